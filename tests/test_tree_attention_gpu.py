"""tree_attention where its general bounds are too wide to see a fault: the
weights of bf16 queries."""
import pytest
import torch

import tree_reference as ref
from decode_megakernel_llama_gb300.build import build
from test_tree_ops_gpu import Case

pytestmark = pytest.mark.gpu
BF, I32 = torch.bfloat16, torch.int32


@pytest.fixture(scope="module")
def dev(cuda_dev):
    build()
    return cuda_dev


def rounded_once(q, k, v, lengths, masks, counts, scale):
    """(out, bound) in float64 for bf16 queries whose result is rounded to bf16 once, and its weights to no fewer than
    16 bits. With p the normalised weights and A = sum p |v|, the result before its rounding is at most A rel off:
      2 d      the scores' error: fp32 sums of hd exact products, a step each (2 u: a tensor core's sum may cut), and the
               scale and the difference from the maximum, 4 u max|s|
      2^-16    the weights: a bf16 term and the rest as another (half a step, 2^-8, of half a step)
      2^-20    exp2
      (2 n/16 + 80) 2^-23   the running sums of both terms over the n rows, 16 at a time, and their joins
    and the rounding is half a step, 2^-8. One term (2^-8 of every weight) exceeds it for one element in ten."""
    B, T, Hq, hd = q.shape
    G = Hq // k.shape[1]
    out = torch.full((B, T, Hq, hd), float("nan"), dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(out)
    for b in range(B):
        n, c = int(lengths[b]), T if counts is None else int(counts[b])
        bits = (masks[b, :c, None] >> torch.arange(c, device=q.device)) & 1
        seen = torch.cat([torch.ones(c, n, dtype=torch.bool, device=q.device), bits.bool()], 1)
        for h in range(Hq):
            kk, vv, qq = (x.double() for x in (k[b, h // G, :n + c], v[b, h // G, :n + c], q[b, :c, h]))
            s = (scale * qq @ kk.T).masked_fill(~seen, float("-inf"))
            p = torch.softmax(s, -1)
            d = scale * (qq.abs() @ kk.abs().T) * 2 * hd * ref.U
            d = d.masked_fill(~seen, 0.0).amax(-1) + 4 * ref.U * s.masked_fill(~seen, 0.0).abs().amax(-1)
            rel = 2 * d + 2.0 ** -16 + 2.0 ** -20 + (2 * (n + c) / 16 + 80) * 2.0 ** -23
            a = (p @ vv.abs()) * rel[:, None]
            out[b, :c, h] = p @ vv
            tol[b, :c, h] = a + ref.BF * (out[b, :c, h].abs() + a)
    return out, tol


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("T,Hq,Hkv,lengths,counts", [
    (1, 4, 4, [9, 200, 0], None), (3, 8, 2, [63, 1], None), (5, 10, 2, [130], None),      # 16 and 32 columns
    (33, 16, 2, [90, 7], [33, 20]), (61, 8, 2, [300, 129], [61, 44]),                     # 128 rows
    (40, 16, 4, [700, 350, 64, 0, 500, 40, 90, 260], None),
])
def test_bf16_results_are_rounded_once(dev, hd, T, Hq, Hkv, lengths, counts):
    c = Case(dev, lengths, T, Hq, Hkv, hd, BF, counts=counts)
    c.run()
    torch.cuda.synchronize()
    want, tol = rounded_once(c.q, c.k, c.v, c.lengths, c.masks, c.counts, c.scale)
    on = ~want.isnan()
    err = (c.out.double() - want).abs()[on]
    assert (err <= tol[on]).all(), (int((err > tol[on]).sum()), err.numel(), float((err / tol[on]).max()))
