"""tree_attention where its general bounds and ordinary calls see no fault: the
weights of bf16 queries, waits that run out."""
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


WAITS = [  # heads, type, nodes and query rows, lengths, max_len: 16 and 32 columns and 128 rows; one CTA, a cluster, many CTAs
    (64, torch.float32, 4, 4, 1, [9000], 1), (64, BF, 8, 4, 1, [9000, 4000], 9000), (64, torch.float32, 8, 32, 8, [9000], 9000),
    (128, torch.float32, 8, 4, 1, [9000], 1), (128, BF, 4, 4, 1, [9000], 9000), (128, BF, 8, 8, 2, [30000], 30000),
    (64, torch.float32, 61, 32, 8, [3000, 5000, 900, 2000] * 2, 5000), (64, BF, 61, 32, 8, [3000, 5000, 900, 2000] * 2, 5000),
    (128, BF, 61, 32, 8, [3000, 5000, 900, 2000] * 2, 5000), (64, BF, 61, 8, 1, [60000], 60000), (128, BF, 61, 8, 1, [60000], 60000),
]


@pytest.mark.parametrize("hd,dtype,T,Hq,Hkv,lengths,max_len", WAITS)
def test_a_wait_that_runs_out(dev, hd, dtype, T, Hq, Hkv, lengths, max_len):
    """A limit of a nanosecond, which copies from memory exceed: the status word says so, a row is NaN or right, and the
    next call, which waits as long as it has to, is right."""
    c = Case(dev, lengths, T, Hq, Hkv, hd, dtype)
    c.run(max_len=max_len)
    want, st = c.out.clone(), torch.zeros(1, dtype=I32, device=dev)
    flush = torch.empty(1 << 28, dtype=torch.uint8, device=dev)
    lost = 0
    for rep in range(20):
        c.out.fill_(99.0)
        st.zero_()
        flush.zero_()  # the cache's rows come from memory
        c.run(max_len=max_len, wait_ns=1, status=st)
        nan = c.out.isnan()
        assert int(st) == int(nan.any())
        assert torch.equal(nan.all(-1), nan.any(-1))
        assert torch.equal(c.out[~nan], want[~nan])
        lost += int(nan.sum())
    assert lost > 0
    st.zero_()
    c.out.fill_(99.0)
    c.run(max_len=max_len, status=st)
    assert int(st) == 0 and torch.equal(c.out, want)


def test_a_wait_that_runs_out_in_a_model(cuda_dev):
    """mk_set_wait_timeout reaches the attention of mk_verify; its status is reported once and the handle works again."""
    from decode_megakernel_llama_gb300 import _lib, synth
    from decode_megakernel_llama_gb300.configs import TINY
    build()
    dev = torch.device("cuda:0")
    k, v = synth.kv_cache(TINY, 600, 1, dev)
    synth.prefill_cache(k, v, 500)
    mk = _lib.Megakernel(TINY, synth.make_weights(TINY, dev, 0), k, v)
    tk = torch.tensor([3, 5, 7], dtype=I32, device=dev)
    pr = torch.tensor([-1, 0, 0], dtype=I32, device=dev)
    out, lg = torch.zeros(3, dtype=I32, device=dev), torch.zeros(3, TINY.vocab, device=dev)
    mk.verify(tk, pr, 500, out, lg)
    assert mk.status() == 0
    want = out.tolist(), lg.clone()
    mk.set_wait_timeout(1)
    mk.verify(tk, pr, 500, out, lg)
    assert mk.status() == _lib.MK_ERR_TIMEOUT
    assert lg.isnan().all()
    mk.set_wait_timeout(2_000_000_000)
    mk.verify(tk, pr, 500, out, lg)
    assert mk.status() == 0
    assert out.tolist() == want[0] and torch.equal(lg, want[1])
    mk.close()
