"""tree_attention where its general bounds and ordinary calls see no fault: the
weights of bf16 queries, waits that run out, splits through the workspace."""
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


# Caches so long that their rows are split over more CTAs than a cluster holds, the parts joined by a second kernel out
# of a workspace: 16 and 32 columns and 128 rows (the last number), one sequence and several.
SPLIT = [
    (64, torch.float32, 4, 8, 2, [20000], 16), (128, BF, 4, 8, 2, [20000], 16), (64, BF, 1, 16, 1, [70000], 16),
    (64, BF, 8, 8, 2, [24000], 32), (128, torch.float32, 8, 8, 2, [24000], 32), (128, torch.float32, 33, 4, 2, [16000], 32),
    (64, torch.float32, 40, 16, 2, [40000], 128), (64, BF, 61, 8, 1, [60000], 128), (128, BF, 61, 8, 1, [60000], 128),
    (64, torch.float32, 5, 6, 2, [30000, 5, 17000], 16), (64, BF, 40, 16, 2, [9000, 40000], 128),
]


def split_args(c, max_len, **kw):
    """The C call's arguments for a Case, without a workspace."""
    from decode_megakernel_llama_gb300 import _lib
    B, T, Hq, hd = c.q.shape
    ptr = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    return _lib.mk_tree_args(**{**dict(
        batch=B, nodes=T, n_heads=Hq, n_kv_heads=c.k.shape[1], head_dim=hd, dtype=int(c.q.dtype == BF),
        slots=c.k.shape[0], max_seq=c.k.shape[2], max_len=max_len, scale=c.scale, q_batch_stride=T * Hq * hd,
        q_token_stride=Hq * hd, out_batch_stride=T * Hq * hd, out_token_stride=Hq * hd, q=ptr(c.q), out=ptr(c.out),
        k_cache=ptr(c.k), v_cache=ptr(c.v), lengths=ptr(c.lengths), counts=ptr(c.counts), slot_of=ptr(c.slots),
        masks=ptr(c.masks)), **kw})


def work_bytes(c, max_len, rows):
    """The workspace asked for, which has to be whole parts of the kernel of so many rows."""
    import ctypes

    from decode_megakernel_llama_gb300 import _lib
    n = _lib.load().mk_tree_attention_workspace(ctypes.byref(split_args(c, max_len)))
    B, T, Hq, hd = c.q.shape
    tiles = -(-T * (Hq // c.k.shape[1]) // rows)
    part = 4 * rows * (hd + 2) * B * c.k.shape[1] * tiles
    assert n > part and n % part == 0, (n, part)
    return n


@pytest.mark.parametrize("hd,dtype,T,Hq,Hkv,lengths,rows", SPLIT)
def test_splits_through_the_workspace(dev, hd, dtype, T, Hq, Hkv, lengths, rows):
    """Against the plain form; equal bits again, in two streams at once and in two graphs replayed side by side."""
    longest = max(lengths)
    cases = [Case(dev, lengths, T, Hq, Hkv, hd, dtype, seed=s) for s in (1, 2)]
    for c in cases:
        work_bytes(c, longest, rows)
        c.run(max_len=longest)
        c.check()
    want = [c.out.clone() for c in cases]
    streams, graphs = [torch.cuda.Stream() for _ in cases], []
    for c in cases:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            c.run(max_len=longest)
    for rep in range(6):
        for c in cases:
            c.out.fill_(99.0)
        torch.cuda.synchronize()
        for c, s, gr in zip(cases, streams, graphs):
            if rep % 2:
                with torch.cuda.stream(s):
                    gr.replay()
            else:
                c.run(max_len=longest, stream=s)
        torch.cuda.synchronize()
        for c, w in zip(cases, want):
            assert torch.equal(c.out, w)


@pytest.mark.parametrize("hd,dtype,T,Hq,Hkv,lengths,rows", SPLIT)
def test_a_workspace_of_the_size_asked_for_too_small_or_none(dev, hd, dtype, T, Hq, Hkv, lengths, rows):
    """With less than it asks for a call does without; it never writes outside what it was given."""
    import ctypes

    from decode_megakernel_llama_gb300 import _lib
    longest = max(lengths)
    c = Case(dev, lengths, T, Hq, Hkv, hd, dtype)
    n = work_bytes(c, longest, rows)
    stream = torch.cuda.current_stream().cuda_stream
    for given in (n, n - 4, n // 2, 16, 0, None):
        room = torch.full((n + 4096,), 77, dtype=torch.uint8, device=dev)
        kw = {} if given is None else dict(workspace=room.data_ptr(), workspace_bytes=given)
        c.out.fill_(99.0)
        _lib.check(_lib.load().mk_tree_attention(ctypes.byref(split_args(c, longest, **kw)), stream))
        c.check()
        assert (room[(n if given == n else 0):] == 77).all(), given
        assert given != n or not (room[:n] == 77).all()


@pytest.mark.parametrize("hd,dtype,T,Hq,Hkv,rows", [(64, torch.float32, 5, 6, 2, 16), (128, BF, 8, 8, 2, 32),
                                                    (64, BF, 40, 16, 2, 128)])
def test_split_sequences_of_no_node_no_slot_and_junk(dev, hd, dtype, T, Hq, Hkv, rows):
    c = Case(dev, [30000, 6, 20000, 50], T, Hq, Hkv, hd, dtype, counts=[T, 0, 2, T], slots=[2, 0, 3, 4], n_slots=5,
             S=30100)
    work_bytes(c, 30000, rows)
    c.k[:, :, 30000 + T:] = float("nan")
    c.v[:, :, 30000 + T:] = float("inf")
    c.k[3, :, 20002:], c.v[3, :, 20002:] = float("inf"), float("nan")
    c.masks[0, 1] = -(1 << 63)  # a bit behind the tree
    c.run(max_len=30000)
    c.check()
    c.slots[3] = 5  # outside the cache: its rows are left alone
    keep = c.out.clone()
    c.out.fill_(99.0)
    c.run(max_len=30000)
    torch.cuda.synchronize()
    assert (c.out[3] == 99.0).all() and torch.equal(c.out[:3], keep[:3])
    # a drafted row that is not finite reaches those that see it, and no other
    c.masks[0, :3] = torch.tensor([1, 2, 4], device=dev)
    c.masks[0, 3:] &= ~2
    c.run(max_len=30000)
    keep = c.out.clone()
    c.v[2, :, 30001, 3] = float("inf")
    c.run(max_len=30000)
    torch.cuda.synchronize()
    assert (c.out[0, 1, :, 3] == float("inf")).all()
    c.out[0, 1] = keep[0, 1]
    assert torch.equal(c.out, keep)


@pytest.mark.parametrize("B,T,Hq,Hkv,hd,dtype", [(3, 64, 8, 1, 128, torch.float32), (1, 64, 16, 1, 64, BF), (2, 33, 8, 2, 64, BF),
                                                 (1, 1, 8, 8, 128, torch.float32)])
def test_the_binding_and_the_c_call_split_alike(dev, B, T, Hq, Hkv, hd, dtype):
    """The workspace is asked for whatever the length: equal bits on either way, and with a stream given."""
    import ctypes

    from decode_megakernel_llama_gb300 import _lib
    for n in (3400, 4030, 4095, 9000):
        c = Case(dev, [n] * B, T, Hq, Hkv, hd, dtype)
        size = _lib.load().mk_tree_attention_workspace(ctypes.byref(split_args(c, n)))
        assert size > 0 if B == 3 else size >= 0  # (for the first shape all of these lengths pay)
        work = torch.empty(size, dtype=torch.uint8, device=dev)
        a = split_args(c, n, workspace=work.data_ptr() if size else None, workspace_bytes=size)
        _lib.check(_lib.load().mk_tree_attention(ctypes.byref(a), torch.cuda.current_stream().cuda_stream))
        want = c.out.clone()
        for kw in ({}, dict(stream=torch.cuda.Stream())):
            torch.cuda.synchronize()
            c.out.fill_(99.0)
            torch.cuda.synchronize()
            c.run(max_len=n, **kw)
            torch.cuda.synchronize()
            assert torch.equal(c.out, want), n
        if n == 4030:
            c.check()
