"""The operators of a cache in pages as a program uses them: together, in streams and graphs, with waits that run out, far
out in a large pool, over drawn sizes, and around the model's own cache."""
import ctypes
import random

import pytest
import torch

from decode_megakernel_llama_gb300 import _lib, synth
from decode_megakernel_llama_gb300.build import build
from decode_megakernel_llama_gb300.configs import TINY
from tests import paged_reference as ref
from tests.test_paged_gpu import Paged

pytestmark = pytest.mark.gpu
I32, BF = torch.int32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()


@pytest.mark.parametrize("hd,type,cache,lens,news,Hq,Hkv", [
    (64, "bf16", "bf16", [3000, 900], [1, 1], 8, 2), (128, "f32", "bf16", [2000], [4], 4, 1),
    (64, "bf16", "e4m3", [3000, 900], [1, 1], 8, 2), (128, "bf16", "e4m3", [4000], [3], 6, 2),
    (64, "bf16", "bf16", [2000, 700], [300, 64], 8, 2), (64, "f32", "e4m3", [1500], [200], 8, 2),
    (128, "bf16", "bf16", [900], [900], 8, 1), (64, "bf16", "bf16", [1000] * 80, [1] * 80, 8, 2),
    (64, "bf16", "bf16", [40000], [1], 8, 1),
])
def test_a_wait_that_runs_out(hd, type, cache, lens, news, Hq, Hkv):
    """A limit of a nanosecond, which copies from memory exceed: the status word says so, a row is NaN or right, and the
    next call, which waits as long as it has to, is right."""
    p = Paged(lens, news, Hq, Hkv, hd, 16, type, cache, seed=1)
    kw = dict(max_new=max(news), max_len=max(lens))
    p.run(**kw)
    p.check()
    want = p.out.clone()
    flush = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    lost = 0
    for _ in range(12):
        p.out.fill_(99.0)
        p.status.zero_()
        flush.zero_()  # the rows come from memory
        p.run(wait_ns=1, **kw)
        nan = p.out.isnan()
        assert int(p.status) == int(nan.any()) or int(p.status) == 1
        assert torch.equal(nan.all(-1), nan.any(-1))
        assert torch.equal(p.out[~nan], want[~nan])
        lost += int(nan.sum())
    assert lost > 0
    p.status.zero_()
    p.run(**kw)
    p.check()
    assert torch.equal(p.out, want)


def test_two_streams_at_once():
    """Calls that split through workspaces, in two streams side by side, many times."""
    a = Paged([30000, 9000], [1, 1], 8, 2, 64, 16, "bf16", "bf16", seed=2)
    b = Paged([12000], [5], 4, 1, 128, 64, "f32", "e4m3", seed=3)
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    for s in (sa, sb):
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(30):
        for p, s in ((a, sa), (b, sb)):
            with torch.cuda.stream(s):
                p.run(max_new=5, max_len=30000 if p is a else 12000)
    torch.cuda.synchronize()
    a.check()
    b.check()


def test_two_graphs_with_workspaces_of_their_own():
    a = Paged([30000, 9000], [1, 1], 8, 2, 64, 16, "bf16", "bf16", seed=4)
    b = Paged([28000, 11000], [1, 1], 8, 2, 64, 16, "bf16", "e4m3", seed=5)
    graphs = []
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        a.run(max_new=1)
        b.run(max_new=1)
    torch.cuda.current_stream().wait_stream(s)
    for p in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            p.run(max_new=1)
        graphs.append(g)
        p.out.fill_(7.0)
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(10):
        for g, st in zip(graphs, (sa, sb)):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    a.check()
    b.check()


def test_a_workspace_too_small_or_none():
    """The call does without and is right; nothing outside what it is given is written."""
    p = Paged([30000], [2], 8, 2, 64, 16, seed=6)
    row = p.Hq * p.hd
    rec = dict(n_tokens=2, batch=1, max_pages=p.table.shape[1], n_heads=8, n_kv_heads=2, head_dim=64, dtype=1, cache_dtype=1,
               n_pages=p.k.shape[0], page_size=16, max_new=2, max_len=30000, window=0, sinks=0, scale=0.125, q_stride=row,
               out_stride=row, q=p.q.data_ptr(), out=p.out.data_ptr(), k_pages=p.k.data_ptr(), v_pages=p.v.data_ptr(),
               table=p.table.data_ptr(), starts=p.starts.data_ptr(), lengths=p.lengths.data_ptr(), status=p.status.data_ptr())
    lib, stream = _lib.load(), torch.cuda.current_stream().cuda_stream
    need = lib.mk_paged_attention_workspace(ctypes.byref(_lib.mk_paged_args(**rec)))
    assert need > 0
    for size in (0, 64, need - 16, need):
        work = torch.full((need + 64,), 0xAB, dtype=torch.uint8, device="cuda")
        p.out.fill_(7.0)
        args = _lib.mk_paged_args(**rec, workspace=work.data_ptr() if size else None, workspace_bytes=size)
        assert lib.mk_paged_attention(ctypes.byref(args), stream) == 0
        p.check()
        assert bool((work[size:] == 0xAB).all())
        assert size == need or bool((work == 0xAB).all())


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_pages_behind_4_gib(cache):
    """A pool whose last pages lie more than 2^32 bytes in: written, attended over and read back there."""
    Hkv, hd, ps = 8, 128, 128
    pages = (1 << 33) // (Hkv * hd * ps * (2 if cache == "bf16" else 1)) + 8
    dev = torch.device("cuda")
    view = BF if cache == "bf16" else ref.E4M3
    kp, vp = (torch.empty(pages, Hkv, ps, hd, dtype=BF if cache == "bf16" else torch.uint8, device=dev).view(view) for _ in range(2))
    ks, vs = (None, None) if cache == "bf16" else (torch.empty(pages, Hkv, ps, hd // 32, dtype=torch.uint8, device=dev)
                                                   for _ in range(2))
    g = torch.Generator().manual_seed(7)
    k, v = (torch.randn(1, 1, Hkv, 300, hd, generator=g).to(BF).to(dev) for _ in range(2))
    table = torch.tensor([[pages - 1, pages - 3, pages - 2]], dtype=I32, device=dev)
    n = torch.tensor([300], dtype=I32, device=dev)
    sc = dict(k_scales=None if ks is None else ks[None], v_scales=None if vs is None else vs[None])
    _lib.kv_write_pages(k, v, kp[None], vp[None], table, n, **sc)
    k2, v2 = torch.zeros_like(k), torch.zeros_like(v)
    _lib.kv_read_pages(kp[None], vp[None], k2, v2, table, n, **sc)
    if cache == "bf16":
        assert torch.equal(k, k2) and torch.equal(v, v2)
    else:
        assert torch.equal(k2.double(), ref.values(*ref.quantise(k.double())))
    for new in (1, 120):
        q = torch.randn(new, 16, hd, generator=g).to(BF).to(dev)
        out = torch.zeros_like(q)
        starts = torch.tensor([0, new], dtype=I32, device=dev)
        _lib.paged_attention(q, kp, vp, table, starts, n, out, k_scales=ks, v_scales=vs)
        small = torch.arange(3, dtype=I32)[None]
        pool = [torch.cat([x[0, 0], x.new_zeros(Hkv, 84, hd)], 1).double().view(Hkv, 3, ps, hd).transpose(0, 1) for x in (k2, v2)]
        want, tol = ref.attention(q, *pool, small, [0, new], [300], hd ** -0.5, 0, 0)
        assert bool(((out.double() - want).abs() <= tol).all())


def test_drawn_sizes():
    """Sizes, masks and layouts over their whole ranges."""
    rng = random.Random(20)
    for _ in range(60):
        B, Hkv, G = rng.randint(1, 6), rng.choice([1, 2, 3]), rng.choice([1, 2, 3, 4, 5, 8, 16])
        news = [rng.choice([0, 1, 1, 2, rng.randint(1, 40), rng.randint(1, 300)]) for _ in range(B)]
        lens = [n + rng.choice([0, 1, rng.randint(0, 200), rng.randint(0, 3000)]) for n in news]
        if sum(news) == 0:
            continue
        p = Paged(lens, news, Hkv * G, Hkv, rng.choice([64, 128]), rng.choice([8, 16, 32, 64, 128, 256]),
                  rng.choice(["f32", "bf16"]), rng.choice(["bf16", "e4m3"]), rng.choice([0, 0, 1, rng.randint(1, 2000)]),
                  rng.choice([0, 1, 4, rng.randint(1, 300)]), rng.choice([0, 5]), seed=rng.randint(0, 10 ** 6))
        p.run(**rng.choice([dict(), dict(max_new=max(news), max_len=max(lens)), dict(max_new=1, max_len=1)]))
        p.check()


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_a_prompt_in_chunks_then_tokens(cache):
    """Append and attend together: a prompt in three chunks, then single tokens, two sequences with other lengths, their
    pages in any order; each step's queries against all rows written so far."""
    Hq, Hkv, hd, ps, dev = 8, 2, 64, 16, torch.device("cuda")
    g = torch.Generator().manual_seed(8)
    order = torch.randperm(2 * 24, generator=g).view(2, 24)
    table = order.to(I32).to(dev)
    pool = torch.zeros(48, Hkv, ps, hd, dtype=BF if cache == "bf16" else torch.uint8, device=dev)
    kp, vp = (pool.clone().view(BF if cache == "bf16" else ref.E4M3) for _ in range(2))
    ks, vs = (None, None) if cache == "bf16" else (torch.full((48, Hkv, ps, hd // 32), 127, dtype=torch.uint8, device=dev)
                                                   for _ in range(2))
    freq = _lib.rope_frequencies(hd, 5e5)[0].to(dev)
    done = [0, 0]
    for news in ([130, 40], [65, 1], [33, 90], [1, 1], [1, 1], [1, 0], [2, 3]):
        n = sum(news)
        pos = [done[b] + i for b in (0, 1) for i in range(news[b])]
        seq = [b for b in (0, 1) for _ in range(news[b])]
        done = [done[b] + news[b] for b in (0, 1)]
        qkv = torch.randn(n, (Hq + 2 * Hkv) * hd, generator=g).to(BF).to(dev)
        q = torch.empty(n, Hq, hd, dtype=BF, device=dev)
        place = dict(slots=torch.tensor([int(order[b, p // ps]) for b, p in zip(seq, pos)], dtype=I32, device=dev))
        args = (torch.tensor(pos, dtype=I32, device=dev), torch.tensor([p % ps for p in pos], dtype=I32, device=dev), freq)
        if cache == "bf16":
            _lib.rope_append(qkv, q, kp, vp, *args, **place)
        else:
            _lib.rope_append_e4m3(qkv, q, kp, vp, ks, vs, *args, **place)
        out = torch.empty_like(q)
        starts = torch.tensor([0, news[0], n], dtype=I32, device=dev)
        lengths = torch.tensor(done, dtype=I32, device=dev)
        _lib.paged_attention(q, kp, vp, table, starts, lengths, out, k_scales=ks, v_scales=vs, max_new=max(news))
        k64, v64 = (kp.double(), vp.double()) if cache == "bf16" else (ref.values(kp, ks), ref.values(vp, vs))
        want, tol = ref.attention(q, k64, v64, order, starts.tolist(), done, hd ** -0.5, 0, 0)
        assert bool(((out.double() - want).abs() <= tol).all())


def test_a_models_cache_saved_and_restored():
    """mk_prefill fills the model's cache, its rows go to pages, the cache is cleared and restored: decoding goes on with
    the same bits; and the pages serve paged_attention as the model's cache would."""
    dev = torch.device("cuda:0")
    k, v = synth.kv_cache(TINY, 64, 1, dev)
    mk = _lib.Megakernel(TINY, synth.make_weights(TINY, dev, 0), k, v)
    prompt = synth.prompt_tokens(TINY.vocab, 30).to(device=dev, dtype=I32)
    tok = torch.zeros(1, dtype=I32, device=dev)
    lg = [torch.zeros(TINY.vocab, device=dev) for _ in range(2)]
    mk.prefill(prompt, 0, tok)
    first = tok.clone()
    kp, vp = (torch.zeros(TINY.n_layers, 9, TINY.n_kv_heads, 8, TINY.head_dim, dtype=BF, device=dev) for _ in range(2))
    table = torch.tensor([[7, 0, 3, 5]], dtype=I32, device=dev)
    n = torch.tensor([30], dtype=I32, device=dev)
    _lib.kv_write_pages(k, v, kp, vp, table, n)
    saved = k.clone(), v.clone()
    mk.step_dev(first, 30, tok, lg[0])
    k.zero_()
    v.zero_()
    _lib.kv_read_pages(kp, vp, k, v, table, n)
    assert torch.equal(k[:, :, :, :30], saved[0][:, :, :, :30]) and torch.equal(v[:, :, :, :30], saved[1][:, :, :, :30])
    mk.step_dev(first, 30, tok, lg[1])
    torch.cuda.synchronize()
    assert mk.status() == 0 and torch.equal(lg[0], lg[1])
    q = torch.randn(5, TINY.n_heads, TINY.head_dim, device=dev)
    a, b = torch.zeros_like(q), torch.zeros_like(q)
    starts = torch.tensor([0, 5], dtype=I32, device=dev)
    _lib.paged_attention(q, kp[1], vp[1], table, starts, n, a)
    _lib.paged_attention(q, k[1], v[1], torch.zeros(1, 1, dtype=I32, device=dev), starts, n, b)
    assert torch.equal(a, b)
    mk.close()


@pytest.mark.parametrize("hd,Hkv,new,cache", [(64, 8, 100, "bf16"), (64, 8, 100, "e4m3"), (64, 8, 8, "bf16"), (128, 8, 8, "bf16"),
                                              (128, 8, 1, "e4m3")])
def test_sums_over_a_long_cache_are_not_cut(hd, Hkv, new, cache):
    """fp32 queries, values all positive: a sum that cuts instead of rounding falls behind with every product. At most 48
    products of 16 rows (heads of 128: 8 * 32 tiles, and the sums of the weights, which are not cut, 62) add to a sum that
    may cut, 2^-23 of it each; what adds those up, rounds: 2^-24 for each of 235 pairs of tiles and some joins. Beside them
    the scores' error twice and the weights', as in paged_reference.attention."""
    L, G = 60000, 4
    p = Paged([L], [new], Hkv * G, Hkv, hd, 128, "f32", "bf16", seed=9, poison=False, q_scale=0.5)
    p.v = p.v.abs()
    if cache == "e4m3":
        (p.k, p.ks), (p.v, p.vs) = (ref.quantise(x.double()) for x in (p.k, p.v))
        p.k64, p.v64 = ref.values(p.k, p.ks), ref.values(p.v, p.vs)
    else:
        p.k64, p.v64 = p.k.double(), p.v.double()
    p.run(max_new=new)
    torch.cuda.synchronize()
    want, tol = ref.attention(p.q, p.k64, p.v64, p.table.cpu(), p.starts.cpu(), p.lengths.cpu(), hd ** -0.5, 0, 0)
    n = torch.arange(L - new + 1, L + 1, device="cuda")[:, None, None]
    loose = (3 * n / 16 + 80) * 2.0 ** -23  # (that bound's share of the sums, of sum p|v| = the result here)
    cut = 48 if hd == 64 else 8 * 32
    tight = tol - want * loose + want * ((cut + 62) * 2.0 ** -23 + 300 * 2.0 ** -24)
    assert bool(((p.out.double() - want).abs() <= tight).all())


@pytest.mark.parametrize("type", ["f32", "bf16"])
@pytest.mark.parametrize("hd,new", [(64, 300), (128, 300), (64, 3), (128, 8)])
def test_scores_that_keep_rising(type, hd, new):
    """Keys that grow along the sequence: maxima are raised in tile after tile."""
    p = Paged([5000], [new], 4, 1, hd, 64, type, "bf16", seed=10, poison=False)
    order = p.table[0].long()
    ramp = torch.linspace(0.1, 8.0, order.numel() * 64, device="cuda").view(-1, 1, 64, 1)
    p.k[order] = (p.k[order].abs().float() * ramp).to(BF)
    p.q.copy_(p.q.abs())
    p.k64 = p.k.double()
    p.run(max_new=new)
    p.check()
