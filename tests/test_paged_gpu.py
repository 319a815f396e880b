"""Operators of a cache in pages against plain 64-bit forms: attention of ragged new tokens, rows quantised as they are
written, and rows moved between pages and a contiguous cache. Bounds: paged_reference.py and tree_reference.py."""
import math

import pytest
import torch

from decode_megakernel_llama_gb300 import _lib
from decode_megakernel_llama_gb300.build import build
from tests import paged_reference as ref
from tests import tree_reference as tree

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()


class Paged:
    """Seeded inputs of a paged attention call; rows that no token sees hold NaN (`poison`)."""

    def __init__(self, lens, news, Hq=8, Hkv=2, hd=64, ps=16, type="bf16", cache="bf16", window=0, sinks=0, pad=0, seed=0,
                 poison=True, extra_pages=2, q_scale=1.5):
        g = torch.Generator().manual_seed(seed)
        dev = torch.device("cuda")
        self.window, self.sinks, self.Hq, self.hd = window, sinks, Hq, hd
        M = max(1, max(-(-x // ps) for x in lens))
        pages = sum(-(-x // ps) for x in lens) + extra_pages
        order = torch.randperm(pages, generator=g)
        self.table = torch.full((len(lens), M), -1, dtype=torch.int32)
        seen = torch.zeros(pages, ps, dtype=torch.bool)
        at = 0
        for b, (n, x) in enumerate(zip(news, lens)):
            need = -(-x // ps)
            self.table[b, :need] = order[at:at + need].int()
            at += need
            for j in range(x):
                low = max(0, x - n) - window  # the first token's position less the window
                if n and (not window or j > low or j < sinks):
                    seen[self.table[b, j // ps], j % ps] = True
        total = sum(news) + pad
        self.q = (q_scale * torch.randn(total, Hq, hd, generator=g)).to(DT[type]).to(dev)
        k, v = (torch.randn(pages, Hkv, ps, hd, generator=g).bfloat16() for _ in range(2))
        hide = ~seen[:, None, :, None].expand_as(k) if poison else torch.zeros_like(k, dtype=torch.bool)
        if cache == "bf16":
            self.k, self.v = (torch.where(hide, math.nan, x).bfloat16().to(dev) for x in (k, v))
            self.ks = self.vs = None
            self.k64, self.v64 = self.k.double(), self.v.double()
        else:
            (self.k, self.ks), (self.v, self.vs) = (
                tuple(x.to(dev) for x in ref.quantise(torch.where(hide, math.nan, x.double()))) for x in (k, v))
            self.k64, self.v64 = ref.values(self.k, self.ks), ref.values(self.v, self.vs)
        self.starts = torch.tensor([sum(news[:b]) for b in range(len(news) + 1)], dtype=torch.int32).to(dev)
        self.lengths = torch.tensor(lens, dtype=torch.int32).to(dev)
        self.table = self.table.to(dev)
        self.out = torch.full_like(self.q, 7.0)
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)

    def run(self, **kw):
        _lib.paged_attention(self.q, self.k, self.v, self.table, self.starts, self.lengths, self.out, window=self.window,
                             sinks=self.sinks, k_scales=self.ks, v_scales=self.vs, status=self.status, **kw)

    def check(self, scale=None):
        torch.cuda.synchronize()
        assert int(self.status) == 0
        scale = self.hd ** -0.5 if scale is None else scale
        want, tol = ref.attention(self.q, self.k64, self.v64, self.table.cpu(), self.starts.cpu(), self.lengths.cpu(),
                                  scale, self.window, self.sinks)
        outside = torch.isnan(tol).all(-1).all(-1) & torch.isnan(want).all(-1).all(-1)
        count = int(self.starts[-1])
        assert bool((self.out[count:] == 7.0).all()), "rows behind the last sequence were written"
        got, want, tol = self.out[:count].double(), want[:count], tol[:count]
        odd = ~torch.isfinite(want)
        # (an infinite value that a token sees times a weight's lower terms, zeros or of the other sign, is no number:
        # the result is not finite where the formula's is not)
        assert torch.equal(torch.isfinite(got), ~odd)
        bad = ((got - want).abs() > tol) & ~odd
        assert not bool(bad.any()), f"{int(bad.sum())} of {bad.numel()} off, worst {float(((got - want).abs() / tol)[~odd].max())} bounds, {outside.sum()}"


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("type", ["f32", "bf16"])
@pytest.mark.parametrize("Hq,Hkv,hd,ps,lens,news", [
    (4, 1, 64, 16, [1], [1]),
    (8, 2, 64, 16, [5, 16, 17, 0, 128, 129], [1, 1, 1, 0, 1, 1]),
    (8, 8, 64, 8, [200, 3], [3, 3]),
    (6, 2, 128, 32, [333, 31, 64], [5, 31, 1]),
    (3, 1, 128, 64, [257, 513, 640], [1, 2, 7]),
    (16, 1, 64, 128, [700, 127], [9, 127]),
    (8, 2, 64, 256, [1000, 300], [40, 300]),
    (32, 8, 64, 16, [191], [1]),
    (4, 4, 128, 16, [400], [400]),
    (8, 1, 128, 512, [777, 5], [100, 5]),
])
def test_attention(type, cache, Hq, Hkv, hd, ps, lens, news):
    p = Paged(lens, news, Hq, Hkv, hd, ps, type, cache, pad=3, seed=len(lens) + hd)
    p.run()
    p.check()


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("type", ["f32", "bf16"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (7, 4), (64, 0), (128, 128), (130, 200), (500, 4), (129, 1)])
@pytest.mark.parametrize("Hq,Hkv,hd,ps,lens,news", [
    (8, 2, 64, 16, [900, 130, 3], [1, 1, 1]),
    (8, 2, 128, 32, [700, 400, 60], [13, 8, 60]),
    (4, 4, 64, 64, [1200, 129], [300, 129]),
])
def test_window_and_first_tokens(type, cache, window, sinks, Hq, Hkv, hd, ps, lens, news):
    p = Paged(lens, news, Hq, Hkv, hd, ps, type, cache, window, sinks, pad=1, seed=window + sinks)
    p.run(max_new=max(news), max_len=max(lens))
    p.check()


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("Hq,Hkv,hd,type", [(8, 2, 64, "bf16"), (4, 2, 128, "bf16"), (8, 8, 64, "f32"), (16, 4, 128, "f32")])
def test_long_contexts_are_split(Hq, Hkv, hd, type, cache):
    p = Paged([9001, 4000], [1, 2], Hq, Hkv, hd, 64, type, cache, seed=3)
    p.run(max_new=2, max_len=9001)
    p.check()


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("Hq,Hkv,hd,type", [(8, 2, 64, "bf16"), (8, 1, 128, "bf16"), (4, 1, 64, "f32"), (2, 1, 128, "f32")])
def test_a_prompt_behind_a_prefix(Hq, Hkv, hd, type, cache):
    p = Paged([2500, 600], [1037, 600], Hq, Hkv, hd, 16, type, cache, pad=2, seed=4)
    p.run(max_new=1037, max_len=2500)
    p.check()


def test_bounds_that_are_exceeded_only_choose_the_launch():
    p = Paged([1500, 700], [70, 3], seed=5)
    p.run(max_new=1, max_len=5)
    p.check()


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("type", ["f32", "bf16"])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("new,window", [(5, 0), (5, 40), (150, 0), (150, 60)])
def test_rows_that_some_tokens_see_may_hold_anything(type, cache, hd, new, window):
    """A token that does not see a row is not touched by its NaN or infinities; one that sees it is not finite there."""
    p = Paged([400], [new], 4, 2, hd, 16, type, cache, window, 2, seed=6)
    for j in (400 - new + 1, 400 - new // 2, 399, 400 - new - 20):
        page, row = int(p.table[0, j // 16]), j % 16
        if cache == "bf16":
            p.k[page, 0, row, 3] = math.nan
            p.v[page, 1, row, hd - 1] = math.inf if j % 2 else math.nan
        else:
            p.ks[page, 0, row, 0] = 255
            p.vs[page, 1, row, hd // 32 - 1] = 255
    if cache == "bf16":
        p.k64, p.v64 = p.k.double(), p.v.double()
    else:
        p.k64, p.v64 = ref.values(p.k, p.ks), ref.values(p.v, p.vs)
    p.run()
    p.check()


def test_tokens_before_the_first_row_get_zeros_and_empty_sequences_nothing():
    """Fewer rows than new tokens: the first ones stand before row 0."""
    p = Paged([3, 0, 20], [8, 2, 0], seed=7)
    p.run()
    torch.cuda.synchronize()
    assert bool((p.out[:5] == 0).all()) and bool((p.out[8:10] == 0).all())
    p.check()


def test_pages_outside_the_pool_read_as_zeros_and_shared_pages_are_read_by_all():
    p = Paged([100, 100], [4, 4], poison=False, seed=8)
    p.table[1, :3] = p.table[0, :3]
    p.table[0, 4] = 10 ** 9
    p.table[1, 5] = -7
    p.run()
    p.check()


def test_strided_queries_and_another_stream():
    p = Paged([300, 77], [20, 3], seed=9)
    wide = torch.randn(p.q.shape[0], p.Hq + 3, p.hd, device="cuda").bfloat16()
    wide[:, :p.Hq] = p.q
    into = torch.full_like(wide, 7.0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    _lib.paged_attention(wide[:, :p.Hq], p.k, p.v, p.table, p.starts, p.lengths, into[:, :p.Hq], stream=s)
    s.synchronize()
    assert bool((into[:, p.Hq:] == 7.0).all())
    p.out = into[:, :p.Hq].contiguous()
    p.check()


def test_a_contiguous_cache_is_one_page_a_sequence():
    """Any number of rows a page, a table of one page."""
    p = Paged([201, 30], [50, 30], ps=16, seed=10, poison=False)
    k = torch.randn(3, 2, 203, 64, device="cuda").bfloat16()
    v = torch.randn_like(k)
    table = torch.tensor([[2], [0]], dtype=torch.int32, device="cuda")
    p.k, p.v, p.table, p.k64, p.v64 = k, v, table, k.double(), v.double()
    p.run()
    p.check()


def test_captured_and_replayed_with_other_contents():
    p = Paged([500, 90], [3, 3], seed=11)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        p.run()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        p.run()
    p.q.copy_(torch.randn_like(p.q))
    p.lengths.sub_(7)  # (the rows that were the last are behind the sequences)
    p.out.fill_(7.0)
    g.replay()
    p.check()


# ---------------------------------------------------------------- rows in 8 bits
def _rope_case(n, Hq, Hkv, hd, rot, type, norm, seed, pages=9, ps=16):
    g = torch.Generator().manual_seed(seed)
    dev = torch.device("cuda")
    c = dict(qkv=torch.randn(n, (Hq + 2 * Hkv) * hd, generator=g).to(DT[type]).to(dev))
    place = torch.randperm(pages * ps, generator=g)[:n]
    c["slots"], c["rows"] = (place // ps).int().to(dev), (place % ps).int().to(dev)
    c["pos"] = torch.randint(0, 100000, (n,), generator=g).int().to(dev)
    c["freq"], _ = _lib.rope_frequencies(rot, 5e5)
    c["freq"] = c["freq"].to(dev)
    c["qn"], c["kn"] = ((1 + 0.1 * torch.randn(hd, generator=g)).bfloat16().to(dev) if norm else None for _ in range(2))
    c["k"], c["v"] = (torch.full((pages, Hkv, ps, hd), 0x55, dtype=torch.uint8, device=dev).view(ref.E4M3) for _ in range(2))
    c["ks"], c["vs"] = (torch.full((pages, Hkv, ps, hd // 32), 99, dtype=torch.uint8, device=dev) for _ in range(2))
    c["q"] = torch.full((n, Hq, hd), 7.0, dtype=DT[type], device=dev)
    return c


def _near(rows, tol, codes, scales):
    """8-bit rows against float64 ones that are known to tol: the byte is that of a value within tol, the values are
    within half a step (2^-4 of the value, 2^-10 of the block's power where it is small) and tol."""
    s = scales.long()
    mag = rows.abs().unflatten(-1, (-1, 32))
    t = tol.unflatten(-1, (-1, 32))
    low, high = ref.exponents((mag - t).clamp(min=0).flatten(-2)), ref.exponents((mag + t).flatten(-2))
    assert bool(((s >= low) & (s <= high)).all())
    step = ref.power(s - 127).repeat_interleave(32, -1)
    err = (ref.values(codes, scales) - rows).abs()
    assert bool((err <= tol + torch.maximum((rows.abs() + tol) * 2.0 ** -4, step * 2.0 ** -10)).all())


@pytest.mark.parametrize("type", ["f32", "bf16"])
@pytest.mark.parametrize("n,Hq,Hkv,hd,rot,norm,inter", [
    (1, 32, 8, 64, 64, False, False), (1, 3, 1, 128, 128, True, False), (7, 6, 2, 64, 32, True, False),
    (33, 4, 4, 128, 32, False, True), (40, 5, 1, 64, 22, True, False), (100, 8, 2, 128, 94, False, True),
    (1000, 8, 2, 64, 64, True, False), (1001, 4, 1, 128, 64, True, False), (1300, 2, 1, 64, 64, False, True),
])
def test_append_in_8_bits(type, n, Hq, Hkv, hd, rot, norm, inter):
    pages, ps = (9, 16) if n < 140 else (90, 16)
    c = _rope_case(n, Hq, Hkv, hd, rot, type, norm, n + rot, pages, ps)
    _lib.rope_append_e4m3(c["qkv"], c["q"], c["k"], c["v"], c["ks"], c["vs"], c["pos"], c["rows"], c["freq"],
                          slots=c["slots"], q_norm=c["qn"], k_norm=c["kn"], interleaved=inter)
    (q, qm), (k, km), v = tree.rope(c["qkv"], Hq, Hkv, hd, c["pos"], c["freq"], c["qn"], c["kn"], 1e-5, 1.0, inter)
    err = (c["q"].double() - q).abs()
    own = tree.BF if type == "bf16" else 0.0
    assert bool((err <= tree.ROPE_TOL * qm * (1 + own) + own * q.abs() + 1e-30).all())
    sl, r = c["slots"].long(), c["rows"].long()
    _near(k, tree.ROPE_TOL * km, c["k"].view(torch.uint8)[sl, :, r].view(ref.E4M3), c["ks"][sl, :, r])
    # values are quantised as they come: bit for bit
    codes, scales = ref.quantise(v)
    assert torch.equal(c["v"].view(torch.uint8)[sl, :, r], codes.view(torch.uint8)) and torch.equal(c["vs"][sl, :, r], scales)
    # and nothing else is written
    other = torch.ones(pages, ps, dtype=torch.bool, device="cuda")
    other[sl, r] = False
    for x, was in ((c["k"].view(torch.uint8), 0x55), (c["v"].view(torch.uint8), 0x55), (c["ks"], 99), (c["vs"], 99)):
        assert bool((x.transpose(1, 2)[other] == was).all())


def test_append_in_8_bits_leaves_what_is_outside():
    c = _rope_case(4, 2, 1, 64, 64, "f32", False, 1)
    c["rows"][:] = torch.tensor([-1, 16, 3, 3], dtype=torch.int32)
    c["slots"][:] = torch.tensor([0, 0, -1, 9], dtype=torch.int32)
    _lib.rope_append_e4m3(c["qkv"], c["q"], c["k"], c["v"], c["ks"], c["vs"], c["pos"], c["rows"], c["freq"], slots=c["slots"])
    torch.cuda.synchronize()
    assert bool((c["k"].view(torch.uint8) == 0x55).all()) and bool((c["vs"] == 99).all())
    assert bool((c["q"] != 7.0).any())


def test_append_in_8_bits_keeps_the_whole_angle():
    """Heads of ones and zeros come out as cosines and sines. Of each, sincospif is within one unit in the last place,
    2 u of it, and the correction rounds once, u: 3 u of the value, also where it is next to 0; the angle, 16,000 turns
    at most after three roundings in 64 bits, is within 16000 * 2 pi * 3 * 2^-53 = 3.4e-11."""
    n, hd = 500, 64
    c = _rope_case(n, 1, 1, hd, hd, "f32", False, 5, 40)
    c["qkv"].view(n, 3, hd)[:] = torch.cat([torch.ones(hd // 2), torch.zeros(hd // 2)]).cuda()
    _lib.rope_append_e4m3(c["qkv"], c["q"], c["k"], c["v"], c["ks"], c["vs"], c["pos"], c["rows"], c["freq"], slots=c["slots"])
    angle = c["pos"].double()[:, None] * c["freq"].double()
    want = torch.cat([angle.cos(), angle.sin()], -1)
    assert bool(((c["q"][:, 0].double() - want).abs() <= 3 * tree.U * want.abs() + 1e-10).all())


@pytest.mark.parametrize("type", ["f32", "bf16"])
def test_append_in_8_bits_norms_an_infinite_key(type):
    """An infinite mean leaves zeros, and no number where the infinity was: in its block alone."""
    n, hd = 5, 128
    c = _rope_case(n, 2, 1, hd, 64, type, True, 3)
    c["qkv"].view(n, 4, hd)[2, 2, 100] = math.inf
    _lib.rope_append_e4m3(c["qkv"], c["q"], c["k"], c["v"], c["ks"], c["vs"], c["pos"], c["rows"], c["freq"],
                          slots=c["slots"], q_norm=c["qn"], k_norm=c["kn"])
    at = int(c["slots"][2]), 0, int(c["rows"][2])
    assert c["ks"][at].tolist() == [27, 27, 27, 255]
    assert bool((c["k"].view(torch.uint8)[at][:96] & 127 == 0).all())
    assert bool(torch.isfinite(c["q"]).all()) and not bool((c["vs"][at] == 255).any())


def _hard_rows(g, *shape):
    """bf16 rows with blocks at the format's edges: zeros, powers over the whole range, values that round to ties or sit
    at 448 and 57344, infinities and NaN."""
    x = torch.randn(*shape, generator=g) * torch.exp2(torch.randint(-130, 18, (*shape[:-1], 1), generator=g).float())
    x = x.bfloat16()
    flat = x.view(-1, 32)
    flat[0] = 0
    flat[1] = 448.0
    flat[2, 5] = 450.0
    flat[3, 0] = math.inf
    flat[4, 31] = math.nan
    flat[5] = torch.arange(32) * 0.5 + 17.0
    flat[5, 0] = 448.0
    flat[6, 3] = 57344.0
    flat[7, 3] = 1e30
    flat[8] = 2.0 ** -130
    flat[9] = -0.0
    return x


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("L,B,Hkv,S,hd,ps,lens,first", [
    (1, 1, 1, 10, 64, 8, [10], None), (2, 3, 2, 100, 64, 16, [100, 1, 37], None), (3, 2, 1, 300, 128, 128, [257, 300], [250, 7]),
    (2, 4, 3, 61, 128, 32, [0, 61, 33, 32], [0, 0, 40, 31]),
])
def test_rows_to_pages_and_back(cache, L, B, Hkv, S, hd, ps, lens, first):
    g = torch.Generator().manual_seed(S)
    dev = torch.device("cuda")
    k, v = (_hard_rows(g, L, B, Hkv, S, hd).to(dev) for _ in range(2))
    M = -(-S // ps)
    P = B * M + 1
    table = torch.randperm(P, generator=g)[:B * M].view(B, M).int()
    slots = torch.randperm(B, generator=g).int()
    from_ = first or [0] * B
    cols = (1, 2) if cache == "bf16" else (1, 1)
    pools = [torch.full((L, P, Hkv, ps, hd * cols[1]), 0x41, dtype=torch.uint8, device=dev) for _ in range(2)]
    view = torch.bfloat16 if cache == "bf16" else ref.E4M3
    kp, vp = (x.view(view) for x in pools)
    ks, vs = ((None, None) if cache == "bf16" else
              (torch.full((L, P, Hkv, ps, hd // 32), 3, dtype=torch.uint8, device=dev) for _ in range(2)))
    args = dict(slots=slots.to(dev), first=None if first is None else torch.tensor(first, dtype=torch.int32, device=dev),
                k_scales=ks, v_scales=vs)
    if cache == "bf16":
        pools = [torch.full((L, P, Hkv, ps, hd), 3.0, dtype=torch.bfloat16, device=dev) for _ in range(2)]
        kp, vp = pools
    lengths = torch.tensor(lens, dtype=torch.int32, device=dev)
    was = [None if x is None else x.clone() for x in (kp, vp, ks, vs)]
    _lib.kv_write_pages(k, v, kp, vp, table.to(dev), lengths, **args)
    for src, pool, sc, old, old_sc in ((k, kp, ks, was[0], was[2]), (v, vp, vs, was[1], was[3])):
        want = old.clone().view(torch.uint8) if cache != "bf16" else old.clone()
        want_sc = None if sc is None else old_sc.clone()
        for b in range(B):
            for j in range(from_[b], lens[b]):
                page, row = int(table[b, j // ps]), j % ps
                x = src[:, int(slots[b]), :, j]
                if cache == "bf16":
                    want[:, page, :, row] = x
                else:
                    codes, e = ref.quantise(x.double())
                    want[:, page, :, row], want_sc[:, page, :, row] = codes.view(torch.uint8), e
        if cache == "bf16":
            assert torch.equal(pool.view(torch.int16), want.view(torch.int16))
        else:
            assert torch.equal(sc, want_sc)
            assert torch.equal(pool.view(torch.uint8), want)
    k2, v2 = (torch.full_like(k, 5.0) for _ in range(2))
    _lib.kv_read_pages(kp, vp, k2, v2, table.to(dev), lengths, **args)
    for src, dst in ((k, k2), (v, v2)):
        for b in range(B):
            sl = int(slots[b])
            x = src[:, sl, :, from_[b]:lens[b]]
            if cache != "bf16":
                x = ref.values(*ref.quantise(x.double())).bfloat16()
            assert torch.equal(dst[:, sl, :, from_[b]:lens[b]].nan_to_num(9.0), x.nan_to_num(9.0) if cache != "bf16" else x.nan_to_num(9.0))
            assert bool((dst[:, sl, :, :from_[b]] == 5.0).all()) and bool((dst[:, sl, :, max(lens[b], from_[b]):] == 5.0).all())


def test_every_code_and_power_reads_back():
    """All codes (but NaN's) under all powers that are written, as bf16 values."""
    dev = torch.device("cuda")
    codes = torch.arange(256, dtype=torch.uint8).view(1, 1, 1, 4, 64).repeat(1, 108, 1, 2, 1)
    codes[(codes & 127) == 127] = 0
    scales = torch.arange(27, 135, dtype=torch.uint8).view(1, 108, 1, 1, 1).expand(1, 108, 1, 8, 2).contiguous()
    k, v = (torch.zeros(1, 108, 1, 8, 64, dtype=torch.bfloat16, device=dev) for _ in range(2))
    kp, ks = codes.to(dev).view(ref.E4M3), scales.to(dev)
    table = torch.arange(108, dtype=torch.int32, device=dev)[:, None]
    _lib.kv_read_pages(kp, kp.clone(), k, v, table, torch.full((108,), 8, dtype=torch.int32, device=dev), k_scales=ks,
                       v_scales=ks.clone())
    assert torch.equal(k[0].double(), ref.values(kp, ks)[0]) and torch.equal(k, v)


def test_moves_leave_what_is_outside():
    dev = torch.device("cuda")
    k, v = (torch.randn(1, 2, 1, 20, 64, device=dev).bfloat16() for _ in range(2))
    kp, vp = (torch.full((1, 3, 1, 8, 64), 3.0, device=dev).bfloat16() for _ in range(2))
    table = torch.tensor([[0, 7, 1], [2, 2, 2]], dtype=torch.int32, device=dev)
    _lib.kv_write_pages(k, v, kp, vp, table, torch.tensor([99, 99], dtype=torch.int32, device=dev),
                        slots=torch.tensor([1, 2], dtype=torch.int32, device=dev))
    assert torch.equal(kp[0, 0, 0], k[0, 1, 0, :8]) and torch.equal(kp[0, 1, 0, :4], k[0, 1, 0, 16:])
    assert bool((kp[0, 1, 0, 4:] == 3.0).all()) and bool((kp[0, 2] == 3.0).all())
