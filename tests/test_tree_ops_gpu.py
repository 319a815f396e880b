"""The drafted-tree operators against their plain 64-bit forms
(tests/tree_reference.py holds the forms and derives the error bounds)."""
import pytest
import torch

import tree_reference as ref
from decode_megakernel_llama_gb300 import _lib
from decode_megakernel_llama_gb300.build import build

pytestmark = pytest.mark.gpu
BF, I32 = torch.bfloat16, torch.int32


@pytest.fixture(scope="module")
def dev(cuda_dev):
    build()
    return cuda_dev


def normal(gen, *shape, dtype=torch.float32, dev="cuda:0"):
    return torch.randn(*shape, generator=gen).to(dtype).to(dev)


# ---------------------------------------------------------------- rope_append
def rope_case(dev, n, Hq, Hkv, hd, rot, dtype, norm, inter, slots=3, S=64, base=0, mscale=1.0, pad=0, in_place=False,
              seed=0):
    g = torch.Generator().manual_seed(seed + n * 7 + Hq + hd + rot)
    width = (Hq + 2 * Hkv) * hd
    buf = normal(g, n, width + pad, dtype=dtype)
    qkv = buf[:, :width]
    before = qkv.clone()
    k, v = normal(g, slots, Hkv, S, hd, dtype=BF), normal(g, slots, Hkv, S, hd, dtype=BF)
    k0, v0 = k.clone(), v.clone()
    spots = torch.randperm(slots * S, generator=g)[:n]
    sl, rows = (spots // S).to(I32).to(dev), (spots % S).to(I32).to(dev)
    pos = (base + torch.randint(0, 500, (n,), generator=g)).to(I32).to(dev)
    freq, _ = _lib.rope_frequencies(rot, 5e5) if rot > 0 else (None, 1)
    freq = freq.to(dev)
    qn = (1 + 0.1 * normal(g, hd)).to(BF) if norm else None
    kn = (1 + 0.1 * normal(g, hd)).to(BF) if norm else None
    q_out = qkv[:, : Hq * hd].view(n, Hq, hd) if in_place else torch.full((n, Hq, hd), 7.0, dtype=dtype, device=dev)
    _lib.rope_append(qkv, q_out, k, v, pos, rows, freq, slots=sl, q_norm=qn, k_norm=kn, eps=1e-5, mscale=mscale,
                     interleaved=inter)
    torch.cuda.synchronize()
    (q_ref, q_mag), (k_ref, k_mag), v_ref = ref.rope(before, Hq, Hkv, hd, pos, freq, qn, kn, 1e-5, mscale, inter)
    half_step = 0.0 if dtype == torch.float32 else ref.BF
    err = (q_out.double() - q_ref).abs()
    tol = ref.ROPE_TOL * q_mag
    assert (err <= tol + half_step * (q_ref.abs() + tol)).all(), (err - tol).max()
    sl, rows = sl.long(), rows.long()
    got = k[sl, :, rows].double()
    tol = ref.ROPE_TOL * k_mag
    assert ((got - k_ref).abs() <= tol + ref.BF * (k_ref.abs() + tol)).all()
    assert torch.equal(v[sl, :, rows], before.view(n, -1, hd)[:, Hq + Hkv:].to(BF))
    k[sl, :, rows], v[sl, :, rows] = k0[sl, :, rows], v0[sl, :, rows]
    assert torch.equal(k, k0) and torch.equal(v, v0)  # every other row as it was
    if pad:
        assert torch.equal(buf[:, :width][:, Hq * hd:], before[:, Hq * hd:])


@pytest.mark.parametrize("dtype", [torch.float32, BF])
@pytest.mark.parametrize("n,Hq,Hkv,hd,rot", [(1, 4, 2, 64, 64), (1, 32, 8, 64, 64), (5, 1, 1, 128, 128), (3, 9, 3, 64, 32),
                                             (64, 24, 8, 128, 32), (7, 4, 4, 64, 2), (2, 4, 1, 128, 126),
                                             (33, 5, 5, 64, 38), (150, 2, 1, 128, 64)])
@pytest.mark.parametrize("norm,inter", [(False, False), (True, False), (False, True), (True, True)])
def test_rope_append_matches_the_formula(dev, dtype, n, Hq, Hkv, hd, rot, norm, inter):
    rope_case(dev, n, Hq, Hkv, hd, rot, dtype, norm, inter)


def test_rope_append_far_positions_scale_strides_in_place(dev):
    rope_case(dev, 20, 8, 2, 64, 64, torch.float32, True, False, base=131072 - 500, mscale=1.2079)
    rope_case(dev, 20, 8, 2, 128, 128, torch.float32, False, True, base=131072 - 500)
    rope_case(dev, 20, 8, 2, 64, 48, torch.float32, True, False, pad=20)
    rope_case(dev, 20, 8, 2, 64, 64, BF, True, True, pad=12)
    rope_case(dev, 20, 8, 2, 64, 64, torch.float32, True, False, in_place=True)
    rope_case(dev, 20, 8, 2, 128, 20, BF, False, True, in_place=True, pad=4)


def test_rope_append_large_prompt(dev):
    rope_case(dev, 3000, 8, 2, 64, 64, torch.float32, True, False, slots=2, S=1600)


@pytest.mark.parametrize("n,Hq,Hkv,hd,rot,dtype,kw", [
    (1024, 4, 4, 64, 64, torch.float32, dict(norm=True)), (1025, 32, 8, 64, 64, torch.float32, dict(norm=True)),
    (1300, 24, 8, 128, 32, BF, dict(norm=True, inter=True)), (2500, 9, 3, 64, 38, torch.float32, dict(pad=4)),
    (1100, 5, 1, 128, 126, BF, dict(pad=8)), (2999, 2, 1, 64, 2, BF, dict(inter=True, in_place=True)),
    (1500, 8, 2, 128, 128, torch.float32, dict(norm=True, in_place=True)),
    (1700, 3, 2, 64, 48, BF, dict(norm=True, pad=4)),              # rows that start at 8 bytes of 16
    (1030, 40, 8, 128, 64, torch.float32, dict(norm=True)),        # rows of 28 KB
    (32, 24, 8, 128, 128, BF, dict(norm=True)), (33, 7, 1, 64, 64, torch.float32, dict(norm=True)),
    (216, 24, 8, 128, 96, BF, dict(norm=True)), (300, 4, 2, 64, 32, torch.float32, dict()),
    (457, 5, 3, 128, 24, BF, dict(inter=True, norm=True)), (912, 3, 1, 64, 40, BF, dict(norm=True, in_place=True)),
    (913, 3, 1, 128, 112, torch.float32, dict(norm=True)), (940, 12, 4, 128, 128, BF, dict(inter=True)),
    (1000, 6, 2, 128, 64, BF, dict(norm=True, pad=4)), (1200, 6, 2, 64, 56, torch.float32, dict(norm=True)),
])
def test_rope_append_long_prompts(dev, n, Hq, Hkv, hd, rot, dtype, kw):
    rope_case(dev, n, Hq, Hkv, hd, rot, dtype, **{"norm": False, "inter": False, **kw}, slots=2, S=n, base=100000)


def test_rope_append_long_prompts_in_streams_and_graphs(dev):
    g = torch.Generator().manual_seed(9)
    n, Hq, Hkv, hd = 1600, 6, 2, 64
    freq = _lib.rope_frequencies(hd, 1e4)[0].to(dev)
    rows = torch.arange(n, dtype=I32, device=dev)
    rows[5], rows[1400] = -1, n
    sides = []
    for _ in range(2):
        x = normal(g, n, (Hq + 2 * Hkv) * hd)
        q, k, v = torch.empty(n, Hq, hd, device=dev), *(torch.zeros(1, Hkv, n, hd, dtype=BF, device=dev) for _ in "kv")
        sides.append((x, q, k, v, torch.cuda.Stream(), torch.cuda.CUDAGraph()))
    torch.cuda.synchronize()
    for x, q, k, v, s, gr in sides:
        _lib.rope_append(x, q, k, v, rows, rows, freq, stream=s)
    torch.cuda.synchronize()
    for x, q, k, v, s, gr in sides:
        with torch.cuda.graph(gr):
            _lib.rope_append(x, q, k, v, rows, rows, freq)
        x.mul_(-2)
    want = [(-2 * q, -2 * k, -2 * v) for x, q, k, v, s, gr in sides]  # (exact: signs and a power of two)
    torch.cuda.synchronize()
    for x, q, k, v, s, gr in sides:
        with torch.cuda.stream(s):
            gr.replay()
    torch.cuda.synchronize()
    for (x, q, k, v, s, gr), w in zip(sides, want):
        (q_ref, mag), _, _ = ref.rope(x, Hq, Hkv, hd, rows, freq, None, None, 0, 1.0, False)
        assert ((q.double() - q_ref).abs() <= ref.ROPE_TOL * mag).all()
        assert torch.equal(q, w[0]) and torch.equal(k, w[1]) and torch.equal(v, w[2])
        assert (k[:, :, 5] == 0).all() and (v[:, :, 1400] == 0).all()


def test_rope_append_rows_outside_the_cache_are_not_written(dev):
    g = torch.Generator().manual_seed(5)
    n, Hq, Hkv, hd, S = 8, 2, 1, 64, 16
    qkv = normal(g, n, (Hq + 2 * Hkv) * hd)
    k, v = normal(g, 2, Hkv, S, hd, dtype=BF), normal(g, 2, Hkv, S, hd, dtype=BF)
    k0, v0 = k.clone(), v.clone()
    q = torch.zeros(n, Hq, hd, device=dev)
    rows = torch.tensor([0, -1, S, 3, 4, 5, 2 ** 31 - 1, -2 ** 31], dtype=I32, device=dev)
    sl = torch.tensor([0, 0, 0, 2, -1, 1, 0, 1], dtype=I32, device=dev)
    pos = torch.arange(n, dtype=I32, device=dev)
    freq = _lib.rope_frequencies(hd, 1e4)[0].to(dev)
    _lib.rope_append(qkv, q, k, v, pos, rows, freq, slots=sl)
    (q_ref, mag), _, _ = ref.rope(qkv, Hq, Hkv, hd, pos, freq, None, None, 0, 1.0, False)
    assert ((q.double() - q_ref).abs() <= ref.ROPE_TOL * mag).all()
    x = qkv.view(n, -1, hd)
    assert torch.equal(v[0, :, 0], x[0, 3:].to(BF)) and torch.equal(v[1, :, 5], x[5, 3:].to(BF))
    for c, c0 in ((k, k0), (v, v0)):
        c[0, :, 0], c[1, :, 5] = c0[0, :, 0], c0[1, :, 5]
        assert torch.equal(c, c0)


# ------------------------------------------------------------- tree_attention
class Case:
    def __init__(self, dev, lengths, T, Hq, Hkv, hd, dtype, counts=None, S=None, slots=None, n_slots=None, seed=0,
                 roots=1, q_scale=1.5):
        g = torch.Generator().manual_seed(seed + 31 * T + Hq + hd + sum(lengths))
        B = len(lengths)
        self.S = S or max(lengths) + T
        n_slots = n_slots or B
        self.q = (q_scale * torch.randn(B, T, Hq, hd, generator=g)).to(dtype).to(dev)
        self.k = normal(g, n_slots, Hkv, self.S, hd, dtype=BF)
        self.v = normal(g, n_slots, Hkv, self.S, hd, dtype=BF)
        self.out = torch.full((B, T, Hq, hd), 99.0, dtype=dtype, device=dev)
        self.lengths = torch.tensor(lengths, dtype=I32, device=dev)
        self.counts = None if counts is None else torch.tensor(counts, dtype=I32, device=dev)
        self.slots = None if slots is None else torch.tensor(slots, dtype=I32, device=dev)
        words = [ref.mask_words(ref.random_parents(T, g, roots)) for _ in range(B)]
        self.masks = torch.tensor([[ref.signed(w) for w in r] for r in words], dtype=torch.int64, device=dev)
        self.scale = hd ** -0.5

    def run(self, **kw):
        _lib.tree_attention(self.q, self.k, self.v, self.lengths, self.masks, self.out, counts=self.counts,
                            slots=self.slots, **kw)

    def check(self):
        torch.cuda.synchronize()
        want, tol = ref.attention(self.q, self.k, self.v, self.lengths, self.masks, self.counts, self.slots, self.scale)
        got = self.out.double()
        behind = want.isnan()
        assert (got[behind] == 99.0).all()  # nodes behind the last one: not written
        err = (got - want).abs()[~behind]
        assert got[~behind].isfinite().all()
        worst = (err / tol[~behind]).max() if err.numel() else 0
        assert (err <= tol[~behind]).all(), (float(err.max()), float(worst))


@pytest.mark.parametrize("dtype", [torch.float32, BF])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("T,Hq,Hkv", [(1, 1, 1), (1, 32, 8), (2, 4, 2), (8, 4, 1), (17, 6, 2), (16, 16, 2), (33, 24, 8),
                                      (64, 8, 2), (64, 16, 1), (31, 32, 2)])
@pytest.mark.parametrize("length", [0, 1, 63, 200])
def test_tree_attention_matches_the_formula(dev, dtype, hd, T, Hq, Hkv, length):
    c = Case(dev, [length], T, Hq, Hkv, hd, dtype)
    c.run()
    c.check()


@pytest.mark.parametrize("dtype", [torch.float32, BF])
@pytest.mark.parametrize("length", [64, 127, 128, 129, 255, 256, 257, 511, 513, 1023, 2049, 5000])
def test_tree_attention_lengths_around_tiles(dev, dtype, length):
    for hd, T, Hq, Hkv in ((64, 12, 8, 2), (128, 3, 4, 2)):
        c = Case(dev, [length], T, Hq, Hkv, hd, dtype, S=length + T + 37)
        c.run(max_len=length)
        c.check()


@pytest.mark.parametrize("dtype", [torch.float32, BF])
@pytest.mark.parametrize("hd", [64, 128])
def test_tree_attention_ragged_batch_slots_and_counts(dev, dtype, hd):
    c = Case(dev, [700, 0, 129, 1, 64], 20, 8, 2, hd, dtype, counts=[20, 1, 0, 13, 7], slots=[4, 6, 0, 2, 5], n_slots=7,
             S=760, roots=3)
    c.run()
    c.check()
    c.out.fill_(99.0)
    c.run(max_len=5)  # only a hint: longer sequences are still right
    c.check()


@pytest.mark.parametrize("dtype", [torch.float32, BF])
@pytest.mark.parametrize("hd", [64, 128])
def test_tree_attention_empty_rows_and_junk_behind_masks(dev, dtype, hd):
    """No committed rows and masks of no bit: zeros. Rows that a node does not see may hold anything."""
    T = 9
    c = Case(dev, [0, 150], T, 4, 2, hd, dtype, counts=[T, 5], S=300)
    c.masks[0, 2] = 0
    c.masks[0, 3] = 1 << 40  # a bit behind the tree
    c.masks[0, 4] = -1       # every bit: the T nodes
    c.masks[1, 3] = 1 << 3
    nan, inf = float("nan"), float("inf")
    for x in (c.k, c.v):
        x[:, :, 200:] = nan
        x[0, :, T:] = inf
        x[1, :, 155:] = nan          # behind the sequence's five nodes
    c.run()
    c.check()
    assert (c.out[0, 2:4] == 0).all()
    # a node whose keys and values are not finite reaches those that see it, and no other
    keep = c.out.clone()
    c.v[1, :, 154] = inf
    c.k[1, 0, 154] = nan
    c.v[1, 1, 154, 3] = nan
    c.masks[1, :4] &= ~(1 << 4)
    c.masks[1, 4] |= 1 << 4
    c.run()
    torch.cuda.synchronize()
    assert torch.equal(c.out[1, :4], keep[1, :4])
    assert not c.out[1, 4].isfinite().all()
    assert torch.equal(c.out[0], keep[0])


@pytest.mark.parametrize("dtype", [torch.float32, BF])
def test_tree_attention_strided_queries_and_outputs(dev, dtype):
    c = Case(dev, [90, 33], 6, 4, 2, 64, dtype)
    B, T, Hq, hd = c.q.shape
    wide = torch.zeros(B, T + 2, 8, hd, dtype=dtype, device=dev)
    wide[:, :T, :4] = c.q
    c.q = wide[:, :T, :4]
    out = torch.full((T, B, Hq, hd), 99.0, dtype=dtype, device=dev)
    c.out = out.transpose(0, 1)
    c.run()
    c.check()


@pytest.mark.parametrize("dtype", [torch.float32, BF])
def test_tree_attention_large_scores(dev, dtype):
    """Scores of hundreds, rising along the cache: the running maximum changes in every tile."""
    c = Case(dev, [600], 5, 4, 1, 64, dtype, q_scale=30.0)
    c.k[0, 0] *= torch.linspace(0.1, 2.0, c.S, device=dev).to(BF)[:, None]
    c.run()
    c.check()
    c.out.fill_(99.0)
    c.k = c.k.flip(2).contiguous()
    c.run()
    c.check()


def test_tree_attention_lengths_are_cut_to_the_cache(dev):
    c = Case(dev, [40, 40, 40, 40], 4, 2, 1, 64, torch.float32, S=44)
    c.run()
    want = c.out.clone()
    c.out.fill_(99.0)
    c.lengths = torch.tensor([40, 44, 2 ** 31 - 1, -5], dtype=I32, device=dev)
    c.counts = torch.tensor([2 ** 31 - 1, 4, 4, -1], dtype=I32, device=dev)
    c.run()
    torch.cuda.synchronize()
    assert torch.equal(c.out[0], want[0])
    assert (c.out[1:] == 99.0).all()  # no room for a node, or none
    c.slots = torch.tensor([0, 4, -1, 2 ** 31 - 1], dtype=I32, device=dev)
    c.lengths.fill_(40)
    c.counts.fill_(4)
    c.out.fill_(99.0)
    c.run()
    torch.cuda.synchronize()
    assert torch.equal(c.out[0], want[0]) and (c.out[1:] == 99.0).all()


def test_tree_attention_offsets_past_32_bits(dev):
    S, hd, Hkv, T = (1 << 20) + 64, 128, 8, 5
    k = torch.empty(3, Hkv, S, hd, dtype=BF, device=dev)
    v = torch.empty(3, Hkv, S, hd, dtype=BF, device=dev)
    assert k.numel() > 2 ** 31
    g = torch.Generator().manual_seed(3)
    c = Case(dev, [300], T, Hkv, Hkv, hd, torch.float32, n_slots=1)
    k[2, :, :305], v[2, :, :305] = c.k[0], c.v[0]
    c.run()
    c.check()
    want = c.out.clone()
    c.out.fill_(99.0)
    small = c.k, c.v
    c.k, c.v, c.slots = k, v, torch.tensor([2], dtype=I32, device=dev)
    c.run(max_len=300)
    torch.cuda.synchronize()
    assert torch.equal(c.out, want) or (c.out - want).abs().max() < 1e-5
    # and its last rows, far out in the slot
    c.k, c.v, c.slots = small[0], small[1], None
    del k, v
    far = 1 << 20
    kk = torch.randn(1, 1, S, hd, device=dev).to(BF)
    vv = torch.randn(1, 1, S, hd, device=dev).to(BF)
    d = Case(dev, [70], T, 1, 1, hd, BF)
    d.k, d.v, d.lengths = kk, vv, torch.tensor([far], dtype=I32, device=dev)
    d.run()
    d.check()


def test_tree_attention_is_repeatable_in_streams_and_graphs(dev):
    cases = [Case(dev, [900, 30], 16, 8, 2, 64, torch.float32, seed=s) for s in (1, 2)]
    for c in cases:
        c.run()
    torch.cuda.synchronize()
    want = [c.out.clone() for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    for rep in range(10):
        for c in cases:
            c.out.fill_(99.0)
        torch.cuda.synchronize()
        for c, s in zip(cases, streams):
            c.run(stream=s)
        torch.cuda.synchronize()
        for c, w in zip(cases, want):
            assert torch.equal(c.out, w)
    # captured once, replayed on new inputs, two graphs alive at once
    graphs = []
    for c in cases:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            c.run()
        graphs.append(gr)
    for c in cases:
        c.q.mul_(-1)
        c.lengths.add_(-7)
    for gr, s in zip(graphs, streams):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            gr.replay()
    torch.cuda.synchronize()
    for c in cases:
        c.check()


@pytest.mark.parametrize("hd,T,Hq,Hkv,dtype", [(64, 12, 8, 2, torch.float32), (64, 40, 8, 2, BF), (128, 20, 6, 2, BF),
                                               (128, 3, 2, 1, torch.float32)])
def test_tree_attention_long_caches_in_streams_and_graphs(dev, hd, T, Hq, Hkv, dtype):
    """Caches split through the workspace: repeated, in two streams at once, and in two graphs replayed side by side."""
    cases = [Case(dev, [6000], T, Hq, Hkv, hd, dtype, seed=s) for s in (1, 2)]
    for c in cases:
        c.run(max_len=6000)
        c.check()
    want = [c.out.clone() for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    graphs = []
    for c in cases:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            c.run(max_len=6000)
        graphs.append(gr)
    for rep in range(6):
        for c in cases:
            c.out.fill_(99.0)
        torch.cuda.synchronize()
        for c, s, gr in zip(cases, streams, graphs):
            if rep % 2:
                with torch.cuda.stream(s):
                    gr.replay()
            else:
                c.run(max_len=6000, stream=s)
        torch.cuda.synchronize()
        for c, w in zip(cases, want):
            assert torch.equal(c.out, w)


# Large trees (128 rows and more) of ragged batches, in caches far longer than the sequences.
LARGE = [(64, torch.float32), (64, BF), (128, torch.float32), (128, BF)]
FAR = 16400


@pytest.mark.parametrize("hd,dtype", LARGE)
def test_tree_attention_large_trees_ragged(dev, hd, dtype):
    c = Case(dev, [700, 0, 129, 1, 64, 3000, 127, 128], 40, 8, 2, hd, dtype, counts=[40, 1, 0, 13, 7, 40, 33, 32],
             slots=[4, 6, 0, 2, 5, 7, 1, 8], n_slots=9, S=FAR, roots=3)
    c.run()
    c.check()
    c.out.fill_(99.0)
    c.slots[3], c.lengths[6], c.counts[7] = 9, FAR, -1  # outside the caches, no room, no node
    c.run()
    torch.cuda.synchronize()
    assert (c.out[[3, 6, 7]] == 99.0).all()
    c.slots[3], c.lengths[6] = 3, 0  # (for the plain form: the same, said in bounds)
    c.counts[3] = c.counts[6] = c.counts[7] = 0
    c.check()
    c.counts.fill_(0)  # no work at all
    c.out.fill_(99.0)
    c.run()
    torch.cuda.synchronize()
    assert (c.out == 99.0).all()


@pytest.mark.parametrize("hd,dtype", LARGE)
def test_tree_attention_large_trees_of_many_short_sequences(dev, hd, dtype):
    B = 33
    c = Case(dev, [(7 * b) % 150 for b in range(B)], 17, 32, 4, hd, dtype, S=4400, counts=[1 + (5 * b) % 17 for b in range(B)])
    c.run()
    c.check()


@pytest.mark.parametrize("hd,dtype", LARGE)
def test_tree_attention_large_trees_junk(dev, hd, dtype):
    T = 40
    c = Case(dev, [0, 150, 600, 90, 255, 256, 1000, 5], T, 8, 2, hd, dtype, counts=[T, 5, T, T, T, T, T, T], S=FAR)
    c.masks[0, 2] = 0
    c.masks[0, 3] = 1 << 45  # a bit behind the tree
    c.masks[2, 35] = -1      # every bit: the T nodes
    nan, inf = float("nan"), float("inf")
    for x in (c.k, c.v):
        x[:, :, 1100:] = nan
        x[0, :, T:] = inf
        x[1, :, 155:] = nan
    c.run()
    c.check()
    assert (c.out[0, 2:4] == 0).all()
    # keys and values of nodes that nobody but themselves sees; two tiles of one sequence, and other sequences
    hit = [(1, 154 - 150), (3, 20), (3, 39), (4, 0), (6, 30)]
    for b, t in hit:
        c.masks[b] &= ~(1 << t)
        c.masks[b, t] |= 1 << t
    c.run()
    torch.cuda.synchronize()
    keep = c.out.clone()
    for b, t in hit:
        at = int(c.lengths[b]) + t
        c.v[b, :, at] = inf
        c.k[b, 0, at] = nan
        c.v[b, 1, at, 3] = nan
    c.run()
    torch.cuda.synchronize()
    for b in range(8):
        for t in range(T):
            if (b, t) in hit:
                assert not c.out[b, t].isfinite().all()
            else:
                assert torch.equal(c.out[b, t], keep[b, t]), (b, t)


@pytest.mark.parametrize("hd,dtype", LARGE)
def test_tree_attention_large_trees_in_streams_and_graphs(dev, hd, dtype):
    cases = [Case(dev, [3000, 100, 2047, 900, 31, 4000, 500, 1], 40, 8, 2, hd, dtype, S=FAR, seed=s) for s in (1, 2)]
    for c in cases:
        c.run()
        c.check()
    want = [c.out.clone() for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    graphs = []
    for c in cases:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            c.run()
        graphs.append(gr)
    for rep in range(6):
        for c in cases:
            c.out.fill_(99.0)
        torch.cuda.synchronize()
        for c, s, gr in zip(cases, streams, graphs):
            if rep % 2:
                with torch.cuda.stream(s):
                    gr.replay()
            else:
                c.run(stream=s)
        torch.cuda.synchronize()
        for c, w in zip(cases, want):
            assert torch.equal(c.out, w)
    for c in cases:  # other lengths in the same graph
        c.lengths.copy_(c.lengths.flip(0))
        c.out.fill_(99.0)
    graphs[0].replay()
    graphs[1].replay()
    for c in cases:
        c.check()


@pytest.mark.parametrize("T,lengths", [(16, [16000, 16000]), (40, [9000, 15000]), (33, [16000] * 4)])
def test_tree_attention_partly_filled_row_tiles_over_long_caches(dev, T, lengths):
    """Row tiles with warps that have no row, and caches from memory: warps and products drift apart; no wait runs out."""
    c = Case(dev, lengths, T, 32, 8, 64, BF, S=FAR)
    status = torch.zeros(1, dtype=I32, device=dev)
    for _ in range(5):
        c.out.fill_(99.0)
        c.run(max_len=max(lengths), status=status)
    c.check()
    assert int(status) == 0


def test_tree_attention_far_scores_and_status(dev):
    """Scores below -1e30 are scores all the same; the status word stays 0."""
    c = Case(dev, [70], 3, 2, 1, 64, torch.float32)
    c.q = torch.full_like(c.q, 3e18)
    c.k = -torch.full_like(c.k, 3e15)
    c.k[0, 0, 5] *= 0.5  # the largest score by far: its value comes back
    st = torch.zeros(1, dtype=I32, device=dev)
    c.run(status=st)
    torch.cuda.synchronize()
    assert int(st) == 0
    assert torch.equal(c.out, c.v[0, 0, 5].float().expand_as(c.out))


# ---------------------------------------------------------------- tree_masks
@pytest.mark.parametrize("T", [1, 2, 31, 33, 64])
def test_tree_masks_of_random_trees(dev, T):
    g = torch.Generator().manual_seed(T)
    B = 5
    parents = [ref.random_parents(T, g, roots=1 + b % 2 if T > 1 else 1) for b in range(B)]
    p = torch.tensor(parents, dtype=I32, device=dev)
    m = torch.full((B, T), 17, dtype=torch.int64, device=dev)
    d = torch.full((B, T), 17, dtype=I32, device=dev)
    counts = torch.tensor([T, T, max(0, T - 1), 0, 1], dtype=I32, device=dev)
    _lib.tree_masks(p, m, d, counts)
    for b in range(B):
        n = int(counts[b])
        words = ref.mask_words(parents[b])
        assert m[b].tolist() == [ref.signed(w) for w in words[:n]] + [17] * (T - n)
        assert d[b].tolist() == [bin(w).count("1") - 1 for w in words[:n]] + [17] * (T - n)


def test_tree_masks_of_bad_parents_are_roots(dev):
    p = torch.tensor([[5, 0, 2, 9, -7, 3]], dtype=I32, device=dev)
    m = torch.zeros(1, 6, dtype=torch.int64, device=dev)
    d = torch.zeros(1, 6, dtype=I32, device=dev)
    _lib.tree_masks(p, m, d)
    assert m[0].tolist() == [1, 3, 4, 8, 16, 40] and d[0].tolist() == [0, 1, 0, 0, 0, 1]


# ------------------------------------------------------------- cache moves
@pytest.mark.parametrize("L,B,Hkv,S,hd,T", [(1, 1, 1, 5, 64, 1), (2, 1, 2, 100, 64, 16), (3, 4, 2, 90, 128, 64),
                                            (1, 2, 3, 70, 64, 33)])
def test_kv_compact(dev, L, B, Hkv, S, hd, T):
    g = torch.Generator().manual_seed(S)
    k, v = normal(g, L, B, Hkv, S, hd, dtype=BF), normal(g, L, B, Hkv, S, hd, dtype=BF)
    starts = torch.randint(0, max(1, S - T + 1), (B,), generator=g)
    counts = torch.randint(0, T + 1, (B,), generator=g)
    counts[0] = T
    nodes = torch.stack([torch.randperm(T, generator=g).sort().values if b % 2 else torch.randperm(T, generator=g)
                         for b in range(B)])
    want = [ref.compact(x, starts, nodes, counts) for x in (k, v)]
    _lib.kv_compact(k, v, *(x.to(I32).to(dev) for x in (starts, nodes, counts)))
    assert torch.equal(k, want[0]) and torch.equal(v, want[1])


def test_kv_compact_repeated_bad_and_far_nodes(dev):
    g = torch.Generator().manual_seed(1)
    k, v = normal(g, 1, 4, 2, 40, 64, dtype=BF), normal(g, 1, 4, 2, 40, 64, dtype=BF)
    starts = torch.tensor([30, 39, -1, 2 ** 31 - 1])
    nodes = torch.tensor([[3, 3, -1, 10, 9, 2], [0, 1, 2, 3, 4, 5], [1] * 6, [1] * 6])
    counts = torch.tensor([100, 6, 6, 6])  # cut to the six nodes
    want = []
    for x in (k, v):
        w = x.clone()
        for i, nd in enumerate([3, 3, None, None, 9, 2]):
            if nd is not None:
                w[:, 0, :, 30 + i] = x[:, 0, :, 30 + nd]
        want.append(w)
    _lib.kv_compact(k, v, *(x.to(I32).to(dev) for x in (starts, nodes, counts)))
    assert torch.equal(k, want[0]) and torch.equal(v, want[1])


@pytest.mark.parametrize("L,B,Hkv,S,hd", [(1, 1, 1, 3, 64), (2, 3, 2, 77, 64), (2, 8, 2, 130, 128), (1, 13, 1, 40, 64),
                                          (1, 30, 2, 33, 64), (1, 64, 1, 50, 128)])
def test_kv_reorder(dev, L, B, Hkv, S, hd):
    g = torch.Generator().manual_seed(B)
    for rep in range(4):
        k, v = normal(g, L, B, Hkv, S, hd, dtype=BF), normal(g, L, B, Hkv, S, hd, dtype=BF)
        lengths = torch.randint(-2, S + 3, (B,), generator=g)
        sources = [torch.randperm(B, generator=g), torch.zeros(B, dtype=torch.int64), torch.arange(B).roll(1),
                   torch.randint(-2, B + 3, (B,), generator=g)][rep]
        want = [ref.reorder(x, sources, lengths) for x in (k, v)]
        _lib.kv_reorder(k, v, sources.to(I32).to(dev), lengths.to(I32).to(dev))
        assert torch.equal(k, want[0]) and torch.equal(v, want[1])


def test_cache_moves_past_32_bit_offsets(dev):
    L, B, Hkv, S, hd = 9, 2, 1, 1 << 20, 128
    k = torch.zeros(L, B, Hkv, S, hd, dtype=BF, device=dev)
    v = torch.zeros(1, dtype=BF, device=dev).expand(1)
    assert k.numel() > 2 ** 31
    v = torch.zeros_like(k)
    g = torch.Generator().manual_seed(2)
    k[8, 1, 0, -64:] = normal(g, 64, hd, dtype=BF)
    v[8, 1, 0, -64:] = normal(g, 64, hd, dtype=BF)
    want = k[8, 1, 0, -64:].clone()
    _lib.kv_compact(k, v, torch.tensor([0, S - 64], dtype=I32, device=dev),
                    torch.tensor([[0, 1], [40, 50]], dtype=I32, device=dev),
                    torch.tensor([0, 2], dtype=I32, device=dev))
    want[:2] = want[[40, 50]]
    assert torch.equal(k[8, 1, 0, -64:], want)
    _lib.kv_reorder(k, v, torch.tensor([1, 1], dtype=I32, device=dev), torch.tensor([S, S], dtype=I32, device=dev))
    assert torch.equal(k[8, 0, 0, -64:], want) and torch.equal(k[8, 1, 0, -64:], want)


def test_cache_moves_in_a_graph(dev):
    g = torch.Generator().manual_seed(9)
    k, v = normal(g, 2, 4, 2, 64, 64, dtype=BF), normal(g, 2, 4, 2, 64, 64, dtype=BF)
    src = torch.tensor([1, 0, 3, 2], dtype=I32, device=dev)
    ln = torch.tensor([64, 64, 10, 10], dtype=I32, device=dev)
    starts, counts = torch.full((4,), 8, dtype=I32, device=dev), torch.full((4,), 3, dtype=I32, device=dev)
    nodes = torch.tensor([[0, 2, 5]] * 4, dtype=I32, device=dev)
    k0, v0 = k.clone(), v.clone()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        _lib.kv_reorder(k, v, src, ln)
        _lib.kv_compact(k, v, starts, nodes, counts)
    for _ in range(3):
        gr.replay()
        k0, v0 = (ref.compact(ref.reorder(x, src, ln), starts, nodes, counts) for x in (k0, v0))
    assert torch.equal(k, k0) and torch.equal(v, v0)


# ---------------------------------------------------------------- together
@pytest.mark.parametrize("dtype", [torch.float32, BF])
@pytest.mark.parametrize("hd,T,Hq,Hkv", [(64, 5, 4, 2), (64, 21, 8, 2), (128, 13, 6, 2)])
def test_a_step_of_trees_in_one_graph(dev, dtype, hd, T, Hq, Hkv):
    """Masks and depths, rotation and append by depth, attention, compaction of a path: a padded batch in slots out of
    order, captured on a stream of its own, replayed on other trees."""
    B, n_slots, S = 3, 4, 320
    g = torch.Generator().manual_seed(hd + T)
    width = (Hq + 2 * Hkv) * hd
    qkv = torch.zeros(B, T, width, dtype=dtype, device=dev)
    out = torch.zeros(B, T, Hq, hd, dtype=dtype, device=dev)
    k, v = (torch.zeros(1, n_slots, Hkv, S, hd, dtype=BF, device=dev) for _ in range(2))
    ints = {n: torch.zeros(*s, dtype=I32, device=dev) for n, s in
            dict(parents=(B, T), depths=(B, T), counts=(B,), lengths=(B,), positions=(B * T,), rows=(B * T,),
                 token_slots=(B * T,), slots=(B,), starts=(n_slots,), moved=(n_slots,), nodes=(n_slots, T)).items()}
    masks = torch.zeros(B, T, dtype=torch.int64, device=dev)
    freq = _lib.rope_frequencies(hd, 1e4)[0].to(dev)
    q = qkv.view(B, T, -1, hd)[:, :, :Hq]
    i, step = ints, torch.arange(T, dtype=I32, device=dev)

    def run():
        _lib.tree_masks(i["parents"], masks, depths=i["depths"], counts=i["counts"])
        i["positions"].copy_((i["lengths"][:, None] + i["depths"]).view(-1))
        i["rows"].copy_(torch.where(step < i["counts"][:, None], i["lengths"][:, None] + step, -1).view(-1))
        flat = qkv.view(B * T, width)
        _lib.rope_append(flat, flat[:, :Hq * hd].view(B * T, Hq, hd), k[0], v[0], i["positions"], i["rows"], freq,
                         slots=i["token_slots"])
        _lib.tree_attention(q, k[0], v[0], i["lengths"], masks, out, counts=i["counts"], slots=i["slots"])
        _lib.kv_compact(k, v, i["starts"], i["nodes"], i["moved"])

    def fill(seed):
        """New contents of every array; what run() has to make of them, from the 64-bit forms."""
        g.manual_seed(seed)
        lengths, counts, slots = [130, 3, 250], [T, T - 3, 2], [2, 0, 3] if seed % 2 else [1, 3, 2]
        parents = torch.full((B, T), -1, dtype=I32)
        for b in range(B):
            parents[b, :counts[b]] = torch.tensor(ref.random_parents(counts[b], g), dtype=I32)
        i["parents"].copy_(parents)
        for name, x in (("lengths", lengths), ("counts", counts), ("slots", slots)):
            i[name].copy_(torch.tensor(x, dtype=I32))
        i["token_slots"].copy_(torch.tensor(slots, dtype=I32).repeat_interleave(T))
        paths = []
        for b in range(B):
            at, path = counts[b] - 1, []
            while at >= 0:
                path.insert(0, at)
                at = int(parents[b, at])
            paths.append(path)
        starts, moved, nodes = torch.zeros(n_slots, dtype=I32), torch.zeros(n_slots, dtype=I32), torch.zeros(n_slots, T, dtype=I32)
        for b in range(B):
            starts[slots[b]], moved[slots[b]] = lengths[b], len(paths[b])
            nodes[slots[b], :len(paths[b])] = torch.tensor(paths[b], dtype=I32)
        for name, x in (("starts", starts), ("moved", moved), ("nodes", nodes)):
            i[name].copy_(x)
        qkv.copy_(normal(g, B, T, width, dtype=dtype))
        k.copy_(normal(g, *k.shape, dtype=BF))
        v.copy_(normal(g, *v.shape, dtype=BF))
        out.fill_(99.0)
        masks.fill_(-1)
        i["depths"].fill_(0)
        return lengths, counts, slots, parents, paths, qkv.clone(), k.clone(), v.clone()

    def check(lengths, counts, slots, parents, paths, qkv0, k0, v0):
        words = torch.full((B, T), -1, dtype=torch.int64)
        for b in range(B):
            w = ref.mask_words(parents[b, :counts[b]].tolist())
            words[b, :counts[b]] = torch.tensor([ref.signed(x) for x in w])
            depth = torch.tensor([bin(x).count("1") - 1 for x in w], dtype=I32, device=dev)
            assert torch.equal(i["depths"][b, :counts[b]], depth)
            (q_ref, q_mag), (k_ref, k_mag), v_ref = ref.rope(qkv0[b, :counts[b]], Hq, Hkv, hd, lengths[b] + depth, freq,
                                                             None, None, 0.0, 1.0, False)
            tol = ref.ROPE_TOL * q_mag
            half = 0.0 if dtype == torch.float32 else ref.BF
            got = q[b, :counts[b]].double()
            assert ((got - q_ref).abs() <= tol + half * (q_ref.abs() + tol)).all()
            # the cache as it was, with the path's rows (all of them, unmoved, behind)
            kb, vb = k0[0, slots[b]], v0[0, slots[b]]
            rows = slice(lengths[b], lengths[b] + counts[b])
            vb[:, rows] = v_ref.to(BF).transpose(0, 1)
            tol = ref.ROPE_TOL * k_mag
            tol = tol + ref.BF * (k_ref.abs() + tol)
            bound = torch.zeros(Hkv, S, hd, dtype=torch.float64, device=dev)
            want = kb.double()
            want[:, rows], bound[:, rows] = k_ref.transpose(0, 1), tol.transpose(0, 1)
            for to, node in enumerate(paths[b]):  # a path's nodes only move down: in order is as if at once
                for x in (want, bound, vb):
                    x[:, lengths[b] + to] = x[:, lengths[b] + node]
            assert torch.equal(v[0, slots[b]], vb)
            assert ((k[0, slots[b]].double() - want).abs() <= bound).all()
        assert torch.equal(masks.cpu(), words)
        return words

    def attended(lengths, counts, slots, words, kk, vv):
        cn, sl = torch.tensor(counts), torch.tensor(slots)
        o, tol = ref.attention(q, kk[0], vv[0], lengths, words, cn, sl, hd ** -0.5)
        on = ~o.isnan()
        assert ((out.double() - o).abs()[on] <= tol[on]).all()
        for b in range(B):
            assert (out[b, counts[b]:] == 99.0).all()

    side = torch.cuda.Stream()
    fill(0)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        run()
    for seed in (1, 2):
        made = fill(seed)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graph.replay()
        torch.cuda.synchronize()
        words = check(*made)
        # attention read the appended rows before the path moved: what the moves did not touch lies there still,
        # and the moved rows' first copies are redone here
        kk, vv = made[6].clone(), made[7].clone()
        again = made[5].view(B * T, width).clone()
        _lib.rope_append(again, torch.empty(B * T, Hq, hd, dtype=dtype, device=dev), kk[0], vv[0], i["positions"],
                         i["rows"], freq, slots=i["token_slots"])
        torch.cuda.synchronize()
        attended(*made[:3], words, kk, vv)
