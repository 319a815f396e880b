"""Sums of paged_attention over long caches, whatever bounds and workspace the call is given."""
import ctypes

import pytest
import torch

from decode_megakernel_llama_gb300 import _lib
from decode_megakernel_llama_gb300.build import build
from tests import paged_reference as ref
from tests.test_paged_gpu import Paged

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()


def call(p, workspace, **kw):
    """mk_paged_attention on p through the C ABI, with the workspace that it asks for or none."""
    row = p.Hq * p.hd
    at = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    rec = dict(n_tokens=p.q.shape[0], batch=p.lengths.numel(), max_pages=p.table.shape[1], n_heads=p.Hq,
               n_kv_heads=p.k.shape[1], head_dim=p.hd, dtype=0 if p.q.dtype == torch.float32 else 1,
               cache_dtype=1 if p.ks is None else 2, n_pages=p.k.shape[0], page_size=p.k.shape[2], window=p.window,
               sinks=p.sinks, scale=p.hd ** -0.5, q_stride=row, out_stride=row, q=at(p.q), out=at(p.out), k_pages=at(p.k),
               v_pages=at(p.v), k_scales=at(p.ks), v_scales=at(p.vs), table=at(p.table), starts=at(p.starts),
               lengths=at(p.lengths), status=at(p.status), **kw)
    lib, work = _lib.load(), None
    need = lib.mk_paged_attention_workspace(ctypes.byref(_lib.mk_paged_args(**rec)))
    assert need >= 0
    if workspace and need:
        work = torch.empty(need, dtype=torch.uint8, device="cuda")
        rec.update(workspace=work.data_ptr(), workspace_bytes=need)
    assert lib.mk_paged_attention(ctypes.byref(_lib.mk_paged_args(**rec)), torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    assert int(p.status) == 0


@pytest.mark.parametrize("sign", ["plus", "minus", "by dim"])
@pytest.mark.parametrize("how", ["bounds", "no workspace", "a bound that is exceeded"])
@pytest.mark.parametrize("hd,Hkv,new,cache", [(64, 2, 3, "bf16"), (64, 2, 8, "e4m3"), (64, 2, 60, "bf16"), (128, 2, 3, "e4m3"),
                                              (128, 2, 8, "bf16"), (128, 2, 60, "bf16"), (64, 1, 300, "bf16")])
def test_sums_do_not_hang_on_bounds_workspace_or_sign(hd, Hkv, new, cache, how, sign):
    """fp32 queries, values of one sign in a dim, so that a sum that cuts what it cannot hold falls behind with every
    product. At most 8 tiles of a group (or 2, of many rows) are added up by a tensor core, 8 * 8 * 3 products that cut at most
    2^-23 each; what adds those up rounds, 2^-24 for each of 30 sums of tiles (or 118) and some joins: 200. Beside them the
    weights' sums, which one thread adds up over 235 tiles where they are not the product's (2^-24 each, 235 and the warp's 8),
    the scores' error twice and the weights', as in paged_reference.attention."""
    L, G = 60000, 4
    p = Paged([L], [new], Hkv * G, Hkv, hd, 128, "f32", "bf16", seed=9, poison=False, q_scale=0.5)
    to = {"plus": 1.0, "minus": -1.0, "by dim": torch.where(torch.arange(hd, device="cuda") % 3 == 0, -1.0, 1.0)}[sign]
    p.v = (p.v.abs() * to).to(BF)
    if cache == "e4m3":
        (p.k, p.ks), (p.v, p.vs) = (ref.quantise(x.double()) for x in (p.k, p.v))
        p.k64, p.v64 = ref.values(p.k, p.ks), ref.values(p.v, p.vs)
    else:
        p.k64, p.v64 = p.k.double(), p.v.double()
    call(p, how != "no workspace", max_new=new, max_len=1 if how == "a bound that is exceeded" else L)
    want, tol = ref.attention(p.q, p.k64, p.v64, p.table.cpu(), p.starts.cpu(), p.lengths.cpu(), hd ** -0.5, 0, 0)
    n = torch.arange(L - new + 1, L + 1, device="cuda")[:, None, None]
    loose = (3 * n / 16 + 80) * 2.0 ** -23  # (that bound's share of the sums, of sum p|v| = |the result| here)
    tight = tol - want.abs() * loose + want.abs() * (8 * 8 * 3 * 2.0 ** -23 + (200 + 243) * 2.0 ** -24)
    err = (p.out.double() - want).abs()
    assert bool((err <= tight).all()), f"worst {float((err / want.abs()).max()):.2e} of a result, {float((err / tight).max())} bounds"


@pytest.mark.parametrize("hd,cache", [(64, "bf16"), (128, "bf16"), (64, "e4m3"), (128, "e4m3")])
def test_bf16_results_of_a_million_rows_are_rounded_once(hd, cache):
    """One CTA over 2^20 rows (the bound says one). A result is the rounding of a value within `off` of the formula's, so it
    lies between the roundings of the ends: off is twice the scores' error (3 hd products in fp32 each) and 2^-20, the
    weights' 2^-16, 8 * 8 * 2 products that cut at most 2^-23, and what adds those up (512 of them) and the weights (4,096 of a
    thread, 8 over a warp), 2^-24 each. Sums that cut left results 2.6e-3 short."""
    L, new, G = 1 << 20, 3, 4
    g = torch.Generator(device="cuda").manual_seed(1)
    q = (0.5 * torch.randn(new, G, hd, generator=g, device="cuda")).to(BF)
    k, v = (torch.randn(1, 1, L, hd, generator=g, device="cuda").to(BF) for _ in range(2))
    v = v.abs()
    ks = vs = None
    k64, v64 = k, v
    if cache == "e4m3":  # (one power for all: every value fits)
        k, v = (x.float().clamp(-7, 7).mul(64).to(ref.E4M3) for x in (k, v))
        ks = vs = torch.full((1, 1, L, hd // 32), 127 - 6, dtype=torch.uint8, device="cuda")
        k64, v64 = (x.float() / 64 for x in (k, v))
    out = torch.zeros_like(q)
    i32 = dict(dtype=torch.int32, device="cuda")
    _lib.paged_attention(q, k, v, torch.zeros(1, 1, **i32), torch.tensor([0, new], **i32), torch.tensor([L], **i32), out,
                         k_scales=ks, v_scales=None if vs is None else vs.clone(), max_new=new, max_len=1)
    for t in range(new):
        n = L - new + t + 1
        kk, vv, qq = k64[0, 0, :n].double(), v64[0, 0, :n].double(), q[t].double()
        want = torch.softmax(hd ** -0.5 * qq @ kk.T, -1) @ vv
        d = hd ** -0.5 * (qq.abs() @ kk.abs().T).amax(-1, keepdim=True) * 3 * hd * 2.0 ** -24
        off = 2 * d + 2.0 ** -20 + 2.0 ** -16 + 128 * 2.0 ** -23 + (512 + 4096 + 8) * 2.0 ** -24
        low, high = (want * (1 - off)).to(BF), (want * (1 + off)).to(BF)
        assert bool(((out[t] >= low) & (out[t] <= high)).all()), float((out[t].double() - want).mean() / want.mean())


def _need(**kw):
    a = dict(n_tokens=1, batch=1, max_pages=8192, n_heads=32, n_kv_heads=8, head_dim=128, dtype=1, cache_dtype=1,
             n_pages=20000, page_size=16, scale=0.1, q=1 << 30, out=1 << 50, k_pages=1 << 51, v_pages=1 << 52, table=1 << 53,
             starts=1 << 53, lengths=1 << 53)
    a.update(kw)
    a.update(q_stride=a["n_heads"] * a["head_dim"], out_stride=a["n_heads"] * a["head_dim"])
    return _lib.load().mk_paged_attention_workspace(ctypes.byref(_lib.mk_paged_args(**a)))


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("hd", [64, 128])
def test_the_workspace_stays_small(dtype, hd):
    """Prompts with no bound on the rows, tokens far above the bound on a sequence's: eight waves of partial results at most,
    8 * 152 of (128 * 128 + 256) floats; a long context of one sequence still gets one. (The addresses are not followed.)"""
    most = 8 * 152 * (128 * 128 + 256) * 4
    for kw in (dict(n_tokens=4096), dict(n_tokens=4096, max_len=32768), dict(n_tokens=100000, max_new=1),
               dict(n_tokens=8192, batch=8, max_new=1), dict(n_tokens=30000, batch=4, max_new=40, max_len=100000),
               dict(n_tokens=300), dict(n_tokens=1000, batch=1000, max_new=1)):
        assert 0 <= _need(dtype=dtype, head_dim=hd, **kw) <= most, kw
    for kw in (dict(n_tokens=1), dict(n_tokens=40, max_new=40)):
        assert 0 < _need(dtype=dtype, head_dim=hd, **kw) <= most, kw


@pytest.mark.parametrize("type", ["f32", "bf16"])
def test_many_more_tokens_than_the_bound_says(type):
    """A launch padded to 5,000 tokens, of which two sequences have one each: the right results, the others untouched."""
    p = Paged([9000, 20000], [1, 1], 8, 2, 128, 64, type, "bf16", pad=4998, seed=12)
    p.run(max_new=1, max_len=20000)
    p.check()


@pytest.mark.parametrize("lens,news,Hq,Hkv,hd,cache", [
    ([476, 400, 392], [195, 150, 90], 64, 8, 64, "bf16"), ([391, 380], [240, 200], 16, 4, 64, "e4m3"),
    ([143] * 6, [141] * 6, 8, 4, 64, "bf16"), ([1265, 1100], [1024, 700], 4, 1, 64, "e4m3"),
    ([19261, 9706, 14000], [1, 1, 1], 8, 8, 64, "e4m3"), ([6996, 1500, 4000], [1, 1, 1], 24, 8, 128, "bf16"),
    ([554], [221], 32, 4, 128, "e4m3"),
])
def test_fp32_results_are_as_near_as_those_of_fp32_operations(lens, news, Hq, Hkv, hd, cache):
    """The error's norm against the same formula in torch's fp32, whose sums of 64 to 128 products round after each: at most 1.5
    times that. A tensor core that adds a score's or a result's small terms to the large ones cuts by the large ones' size,
    three times as often as it must (1.9 to 2.7 times that error): so the small terms come first, and sums stay short."""
    p = Paged(lens, news, Hq, Hkv, hd, 32, "f32", cache, seed=21, poison=False)
    p.run(max_new=max(news), max_len=max(lens))
    want = ref.attention(p.q, p.k64, p.v64, p.table.cpu(), p.starts.cpu(), p.lengths.cpu(), hd ** -0.5, 0, 0)[0]
    plain = torch.empty_like(p.out)
    for b, (n, L) in enumerate(zip(news, lens)):
        lo = sum(news[:b])
        k, v = (ref.rows_of(x, p.table[b].cpu(), L).float() for x in (p.k64, p.v64))
        q = p.q[lo:lo + n].view(n, Hkv, Hq // Hkv, hd).transpose(0, 1).reshape(Hkv, -1, hd)
        s = (q @ k.transpose(1, 2)) * hd ** -0.5
        pos = torch.arange(L - n, L, device="cuda").repeat_interleave(Hq // Hkv)
        s = torch.where(torch.arange(L, device="cuda")[None] <= pos[:, None], s, -torch.inf)
        w = torch.exp(s - s.amax(-1, keepdim=True))
        o = (w @ v) / w.sum(-1, keepdim=True)
        plain[lo:lo + n] = o.view(Hkv, n, Hq // Hkv, hd).transpose(0, 1).reshape(n, Hq, hd)
    ours, theirs = (float((x.double() - want).norm() / want.norm()) for x in (p.out, plain))
    assert ours <= 1.5 * theirs, (ours, theirs, ours / theirs)


@pytest.mark.parametrize("hd", [64, 128])
def test_many_bf16_rows_over_a_million_are_split(hd):
    """1,216 tokens of 16 heads, as many tiles of 128 query rows as the GPU has SMs, over 2^20 rows: one split's sums that cut
    left the results 3.4e-3 short. A split has 2^18 rows at most, half of them a group's, whose 2 * 2^17 / 16 products cut 2^-23
    each: 2^-9. Beside it the scores' error twice and 2^-20, the weights' 2^-16, and 4,104 roundings of the weights' sums."""
    L, new, G = 1 << 20, 1216, 16
    g = torch.Generator(device="cuda").manual_seed(1)
    q = (0.5 * torch.randn(new, G, hd, generator=g, device="cuda")).to(BF)
    k, v = (torch.randn(1, 1, L, hd, generator=g, device="cuda").to(BF) for _ in range(2))
    v = (v.abs() * torch.linspace(0.5, 1, hd, device="cuda").to(BF)).to(BF)
    out = torch.zeros_like(q)
    i32 = dict(dtype=torch.int32, device="cuda")
    for kw in (dict(), dict(max_new=new, max_len=L)):
        _lib.paged_attention(q, k, v, torch.zeros(1, 1, **i32), torch.tensor([0, new], **i32), torch.tensor([L], **i32), out, **kw)
        for t in (0, 600, new - 1):
            n = L - new + t + 1
            kk, vv, qq = k[0, 0, :n].double(), v[0, 0, :n].double(), q[t].double()
            want = torch.softmax(hd ** -0.5 * qq @ kk.T, -1) @ vv
            d = hd ** -0.5 * (qq.abs() @ kk.abs().T).amax(-1, keepdim=True) * 3 * hd * 2.0 ** -24
            off = 2 * d + 2.0 ** -20 + 2.0 ** -16 + 2.0 ** -9 + 4104 * 2.0 ** -24
            low, high = (want * (1 - off)).to(BF), (want * (1 + off)).to(BF)
            assert bool(((out[t] >= low) & (out[t] <= high)).all()), float(((out[t].double() - want) / want).mean())
