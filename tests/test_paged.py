"""Host side of the operators of a cache in pages: refusals (the argument checks come before any CUDA call), the binding's
own, and the plain forms that the GPU tests use."""
import ctypes
import os
import sys

import pytest
import torch

from decode_megakernel_llama_gb300 import _lib
from decode_megakernel_llama_gb300.build import build

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from tests import paged_reference as ref  # noqa: E402

FAKE = 1 << 30  # an aligned address that nothing may follow
FAR = 1 << 40


@pytest.fixture(scope="module")
def lib():
    build()
    return _lib.load()


def paged_args(**kw):
    a = dict(n_tokens=40, batch=3, max_pages=8, n_heads=8, n_kv_heads=2, head_dim=64, dtype=1, cache_dtype=1, n_pages=20,
             page_size=16, max_new=0, max_len=0, window=0, sinks=0, scale=0.1, q_stride=512, out_stride=512, q=FAKE,
             out=FAR, k_pages=2 * FAKE, v_pages=3 * FAKE, k_scales=None, v_scales=None, table=4 * FAKE, starts=4 * FAKE,
             lengths=4 * FAKE)
    a.update(kw)
    return _lib.mk_paged_args(**a)


Q8 = dict(cache_dtype=2, k_scales=5 * FAKE, v_scales=6 * FAKE)


@pytest.mark.parametrize("bad,code", [
    (dict(q=None), -1), (dict(out=None), -1), (dict(k_pages=None), -1), (dict(v_pages=None), -1), (dict(table=None), -1),
    (dict(starts=None), -1), (dict(lengths=None), -1), (dict(dtype=2), -1), (dict(cache_dtype=0), -1),
    (dict(cache_dtype=3), -1), (dict(cache_dtype=2), -1), (dict(cache_dtype=2, k_scales=FAR), -1),
    (dict(k_scales=FAR), -1), (dict(v_scales=FAR), -1), (dict(head_dim=96), -4), (dict(n_tokens=-1), -1),
    (dict(batch=-1), -1), (dict(max_pages=0), -1), (dict(n_heads=0), -1), (dict(n_kv_heads=0), -1), (dict(n_pages=0), -1),
    (dict(n_heads=7), -4), (dict(n_heads=34, q_stride=4096, out_stride=4096), -4), (dict(page_size=0), -1),
    (dict(page_size=4), -1), (dict(page_size=24), -1), (dict(page_size=7, max_pages=1), -1),
    (dict(page_size=20, max_pages=1, **Q8), -1), (dict(page_size=1 << 20, max_pages=1 << 12), -4),
    (dict(scale=0.0), -1), (dict(scale=float("nan")), -1), (dict(scale=-1.0), -1), (dict(window=-1), -1),
    (dict(sinks=-1), -1), (dict(max_new=-1), -1), (dict(max_len=-1), -1),
    (dict(n_pages=1 << 30), -4), (dict(n_tokens=1 << 28), -4), (dict(batch=(1 << 20) + 1), -4), (dict(q_stride=504), -1),
    (dict(q_stride=516), -1), (dict(out_stride=508), -1), (dict(q=FAKE + 8), -1), (dict(out=FAR + 8), -1),
    (dict(k_pages=2 * FAKE + 8), -1), (dict(v_pages=3 * FAKE + 2), -1),
    (dict(cache_dtype=2, k_scales=5 * FAKE + 8, v_scales=6 * FAKE), -1), (dict(workspace=FAKE + 4), -1),
    (dict(workspace_bytes=-1), -1), (dict(wait_ns=-1), -1), (dict(out=FAKE), -1), (dict(out=FAKE + 40960 - 1024), -1),
    (dict(out=2 * FAKE + 16), -1), (dict(out=3 * FAKE), -1), (dict(out=5 * FAKE, **Q8), -1),
])
def test_paged_attention_refuses(lib, bad, code):
    assert lib.mk_paged_attention_workspace(ctypes.byref(paged_args(**bad))) == code
    assert lib.mk_paged_attention(ctypes.byref(paged_args(**bad)), None) == code
    assert b"mk_paged_attention" in lib.mk_last_error()


def test_paged_attention_of_nothing_does_nothing(lib):
    for kw in (dict(n_tokens=0), dict(batch=0)):
        assert lib.mk_paged_attention(ctypes.byref(paged_args(**kw)), None) == 0
        assert lib.mk_paged_attention_workspace(ctypes.byref(paged_args(**kw))) == 0
    assert lib.mk_paged_attention(None, None) == -1


def rope_args(**kw):
    a = dict(n=4, n_heads=4, n_kv_heads=2, head_dim=64, rot=64, interleaved=0, dtype=0, slots=3, max_seq=16, eps=1e-5,
             mscale=1.0, qkv_stride=512, q_stride=256, qkv=FAKE, q_out=2 * FAKE, k_cache=3 * FAKE, v_cache=4 * FAKE,
             positions=FAR, rows=FAR, slot_of=None, inv_freq=FAR, q_norm=None, k_norm=None)
    a.update(kw)
    return _lib.mk_rope_args(**a)


@pytest.mark.parametrize("bad,scales", [
    (dict(), (None, FAR)), (dict(), (FAR, None)), (dict(qkv=None), (FAR, 2 * FAR)), (dict(k_cache=3 * FAKE + 8), (FAR, 2 * FAR)),
    (dict(rot=66), (FAR, 2 * FAR)), (dict(), (FAR, FAR + 64)), (dict(), (3 * FAKE + 100, FAR)), (dict(), (FAR, FAKE + 8)),
    (dict(v_cache=3 * FAKE + 64 * 16 * 2), (FAR, 2 * FAR)), (dict(q_out=4 * FAKE), (FAR, 2 * FAR)),
])
def test_rope_append_e4m3_refuses(lib, bad, scales):
    assert lib.mk_rope_append_e4m3(ctypes.byref(rope_args(**bad)), *scales, None) == -1
    assert b"mk_rope_append_e4m3" in lib.mk_last_error()


def test_rope_append_e4m3_of_no_tokens_does_nothing(lib):
    assert lib.mk_rope_append_e4m3(ctypes.byref(rope_args(n=0)), FAR, 2 * FAR, None) == 0


def pages_args(**kw):
    a = dict(n_layers=2, slots=3, n_kv_heads=2, max_seq=100, head_dim=64, n_pages=20, page_size=16, cache_dtype=1, batch=2,
             max_pages=7, k=FAKE, v=2 * FAKE, k_pages=3 * FAKE, v_pages=4 * FAKE, k_scales=None, v_scales=None, table=FAR,
             lengths=FAR, first=None, slot_of=None)
    a.update(kw)
    return _lib.mk_pages_args(**a)


@pytest.mark.parametrize("bad,code", [
    (dict(k=None), -1), (dict(v=None), -1), (dict(k_pages=None), -1), (dict(v_pages=None), -1), (dict(table=None), -1),
    (dict(lengths=None), -1), (dict(cache_dtype=0), -1), (dict(cache_dtype=2), -1), (dict(k_scales=FAR), -1),
    (dict(head_dim=32), -4), (dict(n_layers=0), -1), (dict(slots=0), -1), (dict(n_kv_heads=0), -1), (dict(max_seq=0), -1),
    (dict(n_pages=0), -1), (dict(batch=-1), -1), (dict(max_pages=0), -1), (dict(page_size=12), -1), (dict(page_size=4), -1),
    (dict(k=FAKE + 8), -1), (dict(v_pages=4 * FAKE + 4), -1), (dict(n_layers=40000), -4), (dict(batch=65536), -4),
    (dict(v=FAKE + 64), -1), (dict(k_pages=2 * FAKE), -1), (dict(cache_dtype=2, k_scales=FAKE, v_scales=FAR), -1),
    (dict(cache_dtype=2, k_scales=FAR, v_scales=FAR + 32), -1),
])
def test_moves_refuse(lib, bad, code):
    for name in ("mk_kv_write_pages", "mk_kv_read_pages"):
        assert getattr(lib, name)(ctypes.byref(pages_args(**bad)), None) == code
        assert name.encode() in lib.mk_last_error()


def test_moves_of_no_sequence_do_nothing(lib):
    for name in ("mk_kv_write_pages", "mk_kv_read_pages"):
        assert getattr(lib, name)(ctypes.byref(pages_args(batch=0)), None) == 0


# ---------------------------------------------------------------- the binding
def _cpu_call(**kw):
    bf, i32 = torch.bfloat16, torch.int32
    a = dict(q=torch.zeros(4, 4, 64, dtype=bf), k_pages=torch.zeros(3, 2, 16, 64, dtype=bf),
             v_pages=torch.zeros(3, 2, 16, 64, dtype=bf), table=torch.zeros(2, 2, dtype=i32), starts=torch.zeros(3, dtype=i32),
             lengths=torch.zeros(2, dtype=i32), out=torch.zeros(4, 4, 64, dtype=bf))
    a.update(kw)
    _lib.paged_attention(**a)


@pytest.mark.parametrize("kw,word", [
    (dict(), "CUDA"), (dict(q=torch.zeros(4, 4, 64, dtype=torch.float16)), "q must be"), (dict(q=torch.zeros(4, 256)), "3 dim"),
    (dict(out=torch.zeros(4, 4, 64)), "out"), (dict(k_pages=torch.zeros(3, 2, 16, 64)), "k_pages"),
    (dict(v_pages=torch.zeros(3, 2, 8, 64, dtype=torch.bfloat16)), "v_pages"), (dict(lengths=torch.zeros(3, dtype=torch.int32)), "lengths"),
    (dict(starts=torch.zeros(2, dtype=torch.int32)), "starts"), (dict(table=torch.zeros(2, 2)), "table"),
    (dict(k_scales=torch.zeros(3, 2, 16, 2, dtype=torch.uint8)), "scales"), (dict(window=-1), "window"),
    (dict(k_pages=torch.zeros(3, 2, 16, 64).to(torch.float8_e4m3fn), v_pages=torch.zeros(3, 2, 16, 64).to(torch.float8_e4m3fn)),
     "k_scales"),
])
def test_the_binding_says_what_is_wrong(lib, kw, word):
    with pytest.raises(_lib.MKError, match=word):
        _cpu_call(**kw)


def test_the_moves_binding_says_what_is_wrong(lib):
    bf, i32 = torch.bfloat16, torch.int32
    k = torch.zeros(2, 1, 2, 30, 64, dtype=bf)
    p = torch.zeros(2, 3, 2, 16, 64, dtype=bf)
    t, n = torch.zeros(1, 2, dtype=i32), torch.zeros(1, dtype=i32)
    for fn, args in ((_lib.kv_write_pages, (k, k, p, p)), (_lib.kv_read_pages, (p, p, k, k))):
        with pytest.raises(_lib.MKError, match="CUDA"):
            fn(*args, t, n)
        with pytest.raises(_lib.MKError, match="lengths"):
            fn(*args, t, t)
        with pytest.raises(_lib.MKError, match="sequences"):
            fn(*args, torch.zeros(2, 2, dtype=i32), torch.zeros(2, dtype=i32))
    with pytest.raises(_lib.MKError, match="float8"):
        _lib.rope_append_e4m3(torch.zeros(1, 256), torch.zeros(1, 2, 64), p[0], p[0], p[0], p[0], n, n, torch.zeros(32))


# ---------------------------------------------------------------- the plain forms
def test_the_plain_quantiser_is_the_format():
    """Against the definition, value by value: the nearest of all codes under the smallest power that holds the block."""
    g = torch.Generator().manual_seed(0)
    x = (torch.randn(40, 64, generator=g) * torch.exp2(torch.randint(-120, 16, (40, 1), generator=g).float())).double()
    x[0], x[1, :32] = 0.0, 448.0
    codes, s = ref.quantise(x)
    table = ref.code_values()[:127]
    for r in range(40):
        for b in range(2):
            y = x[r, 32 * b:32 * b + 32]
            fits = [e for e in range(-100, 8) if float(y.abs().max()) <= 448.0 * 2.0 ** e]
            e = fits[0] if fits else 7
            assert int(s[r, b]) == e + 127
            v = ref.values(codes, s)[r, 32 * b:32 * b + 32]
            step = (table[None] * 2.0 ** e - y.abs().clamp(max=448.0 * 2.0 ** e)[:, None]).abs().amin(1)
            assert torch.equal((v.abs() - y.abs().clamp(max=448.0 * 2.0 ** e)).abs(), step)
    assert torch.equal(ref.values(codes, s), ref.values(codes, s).bfloat16().double())


def test_the_plain_attention_is_a_softmax():
    """One page, one head: the textbook formula, with a window and first tokens."""
    g = torch.Generator().manual_seed(1)
    q, k, v = torch.randn(3, 1, 64, generator=g), torch.randn(1, 1, 16, 64, generator=g).double(), torch.randn(1, 1, 16, 64, generator=g).double()
    out, tol = ref.attention(q, k, v, torch.tensor([[0]]), [0, 3], [12], 0.125, 4, 2)
    for i, pos in enumerate((9, 10, 11)):
        rows = [0, 1] + list(range(pos - 3, pos + 1))
        p = torch.softmax(0.125 * k[0, 0, rows] @ q[i, 0].double(), 0)
        assert torch.allclose(out[i, 0], p @ v[0, 0, rows], rtol=0, atol=1e-14)
    # (the bound: 2 A d with A = sum p|v| near 2, d = 0.125 sum|q k| 192 u near 6e-5, and A 80 * 2^-23)
    assert bool((tol > 0).all()) and float(tol.max()) < 1e-3
