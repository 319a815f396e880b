"""Host side of the drafted-tree operators: refusals (the argument checks come
before any CUDA call), the frequencies of scaled contexts against their closed
forms, and the walk that accepts a path."""
import ctypes
import math

import numpy as np
import pytest

from decode_megakernel_llama_gb300 import _lib
from decode_megakernel_llama_gb300.build import build

FAKE = 1 << 20  # an aligned address that nothing may follow


@pytest.fixture(scope="module")
def lib():
    build()
    return _lib.load()


def rope_args(**kw):
    a = dict(n=4, n_heads=4, n_kv_heads=2, head_dim=64, rot=64, interleaved=0, dtype=0, slots=1, max_seq=16, eps=1e-5,
             mscale=1.0, qkv_stride=512, q_stride=256, qkv=FAKE, q_out=FAKE, k_cache=FAKE, v_cache=FAKE, positions=FAKE,
             rows=FAKE, slot_of=None, inv_freq=FAKE, q_norm=None, k_norm=None)
    a.update(kw)
    return _lib.mk_rope_args(**a)


@pytest.mark.parametrize("bad,code", [
    (dict(qkv=None), -1), (dict(q_out=None), -1), (dict(k_cache=None), -1), (dict(v_cache=None), -1),
    (dict(positions=None), -1), (dict(rows=None), -1), (dict(inv_freq=None), -1), (dict(dtype=2), -1),
    (dict(head_dim=96), -4), (dict(n=-1), -1), (dict(n_heads=0), -1), (dict(n_kv_heads=0), -1), (dict(slots=0), -1),
    (dict(max_seq=0), -1), (dict(rot=0), -1), (dict(rot=7), -1), (dict(rot=66), -1), (dict(eps=float("nan")), -1),
    (dict(eps=-1.0), -1), (dict(mscale=float("inf")), -1), (dict(qkv_stride=511), -1), (dict(qkv_stride=514), -1),
    (dict(q_stride=255), -1), (dict(q_stride=258), -1), (dict(qkv=FAKE + 4), -1), (dict(k_cache=FAKE + 4), -1),
    (dict(q_norm=FAKE + 2), -1), (dict(inv_freq=FAKE + 4), -1), (dict(n_heads=2 ** 26), -1),
])
def test_rope_append_refuses(lib, bad, code):
    assert lib.mk_rope_append(ctypes.byref(rope_args(**bad)), None) == code
    assert b"mk_rope_append" in lib.mk_last_error()


def test_rope_append_of_no_tokens_does_nothing(lib):
    assert lib.mk_rope_append(ctypes.byref(rope_args(n=0)), None) == 0
    assert lib.mk_rope_append(None, None) == -1


def tree_args(**kw):
    a = dict(batch=2, nodes=8, n_heads=8, n_kv_heads=2, head_dim=64, dtype=0, slots=2, max_seq=64, max_len=0, scale=0.1,
             q_batch_stride=4096, q_token_stride=512, out_batch_stride=4096, out_token_stride=512, q=FAKE, out=FAKE,
             k_cache=FAKE, v_cache=FAKE, lengths=FAKE, counts=None, slot_of=None, masks=FAKE)
    a.update(kw)
    return _lib.mk_tree_args(**a)


@pytest.mark.parametrize("bad,code", [
    (dict(q=None), -1), (dict(out=None), -1), (dict(k_cache=None), -1), (dict(v_cache=None), -1),
    (dict(lengths=None), -1), (dict(masks=None), -1), (dict(dtype=-1), -1), (dict(head_dim=32), -4),
    (dict(batch=-1), -1), (dict(nodes=0), -1), (dict(nodes=65), -1), (dict(n_heads=7), -4),
    (dict(n_heads=34, q_token_stride=4096, out_token_stride=4096), -4), (dict(n_kv_heads=0), -1), (dict(slots=0), -1),
    (dict(max_seq=0), -1), (dict(max_len=-1), -1), (dict(max_len=65), -1), (dict(scale=0.0), -1),
    (dict(scale=float("nan")), -1), (dict(scale=float("inf")), -1), (dict(q_token_stride=504), -1),
    (dict(q_token_stride=516), -1), (dict(out_token_stride=504), -1), (dict(q_batch_stride=-8), -1),
    (dict(out_batch_stride=4), -1), (dict(q=FAKE + 8), -1), (dict(out=FAKE + 8), -1), (dict(k_cache=FAKE + 2), -1),
    (dict(v_cache=FAKE + 8), -1), (dict(masks=FAKE + 4), -1), (dict(batch=40000), -4),
    (dict(workspace=FAKE + 4), -1), (dict(workspace_bytes=-1), -1), (dict(out_batch_stride=0), -1),
    (dict(out_batch_stride=512 * 7), -1), (dict(out_batch_stride=504, out_token_stride=4096), -1),
])
def test_tree_attention_refuses(lib, bad, code):
    assert lib.mk_tree_attention_workspace(ctypes.byref(tree_args(**bad))) == code
    assert lib.mk_tree_attention(ctypes.byref(tree_args(**bad)), None) == code
    assert b"mk_tree_attention" in lib.mk_last_error()


def test_tree_attention_takes_either_order_of_out(lib):
    """Sequences behind one another or nodes behind one another pass the check of overlap (one kv head too many
    for the next check tells)."""
    for b, t in ((4096, 512), (512, 1024), (512, 2048), (8192, 1024)):
        a = tree_args(out_batch_stride=b, out_token_stride=t, q=FAKE + 8)
        assert lib.mk_tree_attention(ctypes.byref(a), None) == -1
        assert b"aligned" in lib.mk_last_error()


def test_tree_attention_of_no_sequences_does_nothing(lib):
    assert lib.mk_tree_attention(ctypes.byref(tree_args(batch=0)), None) == 0
    assert lib.mk_tree_attention_workspace(ctypes.byref(tree_args(batch=0))) == 0
    assert lib.mk_tree_attention(None, None) == -1 and lib.mk_tree_attention_workspace(None) == -1


def test_packed_records_have_the_structures_layout():
    for packed, cls in ((_lib._ROPE_ARGS, _lib.mk_rope_args), (_lib._TREE_ARGS, _lib.mk_tree_args)):
        assert packed.size == ctypes.sizeof(cls)
        values = list(range(1, 1 + len(cls._fields_)))
        got = cls.from_buffer_copy(packed.pack(*values))
        assert [getattr(got, f) for f, _ in cls._fields_] == values


def test_cache_moves_refuse(lib):
    good = [FAKE, FAKE, 2, 2, 2, 64, 64, 8, FAKE, FAKE, FAKE, None]
    for at, value, code in [(0, None, -1), (1, None, -1), (0, FAKE + 8, -1), (2, 0, -1), (3, 0, -1), (4, 0, -1),
                            (5, 0, -1), (6, 80, -4), (7, 0, -1), (7, 65, -1), (8, None, -1), (9, None, -1),
                            (10, None, -1), (2, 20000, -4), (3, 70000, -4)]:
        a = list(good)
        a[at] = value
        assert lib.mk_kv_compact(*a) == code, (at, value)
        assert b"mk_kv_compact" in lib.mk_last_error()
    good = [FAKE, FAKE, 2, 2, 2, 64, 64, FAKE, FAKE, None]
    for at, value, code in [(0, None, -1), (1, None, -1), (1, FAKE + 8, -1), (2, 0, -1), (3, 0, -1), (3, 65, -4),
                            (6, 96, -4), (7, None, -1), (8, None, -1)]:
        a = list(good)
        a[at] = value
        assert lib.mk_kv_reorder(*a) == code, (at, value)
        assert b"mk_kv_reorder" in lib.mk_last_error()


def test_tree_masks_refuses(lib):
    for a in ([None, None, 1, 4, FAKE, None, None], [FAKE, None, 1, 4, None, None, None],
              [FAKE, None, -1, 4, FAKE, None, None], [FAKE, None, 1, 0, FAKE, None, None],
              [FAKE, None, 1, 65, FAKE, None, None]):
        assert lib.mk_tree_masks(*a) == -1
    assert lib.mk_tree_masks(FAKE, None, 0, 4, FAKE, None, None) == 0


def test_binding_of_an_empty_batch_does_nothing():
    import torch
    empty, m = torch.zeros(0, 5, dtype=torch.int32), torch.zeros(0, 5, dtype=torch.int64)
    _lib.tree_masks(empty, m, depths=empty.clone(), counts=empty[:, 0].contiguous())
    k, q = torch.zeros(2, 2, 32, 64, dtype=torch.bfloat16), torch.zeros(0, 5, 4, 64)
    _lib.tree_attention(q, k, k.clone(), torch.zeros(0, dtype=torch.int32), m, q.clone())


def test_binding_refuses_before_any_launch():
    import torch
    bf, i32 = torch.bfloat16, torch.int32
    k = torch.zeros(2, 2, 32, 64, dtype=bf)
    q = torch.zeros(2, 3, 4, 64)
    ln, m = torch.zeros(2, dtype=i32), torch.zeros(2, 3, dtype=torch.int64)
    ok = dict(q=q, k_cache=k, v_cache=k.clone(), lengths=ln, masks=m, out=torch.empty_like(q))
    for bad in (dict(q=q.half()), dict(q=q[0]), dict(v_cache=k.float()), dict(v_cache=k[:, :1]), dict(lengths=ln.long()),
                dict(lengths=ln[:1]), dict(masks=m[:, :2]), dict(masks=m.int()), dict(out=torch.empty(2, 3, 4, 32)),
                dict(out=torch.empty_like(q).to(bf)), dict(counts=ln[:1]), dict(slots=ln.long()),
                dict(q=torch.zeros(2, 3, 64, 4).transpose(2, 3)), dict(k_cache=k[:1], v_cache=k[:1]),
                dict(lengths=torch.zeros(4, dtype=i32)[::2]), {}):  # {}: all is well but the device
        with pytest.raises(_lib.MKError) as e:
            _lib.tree_attention(**{**ok, **bad})
        assert e.value.code == _lib.MK_ERR_INVALID_ARG
    x, f = torch.zeros(5, 8 * 64), torch.zeros(32, dtype=torch.float64)
    p = torch.zeros(5, dtype=i32)
    ok = dict(qkv=x, q_out=torch.zeros(5, 4, 64), k_cache=k, v_cache=k.clone(), positions=p, rows=p, inv_freq=f)
    for bad in (dict(qkv=x.half()), dict(qkv=x[:, :-1]), dict(q_out=torch.zeros(5, 4, 64, dtype=bf)),
                dict(q_out=torch.zeros(4, 4, 64)), dict(positions=p.long()), dict(rows=p[:4]), dict(slots=p[:4]),
                dict(inv_freq=f.float()), dict(q_norm=torch.zeros(32, dtype=bf)), dict(k_norm=torch.zeros(64)),
                dict(v_cache=k.float()), dict(qkv=torch.zeros(8 * 64, 5).T), {}):
        with pytest.raises(_lib.MKError) as e:
            _lib.rope_append(**{**ok, **bad})
        assert e.value.code == _lib.MK_ERR_INVALID_ARG
    c = torch.zeros(2, 2, 2, 32, 64, dtype=bf)
    z = torch.zeros(2, dtype=i32)
    for call in (lambda: _lib.kv_compact(c, c[:1], z, z[:, None], z), lambda: _lib.kv_compact(c, c, z, z, z),
                 lambda: _lib.kv_compact(c, c, z, z[:, None], z), lambda: _lib.kv_reorder(c, c, z, z[:1]),
                 lambda: _lib.kv_reorder(c[0], c[0], z, z), lambda: _lib.tree_masks(z, m),
                 lambda: _lib.tree_masks(torch.zeros(2, 3, dtype=i32), m[:1])):
        with pytest.raises(_lib.MKError):
            call()


def test_rope_frequencies_closed_forms():
    rot, theta, factor, orig = 64, 5e5, 8.0, 8192.0
    i = np.arange(rot // 2)
    f = theta ** (-2.0 * i / rot)
    close = lambda a, b: np.allclose(np.asarray(a), b, rtol=1e-13, atol=0)  # noqa: E731
    w, m = _lib.rope_frequencies(rot, theta)
    assert close(w, f) and m == 1.0
    w, m = _lib.rope_frequencies(rot, theta, "linear", factor)
    assert close(w, f / factor) and m == 1.0
    w, m = _lib.rope_frequencies(rot, theta, "base", factor)
    # the slowest pair is slowed by the factor itself, the fastest not at all
    assert close(w[-1], f[-1] / factor) and w[0] == 1.0 and m == 1.0
    w, m = _lib.rope_frequencies(rot, theta, "wavelength", factor, orig)
    turns = orig * f / (2 * math.pi)
    assert close(w[turns >= 4], f[turns >= 4]) and close(w[turns <= 1], f[turns <= 1] / factor) and m == 1.0
    mid = (turns > 1) & (turns < 4)
    s = (turns[mid] - 1) / 3
    assert mid.any() and close(w[mid], f[mid] * ((1 - s) / factor + s))
    w, m = _lib.rope_frequencies(rot, theta, "yarn", factor, orig)
    assert abs(m - (0.1 * math.log(factor) + 1)) < 1e-7
    assert close(w[turns > 40], f[turns > 40]) and close(w[turns < 0.7], f[turns < 0.7] / factor)
    assert np.all(np.asarray(w) <= f * (1 + 1e-13)) and np.all(np.asarray(w) >= f / factor * (1 - 1e-13))
    # a factor of one changes nothing, whatever the kind
    for kind in ("linear", "base", "wavelength", "yarn"):
        w, m = _lib.rope_frequencies(rot, theta, kind, 1.0, orig)
        assert close(w, f) and m == 1.0


@pytest.mark.parametrize("a", [dict(rot=0), dict(rot=3), dict(theta=1.0), dict(theta=float("inf")),
                               dict(kind="linear", factor=0.5), dict(kind="base", factor=2.0, rot=2),
                               dict(kind="yarn", factor=2.0, original_len=0.0),
                               dict(kind="wavelength", factor=2.0, low=4.0, high=4.0),
                               dict(kind="yarn", factor=float("nan")), dict(kind="other")])
def test_rope_frequencies_refuses(a):
    with pytest.raises(_lib.MKError):
        _lib.rope_frequencies(**{**dict(rot=64, theta=1e4), **a})


def brute_accept(tokens, parents, draws):
    path = [0]
    while True:
        kids = [i for i in range(path[-1] + 1, len(tokens)) if parents[i] == path[-1] and tokens[i] == draws[path[-1]]]
        if not kids:
            return path
        path.append(kids[0])


def test_tree_accept_walks_to_the_first_matching_child():
    rng = np.random.default_rng(0)
    longest = 0
    for _ in range(500):
        n = int(rng.integers(1, 65))
        parents = [-1] + [int(rng.integers(0, t)) for t in range(1, n)]
        tokens, draws = rng.integers(0, 3, n).tolist(), rng.integers(0, 3, n).tolist()
        got = _lib.tree_accept(tokens, parents, draws)
        assert got == brute_accept(tokens, parents, draws)
        longest = max(longest, len(got))
    assert longest > 3
    assert _lib.tree_accept([7], [-1], [9]) == [0]
    with pytest.raises(_lib.MKError):
        _lib.tree_accept([], [], [])
    with pytest.raises(_lib.MKError):
        _lib.tree_accept([0] * 65, [-1] * 65, [0] * 65)
    with pytest.raises(_lib.MKError):
        _lib.tree_accept([0, 1], [-1], [0, 1])
