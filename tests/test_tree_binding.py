"""The drafted-tree operators' binding and library on the host: refusals and
loading beside those of test_tree_ops.py."""
import ctypes
import os
import subprocess
import sys
import textwrap

import pytest

from decode_megakernel_llama_gb300 import _lib
from decode_megakernel_llama_gb300.build import build
from test_tree_ops import tree_args

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    build()
    return _lib.load()


def test_a_negative_limit_of_waits_is_refused(lib):
    a = tree_args(wait_ns=-1)
    assert lib.mk_tree_attention(ctypes.byref(a), None) == _lib.MK_ERR_INVALID_ARG
    assert b"wait_ns" in lib.mk_last_error()


def test_the_binding_has_the_headers_numbers():
    text = open(_lib.HEADER).read()
    for name in ("MK_MAX_TREE", "MK_F32", "MK_BF16"):
        assert f"#define {name} {getattr(_lib, name)}" in text, name


def run_fresh(code):
    """Code in an interpreter of its own, from the repository's root; what it printed."""
    r = subprocess.run([sys.executable, "-c", textwrap.dedent(code)], cwd=ROOT, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-3000:]
    return r.stdout.split()


def test_the_library_loads_without_torch_and_without_the_extension(lib):
    out = run_fresh("""
        import sys
        sys.modules["torch"] = None  # (an import of it fails)
        from decode_megakernel_llama_gb300 import _lib, build
        for _ in range(2):
            assert _lib.load().mk_plan_inspect is not None
        print(build.build() == build.LIB, sys.modules["torch"])
        for _ in range(2):
            try:
                _lib.kv_reorder(None, None, None, None)
            except ImportError:
                print("refused")
    """)
    assert out == ["True", "None", "refused", "refused"]
    out = run_fresh("""
        from decode_megakernel_llama_gb300 import _lib, build
        build.extension_path = lambda: "/nowhere/mk_torch.so"
        assert _lib.load().mk_plan_inspect is not None
        import torch
        x = torch.zeros(1, 1, 1, 4, 64, dtype=torch.bfloat16)
        i = torch.zeros(1, dtype=torch.int32)
        for _ in range(2):
            try:
                _lib.kv_reorder(x, x, i, i)
            except ImportError as e:
                print("/nowhere" in str(e))
        print(_lib._quick, _lib.rope_frequencies(64, 1e4)[1])
    """)
    assert out == ["True", "True", "None", "1.0"]


def test_threads_that_load_at_once(lib):
    """Sixteen first calls while the module is being loaded: each is answered as a call of CPU tensors is."""
    out = run_fresh("""
        import importlib.util, threading, time
        import torch
        from decode_megakernel_llama_gb300 import _lib
        made = importlib.util.module_from_spec
        def slow(spec):
            time.sleep(0.3)
            return made(spec)
        importlib.util.module_from_spec = slow
        x = torch.zeros(1, 1, 1, 4, 64, dtype=torch.bfloat16)
        i = torch.zeros(1, dtype=torch.int32)
        gate, seen = threading.Barrier(16), []
        def first():
            gate.wait()
            try:
                _lib.kv_reorder(x, x, i, i)
            except Exception as e:
                seen.append(type(e).__name__ + ("CUDA" in str(e)) * "!")
        threads = [threading.Thread(target=first) for _ in range(16)]
        [t.start() for t in threads], [t.join() for t in threads]
        print(*seen)
    """)
    assert out == ["MKError!"] * 16


def test_the_extension_belongs_to_one_torch_and_python(lib, monkeypatch):
    import torch

    from decode_megakernel_llama_gb300 import build as mkbuild
    here = mkbuild.extension_path()
    assert os.path.exists(here) and not mkbuild._stale(here, [mkbuild.TORCH_SOURCE])
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    other = mkbuild.extension_path()
    assert other != here and mkbuild._stale(other, [mkbuild.TORCH_SOURCE])
    monkeypatch.undo()
    assert mkbuild.extension_path() == here


def test_an_extension_that_does_not_compile_leaves_the_library(lib, monkeypatch, tmp_path):
    """The library is there (and up to date) before the failure is raised, and no half-made file beside it."""
    from decode_megakernel_llama_gb300 import build as mkbuild
    done = []
    monkeypatch.setattr(mkbuild, "extension_path", lambda: str(tmp_path / "x.so"))
    monkeypatch.setattr(mkbuild, "torch_command", lambda out: ["false"])
    monkeypatch.setattr(mkbuild, "_build_lib", lambda *a: done.append(a))
    monkeypatch.setattr(mkbuild, "LIB", str(tmp_path / "libmk.so"))
    with pytest.raises(RuntimeError, match="compile failed"):
        mkbuild.build()
    assert len(done) == 1 and not list(tmp_path.iterdir())


K, V, X, Q = (1 << n for n in (30, 31, 32, 33))  # aligned addresses far from one another, that nothing may follow


@pytest.mark.parametrize("bad", [
    dict(v_cache=K), dict(v_cache=K + 2 * 16 * 2 * 64 - 16), dict(k_cache=V + 1024), dict(q_out=K + 64), dict(q_out=V - 16),
    dict(qkv=K), dict(k_cache=X + 3 * 2048), dict(q_out=X, q_stride=256), dict(q_out=X + 16, q_stride=512),
    dict(q_out=X + 2048, q_stride=512), dict(q_out=X - 2048, q_stride=512), dict(q_out=X + 2048 - 16, q_stride=512),
    dict(q_out=X + 2048, qkv_stride=800, q_stride=804), dict(q_out=X + 2048, qkv_stride=764, q_stride=764),
    dict(q_out=X + 2032, qkv_stride=800, q_stride=800), dict(q_out=X - 1008, qkv_stride=800, q_stride=800),
    dict(n=1, q_out=X + 16), dict(n=1, q_out=X - 16),
])
def test_rope_append_refuses_what_overlaps(lib, bad):
    """Four tokens of 4 + 2 + 2 heads of 64 in fp32: rows of qkv of 2,048 bytes, of q_out of 1,024."""
    from test_tree_ops import rope_args
    a = rope_args(**{**dict(k_cache=K, v_cache=V, qkv=X, q_out=Q), **bad})
    assert lib.mk_rope_append(ctypes.byref(a), None) == _lib.MK_ERR_INVALID_ARG
    assert b"overlap" in lib.mk_last_error()


def test_cache_moves_refuse_caches_that_overlap(lib):
    size = 2 * 2 * 2 * 2 * 64 * 64  # bytes of [2][2][2][64][64]
    for v in (K, K + 16, K + size - 16, K - size + 16):
        assert lib.mk_kv_compact(K, v, 2, 2, 2, 64, 64, 8, X, X, X, None) == _lib.MK_ERR_INVALID_ARG
        assert b"overlap" in lib.mk_last_error()
        assert lib.mk_kv_reorder(K, v, 2, 2, 2, 64, 64, X, X, None) == _lib.MK_ERR_INVALID_ARG
        assert b"overlap" in lib.mk_last_error()


def test_heads_of_no_elements_are_refused():
    import torch
    q, k = torch.zeros(1, 1, 2, 0), torch.zeros(1, 1, 8, 0, dtype=torch.bfloat16)
    n, m = torch.zeros(1, dtype=torch.int32), torch.zeros(1, 1, dtype=torch.int64)
    with pytest.raises(_lib.MKError):
        _lib.tree_attention(q, k, k.clone(), n, m, q.clone())
