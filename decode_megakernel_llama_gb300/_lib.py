"""Thin ctypes binding of libmk.so (include/mk.h): argument marshalling only.

Every step of the decode path runs in the library's CUDA kernels; this module
only turns torch tensors into device pointers and sizes. If the library is
missing it raises instead of falling back to anything else.
"""
from __future__ import annotations

import ctypes
import os
import re
import struct
import threading

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "_build", "libmk.so")
HEADER = os.path.join(os.path.dirname(PKG), "include", "mk.h")

MK_OK = 0
MK_ERR_INVALID_ARG = -1
MK_ERR_CUDA = -2
MK_ERR_LAUNCH = -3
MK_ERR_UNSUPPORTED = -4
MK_ERR_TIMEOUT = -5
MK_ERR_NOMEM = -6
MK_INSTR_WORDS = 16
MK_F32, MK_BF16, MK_E4M3 = 0, 1, 2
MK_MAX_TREE = 64
ROPE_KINDS = {"none": 0, "linear": 1, "base": 2, "wavelength": 3, "yarn": 4}


class MKError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"mk error {code}: {msg}")
        self.code = code


class mk_config(ctypes.Structure):
    _fields_ = [("n_layers", ctypes.c_int32), ("d_model", ctypes.c_int32),
                ("n_heads", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("ffn_dim", ctypes.c_int32),
                ("vocab", ctypes.c_int32), ("max_seq", ctypes.c_int32),
                ("max_batch", ctypes.c_int32), ("attn_splits", ctypes.c_int32),
                ("rms_eps", ctypes.c_float), ("rope_theta", ctypes.c_float)]


class mk_layer_weights(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("attn_norm", "wq", "wk", "wv", "wo", "mlp_norm",
                                               "w_gate", "w_up", "w_down")]


class mk_weights(ctypes.Structure):
    _fields_ = [("embed", ctypes.c_void_p), ("final_norm", ctypes.c_void_p),
                ("layers", ctypes.POINTER(mk_layer_weights))]


class mk_kv_cache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p)]


class mk_rope_args(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int32) for n in ("n", "n_heads", "n_kv_heads", "head_dim", "rot", "interleaved", "dtype",
                                               "slots", "max_seq")]
                + [("eps", ctypes.c_float), ("mscale", ctypes.c_float), ("qkv_stride", ctypes.c_int64),
                   ("q_stride", ctypes.c_int64)]
                + [(n, ctypes.c_void_p) for n in ("qkv", "q_out", "k_cache", "v_cache", "positions", "rows", "slot_of",
                                                  "inv_freq", "q_norm", "k_norm")])


class mk_tree_args(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int32) for n in ("batch", "nodes", "n_heads", "n_kv_heads", "head_dim", "dtype", "slots",
                                               "max_seq", "max_len")]
                + [("scale", ctypes.c_float)]
                + [(n, ctypes.c_int64) for n in ("q_batch_stride", "q_token_stride", "out_batch_stride",
                                                 "out_token_stride")]
                + [(n, ctypes.c_void_p) for n in ("q", "out", "k_cache", "v_cache", "lengths", "counts", "slot_of",
                                                  "masks", "workspace")]
                + [("workspace_bytes", ctypes.c_int64), ("status", ctypes.c_void_p), ("wait_ns", ctypes.c_int64)])


class mk_paged_args(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int32) for n in ("n_tokens", "batch", "max_pages", "n_heads", "n_kv_heads", "head_dim",
                                               "dtype", "cache_dtype", "n_pages", "page_size", "max_new", "max_len",
                                               "window", "sinks")]
                + [("scale", ctypes.c_float), ("q_stride", ctypes.c_int64), ("out_stride", ctypes.c_int64)]
                + [(n, ctypes.c_void_p) for n in ("q", "out", "k_pages", "v_pages", "k_scales", "v_scales", "table",
                                                  "starts", "lengths", "workspace")]
                + [("workspace_bytes", ctypes.c_int64), ("status", ctypes.c_void_p), ("wait_ns", ctypes.c_int64)])


class mk_pages_args(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int32) for n in ("n_layers", "slots", "n_kv_heads", "max_seq", "head_dim", "n_pages",
                                               "page_size", "cache_dtype", "batch", "max_pages")]
                + [(n, ctypes.c_void_p) for n in ("k", "v", "k_pages", "v_pages", "k_scales", "v_scales", "table",
                                                  "lengths", "first", "slot_of")])


# The same as one packed record each (native layout): filling a ctypes
# structure field by field costs more than the launch it is for.
_ROPE_ARGS = struct.Struct("@9i2f2q10P")
_TREE_ARGS = struct.Struct("@9if4q9PqPq")
_PAGED_ARGS = struct.Struct("@14if2q10PqPq")
_PAGES_ARGS = struct.Struct("@10i10P")


_lib = None
_quick = None  # the extension module of the standalone operators (csrc/mk_torch.cpp)
_loading = threading.RLock()
_VP = ctypes.c_void_p
_I32 = ctypes.c_int32
_PI32 = ctypes.POINTER(ctypes.c_int32)


def load(path: str | None = None):
    """Loads libmk.so (built by decode_megakernel_llama_gb300.build). The
    environment variable MK_LIB selects another build of the same library
    (e.g. the address-checked one)."""
    global _lib
    if _lib is None:
        with _loading:
            if _lib is None:
                _lib = _load(path)
    return _lib


def _load(path: str | None):
    path = path or os.environ.get("MK_LIB") or LIB_PATH
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing: run decode_megakernel_llama_gb300.build.build() "
                          "(there is no fallback implementation)")
    L = ctypes.CDLL(path)
    L.mk_last_error.restype = ctypes.c_char_p
    L.mk_create.argtypes = [ctypes.POINTER(mk_config), ctypes.POINTER(mk_weights),
                            ctypes.POINTER(mk_kv_cache), ctypes.POINTER(_VP)]
    L.mk_decode_step.argtypes = [_VP, _I32, _I32, _VP, _VP, _VP]
    L.mk_decode_step_dev.argtypes = [_VP, _VP, _I32, _VP, _VP, _VP]
    L.mk_decode_step_host.argtypes = [_VP, _PI32, _I32, _VP, _PI32, _VP]
    L.mk_decode_step_unfused.argtypes = [_VP, _I32, _I32, _VP, _VP, _VP]
    L.mk_decode_step_batch.argtypes = [_VP, _VP, _VP, _I32, _VP, _VP, _VP]
    L.mk_get_status.argtypes = [_VP]
    L.mk_set_wait_timeout.argtypes = [_VP, ctypes.c_uint64]
    L.mk_set_trace.argtypes = [_VP, _I32]
    L.mk_set_sampling.argtypes = [_VP, ctypes.c_float, ctypes.c_uint64]
    L.mk_read_trace.argtypes = [_VP, ctypes.POINTER(ctypes.c_int64), _I32]
    L.mk_plan_size.argtypes = [_VP, _PI32, _PI32]
    L.mk_plan_inspect.argtypes = [ctypes.POINTER(mk_config), _I32, _PI32, _I32, _PI32, _PI32]
    L.mk_debug_read.argtypes = [_VP, ctypes.POINTER(ctypes.c_uint64)]
    L.mk_decode_step_noalloc.argtypes = [ctypes.POINTER(mk_config), ctypes.POINTER(mk_weights),
                                         ctypes.POINTER(mk_kv_cache), _I32, _I32, _VP, _VP, _VP]
    L.mk_set_sampling_filter.argtypes = [_VP, _I32, ctypes.c_float]
    L.mk_sampling_noise.argtypes = [_I32, _I32, _I32, ctypes.c_uint64, _VP, _VP, _VP, _VP]
    L.mk_draw_from_logits.argtypes = [_VP, _I32, _I32, ctypes.c_float, _I32, ctypes.c_float, _VP, ctypes.c_uint64,
                                      _VP, _VP]
    L.mk_w2_pack.argtypes = [_VP, ctypes.c_int64, ctypes.c_int64, _VP]
    L.mk_w2_unpack.argtypes = [_VP, ctypes.c_int64, ctypes.c_int64, _VP]
    L.mk_w2a8_gemv.argtypes = [_VP, ctypes.c_float, _I32, _I32, _VP, _VP, _VP]
    L.mk_twell_down.argtypes = [_VP, _I32, _I32, _VP, _VP, _VP]
    L.mk_twell_ffn.argtypes = [_VP, _VP, _VP, _I32, _I32, _VP, _VP, _VP, _VP]
    L.mk_prefill.argtypes = [_VP, _VP, _I32, _I32, _VP, _VP, _VP]
    L.mk_verify.argtypes = [_VP, _VP, _VP, _I32, _I32, _VP, _VP, _VP]
    L.mk_tc_gemm.argtypes = [_VP, _I32, _I32, _VP, _VP, _I32, _VP, _VP, _VP, _VP]
    L.mk_rope_append.argtypes = [_VP, _VP]  # a packed record, or byref of the structure
    L.mk_rope_frequencies.argtypes = [_I32, _I32] + [ctypes.c_double] * 5 + [_VP, ctypes.POINTER(ctypes.c_float)]
    L.mk_tree_attention.argtypes = [_VP, _VP]
    L.mk_tree_attention_workspace.argtypes = [_VP]
    L.mk_tree_attention_workspace.restype = ctypes.c_int64
    L.mk_tree_masks.argtypes = [_VP, _VP, _I32, _I32, _VP, _VP, _VP]
    L.mk_tree_accept.argtypes = [_VP, _VP, _VP, _I32, _VP]
    L.mk_kv_compact.argtypes = [_VP, _VP] + [_I32] * 6 + [_VP] * 4
    L.mk_kv_reorder.argtypes = [_VP, _VP] + [_I32] * 5 + [_VP] * 3
    L.mk_paged_attention.argtypes = [_VP, _VP]
    L.mk_paged_attention_workspace.argtypes = [_VP]
    L.mk_paged_attention_workspace.restype = ctypes.c_int64
    L.mk_rope_append_e4m3.argtypes = [_VP] * 4
    L.mk_kv_write_pages.argtypes = [_VP, _VP]
    L.mk_kv_read_pages.argtypes = [_VP, _VP]
    L.mk_destroy.argtypes = [_VP]
    L.mk_destroy.restype = None
    return L


def load_extension():
    """Loads the extension module of the drafted-tree operators (rope_append, tree_attention, kv_compact, kv_reorder)
    and of those of pages (paged_attention, rope_append_e4m3, kv_write_pages, kv_read_pages), which their first call
    does otherwise, and gives it the library's entry points. Nothing else needs it."""
    global _quick
    with _loading:
        if _quick is None:
            import importlib.util

            from .build import extension_path
            L, path = load(), extension_path()  # (imports torch, whose libraries the module needs)
            if not os.path.exists(path):
                raise ImportError(f"{path} is missing: run decode_megakernel_llama_gb300.build.build()")
            spec = importlib.util.spec_from_file_location("mk_torch", path)
            mod = importlib.util.module_from_spec(spec)
            spec.loader.exec_module(mod)
            mod.bind(*(ctypes.cast(f, ctypes.c_void_p).value for f in (
                L.mk_rope_append, L.mk_tree_attention, L.mk_tree_attention_workspace, L.mk_kv_compact,
                L.mk_kv_reorder, L.mk_paged_attention, L.mk_paged_attention_workspace, L.mk_rope_append_e4m3,
                L.mk_kv_write_pages, L.mk_kv_read_pages)))
            _quick = mod
    return _quick


def declared_symbols(header: str = HEADER) -> list[str]:
    """Function names declared in include/mk.h."""
    text = open(header).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(mk_[a-z_0-9]+)\s*\(", text)))


def check(rc: int) -> int:
    if rc < 0:
        raise MKError(rc, load().mk_last_error().decode())
    return rc


def make_config(shape, max_seq: int, max_batch: int = 1, attn_splits: int = 0) -> mk_config:
    return mk_config(shape.n_layers, shape.d_model, shape.n_heads, shape.n_kv_heads,
                     shape.head_dim, shape.ffn_dim, shape.vocab, int(max_seq), int(max_batch),
                     int(attn_splits), float(shape.rms_eps), float(shape.rope_theta))


def plan_inspect(shape, n_sm: int, max_seq: int, attn_splits: int = 0, max_batch: int = 1):
    """Host-only plan: returns (instr int32 [n, 16] as list of lists, queue lengths, n_counters).
    max_batch > 1 gives the fused batched step's plan where the model supports it."""
    import numpy as np
    L = load()
    cfg = make_config(shape, max_seq, max_batch, attn_splits)
    qlen = (ctypes.c_int32 * n_sm)()
    nctr = ctypes.c_int32(0)
    n = check(L.mk_plan_inspect(ctypes.byref(cfg), n_sm, None, 0, qlen, ctypes.byref(nctr)))
    buf = np.zeros((n, MK_INSTR_WORDS), dtype=np.int32)
    check(L.mk_plan_inspect(ctypes.byref(cfg), n_sm,
                            buf.ctypes.data_as(_PI32), n, qlen, ctypes.byref(nctr)))
    return buf, np.array(list(qlen), dtype=np.int64), int(nctr.value)


def _stream_ptr(stream) -> int:
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream)


def _weights_struct(shape, weights: dict):
    layers = (mk_layer_weights * shape.n_layers)()
    for i, lw in enumerate(weights["layers"]):
        for k in ("attn_norm", "wq", "wk", "wv", "wo", "mlp_norm", "w_gate", "w_up", "w_down"):
            setattr(layers[i], k, lw[k].data_ptr())
    w = mk_weights(weights["embed"].data_ptr(), weights["final_norm"].data_ptr(),
                   ctypes.cast(layers, ctypes.POINTER(mk_layer_weights)))
    return w, layers


def decode_step_noalloc(shape, weights: dict, k_cache, v_cache, token: int, pos: int, out_token,
                        logits=None, attn_splits: int = 0, stream=None) -> None:
    """mk_decode_step_noalloc: one decode step without a handle and without
    any device allocation (scratch lives in the library's static array)."""
    cfg = make_config(shape, int(k_cache.shape[3]), int(k_cache.shape[1]), attn_splits)
    w, layers = _weights_struct(shape, weights)
    kv = mk_kv_cache(k_cache.data_ptr(), v_cache.data_ptr())
    check(load().mk_decode_step_noalloc(ctypes.byref(cfg), ctypes.byref(w), ctypes.byref(kv),
                                        int(token), int(pos),
                                        logits.data_ptr() if logits is not None else None,
                                        out_token.data_ptr(), _stream_ptr(stream)))


def sampling_noise(n: int, position: int, slot: int, seed: int, out_words=None, out_noise=None,
                   words=None, stream=None) -> None:
    """mk_sampling_noise: the sampling epilogue's Philox words and Gumbel noise for
    vocabulary entries 0..n-1 (int32/uint32 and float32 CUDA tensors [n]); with
    `words` given, the noise of those words instead."""
    ptr = lambda t: t.data_ptr() if t is not None else None
    check(load().mk_sampling_noise(int(n), int(position), int(slot), int(seed) & ((1 << 64) - 1),
                                   ptr(words), ptr(out_words), ptr(out_noise), _stream_ptr(stream)))


def draw_from_logits(logits, temperature: float, top_k: int, top_p: float, positions, seed: int, out_tokens,
                     stream=None) -> None:
    """mk_draw_from_logits: logits float32 CUDA tensor [B][V]; positions and
    out_tokens int32 CUDA tensors [B]; sequence b draws on slot b's noise."""
    B, V = int(logits.shape[0]), int(logits.shape[1])
    check(load().mk_draw_from_logits(logits.data_ptr(), B, V, float(temperature), int(top_k), float(top_p),
                                     positions.data_ptr(), int(seed) & ((1 << 64) - 1), out_tokens.data_ptr(),
                                     _stream_ptr(stream)))


def w2_pack(q):
    """Host: ternary int8 codes [rows][cols] (numpy) -> packed uint32 [rows][cols / 16]
    in the library's W2 layout (mk_w2_pack)."""
    import numpy as np
    q = np.ascontiguousarray(q, dtype=np.int8)
    rows, cols = q.shape
    out = np.empty((rows, cols // 16), dtype=np.uint32)
    check(load().mk_w2_pack(q.ctypes.data, rows, cols, out.ctypes.data))
    return out


def w2_unpack(packed, cols: int):
    """Host: the inverse of w2_pack (mk_w2_unpack)."""
    import numpy as np
    packed = np.ascontiguousarray(packed, dtype=np.uint32)
    rows = packed.shape[0]
    out = np.empty((rows, cols), dtype=np.int8)
    check(load().mk_w2_unpack(packed.ctypes.data, rows, cols, out.ctypes.data))
    return out


def w2a8_gemv(packed, beta: float, rows: int, cols: int, x, y, stream=None) -> None:
    """mk_w2a8_gemv on CUDA tensors: packed (uint32/int32 [rows][cols/16]),
    x float32 [cols], y float32 [rows]."""
    check(load().mk_w2a8_gemv(packed.data_ptr(), float(beta), int(rows), int(cols), x.data_ptr(),
                              y.data_ptr(), _stream_ptr(stream)))


def twell_down(w_down_t, h, y, stream=None) -> None:
    """mk_twell_down on CUDA tensors: w_down_t bf16 [F][d], h float32 [F],
    y float32 [d] = W_down h over the non-zero entries of h."""
    F, d = w_down_t.shape
    rc = load().mk_twell_down(w_down_t.data_ptr(), int(F), int(d), h.data_ptr(), y.data_ptr(), _stream_ptr(stream))
    if rc != 0:
        raise MKError(rc, f"mk_twell_down returned {rc}")


def twell_ffn(w_gate, w_up, w_down_t, x, h, y, stream=None) -> None:
    """mk_twell_ffn on CUDA tensors: w_gate / w_up bf16 [F][d], w_down_t bf16
    [F][d], x float32 [d]; writes h float32 [F] = relu(W_gate x) * (W_up x) and
    y float32 [d] = W_down h."""
    F, d = w_gate.shape
    rc = load().mk_twell_ffn(w_gate.data_ptr(), w_up.data_ptr(), w_down_t.data_ptr(), int(F), int(d),
                             x.data_ptr(), h.data_ptr(), y.data_ptr(), _stream_ptr(stream))
    if rc != 0:
        raise MKError(rc, f"mk_twell_ffn returned {rc}")


def tc_gemm(w, bhi, blo, y, r=None, status=None, stream=None) -> None:
    """mk_tc_gemm on CUDA tensors: w bf16 [M][K], bhi / blo bf16 [N][K], y (and r)
    float32 [N][M]; y = W (bhi + blo)^T (+ r). status: int32 CUDA tensor [1]
    (zeroed by the caller) that turns non-zero if an in-kernel wait expires;
    without it, the call synchronises and raises on expiry."""
    import torch
    M, K = w.shape
    N = bhi.shape[0]
    st = status if status is not None else torch.zeros(1, dtype=torch.int32, device=y.device)
    rc = load().mk_tc_gemm(w.data_ptr(), int(M), int(K), bhi.data_ptr(), blo.data_ptr(), int(N), y.data_ptr(),
                           r.data_ptr() if r is not None else None, st.data_ptr(), _stream_ptr(stream))
    if rc != 0:
        raise MKError(rc, f"mk_tc_gemm returned {rc}")
    if status is None and int(st.item()) != 0:
        raise MKError(MK_ERR_TIMEOUT, "a bounded wait of the tensor-core contraction expired")


def _bad(msg: str):
    raise MKError(MK_ERR_INVALID_ARG, msg)


def _need(t, what: str, dtype, shape, like, dense: bool = True) -> None:
    """Raises unless tensor t has this type, shape (a tuple) and layout and is on the device of `like`."""
    if t.dtype != dtype:
        _bad(f"{what} must be {dtype}, not {t.dtype}")
    if t.shape != shape:
        _bad(f"{what} has shape {tuple(t.shape)}, not {tuple(shape)}")
    if t.device != like.device:
        _bad(f"{what} is on {t.device}, not {like.device}")
    if dense and not t.is_contiguous():
        _bad(f"{what} must be contiguous")


def _run_on(torch, d: int, stream, fn, *args) -> None:
    """fn(*args, stream pointer) with CUDA device d current; without a stream, on that device's current one."""
    if d < 0:
        _bad("tensors must be on a CUDA device")
    if d == torch._C._cuda_getDevice():
        rc = fn(*args, torch._C._cuda_getCurrentRawStream(d) if stream is None else stream.cuda_stream)
    else:
        with torch.cuda.device(d):
            rc = fn(*args, torch._C._cuda_getCurrentRawStream(d) if stream is None else stream.cuda_stream)
    if rc < 0:
        check(rc)


def _io_dtype(torch, t, what: str) -> int:
    if t.dtype is torch.float32:
        return MK_F32
    if t.dtype is torch.bfloat16:
        return MK_BF16
    _bad(f"{what} must be float32 or bfloat16, not {t.dtype}")


def rope_frequencies(rot: int, theta: float, kind: str = "none", factor: float = 1.0, original_len: float = 8192.0,
                     low: float = 1.0, high: float | None = None):
    """mk_rope_frequencies: (float64 CPU tensor [rot / 2] of radians per position, factor on the rotated
    values). kind: "none", "linear", "base", "wavelength" (high defaults to 4) or "yarn" (32)."""
    import torch
    if kind not in ROPE_KINDS:
        _bad(f"kind must be one of {sorted(ROPE_KINDS)}, not {kind!r}")
    if high is None:
        high = 32.0 if kind == "yarn" else 4.0
    out = torch.empty(max(1, int(rot) // 2), dtype=torch.float64)
    m = ctypes.c_float()
    check(load().mk_rope_frequencies(ROPE_KINDS[kind], int(rot), float(theta), float(factor), float(original_len),
                                     float(low), float(high), out.data_ptr(), ctypes.byref(m)))
    return out, m.value


def rope_append(qkv, q_out, k_cache, v_cache, positions, rows, inv_freq, slots=None, q_norm=None, k_norm=None,
                eps: float = 1e-5, mscale: float = 1.0, interleaved: bool = False, stream=None) -> None:
    """mk_rope_append on CUDA tensors: qkv [n][(Hq + 2 Hkv) hd] float32 or bfloat16 (rows may be strided),
    q_out [n][Hq][hd] of the same type (token stride free), k_cache / v_cache bfloat16 [B][Hkv][max_seq][hd]
    (one layer), positions / rows / slots int32 [n], inv_freq float64 [rot / 2], q_norm / k_norm bfloat16 [hd]."""
    q = _quick or load_extension()
    rc = q.rope_append(qkv, q_out, k_cache, v_cache, positions, rows, inv_freq, slots, q_norm, k_norm, eps, mscale,
                       interleaved, stream)
    if rc == MK_OK:
        return
    if rc < 0:
        check(rc)
    # not done: something is wrong, or the call is for another stream or device
    import torch
    bf, i32, dt = torch.bfloat16, torch.int32, _io_dtype(torch, qkv, "qkv")
    if k_cache.dim() != 4 or q_out.dim() != 3 or qkv.dim() != 2 or inv_freq.dim() != 1:
        _bad("qkv, q_out, k_cache, inv_freq must have 2, 3, 4, 1 dimensions")
    B, Hkv, S, hd = k_cache.shape
    n, Hq, _ = q_out.shape
    half, d, per_token = inv_freq.shape[0], qkv.get_device(), (n,)
    if not (qkv.shape == (n, (Hq + 2 * Hkv) * hd) and q_out.shape == (n, Hq, hd) and q_out.dtype is qkv.dtype
            and k_cache.dtype is bf and v_cache.dtype is bf and v_cache.shape == k_cache.shape
            and positions.dtype is i32 and rows.dtype is i32 and positions.shape == per_token
            and rows.shape == per_token and inv_freq.dtype is torch.float64
            and q_out.get_device() == k_cache.get_device() == v_cache.get_device() == positions.get_device()
            == rows.get_device() == inv_freq.get_device() == d and k_cache.is_contiguous()
            and v_cache.is_contiguous() and positions.is_contiguous() and rows.is_contiguous()
            and inv_freq.is_contiguous()):
        for t, what, dtype, shape, dense in (
                (qkv, "qkv", qkv.dtype, (n, (Hq + 2 * Hkv) * hd), False), (q_out, "q_out", qkv.dtype, (n, Hq, hd), False),
                (k_cache, "k_cache", bf, (B, Hkv, S, hd), True), (v_cache, "v_cache", bf, (B, Hkv, S, hd), True),
                (positions, "positions", i32, per_token, True), (rows, "rows", i32, per_token, True),
                (inv_freq, "inv_freq", torch.float64, (half,), True)):
            _need(t, what, dtype, shape, qkv, dense)
    for t, what, dtype, shape in ((slots, "slots", i32, per_token), (q_norm, "q_norm", bf, (hd,)),
                                  (k_norm, "k_norm", bf, (hd,))):
        if t is not None:
            _need(t, what, dtype, shape, qkv)
    if n == 0:
        return
    ts, qs = qkv.stride(), q_out.stride()
    if ts[1] != 1 or qs[2] != 1 or (Hq > 1 and qs[1] != hd):
        _bad("the heads of a token must be contiguous in qkv and q_out")
    width = (Hq + 2 * Hkv) * hd
    rec = _ROPE_ARGS.pack(n, Hq, Hkv, hd, 2 * half, 1 if interleaved else 0, dt, B, S, eps, mscale,
                          ts[0] if n > 1 else width, qs[0] if n > 1 else Hq * hd, qkv.data_ptr(), q_out.data_ptr(),
                          k_cache.data_ptr(), v_cache.data_ptr(), positions.data_ptr(), rows.data_ptr(),
                          0 if slots is None else slots.data_ptr(), inv_freq.data_ptr(),
                          0 if q_norm is None else q_norm.data_ptr(), 0 if k_norm is None else k_norm.data_ptr())
    _run_on(torch, d, stream, load().mk_rope_append, rec)


def tree_attention(q, k_cache, v_cache, lengths, masks, out, scale: float | None = None, counts=None, slots=None,
                   max_len: int = 0, status=None, stream=None, wait_ns: int = 0) -> None:
    """mk_tree_attention on CUDA tensors: q and out [B][T][Hq][hd] float32 or bfloat16 (batch and node strides
    free), k_cache / v_cache bfloat16 [slots][Hkv][max_seq][hd] (one layer), lengths / counts / slots int32 [B],
    masks int64 [B][T] (the 64 bits of the ancestor mask). scale defaults to 1 / sqrt(hd). status: int32 [1]
    (zeroed by the caller) that becomes 1 if a bounded in-kernel wait ran out, after wait_ns nanoseconds (0: 2e9); the
    rows concerned are then NaN. The workspace of long caches comes from torch's allocator, on the call's stream."""
    quick = _quick or load_extension()
    rc = quick.tree_attention(q, k_cache, v_cache, lengths, masks, out, scale, counts, slots, max_len, status, stream,
                              wait_ns)
    if rc == MK_OK:
        return
    if rc < 0:
        check(rc)
    # not done: something is wrong, or the call is for another stream or device
    import torch
    bf, i32, i64, dt = torch.bfloat16, torch.int32, torch.int64, _io_dtype(torch, q, "q")
    if q.dim() != 4 or k_cache.dim() != 4:
        _bad("q and k_cache must have 4 dimensions")
    B, T, Hq, hd = q.shape
    n_slots, Hkv, S, _ = k_cache.shape
    if scale is None:
        scale = max(hd, 1) ** -0.5
    d, per_seq = q.get_device(), (B,)
    if not (out.dtype is q.dtype and out.shape == q.shape and k_cache.dtype is bf and v_cache.dtype is bf
            and k_cache.shape[3] == hd and v_cache.shape == k_cache.shape and lengths.dtype is i32
            and lengths.shape == per_seq and masks.dtype is i64 and masks.shape == (B, T)
            and out.get_device() == k_cache.get_device() == v_cache.get_device() == lengths.get_device()
            == masks.get_device() == d and k_cache.is_contiguous() and v_cache.is_contiguous()
            and lengths.is_contiguous() and masks.is_contiguous()):
        for t, what, dtype, shape, dense in (
                (out, "out", q.dtype, (B, T, Hq, hd), False), (k_cache, "k_cache", bf, (n_slots, Hkv, S, hd), True),
                (v_cache, "v_cache", bf, (n_slots, Hkv, S, hd), True), (lengths, "lengths", i32, per_seq, True),
                (masks, "masks", i64, (B, T), True)):
            _need(t, what, dtype, shape, q, dense)
    for t, what, shape in ((counts, "counts", per_seq), (slots, "slots", per_seq), (status, "status", (1,))):
        if t is not None:
            _need(t, what, i32, shape, q)
    if slots is None and B > n_slots:
        _bad(f"{B} sequences for {n_slots} cache slots")
    if B == 0:
        return
    qs, os = q.stride(), out.stride()
    if qs[3] != 1 or os[3] != 1 or (Hq > 1 and (qs[2] != hd or os[2] != hd)):
        _bad("the heads of a node must be contiguous in q and out")
    row = Hq * hd
    rec = [B, T, Hq, Hkv, hd, dt, n_slots, S, max_len, scale, qs[0] if B > 1 else 0,
           qs[1] if T > 1 else row, os[0] if B > 1 else 0, os[1] if T > 1 else row, q.data_ptr(), out.data_ptr(),
           k_cache.data_ptr(), v_cache.data_ptr(), lengths.data_ptr(), 0 if counts is None else counts.data_ptr(),
           0 if slots is None else slots.data_ptr(), masks.data_ptr(), 0, 0,
           0 if status is None else status.data_ptr(), wait_ns]
    L, work = load(), None
    if d >= 0:
        with torch.cuda.device(d):
            n = L.mk_tree_attention_workspace(_TREE_ARGS.pack(*rec))
            if n < 0:
                check(n)
            if n > 0:
                if stream is None:
                    work = torch.empty(n, dtype=torch.uint8, device=q.device)
                else:
                    with torch.cuda.stream(stream):
                        work = torch.empty(n, dtype=torch.uint8, device=q.device)
                rec[22], rec[23] = work.data_ptr(), n
    _run_on(torch, d, stream, L.mk_tree_attention, _TREE_ARGS.pack(*rec))


def tree_masks(parents, masks, depths=None, counts=None, stream=None) -> None:
    """mk_tree_masks on CUDA tensors: parents int32 [B][T] -> masks int64 [B][T], depths int32 [B][T] or None."""
    import torch
    if parents.dim() != 2:
        _bad("parents must have 2 dimensions")
    B, T = parents.shape
    _need(parents, "parents", torch.int32, (B, T), parents)
    _need(masks, "masks", torch.int64, (B, T), parents)
    if depths is not None:
        _need(depths, "depths", torch.int32, (B, T), parents)
    if counts is not None:
        _need(counts, "counts", torch.int32, (B,), parents)
    if B == 0:
        return
    _run_on(torch, parents.get_device(), stream, load().mk_tree_masks, parents.data_ptr(),
            None if counts is None else counts.data_ptr(), B, T, masks.data_ptr(),
            None if depths is None else depths.data_ptr())


def tree_accept(tokens, parents, draws):
    """mk_tree_accept: the accepted nodes (list, node 0 first) of a verified tree; the three are host sequences of
    n whole numbers. The next token is draws[path[-1]]."""
    n = len(tokens)
    if len(parents) != n or len(draws) != n:
        _bad("tokens, parents and draws must have the same length")
    arr = ctypes.c_int32 * max(1, n)
    path = arr()
    c = check(load().mk_tree_accept(arr(*map(int, tokens)), arr(*map(int, parents)), arr(*map(int, draws)), n, path))
    return list(path[:c])


def _check_caches(torch, k, v, shape, small) -> None:
    """k, v: the whole caches, of `shape`; small: the int32 arrays that go with them, (tensor, name, shape)."""
    d = k.get_device()
    if not (k.dtype is torch.bfloat16 and v.dtype is torch.bfloat16 and v.shape == shape and v.get_device() == d
            and k.is_contiguous() and v.is_contiguous()):
        _need(k, "k", torch.bfloat16, shape, k)
        _need(v, "v", torch.bfloat16, shape, k)
    for t, what, dims in small:
        if not (t.dtype is torch.int32 and t.shape == dims and t.get_device() == d and t.is_contiguous()):
            _need(t, what, torch.int32, dims, k)


def kv_compact(k, v, starts, nodes, counts, stream=None) -> None:
    """mk_kv_compact on CUDA tensors: k / v bfloat16 [L][B][Hkv][max_seq][hd], starts / counts int32 [B], nodes
    int32 [B][n]: rows starts[b] + nodes[b][i] move to starts[b] + i."""
    rc = (_quick or load_extension()).kv_compact(k, v, starts, nodes, counts, stream)
    if rc == MK_OK:
        return
    if rc < 0:
        check(rc)
    import torch
    if k.dim() != 5 or nodes.dim() != 2:
        _bad("the caches must have 5 dimensions, nodes 2")
    shape = k.shape
    L, B, Hkv, S, hd = shape
    n = nodes.shape[1]
    _check_caches(torch, k, v, shape, ((starts, "starts", (B,)), (nodes, "nodes", (B, n)), (counts, "counts", (B,))))
    _run_on(torch, k.get_device(), stream, load().mk_kv_compact, k.data_ptr(), v.data_ptr(), L, B, Hkv, S, hd, n,
            starts.data_ptr(), nodes.data_ptr(), counts.data_ptr())


def kv_reorder(k, v, sources, lengths, stream=None) -> None:
    """mk_kv_reorder on CUDA tensors: k / v bfloat16 [L][B][Hkv][max_seq][hd], sources / lengths int32 [B]: rows
    [0, lengths[b]) of slot b become slot sources[b]'s."""
    rc = (_quick or load_extension()).kv_reorder(k, v, sources, lengths, stream)
    if rc == MK_OK:
        return
    if rc < 0:
        check(rc)
    import torch
    if k.dim() != 5:
        _bad("the caches must have 5 dimensions")
    shape = k.shape
    L, B, Hkv, S, hd = shape
    _check_caches(torch, k, v, shape, ((sources, "sources", (B,)), (lengths, "lengths", (B,))))
    _run_on(torch, k.get_device(), stream, load().mk_kv_reorder, k.data_ptr(), v.data_ptr(), L, B, Hkv, S, hd,
            sources.data_ptr(), lengths.data_ptr())


def _pool(torch, k_pages, v_pages, k_scales, v_scales, lead: int) -> int:
    """Checks a pool of pages ([pages][Hkv][rows][hd] behind `lead` dimensions) and its scales; its type."""
    e4m3 = torch.float8_e4m3fn
    if k_pages.dim() != 4 + lead:
        _bad(f"k_pages must have {4 + lead} dimensions")
    if k_pages.dtype not in (torch.bfloat16, e4m3):
        _bad(f"k_pages must be bfloat16 or float8_e4m3fn, not {k_pages.dtype}")
    q8 = k_pages.dtype is e4m3
    _need(k_pages, "k_pages", k_pages.dtype, k_pages.shape, k_pages)
    _need(v_pages, "v_pages", k_pages.dtype, k_pages.shape, k_pages)
    if (k_scales is not None) != q8 or (v_scales is not None) != q8:
        _bad("float8_e4m3fn pages need k_scales and v_scales, bfloat16 pages none")
    if q8:
        shape = (*k_pages.shape[:-1], k_pages.shape[-1] // 32)
        _need(k_scales, "k_scales", torch.uint8, shape, k_pages)
        _need(v_scales, "v_scales", torch.uint8, shape, k_pages)
    return MK_E4M3 if q8 else MK_BF16


def _at(t) -> int:
    return 0 if t is None else t.data_ptr()


def paged_attention(q, k_pages, v_pages, table, starts, lengths, out, scale: float | None = None, window: int = 0,
                    sinks: int = 0, k_scales=None, v_scales=None, max_new: int = 0, max_len: int = 0, status=None,
                    stream=None, wait_ns: int = 0) -> None:
    """mk_paged_attention on CUDA tensors: q and out [n][Hq][hd] float32 or bfloat16 (token strides free), k_pages /
    v_pages bfloat16 [pages][Hkv][rows][hd] (one layer), or float8_e4m3fn with k_scales / v_scales uint8
    [pages][Hkv][rows][hd / 32]; table int32 [B][pages of a sequence], starts int32 [B + 1] (sequence b has tokens
    starts[b] .. starts[b + 1] - 1 of q), lengths int32 [B] (its rows, the new tokens' own among them). A token sees
    the rows up to its own, with a window the last `window` of them and the first `sinks`. scale defaults to
    1 / sqrt(hd). max_new, max_len: bounds on a sequence's tokens and rows, for the choice of the launch alone.
    status, wait_ns and the workspace: as in tree_attention."""
    rc = (_quick or load_extension()).paged_attention(q, k_pages, v_pages, table, starts, lengths, out, scale, window,
                                                   sinks, k_scales, v_scales, max_new, max_len, status, stream,
                                                   wait_ns)
    if rc == MK_OK:
        return
    if rc < 0:
        check(rc)
    # not done: something is wrong, or the call is for another stream or device
    import torch
    i32, dt = torch.int32, _io_dtype(torch, q, "q")
    if q.dim() != 3 or table.dim() != 2:
        _bad("q must have 3 dimensions, table 2")
    cache = _pool(torch, k_pages, v_pages, k_scales, v_scales, 0)
    n, Hq, hd = q.shape
    P, Hkv, ps, kd = k_pages.shape
    B, M = table.shape
    if kd != hd:
        _bad(f"pages of heads of {kd}, queries of {hd}")
    _need(out, "out", q.dtype, (n, Hq, hd), q, False)
    _need(k_pages, "k_pages", k_pages.dtype, k_pages.shape, q)
    _need(table, "table", i32, (B, M), q)
    _need(starts, "starts", i32, (B + 1,), q)
    _need(lengths, "lengths", i32, (B,), q)
    if status is not None:
        _need(status, "status", i32, (1,), q)
    if scale is None:
        scale = max(hd, 1) ** -0.5
    if n == 0 or B == 0:
        return
    qs, os = q.stride(), out.stride()
    if qs[2] != 1 or os[2] != 1 or (Hq > 1 and (qs[1] != hd or os[1] != hd)):
        _bad("the heads of a token must be contiguous in q and out")
    row, d = Hq * hd, q.get_device()
    if not all(0 <= x < 1 << 31 for x in (window, sinks, max_new, max_len)):
        _bad("window, sinks, max_new or max_len outside [0, 2^31)")
    rec = [n, B, M, Hq, Hkv, hd, dt, cache, P, ps, max_new, max_len, window, sinks, scale, qs[0] if n > 1 else row,
           os[0] if n > 1 else row, q.data_ptr(), out.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), _at(k_scales),
           _at(v_scales), table.data_ptr(), starts.data_ptr(), lengths.data_ptr(), 0, 0, _at(status), wait_ns]
    L, work = load(), None
    if d >= 0:
        with torch.cuda.device(d):
            size = L.mk_paged_attention_workspace(_PAGED_ARGS.pack(*rec))
            if size < 0:
                check(size)
            if size > 0:
                with torch.cuda.stream(stream if stream is not None else torch.cuda.current_stream(d)):
                    work = torch.empty(size, dtype=torch.uint8, device=q.device)
                rec[26], rec[27] = work.data_ptr(), size
    _run_on(torch, d, stream, L.mk_paged_attention, _PAGED_ARGS.pack(*rec))


def rope_append_e4m3(qkv, q_out, k_pages, v_pages, k_scales, v_scales, positions, rows, inv_freq, slots=None,
                     q_norm=None, k_norm=None, eps: float = 1e-5, mscale: float = 1.0, interleaved: bool = False,
                     stream=None) -> None:
    """mk_rope_append_e4m3 on CUDA tensors: rope_append with 8-bit caches, k_pages / v_pages float8_e4m3fn
    [slots][Hkv][rows][hd] with k_scales / v_scales uint8 [slots][Hkv][rows][hd / 32]. With a pool of pages slots are
    the tokens' pages, rows their rows in them."""
    rc = (_quick or load_extension()).rope_append_e4m3(qkv, q_out, k_pages, v_pages, positions, rows, inv_freq, slots,
                                                    q_norm, k_norm, eps, mscale, interleaved, stream, k_scales,
                                                    v_scales)
    if rc == MK_OK:
        return
    if rc < 0:
        check(rc)
    # not done: something is wrong, or the call is for another stream or device
    import torch
    bf, i32, dt = torch.bfloat16, torch.int32, _io_dtype(torch, qkv, "qkv")
    if k_pages.dim() != 4 or q_out.dim() != 3 or qkv.dim() != 2 or inv_freq.dim() != 1:
        _bad("qkv, q_out, k_pages, inv_freq must have 2, 3, 4, 1 dimensions")
    if k_pages.dtype is not torch.float8_e4m3fn:
        _bad(f"k_pages must be float8_e4m3fn, not {k_pages.dtype} (rope_append takes bfloat16)")
    _pool(torch, k_pages, v_pages, k_scales, v_scales, 0)
    B, Hkv, S, hd = k_pages.shape
    n, Hq, _ = q_out.shape
    half = inv_freq.shape[0]
    for t, what, dtype, shape, dense in (
            (qkv, "qkv", qkv.dtype, (n, (Hq + 2 * Hkv) * hd), False), (q_out, "q_out", qkv.dtype, (n, Hq, hd), False),
            (k_pages, "k_pages", k_pages.dtype, (B, Hkv, S, hd), True), (positions, "positions", i32, (n,), True),
            (rows, "rows", i32, (n,), True), (inv_freq, "inv_freq", torch.float64, (half,), True)):
        _need(t, what, dtype, shape, qkv, dense)
    for t, what, dtype, shape in ((slots, "slots", i32, (n,)), (q_norm, "q_norm", bf, (hd,)), (k_norm, "k_norm", bf, (hd,))):
        if t is not None:
            _need(t, what, dtype, shape, qkv)
    if n == 0:
        return
    ts, qs = qkv.stride(), q_out.stride()
    if ts[1] != 1 or qs[2] != 1 or (Hq > 1 and qs[1] != hd):
        _bad("the heads of a token must be contiguous in qkv and q_out")
    width = (Hq + 2 * Hkv) * hd
    rec = _ROPE_ARGS.pack(n, Hq, Hkv, hd, 2 * half, 1 if interleaved else 0, dt, B, S, eps, mscale,
                          ts[0] if n > 1 else width, qs[0] if n > 1 else Hq * hd, qkv.data_ptr(), q_out.data_ptr(),
                          k_pages.data_ptr(), v_pages.data_ptr(), positions.data_ptr(), rows.data_ptr(), _at(slots),
                          inv_freq.data_ptr(), _at(q_norm), _at(k_norm))
    _run_on(torch, qkv.get_device(), stream, load().mk_rope_append_e4m3, rec, k_scales.data_ptr(), v_scales.data_ptr())


def _move_pages(name, k, v, k_pages, v_pages, table, lengths, slots, first, k_scales, v_scales, stream) -> None:
    rc = getattr(_quick or load_extension(), name)(k, v, k_pages, v_pages, table, lengths, slots, first, k_scales, v_scales,
                                                   stream)
    if rc == MK_OK:
        return
    if rc < 0:
        check(rc)
    # not done: something is wrong, or the call is for another stream or device
    import torch
    bf, i32 = torch.bfloat16, torch.int32
    if k.dim() != 5 or table.dim() != 2:
        _bad("the caches must have 5 dimensions, table 2")
    cache = _pool(torch, k_pages, v_pages, k_scales, v_scales, 1)
    L, slots_n, Hkv, S, hd = k.shape
    _, P, _, ps, _ = k_pages.shape
    B, M = table.shape
    _need(k, "k", bf, k.shape, k)
    _need(v, "v", bf, k.shape, k)
    _need(k_pages, "k_pages", k_pages.dtype, (L, P, Hkv, ps, hd), k)
    _need(table, "table", i32, (B, M), k)
    for t, what in ((lengths, "lengths"), (slots, "slots"), (first, "first")):
        if t is not None or what == "lengths":
            _need(t, what, i32, (B,), k)
    if slots is None and B > slots_n:
        _bad(f"{B} sequences for {slots_n} cache slots")
    if B == 0:
        return
    rec = _PAGES_ARGS.pack(L, slots_n, Hkv, S, hd, P, ps, cache, B, M, k.data_ptr(), v.data_ptr(), k_pages.data_ptr(),
                           v_pages.data_ptr(), _at(k_scales), _at(v_scales), table.data_ptr(), lengths.data_ptr(),
                           _at(first), _at(slots))
    _run_on(torch, k.get_device(), stream, getattr(load(), "mk_" + name), rec)


def kv_write_pages(k, v, k_pages, v_pages, table, lengths, slots=None, first=None, k_scales=None, v_scales=None,
                   stream=None) -> None:
    """mk_kv_write_pages on CUDA tensors: rows first[b] (0) .. lengths[b] - 1 of cache slot slots[b] (b) of k / v
    bfloat16 [L][B][Hkv][max_seq][hd] to the pages table[b] of k_pages / v_pages [L][pages][Hkv][rows][hd], bfloat16 or
    float8_e4m3fn with k_scales / v_scales uint8 [L][pages][Hkv][rows][hd / 32]."""
    _move_pages("kv_write_pages", k, v, k_pages, v_pages, table, lengths, slots, first, k_scales, v_scales, stream)


def kv_read_pages(k_pages, v_pages, k, v, table, lengths, slots=None, first=None, k_scales=None, v_scales=None,
                  stream=None) -> None:
    """mk_kv_read_pages on CUDA tensors: the way back of kv_write_pages; 8-bit rows become the bfloat16 values that
    they stand for, exactly."""
    _move_pages("kv_read_pages", k, v, k_pages, v_pages, table, lengths, slots, first, k_scales, v_scales, stream)


class Megakernel:
    """One model bound to the decode megakernel (owns an mk_handle).

    weights: dict from synth.make_weights on a CUDA device (bf16 tensors).
    k_cache, v_cache: bf16 CUDA tensors [L][max_batch][Hkv][max_seq][hd].
    """

    def __init__(self, shape, weights: dict, k_cache, v_cache, attn_splits: int = 0):
        L = load()
        self.shape = shape
        self.max_seq = int(k_cache.shape[3])
        self.max_batch = int(k_cache.shape[1])
        self._keep = (weights, k_cache, v_cache)
        self.cfg = make_config(shape, self.max_seq, self.max_batch, attn_splits)
        w, layers = _weights_struct(shape, weights)
        self._layers = layers
        kv = mk_kv_cache(k_cache.data_ptr(), v_cache.data_ptr())
        h = _VP()
        check(L.mk_create(ctypes.byref(self.cfg), ctypes.byref(w), ctypes.byref(kv), ctypes.byref(h)))
        self.h = h

    def step(self, token: int, pos: int, out_token, logits=None, stream=None) -> None:
        check(load().mk_decode_step(self.h, int(token), int(pos),
                                    logits.data_ptr() if logits is not None else None,
                                    out_token.data_ptr(), _stream_ptr(stream)))

    def step_dev(self, d_token, pos: int, out_token, logits=None, stream=None) -> None:
        check(load().mk_decode_step_dev(self.h, d_token.data_ptr(), int(pos),
                                        logits.data_ptr() if logits is not None else None,
                                        out_token.data_ptr(), _stream_ptr(stream)))

    def step_batch(self, d_tokens, d_positions, out_tokens, logits=None, stream=None) -> None:
        """d_tokens, d_positions, out_tokens: int32 CUDA tensors [B]; logits: float32 CUDA
        tensor [B][vocab] or None. Sequence b uses batch slot b of the KV cache. With
        B == max_batch (head dim 64) all sequences run in one fused launch that reads
        every weight tile once (fp16 GEMV inputs; with a top-k / top-p filter, two
        short draw kernels follow it); otherwise one launch per sequence."""
        check(load().mk_decode_step_batch(self.h, d_tokens.data_ptr(), d_positions.data_ptr(),
                                          int(d_tokens.numel()),
                                          logits.data_ptr() if logits is not None else None,
                                          out_tokens.data_ptr(), _stream_ptr(stream)))

    def prefill(self, d_tokens, start_pos: int, out_token, logits=None, stream=None) -> None:
        """mk_prefill: d_tokens int32 CUDA tensor [n] at positions start_pos ..;
        out_token int32 CUDA tensor [1]; logits float32 CUDA tensor [vocab] or None."""
        check(load().mk_prefill(self.h, d_tokens.data_ptr(), int(d_tokens.numel()), int(start_pos),
                                logits.data_ptr() if logits is not None else None, out_token.data_ptr(),
                                _stream_ptr(stream)))

    def verify(self, d_tokens, d_parents, start_pos: int, out_tokens, logits=None, stream=None) -> None:
        """mk_verify: the n nodes of a drafted tree (int32 CUDA tensors [n]) behind the committed positions
        [0, start_pos) of slot 0; out_tokens int32 CUDA tensor [n], logits float32 CUDA tensor [n][vocab] or None."""
        import torch
        n, i32, dev = int(d_tokens.numel()), torch.int32, self._keep[1].device
        if int(d_parents.numel()) != n or int(out_tokens.numel()) < n:
            _bad("d_parents and out_tokens must have as many entries as d_tokens")
        for t, what in ((d_tokens, "d_tokens"), (d_parents, "d_parents"), (out_tokens, "out_tokens")):
            if t.dtype is not i32 or t.device != dev or not t.is_contiguous():
                _bad(f"{what} must be a contiguous int32 tensor on {dev}")
        if logits is not None and (logits.dtype is not torch.float32 or logits.device != dev
                                   or not logits.is_contiguous() or logits.numel() < n * self.shape.vocab):
            _bad(f"logits must be a contiguous float32 tensor of {n} x {self.shape.vocab} on {dev}")
        check(load().mk_verify(self.h, d_tokens.data_ptr(), d_parents.data_ptr(), n, int(start_pos),
                               logits.data_ptr() if logits is not None else None, out_tokens.data_ptr(),
                               _stream_ptr(stream)))

    def accept(self, tokens, parents, draws, start_pos: int, stream=None):
        """The path of a verified tree that its draws accept (host whole numbers, as given to and returned by
        verify): its cache rows move up to start_pos .., and the nodes come back as a list. Decoding goes on at
        start_pos + len(path) with token draws[path[-1]]."""
        import torch
        if not 0 <= int(start_pos) <= self.max_seq - len(tokens):
            _bad("tree rows outside [0, max_seq)")
        path = tree_accept(tokens, parents, draws)
        if path[-1] != len(path) - 1:  # else every row is in its place
            _, k, v = self._keep
            B = self.max_batch
            host = torch.zeros(2 + len(path), B, dtype=torch.int32)
            host[0, 0], host[1, 0] = int(start_pos), len(path)
            host[2:, 0] = torch.tensor(path, dtype=torch.int32)
            s = stream or torch.cuda.current_stream(k.device)
            with torch.cuda.stream(s):
                dev = host.to(k.device)
                nodes = dev[2:].T.contiguous()
                kv_compact(k, v, dev[0], nodes, dev[1], stream=s)
        return path

    def step_unfused(self, token: int, pos: int, out_token, logits=None, stream=None) -> None:
        check(load().mk_decode_step_unfused(self.h, int(token), int(pos),
                                            logits.data_ptr() if logits is not None else None,
                                            out_token.data_ptr(), _stream_ptr(stream)))

    def step_host(self, host_token, pos: int, host_out_token, host_logits=None, stream=None) -> None:
        """host_token / host_out_token: pinned int32 CPU tensors [1]; host_logits: pinned
        float32 CPU tensor [vocab] or None."""
        check(load().mk_decode_step_host(
            self.h, ctypes.cast(host_token.data_ptr(), _PI32), int(pos),
            host_logits.data_ptr() if host_logits is not None else None,
            ctypes.cast(host_out_token.data_ptr(), _PI32), _stream_ptr(stream)))

    def status(self) -> int:
        return load().mk_get_status(self.h)

    def set_wait_timeout(self, ns: int) -> None:
        check(load().mk_set_wait_timeout(self.h, int(ns)))

    def set_sampling(self, temperature: float, seed: int = 0) -> None:
        """temperature > 0: tokens are drawn from softmax(logits / temperature)
        (Gumbel-max with Philox noise keyed by seed); <= 0: greedy."""
        check(load().mk_set_sampling(self.h, float(temperature), int(seed) & ((1 << 64) - 1)))

    def set_sampling_filter(self, top_k: int = 0, top_p: float = 1.0) -> None:
        """Top-k / top-p filtering of the sampled draw (mk_set_sampling_filter);
        top_k = 0 and top_p = 1 switch it off."""
        check(load().mk_set_sampling_filter(self.h, int(top_k), float(top_p)))

    def set_trace(self, on: bool) -> None:
        check(load().mk_set_trace(self.h, 1 if on else 0))

    def read_trace(self):
        import numpy as np
        need = check(load().mk_read_trace(self.h, None, 0))
        buf = np.zeros((max(1, need), 8), dtype=np.int64)
        n = check(load().mk_read_trace(self.h, buf.ctypes.data_as(ctypes.POINTER(ctypes.c_int64)),
                                       buf.shape[0]))
        return buf[:n]

    def debug_read(self):
        """(checked_build, [site, address, bytes, block<<32|thread])."""
        out = (ctypes.c_uint64 * 4)()
        rc = check(load().mk_debug_read(self.h, out))
        return rc == 1, list(out)

    def plan_size(self):
        n_sm, n_instr = ctypes.c_int32(), ctypes.c_int32()
        check(load().mk_plan_size(self.h, ctypes.byref(n_sm), ctypes.byref(n_instr)))
        return n_sm.value, n_instr.value

    def close(self) -> None:
        if getattr(self, "h", None):
            load().mk_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
