// mk_paged.cu — attention of ragged new tokens (one, a chunk, a whole prompt) over
// a KV cache in pages (mk_paged_attention).
//
// Mathematics, for token i of sequence b at position p = lengths[b] - n_b + i,
// query head h, kv head h / G:
//   s_j = scale * q . k_j for the rows j <= p with no window, j > p - window or
//   j < sinks; o = sum_j exp(s_j - m) v_j / sum_j exp(s_j - m), m = max_j s_j,
// in one pass over the rows with the running maximum and sum. A token that sees
// no row gets zeros.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <stdio.h>

#include <algorithm>
#include <type_traits>

#include "mk_internal.h"
#include "mk_ops.h"

namespace mkops {
namespace {

// Where row j of a sequence lies in the pool, in rows; -1 on a page outside it.
__device__ __forceinline__ int64_t pool_row(const PagedArgs &a, int b, int kvh, int j) {
    const int p = j >> a.shift, page = a.table[(int64_t)b * a.max_pages + p];
    if (page < 0 || page >= a.n_pages) return -1;
    return ((int64_t)page * a.Hkv + kvh) * a.ps + (j - (p << a.shift));
}

// Element d of a row of the pool, in fp32.
template <int HD, bool Q8>
__device__ __forceinline__ float pool_value(const void *pool, const uint8_t *scales, int64_t row, int d) {
    if (row < 0) return 0.f;
    if constexpr (Q8) {
        const uint32_t code = static_cast<const uint8_t *>(pool)[row * HD + d];
        return bf_lo(e4m3_values(code, e4m3_factor(scales[row * (HD / 32) + d / 32])).x);
    } else {
        return bf_lo(static_cast<const uint16_t *>(pool)[row * HD + d]);
    }
}

// A warp per (token, head): 32 rows at a time, a lane the score of one, then all
// lanes HD / 32 dims each of the weighted sum.
template <typename T, int HD, bool Q8>
__global__ void __launch_bounds__(128) paged_simple(const PagedArgs a) {
    __shared__ float qs[4][HD];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, t = blockIdx.x, h = blockIdx.y * 4 + warp;
    pdl_begin();
    if (h >= a.Hq) return;
    int b = 0, n = 0, i = -1;
    for (; b < a.B; ++b) {
        const int lo = min(max(a.starts[b], 0), a.n), hi = min(max(a.starts[b + 1], 0), a.n);
        if (t >= lo && t < hi) {
            n = hi - lo, i = t - lo;
            break;
        }
    }
    if (i < 0) return;
    const int pos = min(max(a.lengths[b], 0), a.cap) - n + i, kvh = h / (a.Hq / a.Hkv);
    const T *q = static_cast<const T *>(a.q) + t * a.q_stride + (int64_t)h * HD;
    for (int d = lane; d < HD; d += 32) {
        if constexpr (sizeof(T) == 4)
            qs[warp][d] = q[d];
        else
            qs[warp][d] = bf_lo(q[d]);
    }
    __syncwarp();
    float m = -INFINITY, l = 0.f, o[HD / 32] = {};
    for (int j0 = 0; j0 <= pos; j0 += 32) {
        const int j = j0 + lane;
        const bool sees = j <= pos && (!a.window || j > pos - a.window || j < a.sinks);
        if (!__any_sync(0xFFFFFFFFu, sees)) continue;
        float x = -INFINITY;
        int64_t row = -1;
        if (sees) {
            row = pool_row(a, b, kvh, j);
            x = 0.f;
            for (int d = 0; d < HD; ++d) x = fmaf(qs[warp][d], pool_value<HD, Q8>(a.kc, a.ks, row, d), x);
            x *= a.scale;
        }
        float top = x;
        for (int s = 16; s > 0; s >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, s));
        top = fmaxf(top, m);
        const float corr = m == top ? 1.f : expf(m - top), w = sees ? expf(x - top) : 0.f;
        m = top;
        l = l * corr + w;
        for (int e = 0; e < HD / 32; ++e) o[e] *= corr;
        for (int s = 0; s < 32; ++s) {
            const float ws = __shfl_sync(0xFFFFFFFFu, w, s);
            const int64_t rs = __shfl_sync(0xFFFFFFFFu, row, s);
            if (__shfl_sync(0xFFFFFFFFu, (int)sees, s))
                for (int e = 0; e < HD / 32; ++e)
                    o[e] = fmaf(ws, pool_value<HD, Q8>(a.vc, a.vs, rs, e * 32 + lane), o[e]);
        }
    }
    for (int s = 16; s > 0; s >>= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, s);
    const float inv = l == 0.f ? 0.f : 1.f / l;
    T *out = static_cast<T *>(a.out) + t * a.o_stride + (int64_t)h * HD;
    for (int e = 0; e < HD / 32; ++e) {
        if constexpr (sizeof(T) == 4)
            out[e * 32 + lane] = o[e] * inv;
        else
            out[e * 32 + lane] = (uint16_t)pack_bf16(o[e] * inv, 0.f);
    }
}

}  // namespace

bool page_shift(int page_size, int max_pages, int *shift) {
    if (page_size < 8) return false;
    *shift = 31;  // one page: every row is its own
    if (max_pages == 1) return true;
    if (page_size & (page_size - 1)) return false;
    for (*shift = 3; (1 << *shift) < page_size;) ++*shift;
    return true;
}

cudaError_t paged_attention_launch(const PagedArgs &a, int hd, bool f32, int max_new, int max_len, int n_sm,
                                   cudaStream_t s) {
    auto go = [&](auto kernel) { return launch_op(kernel, dim3(a.n, (a.Hq + 3) / 4), 128, 0, 0, s, a); };
    auto of = [&](auto type) {
        using T = decltype(type);
        if (a.ks) return hd == 64 ? go(paged_simple<T, 64, true>) : go(paged_simple<T, 128, true>);
        return hd == 64 ? go(paged_simple<T, 64, false>) : go(paged_simple<T, 128, false>);
    };
    return f32 ? of(float{}) : of(uint16_t{});
}

}  // namespace mkops

namespace {

int check_paged(const mk_paged_args *a, mkops::PagedArgs *p) {
    auto bad = [](int code, const char *what) {
        char text[192];
        snprintf(text, sizeof text, "mk_paged_attention: %s", what);
        return mkint::set_error(code, text);
    };
    if (!a || !a->q || !a->out || !a->k_pages || !a->v_pages || !a->table || !a->starts || !a->lengths)
        return bad(MK_ERR_INVALID_ARG, "a required pointer is NULL");
    if (a->dtype != MK_F32 && a->dtype != MK_BF16) return bad(MK_ERR_INVALID_ARG, "dtype is neither MK_F32 nor MK_BF16");
    if (a->cache_dtype != MK_BF16 && a->cache_dtype != MK_E4M3)
        return bad(MK_ERR_INVALID_ARG, "cache_dtype is neither MK_BF16 nor MK_E4M3");
    const bool q8 = a->cache_dtype == MK_E4M3;
    if (q8 ? !a->k_scales || !a->v_scales : a->k_scales || a->v_scales)
        return bad(MK_ERR_INVALID_ARG, "e4m3 pages need both scales, bf16 pages none");
    if (a->head_dim != 64 && a->head_dim != 128) return bad(MK_ERR_UNSUPPORTED, "head_dim must be 64 or 128");
    if (a->n_tokens < 0 || a->batch < 0 || a->max_pages < 1 || a->n_heads < 1 || a->n_kv_heads < 1 || a->n_pages < 1)
        return bad(MK_ERR_INVALID_ARG, "bad size");
    if (a->n_heads % a->n_kv_heads || a->n_heads / a->n_kv_heads > MK_MAX_GROUP)
        return bad(MK_ERR_UNSUPPORTED, "n_heads must be a multiple of n_kv_heads, at most MK_MAX_GROUP times it");
    int shift;
    if (!mkops::page_shift(a->page_size, a->max_pages, &shift))
        return bad(MK_ERR_INVALID_ARG, "page_size must be a power of two from 8 on (any from 8 on with max_pages 1)");
    const int64_t cap = (int64_t)a->max_pages * a->page_size;
    if (cap > (1 << 30)) return bad(MK_ERR_UNSUPPORTED, "max_pages * page_size above 2^30");
    if (!isfinite(a->scale) || !(a->scale > 0.f)) return bad(MK_ERR_INVALID_ARG, "scale must be finite and > 0");
    if (a->window < 0 || a->sinks < 0) return bad(MK_ERR_INVALID_ARG, "window or sinks is negative");
    if (a->max_new < 0 || a->max_new > a->n_tokens || a->max_len < 0 || a->max_len > cap)
        return bad(MK_ERR_INVALID_ARG, "max_new outside [0, n_tokens] or max_len outside [0, max_pages * page_size]");
    const int64_t row = (int64_t)a->n_heads * a->head_dim;
    if (a->n_kv_heads > 65535 || (int64_t)a->n_pages * a->n_kv_heads > INT32_MAX ||
        (int64_t)a->n_tokens * a->n_heads > (1 << 30) || a->batch > (1 << 20))
        return bad(MK_ERR_UNSUPPORTED, "too many tokens, heads, pages or sequences");
    if (a->q_stride < row || a->out_stride < row || (a->q_stride | a->out_stride) % 8)
        return bad(MK_ERR_INVALID_ARG, "a stride is too small or not a multiple of 8 elements");
    const uintptr_t all = reinterpret_cast<uintptr_t>(a->q) | reinterpret_cast<uintptr_t>(a->out) |
                          reinterpret_cast<uintptr_t>(a->k_pages) | reinterpret_cast<uintptr_t>(a->v_pages) |
                          reinterpret_cast<uintptr_t>(a->workspace);
    if ((all & 15u) || (q8 && ((reinterpret_cast<uintptr_t>(a->k_scales) | reinterpret_cast<uintptr_t>(a->v_scales)) & 3u)))
        return bad(MK_ERR_INVALID_ARG, "a pointer is not aligned");
    if (a->workspace_bytes < 0) return bad(MK_ERR_INVALID_ARG, "bad workspace");
    if (a->wait_ns < 0) return bad(MK_ERR_INVALID_ARG, "wait_ns is negative");
    if (a->n_tokens > 0) {
        const int64_t e = a->dtype == MK_F32 ? 4 : 2, rows = (int64_t)a->n_pages * a->n_kv_heads * a->page_size;
        const int64_t out_bytes = ((a->n_tokens - 1) * a->out_stride + row) * e;
        const int64_t q_bytes = ((a->n_tokens - 1) * a->q_stride + row) * e;
        const int64_t pool = rows * a->head_dim * (q8 ? 1 : 2), scales = q8 ? rows * (a->head_dim / 32) : 0;
        using mkops::meet;
        if (meet(a->out, out_bytes, a->q, q_bytes) || meet(a->out, out_bytes, a->k_pages, pool) ||
            meet(a->out, out_bytes, a->v_pages, pool) ||
            (q8 && (meet(a->out, out_bytes, a->k_scales, scales) || meet(a->out, out_bytes, a->v_scales, scales))))
            return bad(MK_ERR_INVALID_ARG, "out overlaps q, the pages or their scales");
    }
    mkops::PagedArgs r{};
    r.n = a->n_tokens, r.B = a->batch, r.max_pages = a->max_pages, r.Hq = a->n_heads, r.Hkv = a->n_kv_heads;
    r.n_pages = a->n_pages, r.ps = a->page_size, r.shift = shift, r.cap = (int)cap;
    r.window = a->window >= cap ? 0 : a->window, r.sinks = a->sinks;  // (a window over all rows is none)
    r.scale = a->scale, r.q_stride = a->q_stride, r.o_stride = a->out_stride, r.q = a->q, r.out = a->out;
    r.kc = a->k_pages, r.vc = a->v_pages, r.ks = a->k_scales, r.vs = a->v_scales;
    r.table = a->table, r.starts = a->starts, r.lengths = a->lengths;
    r.err = a->status, r.wait_ns = (uint64_t)a->wait_ns;
    r.work = static_cast<float *>(a->workspace), r.work_floats = a->workspace ? a->workspace_bytes / 4 : 0;
    *p = r;
    return MK_OK;
}

}  // namespace

extern "C" int mk_paged_attention(const mk_paged_args *a, void *stream) {
    mkops::PagedArgs p;
    const int rc = check_paged(a, &p);
    if (rc || a->batch == 0 || a->n_tokens == 0) return rc;
    const cudaError_t e =
        mkops::paged_attention_launch(p, a->head_dim, a->dtype == MK_F32, a->max_new ? a->max_new : a->n_tokens,
                                      a->max_len ? a->max_len : p.cap, mkops::sm_count(), static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? MK_OK : mkops::cuda_error(e, "mk_paged_attention");
}

extern "C" int64_t mk_paged_attention_workspace(const mk_paged_args *a) {
    mkops::PagedArgs p;
    return check_paged(a, &p);
}
