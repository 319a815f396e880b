// mk_pages.cu — rows between a contiguous KV cache and a pool of pages
// (mk_kv_write_pages, mk_kv_read_pages), as they are or in 8 bits.
//
// Mathematics of an 8-bit row: for each 32 elements the smallest e in [-100, 7]
// with max|x| <= 448 * 2^e; codes e4m3(x / 2^e), rounded once. A power of two makes
// the division and the way back exact, so a row read back is what the tensor cores
// take of it in mk_paged_attention, and no block saturates.
//
// What bounds them: memory, each row read once and written once: 4 sequences of up to 2,050
// rows, 28 layers of 8 kv heads of 128, read from bf16 pages in 238 us = 6.7 TB/s; 8 of up to
// 2,000, 16 layers of heads of 64, written in 8 bits and the pool read back in 215 us = 6.0
// TB/s; 130 rows in 3.3 us, the launch and two dependent loads. A thread owns
// eight elements (16 bytes of bf16, 8 of codes) of kRows rows, K and V: all its
// loads are out before the first value is used. Four neighbouring threads hold a
// block of 32 and find its largest by two shuffles.
#include <cuda_runtime.h>
#include <stdint.h>
#include <stdio.h>

#include <algorithm>
#include <type_traits>

#include "mk_internal.h"
#include "mk_ops.h"

namespace mkops {
namespace {

constexpr int kT = 256;
constexpr int kRows = 4;  // rows of a thread in flight

struct MoveArgs {
    int L, slots, Hkv, max_seq, n_pages, ps, shift, B, max_pages, cap;
    uint4 *k, *v;
    uint8_t *kp, *vp, *ks, *vs;
    const int32_t *table, *lengths, *first, *slot_of;
};

// Eight bf16 as fp32.
__device__ __forceinline__ void widen(uint4 u, float4 &a, float4 &b) {
    a = make_float4(bf_lo(u.x), bf_hi(u.x), bf_lo(u.y), bf_hi(u.y));
    b = make_float4(bf_lo(u.z), bf_hi(u.z), bf_lo(u.w), bf_hi(u.w));
}

// The largest magnitude of the four threads' eight values each; infinity where one is no number.
__device__ __forceinline__ float block_most(uint4 u) {
    // (magnitudes of bf16 as whole numbers: in order, and NaN above infinity)
    const uint32_t w[4] = {u.x & 0x7FFF7FFFu, u.y & 0x7FFF7FFFu, u.z & 0x7FFF7FFFu, u.w & 0x7FFF7FFFu};
    uint32_t m = __vmaxu2(__vmaxu2(w[0], w[1]), __vmaxu2(w[2], w[3]));
    m = __vmaxu2(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
    m = __vmaxu2(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
    m = max(m & 0xFFFFu, m >> 16);
    return m >= 0x7F80u ? INFINITY : __uint_as_float(m << 16);
}

// grid (blocks of rows, L * Hkv, B)
template <int HD, bool Q8, bool WRITE>
__global__ void __launch_bounds__(kT) move_pages(const MoveArgs a) {
    constexpr int CPR = HD / 8;            // threads of a row
    constexpr int RPB = kT / CPR * kRows;  // rows of a CTA at a time
    const int b = blockIdx.z, tid = threadIdx.x, part = tid % CPR;
    pdl_begin();
    const int slot = a.slot_of ? a.slot_of[b] : b;
    const int last = min(a.lengths[b], a.cap), from = a.first ? max(a.first[b], 0) : 0;
    if (slot < 0 || slot >= a.slots) return;
    const int l = blockIdx.y / a.Hkv, h = blockIdx.y % a.Hkv;
    const int64_t row0 = (((int64_t)l * a.slots + slot) * a.Hkv + h) * a.max_seq;
    const int32_t *table = a.table + (int64_t)b * a.max_pages;
    for (int64_t j0 = from + (int64_t)blockIdx.x * RPB; j0 < last; j0 += (int64_t)gridDim.x * RPB) {
        int64_t at[kRows], page_at[kRows];  // a row of the cache and of the pool; -1: none
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
            const int64_t j = j0 + u * (kT / CPR) + tid / CPR;
            at[u] = -1;
            if (j < last) {
                const int p = (int)(j >> a.shift), page = table[p];
                if (page >= 0 && page < a.n_pages) {
                    at[u] = row0 + j;
                    page_at[u] = (((int64_t)l * a.n_pages + page) * a.Hkv + h) * a.ps + (j - ((int64_t)p << a.shift));
                }
            }
        }
        uint4 k[kRows], v[kRows];
        uint2 k8[kRows], v8[kRows];
        uint32_t ks[kRows], vs[kRows];
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
            if (at[u] < 0) {
                k[u] = v[u] = make_uint4(0, 0, 0, 0);
                continue;
            }
            if constexpr (WRITE) {
                k[u] = a.k[at[u] * CPR + part];
                v[u] = a.v[at[u] * CPR + part];
            } else if constexpr (Q8) {
                k8[u] = reinterpret_cast<const uint2 *>(a.kp)[page_at[u] * CPR + part];
                v8[u] = reinterpret_cast<const uint2 *>(a.vp)[page_at[u] * CPR + part];
                ks[u] = a.ks[page_at[u] * (HD / 32) + part / 4];
                vs[u] = a.vs[page_at[u] * (HD / 32) + part / 4];
            } else {
                k[u] = reinterpret_cast<const uint4 *>(a.kp)[page_at[u] * CPR + part];
                v[u] = reinterpret_cast<const uint4 *>(a.vp)[page_at[u] * CPR + part];
            }
        }
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
            if constexpr (WRITE && Q8) {
                float4 x, y;
                const float km = block_most(k[u]), vm = block_most(v[u]);  // (by whole warps)
                if (at[u] < 0) continue;
                const uint32_t k_s = e4m3_scale(km), v_s = e4m3_scale(vm);
                widen(k[u], x, y);
                reinterpret_cast<uint2 *>(a.kp)[page_at[u] * CPR + part] = make_uint2(e4m3_codes(x, k_s), e4m3_codes(y, k_s));
                widen(v[u], x, y);
                reinterpret_cast<uint2 *>(a.vp)[page_at[u] * CPR + part] = make_uint2(e4m3_codes(x, v_s), e4m3_codes(y, v_s));
                if (part % 4 == 0) {
                    a.ks[page_at[u] * (HD / 32) + part / 4] = (uint8_t)k_s;
                    a.vs[page_at[u] * (HD / 32) + part / 4] = (uint8_t)v_s;
                }
            } else {
                if (at[u] < 0) continue;
                if constexpr (WRITE) {
                    reinterpret_cast<uint4 *>(a.kp)[page_at[u] * CPR + part] = k[u];
                    reinterpret_cast<uint4 *>(a.vp)[page_at[u] * CPR + part] = v[u];
                } else {
                    if constexpr (Q8) {
                        const uint32_t kf = e4m3_factor(ks[u]), vf = e4m3_factor(vs[u]);
                        const uint2 k0 = e4m3_values(k8[u].x, kf), k1 = e4m3_values(k8[u].y, kf);
                        const uint2 v0 = e4m3_values(v8[u].x, vf), v1 = e4m3_values(v8[u].y, vf);
                        k[u] = make_uint4(k0.x, k0.y, k1.x, k1.y);
                        v[u] = make_uint4(v0.x, v0.y, v1.x, v1.y);
                    }
                    a.k[at[u] * CPR + part] = k[u];
                    a.v[at[u] * CPR + part] = v[u];
                }
            }
        }
    }
}

int move(const char *who, const mk_pages_args *a, bool write, void *stream) {
    auto bad = [&](int code, const char *what) {
        char text[192];
        snprintf(text, sizeof text, "%s: %s", who, what);
        return mkint::set_error(code, text);
    };
    if (!a || !a->k || !a->v || !a->k_pages || !a->v_pages || !a->table || !a->lengths)
        return bad(MK_ERR_INVALID_ARG, "a required pointer is NULL");
    if (a->cache_dtype != MK_BF16 && a->cache_dtype != MK_E4M3)
        return bad(MK_ERR_INVALID_ARG, "cache_dtype is neither MK_BF16 nor MK_E4M3");
    const bool q8 = a->cache_dtype == MK_E4M3;
    if (q8 ? !a->k_scales || !a->v_scales : a->k_scales || a->v_scales)
        return bad(MK_ERR_INVALID_ARG, "e4m3 pages need both scales, bf16 pages none");
    if (a->head_dim != 64 && a->head_dim != 128) return bad(MK_ERR_UNSUPPORTED, "head_dim must be 64 or 128");
    if (a->n_layers < 1 || a->slots < 1 || a->n_kv_heads < 1 || a->max_seq < 1 || a->n_pages < 1 || a->batch < 0 ||
        a->max_pages < 1)
        return bad(MK_ERR_INVALID_ARG, "bad size");
    int shift;
    if (!page_shift(a->page_size, a->max_pages, &shift))
        return bad(MK_ERR_INVALID_ARG, "page_size must be a power of two from 8 on (any from 8 on with max_pages 1)");
    const uintptr_t all = reinterpret_cast<uintptr_t>(a->k) | reinterpret_cast<uintptr_t>(a->v) |
                          reinterpret_cast<uintptr_t>(a->k_pages) | reinterpret_cast<uintptr_t>(a->v_pages);
    if (all & 15u) return bad(MK_ERR_INVALID_ARG, "a pointer is not aligned");
    if ((int64_t)a->n_layers * a->n_kv_heads > 65535 || a->batch > 65535)
        return bad(MK_ERR_UNSUPPORTED, "n_layers * n_kv_heads or batch above 65535");
    const int64_t rows = (int64_t)a->n_layers * a->slots * a->n_kv_heads * a->max_seq, bytes = rows * a->head_dim * 2;
    const int64_t prows = (int64_t)a->n_layers * a->n_pages * a->n_kv_heads * a->page_size;
    const int64_t pbytes = prows * a->head_dim * (q8 ? 1 : 2), sbytes = q8 ? prows * (a->head_dim / 32) : 0;
    const struct {
        const void *at;
        int64_t bytes;
    } part[] = {{a->k, bytes}, {a->v, bytes}, {a->k_pages, pbytes}, {a->v_pages, pbytes}, {a->k_scales, sbytes},
                {a->v_scales, sbytes}};
    for (int i = 0; i < (q8 ? 6 : 4); ++i)
        for (int j = 0; j < i; ++j)
            if (meet(part[i].at, part[i].bytes, part[j].at, part[j].bytes))
                return bad(MK_ERR_INVALID_ARG, "caches, pages and scales must not overlap");
    if (a->batch == 0) return MK_OK;
    const int64_t each = (int64_t)a->batch * 4;
    for (int i = write ? 2 : 0; i < (!write ? 2 : q8 ? 6 : 4); ++i)  // (what is written)
        if (meet(part[i].at, part[i].bytes, a->table, each * a->max_pages) ||
            meet(part[i].at, part[i].bytes, a->lengths, each) || meet(part[i].at, part[i].bytes, a->first, each) ||
            meet(part[i].at, part[i].bytes, a->slot_of, each))
            return bad(MK_ERR_INVALID_ARG, "what is written overlaps table, lengths, first or slot_of");
    MoveArgs m{};
    m.L = a->n_layers, m.slots = a->slots, m.Hkv = a->n_kv_heads, m.max_seq = a->max_seq, m.n_pages = a->n_pages;
    m.ps = a->page_size, m.shift = shift, m.B = a->batch, m.max_pages = a->max_pages;
    m.cap = (int)std::min((int64_t)a->max_pages * a->page_size, (int64_t)a->max_seq);
    m.k = static_cast<uint4 *>(a->k), m.v = static_cast<uint4 *>(a->v);
    m.kp = static_cast<uint8_t *>(a->k_pages), m.vp = static_cast<uint8_t *>(a->v_pages);
    m.ks = a->k_scales, m.vs = a->v_scales;
    m.table = a->table, m.lengths = a->lengths, m.first = a->first, m.slot_of = a->slot_of;
    const int rpb = kT / (a->head_dim / 8) * kRows, planes = a->n_layers * a->n_kv_heads;
    // (about 16 CTAs an SM in all; a CTA with more rows than its first loops)
    const int64_t blocks = (m.cap + rpb - 1) / rpb, want = (16ll * sm_count()) / ((int64_t)planes * a->batch) + 1;
    const dim3 grid((unsigned)std::min(blocks, want), planes, a->batch);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    auto go = [&](auto kernel) { return launch_op(kernel, grid, kT, 0, 0, s, m); };
    auto of = [&](auto dim) {
        constexpr int HD = decltype(dim)::value;
        if (q8) return write ? go(move_pages<HD, true, true>) : go(move_pages<HD, true, false>);
        return write ? go(move_pages<HD, false, true>) : go(move_pages<HD, false, false>);
    };
    const cudaError_t e = a->head_dim == 64 ? of(std::integral_constant<int, 64>{}) : of(std::integral_constant<int, 128>{});
    return e == cudaSuccess ? MK_OK : cuda_error(e, who);
}

}  // namespace
}  // namespace mkops

extern "C" int mk_kv_write_pages(const mk_pages_args *a, void *stream) {
    return mkops::move("mk_kv_write_pages", a, true, stream);
}

extern "C" int mk_kv_read_pages(const mk_pages_args *a, void *stream) {
    return mkops::move("mk_kv_read_pages", a, false, stream);
}
