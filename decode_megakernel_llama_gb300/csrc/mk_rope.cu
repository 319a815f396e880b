// mk_rope.cu — per-head norms, rotary positions and the append to the KV
// cache in one pass (mk_rope_append), and the host-side frequencies of scaled
// contexts (mk_rope_frequencies).
//
// Mathematics, for token t with rotary position p, head vector x [hd]:
//   x' = x * g / sqrt(mean(x^2) + eps)              (queries, keys; optional)
//   angle_i = p * w_i, w_i radians per position (64 bits)
//   (a, b) -> mscale * (a cos - b sin, b cos + a sin) for the rot/2 pairs
//   (x'_i, x'_{i + rot/2}) or, interleaved, (x'_{2i}, x'_{2i+1});
//   the hd - rot elements behind them pass through.
// The angle is reduced to a fraction of a turn in 64 bits before its sine and
// cosine are taken in 32, so a far position loses nothing: a turn's fraction
// is off by at most p * 2^-53 turns.
//
// What bounds it: the floor is memory, as each element is read once and written once and
// the arithmetic is a few operations an element; a long prompt takes 1.18 times its
// bytes' time (8,192 tokens of 48 heads of 64, fp32, normed: 32.7 us, DRAM 53 % and issue
// slots 40 % busy, 43 % of the warps: the latency of the loads), a few tokens the time of
// their dependent round trips. A CTA takes one token (or four): its
// threads form the token's sines and cosines once for all heads (shared memory)
// while every warp's first loads are already in flight; a head is held by hd/4
// lanes of a warp, four elements a lane, or by hd/8, four elements of each half, so
// the norm is a shuffle sum and the partner of a pair is in the lane itself (the
// whole head rotated), a shuffle away, or in shared memory (rot/2 no multiple of
// four, or pairs that lie neither way). A few tokens are spread over several CTAs each.
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

constexpr int kT = 256;  // threads per CTA
constexpr int kW = kT / 32;
constexpr int kMaxHalf = 64;  // rotated pairs of a head
constexpr int kPerSm = 3;     // CTAs of the form for fewer tokens that an SM holds

template <typename T>
__device__ __forceinline__ float4 load4(const T *p);
template <>
__device__ __forceinline__ float4 load4<float>(const float *p) {
    return *reinterpret_cast<const float4 *>(p);
}
template <>
__device__ __forceinline__ float4 load4<uint16_t>(const uint16_t *p) {
    const uint2 u = *reinterpret_cast<const uint2 *>(p);
    return make_float4(bf_lo(u.x), bf_hi(u.x), bf_lo(u.y), bf_hi(u.y));
}

__device__ __forceinline__ uint2 pack4(float4 v) { return make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w)); }

template <typename T>
__device__ __forceinline__ void store4(T *p, float4 v);
template <>
__device__ __forceinline__ void store4<float>(float *p, float4 v) {
    *reinterpret_cast<float4 *>(p) = v;
}
template <>
__device__ __forceinline__ void store4<uint16_t>(uint16_t *p, float4 v) {
    *reinterpret_cast<uint2 *>(p) = pack4(v);
}

// TPB tokens a CTA (1 or 4), kW / TPB warps each; a lane holds E elements of a head:
// four, or four of each half. (64 registers: with four CTAs an SM instead of three a prompt of 8,192 tokens
// takes 9 % less. Beside memory the instructions bound a long prompt, 140 for 32 x 4
// elements when they took 53 % of the issue slots: so eight elements a lane, which
// share a norm's shuffles, a head's tests and its addresses, and the reciprocal root
// as one instruction.)
// Q8: the cache in e4m3. A block of 32 elements is the four of eight lanes. A value next to
// a code's border lands a whole step away if 32 bits put it on the wrong side, so the sine's
// argument and the reciprocal root are corrected here: of 64 x 4 million keys 319 then differ
// from those of 64 bits, 496 without (4,094 tokens, heads of 128: 32.6 us with the reading
// back, 31.8 without).
template <typename T, int HD, int TPB, int E, bool Q8>
__global__ void __launch_bounds__(kT, TPB == 1 && E == 8 ? kPerSm : 4) rope_append(const RopeArgs a) {
    constexpr int LPH = HD / E;    // lanes of a head
    constexpr int HPW = 32 / LPH;  // heads of a warp
    constexpr int B = 16 / E;      // a warp's heads in flight, HPW each
    constexpr int WPT = kW / TPB;  // warps of a token
    __shared__ float2 turn[TPB][kMaxHalf];
    __shared__ float4 stage[kT * E / 4];  // a head's row, for pairs that are not a lane apart
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int sub = lane / LPH, j = lane % LPH;  // head of the warp, lane of the head
    const int t = blockIdx.x * TPB + warp / WPT, half = a.rot / 2, n_rows = a.Hq + 2 * a.Hkv;
    const bool here = t < a.n;
    const float2 *cs = turn[warp / WPT];
    pdl_begin();
    const T *in = static_cast<const T *>(a.qkv) + (int64_t)t * a.qkv_stride + 4 * j;
    T *qo = static_cast<T *>(a.q_out) + (int64_t)t * a.q_stride + 4 * j;
    const int row = here ? a.rows[t] : -1, slot = here && a.slot_of ? a.slot_of[t] : 0;
    const int first = (blockIdx.y * WPT + warp % WPT) * HPW + sub, step = gridDim.y * WPT * HPW;
    float4 x[B][E / 4];
    auto load = [&](int h0) {
#pragma unroll
        for (int u = 0; u < B; ++u)
#pragma unroll
            for (int e = 0; e < E / 4; ++e) {
                const int h = h0 + u * step;
                x[u][e] = here && h < n_rows ? load4<T>(in + (int64_t)h * HD + 4 * e * LPH) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
    };
    load(first);
    uint2 gq[E / 4], gk[E / 4];  // the gains, bf16
#pragma unroll
    for (int e = 0; e < E / 4; ++e) {
        const uint2 one = make_uint2(0x3F803F80u, 0x3F803F80u);
        gq[e] = a.q_norm ? *reinterpret_cast<const uint2 *>(a.q_norm + 4 * (e * LPH + j)) : one;
        gk[e] = a.k_norm ? *reinterpret_cast<const uint2 *>(a.k_norm + 4 * (e * LPH + j)) : one;
    }
    for (int i = tid; i < TPB * kMaxHalf; i += kT) {
        const int tt = blockIdx.x * TPB + i / kMaxHalf, e = i % kMaxHalf;
        if (e < half && tt < a.n) {
            // radians to turns in 64 bits; the fraction of a turn fits 32
            const double turns = (double)a.positions[tt] * a.inv_freq[e] * 0.15915494309189533577;
            float s, c;
            const double part = turns - rint(turns);
            sincospif(2.0f * (float)part, &s, &c);
            if constexpr (Q8) {  // what 32 bits cut off the angle, to first order
                const float rest = (float)(part - (double)(float)part) * 6.28318530717959f, s0 = s;
                s = fmaf(rest, c, s), c = fmaf(-rest, s0, c);
            }
            turn[i / kMaxHalf][e] = make_float2(c * a.mscale, s * a.mscale);
        }
    }
    const bool keep = slot >= 0 && slot < a.slots && row >= 0 && row < a.max_seq;
    __syncthreads();
    // (a warp's loop is as long as its first head's: h - sub is the same in all lanes)
    for (int h0 = first; here && h0 - sub < n_rows; h0 += B * step) {
        if (h0 != first) load(h0);
        float ss[B];  // the batch's sums of squares side by side
        if (a.q_norm || a.k_norm) {
#pragma unroll
            for (int u = 0; u < B; ++u) {
                ss[u] = 0.f;
#pragma unroll
                for (int e = 0; e < E / 4; ++e) {
                    const float4 v = x[u][e];
                    ss[u] += v.x * v.x + v.y * v.y + v.z * v.z + v.w * v.w;
                }
            }
#pragma unroll
            for (int o = LPH / 2; o > 0; o >>= 1)
#pragma unroll
                for (int u = 0; u < B; ++u) ss[u] += __shfl_xor_sync(0xFFFFFFFFu, ss[u], o);
        }
#pragma unroll
        for (int u = 0; u < B; ++u) {
            const int h = h0 + u * step;
            if (h - sub >= n_rows) break;
            const bool is_q = h < a.Hq, is_k = !is_q && h < a.Hq + a.Hkv;
            if (is_q ? a.q_norm != nullptr : is_k && a.k_norm != nullptr) {
                const float ms = ss[u] * (1.0f / HD) + a.eps;
                float r = rsqrtf(ms);
                if (Q8 && r > 0.f) r = fmaf(0.5f * r, fmaf(-ms * r, r, 1.0f), r);  // (Newton's step; an infinite sum leaves 0)
#pragma unroll
                for (int e = 0; e < E / 4; ++e) {
                    const uint2 g = is_q ? gq[e] : gk[e];
                    float4 &v = x[u][e];
                    v = make_float4(v.x * r * bf_lo(g.x), v.y * r * bf_hi(g.x), v.z * r * bf_lo(g.y), v.w * r * bf_hi(g.y));
                }
            }
            T *to = qo + (int64_t)h * HD;
            uint16_t *cache = nullptr;
            uint8_t *codes = nullptr, *scale = nullptr;
            if (!is_q && keep && h < n_rows) {
                const int kvh = is_k ? h - a.Hq : h - a.Hq - a.Hkv;
                const int64_t at = ((int64_t)slot * a.Hkv + kvh) * a.max_seq + row;
                if constexpr (Q8) {
                    codes = reinterpret_cast<uint8_t *>(is_k ? a.kc : a.vc) + at * HD + 4 * j;
                    scale = (is_k ? a.ks : a.vs) + at * (HD / 32) + j / 8;
                } else {
                    cache = (is_k ? a.kc : a.vc) + at * HD + 4 * j;
                }
            }
            auto store = [&](int e, float4 y) {
                // (whole warps: a block's largest is found by shuffles; not where all heads are queries)
                if (Q8 && h - sub + HPW > a.Hq) {
                    float most = fmaxf(fmaxf(fabsf(y.x), fabsf(y.y)), fmaxf(fabsf(y.z), fabsf(y.w)));
                    if (!(y.x - y.x == 0.f && y.y - y.y == 0.f && y.z - y.z == 0.f && y.w - y.w == 0.f)) most = INFINITY;
#pragma unroll
                    for (int o = 1; o < 8; o <<= 1) most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, o));
                    if (codes) {
                        const uint32_t s = e4m3_scale(most);
                        *reinterpret_cast<uint32_t *>(codes + 4 * e * LPH) = e4m3_codes(y, s);
                        if ((j & 7) == 0) scale[e * LPH / 8] = (uint8_t)s;
                    }
                }
                if (is_q && h < n_rows)
                    store4<T>(to + 4 * e * LPH, y);
                else if (cache)
                    store4<uint16_t>(cache + 4 * e * LPH, y);
            };
            if (a.interleaved) {
#pragma unroll
                for (int e = 0; e < E / 4; ++e) {
                    const float4 v = x[u][e];
                    const int pair = 2 * (e * LPH + j);
                    float4 y = v;
                    if (is_q || is_k) {
                        if (pair < half) {
                            const float2 c = cs[pair];
                            y.x = v.x * c.x - v.y * c.y;
                            y.y = v.y * c.x + v.x * c.y;
                        }
                        if (pair + 1 < half) {
                            const float2 c = cs[pair + 1];
                            y.z = v.z * c.x - v.w * c.y;
                            y.w = v.w * c.x + v.z * c.y;
                        }
                    }
                    store(e, y);
                }
            } else if (E == 8 && half == HD / 2) {
                // an element's partner is in the lane's other four
                float4 v = x[u][0], w = x[u][E / 4 - 1];
                if (is_q || is_k) {
                    const float2 *c = cs + 4 * j;
                    const float2 c0 = c[0], c1 = c[1], c2 = c[2], c3 = c[3];
                    const float4 o = v;
                    v = make_float4(v.x * c0.x - w.x * c0.y, v.y * c1.x - w.y * c1.y, v.z * c2.x - w.z * c2.y,
                                    v.w * c3.x - w.w * c3.y);
                    w = make_float4(w.x * c0.x + o.x * c0.y, w.y * c1.x + o.y * c1.y, w.z * c2.x + o.z * c2.y,
                                    w.w * c3.x + o.w * c3.y);
                }
                store(0, v);
                store(E / 4 - 1, w);
            } else if (half % 4 == 0 && half / 2 <= LPH) {
                // it is the same element of the lane half / 4 away, of the lane's first four
                const int d = half / 4, from = j < d ? lane + d : lane - d;
                const float4 v = x[u][0];
                const float4 o = make_float4(__shfl_sync(0xFFFFFFFFu, v.x, from), __shfl_sync(0xFFFFFFFFu, v.y, from),
                                             __shfl_sync(0xFFFFFFFFu, v.z, from), __shfl_sync(0xFFFFFFFFu, v.w, from));
                float4 y = v;
                if ((is_q || is_k) && j < 2 * d) {
                    const float2 *c = cs + 4 * (j < d ? j : j - d);
                    const float sg = j < d ? -1.f : 1.f;
                    y.x = v.x * c[0].x + sg * (o.x * c[0].y);
                    y.y = v.y * c[1].x + sg * (o.y * c[1].y);
                    y.z = v.z * c[2].x + sg * (o.z * c[2].y);
                    y.w = v.w * c[3].x + sg * (o.w * c[3].y);
                }
                store(0, y);
                if (E == 8) store(E / 4 - 1, x[u][E / 4 - 1]);
            } else {
                __syncwarp();
#pragma unroll
                for (int e = 0; e < E / 4; ++e) stage[(tid - j) * (E / 4) + e * LPH + j] = x[u][e];
                __syncwarp();
                const float *mine = reinterpret_cast<const float *>(stage + (tid - j) * (E / 4));
#pragma unroll
                for (int q = 0; q < E / 4; ++q) {
                    const float z[4] = {x[u][q].x, x[u][q].y, x[u][q].z, x[u][q].w};
                    float o[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int e = 4 * (q * LPH + j) + i;
                        o[i] = z[i];
                        if ((is_q || is_k) && e < half) {
                            const float2 c = cs[e];
                            o[i] = z[i] * c.x - mine[e + half] * c.y;
                        } else if ((is_q || is_k) && e < a.rot) {
                            const float2 c = cs[e - half];
                            o[i] = z[i] * c.x + mine[e - half] * c.y;
                        }
                    }
                    store(q, make_float4(o[0], o[1], o[2], o[3]));
                }
            }
        }
    }
}

}  // namespace

cudaError_t rope_append_launch(const RopeArgs &a, int hd, bool f32, cudaStream_t s) {
    // Many tokens: four a CTA, two warps each, so that their angles are formed side
    // by side and a warp has several rounds of loads (8,192 tokens of 48 heads of 64 in
    // fp32, normed: 32.7 us = 5.6 TB/s, 38.8 with four elements a lane). Fewer: a token
    // over as many CTAs as the GPU holds, up to one for each round (216 tokens: 2.9 us, 3.3
    // with one CTA each, 4.2 with four elements a lane; 800 tokens of 40 heads of 128:
    // 6.5 us, 7.8 as many, and 1,000, more than two waves, 8.6 and 7.8). A few, where
    // latency counts: four elements a lane (one token: 1.75 us, 1.9 with eight).
    const int per_cta = kW * (hd == 64 ? 2 : 1), rounds = (a.Hq + 2 * a.Hkv + per_cta - 1) / per_cta;
    const int at_once = kPerSm * sm_count();
    const bool many = a.n > 2 * at_once, few = a.n <= 32;
    const int spread = std::max(1, std::min({rounds, 8, at_once / a.n}));
    const dim3 grid(many ? (a.n + 3) / 4 : a.n, many ? 1 : spread);
    auto go = [&](auto kernel) { return launch_op(kernel, grid, kT, 0, 0, s, a); };
    auto pick = [&](auto four, auto one, auto one4) { return many ? go(four) : few ? go(one4) : go(one); };
    auto of = [&](auto type, auto q8) {
        using T = decltype(type);
        constexpr bool Q8 = decltype(q8)::value;
        return hd == 64 ? pick(rope_append<T, 64, 4, 8, Q8>, rope_append<T, 64, 1, 8, Q8>, rope_append<T, 64, 1, 4, Q8>)
                        : pick(rope_append<T, 128, 4, 8, Q8>, rope_append<T, 128, 1, 8, Q8>,
                               rope_append<T, 128, 1, 4, Q8>);
    };
    const bool q8 = a.ks != nullptr;
    if (f32) return q8 ? of(float{}, std::true_type{}) : of(float{}, std::false_type{});
    return q8 ? of(uint16_t{}, std::true_type{}) : of(uint16_t{}, std::false_type{});
}

}  // namespace mkops

namespace {

// Checks and launches mk_rope_append, or with scales mk_rope_append_e4m3.
int rope(const char *who, const mk_rope_args *a, bool q8, uint8_t *ks, uint8_t *vs, void *stream) {
    auto bad = [&](int code, const char *what) {
        char text[192];
        snprintf(text, sizeof text, "%s: %s", who, what);
        return mkint::set_error(code, text);
    };
    if (!a || !a->qkv || !a->q_out || !a->k_cache || !a->v_cache || !a->positions || !a->rows || !a->inv_freq ||
        (q8 && (!ks || !vs)))
        return bad(MK_ERR_INVALID_ARG, "a required pointer is NULL");
    if (a->dtype != MK_F32 && a->dtype != MK_BF16)
        return bad(MK_ERR_INVALID_ARG, "dtype is neither MK_F32 nor MK_BF16");
    if (a->head_dim != 64 && a->head_dim != 128)
        return bad(MK_ERR_UNSUPPORTED, "head_dim must be 64 or 128");
    if (a->n < 0 || a->n_heads < 1 || a->n_kv_heads < 1 || a->slots < 1 || a->max_seq < 1)
        return bad(MK_ERR_INVALID_ARG, "bad size");
    if (a->rot < 2 || a->rot > a->head_dim || a->rot % 2)
        return bad(MK_ERR_INVALID_ARG, "rot must be even, 2 .. head_dim");
    if (!(a->eps >= 0.f) || !isfinite(a->eps) || !isfinite(a->mscale))
        return bad(MK_ERR_INVALID_ARG, "eps or mscale is not a finite number");
    const int64_t q = (int64_t)a->n_heads * a->head_dim, qkv = q + 2 * (int64_t)a->n_kv_heads * a->head_dim;
    if (qkv > INT32_MAX) return bad(MK_ERR_INVALID_ARG, "too many heads");
    if (a->qkv_stride < qkv || a->q_stride < q || a->qkv_stride % 4 || a->q_stride % 4)
        return bad(MK_ERR_INVALID_ARG, "a stride is too small or not a multiple of 4 elements");
    const uintptr_t io = reinterpret_cast<uintptr_t>(a->qkv) | reinterpret_cast<uintptr_t>(a->q_out);
    const uintptr_t both = reinterpret_cast<uintptr_t>(a->k_cache) | reinterpret_cast<uintptr_t>(a->v_cache);
    const uintptr_t cache = reinterpret_cast<uintptr_t>(a->k_cache) | reinterpret_cast<uintptr_t>(a->v_cache) |
                            reinterpret_cast<uintptr_t>(a->q_norm) | reinterpret_cast<uintptr_t>(a->k_norm);
    if ((io & 15u) || (cache & 7u) || (q8 && (both & 15u)) || (reinterpret_cast<uintptr_t>(a->inv_freq) & 7u))
        return bad(MK_ERR_INVALID_ARG, "a pointer is not aligned");
    if (a->n == 0) return MK_OK;
    // What one CTA writes no other may read or write: the caches apart from everything,
    // q_out from qkv but for the same rows in place, or rows in the gaps between qkv's.
    const int64_t e = a->dtype == MK_F32 ? 4 : 2, q_bytes = ((a->n - 1) * a->q_stride + q) * e,
                  qkv_bytes = ((a->n - 1) * a->qkv_stride + qkv) * e,
                  rows = (int64_t)a->slots * a->n_kv_heads * a->max_seq, cache_bytes = rows * a->head_dim * (q8 ? 1 : 2);
    using mkops::meet;
    const struct {
        const void *at;
        int64_t bytes;
    } written[] = {{a->k_cache, cache_bytes}, {a->v_cache, cache_bytes}, {ks, rows * (a->head_dim / 32)},
                   {vs, rows * (a->head_dim / 32)}};
    for (int i = 0; i < (q8 ? 4 : 2); ++i) {
        bool met = meet(written[i].at, written[i].bytes, a->q_out, q_bytes) ||
                   meet(written[i].at, written[i].bytes, a->qkv, qkv_bytes);
        for (int k = 0; k < i; ++k) met = met || meet(written[i].at, written[i].bytes, written[k].at, written[k].bytes);
        if (met) return bad(MK_ERR_INVALID_ARG, "a cache overlaps the other, qkv or q_out");
    }
    const int64_t each = (int64_t)a->n * 4, gains = (int64_t)a->head_dim * 2;
    const struct {
        const void *at;
        int64_t bytes;
    } read[] = {{a->positions, each}, {a->rows, each}, {a->slot_of, a->slot_of ? each : 0},
                {a->inv_freq, (int64_t)a->rot * 4}, {a->q_norm, a->q_norm ? gains : 0}, {a->k_norm, a->k_norm ? gains : 0}};
    for (const auto &r : read) {
        bool met = mkops::meet_rows(a->q_out, a->n, a->q_stride * e, q * e, r.at, r.bytes);
        for (int i = 0; i < (q8 ? 4 : 2); ++i) met = met || meet(written[i].at, written[i].bytes, r.at, r.bytes);
        if (met) return bad(MK_ERR_INVALID_ARG, "what is written overlaps positions, rows, slot_of, inv_freq or a gain");
    }
    if (meet(a->q_out, q_bytes, a->qkv, qkv_bytes)) {
        const int64_t step = a->qkv_stride * e;
        int64_t off = (int64_t)(reinterpret_cast<uintptr_t>(a->q_out) - reinterpret_cast<uintptr_t>(a->qkv));
        const bool same_rows = a->n == 1 || a->q_stride == a->qkv_stride;
        const bool in_place = off == 0 && same_rows;
        off = (off % step + step) % step;
        if (!in_place && !(same_rows && a->n > 1 && off >= qkv * e && off + q * e <= step))
            return bad(MK_ERR_INVALID_ARG, "q_out overlaps qkv other than row by row in place");
    }
    mkops::RopeArgs r{};
    r.n = a->n, r.Hq = a->n_heads, r.Hkv = a->n_kv_heads, r.rot = a->rot, r.interleaved = a->interleaved;
    r.slots = a->slots, r.max_seq = a->max_seq, r.eps = a->eps, r.mscale = a->mscale;
    r.qkv_stride = a->qkv_stride, r.q_stride = a->q_stride;
    r.qkv = a->qkv, r.q_out = a->q_out;
    r.ks = ks, r.vs = vs;
    r.kc = static_cast<uint16_t *>(a->k_cache), r.vc = static_cast<uint16_t *>(a->v_cache);
    r.positions = a->positions, r.rows = a->rows, r.slot_of = a->slot_of, r.inv_freq = a->inv_freq;
    r.q_norm = static_cast<const uint16_t *>(a->q_norm), r.k_norm = static_cast<const uint16_t *>(a->k_norm);
    const cudaError_t err =
        mkops::rope_append_launch(r, a->head_dim, a->dtype == MK_F32, static_cast<cudaStream_t>(stream));
    return err == cudaSuccess ? MK_OK : mkops::cuda_error(err, who);
}

}  // namespace

extern "C" int mk_rope_append(const mk_rope_args *a, void *stream) {
    return rope("mk_rope_append", a, false, nullptr, nullptr, stream);
}

extern "C" int mk_rope_append_e4m3(const mk_rope_args *a, uint8_t *k_scales, uint8_t *v_scales, void *stream) {
    return rope("mk_rope_append_e4m3", a, true, k_scales, v_scales, stream);
}

extern "C" int mk_rope_frequencies(int32_t kind, int32_t rot, double theta, double factor, double original_len,
                                   double low, double high, double *out, float *mscale) {
    using mkint::set_error;
    if (!out || !mscale) return set_error(MK_ERR_INVALID_ARG, "mk_rope_frequencies: NULL pointer");
    if (rot < 2 || rot % 2 || !(theta > 1.0) || !isfinite(theta))
        return set_error(MK_ERR_INVALID_ARG, "mk_rope_frequencies: rot must be even and >= 2, theta finite and > 1");
    if (kind != MK_ROPE_PLAIN && (!(factor >= 1.0) || !isfinite(factor)))
        return set_error(MK_ERR_INVALID_ARG, "mk_rope_frequencies: factor must be finite and >= 1");
    if ((kind == MK_ROPE_WAVELENGTH || kind == MK_ROPE_YARN) &&
        (!(original_len > 0.0) || !(low > 0.0) || !(high > low) || !isfinite(original_len) || !isfinite(high)))
        return set_error(MK_ERR_INVALID_ARG, "mk_rope_frequencies: needs original_len > 0 and 0 < low < high");
    const double two_pi = 6.283185307179586477;
    double base = theta;
    *mscale = 1.f;
    if (kind == MK_ROPE_BASE) {
        if (rot < 4) return set_error(MK_ERR_INVALID_ARG, "mk_rope_frequencies: MK_ROPE_BASE needs rot >= 4");
        base = theta * pow(factor, (double)rot / (rot - 2));
    } else if (kind < MK_ROPE_PLAIN || kind > MK_ROPE_YARN) {
        return set_error(MK_ERR_INVALID_ARG, "mk_rope_frequencies: unknown kind");
    }
    double lo = 0.0, hi = 1.0;
    if (kind == MK_ROPE_YARN) {
        // the pair whose wave turns b times over the original context
        auto pair_of = [&](double b) { return rot * log(original_len / (b * two_pi)) / (2.0 * log(theta)); };
        lo = std::max(0.0, floor(pair_of(high)));
        hi = std::min(rot - 1.0, ceil(pair_of(low)));
        *mscale = (float)(0.1 * log(factor) + 1.0);
    }
    for (int i = 0; i < rot / 2; ++i) {
        const double f = pow(base, -2.0 * i / rot);
        double w = f;
        if (kind == MK_ROPE_LINEAR) {
            w = f / factor;
        } else if (kind == MK_ROPE_WAVELENGTH) {
            const double s = std::min(1.0, std::max(0.0, (original_len * f / two_pi - low) / (high - low)));
            w = f * ((1.0 - s) / factor + s);
        } else if (kind == MK_ROPE_YARN) {
            const double r = std::min(1.0, std::max(0.0, (i - lo) / std::max(1e-3, hi - lo)));
            w = f / factor * r + f * (1.0 - r);
        }
        out[i] = w;
    }
    return MK_OK;
}
