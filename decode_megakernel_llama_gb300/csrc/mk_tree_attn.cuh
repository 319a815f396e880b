// mk_tree_attn.cuh — the attention kernel of a drafted tree (see mk_tree.cu).
//
// A CTA takes NR query rows of one kv head (row = node * G + query head of the
// group) and a range of the sequence's cache rows, 128 of them a tile. Both
// products run on tcgen05 with the CACHE as the A operand, so a tile's 128
// cache rows (then 64 or 128 head dims) fill the instruction's 128 rows
// whatever the number of queries, and all 128 softmax threads have work even
// for one query row:
//   S^T [128 cache rows][N] = K [128][HD] . Q^T         (both K-major)
//   O^T [HD][N]            += V^T [HD][128] . P^T        (both MN-major: V as TMA
//                                                         wrote it, P as the threads write it)
// N = TERMS * NR: fp32 queries and weights enter as three bf16 terms each
// (24 bits: x = t0 + t1 + t2 exactly to half a step of fp32), side by side in
// the B operand, so a tile still costs HD/16 + 8 instructions; the terms'
// columns are added in registers (S) and once at the end (O). bf16 queries are
// one term, their weights are rounded to one bf16 (the result's own type).
//
// Softmax: thread = cache row, register = query row. The reference maximum m
// of a row is raised only when a score exceeds it by 2^8 (the first tile, and
// hardly ever after): exp2(s - m) <= 256 loses nothing in fp32, and the tile
// then needs no reduction over the 128 threads at all; sums of the weights
// stay per thread until the end.
//
// Overlap: warp 4 fills a ring of K and V tiles by TMA, warp 5 issues the
// MMAs. S is read into registers at once, so S(i+1) runs while the exps of
// tile i do, and PV(i) while the scores of i+1 are read. Two CTAs share an SM
// where their shared memory allows.
//
// The splits of a sequence's cache rows form a thread-block cluster: each CTA
// leaves its partial O, sums and maxima in its shared memory, and the cluster
// joins them through distributed shared memory in the splits' order (equal
// inputs give equal bits; no workspace, no second launch).
//
// Masked rows: scores are selected, not added to. A masked weight is 0, and 0
// times a non-finite value would still be NaN, so the V rows behind the
// sequence are zeroed in shared memory, and a drafted row that holds a
// non-finite value is taken out of the product and added at the end, element
// by element, for the rows that see it.
#pragma once
#include <cooperative_groups.h>

#include "mk_ops.h"
#include "mk_tc.cuh"

namespace mkops {

using namespace mktc;

// The sequence's slot, committed rows and nodes, held inside the cache
// whatever the device arrays say.
struct Seq {
    int slot, len, n;
};

__device__ __forceinline__ Seq sequence(const TreeArgs &a, int b) {
    Seq s;
    s.slot = a.slot_of ? a.slot_of[b] : b;
    s.len = min(max(a.lengths[b], 0), a.max_seq);
    s.n = min(a.counts ? min(max(a.counts[b], 0), a.T) : a.T, a.max_seq - s.len);
    if (s.slot < 0 || s.slot >= a.slots) s.n = 0;
    return s;
}

constexpr int kTile = 128;         // cache rows of a tile
constexpr int kSoft = 128;         // softmax threads
constexpr int kAttnThreads = 192;  // + the TMA warp and the MMA warp
constexpr float kNone = -1e30f;    // the maximum of a row that has seen nothing
constexpr float kRaise = 8.f;      // a score this far above m (in powers of two) raises m

template <int HD, int TERMS, int NR>
struct AttnShape {
    static constexpr int N = TERMS * NR;
    static constexpr int kHalf = kTile * 128;       // bytes of 128 rows x 64 dims
    static constexpr int kKv = kHalf * (HD / 64);   // bytes of a K (or V) tile
    static constexpr int kP = ((N + 63) / 64) * kHalf;
    static constexpr int kQ = N * HD * 2;
    static constexpr int kStages = 2;
    static constexpr int kCols = 2 * N <= 32 ? 32 : 2 * N <= 64 ? 64 : 2 * N <= 128 ? 128 : 256;
    static constexpr int kOffP = kStages * 2 * kKv, kOffQ = kOffP + kP, kOffMisc = kOffQ + kQ;
    static constexpr int kMisc = 256 + 8 * NR + 4 * NR * (3 + 4 + 4) + 4 * 16 * NR;
    static constexpr int kSmem = 1024 + kOffMisc + kMisc;
    static_assert(N % 16 == 0 && N <= 256 && 2 * N <= 256, "the instruction's N and the tensor memory");
    static_assert(NR * HD * 4 <= kStages * 2 * kKv, "the partial result fits the ring");
};

// Order-preserving map of a float to an unsigned.
__device__ __forceinline__ uint32_t ordered(float f) {
    const uint32_t u = __float_as_uint(f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t u) {
    return __uint_as_float((u & 0x80000000u) ? (u & 0x7FFFFFFFu) : ~u);
}

__device__ __forceinline__ void soft_sync() { asm volatile("barrier.cta.sync 1, 128;" ::: "memory"); }
__device__ __forceinline__ bool soft_any(bool x) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, 1, 128, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)x)
        : "memory");
    return r != 0;
}

// Values of a tensor-memory load, used only behind its wait.
template <int K>
__device__ __forceinline__ void pin(float *v) {
#pragma unroll
    for (int i = 0; i < K; ++i) asm volatile("" : "+f"(v[i]));
}

// Eight values as TERMS rows of four bf16 pairs whose sum is the values.
template <int TERMS>
__device__ __forceinline__ void split8(float (&x)[8], uint4 (&t)[TERMS]) {
#pragma unroll
    for (int k = 0; k < TERMS; ++k) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            w[i] = pack_bf16(x[2 * i], x[2 * i + 1]);
            if (k + 1 < TERMS) {
                x[2 * i] -= bf_lo(w[i]);
                x[2 * i + 1] -= bf_hi(w[i]);
            }
        }
        t[k] = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

template <int HD, int TERMS, int NR>
__global__ void __launch_bounds__(kAttnThreads, HD == 64 ? 2 : 1)
    tree_attention(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap, const TreeArgs a) {
    using C = AttnShape<HD, TERMS, NR>;
    constexpr int N = C::N, ST = C::kStages;
    namespace cg = cooperative_groups;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *Ps = sm + C::kOffP, *Qs = sm + C::kOffQ;
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + C::kOffMisc);
    uint64_t *kfull = bars, *vfull = kfull + ST, *kfree = vfull + ST, *vfree = kfree + ST;
    uint64_t *s_full = vfree + ST, *s_free = s_full + 1, *p_full = s_free + 1, *o_done = p_full + 1;
    uint32_t *tslot = reinterpret_cast<uint32_t *>(o_done + 1);
    volatile int *err = reinterpret_cast<int *>(tslot + 1);
    volatile int *issued = err + 1;                            // tiles whose K, V copies went out
    uint32_t *bad = const_cast<uint32_t *>(reinterpret_cast<volatile uint32_t *>(issued + 2));  // [2] drafted rows taken out
    uint64_t *maskw = reinterpret_cast<uint64_t *>(sm + C::kOffMisc + 256);
    float *mref = reinterpret_cast<float *>(maskw + NR), *corr = mref + NR, *lsum = corr + NR;
    float *wmax = lsum + NR, *wsum = wmax + 4 * NR, *wgt = wsum + 4 * NR;  // [4][NR], [4][NR], [16][NR]
    float *Os = reinterpret_cast<float *>(sm);  // [NR][HD], in the ring when the tiles are done

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int split = blockIdx.x, S = gridDim.x;
    const int b = blockIdx.y / a.Hkv, kvh = blockIdx.y % a.Hkv, G = a.Hq / a.Hkv;
    const Seq sq = sequence(a, b);
    const int row0 = blockIdx.z * NR, rows = min(NR, sq.n * G - row0);
    if (rows <= 0) return;  // the whole cluster
    const int total = sq.len + sq.n, tiles = (total + kTile - 1) / kTile;
    const int t0 = (int)((int64_t)split * tiles / S), nt = (int)((int64_t)(split + 1) * tiles / S) - t0;
    const int plane = sq.slot * a.Hkv + kvh;
    const float c = a.scale * 1.44269504088896340736f;  // scores in powers of two

    if (tid == 0) {
        for (int s = 0; s < ST; ++s) {
            mbar_init(&kfull[s], 1);
            mbar_init(&vfull[s], 1);
            mbar_init(&kfree[s], 1);
            mbar_init(&vfree[s], 1);
        }
        mbar_init(s_full, 1);
        mbar_init(s_free, kSoft);
        mbar_init(p_full, kSoft);
        mbar_init(o_done, 1);
        *err = 0;
        *issued = 0;
        bad[0] = bad[1] = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 4) tmem_alloc(tslot, C::kCols);
    for (int r = tid; r < NR; r += kAttnThreads) {
        mref[r] = kNone;
        lsum[r] = 0.f;
        maskw[r] = r < rows ? a.masks[(int64_t)b * a.T + (row0 + r) / G] : 0;
    }
    // the queries as the B operand: row term * NR + r, 128-byte swizzled
    for (int i = tid; i < NR * (HD / 8); i += kAttnThreads) {
        const int r = i / (HD / 8), ch = i % (HD / 8), rg = row0 + r;
        uint4 t[TERMS];
        if constexpr (TERMS == 1) {
            t[0] = make_uint4(0u, 0u, 0u, 0u);
            if (r < rows)
                t[0] = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.q) + b * a.q_batch +
                                                        (rg / G) * a.q_token + (int64_t)(kvh * G + rg % G) * HD + 8 * ch);
        } else {
            float x[8] = {};
            if (r < rows) {
                const float4 *q = reinterpret_cast<const float4 *>(static_cast<const float *>(a.q) + b * a.q_batch +
                                                                   (rg / G) * a.q_token +
                                                                   (int64_t)(kvh * G + rg % G) * HD + 8 * ch);
                const float4 u = q[0], v = q[1];
                x[0] = u.x * c, x[1] = u.y * c, x[2] = u.z * c, x[3] = u.w * c;
                x[4] = v.x * c, x[5] = v.y * c, x[6] = v.z * c, x[7] = v.w * c;
            }
            split8<TERMS>(x, t);
        }
#pragma unroll
        for (int k = 0; k < TERMS; ++k) {
            const int n = k * NR + r;
            *reinterpret_cast<uint4 *>(Qs + (ch / 8) * (N * 128) + n * 128 + (((ch % 8) ^ (n & 7)) << 4)) = t[k];
        }
    }
    async_fence();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tslot, tS = tmem, tO = tmem + N;

    if (warp == 4) {
        if (lane == 0) {
            for (int i = 0; i < nt; ++i) {
                const int s = i % ST;
                const uint32_t par = ((i / ST) - 1) & 1;
                uint8_t *k = sm + s * 2 * C::kKv, *v = k + C::kKv;
                if (i >= ST && !mbar_wait(&kfree[s], par, err)) break;
                mbar_expect_tx(&kfull[s], C::kKv);
#pragma unroll
                for (int h = 0; h < HD / 64; ++h)
                    tma_load_3d(k + h * C::kHalf, &kmap, h * 64, (t0 + i) * kTile, plane, &kfull[s]);
                *issued = 2 * i + 1;
                if (i >= ST && !mbar_wait(&vfree[s], par, err)) break;
                mbar_expect_tx(&vfull[s], C::kKv);
#pragma unroll
                for (int h = 0; h < HD / 64; ++h)
                    tma_load_3d(v + h * C::kHalf, &vmap, h * 64, (t0 + i) * kTile, plane, &vfull[s]);
                *issued = 2 * i + 2;
            }
        }
    } else if (warp == 5) {
        if (lane == 0) {
            constexpr uint32_t idS = idesc_bf16(N, false, false), idO = idesc_bf16(N, true, true);
            auto scores = [&](int i) {
                const int s = i % ST;
                if (!mbar_wait(&kfull[s], (i / ST) & 1, err)) return false;
                if (i > 0 && !mbar_wait(s_free, (i - 1) & 1, err)) return false;
                tc_fence_after();
                const uint32_t k = saddr(sm + s * 2 * C::kKv), q = saddr(Qs);
#pragma unroll
                for (int kk = 0; kk < HD / 16; ++kk)
                    umma_bf16(tS, sw128_desc(k + (kk / 4) * C::kHalf + (kk % 4) * 32, 16),
                              sw128_desc(q + (kk / 4) * (N * 128) + (kk % 4) * 32, 16), idS, kk != 0);
                umma_commit(&kfree[s]);
                umma_commit(s_full);
                return true;
            };
            bool ok = nt > 0 && scores(0);
            for (int i = 0; i < nt && ok; ++i) {
                const int s = i % ST;
                if (i + 1 < nt && !(ok = scores(i + 1))) break;
                if (!(ok = mbar_wait(p_full, i & 1, err) && mbar_wait(&vfull[s], (i / ST) & 1, err))) break;
                tc_fence_after();
                const uint32_t v = saddr(sm + s * 2 * C::kKv + C::kKv), p = saddr(Ps);
#pragma unroll
                for (int kk = 0; kk < kTile / 16; ++kk)
                    umma_bf16(tO, sw128_desc(v + kk * 2048, C::kHalf), sw128_desc(p + kk * 2048, C::kHalf), idO,
                              (i | kk) != 0);
                umma_commit(&vfree[s]);
                umma_commit(o_done);
            }
        }
    } else {
        float l[NR];
#pragma unroll
        for (int r = 0; r < NR; ++r) l[r] = 0.f;
        const uint32_t mylane = (uint32_t)(warp * 32) << 16;
        bool ok = true;
        for (int i = 0; i < nt; ++i) {
            // (a wait that ran out: the loop goes on, its barriers matched, and
            // the result becomes NaN)
            ok &= mbar_wait(s_full, i & 1, err);
            tc_fence_after();
            float s[NR];
#pragma unroll
            for (int r0 = 0; r0 < NR; r0 += 16) tmem_ld16(tS + mylane + r0, s + r0);
            if constexpr (TERMS > 1) {
#pragma unroll
                for (int k = 1; k < TERMS; ++k) {
                    float u[NR];
#pragma unroll
                    for (int r0 = 0; r0 < NR; r0 += 16) tmem_ld16(tS + mylane + k * NR + r0, u + r0);
                    tmem_ld_wait();
                    if (k == 1) pin<NR>(s);
                    pin<NR>(u);
#pragma unroll
                    for (int r = 0; r < NR; ++r) s[r] += u[r];
                }
            } else {
                tmem_ld_wait();
                pin<NR>(s);
            }
            tc_fence_before();
            mbar_arrive(s_free);
            const int at = (t0 + i) * kTile, pos = at + tid;
            const bool tail = at + kTile > sq.len;  // drafted rows, or the end
            const int node = pos - sq.len;
            if (tail && node >= 0) {
#pragma unroll
                for (int r = 0; r < NR; ++r)
                    if (node >= sq.n || !((maskw[r] >> node) & 1)) s[r] = -INFINITY;
            }
            constexpr bool kScaled = TERMS > 1;  // the queries carry c already
            float top = -INFINITY;
#pragma unroll
            for (int r = 0; r < NR; ++r) top = fmaxf(top, kScaled ? s[r] - mref[r] : fmaf(s[r], c, -mref[r]));
            if (soft_any(top > kRaise)) {
                // raise the maxima to those of all rows so far
#pragma unroll
                for (int r = 0; r < NR; ++r) {
                    const uint32_t w = __reduce_max_sync(0xFFFFFFFFu, ordered(kScaled ? s[r] : s[r] * c));
                    if (lane == (r & 31)) wmax[warp * NR + r] = unordered(w);
                }
                soft_sync();
                if (tid < NR) {
                    const float old = mref[tid];
                    float m = old;
#pragma unroll
                    for (int w = 0; w < 4; ++w) m = fmaxf(m, wmax[w * NR + tid]);
                    corr[tid] = ex2(old - m);
                    mref[tid] = m;
                }
                soft_sync();
#pragma unroll
                for (int r = 0; r < NR; ++r) l[r] *= corr[r];
                if (i > 0) {
                    ok &= mbar_wait(o_done, (i - 1) & 1, err);
                    tc_fence_after();
                    if (__all_sync(0xFFFFFFFFu, ok)) {
#pragma unroll 1
                        for (int n0 = 0; n0 < N; n0 += 16) {
                            float o[16];
                            tmem_ld16(tO + mylane + n0, o);
                            tmem_ld_wait();
                            pin<16>(o);
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[e] *= corr[n0 % NR + e];
                            tmem_st16(tO + mylane + n0, o);
                        }
                        tmem_st_wait();
                    }
                    tc_fence_before();
                }
            }
#pragma unroll
            for (int r = 0; r < NR; ++r) {
                s[r] = ex2(kScaled ? s[r] - mref[r] : fmaf(s[r], c, -mref[r]));
                l[r] += s[r];
            }
            if (i > 0) ok &= mbar_wait(o_done, (i - 1) & 1, err);  // P is free again
            bool out = false;
            if (tail) {
                const int st = i % ST;
                ok &= mbar_wait(&vfull[st], (i / ST) & 1, err);
                if (node >= 0) {
                    uint8_t *v = sm + st * 2 * C::kKv + C::kKv + tid * 128;
                    bool zero = node >= sq.n;
                    if (!zero) {
                        uint32_t inf = 0;
#pragma unroll
                        for (int h = 0; h < HD / 64; ++h)
#pragma unroll
                            for (int ch = 0; ch < 8; ++ch) {
                                const uint4 u = *reinterpret_cast<const uint4 *>(v + h * C::kHalf + ch * 16);
                                const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    inf |= (uint32_t)((w[e] & 0x7F80u) == 0x7F80u) |
                                           (uint32_t)((w[e] & 0x7F800000u) == 0x7F800000u);
                            }
                        if (inf) {
                            out = zero = true;
                            atomicOr(&bad[node >> 5], 1u << (node & 31));
                        }
                    }
                    if (zero) {
#pragma unroll
                        for (int h = 0; h < HD / 64; ++h)
#pragma unroll
                            for (int ch = 0; ch < 8; ++ch)
                                *reinterpret_cast<uint4 *>(v + h * C::kHalf + ch * 16) = make_uint4(0u, 0u, 0u, 0u);
                    }
                }
            }
            // the weights as the B operand: row = cache row, column = term * NR + r
            uint8_t *p = Ps + tid * 128;
#pragma unroll
            for (int r0 = 0; r0 < NR; r0 += 8) {
                float x[8];
                uint4 t[TERMS];
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = out ? 0.f : s[r0 + e];
                split8<TERMS>(x, t);
#pragma unroll
                for (int k = 0; k < TERMS; ++k) {
                    const int ch = (k * NR + r0) / 8;
                    *reinterpret_cast<uint4 *>(p + (ch / 8) * C::kHalf + (((ch % 8) ^ (tid & 7)) << 4)) = t[k];
                }
            }
            async_fence();
            mbar_arrive(p_full);
        }
        if (nt > 0) ok &= mbar_wait(o_done, (nt - 1) & 1, err);
        tc_fence_after();
        const bool all = !soft_any(!ok);
        // the sums of the 128 threads, warp by warp
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            float x = l[r];
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
            if (lane == (r & 31)) wsum[warp * NR + r] = x;
        }
        // O^T: lane = head dim, column = term * NR + r
        if (warp * 32 < HD) {
#pragma unroll 1
            for (int r0 = 0; r0 < NR; r0 += 16) {
                float o[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] = 0.f;
                if (nt > 0 && all) {
#pragma unroll
                    for (int k = TERMS - 1; k >= 0; --k) {
                        float u[16];
                        tmem_ld16(tO + mylane + k * NR + r0, u);
                        tmem_ld_wait();
                        pin<16>(u);
#pragma unroll
                        for (int e = 0; e < 16; ++e) o[e] += u[e];
                    }
                }
#pragma unroll
                for (int e = 0; e < 16; ++e) Os[(r0 + e) * HD + warp * 32 + lane] = o[e];
            }
        }
        soft_sync();
        if (tid < NR)
            lsum[tid] = all ? wsum[tid] + wsum[NR + tid] + wsum[2 * NR + tid] + wsum[3 * NR + tid]
                            : __uint_as_float(0x7FC00000u);  // a wait ran out: NaN
        if (bad[0] | bad[1]) {
            const uint64_t left = bad[0] | ((uint64_t)bad[1] << 32);
            const int64_t base = (int64_t)plane * a.max_seq * HD;
            for (int i = tid; i < rows * HD; i += kSoft) {
                const int r = i / HD, d = i % HD, rg = row0 + r;
                const int64_t qat = b * a.q_batch + (rg / G) * a.q_token + (int64_t)(kvh * G + rg % G) * HD;
                for (uint64_t w = left & maskw[r]; w; w &= w - 1) {
                    const int64_t at = base + (int64_t)(sq.len + __ffsll(w) - 1) * HD;
                    float x = 0.f;
                    for (int e = 0; e < HD; ++e) {
                        float qv;
                        if constexpr (TERMS == 1)
                            qv = bf_lo(static_cast<const uint16_t *>(a.q)[qat + e]);
                        else
                            qv = static_cast<const float *>(a.q)[qat + e];
                        x = fmaf(qv, bf_lo(a.kc[at + e]), x);
                    }
                    Os[i] = fmaf(ex2(fmaf(x, c, -mref[r])), bf_lo(a.vc[at + d]), Os[i]);
                }
            }
        }
    }
    __syncwarp();
    __syncthreads();
    if (*err && tid == 0) {
        // copies that were issued land before the shared memory goes
        const int ni = *issued;
        for (int j = max(0, ni - 2 * ST); j < ni; ++j) {
            const int i = j / 2;
            uint64_t *bar = (j & 1) ? &vfull[i % ST] : &kfull[i % ST];
            const uint64_t from = gtimer();
            while (!mbar_try(bar, (i / ST) & 1))
                if (gtimer() - from > kWaitNs) break;
        }
        if (a.err) atomicExch(a.err, 1);
    }
    __syncthreads();
    if (warp == 4) {
        tc_fence_after();
        tmem_free(tmem, C::kCols);
    }
    // join the splits
    cg::cluster_group cl = cg::this_cluster();
    if (S > 1) cl.sync();
    for (int r = tid; r < rows; r += kAttnThreads) {
        float m = kNone, sum = 0.f;
        for (int s = 0; s < S; ++s) m = fmaxf(m, *cl.map_shared_rank(mref + r, s));
        for (int s = 0; s < S; ++s) {
            const float w = ex2(*cl.map_shared_rank(mref + r, s) - m);
            wgt[s * NR + r] = w;
            sum = fmaf(w, *cl.map_shared_rank(lsum + r, s), sum);
        }
        corr[r] = sum == 0.f ? 0.f : 1.f / sum;  // no row seen: zeros
    }
    __syncthreads();
    const int64_t obase = b * a.o_batch;
    for (int i = split * kAttnThreads + tid; i < rows * (HD / 4); i += S * kAttnThreads) {
        const int r = i / (HD / 4), d = 4 * (i % (HD / 4)), rg = row0 + r;
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int s = 0; s < S; ++s) {
            const float4 o = *reinterpret_cast<const float4 *>(cl.map_shared_rank(Os + r * HD + d, s));
            const float w = wgt[s * NR + r];
            y.x = fmaf(w, o.x, y.x), y.y = fmaf(w, o.y, y.y), y.z = fmaf(w, o.z, y.z), y.w = fmaf(w, o.w, y.w);
        }
        const float inv = corr[r];
        y.x *= inv, y.y *= inv, y.z *= inv, y.w *= inv;
        const int64_t to = obase + (rg / G) * a.o_token + (int64_t)(kvh * G + rg % G) * HD + d;
        if (a.hi) {
            const uint32_t u = pack_bf16(y.x, y.y), v = pack_bf16(y.z, y.w);
            *reinterpret_cast<uint2 *>(a.hi + to) = make_uint2(u, v);
            *reinterpret_cast<uint2 *>(a.lo + to) =
                make_uint2(pack_bf16(y.x - bf_lo(u), y.y - bf_hi(u)), pack_bf16(y.z - bf_lo(v), y.w - bf_hi(v)));
        } else if constexpr (TERMS == 1) {
            *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.out) + to) =
                make_uint2(pack_bf16(y.x, y.y), pack_bf16(y.z, y.w));
        } else {
            *reinterpret_cast<float4 *>(static_cast<float *>(a.out) + to) = y;
        }
    }
    if (S > 1) cl.sync();  // nobody leaves while its memory is read
}

}  // namespace mkops
