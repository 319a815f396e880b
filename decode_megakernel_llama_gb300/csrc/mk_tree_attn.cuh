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
// then needs no reduction over the 128 threads at all. The sums of the weights
// come out of the second product where its A operand has room: for HD = 64 the
// instruction's rows 64 .. 127 are a constant block whose first row is ones, so
// lane 64 of O^T is sum p; for HD = 128 they stay per thread until the end.
//
// Overlap: warp 4 fills a ring of K and V tiles by TMA, warp 5 issues the
// MMAs. S is read into registers at once, so S(i+1) runs while the exps of
// tile i do, and PV(i) while the scores of i+1 are read. Two CTAs share an SM
// where their shared memory allows.
//
// Up to 8 splits of a sequence's cache rows form a thread-block cluster: each
// CTA leaves its partial O, sums and maxima in its shared memory, and the
// cluster joins them through distributed shared memory in the splits' order
// (equal inputs give equal bits; no workspace, no second launch). More splits
// (a long cache and few sequences) leave their partials in the caller's
// workspace for tree_join.
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
constexpr int kCluster = 8;        // most splits joined in a cluster
constexpr int kMaxSplits = 64;     // most splits joined through the workspace
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
    static constexpr int kOnes = HD == 64 ? 2048 : 0;  // 16 cache rows x 64: ones in the first column
    static constexpr int kOffP = kStages * 2 * kKv, kOffQ = kOffP + kP, kOffOnes = kOffQ + kQ;
    static constexpr int kOffMisc = kOffOnes + kOnes;
    static constexpr int kMisc = 256 + 8 * NR + 4 * NR * (3 + 4 + 3 * 8);
    static constexpr int kSmem = 1024 + kOffMisc + kMisc;
    static_assert(N % 16 == 0 && 2 * N <= 256, "the instruction's N and the tensor memory");
    static_assert(NR * HD * 4 <= kStages * 2 * kKv, "the partial result fits the ring");
};

// Floats of one split's partial result in the workspace: O [NR][HD], the
// maxima and the sums [NR].
__host__ __device__ constexpr int64_t part_floats(int nr, int hd) { return (int64_t)nr * hd + 2 * nr; }

__device__ __forceinline__ float max_warp(float x) {
    float y;
    asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
    return y;
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

// A result of four dims: fp32, bf16, or the hi / lo terms of the handle's path.
template <int TERMS>
__device__ __forceinline__ void put4(const TreeArgs &a, int64_t to, float4 y) {
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

template <int HD, int TERMS, int NR>
__global__ void __launch_bounds__(kAttnThreads, HD == 64 ? 2 : 1)
    tree_attention(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap, const TreeArgs a) {
    using C = AttnShape<HD, TERMS, NR>;
    constexpr int N = C::N, ST = C::kStages;
    constexpr bool kScaled = TERMS > 1;  // the queries carry the scale already
    constexpr bool kOnes = HD == 64;     // the sums come out of the second product
    namespace cg = cooperative_groups;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *Ps = sm + C::kOffP, *Qs = sm + C::kOffQ;
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + C::kOffMisc);
    uint64_t *kfull = bars, *vfull = kfull + ST, *kfree = vfull + ST, *vfree = kfree + ST;
    uint64_t *s_full = vfree + ST, *s_free = s_full + 1, *p_full = s_free + 1, *o_done = p_full + 1;
    uint32_t *tslot = reinterpret_cast<uint32_t *>(o_done + 1);
    volatile int *err = reinterpret_cast<int *>(tslot + 1);
    volatile int *issued = err + 1;  // K and V copies that went out
    uint32_t *bad = const_cast<uint32_t *>(reinterpret_cast<volatile uint32_t *>(issued + 2));  // [2] drafted rows taken out
    uint64_t *maskw = reinterpret_cast<uint64_t *>(sm + C::kOffMisc + 256);
    float *mref = reinterpret_cast<float *>(maskw + NR), *corr = mref + NR, *lsum = corr + NR;
    float *wtmp = lsum + NR;                               // [4][NR]
    float *wgt = wtmp + 4 * NR, *m8 = wgt + 8 * NR, *l8 = m8 + 8 * NR;  // [8][NR] of the cluster's splits
    float *Os = reinterpret_cast<float *>(sm);             // [NR][HD], in the ring when the tiles are done

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int split = blockIdx.x, S = gridDim.x;
    const int b = blockIdx.y / a.Hkv, kvh = blockIdx.y % a.Hkv, G = a.Hq / a.Hkv;
    const int row0 = blockIdx.z * NR;
    const float c = a.scale * 1.44269504088896340736f;  // scores in powers of two

    // the queries as the B operand: row term * NR + r, 128-byte swizzled. (They
    // are read before the sequence's counts are known: rows of nodes behind
    // the last one are columns nobody reads.)
    for (int i = tid; i < NR * (HD / 8); i += kAttnThreads) {
        const int r = i / (HD / 8), ch = i % (HD / 8), rg = row0 + r;
        const bool in = rg < a.T * G;
        const int64_t qat = b * a.q_batch + (rg / G) * a.q_token + (int64_t)(kvh * G + rg % G) * HD + 8 * ch;
        uint4 t[TERMS];
        if constexpr (TERMS == 1) {
            t[0] = make_uint4(0u, 0u, 0u, 0u);
            if (in) t[0] = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.q) + qat);
        } else {
            float x[8] = {};
            if (in) {
                const float4 *q = reinterpret_cast<const float4 *>(static_cast<const float *>(a.q) + qat);
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
    const Seq sq = sequence(a, b);
    const int rows = min(NR, sq.n * G - row0);
    if (rows <= 0) return;  // the whole cluster
    const int total = sq.len + sq.n, tiles = (total + kTile - 1) / kTile;
    const int t0 = (int)((int64_t)split * tiles / S), nt = (int)((int64_t)(split + 1) * tiles / S) - t0;
    const int plane = sq.slot * a.Hkv + kvh;

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
    if constexpr (kOnes)
        for (int i = tid; i < C::kOnes / 16; i += kAttnThreads)  // chunk 0 of row i / 8 sits at chunk (row & 7)
            *reinterpret_cast<uint4 *>(sm + C::kOffOnes + i * 16) =
                make_uint4(i % 8 == ((i / 8) & 7) ? 0x3F80u : 0u, 0u, 0u, 0u);
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
                const uint32_t v = saddr(sm + s * 2 * C::kKv + C::kKv), p = saddr(Ps), ones = saddr(sm + C::kOffOnes);
#pragma unroll
                for (int kk = 0; kk < kTile / 16; ++kk)
                    umma_bf16(tO, sw128_desc(v + kk * 2048, kOnes ? ones - (v + kk * 2048) : C::kHalf),
                              sw128_desc(p + kk * 2048, C::kHalf), idO, (i | kk) != 0);
                umma_commit(&vfree[s]);
                umma_commit(o_done);
            }
        }
    } else {
        float l[kOnes ? 1 : NR];
        if constexpr (!kOnes)
#pragma unroll
            for (int r = 0; r < NR; ++r) l[r] = 0.f;
        const uint32_t mylane = (uint32_t)(warp * 32) << 16;
        const float4 *m4 = reinterpret_cast<const float4 *>(mref);
        bool ok = true;
        for (int i = 0; i < nt; ++i) {
            // (a wait that ran out: the loop goes on, its barriers matched, and
            // the result becomes NaN)
            ok &= mbar_wait(s_full, i & 1, err);
            tc_fence_after();
            float s[N];
#pragma unroll
            for (int n0 = 0; n0 < N; n0 += 16) tmem_ld16(tS + mylane + n0, s + n0);
            tmem_ld_wait();
            pin<N>(s);
            tc_fence_before();
            mbar_arrive(s_free);
#pragma unroll
            for (int r = 0; r < NR; ++r)
#pragma unroll
                for (int k = 1; k < TERMS; ++k) s[r] += s[k * NR + r];
            const int at = (t0 + i) * kTile, pos = at + tid;
            const bool tail = at + kTile > sq.len;  // drafted rows, or the end
            const int node = pos - sq.len;
            if (tail && node >= 0) {
#pragma unroll
                for (int r = 0; r < NR; ++r)
                    if (node >= sq.n || !((maskw[r] >> node) & 1)) s[r] = -INFINITY;
            }
            // y = s - m in powers of two, and the largest of them
            auto shift = [&](float (&y)[NR], const float (&x)[N]) {
                float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int r = 0; r < NR; r += 4) {
                    const float4 m = m4[r / 4];
                    y[r] = kScaled ? x[r] - m.x : fmaf(x[r], c, -m.x);
                    y[r + 1] = kScaled ? x[r + 1] - m.y : fmaf(x[r + 1], c, -m.y);
                    y[r + 2] = kScaled ? x[r + 2] - m.z : fmaf(x[r + 2], c, -m.z);
                    y[r + 3] = kScaled ? x[r + 3] - m.w : fmaf(x[r + 3], c, -m.w);
                    top[(r / 4) & 3] = fmaxf(fmaxf(fmaxf(y[r], y[r + 1]), fmaxf(y[r + 2], y[r + 3])), top[(r / 4) & 3]);
                }
                return fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
            };
            float y[NR];
            if (soft_any(shift(y, s) > kRaise)) {
                // raise the maxima to those of all rows so far
#pragma unroll
                for (int r = 0; r < NR; ++r) {
                    const float w = max_warp(kScaled ? s[r] : s[r] * c);
                    if (lane == (r & 31)) wtmp[warp * NR + r] = w;
                }
                soft_sync();
                if (tid < NR) {
                    const float old = mref[tid];
                    const float m = fmaxf(fmaxf(fmaxf(wtmp[tid], wtmp[NR + tid]),
                                                fmaxf(wtmp[2 * NR + tid], wtmp[3 * NR + tid])), old);
                    corr[tid] = ex2(old - m);
                    mref[tid] = m;
                }
                soft_sync();
                shift(y, s);
                if constexpr (!kOnes)
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
                for (int e = 0; e < 8; ++e) {
                    x[e] = ex2(y[r0 + e]);
                    if constexpr (!kOnes) l[r0 + e] += x[e];
                    if (out) x[e] = 0.f;
                }
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
        if constexpr (!kOnes) {
            // the sums of the 128 threads, warp by warp
#pragma unroll
            for (int r = 0; r < NR; ++r) {
                float x = l[r];
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
                if (lane == (r & 31)) wtmp[warp * NR + r] = x;
            }
        }
        // O^T: lane = head dim (lane 64 of a head of 64: the sums), column = term * NR + r
        if (warp * 32 < HD || (kOnes && warp == 2)) {
#pragma unroll 1
            for (int r0 = 0; r0 < NR; r0 += 16) {
                float o[16];
                if (nt > 0 && all) {
                    float u[16 * TERMS];
#pragma unroll
                    for (int k = 0; k < TERMS; ++k) tmem_ld16(tO + mylane + k * NR + r0, u + 16 * k);
                    tmem_ld_wait();
                    pin<16 * TERMS>(u);
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        o[e] = u[16 * (TERMS - 1) + e];
#pragma unroll
                        for (int k = TERMS - 2; k >= 0; --k) o[e] += u[16 * k + e];
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 16; ++e) o[e] = 0.f;
                }
                if (warp * 32 < HD) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) Os[(r0 + e) * HD + warp * 32 + lane] = o[e];
                } else if (lane == 0) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) lsum[r0 + e] = o[e];
                }
            }
        }
        soft_sync();
        if constexpr (!kOnes)
            if (tid < NR) lsum[tid] = (wtmp[tid] + wtmp[NR + tid]) + (wtmp[2 * NR + tid] + wtmp[3 * NR + tid]);
        if (!all)
            if (tid < NR) lsum[tid] = __uint_as_float(0x7FC00000u);  // a wait ran out: NaN
        if (bad[0] | bad[1]) {
            soft_sync();
            const uint64_t left = bad[0] | ((uint64_t)bad[1] << 32);
            const int64_t base = (int64_t)plane * a.max_seq * HD;
            for (int i = tid; i < rows * HD; i += kSoft) {
                const int r = i / HD, d = i % HD, rg = row0 + r;
                const int64_t qat = b * a.q_batch + (rg / G) * a.q_token + (int64_t)(kvh * G + rg % G) * HD;
                float add = 0.f;  // kOnes: their weights are not in the sums yet
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
                    x = ex2(fmaf(x, c, -mref[r]));
                    add += x;
                    Os[i] = fmaf(x, bf_lo(a.vc[at + d]), Os[i]);
                }
                if (kOnes && d == 0) lsum[r] += add;
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
    if (warp == 4) {
        tc_fence_after();
        tmem_free(tmem, C::kCols);
    }
    if (a.part) {  // leave the partial result to tree_join
        const int64_t unit = (int64_t)blockIdx.z * gridDim.y + blockIdx.y;
        float *p = a.part + (unit * S + split) * part_floats(NR, HD);
        for (int i = tid; i < rows * (HD / 4); i += kAttnThreads)
            reinterpret_cast<float4 *>(p)[i] = reinterpret_cast<const float4 *>(Os)[i];
        for (int r = tid; r < rows; r += kAttnThreads) {
            p[NR * HD + r] = mref[r];
            p[NR * HD + NR + r] = lsum[r];
        }
        return;
    }
    // join the cluster's splits: first every split's maxima and sums, then the
    // rows, shared out over the CTAs
    cg::cluster_group cl = cg::this_cluster();
    if (S > 1) cl.sync();
    for (int i = tid; i < S * NR; i += kAttnThreads) {
        m8[i] = *cl.map_shared_rank(mref + i % NR, i / NR);
        l8[i] = *cl.map_shared_rank(lsum + i % NR, i / NR);
    }
    __syncthreads();
    for (int r = tid; r < rows; r += kAttnThreads) {
        float m = kNone, sum = 0.f;
        for (int s = 0; s < S; ++s) m = fmaxf(m, m8[s * NR + r]);
        for (int s = 0; s < S; ++s) sum = fmaf(ex2(m8[s * NR + r] - m), l8[s * NR + r], sum);
        const float inv = sum == 0.f ? 0.f : 1.f / sum;  // no row seen: zeros
        for (int s = 0; s < S; ++s) wgt[s * NR + r] = ex2(m8[s * NR + r] - m) * inv;
    }
    __syncthreads();
    for (int i = split * kAttnThreads + tid; i < rows * (HD / 4); i += S * kAttnThreads) {
        const int r = i / (HD / 4), d = 4 * (i % (HD / 4)), rg = row0 + r;
        float4 o[8];
#pragma unroll
        for (int s = 0; s < 8; ++s)
            if (s < S) o[s] = *reinterpret_cast<const float4 *>(cl.map_shared_rank(Os + r * HD + d, s));
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int s = 0; s < 8; ++s)
            if (s < S) {
                const float w = wgt[s * NR + r];
                y.x = fmaf(w, o[s].x, y.x), y.y = fmaf(w, o[s].y, y.y);
                y.z = fmaf(w, o[s].z, y.z), y.w = fmaf(w, o[s].w, y.w);
            }
        put4<TERMS>(a, b * a.o_batch + (rg / G) * a.o_token + (int64_t)(kvh * G + rg % G) * HD + d, y);
    }
    if (S > 1) cl.sync();  // nobody leaves while its memory is read
}

// Joins the S splits' partial results of every (row tile, sequence, kv head):
// grid (row tiles, batch * Hkv), a thread per four dims of a row.
template <int HD, int TERMS, int NR>
__global__ void __launch_bounds__(256) tree_join(const TreeArgs a, int S) {
    constexpr int64_t PF = part_floats(NR, HD);
    __shared__ float ms[kMaxSplits * NR], wg[kMaxSplits * NR];
    const int b = blockIdx.y / a.Hkv, kvh = blockIdx.y % a.Hkv, G = a.Hq / a.Hkv, row0 = blockIdx.x * NR;
    const Seq sq = sequence(a, b);
    const int rows = min(NR, sq.n * G - row0);
    if (rows <= 0) return;
    const int64_t unit = (int64_t)blockIdx.x * gridDim.y + blockIdx.y;
    const float *p = a.part + unit * S * PF;
    for (int i = threadIdx.x; i < S * NR; i += 256) {
        const bool in = i % NR < rows;
        ms[i] = in ? p[(i / NR) * PF + NR * HD + i % NR] : kNone;
        wg[i] = in ? p[(i / NR) * PF + NR * HD + NR + i % NR] : 0.f;
    }
    __syncthreads();
    for (int r = threadIdx.x; r < rows; r += 256) {
        float m = kNone, sum = 0.f;
        for (int s = 0; s < S; ++s) m = fmaxf(m, ms[s * NR + r]);
        for (int s = 0; s < S; ++s) sum = fmaf(ex2(ms[s * NR + r] - m), wg[s * NR + r], sum);
        const float inv = sum == 0.f ? 0.f : 1.f / sum;  // no row seen: zeros
        for (int s = 0; s < S; ++s) wg[s * NR + r] = ex2(ms[s * NR + r] - m) * inv;
    }
    __syncthreads();
    for (int i = blockIdx.z * 256 + threadIdx.x; i < rows * (HD / 4); i += gridDim.z * 256) {
        const int r = i / (HD / 4), d = 4 * (i % (HD / 4)), rg = row0 + r;
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int s0 = 0; s0 < S; s0 += 8) {
            float4 o[8];
#pragma unroll
            for (int s = 0; s < 8; ++s)
                if (s0 + s < S) o[s] = *reinterpret_cast<const float4 *>(p + (s0 + s) * PF + r * HD + d);
#pragma unroll
            for (int s = 0; s < 8; ++s)
                if (s0 + s < S) {
                    const float w = wg[(s0 + s) * NR + r];
                    y.x = fmaf(w, o[s].x, y.x), y.y = fmaf(w, o[s].y, y.y);
                    y.z = fmaf(w, o[s].z, y.z), y.w = fmaf(w, o[s].w, y.w);
                }
        }
        put4<TERMS>(a, b * a.o_batch + (rg / G) * a.o_token + (int64_t)(kvh * G + rg % G) * HD + d, y);
    }
}

}  // namespace mkops
