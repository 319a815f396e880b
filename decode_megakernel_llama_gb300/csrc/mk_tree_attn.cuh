// mk_tree_attn.cuh — the attention kernels of a drafted tree (see mk_tree.cu).
//
// Two tcgen05 kernels share everything but which operand the queries are.
//
// tree_attention (few query rows, up to 64 a CTA): the CACHE is the A operand,
// so a tile's 128 cache rows (then 64 or 128 head dims) fill the instruction's
// 128 rows whatever the number of queries, and all softmax threads have work
// even for one query row:
//   S^T [128 cache rows][N] = K [128][HD] . Q^T    (both K-major)
//   O^T [HD][N]            += V^T [HD][128] . P^T   (both MN-major: V as TMA wrote
//                                                    it, P as the threads write it)
// tree_attention_rows (many): 128 query rows are the A operand,
//   S [128 rows][128 cache rows] = Q . K^T, O [128 rows][HD] += P . V,
// P from tensor memory, where it overwrites the scores it came from.
// Measured (MMAs back to back): an instruction of M = 128 costs the larger of
// 44 cycles, its share of shared-memory reads (4 KB of A and 32 N bytes of B at
// 128 B a cycle) and N / 2 cycles, and a chain of 8 is seen complete ~340
// cycles after its last issue. So the first form pays 48 cycles an instruction
// for N = 64 and the second 64 for twice the scores (and none for P).
//
// fp32 queries and weights enter as three bf16 terms each (24 bits: x = t0 + t1 +
// t2 to half a step of fp32): side by side in the first kernel's B operand, N =
// TERMS * NR, added in registers (S) and once at the end (O); as more instructions
// into the same accumulator in the second. bf16 queries are one term, their
// weights are rounded to one bf16 (the result's own type).
//
// Softmax, in one pass with a reference maximum m that is raised only when a
// score exceeds it by 2^8 (the first tile, and hardly ever after): exp2(s - m)
// <= 256 loses nothing in fp32. The first kernel then needs no reduction over
// the 128 threads of a query row but one vote a tile, and the sums of the weights
// come out of the second product where its A operand has room: for HD = 64 the
// instruction's rows 64 .. 127 are a constant block whose first row is ones, so
// lane 64 of O^T is sum p; for HD = 128 they stay per thread until the end. In the
// second kernel a row's statistics are its two threads' own.
//
// Overlap (one CTA an SM): one warp fills a ring of K and V tiles by TMA, one
// issues the MMAs, eight do the softmax, two threads for each lane of tensor
// memory. S is double buffered and so is P: S(i + 2) is issued behind PV(i), so
// neither product's latency stands in the softmax warps' way, and the order of
// the MMAs alone makes both buffers free in time.
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
// sequence are zeroed in shared memory, and so is a drafted row that holds a
// non-finite value, whose product is added at the end, element by element, for
// the rows that see it.
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

constexpr int kTile = 128;      // cache rows of a tile
constexpr int kCluster = 8;     // most splits joined in a cluster
constexpr int kSoft = 256;      // softmax threads: two for each of the 128 lanes of tensor memory
constexpr int kSoftWarps = kSoft / 32, kTmaWarp = kSoftWarps, kMmaWarp = kSoftWarps + 1;
constexpr int kAttnThreads = kSoft + 64;
constexpr int kHalfTile = kTile * 128;  // bytes of 128 rows x 64 dims
constexpr int kSmemMost = 232448;       // shared memory of a CTA
constexpr float kNone = -1e30f;         // the maximum of a row that has seen nothing
constexpr float kRaise = 8.f;           // a score this far above m (in powers of two) raises m

// Most splits joined through the workspace (tree_join keeps their statistics).
__host__ __device__ constexpr int max_splits(int nr) { return 4096 / nr < 64 ? 4096 / nr : 64; }

// Floats of one split's partial result in the workspace: O [NR][HD], the
// maxima and the sums [NR].
__host__ __device__ constexpr int64_t part_floats(int nr, int hd) { return (int64_t)nr * hd + 2 * nr; }

__device__ __forceinline__ float max_warp(float x) {
    float y;
    asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void soft_sync() { asm volatile("barrier.cta.sync 1, 256;" ::: "memory"); }
__device__ __forceinline__ bool soft_any(bool x) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, 1, 256, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)x)
        : "memory");
    return r != 0;
}

// The same between the two warps that share the rows of a lane quarter.
__device__ __forceinline__ bool pair_any(int quarter, bool x) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, %2, 64, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)x), "r"(2 + quarter)
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

// A drafted row, or one behind the sequence, in the V tile at v: thread `row`
// (the row of the tile) zeroes what the product must not see: rows behind the
// last node, and rows with a non-finite value, which it marks in `bad`.
template <int HD>
__device__ __forceinline__ void mend_v(uint8_t *v, int row, int node, int n, uint32_t *bad) {
    v += row * 128;
    bool zero = node >= n;
    if (!zero) {
        uint32_t inf = 0;
#pragma unroll
        for (int h = 0; h < HD / 64; ++h)
#pragma unroll
            for (int ch = 0; ch < 8; ++ch) {
                // (the lanes of a warp start at different chunks: rows are 128 bytes apart)
                const uint4 u = *reinterpret_cast<const uint4 *>(v + h * kHalfTile + ((ch + row) & 7) * 16);
                const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    inf |= (uint32_t)((w[e] & 0x7F80u) == 0x7F80u) | (uint32_t)((w[e] & 0x7F800000u) == 0x7F800000u);
            }
        if (inf) {
            zero = true;
            atomicOr(&bad[node >> 5], 1u << (node & 31));
        }
    }
    if (zero) {
#pragma unroll
        for (int h = 0; h < HD / 64; ++h)
#pragma unroll
            for (int ch = 0; ch < 8; ++ch)
                *reinterpret_cast<uint4 *>(v + h * kHalfTile + ((ch + row) & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
    }
}

// Element d of row r of a partial result: rows of HD floats, with SWZ their
// 16-byte chunks XOR-swizzled by the row (a thread then writes a whole row
// without bank conflicts).
template <int HD, bool SWZ>
__device__ __forceinline__ int o_at(int r, int d) {
    return r * HD + (SWZ ? ((((d >> 2) ^ (r & 7)) << 2) | (d & 3)) : d);
}

// The products of the drafted rows that mend_v took out, element by element
// for the rows that see them (the 128 softmax threads; a rare case).
template <int HD, int TERMS, bool SWZ>
__device__ __noinline__ void add_taken_out(const TreeArgs &a, int b, int kvh, int G, int row0, int rows, Seq sq,
                                           const uint32_t *bad, const float *mref, float *Os, int tid) {
    const float c = a.scale * 1.44269504088896340736f;
    const uint64_t left = bad[0] | ((uint64_t)bad[1] << 32);
    const int64_t base = ((int64_t)sq.slot * a.Hkv + kvh) * a.max_seq * HD;
    for (int i = tid; i < rows * HD; i += kSoft) {
        const int r = i / HD, d = i % HD, rg = row0 + r;
        const int64_t qat = b * a.q_batch + (rg / G) * a.q_token + (int64_t)(kvh * G + rg % G) * HD;
        for (uint64_t w = left & a.masks[(int64_t)b * a.T + rg / G]; w; w &= w - 1) {
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
            float *o = Os + o_at<HD, SWZ>(r, d);
            *o = fmaf(ex2(fmaf(x, c, -mref[r])), bf_lo(a.vc[at + d]), *o);
        }
    }
}

// Barriers and words of a CTA, at the front of its fixed shared memory. The
// ring's unit 2i is tile i's K, unit 2i + 1 its V; U units.
template <int U>
struct Sync {
    uint64_t full[U], free[U];
    // (two of each by the tile's parity: warps of the softmax may be a tile ahead of
    // others, and a wait must never be two phases behind)
    uint64_t s_full[2], p_full[2], o_done[2];
    uint32_t tmem;
    int err, issued;   // a wait ran out; units whose copies went out
    uint32_t bad[2];   // drafted rows taken out of the second product
};

template <int U>
__device__ __forceinline__ void init_sync(Sync<U> *y) {
    for (int u = 0; u < U; ++u) {
        mbar_init(&y->full[u], 1);
        mbar_init(&y->free[u], 1);
    }
    mbar_init(&y->s_full[0], 1);
    mbar_init(&y->s_full[1], 1);
    mbar_init(&y->p_full[0], kSoftWarps);
    mbar_init(&y->p_full[1], kSoftWarps);
    mbar_init(&y->o_done[0], 1);
    mbar_init(&y->o_done[1], 1);
    y->err = y->issued = 0;
    y->bad[0] = y->bad[1] = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    async_fence();
}

// The copies of unit u into its place in the ring.
template <int HD, int U>
__device__ __forceinline__ void load_unit(Sync<U> *y, uint8_t *ring, const CUtensorMap *kmap, const CUtensorMap *vmap,
                                          int u, int t0, int plane) {
    uint64_t *bar = &y->full[u % U];
    uint8_t *at = ring + (u % U) * (kHalfTile * (HD / 64));
    mbar_expect_tx(bar, kHalfTile * (HD / 64));
#pragma unroll
    for (int h = 0; h < HD / 64; ++h)
        tma_load_3d(at + h * kHalfTile, (u & 1) ? vmap : kmap, h * 64, (t0 + u / 2) * kTile, plane, bar);
    *(volatile int *)&y->issued = u + 1;
}

// After a wait ran out: the copies that were issued land before the shared
// memory goes.
template <int U>
__device__ __noinline__ void drain(Sync<U> *y, int *status) {
    const int n = *(volatile int *)&y->issued;
    for (int u = max(0, n - U); u < n; ++u) {
        const uint64_t from = gtimer();
        while (!mbar_try(&y->full[u % U], (u / U) & 1))
            if (gtimer() - from > kWaitNs) break;
    }
    if (status) atomicExch(status, 1);
}

// What a CTA does with its partial result (O in Os, maxima, sums): leaves it
// in the workspace for tree_join, or joins it with the cluster's other splits:
// first every split's maxima and sums, then the rows, shared out over the CTAs.
template <int HD, int TERMS, int NR, bool SWZ>
__device__ __forceinline__ void finish(const TreeArgs &a, int b, int kvh, int G, int row0, int rows, int split, int S,
                                       float *Os, float *mref, float *lsum, float *join) {
    namespace cg = cooperative_groups;
    const int tid = threadIdx.x;
    if (a.part) {
        const int64_t unit = (int64_t)blockIdx.z * gridDim.y + blockIdx.y;
        float *p = a.part + (unit * S + split) * part_floats(NR, HD);
        for (int i = tid; i < rows * (HD / 4); i += kAttnThreads) {
            const int r = i / (HD / 4), d = 4 * (i % (HD / 4));
            reinterpret_cast<float4 *>(p)[i] = *reinterpret_cast<const float4 *>(Os + o_at<HD, SWZ>(r, d));
        }
        for (int r = tid; r < rows; r += kAttnThreads) {
            p[NR * HD + r] = mref[r];
            p[NR * HD + NR + r] = lsum[r];
        }
        return;
    }
    float *wgt = join, *m8 = wgt + kCluster * NR, *l8 = m8 + kCluster * NR;
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
        float4 o[kCluster];
#pragma unroll
        for (int s = 0; s < kCluster; ++s)
            if (s < S) o[s] = *reinterpret_cast<const float4 *>(cl.map_shared_rank(Os + o_at<HD, SWZ>(r, d), s));
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int s = 0; s < kCluster; ++s)
            if (s < S) {
                const float w = wgt[s * NR + r];
                y.x = fmaf(w, o[s].x, y.x), y.y = fmaf(w, o[s].y, y.y);
                y.z = fmaf(w, o[s].z, y.z), y.w = fmaf(w, o[s].w, y.w);
            }
        put4<TERMS>(a, b * a.o_batch + (rg / G) * a.o_token + (int64_t)(kvh * G + rg % G) * HD + d, y);
    }
    if (S > 1) cl.sync();  // nobody leaves while its memory is read
}

// Eight elements of query row rg (node rg / G, head rg % G of the group) as
// TERMS bf16 terms; zeros behind the last node. fp32 queries are scaled here.
template <int HD, int TERMS>
__device__ __forceinline__ void load_query8(const TreeArgs &a, int b, int kvh, int G, int rg, int ch, float c,
                                            uint4 (&t)[TERMS]) {
    const bool in = rg < a.T * G;
    const int64_t at = b * a.q_batch + (rg / G) * a.q_token + (int64_t)(kvh * G + rg % G) * HD + 8 * ch;
    if constexpr (TERMS == 1) {
        t[0] = make_uint4(0u, 0u, 0u, 0u);
        if (in) t[0] = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.q) + at);
    } else {
        float x[8] = {};
        if (in) {
            const float4 *q = reinterpret_cast<const float4 *>(static_cast<const float *>(a.q) + at);
            const float4 u = q[0], v = q[1];
            x[0] = u.x * c, x[1] = u.y * c, x[2] = u.z * c, x[3] = u.w * c;
            x[4] = v.x * c, x[5] = v.y * c, x[6] = v.z * c, x[7] = v.w * c;
        }
        split8<TERMS>(x, t);
    }
}

template <int HD, int TERMS, int NR>
struct AttnShape {
    static constexpr int N = TERMS * NR;
    static constexpr int kKv = kHalfTile * (HD / 64);    // bytes of a K (or V) tile
    static constexpr int kP = ((N + 63) / 64) * kHalfTile;  // of a tile's weights; two of them
    static constexpr int kQ = N * HD * 2;
    static constexpr int kCols = 3 * N <= 64 ? 64 : 3 * N <= 128 ? 128 : 3 * N <= 256 ? 256 : 512;
    static constexpr int kOnes = HD == 64 ? 2048 : 0;  // 16 cache rows x 64: ones in the first column
    static constexpr int kMisc = 512 + 8 * NR + 8 * MK_MAX_TREE + 4 * NR * (3 + 4);
    static constexpr int kRoom = (kSmemMost - 1024 - 2 * kP - kQ - kOnes - kMisc) / kKv;
    static constexpr int U = kRoom > 8 ? 8 : kRoom;
    static constexpr int kOffP = U * kKv, kOffQ = kOffP + 2 * kP, kOffOnes = kOffQ + kQ, kOffMisc = kOffOnes + kOnes;
    static constexpr int kSmem = 1024 + kOffMisc + kMisc;
    static_assert(N % 16 == 0 && N <= 256 && 3 * N <= 512 && U >= 4, "the instruction's N, tensor and shared memory");
    static_assert(NR * HD * 4 + 3 * kCluster * NR * 4 <= U * kKv, "the partial result fits the ring");
};

template <int HD, int TERMS, int NR>
__global__ void __launch_bounds__(kAttnThreads, 1)
    tree_attention(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap, const TreeArgs a) {
    using C = AttnShape<HD, TERMS, NR>;
    constexpr int N = C::N, U = C::U, HR = NR / 2;  // HR: query rows of a softmax thread
    constexpr bool kScaled = TERMS > 1;             // the queries carry the scale already
    constexpr bool kOnes = HD == 64;                // the sums come out of the second product
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *Ps = sm + C::kOffP, *Qs = sm + C::kOffQ;
    Sync<U> *y = reinterpret_cast<Sync<U> *>(sm + C::kOffMisc);
    static_assert(sizeof(Sync<U>) <= 512, "");
    volatile int *err = &y->err;
    uint64_t *seen = reinterpret_cast<uint64_t *>(sm + C::kOffMisc + 512);  // [MK_MAX_TREE] bit r: row r sees it
    float *mref = reinterpret_cast<float *>(seen + MK_MAX_TREE), *corr = mref + NR, *lsum = corr + NR;
    float *wtmp = lsum + NR;                    // [4][NR]
    float *Os = reinterpret_cast<float *>(sm);  // [NR][HD], in the ring when the tiles are done
    float *join = Os + NR * HD;                 // [3][kCluster][NR] behind it

    const int tid = threadIdx.x, warp = warp_index(), lane = tid & 31;
    const int split = blockIdx.x, S = gridDim.x;
    const int b = blockIdx.y / a.Hkv, kvh = blockIdx.y % a.Hkv, G = a.Hq / a.Hkv;
    const int row0 = blockIdx.z * NR;
    const float c = a.scale * 1.44269504088896340736f;  // scores in powers of two
    const Seq sq = sequence(a, b);
    const uint64_t word = tid < NR && row0 + tid < a.T * G ? a.masks[(int64_t)b * a.T + (row0 + tid) / G] : 0;
    if (warp < kSoftWarps) {
        // The queries as the B operand: row term * NR + r, 128-byte swizzled. (Rows
        // of nodes behind the sequence's last one are columns nobody reads.)
        for (int i = tid; i < NR * (HD / 8); i += kSoft) {
            const int r = i / (HD / 8), ch = i % (HD / 8);
            uint4 t[TERMS];
            load_query8<HD, TERMS>(a, b, kvh, G, row0 + r, ch, c, t);
#pragma unroll
            for (int k = 0; k < TERMS; ++k) {
                const int n = k * NR + r;
                *reinterpret_cast<uint4 *>(Qs + (ch / 8) * (N * 128) + n * 128 + (((ch % 8) ^ (n & 7)) << 4)) = t[k];
            }
        }
    }
    const int rows = min(NR, sq.n * G - row0);
    if (rows <= 0) return;  // the whole cluster
    const int total = sq.len + sq.n, tiles = (total + kTile - 1) / kTile;
    const int t0 = (int)((int64_t)split * tiles / S), nt = (int)((int64_t)(split + 1) * tiles / S) - t0;
    const int plane = sq.slot * a.Hkv + kvh;
    if (warp == kTmaWarp) {
        if (elect()) {
            init_sync(y);
            // the first copies need nobody else
            for (int u = 0; u < min(2 * nt, U); ++u) load_unit<HD>(y, sm, &kmap, &vmap, u, t0, plane);
        }
    } else if (warp == kMmaWarp) {
        tmem_alloc(&y->tmem, C::kCols);
        if constexpr (kOnes)
            for (int i = lane; i < C::kOnes / 16; i += 32)  // chunk 0 of row i / 8 sits at chunk (row & 7)
                *reinterpret_cast<uint4 *>(sm + C::kOffOnes + i * 16) =
                    make_uint4(i % 8 == ((i / 8) & 7) ? 0x3F80u : 0u, 0u, 0u, 0u);
    } else {
        if (tid < NR) {
            mref[tid] = kNone;
            lsum[tid] = 0.f;
        }
        if ((t0 + nt) * kTile > sq.len && warp * 32 < NR) {  // a split with drafted rows: the masks by drafted row
            const uint64_t mine = tid < rows ? word : 0;
            uint32_t *out = reinterpret_cast<uint32_t *>(seen) + warp;
            for (int j = 0; j < sq.n; ++j) {
                const uint32_t w = __ballot_sync(0xFFFFFFFFu, (mine >> j) & 1);
                if (lane == 0) out[2 * j] = w;
            }
        }
    }
    async_fence();
    tc_fence_before();
    __syncwarp();
    __syncthreads();
    tc_fence_after();
    const uint32_t tS = uniform(y->tmem), tO = tS + 2 * N;

    if (warp == kTmaWarp) {
        for (int u = U; u < 2 * nt; ++u) {
            if (!__all_sync(0xFFFFFFFFu, mbar_wait(&y->free[u % U], ((u / U) - 1) & 1, err))) break;
            if (elect()) load_unit<HD>(y, sm, &kmap, &vmap, u, t0, plane);
            __syncwarp();
        }
    } else if (warp == kMmaWarp) {
        constexpr uint32_t idS = idesc_bf16(N, false, false), idO = idesc_bf16(N, true, true);
        const uint64_t q = sw128_desc(saddr(Qs), 16);
        const uint32_t ring = saddr(sm), ones = saddr(sm + C::kOffOnes), p0 = saddr(Ps);
        auto scores = [&](int i) {
            const int u = 2 * i;
            if (!__all_sync(0xFFFFFFFFu, mbar_wait(&y->full[u % U], (u / U) & 1, err))) return false;
            tc_fence_after();
            const uint64_t k = sw128_desc(ring + (u % U) * C::kKv, 16);
            if (elect()) {
#pragma unroll
                for (int kk = 0; kk < HD / 16; ++kk)
                    umma_bf16(tS + (i & 1) * N, k + (((kk / 4) * kHalfTile + (kk % 4) * 32) >> 4),
                              q + (((kk / 4) * (N * 128) + (kk % 4) * 32) >> 4), idS, kk != 0);
                umma_commit(&y->free[u % U]);
                umma_commit(&y->s_full[i & 1]);
            }
            __syncwarp();
            return true;
        };
        bool ok = nt > 0 && scores(0) && (nt < 2 || scores(1));
        for (int i = 0; i < nt && ok; ++i) {
            const int u = 2 * i + 1;
            ok = mbar_wait(&y->p_full[i & 1], (i >> 1) & 1, err) && mbar_wait(&y->full[u % U], (u / U) & 1, err);
            if (!(ok = __all_sync(0xFFFFFFFFu, ok))) break;
            tc_fence_after();
            // (the k-th product's first atom moves on by 2048 bytes, so the constant
            // block behind it comes nearer)
            const uint32_t va = ring + (u % U) * C::kKv;
            const uint64_t v = sw128_desc(va, kOnes ? ones - va : kHalfTile);
            const uint64_t p = sw128_desc(p0 + (i & 1) * C::kP, kHalfTile);
            if (elect()) {
#pragma unroll
                for (int kk = 0; kk < kTile / 16; ++kk)
                    umma_bf16(tO, v + ((kk * 2048) >> 4) - (kOnes ? (uint64_t)((kk * 2048) >> 4) << 16 : 0),
                              p + ((kk * 2048) >> 4), idO, (i | kk) != 0);
                umma_commit(&y->free[u % U]);
                umma_commit(&y->o_done[i & 1]);
            }
            __syncwarp();
            if (i + 2 < nt) ok = scores(i + 2);
        }
    } else {
        // thread: cache row `row` of the tile, query rows h0 .. h0 + HR - 1
        const int row = tid & (kTile - 1), h0 = (tid / kTile) * HR, quarter = warp & 3;
        const uint32_t mylane = (uint32_t)(quarter * 32) << 16;
        const float4 *m4 = reinterpret_cast<const float4 *>(mref + h0);
        float l[kOnes ? 1 : HR];
        if constexpr (!kOnes)
#pragma unroll
            for (int r = 0; r < HR; ++r) l[r] = 0.f;
        bool ok = true;
        for (int i = 0; i < nt; ++i) {
            // (a wait that ran out: the loop goes on, its barriers matched, and
            // the result becomes NaN)
            ok &= mbar_wait(&y->s_full[i & 1], (i >> 1) & 1, err);
            tc_fence_after();
            float s[TERMS * HR];
            const uint32_t ts = tS + (i & 1) * N + mylane + h0;
#pragma unroll
            for (int k = 0; k < TERMS; ++k) {
                if constexpr (HR == 8) {
                    tmem_ld8(ts + k * NR, s + k * HR);
                } else {
#pragma unroll
                    for (int r0 = 0; r0 < HR; r0 += 16) tmem_ld16(ts + k * NR + r0, s + k * HR + r0);
                }
            }
            tmem_ld_wait();
            pin<TERMS * HR>(s);
#pragma unroll
            for (int r = 0; r < HR; ++r)
#pragma unroll
                for (int k = 1; k < TERMS; ++k) s[r] += s[k * HR + r];
            const int at = (t0 + i) * kTile;
            const bool tail = at + kTile > sq.len;  // drafted rows, or the end
            const int node = at + row - sq.len;
            if (tail && node >= 0) {
                const uint64_t w = node < sq.n ? seen[node] >> h0 : 0;
#pragma unroll
                for (int r = 0; r < HR; ++r)
                    if (!((w >> r) & 1)) s[r] = -INFINITY;
            }
            // x = s - m in powers of two, and the largest of them
            float x[HR];
            auto shift = [&]() {
                float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int r = 0; r < HR; r += 4) {
                    const float4 m = m4[r / 4];
                    x[r] = kScaled ? s[r] - m.x : fmaf(s[r], c, -m.x);
                    x[r + 1] = kScaled ? s[r + 1] - m.y : fmaf(s[r + 1], c, -m.y);
                    x[r + 2] = kScaled ? s[r + 2] - m.z : fmaf(s[r + 2], c, -m.z);
                    x[r + 3] = kScaled ? s[r + 3] - m.w : fmaf(s[r + 3], c, -m.w);
                    top[(r / 4) & 3] = fmaxf(fmaxf(fmaxf(x[r], x[r + 1]), fmaxf(x[r + 2], x[r + 3])), top[(r / 4) & 3]);
                }
                return fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
            };
            if (soft_any(shift() > kRaise)) {
                // raise the maxima to those of all cache rows so far
#pragma unroll
                for (int r = 0; r < HR; ++r) {
                    const float w = max_warp(kScaled ? s[r] : s[r] * c);
                    if (lane == (r & 31)) wtmp[quarter * NR + h0 + r] = w;
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
                shift();
                if constexpr (!kOnes)
#pragma unroll
                    for (int r = 0; r < HR; ++r) l[r] *= corr[h0 + r];
                if (i > 0) {
                    ok &= mbar_wait(&y->o_done[(i - 1) & 1], ((i - 1) >> 1) & 1, err);
                    tc_fence_after();
#pragma unroll 1
                    for (int n0 = tid < kTile ? 0 : 16; n0 < N; n0 += 32) {
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
            }
            if (tail && tid < kTile) {
                const int u = 2 * i + 1;
                ok &= mbar_wait(&y->full[u % U], (u / U) & 1, err);
                if (node >= 0) mend_v<HD>(sm + (u % U) * C::kKv, row, node, sq.n, y->bad);
            }
            // the weights as the B operand: row = cache row, column = term * NR + r
            // (PV(i - 2), which read this buffer, is behind: S(i) was issued after it)
            uint8_t *p = Ps + (i & 1) * C::kP + row * 128;
#pragma unroll
            for (int r0 = 0; r0 < HR; r0 += 8) {
                float w[8];
                uint4 t[TERMS];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    w[e] = ex2(x[r0 + e]);
                    if constexpr (!kOnes) l[r0 + e] += w[e];
                }
                split8<TERMS>(w, t);
#pragma unroll
                for (int k = 0; k < TERMS; ++k) {
                    const int ch = (k * NR + h0 + r0) / 8;
                    *reinterpret_cast<uint4 *>(p + (ch / 8) * kHalfTile + (((ch % 8) ^ (row & 7)) << 4)) = t[k];
                }
            }
            async_fence();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&y->p_full[i & 1]);
        }
        if (nt > 0) ok &= mbar_wait(&y->o_done[(nt - 1) & 1], ((nt - 1) >> 1) & 1, err);
        tc_fence_after();
        const bool all = !soft_any(!ok);
        if constexpr (!kOnes) {
            // the sums of the 128 cache rows, warp by warp
#pragma unroll
            for (int r = 0; r < HR; ++r) {
                float w = l[r];
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) w += __shfl_xor_sync(0xFFFFFFFFu, w, o);
                if (lane == (r & 31)) wtmp[quarter * NR + h0 + r] = w;
            }
        }
        // O^T: lane = head dim (lane 64 of a head of 64: the sums), column = term * NR + r
        if (quarter * 32 < HD || (kOnes && quarter == 2)) {
#pragma unroll 1
            for (int r0 = tid < kTile ? 0 : 16; r0 < NR; r0 += 32) {
                float o[16];
                if (nt > 0) {
                    float w[16 * TERMS];
#pragma unroll
                    for (int k = 0; k < TERMS; ++k) tmem_ld16(tO + mylane + k * NR + r0, w + 16 * k);
                    tmem_ld_wait();
                    pin<16 * TERMS>(w);
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        o[e] = w[16 * (TERMS - 1) + e];
#pragma unroll
                        for (int k = TERMS - 2; k >= 0; --k) o[e] += w[16 * k + e];
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 16; ++e) o[e] = 0.f;
                }
                if (quarter * 32 < HD) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) Os[(r0 + e) * HD + quarter * 32 + lane] = o[e];
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
        if (y->bad[0] | y->bad[1]) add_taken_out<HD, TERMS, false>(a, b, kvh, G, row0, rows, sq, y->bad, mref, Os, tid);
    }
    __syncwarp();
    __syncthreads();
    if (*err && tid == 0) drain(y, a.err);
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_free(tS, C::kCols);
    }
    finish<HD, TERMS, NR, false>(a, b, kvh, G, row0, rows, split, S, Os, mref, lsum, join);
}

constexpr int kRows = 128;

// Bit e: a row with mask `word` sees the cache row `first` + e, counted from
// the first drafted one (those before it are seen by all).
__device__ __forceinline__ uint32_t seen32(uint64_t word, int first) {
    if (first >= 64) return 0u;
    if (first >= 0) return (uint32_t)(word >> first);
    return first > -32 ? (uint32_t)(word << -first) | ((1u << -first) - 1u) : 0xFFFFFFFFu;
}

template <int HD, int TERMS>
struct RowShape {
    static constexpr int kKv = kHalfTile * (HD / 64);
    static constexpr int kQ = TERMS * kKv;  // 128 rows x HD a term
    // Tensor memory: two buffers of scores, whose 64 columns of a half tile
    // become the half's weights (32 columns each of the first two terms), two of
    // the third term, and O.
    static constexpr int kThird = TERMS > 2 ? kTile / 2 : 0;
    static constexpr int kCols = 512;
    static constexpr int kMisc = 512 + 2 * 4 * kRows;
    static constexpr int kRoom = (kSmemMost - 1024 - kQ - kMisc) / kKv;
    static constexpr int U = kRoom > 8 ? 8 : kRoom;
    static constexpr int kOffQ = U * kKv, kOffMisc = kOffQ + kQ;
    static constexpr int kSmem = 1024 + kOffMisc + kMisc;
    static_assert(2 * kTile + 2 * kThird + HD <= kCols && U >= 4, "tensor and shared memory of an SM");
    static_assert(kRows * HD * 4 + (3 * kCluster + 2) * kRows * 4 <= U * kKv, "the partial result fits the ring");
};

template <int HD, int TERMS>
__global__ void __launch_bounds__(kAttnThreads, 1)
    tree_attention_rows(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                        const TreeArgs a) {
    using C = RowShape<HD, TERMS>;
    constexpr int U = C::U;
    constexpr bool kScaled = TERMS > 1;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *Qs = sm + C::kOffQ;
    Sync<U> *y = reinterpret_cast<Sync<U> *>(sm + C::kOffMisc);
    static_assert(sizeof(Sync<U>) <= 512, "");
    volatile int *err = &y->err;
    float *tops = reinterpret_cast<float *>(sm + C::kOffMisc + 512);  // [2][128] the halves' maxima
    float *Os = reinterpret_cast<float *>(sm);                        // in the ring when the tiles are done,
    float *join = Os + kRows * HD;                                    // and behind it
    float *mref = join + 3 * kCluster * kRows, *lsum = mref + kRows;

    const int tid = threadIdx.x, warp = warp_index(), lane = tid & 31;
    const int split = blockIdx.x, S = gridDim.x;
    const int b = blockIdx.y / a.Hkv, kvh = blockIdx.y % a.Hkv, G = a.Hq / a.Hkv;
    const int row0 = blockIdx.z * kRows;
    const float c = a.scale * 1.44269504088896340736f;
    const Seq sq = sequence(a, b);
    const int row = tid & (kRows - 1), half = (tid / kRows) & 1;  // a softmax thread's query row and half of a tile
    uint64_t word = row0 + row < a.T * G ? a.masks[(int64_t)b * a.T + (row0 + row) / G] : 0;
    if (warp < kSoftWarps) {
        // the queries as the A operand: term k, 128-byte swizzled rows of 64 dims
        for (int i = tid; i < kRows * (HD / 8); i += kSoft) {
            const int r = i / (HD / 8), ch = i % (HD / 8);
            uint4 t[TERMS];
            load_query8<HD, TERMS>(a, b, kvh, G, row0 + r, ch, c, t);
#pragma unroll
            for (int k = 0; k < TERMS; ++k)
                *reinterpret_cast<uint4 *>(Qs + k * C::kKv + (ch / 8) * kHalfTile + r * 128 +
                                           (((ch % 8) ^ (r & 7)) << 4)) = t[k];
        }
    }
    const int rows = min(kRows, sq.n * G - row0);
    if (rows <= 0) return;  // the whole cluster
    const int total = sq.len + sq.n, tiles = (total + kTile - 1) / kTile;
    const int t0 = (int)((int64_t)split * tiles / S), nt = (int)((int64_t)(split + 1) * tiles / S) - t0;
    const int plane = sq.slot * a.Hkv + kvh;
    if (warp == kTmaWarp) {
        if (elect()) {
            init_sync(y);
            for (int u = 0; u < min(2 * nt, U); ++u) load_unit<HD>(y, sm, &kmap, &vmap, u, t0, plane);
        }
    } else if (warp == kMmaWarp) {
        tmem_alloc(&y->tmem, C::kCols);
    }
    async_fence();
    tc_fence_before();
    __syncwarp();
    __syncthreads();
    tc_fence_after();
    const uint32_t tS = uniform(y->tmem), tT = tS + 2 * kTile, tO = tT + 2 * C::kThird;

    if (warp == kTmaWarp) {
        for (int u = U; u < 2 * nt; ++u) {
            if (!__all_sync(0xFFFFFFFFu, mbar_wait(&y->free[u % U], ((u / U) - 1) & 1, err))) break;
            if (elect()) load_unit<HD>(y, sm, &kmap, &vmap, u, t0, plane);
            __syncwarp();
        }
    } else if (warp == kMmaWarp) {
        constexpr uint32_t idS = idesc_bf16(kTile, false, false), idO = idesc_bf16(HD, false, true);
        const uint64_t q = sw128_desc(saddr(Qs), 16);
        const uint32_t ring = saddr(sm);
        auto scores = [&](int i) {
            const int u = 2 * i;
            if (!__all_sync(0xFFFFFFFFu, mbar_wait(&y->full[u % U], (u / U) & 1, err))) return false;
            tc_fence_after();
            const uint64_t k = sw128_desc(ring + (u % U) * C::kKv, 16);
            if (elect()) {
#pragma unroll
                for (int t = 0; t < TERMS; ++t)
#pragma unroll
                    for (int kk = 0; kk < HD / 16; ++kk) {
                        const uint32_t at = (kk / 4) * kHalfTile + (kk % 4) * 32;
                        umma_bf16(tS + (i & 1) * kTile, q + ((t * C::kKv + at) >> 4), k + (at >> 4), idS, (t | kk) != 0);
                    }
                umma_commit(&y->free[u % U]);
                umma_commit(&y->s_full[i & 1]);
            }
            __syncwarp();
            return true;
        };
        bool ok = nt > 0 && scores(0) && (nt < 2 || scores(1));
        for (int i = 0; i < nt && ok; ++i) {
            const int u = 2 * i + 1;
            ok = mbar_wait(&y->p_full[i & 1], (i >> 1) & 1, err) && mbar_wait(&y->full[u % U], (u / U) & 1, err);
            if (!(ok = __all_sync(0xFFFFFFFFu, ok))) break;
            tc_fence_after();
            const uint64_t v = sw128_desc(ring + (u % U) * C::kKv, kHalfTile);
            if (elect()) {
#pragma unroll
                for (int t = 0; t < TERMS; ++t)
#pragma unroll
                    for (int kk = 0; kk < kTile / 16; ++kk) {
                        const uint32_t p = t < 2 ? tS + (i & 1) * kTile + (kk / 4) * 64 + t * 32 + (kk % 4) * 8
                                                 : tT + (i & 1) * C::kThird + kk * 8;
                        umma_bf16_ta(tO, p, v + ((kk * 2048) >> 4), idO, (i | t | kk) != 0);
                    }
                umma_commit(&y->free[u % U]);
                umma_commit(&y->o_done[i & 1]);
            }
            __syncwarp();
            if (i + 2 < nt) ok = scores(i + 2);
        }
    } else {
        const int quarter = warp & 3, half0 = half * (kTile / 2);
        const uint32_t mylane = (uint32_t)(quarter * 32) << 16;
        const bool live = quarter * 32 < rows;  // (rows behind the last: the warp only keeps the barriers)
        if (sq.n < 64) word &= (1ull << sq.n) - 1;
        float m = kNone, l = 0.f;
        bool ok = true;
        for (int i = 0; i < nt; ++i) {
            ok &= mbar_wait(&y->s_full[i & 1], (i >> 1) & 1, err);
            tc_fence_after();
            const int at = (t0 + i) * kTile;
            const bool tail = at + kTile > sq.len;
            if (live) {
                const uint32_t ts = tS + (i & 1) * kTile + half0 + mylane;
                float x[64];
                auto read = [&]() {
#pragma unroll
                    for (int e = 0; e < 64; e += 16) tmem_ld16(ts + e, x + e);
                    tmem_ld_wait();
                    pin<64>(x);
                    if (tail) {
#pragma unroll
                        for (int w = 0; w < 64; w += 32) {
                            const uint32_t see = seen32(word, at + half0 + w - sq.len);
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                if (!((see >> e) & 1)) x[w + e] = -INFINITY;
                        }
                    }
                };
                auto largest = [&]() {
                    float t4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int e = 0; e < 64; e += 8)
#pragma unroll
                        for (int w = 0; w < 4; ++w) t4[w] = fmaxf(fmaxf(t4[w], x[e + 2 * w]), x[e + 2 * w + 1]);
                    return fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3]));
                };
                read();
                const float top = kScaled ? largest() : largest() * c;  // (the scale is positive)
                if (pair_any(quarter, top > m + kRaise)) {
                    // raise the maxima of these rows to those so far; scale O and the sums
                    tops[half * kRows + row] = top;
                    pair_any(quarter, false);
                    const float best = fmaxf(fmaxf(m, top), tops[(half ^ 1) * kRows + row]);
                    const float scale = ex2(m - best);
                    m = best;
                    l *= scale;
                    if (i > 0) {
                        ok &= mbar_wait(&y->o_done[(i - 1) & 1], ((i - 1) >> 1) & 1, err);
                        tc_fence_after();
#pragma unroll 1
                        for (int d = half * (HD / 2); d < (half + 1) * (HD / 2); d += 16) {
                            float o[16];
                            tmem_ld16(tO + mylane + d, o);
                            tmem_ld_wait();
                            pin<16>(o);
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[e] *= scale;
                            tmem_st16(tO + mylane + d, o);
                        }
                    }
                    pair_any(quarter, false);  // (tops is read before it is written again)
                }
                float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int w0 = 0; w0 < 64; w0 += 32) {
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        x[w0 + e] = ex2(kScaled ? x[w0 + e] - m : fmaf(x[w0 + e], c, -m));
                        sum[e & 3] += x[w0 + e];
                    }
#pragma unroll
                    for (int t = 0; t < TERMS; ++t) {
                        uint32_t w[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            float &x0 = x[w0 + 2 * e], &x1 = x[w0 + 2 * e + 1];
                            w[e] = pack_bf16(x0, x1);
                            if (t + 1 < TERMS) {
                                x0 -= bf_lo(w[e]);
                                x1 -= bf_hi(w[e]);
                            }
                        }
                        tmem_st16((t < 2 ? ts + t * 32 : tT + (i & 1) * C::kThird + half * 32 + mylane) + w0 / 2, w);
                    }
                }
                l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
                tmem_st_wait();
            }
            tc_fence_before();
            if (tail && half == 0) {
                const int u = 2 * i + 1, node = at + row - sq.len;
                ok &= mbar_wait(&y->full[u % U], (u / U) & 1, err);
                if (node >= 0) mend_v<HD>(sm + (u % U) * C::kKv, row, node, sq.n, y->bad);
                async_fence();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&y->p_full[i & 1]);
        }
        if (nt > 0) ok &= mbar_wait(&y->o_done[(nt - 1) & 1], ((nt - 1) >> 1) & 1, err);
        tc_fence_after();
        const bool all = !soft_any(!ok);  // (and every copy has landed: the ring is free)
        if (half == 1) tops[row] = l;
        if (live) {
#pragma unroll 1
            for (int d = half * (HD / 2); d < (half + 1) * (HD / 2); d += 16) {
                float o[16];
                if (nt > 0) {
                    tmem_ld16(tO + mylane + d, o);
                    tmem_ld_wait();
                    pin<16>(o);
                } else {
#pragma unroll
                    for (int e = 0; e < 16; ++e) o[e] = 0.f;
                }
#pragma unroll
                for (int e = 0; e < 16; e += 4)
                    *reinterpret_cast<float4 *>(Os + o_at<HD, true>(row, d + e)) =
                        make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
            }
        }
        soft_sync();
        if (half == 0) {
            mref[row] = m;
            lsum[row] = all ? l + tops[row] : __uint_as_float(0x7FC00000u);  // a wait ran out: NaN
        }
        if (y->bad[0] | y->bad[1]) {
            soft_sync();
            add_taken_out<HD, TERMS, true>(a, b, kvh, G, row0, rows, sq, y->bad, mref, Os, tid);
        }
    }
    __syncwarp();
    __syncthreads();
    if (*err && tid == 0) drain(y, a.err);
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_free(tS, C::kCols);
    }
    finish<HD, TERMS, kRows, true>(a, b, kvh, G, row0, rows, split, S, Os, mref, lsum, join);
}

// Joins the S splits' partial results of every (row tile, sequence, kv head):
// grid (row tiles, batch * Hkv), a thread per four dims of a row.
template <int HD, int TERMS, int NR>
__global__ void __launch_bounds__(256) tree_join(const TreeArgs a, int S) {
    constexpr int64_t PF = part_floats(NR, HD);
    __shared__ float ms[max_splits(NR) * NR], wg[max_splits(NR) * NR];
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
