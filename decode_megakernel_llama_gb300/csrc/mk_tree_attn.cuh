// mk_tree_attn.cuh — the attention kernels of a drafted tree (see mk_tree.cu).
//
// Two tcgen05 kernels share everything but which operand the queries are.
//
// tree_attention (few query rows, 16 or 32 a CTA): the CACHE is the A operand, so
// a tile's 128 cache rows (then 64 or 128 head dims) fill the instruction's 128
// rows whatever the number of queries, and all softmax threads have work even for
// one query row:
//   S^T [128 cache rows][N] = K [128][HD] . Q^T    (both K-major)
//   O^T [HD][N]            += V^T [HD][128] . P^T   (both MN-major: V as TMA wrote
//                                                    it, P as the threads write it)
// tree_attention_rows (many): 128 query rows are the A operand,
//   S [128 rows][128 cache rows] = Q . K^T, O [128 rows][HD] += P . V,
// P from tensor memory (for fp32 queries where the scores were).
// Measured (MMAs back to back): an instruction of M = 128 costs the larger of
// 44 cycles, its share of shared-memory reads (4 KB of A and 32 N bytes of B at
// 128 B a cycle) and N / 2 cycles, and a chain of 8 is seen complete ~340
// cycles after its last issue. So the first form pays 56 cycles an instruction
// for 32 fp32 rows (N = 96) and the second 64 for 128 rows, and none of its P
// passes through shared memory.
//
// What bounds them: the first, for a long cache, memory (131,079 rows of 8 kv heads
// of 128: 86.0 us = 6.24 TB/s, 0.93 of the measured copy rate); for a short one
// latency (one token over 191 rows: 5.8 us, of which the launch, the first copies
// and the join of two splits are all but 2). The second the softmax warps' time
// a tile, ~1,550 cycles against 960 of its MMAs and 530 of its exponentials at 31 a
// cycle (8 ragged sequences of up to 8,253 rows, 244 query rows, 64 dims: 58.2 us, of
// which the longest sequence's 65 tiles are 52): a warp's loads, maximum, weights
// and stores come one behind the other, and only two warps share a scheduler. The
// weights' second term costs a third of it (44.3 us with one).
//
// fp32 queries and weights enter as three bf16 terms each (24 bits: x = t0 + t1 +
// t2 to half a step of fp32): side by side in the first kernel's B operand, N =
// terms * NR, added in registers (S) and once at the end (O); as more instructions
// into the same accumulator in the second. bf16 queries are one term, exactly, and
// their weights two (16 bits, 2^-8 of half a step of the bf16 result). With one the
// weights' own rounding was as large as the result's: 0.0023 of the result's norm off
// against 0.0017, which is the rounding of the result alone.
//
// Softmax, in one pass with a reference maximum m that is raised only when a
// score exceeds it by 2^8 (the first tile, and hardly ever after): exp2(s - m)
// <= 256 loses nothing in fp32. The first kernel then needs no reduction over
// the 128 threads of a query row but one vote a tile, and the sums of the weights
// come out of the second product where its A operand has room: for HD = 64 the
// instruction's rows 64 .. 127 are a constant block whose first row is ones, so
// lane 64 of O^T is sum p; for HD = 128 they stay per thread until the end. In the
// second kernel a row's statistics are one thread's own.
//
// Overlap (one CTA an SM): two warps fill rings of K and V tiles by TMA, one issues
// the MMAs, and two groups of four softmax warps take the tiles in turn, each
// with its own buffers of S and P, its own maxima, sums and O (joined at the end
// like two splits), so neither a product's latency nor a group's votes stand in
// the other's way. With rings of four tiles or more and P apart from S, S runs
// three tiles ahead of PV and starts as soon as the scores before are read
// (64 fp32 rows over 8,208: 52.6 -> 44.2 us for one split); else S(i + 2), in the
// second kernel S(i + NB), is issued behind PV(i), and the order of the MMAs alone
// makes the buffers free in time. A commit of a product serves both who waits for its result and the ring's next copy.
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

// bf16 terms of a softmax weight, of queries of `terms`.
__host__ __device__ constexpr int weight_terms(int terms) { return terms == 1 ? 2 : terms; }

constexpr int kTile = 128;      // cache rows of a tile
constexpr int kCluster = 8;     // most splits joined in a cluster
constexpr int kGroup = 128;     // softmax threads of a group: one for each lane of tensor memory
constexpr int kSoft = 2 * kGroup;
// Warps: 0 issues the MMAs, 1 and 2 the copies of K and of V, 3 rests (a group's
// warps w have w & 3 as their quarter of tensor memory), 4 .. 11 do the softmax.
constexpr int kMmaWarp = 0, kKWarp = 1, kVWarp = 2, kFirstSoft = 4, kSoftWarps = kSoft / 32;
constexpr int kAttnThreads = kSoft + 32 * kFirstSoft;
constexpr int kHalfTile = kTile * 128;  // bytes of 128 rows x 64 dims
constexpr int kSmemMost = 232448;       // shared memory of a CTA
constexpr float kNone = -3e38f;         // the maximum of a row that has seen nothing
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

// Barriers of both groups, and of group g: a plain one, and a vote.
__device__ __forceinline__ void soft_sync() { asm volatile("barrier.cta.sync 1, 256;" ::: "memory"); }
__device__ __forceinline__ void group_sync(int g) { asm volatile("barrier.cta.sync %0, 128;" ::"r"(2 + g) : "memory"); }
__device__ __forceinline__ bool group_any(int g, bool x) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, %2, 128, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)x), "r"(2 + g)
        : "memory");
    return r != 0;
}

// (x, y) * c - m: two fp32 in one instruction.
__device__ __forceinline__ void fma2(float &x, float &y, float c, float mx, float my) {
    const float2 r = __ffma2_rn(make_float2(x, y), make_float2(c, c), make_float2(-mx, -my));
    x = r.x, y = r.y;
}

// (x, y) less the bf16 pair w: exact, one instruction for both.
__device__ __forceinline__ void less2(float &x, float &y, uint32_t w) {
    const float2 r = __ffma2_rn(make_float2(bf_lo(w), bf_hi(w)), make_float2(-1.f, -1.f), make_float2(x, y));
    x = r.x, y = r.y;
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
            if (k + 1 < TERMS) less2(x[2 * i], x[2 * i + 1], w[i]);
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

// Barriers and words of a CTA. The ring holds KU tiles of K, then VU of V.
template <int KU, int VU>
struct Sync {
    // full: the copies have landed; done: the product that reads them is (for K the
    // scores are there, for V the tile is in O)
    uint64_t k_full[KU], k_done[KU], v_full[VU], v_done[VU];
    // A group has read its scores, has written its weights (of a tile i: place i % 4, so
    // that a warp or the products, a tile of the group behind, are never two phases late)
    uint64_t s_read[2], p_full[4];
    uint64_t quiet;  // after a wait that ran out: every product that was issued is done
    uint32_t tmem;
    int err, k_issued, v_issued;  // a wait ran out; tiles whose copies went out
    uint32_t bad[2];              // drafted rows taken out of the second product
};

template <int KU, int VU>
__device__ __forceinline__ void init_sync(Sync<KU, VU> *y) {
    for (int u = 0; u < KU; ++u) {
        mbar_init(&y->k_full[u], 1);
        mbar_init(&y->k_done[u], 1);
    }
    for (int u = 0; u < VU; ++u) {
        mbar_init(&y->v_full[u], 1);
        mbar_init(&y->v_done[u], 1);
    }
    for (int g = 0; g < 2; ++g) {
        mbar_init(&y->s_read[g], kSoftWarps / 2);
        mbar_init(&y->p_full[g], kSoftWarps / 2);
        mbar_init(&y->p_full[g + 2], kSoftWarps / 2);
    }
    mbar_init(&y->quiet, 1);
    y->err = y->k_issued = y->v_issued = 0;
    y->bad[0] = y->bad[1] = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    async_fence();
}

// Waits for tile i's copies, or for its product. A waiter must not be two phases
// of a place in the ring behind: the tile before it in its place (2 or more
// before) has to be known to be done. The MMA and copy warps see every tile. A
// softmax group that awaits S(i) has seen S(i - 2), and with it every product
// issued before; one that awaits PV(i - 2) has awaited PV(i - 4), or knows it done by
// S(i - 2), or with three buffers by S(i), which was issued behind PV(i - 3). Of the
// last tile's PV that holds for the group of that tile; the other may pass early:
// what it reads comes behind a barrier with the first.
template <int KU, int VU>
__device__ __forceinline__ bool k_full(Sync<KU, VU> *y, int i, const Wait &w) {
    return mbar_wait(&y->k_full[i % KU], (i / KU) & 1, w);
}
template <int KU, int VU>
__device__ __forceinline__ bool v_full(Sync<KU, VU> *y, int i, const Wait &w) {
    return mbar_wait(&y->v_full[i % VU], (i / VU) & 1, w);
}
template <int KU, int VU>
__device__ __forceinline__ bool s_done(Sync<KU, VU> *y, int i, const Wait &w) {
    return mbar_wait(&y->k_done[i % KU], (i / KU) & 1, w);
}
template <int KU, int VU>
__device__ __forceinline__ bool pv_done(Sync<KU, VU> *y, int i, const Wait &w) {
    return mbar_wait(&y->v_done[i % VU], (i / VU) & 1, w);
}

// The copies of a K (or V) tile into its place in the ring.
template <int HD>
__device__ __forceinline__ void load_tile(uint8_t *at, const CUtensorMap *map, int row, int plane, uint64_t *bar) {
    mbar_expect_tx(bar, kHalfTile * (HD / 64));
#pragma unroll
    for (int h = 0; h < HD / 64; ++h) tma_load_3d(at + h * kHalfTile, map, h * 64, row, plane, bar);
}

// One lane's work: all of a split's K (or V) tiles, into the ring.
template <int HD, int KU, int VU>
__device__ __forceinline__ void load_all(Sync<KU, VU> *y, uint8_t *ring, const CUtensorMap *map, bool is_k, int from,
                                         int to, int t0, int plane, const Wait &w) {
    constexpr int kKv = kHalfTile * (HD / 64);
    for (int i = from; i < to; ++i) {
        if (is_k) {
            if (i >= KU && !s_done(y, i - KU, w)) break;
            load_tile<HD>(ring + (i % KU) * kKv, map, (t0 + i) * kTile, plane, &y->k_full[i % KU]);
            *(volatile int *)&y->k_issued = i + 1;
        } else {
            if (i >= VU && !pv_done(y, i - VU, w)) break;
            load_tile<HD>(ring + (KU + i % VU) * kKv, map, (t0 + i) * kTile, plane, &y->v_full[i % VU]);
            *(volatile int *)&y->v_issued = i + 1;
        }
    }
}

// After a wait that ran out, by the whole CTA behind a barrier: the products and copies
// that were issued (no thread issues more) are done before their shared and tensor
// memory goes, and before anything that the caller writes behind this. The products
// read no barrier and the copies wait for nobody, so both end by themselves; their
// own limit is the default one, however short the call's.
template <int KU, int VU>
__device__ __noinline__ void settle(Sync<KU, VU> *y, int *status) {
    auto land = [](uint64_t *bar, int units, int n) {
        for (int i = max(0, n - units); i < n; ++i) mbar_await(bar + i % units, (i / units) & 1);
    };
    const int warp = warp_index();
    if (warp == kMmaWarp) {
        if (elect()) {  // (the lane that issued them)
            umma_commit(&y->quiet);
            mbar_await(&y->quiet, 0);
        }
    } else if (warp == kKWarp) {
        if (elect()) {
            land(y->k_full, KU, *(volatile int *)&y->k_issued);
            land(y->v_full, VU, *(volatile int *)&y->v_issued);
            if (status) atomicExch(status, 1);
        }
    }
    __syncwarp();
    __syncthreads();
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
        pdl_trigger();  // (brought in earlier, tree_join's CTAs stand in the tiles' way: 86.6 -> 88.7 us at 131k rows)
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
    static constexpr int N = TERMS * NR, PN = weight_terms(TERMS) * NR;  // columns of S and of O
    static constexpr int kKv = kHalfTile * (HD / 64);    // bytes of a K (or V) tile
    static constexpr int kP = ((PN + 63) / 64) * kHalfTile;  // of a tile's weights; two of them
    static constexpr int kQ = N * HD * 2;
    static constexpr int kUsed = 2 * (N + PN), kCols = kUsed <= 64 ? 64 : kUsed <= 128 ? 128 : kUsed <= 256 ? 256 : 512;
    static constexpr int kOnes = HD == 64 ? 2048 : 0;  // 16 cache rows x 64: ones in the first column
    static constexpr int kMisc = 512 + 8 * MK_MAX_TREE + 4 * NR * (2 + 2 + 1 + 8);
    static constexpr int kRoom = (kSmemMost - 1024 - 2 * kP - kQ - kOnes - kMisc) / kKv;
    static constexpr int KU = (kRoom + 1) / 2 > 6 ? 6 : (kRoom + 1) / 2, VU = kRoom / 2 > 6 ? 6 : kRoom / 2;
    // With room for it S runs three tiles ahead of PV and starts as soon as the group
    // has read the scores before; else it follows PV(i), two tiles ahead.
    static constexpr bool kEarly = VU >= 4;
    static constexpr int kAhead = kEarly ? 3 : 2;
    static constexpr int kOffP = (KU + VU) * kKv, kOffQ = kOffP + 2 * kP, kOffOnes = kOffQ + kQ, kOffMisc = kOffOnes + kOnes;
    static constexpr int kSmem = 1024 + kOffMisc + kMisc;
    static_assert(N % 16 == 0 && PN % 16 == 0 && PN <= 256 && kUsed <= 512 && VU >= 2,
                  "the instruction's N, tensor and shared memory");
    static_assert(NR * HD * 4 + 3 * kCluster * NR * 4 <= (KU + VU) * kKv, "the partial result fits the ring");
};

template <int HD, int TERMS, int NR>
__global__ void __launch_bounds__(kAttnThreads, 1)
    tree_attention(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap, const TreeArgs a) {
    using C = AttnShape<HD, TERMS, NR>;
    constexpr int N = C::N, PT = weight_terms(TERMS), PN = C::PN, KU = C::KU, VU = C::VU;
    constexpr bool kScaled = TERMS > 1;             // the queries carry the scale already
    constexpr bool kOnes = HD == 64;                // the sums come out of the second product
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *Ps = sm + C::kOffP, *Qs = sm + C::kOffQ;
    Sync<KU, VU> *y = reinterpret_cast<Sync<KU, VU> *>(sm + C::kOffMisc);
    static_assert(sizeof(Sync<KU, VU>) <= 512, "");
    volatile int *err = &y->err;
    const Wait wt{err, a.wait_ns, a.wait_sleep};
    uint64_t *seen = reinterpret_cast<uint64_t *>(sm + C::kOffMisc + 512);  // [MK_MAX_TREE] bit r: row r sees it
    float *mref = reinterpret_cast<float *>(seen + MK_MAX_TREE), *corr = mref + 2 * NR;  // [2][NR] of the groups
    float *lsum = corr + 2 * NR;                // [NR]
    float *wtmp = lsum + NR;                    // [2][4][NR]
    float *Os = reinterpret_cast<float *>(sm);  // [NR][HD], in the ring when the tiles are done
    float *join = Os + NR * HD;                 // [3][kCluster][NR] behind it

    const int tid = threadIdx.x, warp = warp_index(), lane = tid & 31;
    const int split = blockIdx.x, S = gridDim.x;
    const int b = blockIdx.y / a.Hkv, kvh = blockIdx.y % a.Hkv, G = a.Hq / a.Hkv;
    const int row0 = blockIdx.z * NR;
    const float c = a.scale * 1.44269504088896340736f;  // scores in powers of two
    pdl_wait();
    if (!a.part) pdl_trigger();
    const Seq sq = sequence(a, b);
    const int first = threadIdx.x - kFirstSoft * 32;
    const uint64_t word =
        first >= 0 && first < NR && row0 + first < a.T * G ? a.masks[(int64_t)b * a.T + (row0 + first) / G] : 0;
    if (warp >= kFirstSoft) {
        // The queries as the B operand: row term * NR + r, 128-byte swizzled. (Rows
        // of nodes behind the sequence's last one are columns nobody reads.)
        for (int i = first; i < NR * (HD / 8); i += kSoft) {
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
    if (warp == kKWarp) {
        if (elect()) {
            init_sync(y);
            // the first copies need nobody else
            load_all<HD>(y, sm, &kmap, true, 0, min(nt, KU), t0, plane, wt);
            load_all<HD>(y, sm, &vmap, false, 0, min(nt, VU), t0, plane, wt);
        }
    } else if (warp == kMmaWarp) {
        tmem_alloc(&y->tmem, C::kCols);
        if constexpr (kOnes)
            for (int i = lane; i < C::kOnes / 16; i += 32)  // chunk 0 of row i / 8 sits at chunk (row & 7)
                *reinterpret_cast<uint4 *>(sm + C::kOffOnes + i * 16) =
                    make_uint4(i % 8 == ((i / 8) & 7) ? 0x3F80u : 0u, 0u, 0u, 0u);
    } else if (warp >= kFirstSoft) {
        if (first < 2 * NR) mref[first] = kNone;
        if ((t0 + nt) * kTile > sq.len && first < ((NR + 31) & ~31)) {  // a split with drafted rows: their masks
            const uint64_t mine = first < rows ? word : 0;
            uint32_t *out = reinterpret_cast<uint32_t *>(seen) + first / 32;
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
    const uint32_t tS = uniform(y->tmem), tO = tS + 2 * N;  // S and O of group g: + g * N, + g * PN

    if (warp == kKWarp) {
        if (elect()) load_all<HD>(y, sm, &kmap, true, KU, nt, t0, plane, wt);
    } else if (warp == kVWarp) {
        if (elect()) load_all<HD>(y, sm, &vmap, false, VU, nt, t0, plane, wt);
    } else if (warp == kMmaWarp) {
        constexpr uint32_t idS = idesc_bf16(N, false, false), idO = idesc_bf16(PN, true, true);
        const uint64_t q = sw128_desc(saddr(Qs), 16);
        const uint32_t ring = saddr(sm), ones = saddr(sm + C::kOffOnes), p0 = saddr(Ps);
        auto scores = [&](int i) {
            const uint64_t k = sw128_desc(ring + (i % KU) * C::kKv, 16);
#pragma unroll
            for (int kk = 0; kk < HD / 16; ++kk)
                umma_bf16(tS + (i & 1) * N, k + (((kk / 4) * kHalfTile + (kk % 4) * 32) >> 4),
                          q + (((kk / 4) * (N * 128) + (kk % 4) * 32) >> 4), idS, kk != 0);
            umma_commit(&y->k_done[i % KU]);
        };
        if (elect()) {
            bool ok = true;
            // the scores of tile i (early: once the group has read those of i - 2)
            for (int i = 0; i < min(nt, C::kAhead) && ok; ++i) {
                ok = k_full(y, i, wt) && (i < 2 || mbar_wait(&y->s_read[i & 1], ((i >> 1) - 1) & 1, wt));
                tc_fence_after();
                if (ok) scores(i);
            }
            for (int i = 0; i < nt && ok; ++i) {
                const int j = i + C::kAhead;
                if (C::kEarly && j < nt) {
                    ok = k_full(y, j, wt) && mbar_wait(&y->s_read[j & 1], ((j >> 1) - 1) & 1, wt);
                    tc_fence_after();
                    if (ok) scores(j);
                }
                // (the k-th product's first atom moves on by 2048 bytes, so the constant
                // block behind it comes nearer)
                const uint32_t va = ring + (KU + i % VU) * C::kKv;
                const uint64_t v = sw128_desc(va, kOnes ? ones - va : kHalfTile);
                const uint64_t p = sw128_desc(p0 + (i & 1) * C::kP, kHalfTile);
                if (!(ok = ok && v_full(y, i, wt) && mbar_wait(&y->p_full[i & 3], (i >> 2) & 1, wt))) break;
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < kTile / 16; ++kk)
                    umma_bf16(tO + (i & 1) * PN, v + ((kk * 2048) >> 4) - (kOnes ? (uint64_t)((kk * 2048) >> 4) << 16 : 0),
                              p + ((kk * 2048) >> 4), idO, i >= 2 || kk != 0);
                umma_commit(&y->v_done[i % VU]);
                if (!C::kEarly && j < nt) {
                    ok = k_full(y, j, wt);
                    tc_fence_after();
                    if (ok) scores(j);
                }
            }
        }
    } else if (warp >= kFirstSoft) {
        // group g takes every other tile; thread: cache row `row` of it, all query rows
        const int g = (warp - kFirstSoft) >> 2, quarter = warp & 3, row = quarter * 32 + lane;
        const uint32_t mylane = (uint32_t)(quarter * 32) << 16;
        const uint32_t ts = tS + g * N + mylane, to = tO + g * PN + mylane;
        float *gref = mref + g * NR, *gcorr = corr + g * NR, *gtmp = wtmp + g * 4 * NR;
        const float4 *m4 = reinterpret_cast<const float4 *>(gref);
        float l[kOnes ? 1 : NR];
        if constexpr (!kOnes)
#pragma unroll
            for (int r = 0; r < NR; ++r) l[r] = 0.f;
        bool ok = true;
        for (int i = g; i < nt; i += 2) {
            // (a wait that ran out: the loop goes on, its barriers matched, without
            // another wait, and the result becomes NaN)
            ok = ok && s_done(y, i, wt);
            tc_fence_after();
            float s[TERMS * NR];
#pragma unroll
            for (int n = 0; n < N; n += 16) tmem_ld16(ts + n, s + n);
            tmem_ld_wait();
            pin<N>(s);
            if (C::kEarly) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&y->s_read[g]);
            }
#pragma unroll
            for (int r = 0; r < NR; ++r)
#pragma unroll
                for (int k = 1; k < TERMS; ++k) s[r] += s[k * NR + r];
            const int at = (t0 + i) * kTile;
            const bool tail = at + kTile > sq.len;  // drafted rows, or the end
            const int node = at + row - sq.len;
            if (tail && node >= 0) {
                const uint64_t w = node < sq.n ? seen[node] : 0;
#pragma unroll
                for (int r = 0; r < NR; ++r)
                    if (!((w >> r) & 1)) s[r] = -INFINITY;
            }
            // x = s - m in powers of two, and the largest of them
            float x[NR];
            auto shift = [&]() {
                float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int r = 0; r < NR; r += 4) {
                    const float4 m = m4[r / 4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[r + e] = s[r + e];
                    fma2(x[r], x[r + 1], kScaled ? 1.f : c, m.x, m.y);
                    fma2(x[r + 2], x[r + 3], kScaled ? 1.f : c, m.z, m.w);
                    top[(r / 4) & 3] = fmaxf(fmaxf(fmaxf(x[r], x[r + 1]), fmaxf(x[r + 2], x[r + 3])), top[(r / 4) & 3]);
                }
                return fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
            };
            const bool raise = group_any(g, shift() > kRaise);
            // PV(i - 2) is done: P and O are this group's again (not early: S(i) was issued after it)
            if (C::kEarly && i >= 2) ok = ok && pv_done(y, i - 2, wt);
            if (raise) {
                // raise the maxima to those of all cache rows so far
#pragma unroll
                for (int r = 0; r < NR; ++r) {
                    const float w = max_warp(kScaled ? s[r] : s[r] * c);
                    if (lane == (r & 31)) gtmp[quarter * NR + r] = w;
                }
                group_sync(g);
                if (row < NR) {
                    const float old = gref[row];
                    const float m = fmaxf(fmaxf(fmaxf(gtmp[row], gtmp[NR + row]),
                                                fmaxf(gtmp[2 * NR + row], gtmp[3 * NR + row])), old);
                    gcorr[row] = ex2(old - m);
                    gref[row] = m;
                }
                group_sync(g);
                shift();
                if constexpr (!kOnes)
#pragma unroll
                    for (int r = 0; r < NR; ++r) l[r] *= gcorr[r];
                if (i >= 2) {
                    tc_fence_after();
#pragma unroll 1
                    for (int n0 = 0; n0 < PN; n0 += 16) {
                        float o[16];
                        tmem_ld16(to + n0, o);
                        tmem_ld_wait();
                        pin<16>(o);
#pragma unroll
                        for (int e = 0; e < 16; ++e) o[e] *= gcorr[n0 % NR + e];
                        tmem_st16(to + n0, o);
                    }
                    tmem_st_wait();
                }
            }
            if (tail) {
                ok = ok && v_full(y, i, wt);
                if (node >= 0) mend_v<HD>(sm + (KU + i % VU) * C::kKv, row, node, sq.n, y->bad);
            }
            // the weights as the B operand: row = cache row, column = term * NR + r
            uint8_t *p = Ps + g * C::kP + row * 128;
#pragma unroll
            for (int r0 = 0; r0 < NR; r0 += 8) {
                float w[8];
                uint4 t[PT];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    w[e] = ex2(x[r0 + e]);
                    if constexpr (!kOnes) l[r0 + e] += w[e];
                }
                split8<PT>(w, t);
#pragma unroll
                for (int k = 0; k < PT; ++k) {
                    const int ch = (k * NR + r0) / 8;
                    *reinterpret_cast<uint4 *>(p + (ch / 8) * kHalfTile + (((ch % 8) ^ (row & 7)) << 4)) = t[k];
                }
            }
            async_fence();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&y->p_full[i & 3]);
        }
        if (nt > 0) ok = ok && pv_done(y, nt - 1, wt);  // (and with it every product)
        tc_fence_after();
        if constexpr (!kOnes) {
            // the sums of the 128 cache rows, warp by warp
#pragma unroll
            for (int r = 0; r < NR; ++r) {
                float w = l[r];
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) w += __shfl_xor_sync(0xFFFFFFFFu, w, o);
                if (lane == (r & 31)) gtmp[quarter * NR + r] = w;
            }
        }
        soft_sync();
        tc_fence_after();  // (a group that passed early reads O behind the barrier, too)
        // the groups' factors to the larger maximum, which both keep
        float f0 = 0.f, f1 = 0.f;
        if (first < NR) {
            const float m = fmaxf(mref[first], mref[NR + first]);
            f0 = corr[first] = nt > 0 ? ex2(mref[first] - m) : 0.f;
            f1 = corr[NR + first] = nt > 1 ? ex2(mref[NR + first] - m) : 0.f;
            mref[first] = m;
            if constexpr (!kOnes)
                lsum[first] = f0 * ((wtmp[first] + wtmp[NR + first]) + (wtmp[2 * NR + first] + wtmp[3 * NR + first])) +
                            f1 * ((wtmp[4 * NR + first] + wtmp[5 * NR + first]) + (wtmp[6 * NR + first] + wtmp[7 * NR + first]));
        }
        soft_sync();
        // O^T: lane = head dim (lane 64 of a head of 64: the sums), column = term * NR + r
        if (quarter * 32 < HD || (kOnes && quarter == 2)) {
#pragma unroll 1
            for (int r0 = 16 * g; r0 < NR; r0 += 32) {
                float o[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] = 0.f;
#pragma unroll 1
                for (int h = 0; h < min(nt, 2); ++h) {
                    float w[16 * PT];
#pragma unroll
                    for (int k = 0; k < PT; ++k) tmem_ld16(tO + h * PN + mylane + k * NR + r0, w + 16 * k);
                    tmem_ld_wait();
                    pin<16 * PT>(w);
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        float z = w[16 * (PT - 1) + e];
#pragma unroll
                        for (int k = PT - 2; k >= 0; --k) z += w[16 * k + e];
                        o[e] = fmaf(corr[h * NR + r0 + e], z, o[e]);
                    }
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
        if (y->bad[0] | y->bad[1]) add_taken_out<HD, TERMS, false>(a, b, kvh, G, row0, rows, sq, y->bad, mref, Os, first);
    }
    tc_fence_before();
    __syncwarp();
    __syncthreads();
    if (*err) {  // a wait ran out (nobody waits any more: the same for all threads): the rows are NaN
        settle(y, a.err);
        if (tid < NR) lsum[tid] = __uint_as_float(0x7FC00000u);
        __syncthreads();
    }
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
    // Tensor memory: an O for each group, and NB buffers in which a tile's scores (128
    // columns) become its weights (64 columns each of the first two terms) beside a
    // third term of fp32. With three a group's next scores wait for the other group's last
    // second product, not for its own (8 ragged sequences, weights of one term: 49.1 ->
    // 44.3 us).
    static constexpr int kThird = TERMS > 2 ? kTile / 2 : 0, kCols = 512;
    static constexpr int NB = (kCols - 2 * HD) / (kTile + kThird) > 2 ? 3 : 2;
    static constexpr int kMisc = 512 + 2 * 4 * kRows;
    static constexpr int kRoom = (kSmemMost - 1024 - kQ - kMisc) / kKv;
    static constexpr int KU = (kRoom + 1) / 2 > 6 ? 6 : (kRoom + 1) / 2, VU = kRoom / 2 > 6 ? 6 : kRoom / 2;
    static constexpr int kOffQ = (KU + VU) * kKv, kOffMisc = kOffQ + kQ;
    static constexpr int kSmem = 1024 + kOffMisc + kMisc;
    static_assert(NB * (kTile + kThird) + 2 * HD <= kCols && VU >= NB && KU >= NB, "tensor and shared memory of an SM");
    static_assert(kRows * HD * 4 + 3 * kCluster * kRows * 4 <= (KU + VU) * kKv, "the partial result fits the ring");
};

template <int HD, int TERMS>
__global__ void __launch_bounds__(kAttnThreads, 1)
    tree_attention_rows(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                        const TreeArgs a) {
    using C = RowShape<HD, TERMS>;
    constexpr int KU = C::KU, VU = C::VU, NB = C::NB, PT = weight_terms(TERMS);
    constexpr bool kScaled = TERMS > 1;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *Qs = sm + C::kOffQ;
    Sync<KU, VU> *y = reinterpret_cast<Sync<KU, VU> *>(sm + C::kOffMisc);
    static_assert(sizeof(Sync<KU, VU>) <= 512, "");
    volatile int *err = &y->err;
    const Wait wt{err, a.wait_ns, a.wait_sleep};
    // [2][128]: the groups' maxima, then the rows' maxima and sums, each written by the thread that read what was there
    float *gm = reinterpret_cast<float *>(sm + C::kOffMisc + 512), *mref = gm, *lsum = gm + kRows;
    float *Os = reinterpret_cast<float *>(sm);                      // in the ring when the tiles are done,
    float *join = Os + kRows * HD;                                  // and behind it

    const int tid = threadIdx.x, warp = warp_index(), lane = tid & 31;
    const int split = blockIdx.x, S = gridDim.x;
    const int b = blockIdx.y / a.Hkv, kvh = blockIdx.y % a.Hkv, G = a.Hq / a.Hkv;
    const int row0 = blockIdx.z * kRows;
    const float c = a.scale * 1.44269504088896340736f;
    pdl_wait();
    if (!a.part) pdl_trigger();
    const Seq sq = sequence(a, b);
    const int row = (warp & 3) * 32 + lane;  // a softmax thread's query row
    uint64_t word = row0 + row < a.T * G ? a.masks[(int64_t)b * a.T + (row0 + row) / G] : 0;
    const int st = tid - kFirstSoft * 32;  // a softmax thread's index
    if (warp >= kFirstSoft) {
        // the queries as the A operand: term k, 128-byte swizzled rows of 64 dims
        for (int i = st; i < kRows * (HD / 8); i += kSoft) {
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
    if (warp == kKWarp) {
        if (elect()) {
            init_sync(y);
            // the first copies need nobody else
            load_all<HD>(y, sm, &kmap, true, 0, min(nt, KU), t0, plane, wt);
            load_all<HD>(y, sm, &vmap, false, 0, min(nt, VU), t0, plane, wt);
        }
    } else if (warp == kMmaWarp) {
        tmem_alloc(&y->tmem, C::kCols);
    }
    async_fence();
    tc_fence_before();
    __syncwarp();
    __syncthreads();
    tc_fence_after();
    // scores and third terms of tile i: + i % NB * 128, + i % NB * kThird; O of group g: + g * HD
    const uint32_t tS = uniform(y->tmem), tT = tS + NB * kTile, tO = tT + NB * C::kThird;

    if (warp == kKWarp) {
        if (elect()) load_all<HD>(y, sm, &kmap, true, KU, nt, t0, plane, wt);
    } else if (warp == kVWarp) {
        if (elect()) load_all<HD>(y, sm, &vmap, false, VU, nt, t0, plane, wt);
    } else if (warp == kMmaWarp) {
        constexpr uint32_t idS = idesc_bf16(kTile, false, false), idO = idesc_bf16(HD, false, true);
        const uint64_t q = sw128_desc(saddr(Qs), 16);
        const uint32_t ring = saddr(sm);
        auto scores = [&](int i) {
            const uint64_t k = sw128_desc(ring + (i % KU) * C::kKv, 16);
#pragma unroll
            for (int t = 0; t < TERMS; ++t)
#pragma unroll
                for (int kk = 0; kk < HD / 16; ++kk) {
                    const uint32_t at = (kk / 4) * kHalfTile + (kk % 4) * 32;
                    umma_bf16(tS + (i % NB) * kTile, q + ((t * C::kKv + at) >> 4), k + (at >> 4), idS, (t | kk) != 0);
                }
            umma_commit(&y->k_done[i % KU]);
        };
        if (elect()) {
            bool ok = true;
            for (int i = 0; i < min(nt, NB) && (ok = k_full(y, i, wt)); ++i) {
                tc_fence_after();
                scores(i);
            }
            for (int i = 0; i < nt && ok; ++i) {
                const int j = i + NB;
                const uint64_t v = sw128_desc(ring + (KU + i % VU) * C::kKv, kHalfTile);
                if (!(ok = ok && v_full(y, i, wt) && mbar_wait(&y->p_full[i & 3], (i >> 2) & 1, wt))) break;
                tc_fence_after();
#pragma unroll
                for (int t = 0; t < PT; ++t)
#pragma unroll
                    for (int kk = 0; kk < kTile / 16; ++kk) {
                        const uint32_t p = t < 2 ? tS + (i % NB) * kTile + t * 64 + kk * 8
                                                 : tT + (i % NB) * C::kThird + kk * 8;
                        umma_bf16_ta(tO + (i & 1) * HD, p, v + ((kk * 2048) >> 4), idO, i >= 2 || (t | kk) != 0);
                    }
                umma_commit(&y->v_done[i % VU]);
                if (j < nt) {  // (into the buffer of PV(i))
                    ok = k_full(y, j, wt);
                    tc_fence_after();
                    if (ok) scores(j);
                }
            }
        }
    } else if (warp >= kFirstSoft) {
        // group g takes every other tile, a thread one query row of it
        const int g = (warp - kFirstSoft) >> 2, quarter = warp & 3;
        const uint32_t mylane = (uint32_t)(quarter * 32) << 16;
        const uint32_t to = tO + g * HD + mylane;
        const bool live = quarter * 32 < rows;  // (rows behind the last: the warp only keeps the barriers)
        if (sq.n < 64) word &= (1ull << sq.n) - 1;
        float m = kNone, l = 0.f;
        bool ok = true;
        for (int i = g; i < nt; i += 2) {
            ok = ok && s_done(y, i, wt);
            tc_fence_after();
            const uint32_t ts = tS + (i % NB) * kTile + mylane, tt = tT + (i % NB) * C::kThird + mylane;
            const int at = (t0 + i) * kTile;
            const bool tail = at + kTile > sq.len;
            if (live) {
                float x[kTile];
#pragma unroll
                for (int e = 0; e < kTile; e += 16) tmem_ld16(ts + e, x + e);
                tmem_ld_wait();
                pin<kTile>(x);
                if (tail) {
#pragma unroll
                    for (int w = 0; w < kTile; w += 32) {
                        const uint32_t see = seen32(word, at + w - sq.len);
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (!((see >> e) & 1)) x[w + e] = -INFINITY;
                    }
                }
                float t4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int e = 0; e < kTile; e += 8)
#pragma unroll
                    for (int w = 0; w < 4; ++w) t4[w] = fmaxf(fmaxf(t4[w], x[e + 2 * w]), x[e + 2 * w + 1]);
                float top = fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3]));
                if (!kScaled) top *= c;  // (the scale is positive)
                if (__any_sync(0xFFFFFFFFu, top > m + kRaise)) {
                    // raise the warp's maxima to those of the rows so far; scale O and the sums
                    const float best = fmaxf(m, top), scale = ex2(m - best);
                    m = best;
                    l *= scale;
                    if (i >= 2) {
                        if (NB > 2) ok = ok && pv_done(y, i - 2, wt);  // O is this group's again (NB = 2: S(i) was issued behind it)
                        tc_fence_after();
#pragma unroll 1
                        for (int d = 0; d < HD; d += 16) {
                            float o[16];
                            tmem_ld16(to + d, o);
                            tmem_ld_wait();
                            pin<16>(o);
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[e] *= scale;
                            tmem_st16(to + d, o);
                        }
                    }
                }
                float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                for (int w0 = 0; w0 < kTile; w0 += 32) {
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        float &x0 = x[w0 + e], &x1 = x[w0 + e + 1];
                        fma2(x0, x1, kScaled ? 1.f : c, m, m);
                        x0 = ex2(x0);
                        x1 = ex2(x1);
                        sum[(e >> 1) & 1] = __ffma2_rn(make_float2(x0, x1), make_float2(1.f, 1.f), sum[(e >> 1) & 1]);
                    }
#pragma unroll
                    for (int t = 0; t < PT; ++t) {
                        uint32_t w[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            float &x0 = x[w0 + 2 * e], &x1 = x[w0 + 2 * e + 1];
                            w[e] = pack_bf16(x0, x1);
                            if (t + 1 < PT) less2(x0, x1, w[e]);
                        }
                        tmem_st16((t < 2 ? ts + t * 64 : tt) + w0 / 2, w);
                    }
                }
                l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
                tmem_st_wait();
            }
            tc_fence_before();
            if (tail) {
                const int node = at + row - sq.len;
                ok = ok && v_full(y, i, wt);
                if (node >= 0) mend_v<HD>(sm + (KU + i % VU) * C::kKv, row, node, sq.n, y->bad);
                async_fence();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&y->p_full[i & 3]);
        }
        if (nt > 0) ok = ok && pv_done(y, nt - 1, wt);  // (and with it every product: the ring is free)
        tc_fence_after();
        gm[g * kRows + row] = m;
        soft_sync();
        tc_fence_after();  // (a group that passed early reads O behind the barrier, too)
        // the groups' O to the larger maximum: group 0 writes, group 1 adds
        const float best = fmaxf(m, gm[(g ^ 1) * kRows + row]), scale = g < nt ? ex2(m - best) : 0.f;
        l *= scale;
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
            if (g == h) {
                if (live) {
#pragma unroll 1
                    for (int d = 0; d < HD; d += 16) {
                        float o[16];
                        if (g < nt) {
                            tmem_ld16(to + d, o);
                            tmem_ld_wait();
                            pin<16>(o);
                        } else {
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[e] = 0.f;
                        }
#pragma unroll
                        for (int e = 0; e < 16; e += 4) {
                            float4 *z = reinterpret_cast<float4 *>(Os + o_at<HD, true>(row, d + e));
                            float4 w = make_float4(0.f, 0.f, 0.f, 0.f);
                            if (h) w = *z;
                            w.x = fmaf(scale, o[e], w.x), w.y = fmaf(scale, o[e + 1], w.y);
                            w.z = fmaf(scale, o[e + 2], w.z), w.w = fmaf(scale, o[e + 3], w.w);
                            *z = w;
                        }
                    }
                }
                lsum[row] = h ? lsum[row] + l : l;
                if (h) mref[row] = best;
            }
            soft_sync();
        }
        if (y->bad[0] | y->bad[1]) add_taken_out<HD, TERMS, true>(a, b, kvh, G, row0, rows, sq, y->bad, mref, Os, st);
    }
    tc_fence_before();
    __syncwarp();
    __syncthreads();
    if (*err) {  // a wait ran out (nobody waits any more: the same for all threads): the rows are NaN
        settle(y, a.err);
        if (tid < kRows) lsum[tid] = __uint_as_float(0x7FC00000u);
        __syncthreads();
    }
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
    pdl_begin();  // (behind it the splits' partial results are there)
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
