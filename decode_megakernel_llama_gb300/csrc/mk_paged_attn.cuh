// mk_paged_attn.cuh — the attention kernels over a cache in pages (see mk_paged.cu).
//
// The two tcgen05 kernels of a drafted tree (mk_tree_attn.cuh, whose head states the
// products, the softmax in one pass, the overlap and what a wait that runs out does),
// with what ragged sequences in pages need instead of a tree in a slot:
//   - a CTA finds its sequence and rows from `starts` (find_work), so the grid
//     follows the tokens, not the longest sequence: a batch of one prompt and many
//     single tokens has no empty CTAs to speak of;
//   - a tile of 128 rows is one TMA box a page (16 pages of 8 rows at most, a lane
//     each), the page numbers read a tile ahead; pages that are not there, and what
//     lies behind the sequence, are boxes outside the map, which read as zeros;
//   - tiles that no row of the CTA sees (behind the last token, before the window)
//     are not visited, those that all rows see whole take no mask; the others, five at
//     most (Span), select scores and clean V;
//   - 8-bit pages (Q8): more warps (eight, with many rows four) read codes and powers, put the
//     bf16 values, which are exact, where TMA puts them, and from there on all is as with bf16.
//     So their products are those of the bf16 kernel and only the bytes are half.
#pragma once
#include "mk_tree_attn.cuh"

namespace mkops {

// Threads: four warps for products and copies, the softmax warps (few rows: two groups of
// four; many: of eight, two to 32 rows), and for 8-bit pages those that convert them.
constexpr int kRowSoft = 512;
__host__ __device__ constexpr int soft_threads(bool many) { return many ? kRowSoft : kSoft; }
__host__ __device__ constexpr int conv_warps(bool many) { return many ? 4 : 8; }
constexpr int kParts = 5, kBadRows = kParts * kTile, kBadWords = kBadRows / 32;

__host__ __device__ constexpr int first_conv(bool many) { return kFirstSoft + soft_threads(many) / 32; }
__host__ __device__ constexpr int paged_threads(bool many, bool q8) {
    return 32 * (first_conv(many) + (q8 ? conv_warps(many) : 0));
}
template <bool MANY>
__device__ __forceinline__ bool is_soft(int warp) {
    return warp >= kFirstSoft && warp < first_conv(MANY);
}

// A CTA's rows: query rows row0 .. row0 + rows - 1 of sequence b (row = token of the
// sequence * G + head of the group), whose n tokens begin at tok0 of the call's.
struct Work {
    int b, n, len, tok0, row0, rows;
};

// The grid's places of tiles of NR rows: sequence b's begin at starts[b] * G / NR + min(b, starts[b]), so
// that each has room for its tiles, an empty one takes none, and they rise with b.
__device__ __forceinline__ int place(int b, int start, int NR, int G) { return start * G / NR + min(b, start); }

// (x) the first of y <= 32 sequences that place u is one of's, of more than 32, by a whole warp: a
// 32nd of them is left each time, so two rounds of loads for 1,024, four for 2^20. (Counting the tiles
// of all sequences before took 0.3 ms for 1,024 sequences of 20 rows, 40 ms for 16,384; now 0.2 and 2.8.)
static __device__ __noinline__ int2 narrow(const int32_t *starts, int B, int n, int u, int NR, int G, int lane) {
    int lo = 0, size = B;
    while (size > 32) {
        const int step = (size + 31) / 32, b = lo + lane * step;
        const bool in = lane * step < size && place(b, min(max(starts[b], 0), n), NR, G) <= u;
        const uint32_t m = __ballot_sync(0xFFFFFFFFu, in);
        const int skip = m ? (31 - __clz(m)) * step : 0;
        lo += skip, size = min(step, size - skip);
    }
    return make_int2(lo, size);
}

// The tile of NR rows at place u, by a whole warp; rows = 0: an empty place. A sequence's
// last rows, which see the most, come first.
__device__ __forceinline__ Work find_work(const PagedArgs &a, int u, int NR, int G, int lane) {
    Work w;
    int2 in = make_int2(0, a.B);
    if (a.B > 32) in = narrow(a.starts, a.B, a.n, u, NR, G, lane);
    const int b = in.x + lane;
    int lo = 0, n = 0, len = 0, at = 0;
    if (lane < in.y) {
        lo = min(max(a.starts[b], 0), a.n);
        n = max(min(max(a.starts[b + 1], 0), a.n) - lo, 0);
        len = min(max(a.lengths[b], 0), a.cap);
        at = place(b, lo, NR, G);
    }
    const uint32_t m = __ballot_sync(0xFFFFFFFFu, lane < in.y && at <= u);
    const int first = __shfl_sync(0xFFFFFFFFu, at, 0), l = m ? 31 - __clz(m) : 0;
    w.b = in.x + l;
    w.n = __shfl_sync(0xFFFFFFFFu, n, l);
    w.len = __shfl_sync(0xFFFFFFFFu, len, l);
    w.tok0 = __shfl_sync(0xFFFFFFFFu, lo, l);
    w.row0 = __shfl_sync(0xFFFFFFFFu, (at + (n * G + NR - 1) / NR - 1 - u) * NR, l);  // (behind its tiles: below 0)
    w.rows = first <= u && w.row0 >= 0 ? min(NR, w.n * G - w.row0) : 0;
    w.row0 = max(w.row0, 0);  // (an empty place's queries are read, too)
    // (else the compiler forms them anew in the loops: a chunk of tokens over 8-bit pages 91.1 -> 97.5 us)
    asm volatile("" : "+r"(w.row0), "+r"(w.rows), "+r"(w.b), "+r"(w.n), "+r"(w.len), "+r"(w.tok0));
    return w;
}

// Bits below n of 32.
__device__ __forceinline__ uint32_t below(int n) { return n <= 0 ? 0u : n >= 32 ? 0xFFFFFFFFu : (1u << n) - 1u; }

// The cache rows that a CTA's tokens, at positions p0 .. p1 (p1 - p0 < 128), see: its
// tiles in order are the ns that hold the first `sinks` rows, then those from wt on.
struct Span {
    int base, p0, p1, end, window, sinks, ns, wt, tiles, last;  // base: position of token 0; last: of the CTA, + 1
    __device__ __forceinline__ int tile(int v) const { return v < ns ? v : wt + v - ns; }
    // Which of the kParts tiles that not all rows see whole; -1: all do. (0: the end of
    // the first rows; 1, 2: where the windows begin; 3, 4: where the tokens stand.)
    __device__ __forceinline__ int part(int t) const {
        const int at = t * kTile;
        if (window && at <= p1 - window && at + kTile > sinks) return t < wt ? 0 : 1 + t - wt;
        return at + kTile > p0 + 1 ? 3 + t - max(p0 + 1, 0) / kTile : -1;
    }
    __device__ __forceinline__ int tile_of_part(int k) const {
        return k == 0 ? ns - 1 : k < 3 ? wt + k - 1 : max(p0 + 1, 0) / kTile + k - 3;
    }
    __device__ __forceinline__ bool sees(int pos, int j) const {
        return j <= pos && (!window || j > pos - window || j < sinks);
    }
    __device__ __forceinline__ bool somebody(int j) const {
        return j < end && (!window || j > p0 - window || j < sinks);
    }
    // The query rows of the CTA that see cache row j: [lo, hi).
    __device__ __forceinline__ void columns(int j, int G, int row0, int &lo, int &hi) const {
        lo = max(j - base, 0) * G - row0;
        hi = last * G - row0;
        if (window && j >= sinks) hi = min(max(j - base + window, 0), last) * G - row0;
    }
    // Bit e: the token at pos sees row j + e.
    __device__ __forceinline__ uint32_t sees32(int pos, int j) const {
        uint32_t m = below(pos + 1 - j);
        if (window) m &= ~below(pos - window + 1 - j) | below(sinks - j);
        return m;
    }
};

__device__ __forceinline__ Span span_of(const PagedArgs &a, const Work &w, int G) {
    Span s;
    s.base = w.len - w.n;
    s.last = (w.row0 + w.rows - 1) / G + 1;
    s.p0 = s.base + w.row0 / G;
    s.p1 = s.base + s.last - 1;
    s.end = max(s.p1 + 1, 0);
    s.window = a.window, s.sinks = a.sinks;
    s.wt = a.window ? max(s.p0 - a.window + 1, 0) / kTile : 0;
    s.ns = a.window ? min((min(a.sinks, s.end) + kTile - 1) / kTile, s.wt) : 0;
    s.tiles = s.ns + max((s.end + kTile - 1) / kTile - s.wt, 0);
    return s;
}

// The sequence's queries and results as those of one tree.
template <int TERMS>
__device__ __forceinline__ TreeArgs tree_args(const PagedArgs &a, const Work &w) {
    constexpr int kBytes = TERMS == 1 ? 2 : 4;
    TreeArgs t{};
    t.T = w.n, t.Hq = a.Hq, t.Hkv = a.Hkv, t.scale = a.scale, t.part = a.part;
    t.q_token = a.q_stride, t.o_token = a.o_stride;
    t.q = static_cast<const uint8_t *>(a.q) + w.tok0 * a.q_stride * kBytes;
    t.out = static_cast<uint8_t *>(a.out) + w.tok0 * a.o_stride * kBytes;
    return t;
}

// Row j of sequence b in the pool, counted in rows; -1 on a page that is not there.
__device__ __forceinline__ int64_t pool_row(const PagedArgs &a, int b, int kvh, int j) {
    const int p = j >> a.shift, page = a.table[(int64_t)b * a.max_pages + p];
    if (page < 0 || page >= a.n_pages) return -1;
    return ((int64_t)page * a.Hkv + kvh) * a.ps + (j - (int)((int64_t)p << a.shift));
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

// The CTA's barriers and words, by a whole warp. (landers: arrivals that make a tile of K,
// or of V, full; warps: of a softmax group)
template <int KU, int VU>
__device__ __forceinline__ void init_paged(Sync<KU, VU> *y, uint32_t *bad, int landers, int warps, int lane) {
    static_assert(KU <= 8 && VU <= 8 && kBadWords <= 32, "");
    if (lane < KU) mbar_init(&y->k_full[lane], landers), mbar_init(&y->k_done[lane], 1);
    if (lane < VU) mbar_init(&y->v_full[lane], landers), mbar_init(&y->v_done[lane], 1);
    if (lane < 2) mbar_init(&y->s_read[lane], warps);
    if (lane < 4) mbar_init(&y->p_full[lane], warps);
    if (lane < kBadWords) bad[lane] = 0;
    if (lane < 2) y->bad[lane] = 0;
    if (lane == 0) {
        mbar_init(&y->quiet, 1);
        y->err = y->k_issued = y->v_issued = 0;
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    async_fence();
    __syncwarp();
}

__device__ __forceinline__ bool any_bad(const uint32_t *bad) {
    uint32_t x = 0;
#pragma unroll
    for (int i = 0; i < kBadWords; ++i) x |= bad[i];
    return x != 0;
}

// A warp's work: tiles from .. to - 1 of a split's K (or V), a box of a page a lane. (The
// lanes' copies go out one behind the other, ~48 cycles each: before the CTA's first
// barrier only one tile's do; all that the rings hold took 6,000 cycles there.)
template <int HD, int KU, int VU>
__device__ __forceinline__ void load_pages(Sync<KU, VU> *y, uint8_t *ring, const CUtensorMap *map, bool is_k,
                                           const PagedArgs &a, int b, int kvh, const Span &sp, int t0, int from, int to,
                                           int lane, const Wait &w) {
    constexpr int kKv = kHalfTile * (HD / 64), kHalves = HD / 64;
    const int parts = max(kTile >> a.shift, 1), rows = kTile / parts;
    const int part = lane / kHalves, half = lane % kHalves;
    const bool mine = lane < parts * kHalves;
    const int32_t *table = a.table + (int64_t)b * a.max_pages;
    int at_row = 0, page = a.n_pages;  // of this lane's box
    auto look = [&](int i) {
        const int j = sp.tile(t0 + i) * kTile + part * rows;
        page = a.n_pages;
        if (mine && j < sp.end) page = table[j >> a.shift];
        at_row = a.shift < 31 ? j & (a.ps - 1) : j;
    };
    if (from < to) look(from);
    for (int i = from; i < to; ++i) {
        const bool there = page >= 0 && page < a.n_pages;
        const int plane = (there ? page : a.n_pages) * a.Hkv + kvh, row = at_row;
        if (i + 1 < to) look(i + 1);
        const int u = is_k ? i % KU : i % VU;
        bool ok = true;
        if (is_k ? i >= KU : i >= VU) ok = is_k ? s_done(y, i - KU, w) : pv_done(y, i - VU, w);
        if (!__all_sync(0xFFFFFFFFu, ok)) break;
        uint64_t *bar = is_k ? &y->k_full[u] : &y->v_full[u];
        if (lane == 0) {
            mbar_expect_tx(bar, kKv);
            *(volatile int *)(is_k ? &y->k_issued : &y->v_issued) = i + 1;
        }
        __syncwarp();
        if (mine)
            tma_load_3d(ring + (is_k ? u : KU + u) * kKv + half * kHalfTile + part * rows * 128, map, half * 64, row,
                        plane, bar);
    }
}

// ---- 8-bit pages. A warp for K and one for V copy codes and powers as they lie in the
// pages into rings of stages (bulk copies: a page of a head is contiguous), and the
// converting warps, half of them for K, half for V, make bf16 tiles of them in the products'
// own ring. With `split` the two halves of a tile have rings and warps of their own, so
// that a warp waits, reads and hands over once a tile.
// Measured, a token a sequence, heads of 64 and 128, us a tile: loads into registers a
// tile ahead 1.06, 1.75; one ring of K and V in turn 1.05, 1.45; rings for each, whole
// tiles 0.75 and (halves, for want of room) 1.43; split rings 0.92, 1.23; each warp's own
// copies, bulk 1.20, 1.53, cp.async 0.92, 1.64.
struct Form {  // of an instance
    int rows, stages;  // of a stage; of a ring
    bool split;
};
constexpr int kMostStages = 3;
__host__ __device__ constexpr Form form_of(bool many, int hd, int terms, int nr = 0) {
    // (heads of 128 have room for split rings beside packed weights only)
    return hd == 64 ? Form{128, many && terms > 1 ? 2 : 3, false}
                    : !many && weight_terms(terms) * nr <= 32 ? Form{64, 2, true} : Form{64, 3, false};
}
__host__ __device__ constexpr int stage_bytes(Form f, int hd) { return f.rows * (hd + hd / 32); }
__host__ __device__ constexpr int less_bytes(bool q8, Form f, int hd) {
    return q8 ? 2 * (f.split ? 2 : 1) * f.stages * stage_bytes(f, hd) : 0;
}

struct Stages {  // [K, V][half]
    uint64_t full[2][2][kMostStages], free[2][2][kMostStages];
    uint32_t there[2][2][kMostStages];  // a stage's parts (of a page each) that hold rows of the pool; the others are zeros
    int issued[2][2];
};
constexpr int kOwnBytes = 4 * kBadWords + 256;  // of a CTA: bad rows, and this
static_assert(sizeof(Stages) <= 256 && 4 * kBadWords % 8 == 0, "");

__device__ __forceinline__ void init_stages(Stages *g, int readers, int lane) {
    if (lane < 4 * kMostStages) {
        mbar_init(&g->full[0][0][0] + lane, 1);
        mbar_init(&g->free[0][0][0] + lane, readers);
    }
    if (lane < 4) (&g->issued[0][0])[lane] = 0;
}

// A copying warp: all of a split's K (o = 0) or V.
template <int HD, int HR, int N, bool SPLIT>
__device__ __forceinline__ void stage_pages(Stages *g, uint8_t *stages, int o, const PagedArgs &a, int b, int kvh,
                                            const Span &sp, int t0, int nt, int lane, const Wait &w) {
    constexpr int PER = kTile / HR, kBytes = HR * (HD + HD / 32);
    static_assert(!SPLIT || PER == 2, "");
    const int parts = max(HR >> a.shift, 1), rows = HR / parts, n_items = PER * nt;
    const int32_t *table = a.table + (int64_t)b * a.max_pages;
    const uint8_t *codes = static_cast<const uint8_t *>(o ? a.vc : a.kc), *scales = o ? a.vs : a.ks;
    stages += o * (SPLIT ? 2 : 1) * N * kBytes;
    auto row_of = [&](int e) {
        if (lane >= parts || e >= n_items) return -1;
        const int j = sp.tile(t0 + e / PER) * kTile + e % PER * HR + lane * rows;
        return j < sp.end ? j : -1;
    };
    auto ask = [&](int j) { return j < 0 ? -1 : table[j >> a.shift]; };
    int next = row_of(0), page_next = ask(next);  // (the page is asked for an item before it is used)
    int u = 0;                                    // stage, and whether its last reader is waited for
    uint32_t phase = 0;
    bool used = false;
    for (int e = 0; e < n_items; ++e) {
        const int j = next, page = page_next, half = SPLIT ? e & 1 : 0;
        next = row_of(e + 1);
        page_next = ask(next);
        const bool ok = !used || mbar_wait(&g->free[o][half][u], phase, w);
        if (!__all_sync(0xFFFFFFFFu, ok)) return;
        const bool there = j >= 0 && page >= 0 && page < a.n_pages;
        const uint32_t mask = __ballot_sync(0xFFFFFFFFu, there);
        const int at = a.shift < 31 ? j & (a.ps - 1) : j, n = min(rows, a.ps - at);  // row of the page, rows
        uint64_t *full = &g->full[o][half][u];
        if (lane == 0) {
            g->there[o][half][u] = mask;
            mbar_expect_tx(full, (parts > 1 ? __popc(mask) * rows : there ? n : 0) * (HD + HD / 32));
            *(volatile int *)&g->issued[o][half] = (SPLIT ? e / 2 : e) + 1;
        }
        __syncwarp();
        if (there) {
            uint8_t *to = stages + (half * N + u) * kBytes;
            const int64_t from = ((int64_t)page * a.Hkv + kvh) * a.ps + at;
            bulk_load(to + lane * rows * HD, codes + from * HD, n * HD, full);
            bulk_load(to + HR * HD + lane * rows * (HD / 32), scales + from * (HD / 32), n * (HD / 32), full);
        }
        if ((!SPLIT || half == 1) && ++u == N) {
            u = 0;
            if (used) phase ^= 1;
            used = true;
        }
    }
}

// One of W converting warps: its rows of every tile of K (who < W / 2) or V as bf16
// values into the ring, 128-byte swizzled as TMA writes it. A lane takes 16 elements at a
// time of every eighth row; of heads of 128 neighbouring rows' lanes take different
// halves, so that the eight lanes that read or write at once meet in no bank.
// (The next stage's codes read before these are widened: 0.83 for 0.75 us a tile.)
template <int HD, int KU, int VU, int W, int HR, int NS, bool SPLIT>
__device__ __forceinline__ void convert_pages(Sync<KU, VU> *y, uint8_t *ring, Stages *g, const uint8_t *stages,
                                              const PagedArgs &a, int nt, int who, int lane, const Wait &w) {
    constexpr int kKv = kHalfTile * (HD / 64), PER = SPLIT ? 1 : kTile / HR, H = HD / 64,
                  kBytes = HR * (HD + HD / 32);
    constexpr int ROWS = HR / (W / 2) * (SPLIT ? 2 : 1), N = ROWS / 8 * H;  // a warp's rows of a stage, a lane's loads
    constexpr int B = N < 4 ? N : 4, NB = N / B;  // loads of a batch, batches of a stage
    const bool is_k = who < W / 2;
    const int op = is_k ? 0 : 1, q = who % (W / 2), half = SPLIT ? q / (W / 4) : 0;
    const int sub = lane >> 2, dim = lane & 3, row0 = (SPLIT ? q % (W / 4) : q) * ROWS + sub;
    const int part_bits = min(a.shift, HR == 128 ? 7 : 6), units = is_k ? KU : VU, h0 = H > 1 ? sub & 1 : 0;
    const uint8_t *from = stages + (op * (SPLIT ? 2 : 1) + half) * NS * kBytes;
    const int to0 = h0 * kHalfTile + row0 * 128 + (((2 * dim) ^ sub) << 4), to1 = to0 ^ 16;  // (row0 & 7 is sub)
    const uint32_t all = (1u << (HR >> part_bits)) - 1u;  // (at most 16 parts)
    uint64_t *full = g->full[op][half], *done = is_k ? y->k_done : y->v_done, *ready = is_k ? y->k_full : y->v_full;
    const int items = nt * PER;
    int u = 0, slot = 0;  // the stage, the place in the ring
    uint32_t stage_phase = 0, slot_phase = 1;  // (of a slot: of the products that last read it)
    for (int e = 0; e < items; ++e) {
        bool ok = mbar_wait(full + u, stage_phase, w);
        if (e >= units * PER && e % PER == 0) ok = ok && mbar_wait(done + slot, slot_phase, w);
        if (!__all_sync(0xFFFFFFFFu, ok)) return;
        const uint8_t *codes = from + u * kBytes + row0 * HD + h0 * 64 + dim * 16;
        const uint8_t *scales = from + u * kBytes + HR * HD + row0 * (HD / 32) + h0 * 2 + (dim >> 1);
        uint8_t *to = ring + (is_k ? slot : KU + slot) * kKv + (SPLIT ? half : e % PER) * HR * 128;
        const uint32_t there = g->there[op][half][u];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            uint4 x[B];
            uint32_t f[B];
#pragma unroll
            for (int k = 0; k < B; ++k) {
                const int r = (b * B + k) / H * 8, flip = k % H;  // (the other half of the dims: 64 bytes on, or back)
                x[k] = *reinterpret_cast<const uint4 *>(codes + r * HD + (flip ? 64 - 128 * h0 : 0));
                f[k] = scales[r * (HD / 32) + (flip ? 2 - 4 * h0 : 0)];
            }
            if (there != all) {  // rows that are not there: zeros
#pragma unroll
                for (int k = 0; k < B; ++k)
                    if (!((there >> ((row0 + (b * B + k) / H * 8) >> part_bits)) & 1))
                        x[k] = make_uint4(0, 0, 0, 0), f[k] = 127;
            }
#pragma unroll
            for (int k = 0; k < B; ++k) {
                const uint32_t s = e4m3_factor(f[k]);
                const uint2 v0 = e4m3_values(x[k].x, s), v1 = e4m3_values(x[k].y, s), v2 = e4m3_values(x[k].z, s),
                            v3 = e4m3_values(x[k].w, s);
                uint8_t *at = to + (b * B + k) / H * 8 * 128 + (k % H ? kHalfTile - 2 * kHalfTile * h0 : 0);
                *reinterpret_cast<uint4 *>(at + to0) = make_uint4(v0.x, v0.y, v1.x, v1.y);
                *reinterpret_cast<uint4 *>(at + to1) = make_uint4(v2.x, v2.y, v3.x, v3.y);
            }
        }
        async_fence();
        __syncwarp();
        if (lane == 0) {
            mbar_arrive(&g->free[op][half][u]);
            mbar_arrive(ready + slot);
        }
        if (++u == NS) u = 0, stage_phase ^= 1;
        if (e % PER == PER - 1 && ++slot == units) slot = 0, slot_phase ^= 1;
    }
}

// After a wait that ran out: the copies that were issued have landed.
static __device__ __noinline__ void settle_stages(Stages *g, int stages) {
    for (int i = 0; i < 4; ++i) {
        const int n = *(volatile int *)(&g->issued[0][0] + i);
        for (int e = max(0, n - stages); e < n; ++e)
            mbar_await(&g->full[0][0][0] + i * kMostStages + e % stages, (e / stages) & 1);
    }
}

// The products of the V rows that were taken out of their tiles (a value that is no
// number), element by element for the query rows that see them; a rare case.
template <int HD, int TERMS, bool MANY, bool Q8>
__device__ __noinline__ void add_hidden_rows(const PagedArgs &a, const TreeArgs &t, const Work &wk, const Span &sp, int kvh,
                                             int G, const uint32_t *bad, const float *mref, float *Os, int tid) {
    const float c = a.scale * 1.44269504088896340736f;
    for (int i = tid; i < wk.rows * HD; i += soft_threads(MANY)) {
        const int r = i / HD, d = i % HD, rg = wk.row0 + r, pos = sp.base + rg / G;
        const int64_t qat = (rg / G) * t.q_token + (int64_t)(kvh * G + rg % G) * HD;
        for (int word = 0; word < kBadWords; ++word)
            for (uint32_t w = bad[word]; w; w &= w - 1) {
                const int j = sp.tile_of_part(word / 4) * kTile + word % 4 * 32 + __ffs(w) - 1;
                if (!sp.sees(pos, j)) continue;
                const int64_t at = pool_row(a, wk.b, kvh, j);
                float x = 0.f;
                for (int e = 0; e < HD; ++e) {
                    float qv;
                    if constexpr (TERMS == 1)
                        qv = bf_lo(static_cast<const uint16_t *>(t.q)[qat + e]);
                    else
                        qv = static_cast<const float *>(t.q)[qat + e];
                    x = fmaf(qv, pool_value<HD, Q8>(a.kc, a.ks, at, e), x);
                }
                float *o = Os + o_at<HD, MANY>(r, d);
                *o = fmaf(ex2(fmaf(x, c, -mref[r])), pool_value<HD, Q8>(a.vc, a.vs, at, d), *o);
            }
    }
}

// The kernels' shared memory, for them and for their launches.
template <int HD, int TERMS, int NR, bool Q8, int PER>
using PagedShape =
    AttnShape<HD, TERMS, NR, less_bytes(Q8, form_of(false, HD, TERMS, NR), HD), PER, true>;
// (sum_bytes: the results of many rows of fp32 queries, summed tile by tile)
__host__ __device__ constexpr int sum_bytes(int hd, int terms) { return terms > 1 ? 2 * kRows * hd * 4 : 0; }
template <int HD, int TERMS, bool Q8>
using PagedRowShape =
    RowShape<HD, TERMS, kOwnBytes, less_bytes(Q8, form_of(true, HD, TERMS), HD) + sum_bytes(HD, TERMS)>;

// Few rows: up to 16 or 32 query rows of a kv head a CTA, S = K q^T and O = V^T P. What
// bounds it: for bf16 pages memory and the longest sequences at the end (32 of 199 to
// 4,099 rows, 8 kv heads of 64: 35.6 us = 4.0 TB/s over all, DRAM 46 % busy), for 8-bit pages
// the widening (8 of 27,767 to 32,768 rows, heads of 128: 147.8 us = 3.5 TB/s, issue slots
// 60 %), for one token over a short context latency (192 rows, fp32: 6.2 us).
template <int HD, int TERMS, int NR, bool Q8, int PER>
__global__ void __launch_bounds__(paged_threads(false, Q8), PER)
    paged_attention(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap, const __grid_constant__ PagedArgs a) {
    constexpr Form F = form_of(false, HD, TERMS, NR);
    using C = PagedShape<HD, TERMS, NR, Q8, PER>;
    constexpr int kThreads = paged_threads(false, Q8);
    constexpr int N = C::N, PT = weight_terms(TERMS), PN = C::PN, KU = C::KU, VU = C::VU;
    constexpr bool kScaled = TERMS > 1;             // the queries carry the scale already
    constexpr bool kOnes = HD == 64;                // the sums come out of the second product
    // A tensor core's sum cuts what it cannot hold, towards zero: 60,000 rows of a CTA left
    // results 1.5e-4 of their norm short, a million 2.6e-3 (also with heads of 64, whose weights' sums
    // come out of the same product). So a group's product starts anew every kSumTiles of its tiles,
    // and what there was is added up, rounded, in tensor memory of its own (F), however many CTAs
    // share the rows. (Eight tiles instead of four cost as much and left up to 1.7 times the
    // error of fp32 operations. Its instructions: one token over 192 rows 6.46 -> 6.48 us, the decode
    // batch 35.63 -> 35.85, 8-bit tokens 146.2 -> 146.4, fp32 ones with heads of 128 3 to 5 %, which
    // spill; in a function of its own, or with the raising of the maxima, the batch took 1.2 to 1.5
    // us more, with columns by eights 0.8.)
    constexpr int kSumTiles = 4;
    static_assert(C::kUsed + 2 * NR <= C::kCols, "S, O and F of both groups");
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *Ps = sm + C::kOffP, *Qs = sm + C::kOffQ;
    Sync<KU, VU> *y = reinterpret_cast<Sync<KU, VU> *>(sm + C::kOffMisc);
    static_assert(sizeof(Sync<KU, VU>) <= 512, "");
    volatile int *err = &y->err;
    const Wait wt{err, a.wait_ns, a.wait_sleep};
    uint32_t *bad = reinterpret_cast<uint32_t *>(sm + C::kOffMisc + 512);  // [kBadWords]
    Stages *stage = reinterpret_cast<Stages *>(bad + kBadWords);
    uint8_t *stages = sm + C::kOffMore;
    static_assert(kOwnBytes <= 8 * MK_MAX_TREE, "");
    float *mref = reinterpret_cast<float *>(sm + C::kOffMisc + 512 + kOwnBytes), *corr = mref + 2 * NR;  // [2][NR] of the groups
    float *lsum = corr + 2 * NR;                // [NR]
    float *wtmp = lsum + NR;                    // [2][4][NR]
    float *Os = reinterpret_cast<float *>(sm);  // [NR][HD], in the ring when the tiles are done

    const int tid = threadIdx.x, warp = warp_index(), lane = tid & 31;
    const int S = gridDim.x / a.units, split = blockIdx.x % S, kvh = blockIdx.y, G = a.Hq / a.Hkv;
    const int turn = blockIdx.x / S;
    const float c = a.scale * 1.44269504088896340736f;  // scores in powers of two
    // (what needs nothing of the kernel before comes before its end is awaited)
    if (warp == kKWarp) {
        if constexpr (Q8) init_stages(stage, conv_warps(false) / (F.split ? 4 : 2), lane);
        init_paged(y, bad, Q8 ? conv_warps(false) / 2 * (F.split ? 1 : kTile / F.rows) : 1, soft_threads(false) / 64, lane);
    }
    pdl_wait();
    if (!a.part) pdl_trigger();
    if (warp == kMmaWarp) tmem_alloc(&y->tmem, C::kCols);
    const Work wk = find_work(a, turn, NR, G, lane);
    const int row0 = wk.row0, rows = wk.rows;
    const TreeArgs t = tree_args<TERMS>(a, wk);
    const int first = threadIdx.x - kFirstSoft * 32;
    if (is_soft<false>(warp)) {
        // The queries as the B operand: row term * NR + r, 128-byte swizzled. (Rows
        // behind the sequence's last token are zeros, and columns nobody reads.)
#pragma unroll
        for (int i0 = 0; i0 < NR * (HD / 8); i0 += kSoft) {
            const int i = i0 + first, r = i / (HD / 8), ch = i % (HD / 8);
            if (NR * (HD / 8) < kSoft && i >= NR * (HD / 8)) break;
            uint4 q[TERMS];
            load_query8<HD, TERMS>(t, 0, kvh, G, row0 + r, ch, c, q);
#pragma unroll
            for (int k = 0; k < TERMS; ++k) {
                const int n = k * NR + r;
                *reinterpret_cast<uint4 *>(Qs + (ch / 8) * (N * 128) + n * 128 + (((ch % 8) ^ (n & 7)) << 4)) = q[k];
            }
        }
    }
    if (rows <= 0) {  // the whole cluster
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
        if (warp == kMmaWarp) tmem_free(uniform(y->tmem), C::kCols);
        return;
    }
    const Span sp = span_of(a, wk, G);
    const int t0 = (int)((int64_t)split * sp.tiles / S), nt = (int)((int64_t)(split + 1) * sp.tiles / S) - t0;
    if (!Q8 && warp == kKWarp) {  // the first copy needs nobody else
        load_pages<HD>(y, sm, &kmap, true, a, wk.b, kvh, sp, t0, 0, min(nt, 1), lane, wt);
    } else if (warp == kMmaWarp) {
        if constexpr (kOnes)
            for (int i = lane; i < C::kOnes / 16; i += 32)  // chunk 0 of row i / 8 sits at chunk (row & 7)
                *reinterpret_cast<uint4 *>(sm + C::kOffOnes + i * 16) =
                    make_uint4(i % 8 == ((i / 8) & 7) ? 0x3F80u : 0u, 0u, 0u, 0u);
    } else if (is_soft<false>(warp)) {
        if (first < 2 * NR) mref[first] = kNone;
    }
    async_fence();
    tc_fence_before();
    __syncwarp();
    __syncthreads();
    tc_fence_after();
    // S, O and F of group g: + g * N, + g * PN, + g * NR
    const uint32_t tS = uniform(y->tmem), tO = tS + 2 * N, tF = tO + 2 * PN;

    if (warp >= first_conv(false)) {
        if constexpr (Q8)
            convert_pages<HD, KU, VU, conv_warps(false), F.rows, F.stages, F.split>(y, sm, stage, stages, a, nt,
                                                                                    warp - first_conv(false), lane, wt);
    } else if (Q8 && (warp == kKWarp || warp == kVWarp)) {
        if constexpr (Q8)
            stage_pages<HD, F.rows, F.stages, F.split>(stage, stages, warp == kVWarp, a, wk.b, kvh, sp, t0, nt, lane, wt);
    } else if (!Q8 && warp == kKWarp) {
        load_pages<HD>(y, sm, &kmap, true, a, wk.b, kvh, sp, t0, 1, nt, lane, wt);
    } else if (!Q8 && warp == kVWarp) {
        load_pages<HD>(y, sm, &vmap, false, a, wk.b, kvh, sp, t0, 0, nt, lane, wt);
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
                const uint64_t p = sw128_desc(p0 + (i & 1) * C::kP, kHalfTile);  // (packed: 64 bytes into the rows)
                if (!(ok = ok && v_full(y, i, wt) && mbar_wait(&y->p_full[i & 3], (i >> 2) & 1, wt))) break;
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < kTile / 16; ++kk)
                    umma_bf16(tO + (i & 1) * PN, v + ((kk * 2048) >> 4) - (kOnes ? (uint64_t)((kk * 2048) >> 4) << 16 : 0),
                              p + ((kk * 2048) >> 4), idO, (i >> 1) % kSumTiles != 0 || kk != 0);
                umma_commit(&y->v_done[i % VU]);
                if (!C::kEarly && j < nt) {
                    ok = k_full(y, j, wt);
                    tc_fence_after();
                    if (ok) scores(j);
                }
            }
        }
    } else if (is_soft<false>(warp)) {
        // group g takes every other tile; thread: cache row `row` of it, all query rows
        const int g = (warp - kFirstSoft) >> 2, quarter = warp & 3, row = quarter * 32 + lane;
        const uint32_t mylane = (uint32_t)(quarter * 32) << 16;
        const uint32_t ts = tS + g * N + mylane, to = tO + g * PN + mylane, tf = tF + g * NR + mylane;
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
            const int tile = sp.tile(t0 + i), j = tile * kTile + row, part = sp.part(tile);
            if (part >= 0) {  // not all rows see all of it: columns [lo, hi) see this one
                int lo, hi;
                sp.columns(j, G, row0, lo, hi);
#pragma unroll
                for (int r = 0; r < NR; ++r)
                    if (r < lo || r >= hi) s[r] = -INFINITY;
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
                    const int n1 = (i >> 1) > kSumTiles ? PN + NR : PN;  // (F behind O, once there is one)
#pragma unroll 1
                    for (int n0 = 0; n0 < n1; n0 += 16) {
                        const uint32_t at = n0 < PN ? to + n0 : tf + n0 - PN;
                        float o[16];
                        tmem_ld16(at, o);
                        tmem_ld_wait();
                        pin<16>(o);
#pragma unroll
                        for (int e = 0; e < 16; ++e) o[e] *= gcorr[n0 % NR + e];
                        tmem_st16(at, o);
                    }
                    tmem_st_wait();
                }
            }
            if (i >= 2 && (i >> 1) % kSumTiles == 0) {  // O starts anew with this tile
                tc_fence_after();
#pragma unroll 1
                for (int r0 = 0; r0 < NR; r0 += 16) {
                    float z[16], w[16];
                    tmem_ld16(to + (PT - 1) * NR + r0, z);
                    tmem_ld_wait();
                    pin<16>(z);
#pragma unroll 1
                    for (int k = PT - 2; k >= 0; --k) {
                        tmem_ld16(to + k * NR + r0, w);
                        tmem_ld_wait();
                        pin<16>(w);
#pragma unroll
                        for (int e = 0; e < 16; ++e) z[e] += w[e];
                    }
                    if ((i >> 1) > kSumTiles) {
                        tmem_ld16(tf + r0, w);
                        tmem_ld_wait();
                        pin<16>(w);
#pragma unroll
                        for (int e = 0; e < 16; ++e) z[e] += w[e];
                    }
                    tmem_st16(tf + r0, z);
                }
                tmem_st_wait();
            }
            if (part >= 0) {
                ok = ok && v_full(y, i, wt);
                mend_v<HD>(sm + (KU + i % VU) * C::kKv, row, sp.somebody(j) ? part * kTile + row : kBadRows, kBadRows, bad);
            }
            // the weights as the B operand: row = cache row, column = term * NR + r
            uint8_t *p = Ps + (C::kPacked ? 0 : g * C::kP) + row * 128;
            constexpr int kChunks = C::kPacked ? 4 : 0;  // of the row, before group 1's
#pragma unroll
            for (int r0 = 0; r0 < NR; r0 += 8) {
                float w[8];
                uint4 u[PT];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    w[e] = ex2(x[r0 + e]);
                    if constexpr (!kOnes) l[r0 + e] += w[e];
                }
                split8<PT>(w, u);
#pragma unroll
                for (int k = 0; k < PT; ++k) {
                    const int ch = (k * NR + r0) / 8 + g * kChunks;
                    *reinterpret_cast<uint4 *>(p + (ch / 8) * kHalfTile + (((ch % 8) ^ (row & 7)) << 4)) = u[k];
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
                        w[e] = z;
                    }
                    if ((nt - h + 1) / 2 > kSumTiles) {
                        float f[16];
                        tmem_ld16(tF + h * NR + mylane + r0, f);
                        tmem_ld_wait();
                        pin<16>(f);
#pragma unroll
                        for (int e = 0; e < 16; ++e) w[e] += f[e];
                    }
#pragma unroll
                    for (int e = 0; e < 16; ++e) o[e] = fmaf(corr[h * NR + r0 + e], w[e], o[e]);
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
        if (any_bad(bad)) add_hidden_rows<HD, TERMS, false, Q8>(a, t, wk, sp, kvh, G, bad, mref, Os, first);
    }
    tc_fence_before();
    __syncwarp();
    __syncthreads();
    if (*err) {  // a wait ran out (nobody waits any more: the same for all threads): the rows are NaN
        if constexpr (Q8)
            if (warp == kKWarp && elect()) settle_stages(stage, F.stages);
        settle(y, a.err);
        if (tid < NR) lsum[tid] = __uint_as_float(0x7FC00000u);
        __syncthreads();
    }
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_free(tS, C::kCols);
    }
    finish<HD, TERMS, NR, false, kThreads>(t, (int64_t)turn * a.Hkv + kvh, 0, kvh, G, row0, rows, split, S, Os, mref,
                                   lsum);
}

// Barriers of the softmax threads, and of a pair of their warps: a plain one, and a vote.
__device__ __forceinline__ void rows_sync() { asm volatile("barrier.cta.sync 1, 512;" ::: "memory"); }
__device__ __forceinline__ void pair_sync(int id) { asm volatile("barrier.cta.sync %0, 64;" ::"r"(id) : "memory"); }
__device__ __forceinline__ bool pair_any(int id, bool x) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, %2, 64, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)x), "r"(id)
        : "memory");
    return r != 0;
}

// A thread's N consecutive dims of a result.
template <int TERMS, int N>
__device__ __forceinline__ void put_row(const TreeArgs &t, int64_t at, const float (&o)[N]) {
#pragma unroll
    for (int e = 0; e < N; e += 8) {
        if constexpr (TERMS == 1) {
            *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(t.out) + at + e) =
                make_uint4(pack_bf16(o[e], o[e + 1]), pack_bf16(o[e + 2], o[e + 3]), pack_bf16(o[e + 4], o[e + 5]),
                           pack_bf16(o[e + 6], o[e + 7]));
        } else {
            float4 *to = reinterpret_cast<float4 *>(static_cast<float *>(t.out) + at + e);
            to[0] = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
            to[1] = make_float4(o[e + 4], o[e + 5], o[e + 6], o[e + 7]);
        }
    }
}

// Many rows: 128 query rows of a kv head a CTA, S = q K^T and O = P V with P in tensor
// memory, in place of the scores it comes from. 16 warps for the softmax, two to 32 rows,
// half of a tile's columns each: with eight 8-bit chunks took 156 us for 125. What bounds it is neither the
// products (tensor pipe 33 % of the active cycles) nor memory: a prompt of 4,096 tokens, 32 heads of 64, takes
// 139 us (494 TFLOP/s of the formula's operations), 111 tiles an SM of 0.75 us and the set-up and end
// of seven CTAs an SM; 4 x 33 tokens, window 4,096, heads of 128, 32.6 us (1.07 a tile, 80 CTAs for
// 152 SMs); fp32 chunks over 6,001 rows of 8 bits 91.2 us (1.74 a tile). With fp32 queries a tensor core's sums,
// which cut what they cannot hold, are too short: two tiles of a group are summed there, and
// those sums in shared memory (80 us without, off by up to 1.3e-5 of the norm over 32,000 rows; 1.7e-6 with, over a million).
template <int HD, int TERMS, bool Q8>
__global__ void __launch_bounds__(paged_threads(true, Q8), 1)
    paged_attention_rows(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                         const __grid_constant__ PagedArgs a) {
    constexpr Form F = form_of(true, HD, TERMS);
    using C = PagedRowShape<HD, TERMS, Q8>;
    constexpr int kThreads = paged_threads(true, Q8);
    constexpr int KU = C::KU, VU = C::VU, NB = C::NB, PT = weight_terms(TERMS);
    constexpr bool kScaled = TERMS > 1;
    constexpr int kHalf = kTile / 2;  // a softmax thread's columns of a tile
    // Scores that a thread keeps from the maximum to the weights; with 8-bit pages, whose
    // converting warps leave 80 registers, it reads them again.
    constexpr int kKeep = Q8 ? 32 : kHalf;
    // A tensor core's sum cuts what it cannot hold, towards zero: over 125 tiles of three
    // terms the results of fp32 queries were 1.3e-5 of their norm off (the sums of the
    // weights, rounded, are not cut alike). So theirs are summed by the softmax threads, a
    // group's two tiles at a time, in shared memory, and no product adds to more (each tile:
    // 104 us for 80 without, 24 heads of 64 over 6,001 rows, 301 tokens and fewer).
    constexpr bool kSums = TERMS > 1;
    static_assert(!kSums || NB == 2, "S(i) is issued behind PV(i - 2)");
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *Qs = sm + C::kOffQ;
    Sync<KU, VU> *y = reinterpret_cast<Sync<KU, VU> *>(sm + C::kOffMisc);
    static_assert(sizeof(Sync<KU, VU>) <= 512, "");
    volatile int *err = &y->err;
    const Wait wt{err, a.wait_ns, a.wait_sleep};
    // [2][128]: the groups' maxima, then the rows' maxima and sums
    uint32_t *bad = reinterpret_cast<uint32_t *>(sm + C::kOffMisc + 512);  // [kBadWords]
    Stages *stage = reinterpret_cast<Stages *>(bad + kBadWords);
    uint8_t *stages = sm + C::kOffMore;
    float *acc = reinterpret_cast<float *>(stages + less_bytes(Q8, F, HD));  // kSums: [2][128][HD], of the groups
    float *gm = reinterpret_cast<float *>(sm + C::kOffMisc + 512 + kOwnBytes), *mref = gm, *lsum = gm + kRows;
    float *Os = reinterpret_cast<float *>(sm);                      // in the ring when the tiles are done,
    float *join = Os + kRows * HD;                                  // and behind it

    const int tid = threadIdx.x, warp = warp_index(), lane = tid & 31;
    const int S = gridDim.x / a.units, split = blockIdx.x % S, kvh = blockIdx.y, G = a.Hq / a.Hkv;
    const int turn = blockIdx.x / S;
    const float c = a.scale * 1.44269504088896340736f;
    // (what needs nothing of the kernel before comes before its end is awaited)
    if (warp == kKWarp) {
        if constexpr (Q8) init_stages(stage, conv_warps(true) / (F.split ? 4 : 2), lane);
        init_paged(y, bad, Q8 ? conv_warps(true) / 2 * (F.split ? 1 : kTile / F.rows) : 1, soft_threads(true) / 64, lane);
    }
    pdl_wait();
    if (!a.part) pdl_trigger();
    if (warp == kMmaWarp) tmem_alloc(&y->tmem, C::kCols);
    const Work wk = find_work(a, turn, kRows, G, lane);
    const int row0 = wk.row0, rows = wk.rows;
    const TreeArgs t = tree_args<TERMS>(a, wk);
    const int row = (warp & 3) * 32 + lane;  // a softmax thread's query row
    const int st = tid - kFirstSoft * 32;  // a softmax thread's index
    if (is_soft<true>(warp)) {
        // the queries as the A operand: term k, 128-byte swizzled rows of 64 dims
#pragma unroll
        for (int i0 = 0; i0 < kRows * (HD / 8); i0 += kRowSoft) {
            const int r = (i0 + st) / (HD / 8), ch = (i0 + st) % (HD / 8);
            uint4 q[TERMS];
            load_query8<HD, TERMS>(t, 0, kvh, G, row0 + r, ch, c, q);
#pragma unroll
            for (int k = 0; k < TERMS; ++k)
                *reinterpret_cast<uint4 *>(Qs + k * C::kKv + (ch / 8) * kHalfTile + r * 128 +
                                           (((ch % 8) ^ (r & 7)) << 4)) = q[k];
        }
    }
    if (rows <= 0) {  // the whole cluster
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
        if (warp == kMmaWarp) tmem_free(uniform(y->tmem), C::kCols);
        return;
    }
    const Span sp = span_of(a, wk, G);
    const int t0 = (int)((int64_t)split * sp.tiles / S), nt = (int)((int64_t)(split + 1) * sp.tiles / S) - t0;
    if (!Q8 && warp == kKWarp) {  // the first copy needs nobody else
        load_pages<HD>(y, sm, &kmap, true, a, wk.b, kvh, sp, t0, 0, min(nt, 1), lane, wt);
    }
    async_fence();
    tc_fence_before();
    __syncwarp();
    __syncthreads();
    tc_fence_after();
    // scores and third terms of tile i: + i % NB * 128, + i % NB * kThird; O of group g: + g * HD
    const uint32_t tS = uniform(y->tmem), tT = tS + NB * kTile, tO = tT + NB * C::kThird;

    if (warp >= first_conv(true)) {
        if constexpr (Q8)
            convert_pages<HD, KU, VU, conv_warps(true), F.rows, F.stages, F.split>(y, sm, stage, stages, a, nt,
                                                                                    warp - first_conv(true), lane, wt);
    } else if (Q8 && (warp == kKWarp || warp == kVWarp)) {
        if constexpr (Q8)
            stage_pages<HD, F.rows, F.stages, F.split>(stage, stages, warp == kVWarp, a, wk.b, kvh, sp, t0, nt, lane, wt);
    } else if (!Q8 && warp == kKWarp) {
        load_pages<HD>(y, sm, &kmap, true, a, wk.b, kvh, sp, t0, 1, nt, lane, wt);
    } else if (!Q8 && warp == kVWarp) {
        load_pages<HD>(y, sm, &vmap, false, a, wk.b, kvh, sp, t0, 0, nt, lane, wt);
    } else if (warp == kMmaWarp) {
        constexpr uint32_t idS = idesc_bf16(kTile, false, false), idO = idesc_bf16(HD, false, true);
        const uint64_t q = sw128_desc(saddr(Qs), 16);
        const uint32_t ring = saddr(sm);
        auto scores = [&](int i) {
            const uint64_t k = sw128_desc(ring + (i % KU) * C::kKv, 16);
#pragma unroll
            for (int t = TERMS - 1; t >= 0; --t)  // (the small terms first: a sum cuts by its size)
#pragma unroll
                for (int kk = 0; kk < HD / 16; ++kk) {
                    const uint32_t at = (kk / 4) * kHalfTile + (kk % 4) * 32;
                    umma_bf16(tS + (i % NB) * kTile, q + ((t * C::kKv + at) >> 4), k + (at >> 4), idS,
                              t != TERMS - 1 || kk != 0);
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
                for (int t = PT - 1; t >= 0; --t)
#pragma unroll
                    for (int kk = 0; kk < kTile / 16; ++kk) {
                        const uint32_t p = t < 2 ? tS + (i % NB) * kTile + kk / 2 * 32 + t * 16 + kk % 2 * 8
                                                 : tT + (i % NB) * C::kThird + kk * 8;
                        umma_bf16_ta(tO + (i & 1) * HD, p, v + ((kk * 2048) >> 4), idO,
                                     (kSums ? (i & 2) != 0 : i >= 2) || t != PT - 1 || kk != 0);
                    }
                umma_commit(&y->v_done[i % VU]);
                if (j < nt) {  // (into the buffer of PV(i))
                    ok = k_full(y, j, wt);
                    tc_fence_after();
                    if (ok) scores(j);
                }
            }
        }
    } else if (is_soft<true>(warp)) {
        // group g takes every other tile; two warps have a row of it each in their lanes, and
        // half (h) of its columns: their maximum is one, their sums are added at the end
        const int sw = warp - kFirstSoft, g = (sw >> 2) & 1, h = sw >> 3, quarter = warp & 3, pair = 2 + g * 4 + quarter;
        const uint32_t mylane = (uint32_t)(quarter * 32) << 16;
        const uint32_t to = tO + g * HD + h * (HD / 2) + mylane;
        const bool live = quarter * 32 < rows;  // (rows behind the last: the warps only keep the barriers)
        const int pos = sp.base + (row0 + row) / G;  // the row's token
        float m = kNone, l = 0.f;
        bool ok = true;
        for (int i = g; i < nt; i += 2) {
            ok = ok && s_done(y, i, wt);
            tc_fence_after();
            const uint32_t ts = tS + (i % NB) * kTile + h * kHalf + mylane;
            const uint32_t tt = tT + (i % NB) * C::kThird + h * (kHalf / 2) + mylane;
            const int tile = sp.tile(t0 + i), at = tile * kTile, part = sp.part(tile);
            if (live) {
                float x[kKeep];
                // The scores of columns w0 .. w0 + kKeep - 1 of the half, hidden ones -inf.
                auto load = [&](int w0) {
#pragma unroll
                    for (int e = 0; e < kKeep; e += 16) tmem_ld16(ts + w0 + e, x + e);
                    tmem_ld_wait();
                    pin<kKeep>(x);
                    if (part >= 0) {
#pragma unroll
                        for (int w = 0; w < kKeep; w += 32) {
                            const uint32_t see = sp.sees32(pos, at + h * kHalf + w0 + w);
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                if (!((see >> e) & 1)) x[w + e] = -INFINITY;
                        }
                    }
                };
                float t4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int w0 = 0; w0 < kHalf; w0 += kKeep) {
                    load(w0);
#pragma unroll
                    for (int e = 0; e < kKeep; e += 8)
#pragma unroll
                        for (int w = 0; w < 4; ++w) t4[w] = fmaxf(fmaxf(t4[w], x[e + 2 * w]), x[e + 2 * w + 1]);
                }
                float top = fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3]));
                if (!kScaled) top *= c;  // (the scale is positive)
                float scale = 1.f;
                const bool raise = pair_any(pair, top > m + kRaise);
                if (raise) {
                    // raise the warps' maxima to those of the rows so far; scale O and the sums
                    float *seen = gm + g * kRows + row;
                    if (h) *seen = top;
                    pair_sync(pair);
                    if (!h) *seen = fmaxf(fmaxf(*seen, top), m);
                    pair_sync(pair);
                    const float best = *seen;
                    scale = ex2(m - best);
                    m = best;
                    l *= scale;
                    if (kSums ? (i & 2) != 0 : i >= 2) {
                        if (NB > 2) ok = ok && pv_done(y, i - 2, wt);  // O is this group's again (NB = 2: S(i) was issued behind it)
                        tc_fence_after();
#pragma unroll 1
                        for (int d = 0; d < HD / 2; d += 16) {
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
                // (PV(i - 2) is done: S(i) was issued behind it)
                if (kSums && i >= 4 && ((i & 2) == 0 || raise)) {
                    const bool take = (i & 2) == 0;
#pragma unroll
                    for (int d = 0; d < HD / 2; d += 16) {
                        float o[16];
                        tmem_ld16(to + d, o);
                        tmem_ld_wait();
                        pin<16>(o);
#pragma unroll
                        for (int e = 0; e < 16; e += 4) {
                            float4 *z = reinterpret_cast<float4 *>(acc + g * kRows * HD + o_at<HD, true>(row, h * (HD / 2) + d + e));
                            float4 w = make_float4(0.f, 0.f, 0.f, 0.f);
                            if (i >= 6) w = *z;
                            if (take) w = make_float4(w.x + o[e], w.y + o[e + 1], w.z + o[e + 2], w.w + o[e + 3]);
                            *z = make_float4(w.x * scale, w.y * scale, w.z * scale, w.w * scale);
                        }
                    }
                }
                float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                for (int w0 = 0; w0 < kHalf; w0 += 32) {
                    if (kKeep < kHalf) load(w0);
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        float &x0 = x[w0 % kKeep + e], &x1 = x[w0 % kKeep + e + 1];
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
                            float &x0 = x[w0 % kKeep + 2 * e], &x1 = x[w0 % kKeep + 2 * e + 1];
                            w[e] = pack_bf16(x0, x1);
                            if (t + 1 < PT) less2(x0, x1, w[e]);
                        }
                        // (into the columns that the 32 scores were in)
                        tmem_st16(t < 2 ? ts + w0 + t * 16 : tt + w0 / 2, w);
                    }
                }
                l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
                tmem_st_wait();
            }
            tc_fence_before();
            if (part >= 0) {
                ok = ok && v_full(y, i, wt);
                if (!h)
                    mend_v<HD>(sm + (KU + i % VU) * C::kKv, row, sp.somebody(at + row) ? part * kTile + row : kBadRows,
                               kBadRows, bad);
                async_fence();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&y->p_full[i & 3]);
        }
        if (nt > 0) ok = ok && pv_done(y, nt - 1, wt);  // (and with it every product: the ring is free)
        tc_fence_after();
        // (the pair's raises are over: each of its warps has read the last one's before this)
        if (!h) gm[g * kRows + row] = m;
        rows_sync();
        tc_fence_after();  // (a group that passed early reads O behind the barrier, too)
        // the groups' O and sums to the larger maximum; a row's four threads take a quarter of
        // its dims each, from both groups' O
        const float best = fmaxf(m, gm[(g ^ 1) * kRows + row]), scale = g < nt ? ex2(m - best) : 0.f;
        float *sums = join, *scales = sums + 4 * kRows;  // [4][128], [2][128], in the ring
        sums[(g * 2 + h) * kRows + row] = l * scale;
        if (!h) scales[g * kRows + row] = scale;
        const bool direct = S == 1 && !a.part && !any_bad(bad);
        rows_sync();
        const float sum = (sums[row] + sums[kRows + row]) + (sums[2 * kRows + row] + sums[3 * kRows + row]);
        if (live) {  // (whole warps: they load together)
            // one split: the result (no row seen: zeros; a wait that ran out: NaN); else its part of it
            const float inv = !direct ? 1.f : *err ? __uint_as_float(0x7FC00000u) : sum == 0.f ? 0.f : 1.f / sum;
            const float f0 = scales[row] * inv, f1 = scales[kRows + row] * inv;
            const int d0 = (g * 2 + h) * (HD / 4);
            float o[HD / 4], p[HD / 4];
#pragma unroll
            for (int d = 0; d < HD / 4; d += 16) {
                if (nt > 0) tmem_ld16(tO + mylane + d0 + d, o + d);
                if (nt > 1) tmem_ld16(tO + HD + mylane + d0 + d, p + d);
            }
            tmem_ld_wait();
            pin<HD / 4>(o);
            pin<HD / 4>(p);
            if constexpr (kSums) {
#pragma unroll
                for (int e = 0; e < HD / 4; ++e) {
                    const float *z = acc + o_at<HD, true>(row, d0 + e);
                    if (nt > 4) o[e] += z[0];
                    if (nt > 5) p[e] += z[kRows * HD];
                }
            }
#pragma unroll
            for (int e = 0; e < HD / 4; ++e) {
                o[e] = nt > 0 ? f0 * o[e] : direct ? inv : 0.f;  // (no tile: 0, or NaN)
                if (nt > 1) o[e] = fmaf(f1, p[e], o[e]);
            }
            if (!direct) {
#pragma unroll
                for (int e = 0; e < HD / 4; e += 4)
                    *reinterpret_cast<float4 *>(Os + o_at<HD, true>(row, d0 + e)) = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
            } else if (row < rows) {
                const int rg = row0 + row;
                put_row<TERMS, HD / 4>(t, (rg / G) * t.o_token + (int64_t)(kvh * G + rg % G) * HD + d0, o);
            }
        }
        if (!direct) {
            if (st < kRows) mref[row] = best, lsum[row] = sum;  // (st is the row here; the maxima have been read)
            rows_sync();
        }
        if (!direct && any_bad(bad)) add_hidden_rows<HD, TERMS, true, Q8>(a, t, wk, sp, kvh, G, bad, mref, Os, st);
    }
    tc_fence_before();
    __syncwarp();
    __syncthreads();
    if (*err) {  // a wait ran out (nobody waits any more: the same for all threads): the rows are NaN
        if constexpr (Q8)
            if (warp == kKWarp && elect()) settle_stages(stage, F.stages);
        settle(y, a.err);
        if (tid < kRows) lsum[tid] = __uint_as_float(0x7FC00000u);
        __syncthreads();
    }
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_free(tS, C::kCols);
    }
    if (S == 1 && !a.part && !any_bad(bad)) return;  // (written, or NaN)
    finish<HD, TERMS, kRows, true, kThreads>(t, (int64_t)turn * a.Hkv + kvh, 0, kvh, G, row0, rows, split, S, Os, mref,
                                   lsum);
}

// Joins the S splits' partial results of every unit: grid (tiles of rows, kv heads, dims).
template <int HD, int TERMS, int NR>
__global__ void __launch_bounds__(256) paged_join(const __grid_constant__ PagedArgs a, int S) {
    constexpr int64_t PF = part_floats(NR, HD);
    __shared__ float ms[max_splits(NR) * NR], wg[max_splits(NR) * NR];
    const int kvh = blockIdx.y, G = a.Hq / a.Hkv;
    pdl_begin();  // (behind it the splits' partial results are there)
    const Work wk = find_work(a, blockIdx.x, NR, G, threadIdx.x & 31);
    if (wk.rows <= 0) return;
    const TreeArgs t = tree_args<TERMS>(a, wk);
    join_splits<HD, TERMS, NR>(t, a.part + ((int64_t)blockIdx.x * a.Hkv + kvh) * S * PF, 0, kvh, G, wk.row0, wk.rows, S, ms,
                               wg);
}

}  // namespace mkops
