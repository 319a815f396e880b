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
#include "mk_paged_attn.cuh"

namespace mkops {
namespace {

// The two kernels by what their launch needs. kTileUs: a tile of one CTA; kFixedUs:
// launch, set-up and end; kJoinUs: the workspace's second launch.
template <int HD_, int TERMS_, int NR_, bool Q8_, int PER_ = 1>
struct PagedFew {
    static constexpr int kThreads = paged_threads(false, Q8_), HD = HD_, TERMS = TERMS_, NR = NR_,
                         kSmem = PagedShape<HD, TERMS, NR, Q8_, PER_>::kSmem;
    static constexpr bool Q8 = Q8_;
    static constexpr double kTileUs = Q8_ ? (HD == 64 ? 0.8 : NR_ == 16 && TERMS_ == 1 ? 1.15 : 1.55)
                                          : (HD == 64 ? 0.6 : 1.0) - (TERMS == 1 ? HD / 64 * 0.1 : 0.0);
    static constexpr double kFixedUs = 4.5, kJoinUs = 4.5;
    static auto fn() { return paged_attention<HD, TERMS, NR, Q8, PER_>; }
};
template <int HD_, int TERMS_, bool Q8_>
struct PagedMany {
    static constexpr int kThreads = paged_threads(true, Q8_), HD = HD_, TERMS = TERMS_, NR = kRows,
                         kSmem = PagedRowShape<HD, TERMS, Q8_>::kSmem;
    static constexpr bool Q8 = Q8_;
    static constexpr double kTileUs = (HD == 128 ? 1.1 : TERMS == 1 ? 0.78 : 1.4) *
                                      (!Q8_ ? 1.0 : TERMS == 1 ? 1.75 : 1.25);
    static constexpr double kFixedUs = 8.0, kJoinUs = 7.0;
    static auto fn() { return paged_attention_rows<HD, TERMS, Q8>; }
};

struct Plan {
    int S, U;  // splits of a unit's tiles; places of tiles of query rows, over all sequences
    bool ws;
    double us;  // its estimated time
};

// What a call's host knows: bounds on a sequence's tokens and rows.
struct Bounds {
    int max_new, max_len, n_sm;
};

// The split with the least estimated time. Units (tiles of query rows x kv heads)
// that do not fit the GPU at once follow one another, so more than a wave of them
// cost their mean, less the longest (the mean of a prompt's tiles is about half of
// the longest's). A tile takes kTileUs, or its share of the memory's rate when the CTAs
// at work read more than that (the tiles of a sequence's query rows share what they read).
template <class K>
Plan plan(const PagedArgs &a, const Bounds &h, bool ws) {
    const int G = a.Hq / a.Hkv;
    const int U = (int)(((int64_t)a.n * G + K::NR - 1) / K::NR) + std::min(a.B, a.n) - 1;  // (places: find_work)
    const int64_t real = std::min<int64_t>(U, (int64_t)a.B * (((int64_t)h.max_new * G + K::NR - 1) / K::NR));
    const int64_t units = real * a.Hkv;
    double rows = h.max_len, mean = h.max_len - 0.5 * std::min(h.max_new, h.max_len);
    if (a.window) {
        const double seen = (double)a.window + a.sinks + kTile + K::NR / G;
        rows = std::min(rows, seen), mean = std::min(mean, seen);
    }
    const int tiles = std::max(1, (int)((rows + kTile - 1) / kTile));
    const double mean_tiles = std::max(1.0, mean / kTile);
    constexpr double kRate = 6.5e6;  // bytes a microsecond
    constexpr double kTileBytes = 2.0 * kTile * K::HD * (K::Q8 ? 1.03 : 2.0);
    const double sharers = (double)std::max<int64_t>(1, ((int64_t)h.max_new * G + K::NR - 1) / K::NR);
    auto tile_us = [&](double ctas) { return std::max(K::kTileUs, ctas / sharers * kTileBytes / kRate); };
    // Many rows of bf16 queries have no room to begin a tensor core's sum anew, and it cuts what it
    // cannot hold, n * 2^-27 over n rows: so at most 262,144 rows a split, half of the result's own
    // rounding, as far as a cluster's splits go (a million rows in one split were 3.4e-3 short).
    const int least = K::NR == kRows && K::TERMS == 1 ? std::min((tiles + 2047) / 2048, kCluster) : 1;
    Plan best{1, U, false, 1e30};
    for (int k = 0; k < 4 && (1 << k) <= tiles; ++k) {
        if ((1 << k) < least && k < 3) continue;
        const int S = 1 << k, at_once = active_clusters<K>(k, h.n_sm);
        const int64_t waves = (units + at_once - 1) / at_once;
        const double each = waves > 1 ? mean_tiles / S + 0.5 : (tiles + S - 1) / S;
        const double us = (double)waves * (each * tile_us((double)S * std::min<int64_t>(units, at_once)) + K::kFixedUs) +
                          (k ? 0.8 + 0.2 * k : 0.0);
        if (us < best.us) best = Plan{S, U, false, us};
    }
    if (ws && units > 0) {
        // (any number of splits, in whole waves: 64 units leave 24 of 152 SMs idle in two
        // splits, and none to speak of in seven: 8 sequences of 32,768 rows of 8 bits, heads of
        // 128, 154.9 -> 145.9 us)
        // (At most eight waves of partial results, 81 MB where a CTA has 128 rows of 128 dims: the
        // workspace has room for all of the call's tokens, not for the bound on a sequence's alone.
        // Tokens far above that bound, 100,000 for one, had asked for 27 GB.)
        const int at_once = active_clusters<K>(0, h.n_sm);
        const int most = (int)std::min<int64_t>(std::min(max_splits(K::NR), tiles / 2), 8ll * at_once / ((int64_t)U * a.Hkv));
        for (int S = std::max(2, least); S <= most; ++S) {
            const int64_t waves = (units * S + at_once - 1) / at_once;
            const double tile = tile_us((double)std::min<int64_t>(units * S, at_once));
            const double us = (double)waves * (((tiles + S - 1) / S) * tile + K::kFixedUs) + K::kJoinUs +
                              8.0 * units * S * part_floats(K::NR, K::HD) / kRate;
            if (us < best.us) best = Plan{S, U, true, us};
        }
    }
    return best;
}

template <class K>
cudaError_t launch(PagedArgs a, const Bounds &h, cudaStream_t s, int64_t *want) {
    cudaError_t e = configure<K>();
    if (e != cudaSuccess) return e;
    Plan p = plan<K>(a, h, want || a.work);
    const int64_t need = p.ws ? (int64_t)p.U * a.Hkv * p.S * part_floats(K::NR, K::HD) : 0;
    if (want) {
        *want = need;
        return cudaSuccess;
    }
    if (need > a.work_floats) p = plan<K>(a, h, false);
    a.part = p.ws ? a.work : nullptr;
    a.units = p.U;
    if (a.wait_ns == 0) a.wait_ns = kWaitNs;
    a.wait_sleep = (uint32_t)std::min<uint64_t>(a.wait_ns, kSleepNs);
    CUtensorMap kmap{}, vmap{};
    if (!K::Q8) {
        const int box = a.shift < 31 ? std::min(a.ps, kTile) : kTile;
        if (!cache_map(&kmap, a.kc, a.n_pages * a.Hkv, a.ps, K::HD, box) ||
            !cache_map(&vmap, a.vc, a.n_pages * a.Hkv, a.ps, K::HD, box))
            return cudaErrorInvalidValue;
    }
    e = launch_op(K::fn(), dim3(p.S * p.U, a.Hkv), K::kThreads, K::kSmem, p.ws ? 1 : p.S, s, kmap, vmap, a);
    if (e != cudaSuccess || !p.ws) return e;
    return launch_op(paged_join<K::HD, K::TERMS, K::NR>, dim3(p.U, a.Hkv, (K::NR * K::HD / 4 + 255) / 256), 256, 0, 0, s, a,
                     p.S);
}

// The kernel of 16 or 32 columns that holds a sequence's rows of a kv head, or, for
// more rows, several CTAs of 32 or the kernel of 128 rows, whichever plan is shorter.
template <int HD, int TERMS, bool Q8>
cudaError_t dispatch(const PagedArgs &a, const Bounds &h, cudaStream_t s, int64_t *want) {
    const int64_t rows = (int64_t)h.max_new * (a.Hq / a.Hkv);
    // (32 columns of three terms and heads of 128 leave no room for 8-bit pages' stages)
    constexpr bool kNarrow = HD == 128 && TERMS == 3 && Q8;
    // More units than SMs: two CTAs an SM with half the ring each, so that one's set-up and
    // end lie behind the other's tiles (bf16, 64 x 1,000 rows 40.7 -> 31.0 us, 32 x 199 to
    // 4,099 37.7 -> 35.4; with fewer the ring counts: 19 x 4,000 32.8 -> 34.8).
    if constexpr (HD == 64 && !Q8)
        if (rows <= 16 && std::min(a.B, a.n) * a.Hkv > h.n_sm)
            return launch<PagedFew<HD, TERMS, 16, Q8, 2>>(a, h, s, want);
    if (rows <= 16 || kNarrow) return launch<PagedFew<HD, TERMS, 16, Q8>>(a, h, s, want);
    // (three terms of a head of 128 and two O of 128 columns exceed tensor memory)
    if constexpr (!(HD == 128 && TERMS == 3))
        if (rows > 32) {
            const bool ws = want || a.work;
            if (plan<PagedMany<HD, TERMS, Q8>>(a, h, ws).us < plan<PagedFew<HD, TERMS, 32, Q8>>(a, h, ws).us)
                return launch<PagedMany<HD, TERMS, Q8>>(a, h, s, want);
        }
    if constexpr (!kNarrow) return launch<PagedFew<HD, TERMS, 32, Q8>>(a, h, s, want);
    return cudaErrorInvalidValue;  // (not reached)
}

template <int HD, int TERMS>
cudaError_t dispatch(const PagedArgs &a, const Bounds &h, cudaStream_t s, int64_t *want) {
    return a.ks ? dispatch<HD, TERMS, true>(a, h, s, want) : dispatch<HD, TERMS, false>(a, h, s, want);
}

cudaError_t dispatch(const PagedArgs &a, int hd, bool f32, const Bounds &h, cudaStream_t s, int64_t *want) {
    if (f32) return hd == 64 ? dispatch<64, 3>(a, h, s, want) : dispatch<128, 3>(a, h, s, want);
    return hd == 64 ? dispatch<64, 1>(a, h, s, want) : dispatch<128, 1>(a, h, s, want);
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
    if (q8 && a->page_size % 8) return bad(MK_ERR_INVALID_ARG, "page_size of e4m3 pages must be a multiple of 8");
    const int64_t cap = (int64_t)a->max_pages * a->page_size;
    if (cap > (1 << 29)) return bad(MK_ERR_UNSUPPORTED, "max_pages * page_size above 2^29");
    if (!isfinite(a->scale) || !(a->scale > 0.f)) return bad(MK_ERR_INVALID_ARG, "scale must be finite and > 0");
    if (a->window < 0 || a->sinks < 0) return bad(MK_ERR_INVALID_ARG, "window or sinks is negative");
    if (a->max_new < 0 || a->max_len < 0) return bad(MK_ERR_INVALID_ARG, "max_new or max_len is negative");
    const int64_t row = (int64_t)a->n_heads * a->head_dim;
    if (a->n_kv_heads > 65535 || ((int64_t)a->n_pages + 1) * a->n_kv_heads > INT32_MAX ||
        (int64_t)a->n_tokens * a->n_heads > (1 << 29) || a->batch > (1 << 20))
        return bad(MK_ERR_UNSUPPORTED, "too many tokens, heads, pages or sequences");
    if (a->q_stride < row || a->out_stride < row || (a->q_stride | a->out_stride) % 8)
        return bad(MK_ERR_INVALID_ARG, "a stride is too small or not a multiple of 8 elements");
    const uintptr_t all = reinterpret_cast<uintptr_t>(a->q) | reinterpret_cast<uintptr_t>(a->out) |
                          reinterpret_cast<uintptr_t>(a->k_pages) | reinterpret_cast<uintptr_t>(a->v_pages) |
                          reinterpret_cast<uintptr_t>(a->workspace);
    if ((all & 15u) || (q8 && ((reinterpret_cast<uintptr_t>(a->k_scales) | reinterpret_cast<uintptr_t>(a->v_scales)) & 15u)))
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
        // what is written apart from everything else: the rows of out, the workspace and the status word
        const int64_t b = a->batch, work = a->workspace ? a->workspace_bytes : 0, word = a->status ? 4 : 0;
        const struct {
            const void *at;
            int64_t bytes;
        } read[] = {{a->table, b * a->max_pages * 4}, {a->starts, b ? (b + 1) * 4 : 0}, {a->lengths, b * 4},
                    {a->q, q_bytes}, {a->k_pages, pool}, {a->v_pages, pool}, {a->k_scales, scales},
                    {a->v_scales, scales}};
        auto out_meets = [&](const void *at, int64_t bytes) {
            return mkops::meet_rows(a->out, a->n_tokens, a->out_stride * e, row * e, at, bytes);
        };
        bool met = out_meets(a->workspace, work) || out_meets(a->status, word) || meet(a->workspace, work, a->status, word);
        for (int i = 0; i < 8; ++i)
            met = met || (i < 3 && out_meets(read[i].at, read[i].bytes)) ||
                  meet(a->workspace, work, read[i].at, read[i].bytes) || meet(a->status, word, read[i].at, read[i].bytes);
        if (met) return bad(MK_ERR_INVALID_ARG, "out, the workspace or status overlaps something else");
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

mkops::Bounds bounds_of(const mk_paged_args *a, const mkops::PagedArgs &p) {
    return {a->max_new ? std::min(a->max_new, a->n_tokens) : a->n_tokens, a->max_len ? std::min(a->max_len, p.cap) : p.cap,
            mkops::sm_count()};
}

}  // namespace

extern "C" int mk_paged_attention(const mk_paged_args *a, void *stream) {
    mkops::PagedArgs p;
    const int rc = check_paged(a, &p);
    if (rc || a->batch == 0 || a->n_tokens == 0) return rc;
    const mkops::Bounds h = bounds_of(a, p);
    const cudaError_t e =
        mkops::dispatch(p, a->head_dim, a->dtype == MK_F32, h, static_cast<cudaStream_t>(stream), nullptr);
    return e == cudaSuccess ? MK_OK : mkops::cuda_error(e, "mk_paged_attention");
}

extern "C" int64_t mk_paged_attention_workspace(const mk_paged_args *a) {
    mkops::PagedArgs p;
    const int rc = check_paged(a, &p);
    if (rc || a->batch == 0 || a->n_tokens == 0) return rc;
    const mkops::Bounds h = bounds_of(a, p);
    int64_t floats = 0;
    const cudaError_t e = mkops::dispatch(p, a->head_dim, a->dtype == MK_F32, h, nullptr, &floats);
    return e == cudaSuccess ? floats * 4 : mkops::cuda_error(e, "mk_paged_attention_workspace");
}
