// mk_tree.cu — attention of a tree of drafted tokens over the KV cache
// (mk_tree_attention), the ancestor masks of such a tree (mk_tree_masks) and
// the host-side walk that accepts a path of it (mk_tree_accept).
//
// Mathematics, for node t of sequence b, query head h, kv head h / G:
//   s_j = scale * q . k_j for the cache rows j the node sees: every row below
//   lengths[b], and row lengths[b] + i where bit i of masks[b][t] is set;
//   o = sum_j exp(s_j - m) v_j / sum_j exp(s_j - m), m = max_j s_j,
// in one pass over the rows with the running maximum and sum. A node that
// sees no row gets zeros.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <stdio.h>

#include <algorithm>
#include <atomic>

#include "mk_internal.h"
#include "mk_ops.h"
#include "mk_tree_attn.cuh"

namespace mkops {
namespace {

// One warp per sequence; lane l walks up from nodes l and l + 32. (rows and
// length, of a single sequence, are the pass through a model's.)
__global__ void __launch_bounds__(32) tree_masks(const int32_t *__restrict__ parents,
                                                 const int32_t *__restrict__ counts, int T, int start,
                                                 uint64_t *masks, int32_t *depths, int32_t *rows, int32_t *length) {
    __shared__ int32_t up[MK_MAX_TREE];
    pdl_begin();
    const int b = blockIdx.x, n = counts ? min(max(counts[b], 0), T) : T;
    for (int t = threadIdx.x; t < n; t += 32) {
        const int p = parents[(int64_t)b * T + t];
        up[t] = p < t ? p : -1;  // a parent comes before its child
    }
    __syncwarp();
    for (int t = threadIdx.x; t < n; t += 32) {
        uint64_t m = 0;
        int depth = -1;
        for (int x = t; x >= 0; x = up[x]) {  // falls with every step
            m |= 1ull << x;
            ++depth;
        }
        masks[(int64_t)b * T + t] = m;
        if (depths) depths[(int64_t)b * T + t] = start + depth;
        if (rows) rows[t] = start + t;
    }
    if (length && threadIdx.x == 0) *length = start;
}

}  // namespace

int sm_count() {
    static const int n = [] {
        int dev = 0, sms = 0;
        if (cudaGetDevice(&dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms < 1) {
            (void)cudaGetLastError();
            sms = 152;
        }
        return sms;
    }();
    return n;
}

int cuda_error(cudaError_t e, const char *what) {
    char text[256];
    snprintf(text, sizeof text, "%s: %s", what, cudaGetErrorString(e));
    return mkint::set_error(MK_ERR_CUDA, text);
}

namespace {

typedef CUresult (*EncodeTiled)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encoder() {
    static const EncodeTiled fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<EncodeTiled>(p);
    }();
    return fn;
}

}  // namespace

// The cache of one layer as [planes][max_seq][hd], boxes of `box` rows x 64
// dims, 128-byte swizzle. Made for each call (it holds the address).
bool cache_map(CUtensorMap *map, const void *cache, int planes, int max_seq, int hd, int box_rows) {
    const EncodeTiled enc = encoder();
    if (!enc) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)hd, (cuuint64_t)max_seq, (cuuint64_t)planes};
    const cuuint64_t strides[2] = {(cuuint64_t)hd * 2, (cuuint64_t)max_seq * hd * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)box_rows, 1}, one[3] = {1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(cache), dims, strides, box, one,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

namespace {

// How a call splits the cache rows of its (row tile, sequence, kv head) units:
// S CTAs of one cluster, or (ws) S CTAs whose partial results go through the
// workspace.
struct Plan {
    int S;
    bool ws;
    double us;  // its estimated time
};

// The two kernels by what their launch needs.
template <int HD_, int TERMS_, int NR_>
struct Few {
    static constexpr int kThreads = kAttnThreads, HD = HD_, TERMS = TERMS_, NR = NR_, kSmem = AttnShape<HD, TERMS, NR>::kSmem;
    static constexpr double kTileUs = (HD == 64 ? 0.6 : 1.0) - (TERMS == 1 ? HD / 64 * 0.1 : 0.0), kFixedUs = 5.0, kJoinUs = 4.5;
    static auto fn() { return tree_attention<HD, TERMS, NR>; }
};
template <int HD_, int TERMS_>
struct Many {
    static constexpr int kThreads = kAttnThreads, HD = HD_, TERMS = TERMS_, NR = kRows, kSmem = RowShape<HD, TERMS>::kSmem;
    static constexpr double kTileUs = HD == 64 && TERMS == 1 ? 0.8 : 1.2, kFixedUs = 6.5, kJoinUs = 7.0;
    static auto fn() { return tree_attention_rows<HD, TERMS>; }
};

// The split with the least estimated time, in microseconds: waves of resident
// CTAs x (the tiles of a split x K::kTileUs + a fixed part). The tile times are
// those of one split over a cache (S = 1: 65 tiles of 32 fp32 rows with heads of 64
// 43.1 us, of 32 bf16 rows 36.1, of 128 bf16 rows 58.2; 17 tiles with heads of 128 of
// 32 fp32 rows 21.4 us, of 32 bf16 rows 20.7, of 128 bf16 rows 26.6; each
// with K::kFixedUs of launch, set-up and end); more than a
// cluster's splits cost K::kJoinUs: a second launch and the partial results'
// way through memory. (That pays from about 3,000 rows on where whole waves of clusters
// leave SMs free: two trees of 38 nodes, 16 heads of 128 a kv head, fp32, 3,875 rows
// 16.9 us, in clusters 21.4.)
template <class K>
Plan plan(const TreeArgs &a, int max_len, int n_sm, bool ws) {
    const int row_tiles = (a.T * (a.Hq / a.Hkv) + K::NR - 1) / K::NR;
    const int64_t units = (int64_t)a.B * a.Hkv * row_tiles;
    const int tiles = (std::min((int64_t)max_len + a.T, (int64_t)a.max_seq) + kTile - 1) / kTile;
    Plan best{1, false, 1e30};
    for (int k = 0; k < 4 && (1 << k) <= tiles; ++k) {
        const int S = 1 << k, at_once = active_clusters<K>(k, n_sm);
        const double us =
            (double)((units + at_once - 1) / at_once) * (((tiles + S - 1) / S) * K::kTileUs + K::kFixedUs) +
            (k ? 0.8 + 0.2 * k : 0.0);  // (the cluster's join)
        if (us < best.us) best = Plan{S, false, us};
    }
    if (ws) {
        const int64_t room = active_clusters<K>(0, n_sm) / units;
        const int S = (int)std::min<int64_t>(std::min<int64_t>(room, max_splits(K::NR)), tiles / 2);
        const double us = ((tiles + S - 1) / std::max(S, 1)) * K::kTileUs + K::kFixedUs + K::kJoinUs;
        if (S > 1 && us < best.us) best = Plan{S, true, us};
    }
    return best;
}

template <class K>
cudaError_t launch(TreeArgs a, int max_len, int n_sm, cudaStream_t s, int64_t *want) {
    const int row_tiles = (a.T * (a.Hq / a.Hkv) + K::NR - 1) / K::NR;
    cudaError_t e = configure<K>();
    if (e != cudaSuccess) return e;
    Plan p = plan<K>(a, max_len, n_sm, want || a.work);
    const int64_t need = p.ws ? (int64_t)a.B * a.Hkv * row_tiles * p.S * part_floats(K::NR, K::HD) : 0;
    if (want) {
        *want = need;
        return cudaSuccess;
    }
    if (need > a.work_floats) p = plan<K>(a, max_len, n_sm, false);
    a.part = p.ws ? a.work : nullptr;
    if (a.wait_ns == 0) a.wait_ns = kWaitNs;
    a.wait_sleep = (uint32_t)std::min<uint64_t>(a.wait_ns, kSleepNs);
    CUtensorMap kmap, vmap;
    if (!cache_map(&kmap, a.kc, a.slots * a.Hkv, a.max_seq, K::HD, kTile) ||
        !cache_map(&vmap, a.vc, a.slots * a.Hkv, a.max_seq, K::HD, kTile))
        return cudaErrorInvalidValue;
    e = launch_op(K::fn(), dim3(p.S, a.B * a.Hkv, row_tiles), kAttnThreads, K::kSmem, p.ws ? 1 : p.S, s, kmap, vmap, a);
    if (e != cudaSuccess || !p.ws) return e;
    return launch_op(tree_join<K::HD, K::TERMS, K::NR>,
                     dim3(row_tiles, a.B * a.Hkv, (K::NR * K::HD / 4 + 255) / 256), 256, 0, 0, s, a, p.S);
}

// The kernel of 16 or 32 columns that holds the tree's rows of a kv head; for more
// rows, several CTAs of 32 or the kernel of 128 rows, whichever plan is shorter.
// (Measured, 64 bf16 rows over 8,208 cache rows: 13.0 us with 32 columns, 16.1 with
// 128 rows; 244 bf16 rows and 64 (sequence, kv head) pairs: 58.2 us with 128 rows, four
// waves of 36 with 32 columns.)
template <int HD, int TERMS>
cudaError_t dispatch(const TreeArgs &a, int max_len, int n_sm, cudaStream_t s, int64_t *want) {
    const int rows = a.T * (a.Hq / a.Hkv);
    if (rows <= 16) return launch<Few<HD, TERMS, 16>>(a, max_len, n_sm, s, want);
    // (three terms of a head of 128 and two O of 128 columns exceed tensor memory)
    if constexpr (!(HD == 128 && TERMS == 3))
        if (rows > 32) {
            const bool ws = want || a.work;
            if (plan<Many<HD, TERMS>>(a, max_len, n_sm, ws).us < plan<Few<HD, TERMS, 32>>(a, max_len, n_sm, ws).us)
                return launch<Many<HD, TERMS>>(a, max_len, n_sm, s, want);
        }
    return launch<Few<HD, TERMS, 32>>(a, max_len, n_sm, s, want);
}

cudaError_t dispatch(const TreeArgs &a, int hd, bool f32, int max_len, int n_sm, cudaStream_t s, int64_t *want) {
    if (f32) return hd == 64 ? dispatch<64, 3>(a, max_len, n_sm, s, want) : dispatch<128, 3>(a, max_len, n_sm, s, want);
    return hd == 64 ? dispatch<64, 1>(a, max_len, n_sm, s, want) : dispatch<128, 1>(a, max_len, n_sm, s, want);
}

}  // namespace

cudaError_t tree_attention_launch(const TreeArgs &a, int hd, bool f32, int max_len, int n_sm, cudaStream_t s) {
    return dispatch(a, hd, f32, max_len, n_sm, s, nullptr);
}

cudaError_t tree_attention_work_floats(const TreeArgs &a, int hd, bool f32, int max_len, int n_sm, int64_t *floats) {
    return dispatch(a, hd, f32, max_len, n_sm, nullptr, floats);
}

cudaError_t tree_masks_launch(const int32_t *parents, const int32_t *counts, int B, int T, uint64_t *masks,
                              int32_t *depths, cudaStream_t s) {
    return launch_op(tree_masks, dim3(B), 32, 0, 0, s, parents, counts, T, 0, masks, depths, nullptr, nullptr);
}

cudaError_t tree_plan_launch(const int32_t *parents, int n, int start, uint64_t *masks, int32_t *positions,
                             int32_t *rows, int32_t *length, cudaStream_t s) {
    return launch_op(tree_masks, dim3(1), 32, 0, 0, s, parents, nullptr, n, start, masks, positions, rows, length);
}

}  // namespace mkops

namespace {

int check_tree(const mk_tree_args *a) {
    using mkint::set_error;
    if (!a || !a->q || !a->out || !a->k_cache || !a->v_cache || !a->lengths || !a->masks)
        return set_error(MK_ERR_INVALID_ARG, "mk_tree_attention: a required pointer is NULL");
    if (a->dtype != MK_F32 && a->dtype != MK_BF16)
        return set_error(MK_ERR_INVALID_ARG, "mk_tree_attention: dtype is neither MK_F32 nor MK_BF16");
    if (a->head_dim != 64 && a->head_dim != 128)
        return set_error(MK_ERR_UNSUPPORTED, "mk_tree_attention: head_dim must be 64 or 128");
    if (a->batch < 0 || a->n_heads < 1 || a->n_kv_heads < 1 || a->slots < 1 || a->max_seq < 1)
        return set_error(MK_ERR_INVALID_ARG, "mk_tree_attention: bad size");
    if (a->nodes < 1 || a->nodes > MK_MAX_TREE)
        return set_error(MK_ERR_INVALID_ARG, "mk_tree_attention: nodes outside [1, MK_MAX_TREE]");
    if (a->n_heads % a->n_kv_heads || a->n_heads / a->n_kv_heads > MK_MAX_GROUP)
        return set_error(MK_ERR_UNSUPPORTED,
                         "mk_tree_attention: n_heads must be a multiple of n_kv_heads, at most MK_MAX_GROUP times it");
    if (!isfinite(a->scale) || !(a->scale > 0.f))
        return set_error(MK_ERR_INVALID_ARG, "mk_tree_attention: scale must be finite and > 0");
    if (a->max_len < 0 || a->max_len > a->max_seq)
        return set_error(MK_ERR_INVALID_ARG, "mk_tree_attention: max_len outside [0, max_seq]");
    if ((int64_t)a->batch * a->n_kv_heads > 65535 || (int64_t)a->slots * a->n_kv_heads > INT32_MAX)
        return set_error(MK_ERR_UNSUPPORTED, "mk_tree_attention: batch * n_kv_heads above 65535");
    const int64_t row = (int64_t)a->n_heads * a->head_dim;
    if (a->q_token_stride < row || a->out_token_stride < row || a->q_batch_stride < 0 || a->out_batch_stride < 0 ||
        (a->q_token_stride | a->out_token_stride | a->q_batch_stride | a->out_batch_stride) % 8)
        return set_error(MK_ERR_INVALID_ARG, "mk_tree_attention: a stride is too small or not a multiple of 8 elements");
    // the rows of out must not meet: whole sequences behind one another, or whole nodes
    if (a->batch > 1 && a->out_batch_stride < (a->nodes - 1) * a->out_token_stride + row &&
        (a->out_batch_stride < row || a->out_token_stride < (a->batch - 1) * a->out_batch_stride + row))
        return set_error(MK_ERR_INVALID_ARG, "mk_tree_attention: the rows of out overlap");
    if ((reinterpret_cast<uintptr_t>(a->q) | reinterpret_cast<uintptr_t>(a->out) |
         reinterpret_cast<uintptr_t>(a->k_cache) | reinterpret_cast<uintptr_t>(a->v_cache)) & 15u ||
        reinterpret_cast<uintptr_t>(a->masks) & 7u)
        return set_error(MK_ERR_INVALID_ARG, "mk_tree_attention: a pointer is not aligned");
    if (a->workspace_bytes < 0 || (a->workspace && (reinterpret_cast<uintptr_t>(a->workspace) & 15u)))
        return set_error(MK_ERR_INVALID_ARG, "mk_tree_attention: bad workspace");
    if (a->wait_ns < 0) return set_error(MK_ERR_INVALID_ARG, "mk_tree_attention: wait_ns is negative");
    return MK_OK;
}

mkops::TreeArgs tree_of(const mk_tree_args *a) {
    mkops::TreeArgs t{};
    t.B = a->batch, t.T = a->nodes, t.Hq = a->n_heads, t.Hkv = a->n_kv_heads, t.slots = a->slots;
    t.max_seq = a->max_seq, t.scale = a->scale;
    t.q_batch = a->q_batch_stride, t.q_token = a->q_token_stride;
    t.o_batch = a->out_batch_stride, t.o_token = a->out_token_stride;
    t.q = a->q, t.out = a->out;
    t.kc = static_cast<const uint16_t *>(a->k_cache), t.vc = static_cast<const uint16_t *>(a->v_cache);
    t.lengths = a->lengths, t.counts = a->counts, t.slot_of = a->slot_of, t.masks = a->masks;
    t.work = static_cast<float *>(a->workspace);
    t.work_floats = a->workspace ? a->workspace_bytes / 4 : 0;
    t.err = a->status;
    t.wait_ns = (uint64_t)a->wait_ns;
    return t;
}

}  // namespace

extern "C" int mk_tree_attention(const mk_tree_args *a, void *stream) {
    const int rc = check_tree(a);
    if (rc || a->batch == 0) return rc;
    const cudaError_t e =
        mkops::tree_attention_launch(tree_of(a), a->head_dim, a->dtype == MK_F32, a->max_len ? a->max_len : a->max_seq,
                                     mkops::sm_count(), static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? MK_OK : mkops::cuda_error(e, "mk_tree_attention");
}

extern "C" int64_t mk_tree_attention_workspace(const mk_tree_args *a) {
    const int rc = check_tree(a);
    if (rc || a->batch == 0) return rc;
    int64_t floats = 0;
    const cudaError_t e =
        mkops::tree_attention_work_floats(tree_of(a), a->head_dim, a->dtype == MK_F32,
                                          a->max_len ? a->max_len : a->max_seq, mkops::sm_count(), &floats);
    return e == cudaSuccess ? floats * 4 : mkops::cuda_error(e, "mk_tree_attention_workspace");
}

extern "C" int mk_tree_masks(const int32_t *d_parents, const int32_t *d_counts, int32_t batch, int32_t nodes,
                             uint64_t *d_masks, int32_t *d_depths, void *stream) {
    using mkint::set_error;
    if (!d_parents || !d_masks) return set_error(MK_ERR_INVALID_ARG, "mk_tree_masks: a required pointer is NULL");
    if (batch < 0 || nodes < 1 || nodes > MK_MAX_TREE)
        return set_error(MK_ERR_INVALID_ARG, "mk_tree_masks: bad batch, or nodes outside [1, MK_MAX_TREE]");
    if (batch == 0) return MK_OK;
    const cudaError_t e = mkops::tree_masks_launch(d_parents, d_counts, batch, nodes, d_masks, d_depths,
                                                   static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? MK_OK : mkops::cuda_error(e, "mk_tree_masks");
}

extern "C" int mk_tree_accept(const int32_t *tokens, const int32_t *parents, const int32_t *draws, int32_t n,
                              int32_t *path) {
    using mkint::set_error;
    if (!tokens || !parents || !draws || !path)
        return set_error(MK_ERR_INVALID_ARG, "mk_tree_accept: a required pointer is NULL");
    if (n < 1 || n > MK_MAX_TREE) return set_error(MK_ERR_INVALID_ARG, "mk_tree_accept: n outside [1, MK_MAX_TREE]");
    int count = 0, at = 0;
    path[count++] = 0;
    for (int i = 1; i < n; ++i)  // children come behind their parents
        if (parents[i] == at && tokens[i] == draws[at]) {
            at = i;
            path[count++] = i;
        }
    return count;
}
