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

#include "mk_internal.h"
#include "mk_ops.h"
#include "mk_tree_attn.cuh"

namespace mkops {
namespace {

// One warp per sequence; lane l walks up from nodes l and l + 32.
__global__ void __launch_bounds__(32) tree_masks(const int32_t *__restrict__ parents,
                                                 const int32_t *__restrict__ counts, int T, uint64_t *masks,
                                                 int32_t *depths) {
    __shared__ int32_t up[MK_MAX_TREE];
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
        if (depths) depths[(int64_t)b * T + t] = depth;
    }
}

}  // namespace

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

// The cache of one layer as [planes][max_seq][hd], boxes of 128 rows x 64
// dims, 128-byte swizzle. Made for each call (it holds the address).
bool cache_map(CUtensorMap *map, const void *cache, int planes, int max_seq, int hd) {
    const EncodeTiled enc = encoder();
    if (!enc) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)hd, (cuuint64_t)max_seq, (cuuint64_t)planes};
    const cuuint64_t strides[2] = {(cuuint64_t)hd * 2, (cuuint64_t)max_seq * hd * 2};
    const cuuint32_t box[3] = {64, kTile, 1}, one[3] = {1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(cache), dims, strides, box, one,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int HD, int TERMS, int NR>
cudaError_t launch(const TreeArgs &a, int max_len, int n_sm, cudaStream_t s) {
    using C = AttnShape<HD, TERMS, NR>;
    CUtensorMap kmap, vmap;
    if (!cache_map(&kmap, a.kc, a.slots * a.Hkv, a.max_seq, HD) ||
        !cache_map(&vmap, a.vc, a.slots * a.Hkv, a.max_seq, HD))
        return cudaErrorInvalidValue;
    const auto kernel = tree_attention<HD, TERMS, NR>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    const int row_tiles = (a.T * (a.Hq / a.Hkv) + NR - 1) / NR;
    const int64_t units = (int64_t)a.B * a.Hkv * row_tiles;
    const int tiles = (std::min(max_len + a.T, a.max_seq) + kTile - 1) / kTile;
    int S = 1;
    while (S < 16 && units * S * 2 <= n_sm * (HD == 64 ? 2 : 1) && S * 2 <= tiles) S *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(S, a.B * a.Hkv, row_tiles);
    cfg.blockDim = dim3(kAttnThreads);
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = S;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, kmap, vmap, a);
}

}  // namespace

cudaError_t tree_attention_launch(const TreeArgs &a, int hd, bool f32, int max_len, int n_sm, cudaStream_t s) {
    const int rows = a.T * (a.Hq / a.Hkv);
    if (f32) {
        if (hd == 64) return rows <= 16 ? launch<64, 3, 16>(a, max_len, n_sm, s) : launch<64, 3, 32>(a, max_len, n_sm, s);
        return rows <= 16 ? launch<128, 3, 16>(a, max_len, n_sm, s) : launch<128, 3, 32>(a, max_len, n_sm, s);
    }
    if (hd == 64)
        return rows <= 16   ? launch<64, 1, 16>(a, max_len, n_sm, s)
               : rows <= 32 ? launch<64, 1, 32>(a, max_len, n_sm, s)
                            : launch<64, 1, 64>(a, max_len, n_sm, s);
    return rows <= 16   ? launch<128, 1, 16>(a, max_len, n_sm, s)
           : rows <= 32 ? launch<128, 1, 32>(a, max_len, n_sm, s)
                        : launch<128, 1, 64>(a, max_len, n_sm, s);
}

cudaError_t tree_masks_launch(const int32_t *parents, const int32_t *counts, int B, int T, uint64_t *masks,
                              int32_t *depths, cudaStream_t s) {
    tree_masks<<<B, 32, 0, s>>>(parents, counts, T, masks, depths);
    return cudaGetLastError();
}

}  // namespace mkops

extern "C" int mk_tree_attention(const mk_tree_args *a, void *stream) {
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
    if ((reinterpret_cast<uintptr_t>(a->q) | reinterpret_cast<uintptr_t>(a->out) |
         reinterpret_cast<uintptr_t>(a->k_cache) | reinterpret_cast<uintptr_t>(a->v_cache)) & 15u ||
        reinterpret_cast<uintptr_t>(a->masks) & 7u)
        return set_error(MK_ERR_INVALID_ARG, "mk_tree_attention: a pointer is not aligned");
    int dev = 0, n_sm = 0;
    if (a->batch == 0) return MK_OK;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&n_sm, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return mkops::cuda_error(e, "mk_tree_attention");
    mkops::TreeArgs t{};
    t.B = a->batch, t.T = a->nodes, t.Hq = a->n_heads, t.Hkv = a->n_kv_heads, t.slots = a->slots;
    t.max_seq = a->max_seq, t.scale = a->scale;
    t.q_batch = a->q_batch_stride, t.q_token = a->q_token_stride;
    t.o_batch = a->out_batch_stride, t.o_token = a->out_token_stride;
    t.q = a->q, t.out = a->out;
    t.kc = static_cast<const uint16_t *>(a->k_cache), t.vc = static_cast<const uint16_t *>(a->v_cache);
    t.lengths = a->lengths, t.counts = a->counts, t.slot_of = a->slot_of, t.masks = a->masks;
    e = mkops::tree_attention_launch(t, a->head_dim, a->dtype == MK_F32, a->max_len ? a->max_len : a->max_seq, n_sm,
                                     static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? MK_OK : mkops::cuda_error(e, "mk_tree_attention");
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
