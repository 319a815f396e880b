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

#include "mk_internal.h"
#include "mk_ops.h"

namespace mkops {
namespace {

constexpr int kT = 256;
constexpr int kW = kT / 32;

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

// One CTA per (query head, node, sequence); warp w takes every 8th row, lane
// l the dims E l .. E l + E - 1.
template <typename TQ, int HD>
__global__ void __launch_bounds__(kT) tree_attention_simple(const TreeArgs a) {
    constexpr int E = HD / 32;
    __shared__ float ms[kW], ls[kW], os[kW][HD];
    const int h = blockIdx.x, t = blockIdx.y, b = blockIdx.z;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Seq s = sequence(a, b);
    if (t >= s.n) return;
    const TQ *q = static_cast<const TQ *>(a.q) + b * a.q_batch + t * a.q_token + (int64_t)h * HD + E * lane;
    float qv[E], o[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
        if constexpr (sizeof(TQ) == 4)
            qv[e] = q[e] * a.scale;
        else
            qv[e] = bf_lo(q[e]) * a.scale;
        o[e] = 0.f;
    }
    const int64_t at = ((int64_t)s.slot * a.Hkv + h / (a.Hq / a.Hkv)) * a.max_seq * HD + E * lane;
    const uint64_t mask = a.masks[(int64_t)b * a.T + t];
    float m = -INFINITY, l = 0.f;
    for (int j = warp; j < s.len + s.n; j += kW) {
        if (j >= s.len && !((mask >> (j - s.len)) & 1)) continue;
        const uint16_t *k = a.kc + at + (int64_t)j * HD, *v = a.vc + at + (int64_t)j * HD;
        float x = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) x = fmaf(qv[e], bf_lo(k[e]), x);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, d);
        const float mn = fmaxf(m, x), c = m == mn ? 1.f : expf(m - mn), p = expf(x - mn);
        l = l * c + p;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = fmaf(p, bf_lo(v[e]), o[e] * c);
        m = mn;
    }
    if (lane == 0) ms[warp] = m, ls[warp] = l;
#pragma unroll
    for (int e = 0; e < E; ++e) os[warp][E * lane + e] = o[e];
    __syncthreads();
    for (int d = threadIdx.x; d < HD; d += kT) {
        float M = -INFINITY, L = 0.f, O = 0.f;
        for (int w = 0; w < kW; ++w) M = fmaxf(M, ms[w]);
        for (int w = 0; w < kW; ++w) {
            const float c = ms[w] == -INFINITY ? 0.f : expf(ms[w] - M);
            L = fmaf(ls[w], c, L);
            O = fmaf(os[w][d], c, O);
        }
        const float y = M == -INFINITY ? 0.f : O / L;
        const int64_t to = b * a.o_batch + t * a.o_token + (int64_t)h * HD + d;
        if (a.hi) {
            const uint32_t u = pack_bf16(y, 0.f);
            a.hi[to] = (uint16_t)u;
            a.lo[to] = (uint16_t)pack_bf16(y - bf_lo(u), 0.f);
        } else if constexpr (sizeof(TQ) == 4) {
            static_cast<float *>(a.out)[to] = y;
        } else {
            static_cast<uint16_t *>(a.out)[to] = (uint16_t)pack_bf16(y, 0.f);
        }
    }
}

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

cudaError_t tree_attention_launch(const TreeArgs &a, int hd, bool f32, int max_len, int n_sm, cudaStream_t s) {
    const dim3 grid(a.Hq, a.T, a.B);
    if (f32) {
        if (hd == 64)
            tree_attention_simple<float, 64><<<grid, kT, 0, s>>>(a);
        else
            tree_attention_simple<float, 128><<<grid, kT, 0, s>>>(a);
    } else {
        if (hd == 64)
            tree_attention_simple<uint16_t, 64><<<grid, kT, 0, s>>>(a);
        else
            tree_attention_simple<uint16_t, 128><<<grid, kT, 0, s>>>(a);
    }
    return cudaGetLastError();
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
