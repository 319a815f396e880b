// mk_kv.cu — moves of rows inside the KV cache: mk_kv_compact (the accepted
// path of a drafted tree, behind the committed rows) and mk_kv_reorder (slots
// copied, forked and exchanged).
//
// Both are pure copies: their floor is the memory's rate, each moved row read once
// and written once (reorder: 2,000 rows of 6 of 8 slots, 16 layers, 620 MB, 101 us =
// 6.1 TB/s; compact, whose rows are few and mostly in L2, is bound by three dependent
// loads: 8 x 40 rows of 28 layers, 73 MB, 13.7 us). The one thing to get right is that sources and
// targets overlap, so every thread has all its loads behind it before the
// first store that could touch another's source:
//   compact: one CTA holds all moved rows of one (layer, slot, head), K and V,
//     in registers, a barrier between its loads and its stores (no other CTA
//     touches those rows);
//   reorder: a thread owns one 16-byte column of a cache row in ALL slots;
//     it loads what every slot will hold and then stores, so any mapping of
//     slots, cycles too, needs no second buffer and no barrier.
#include <cuda_runtime.h>
#include <stdint.h>

#include "mk_internal.h"
#include "mk_ops.h"

namespace mkops {
namespace {

constexpr int kMaxNodes = 64;
constexpr int kT = 256;

// grid (L * Hkv, B): CTA of (layer, head) and slot; K and V, so that twice the
// loads are in flight.
template <int HD>
__global__ void __launch_bounds__(kT) kv_compact(uint16_t *kc, uint16_t *vc, int L, int B, int Hkv, int max_seq, int T,
                                                 const int32_t *__restrict__ starts, const int32_t *__restrict__ nodes,
                                                 const int32_t *__restrict__ counts) {
    constexpr int CPR = HD / 8;                   // 16-byte chunks of a row
    constexpr int NC = kMaxNodes * CPR / kT;      // chunks of a thread
    const int b = blockIdx.y, tid = threadIdx.x;
    pdl_begin();
    const int l = blockIdx.x / Hkv, h = blockIdx.x % Hkv;
    const int start = starts[b], n = min(counts[b], T);
    if (start < 0 || n <= 0) return;
    const int64_t at = (((int64_t)l * B + b) * Hkv + h) * max_seq * HD;
    uint4 *krows = reinterpret_cast<uint4 *>(kc + at), *vrows = reinterpret_cast<uint4 *>(vc + at);
    uint4 k[NC], v[NC];
    bool move[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const int i = (tid + c * kT) / CPR, part = tid % CPR;
        move[c] = false;
        if (i < n) {
            const int node = nodes[(int64_t)b * T + i];
            const int64_t src = (int64_t)start + node, dst = (int64_t)start + i;
            move[c] = node >= 0 && node != i && src < max_seq && dst < max_seq;
            if (move[c]) {
                k[c] = krows[src * CPR + part];
                v[c] = vrows[src * CPR + part];
            }
        }
    }
    __syncthreads();
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const int64_t to = ((int64_t)start + (tid + c * kT) / CPR) * CPR + tid % CPR;
        if (move[c]) {
            krows[to] = k[c];
            vrows[to] = v[c];
        }
    }
}

// grid (blocks of a plane, 2 * L * Hkv); V = uint4 (NB <= 32) or uint2 (64).
template <typename V, int NB>
__global__ void __launch_bounds__(kT) kv_reorder(V *kc, V *vc, int L, int B, int Hkv, int max_seq, int cpr,
                                                 const int32_t *__restrict__ sources,
                                                 const int32_t *__restrict__ lengths) {
    __shared__ int src[NB], len[NB];
    __shared__ int most;
    const int tid = threadIdx.x;
    if (tid == 0) most = 0;
    pdl_begin();
    __syncthreads();
    if (tid < NB) {
        int s = tid < B ? sources[tid] : tid;
        int n = tid < B ? min(max(lengths[tid], 0), max_seq) : 0;
        if (s < 0 || s >= B || s == tid) n = 0;  // stays as it is
        src[tid] = n ? s : 0;
        len[tid] = n;
        if (n) atomicMax(&most, n);
    }
    __syncthreads();
    const int plane = blockIdx.y % (L * Hkv), l = plane / Hkv, h = plane % Hkv;
    V *cache = blockIdx.y < L * Hkv ? kc : vc;
    const int64_t slot_stride = (int64_t)Hkv * max_seq * cpr;
    V *base = cache + ((int64_t)l * B * Hkv + h) * max_seq * cpr;
    const int64_t total = (int64_t)most * cpr;
    for (int64_t i = (int64_t)blockIdx.x * kT + tid; i < total; i += (int64_t)gridDim.x * kT) {
        const int row = (int)(i / cpr);
        V v[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b)
            if (row < len[b]) v[b] = base[src[b] * slot_stride + i];
#pragma unroll
        for (int b = 0; b < NB; ++b)
            if (row < len[b]) base[b * slot_stride + i] = v[b];
    }
}

int check_cache(const char *who, const void *k, const void *v, int L, int B, int Hkv, int max_seq, int hd) {
    using mkint::set_error;
    if (!k || !v) return set_error(MK_ERR_INVALID_ARG, who);
    if (L < 1 || B < 1 || Hkv < 1 || max_seq < 1) return set_error(MK_ERR_INVALID_ARG, who);
    if (hd != 64 && hd != 128) return set_error(MK_ERR_UNSUPPORTED, who);
    if ((reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v)) & 15u)
        return set_error(MK_ERR_INVALID_ARG, who);
    if ((int64_t)L * Hkv > 32767 || B > 65535) return set_error(MK_ERR_UNSUPPORTED, who);
    return MK_OK;
}

// (kv_reorder's CTAs take K or V: a shared row would move twice)
bool caches_meet(const void *k, const void *v, int L, int B, int Hkv, int max_seq, int hd) {
    const int64_t bytes = 2 * (int64_t)L * B * Hkv * max_seq * hd;
    return meet(k, bytes, v, bytes);
}

}  // namespace
}  // namespace mkops

extern "C" int mk_kv_compact(void *k, void *v, int32_t n_layers, int32_t slots, int32_t n_kv_heads, int32_t max_seq,
                             int32_t head_dim, int32_t nodes_per_slot, const int32_t *d_starts, const int32_t *d_nodes,
                             const int32_t *d_counts, void *stream) {
    using mkint::set_error;
    const int rc = mkops::check_cache("mk_kv_compact: bad cache (pointer, alignment, size or head_dim)", k, v,
                                      n_layers, slots, n_kv_heads, max_seq, head_dim);
    if (rc) return rc;
    if (!d_starts || !d_nodes || !d_counts)
        return set_error(MK_ERR_INVALID_ARG, "mk_kv_compact: a required pointer is NULL");
    if (nodes_per_slot < 1 || nodes_per_slot > mkops::kMaxNodes)
        return set_error(MK_ERR_INVALID_ARG, "mk_kv_compact: nodes_per_slot outside [1, MK_MAX_TREE]");
    if (mkops::caches_meet(k, v, n_layers, slots, n_kv_heads, max_seq, head_dim))
        return set_error(MK_ERR_INVALID_ARG, "mk_kv_compact: k and v overlap");
    const dim3 grid(n_layers * n_kv_heads, slots);
    uint16_t *kc = static_cast<uint16_t *>(k), *vc = static_cast<uint16_t *>(v);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    auto go = [&](auto kernel) {
        return mkops::launch_op(kernel, grid, mkops::kT, 0, 0, s, kc, vc, n_layers, slots, n_kv_heads, max_seq,
                                nodes_per_slot, d_starts, d_nodes, d_counts);
    };
    const cudaError_t e = head_dim == 64 ? go(mkops::kv_compact<64>) : go(mkops::kv_compact<128>);
    return e == cudaSuccess ? MK_OK : mkops::cuda_error(e, "mk_kv_compact");
}

extern "C" int mk_kv_reorder(void *k, void *v, int32_t n_layers, int32_t slots, int32_t n_kv_heads, int32_t max_seq,
                             int32_t head_dim, const int32_t *d_sources, const int32_t *d_lengths, void *stream) {
    using mkint::set_error;
    const int rc = mkops::check_cache("mk_kv_reorder: bad cache (pointer, alignment, size or head_dim)", k, v,
                                      n_layers, slots, n_kv_heads, max_seq, head_dim);
    if (rc) return rc;
    if (!d_sources || !d_lengths)
        return set_error(MK_ERR_INVALID_ARG, "mk_kv_reorder: a required pointer is NULL");
    if (slots > 64) return set_error(MK_ERR_UNSUPPORTED, "mk_kv_reorder: more than 64 slots");
    if (mkops::caches_meet(k, v, n_layers, slots, n_kv_heads, max_seq, head_dim))
        return set_error(MK_ERR_INVALID_ARG, "mk_kv_reorder: k and v overlap");
    const int planes = 2 * n_layers * n_kv_heads;
    const int64_t chunks = (int64_t)max_seq * head_dim / 8;
    int64_t per = (chunks + mkops::kT - 1) / mkops::kT;
    const int64_t want = (mkops::sm_count() * 16 + planes - 1) / planes;
    if (per > want) per = want;
    const dim3 grid((unsigned)per, planes);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int cpr = head_dim / 8;
    auto go = [&](auto kernel, auto *kc, auto *vc, int c) {
        return mkops::launch_op(kernel, grid, mkops::kT, 0, 0, s, kc, vc, n_layers, slots, n_kv_heads, max_seq, c,
                                d_sources, d_lengths);
    };
    uint4 *k4 = static_cast<uint4 *>(k), *v4 = static_cast<uint4 *>(v);
    const cudaError_t e = slots <= 4    ? go(mkops::kv_reorder<uint4, 4>, k4, v4, cpr)
                          : slots <= 8  ? go(mkops::kv_reorder<uint4, 8>, k4, v4, cpr)
                          : slots <= 16 ? go(mkops::kv_reorder<uint4, 16>, k4, v4, cpr)
                          : slots <= 32 ? go(mkops::kv_reorder<uint4, 32>, k4, v4, cpr)
                                        : go(mkops::kv_reorder<uint2, 64>, static_cast<uint2 *>(k),
                                             static_cast<uint2 *>(v), 2 * cpr);
    return e == cudaSuccess ? MK_OK : mkops::cuda_error(e, "mk_kv_reorder");
}
