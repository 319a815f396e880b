// mk_ops.h — what the standalone operators' sources share (mk_rope.cu,
// mk_tree.cu, mk_kv.cu), and their launches for the C ABI and for the paths of
// the handle (mk_prefill.cu). Not part of the C ABI.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/mk.h"

namespace mkops {

#ifdef __CUDACC__
__device__ __forceinline__ float bf_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf_hi(uint32_t u) { return __uint_as_float(u & 0xFFFF0000u); }

// Programmatic dependent launch: the operators are launched so that they may be
// brought in while the kernel before them in the stream runs; they touch memory
// only behind pdl_wait, which waits for that kernel's end. pdl_trigger lets the
// next one be brought in. Without the launch attribute both do nothing.
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_trigger() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void pdl_begin() {
    pdl_wait();
    pdl_trigger();
}

// Two fp32 rounded to nearest even as bf16, `lo` in the low half.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t u;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(u) : "f"(hi), "f"(lo));
    return u;
}
#endif

// Launches a kernel that begins with pdl_begin, in clusters of `cluster` CTAs
// along x (0: none). Measured in a stream of calls from the host: a rope token
// 4.1 us without the attribute, 3.1 with it; a token's attention 8.2 and 6.0.
template <typename... KArgs, typename... Args>
inline cudaError_t launch_op(void (*kernel)(KArgs...), dim3 grid, int threads, int smem, int cluster, cudaStream_t s,
                             Args &&...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
}

// Whether two ranges of bytes share one.
inline bool meet(const void *a, int64_t a_bytes, const void *b, int64_t b_bytes) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y ? y - x < (uint64_t)a_bytes : x - y < (uint64_t)b_bytes;
}

// SMs of the GPU (of the device that is current at the first call: a machine's are alike).
int sm_count();

// Sets the calling thread's error text from a CUDA error; returns MK_ERR_CUDA.
int cuda_error(cudaError_t e, const char *what);

struct RopeArgs {
    int n, Hq, Hkv, rot, interleaved, slots, max_seq;
    float eps, mscale;
    int64_t qkv_stride, q_stride;  // elements from one token to the next
    const void *qkv;
    void *q_out;
    uint16_t *kc, *vc;
    const int32_t *positions, *rows, *slot_of;
    const double *inv_freq;
    const uint16_t *q_norm, *k_norm;
};

cudaError_t rope_append_launch(const RopeArgs &a, int hd, bool f32, cudaStream_t s);

// Attention of a tree of drafted tokens. Out: out (fp32 or bf16), or, with
// hi set, the hi / lo bf16 terms of the fp32 result at out's strides.
struct TreeArgs {
    int B, T, Hq, Hkv, slots, max_seq;
    float scale;
    int64_t q_batch, q_token, o_batch, o_token;  // strides in elements
    const void *q;
    void *out;
    uint16_t *hi, *lo;
    const uint16_t *kc, *vc;
    const int32_t *lengths, *counts, *slot_of;
    const uint64_t *masks;
    int *err;     // set to 1 if a bounded wait runs out (nullable)
    uint64_t wait_ns;    // limit of a wait, and how long a thread sleeps in it (set by the launch)
    uint32_t wait_sleep;
    float *part;  // the splits' partial results (set by the launch from work)
    float *work;  // the caller's workspace (nullable)
    int64_t work_floats;
};

cudaError_t tree_attention_launch(const TreeArgs &a, int hd, bool f32, int max_len, int n_sm, cudaStream_t s);

// Floats of workspace (TreeArgs::work) with which a call splits long caches
// over more than a cluster's CTAs; 0: it would not use any.
cudaError_t tree_attention_work_floats(const TreeArgs &a, int hd, bool f32, int max_len, int n_sm, int64_t *floats);

cudaError_t tree_masks_launch(const int32_t *parents, const int32_t *counts, int B, int T, uint64_t *masks,
                              int32_t *depths, cudaStream_t s);

// One tree behind `start` committed rows: masks, positions (start + depth), rows
// (start + index) of its n nodes, and *length = start.
cudaError_t tree_plan_launch(const int32_t *parents, int n, int start, uint64_t *masks, int32_t *positions,
                             int32_t *rows, int32_t *length, cudaStream_t s);

}  // namespace mkops
