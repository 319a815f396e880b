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

// ---- rows in 8 bits: e4m3 codes with a power of two 2^(s - 127) for each 32 elements.
constexpr uint32_t kNoScale = 255;  // the block holds no numbers

// The byte s of a block from its largest magnitude: 448 = 1.75 * 2^8, so the
// exponent is that of `most` less 8, one more where its mantissa exceeds 1.75.
__device__ __forceinline__ uint32_t e4m3_scale(float most) {
    const uint32_t bits = __float_as_uint(most);
    if (bits >= 0x7F800000u) return kNoScale;
    const int s = (int)(bits >> 23) - 8 + ((bits & 0x7FFFFFu) > 0x600000u);
    return (uint32_t)min(max(s, 127 - 100), 127 + 7);
}

// Four values as codes: x * 2^(127 - s) is exact, and rounded once.
__device__ __forceinline__ uint32_t e4m3_codes(float4 x, uint32_t s) {
    const float up = __uint_as_float((254u - s) << 23);
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(x.y * up), "f"(x.x * up));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(x.w * up), "f"(x.z * up));
    return s == kNoScale ? 0u : (uint32_t)lo | (uint32_t)hi << 16;
}

// The factor of e4m3_values, twice: a code's bits put at bf16's place are its value
// * 2^-120, denormals too, and 2^(s - 7) is a bf16 number up to s = 134; above: not a number.
__device__ __forceinline__ uint32_t e4m3_factor2(uint32_t s2) {  // of s in both halves
    return s2 > 134 * 0x00010001u ? 0x7FFF7FFFu : s2 * 128u + 120 * 0x00800080u;
}
__device__ __forceinline__ uint32_t e4m3_factor(uint32_t s) { return e4m3_factor2(s * 0x00010001u); }

// Four codes as bf16 (exact for s >= 3: a code's last bit is 2^-9, bf16's 2^-133). A code c = 128 sign + m belongs at 2^15 sign +
// 16 m: 16 c + 240 (c & 128), two multiplications (shifts and masks took twice the ALU's time).
__device__ __forceinline__ uint2 e4m3_values(uint32_t codes, uint32_t factor) {
    uint2 y;
    uint32_t u = __byte_perm(codes, 0, 0x4140), v = __byte_perm(codes, 0, 0x4342);
    u = u * 16u + (u & 0x00800080u) * 240u;
    v = v * 16u + (v & 0x00800080u) * 240u;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(y.x) : "r"(u), "r"(factor));
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(y.y) : "r"(v), "r"(factor));
    return y;
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
    if (a_bytes <= 0 || b_bytes <= 0) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y ? y - x < (uint64_t)a_bytes : x - y < (uint64_t)b_bytes;
}

// The same for n rows of `row` bytes, `step` apart (what lies between them is not theirs).
inline bool meet_rows(const void *a, int64_t n, int64_t step, int64_t row, const void *b, int64_t b_bytes) {
    if (n <= 0 || b_bytes <= 0) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    if (y <= x) return x - y < (uint64_t)b_bytes;
    const uint64_t k = (y - x) / (uint64_t)step, at = (y - x) % (uint64_t)step;  // b begins `at` behind row k's start
    if (k >= (uint64_t)n) return false;
    return at < (uint64_t)row || (k + 1 < (uint64_t)n && (uint64_t)b_bytes > (uint64_t)step - at);
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
    uint16_t *kc, *vc;  // bf16, or with ks set e4m3 codes
    uint8_t *ks, *vs;
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

// log2 of a pool's page size, 31 with one page a sequence; false for a size that is not allowed.
bool page_shift(int page_size, int max_pages, int *shift);

// Attention of ragged new tokens over a cache in pages.
struct PagedArgs {
    int n, B, max_pages, Hq, Hkv, n_pages, ps, shift;  // ps = 1 << shift, or one page a sequence (shift 31)
    int cap, window, sinks;                            // most rows of a sequence; window 0: none
    int units;                                         // tiles of query rows in the grid (set by the launch)
    float scale;
    int64_t q_stride, o_stride;
    const void *q;
    void *out;
    const void *kc, *vc;
    const uint8_t *ks, *vs;  // of e4m3 pages, else NULL
    const int32_t *table, *starts, *lengths;
    int *err;  // as in TreeArgs, and the following
    uint64_t wait_ns;
    uint32_t wait_sleep;
    float *part;
    float *work;
    int64_t work_floats;
};

cudaError_t tree_masks_launch(const int32_t *parents, const int32_t *counts, int B, int T, uint64_t *masks,
                              int32_t *depths, cudaStream_t s);

// One tree behind `start` committed rows: masks, positions (start + depth), rows
// (start + index) of its n nodes, and *length = start.
cudaError_t tree_plan_launch(const int32_t *parents, int n, int start, uint64_t *masks, int32_t *positions,
                             int32_t *rows, int32_t *length, cudaStream_t s);

}  // namespace mkops
