// kv.cuh -- shared by the paged 8-bit key/value cache kernels: the cache and
// batch as kernels see them, device-side checks, code conversions, launch.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kernels.h"
#include "ptx.cuh"

namespace w4a16 {

constexpr int kKvInt8 = 0, kKvE4m3 = 1;
constexpr float kKvScaleMin = 8.673617379884035e-19f;   // 2^-60

__device__ __forceinline__ void kv_report(int *status) { atomicExch(status, kStatusBadArg); }

// One sequence of a batch: rows [q0, q0 + n) of the token tensors, at
// positions [len - n, len) of its cache.
struct KvSeq {
    int q0, n, len;
};

// Device-side arrays are not trusted: rows stay in [0, n_tokens], the length
// within the table's width; whatever had to be clamped is reported.
__device__ __forceinline__ KvSeq kv_sequence(const KvBatch &b, int page_shift, int i, int *status) {
    const int s0 = b.q_starts[i], s1 = b.q_starts[i + 1], len = b.kv_lens[i];
    const int cap = b.max_blocks << page_shift;
    KvSeq s;
    s.q0 = min(max(s0, 0), b.n_tokens);
    s.n = min(max(s1, s.q0), b.n_tokens) - s.q0;
    s.len = min(max(len, 0), cap);
    if (s.q0 != s0 || s.q0 + s.n != s1 || s.len != len || s.n > s.len) kv_report(status);
    return s;
}

// The page of position block `blk` (below the table's width) of sequence i, or -1 (reported).
__device__ __forceinline__ int kv_page(const KvCache &c, const KvBatch &b, int i, int blk, int *status) {
    const int p = b.block_table[(long long)i * b.max_blocks + blk];
    if (p >= 0 && p < c.n_pages) return p;
    kv_report(status);
    return -1;
}

// Rows of the output that no sequence owns, before `lo` and from `hi` on: zeros,
// and a log-sum-exp of -inf.  A row a CTA, all CTAs and threads of the launch.
__device__ __forceinline__ void kv_empty_rows(const KvAttentionArgs &a, const KvBatch &b, int head_dim, int lo, int hi) {
    const int vecs = a.n_heads * head_dim / 8;
    for (long long r = blockIdx.x; r < (long long)lo + b.n_tokens - hi; r += gridDim.x) {
        const long long row = r < lo ? r : r - lo + hi;
        for (int i = threadIdx.x; i < vecs; i += blockDim.x)
            static_cast<uint4 *>(a.out)[row * vecs + i] = make_uint4(0, 0, 0, 0);
        for (int i = threadIdx.x; a.lse && i < a.n_heads; i += blockDim.x) a.lse[row * a.n_heads + i] = -INFINITY;
    }
}

// Test hook: whether this CTA of an attention kernel issues no copies, so that its waits run out.
__device__ __forceinline__ bool kv_holds(int hold) { return hold != 0 && (hold < 2 || blockIdx.x % hold == 0); }

// ---- activations
template <int DT>
__device__ __forceinline__ float kv_act(uint16_t v) {
    return DT == 0 ? __half2float(__ushort_as_half(v)) : __bfloat162float(__ushort_as_bfloat16(v));
}
template <int DT>
__device__ __forceinline__ uint16_t kv_to_act(float v) {
    return DT == 0 ? __half_as_ushort(__float2half_rn(v)) : __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

// ---- codes
// Four codes of a word as fp32.
template <int KT>
__device__ __forceinline__ void kv_decode4(uint32_t w, float (&v)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (KT == kKvInt8) {
            v[i] = (float)(int8_t)(w >> (8 * i));
        } else {
            const __half_raw h = __nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)(w >> (8 * i)), __NV_E4M3);
            v[i] = __half2float(h);
        }
    }
}

// Four values as a word of codes: to the nearest, ties to even.  int8: adding
// 1.5 * 2^23 rounds to an integer whose low byte is the code; |v| <= 127 (a
// block's scale is its largest value's), so nothing needs saturating.  What a
// value that is not finite gives is the caller's to replace.
template <int KT>
__device__ __forceinline__ uint32_t kv_encode4(float a, float b, float c, float d) {
    if (KT == kKvInt8) {
        const float big = 12582912.0f;
        const uint32_t x = __byte_perm(__float_as_uint(__fadd_rn(a, big)), __float_as_uint(__fadd_rn(b, big)), 0x0040);
        const uint32_t y = __byte_perm(__float_as_uint(__fadd_rn(c, big)), __float_as_uint(__fadd_rn(d, big)), 0x0040);
        return __byte_perm(x, y, 0x5410);
    }
    return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3) |
           (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3) << 16;
}

__host__ __device__ inline int kv_log2(int v) {
    int s = 0;
    while ((1 << s) < v) ++s;
    return s;
}

// Launch with programmatic dependent launch when `pdl`: the kernel starts
// while the one before it drains, and waits (grid_dependency_wait) before it
// touches memory.
template <typename... P, typename... A>
inline cudaError_t kv_launch(void (*kern)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t s, bool pdl,
                             A &&...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, static_cast<P>(args)...);
}

// Early launch of the next kernel on the stream, only once everything before
// this kernel has completed: a GEMM reads its weights before its own wait, and
// may rely on kernels further back than the one right before it.
__device__ __forceinline__ void kv_begin() {
    grid_dependency_wait();
    grid_dependents_launch();
}

}  // namespace w4a16
