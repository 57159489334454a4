// kv_append.cu -- quantise new keys and values into the pages of an 8-bit
// cache, and read cached tokens back.
//
// Append.  For a page and kv head, with amax = max |x| over the page's new
// tokens and s_old the scale of the tokens already in it (0 without any),
//     s = max(s_old, amax / qmax, 2^-60),   code = RN(x * RN(1 / s)),
// and when s > s_old the older codes are rounded again against s.  The
// products and the division are fp32: RN(1 / s) is one rounding away from
// 1 / s, far below half a code step, so one reciprocal serves a whole block.
#include "kv.cuh"

namespace w4a16 {
namespace {

template <int KT>
__device__ __forceinline__ float kv_qmax() {
    return KT == kKvInt8 ? 127.0f : 448.0f;
}

// Units: (sequence, touched page).  n new tokens touch at most n / ps + 2
// pages wherever they begin, so sequence b owns units from
// q_starts[b] / ps + 2 b on: a search over the starts finds a unit's
// sequence, with no scan and no count on the host.  Units past a sequence's
// last page do nothing.
__device__ __forceinline__ int append_base(const KvBatch &b, int shift, int i) {
    return (min(max(b.q_starts[i], 0), b.n_tokens) >> shift) + 2 * i;
}

// One CTA per (unit, kv head, K or V): a thread holds 16 values of one slot.
// Plain loads and stores: the bytes are few and read once.
template <int DT, int KT>
__global__ void append_kernel(KvCache c, KvBatch b, const uint16_t *k_new, long long k_stride, const uint16_t *v_new,
                              long long v_stride, int *status) {
    kv_begin();
    __shared__ uint32_t warp_max[32];
    __shared__ int s_seq;
    const int shift = c.page_shift;
    const int unit = blockIdx.x, head = blockIdx.y, is_v = blockIdx.z;
    if (threadIdx.x == 0) {
        int lo = 0, hi = b.n_seqs - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (append_base(b, shift, mid) <= unit) lo = mid;
            else hi = mid - 1;
        }
        s_seq = lo;
    }
    __syncthreads();
    const int i = s_seq;
    const KvSeq s = kv_sequence(b, shift, i, status);
    const int first = s.len - s.n;                       // position of the first new token
    const int nth = unit - append_base(b, shift, i);
    const int blk = (max(first, 0) >> shift) + nth;
    if (s.n == 0 || nth < 0 || blk > (s.len - 1) >> shift) return;
    const int page = kv_page(c, b, i, blk, status);
    if (page < 0) return;
    const int old = max(first - (blk << shift), 0);      // slots filled before this call
    const int vecs = c.head_dim / 16;
    const int slot = threadIdx.x / vecs, d0 = threadIdx.x % vecs * 16;
    const int pos = (blk << shift) + slot;
    const bool is_new = pos >= first && pos >= 0 && pos < s.len;

    uint32_t x[8];
    uint32_t top = 0;                                    // |x| as bits: ordered as integers, NaN on top
    if (is_new) {
        const uint16_t *src = (is_v ? v_new + (long long)(s.q0 + pos - first) * v_stride
                                    : k_new + (long long)(s.q0 + pos - first) * k_stride) + head * c.head_dim + d0;
        const uint4 a = ldg_stream_v4(src), z = ldg_stream_v4(src + 8);
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = z.x, x[5] = z.y, x[6] = z.z, x[7] = z.w;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            top = max(top, x[j] & 0x7fffu);
            top = max(top, (x[j] >> 16) & 0x7fffu);
        }
    }
    top = __reduce_max_sync(0xffffffffu, top);
    if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = top;
    float *sp = (is_v ? c.v_scale : c.k_scale) + (long long)page * c.n_kv_heads + head;
    const float s_old = old > 0 ? *sp : 0.0f;
    __syncthreads();
    for (int w = 0; w < (int)blockDim.x / 32; ++w) top = max(top, warp_max[w]);
    const float need = __fdiv_rn(kv_act<DT>((uint16_t)top), kv_qmax<KT>());
    float s_new = need <= s_old ? s_old : need;          // a NaN on either side stays
    if (s_old != s_old) s_new = s_old;
    if (s_new < kKvScaleMin) s_new = kKvScaleMin;
    const float r = __frcp_rn(s_new);
    uint8_t *dst = (is_v ? c.v : c.k) + page * c.page_stride + head * c.head_stride + slot * c.token_stride + d0;
    uint4 o;
    uint32_t *ow = &o.x;
    if (is_new) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            ow[j] = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint16_t h = (uint16_t)(x[2 * j + e / 2] >> (16 * (e & 1)));
                ow[j] |= kv_encode<KT>(kv_act<DT>(h) * r) << (8 * e);
            }
        }
        *reinterpret_cast<uint4 *>(dst) = o;
    } else if (slot < old && s_new != s_old) {
        const uint4 q = *reinterpret_cast<const uint4 *>(dst);
        const uint32_t qw[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float v[4];
            kv_decode4<KT>(qw[j], v);
            ow[j] = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) ow[j] |= kv_encode<KT>(__fmul_rn(__fmul_rn(v[e], s_old), r)) << (8 * e);
        }
        *reinterpret_cast<uint4 *>(dst) = o;
    }
    if (threadIdx.x == 0) *sp = s_new;
}

// Read: 16 values a thread, K and V of `per` tokens a CTA.
template <int DT, int KT>
__global__ void read_kernel(KvCache c, KvBatch b, uint16_t *k_out, uint16_t *v_out, int *status) {
    kv_begin();
    const int vecs = c.n_kv_heads * c.head_dim / 16;
    const long long at = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    if (at >= (long long)b.n_tokens * vecs) return;
    const int t = (int)(at / vecs), e = (int)(at % vecs);
    int lo = 0, hi = b.n_seqs - 1;
    while (lo < hi) {                                    // the last sequence that starts at or before t
        const int mid = (lo + hi + 1) >> 1;
        if (b.q_starts[mid] <= t) lo = mid;
        else hi = mid - 1;
    }
    const KvSeq s = kv_sequence(b, c.page_shift, lo, status);
    const int pos = s.len - s.n + t - s.q0;
    const int head = e * 16 / c.head_dim, d0 = e * 16 % c.head_dim;
    int page = -1;
    if (t >= s.q0 && t < s.q0 + s.n && pos >= 0) page = kv_page(c, b, lo, pos >> c.page_shift, status);
#pragma unroll
    for (int is_v = 0; is_v < 2; ++is_v) {
        uint4 q = make_uint4(0, 0, 0, 0);
        float scale = 0.0f;
        if (page >= 0) {
            const uint8_t *src = (is_v ? c.v : c.k) + page * c.page_stride + head * c.head_stride +
                                 (pos & ((1 << c.page_shift) - 1)) * c.token_stride + d0;
            q = ldg_stream_v4(src);
            scale = (is_v ? c.v_scale : c.k_scale)[(long long)page * c.n_kv_heads + head];
        }
        const uint32_t qw[4] = {q.x, q.y, q.z, q.w};
        uint32_t o[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float v[4];
            kv_decode4<KT>(qw[j], v);
#pragma unroll
            for (int e2 = 0; e2 < 2; ++e2)
                o[2 * j + e2] = (uint32_t)kv_to_act<DT>(v[2 * e2] * scale) |
                                (uint32_t)kv_to_act<DT>(v[2 * e2 + 1] * scale) << 16;
        }
        uint4 *dst = reinterpret_cast<uint4 *>((is_v ? v_out : k_out) + at * 16);
        dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
        dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
    }
}

}  // namespace

cudaError_t launch_kv_append(const KvCache &c, const KvBatch &b, const void *k_new, long long k_stride,
                             const void *v_new, long long v_stride, int dtype, const DeviceInfo &dev, cudaStream_t s,
                             bool pdl) {
    const int ps = 1 << c.page_shift;
    const dim3 grid((b.n_tokens >> c.page_shift) + 2 * b.n_seqs, c.n_kv_heads, 2);
    const dim3 block(ps * c.head_dim / 16);
    auto kern = dtype == 0 ? (c.kv_dtype == kKvInt8 ? append_kernel<0, kKvInt8> : append_kernel<0, kKvE4m3>)
                           : (c.kv_dtype == kKvInt8 ? append_kernel<1, kKvInt8> : append_kernel<1, kKvE4m3>);
    return kv_launch(kern, grid, block, 0, s, pdl, c, b, static_cast<const uint16_t *>(k_new), k_stride,
                     static_cast<const uint16_t *>(v_new), v_stride, dev.status);
}

cudaError_t launch_kv_read(const KvCache &c, const KvBatch &b, void *k_out, void *v_out, int dtype,
                           const DeviceInfo &dev, cudaStream_t s, bool pdl) {
    const long long threads = (long long)b.n_tokens * c.n_kv_heads * c.head_dim / 16;
    auto kern = dtype == 0 ? (c.kv_dtype == kKvInt8 ? read_kernel<0, kKvInt8> : read_kernel<0, kKvE4m3>)
                           : (c.kv_dtype == kKvInt8 ? read_kernel<1, kKvInt8> : read_kernel<1, kKvE4m3>);
    return kv_launch(kern, dim3((unsigned)((threads + 255) / 256)), dim3(256), 0, s, pdl, c, b,
                     static_cast<uint16_t *>(k_out), static_cast<uint16_t *>(v_out), dev.status);
}

}  // namespace w4a16
