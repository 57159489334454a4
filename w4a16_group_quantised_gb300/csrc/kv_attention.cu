// kv_attention.cu -- attention over the paged 8-bit cache.
//
// First form: one warp per (token, query head), fp32 throughout, one key
// after another with a running maximum and sum.
#include "kv.cuh"

namespace w4a16 {
namespace {

template <int DT, int KT, int D>
__global__ void attention_kernel(KvAttentionArgs a, KvCache c, KvBatch b, int *status) {
    kv_begin();
    constexpr int P = D / 32;                            // dims per lane
    const int lane = threadIdx.x & 31;
    const long long wid = (long long)blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32;
    if (wid >= (long long)b.n_tokens * a.n_heads) return;
    const int t = (int)(wid / a.n_heads), head = (int)(wid % a.n_heads);
    int lo = 0, hi = b.n_seqs - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (b.q_starts[mid] <= t) lo = mid;
        else hi = mid - 1;
    }
    const KvSeq s = kv_sequence(b, c.page_shift, lo, status);
    const int kvh = head / (a.n_heads / c.n_kv_heads);
    float q[P], o[P];
#pragma unroll
    for (int p = 0; p < P; ++p) {
        q[p] = kv_act<DT>(static_cast<const uint16_t *>(a.q)[t * a.q_stride + head * D + lane * P + p]);
        o[p] = 0.0f;
    }
    float m = -INFINITY, l = 0.0f;
    const int i = s.len - s.n + t - s.q0;
    if (t >= s.q0 && t < s.q0 + s.n)
        for (int j = 0; j <= i; ++j) {
            if (a.window > 0 && i - j >= a.window && j >= a.sinks) {
                j = i - a.window;                        // on to the window's first key
                continue;
            }
            const int page = kv_page(c, b, lo, j >> c.page_shift, status);
            if (page < 0) continue;
            const long long at = page * c.page_stride + kvh * c.head_stride +
                                 (j & ((1 << c.page_shift) - 1)) * c.token_stride + lane * P;
            const long long sc = (long long)page * c.n_kv_heads + kvh;
            float kv[4], vv[4];
            kv_decode4<KT>(P == 4 ? *reinterpret_cast<const uint32_t *>(c.k + at) : *reinterpret_cast<const uint16_t *>(c.k + at), kv);
            kv_decode4<KT>(P == 4 ? *reinterpret_cast<const uint32_t *>(c.v + at) : *reinterpret_cast<const uint16_t *>(c.v + at), vv);
            float x = 0.0f;
#pragma unroll
            for (int p = 0; p < P; ++p) x += q[p] * kv[p];
            for (int d = 16; d; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
            x *= a.scale * c.k_scale[sc];
            const float m2 = fmaxf(m, x);
            const float f = m == -INFINITY ? 0.0f : expf(m - m2), w = expf(x - m2);
            l = l * f + w;
#pragma unroll
            for (int p = 0; p < P; ++p) o[p] = o[p] * f + w * c.v_scale[sc] * vv[p];
            m = m2;
        }
    const float r = l > 0.0f ? 1.0f / l : (l == l ? 0.0f : l);
#pragma unroll
    for (int p = 0; p < P; ++p)
        static_cast<uint16_t *>(a.out)[wid * D + lane * P + p] = kv_to_act<DT>(o[p] * r);
    if (a.lse && lane == 0) a.lse[wid] = l > 0.0f ? m + logf(l) : (l == l ? -INFINITY : l);
}

}  // namespace

cudaError_t launch_kv_attention(const KvAttentionArgs &a, const KvCache &c, const KvBatch &b, const DeviceInfo &dev,
                                cudaStream_t s, bool pdl) {
    const long long warps = (long long)b.n_tokens * a.n_heads;
    auto pick = [&](auto d64, auto d128) { return c.head_dim == 64 ? d64 : d128; };
    auto kern = a.dtype == 0
                    ? (c.kv_dtype == kKvInt8 ? pick(attention_kernel<0, kKvInt8, 64>, attention_kernel<0, kKvInt8, 128>)
                                             : pick(attention_kernel<0, kKvE4m3, 64>, attention_kernel<0, kKvE4m3, 128>))
                    : (c.kv_dtype == kKvInt8 ? pick(attention_kernel<1, kKvInt8, 64>, attention_kernel<1, kKvInt8, 128>)
                                             : pick(attention_kernel<1, kKvE4m3, 64>, attention_kernel<1, kKvE4m3, 128>));
    return kv_launch(kern, dim3((unsigned)((warps + 7) / 8)), dim3(256), 0, s, pdl, a, c, b, dev.status);
}

long long kv_attention_workspace(int, int, int, int, int, const DeviceInfo &) { return 0; }

}  // namespace w4a16
