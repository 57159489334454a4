// kv_append.cu -- quantise new keys and values into the pages of an 8-bit
// cache, and read cached tokens back.
//
// Append.  For a page and kv head, with amax = max |x| over the page's new
// tokens and s_old the scale of the tokens already in it (0 without any),
//     s = max(s_old, amax / qmax, 2^-60),   code = RN(x * RN(1 / s)),
// and when s > s_old the older codes are rounded again against s.  The
// products and the division are fp32: RN(1 / s) is one rounding away from
// 1 / s, far below half a code step, so one reciprocal serves a whole block.
// A block with a value that is not finite gets a scale that is not, and codes
// of 0: the scale tells whoever sees the block (0 * inf is NaN), while a NaN
// code would also reach rows that do not, through a weight of 0.
#include <algorithm>

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

// The largest i with key(i) <= at, or 0: every lane of a warp calls.  Up to
// kScan sequences are looked at 32 at a time, in one round trip to memory for
// most batches; more are searched by halves.
constexpr int kScan = 256;
template <typename Key>
__device__ __forceinline__ int warp_find(int n, int at, Key key) {
    const int lane = threadIdx.x & 31;
    if (n <= kScan) {
        int below = 0;
#pragma unroll 2
        for (int base = 0; base < n; base += 32)
            below += __popc(__ballot_sync(0xffffffffu, base + lane < n && key(base + lane) <= at));
        return max(below - 1, 0);
    }
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (key(mid) <= at) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// One CTA per (unit, kv head): a thread holds 16 values of one slot of K and of
// V.  The bytes are few and read once; what counts is the chain of dependent
// loads (starts, then values and page id together, then the scales), and how
// much is on its way during one: K and V apart, 32 bytes a thread, took 28 us
// where both together take 23 us for 15,200 tokens of 8 heads.
// That call with its read-back takes 37 us against 28 us for its bytes at a
// copy's bandwidth; 64 sequences' single tokens take 6.5 us.
constexpr int kRows = 65535;               // of a grid: units go on in the next plane
template <int DT, int KT>
__global__ void append_kernel(KvCache c, KvBatch b, const uint16_t *k_new, long long k_stride, const uint16_t *v_new,
                              long long v_stride, int *status) {
    kv_begin();
    __shared__ uint32_t warp_max[2][32];
    const int shift = c.page_shift;
    const int unit = blockIdx.z * kRows + blockIdx.y, head = blockIdx.x;
    const int i = warp_find(b.n_seqs, unit, [&](int j) { return append_base(b, shift, j); });
    const KvSeq s = kv_sequence(b, shift, i, status);
    const int first = s.len - s.n;                       // position of the first new token
    const int nth = unit - append_base(b, shift, i);
    const int blk = (max(first, 0) >> shift) + nth;
    if (s.n == 0 || nth < 0 || blk > (s.len - 1) >> shift) return;
    const int page = b.block_table[(long long)i * b.max_blocks + blk];
    const int old = max(first - (blk << shift), 0);      // slots filled before this call
    const int vecs = c.head_dim / 16;
    const int slot = threadIdx.x / vecs, d0 = threadIdx.x % vecs * 16;
    const int pos = (blk << shift) + slot;
    const bool is_new = pos >= first && pos >= 0 && pos < s.len;

    uint32_t x[2][8], top[2] = {0, 0};                   // |x| as bits: ordered as integers, NaN on top
    if (is_new) {
        const long long row = s.q0 + pos - first;
        const uint16_t *src[2] = {k_new + row * k_stride + head * c.head_dim + d0,
                                  v_new + row * v_stride + head * c.head_dim + d0};
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const uint4 a = ldg_stream_v4(src[t]), z = ldg_stream_v4(src[t] + 8);
            x[t][0] = a.x, x[t][1] = a.y, x[t][2] = a.z, x[t][3] = a.w;
            x[t][4] = z.x, x[t][5] = z.y, x[t][6] = z.z, x[t][7] = z.w;
        }
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int j = 0; j < 8; ++j) top[t] = max(top[t], max(x[t][j] & 0x7fffu, (x[t][j] >> 16) & 0x7fffu));
    }
    if (page < 0 || page >= c.n_pages) {                 // the same for the whole CTA
        if (threadIdx.x == 0) kv_report(status);
        return;
    }
    const long long at_scale = (long long)page * c.n_kv_heads + head;
    const float s_old[2] = {old > 0 ? c.k_scale[at_scale] : 0.0f, old > 0 ? c.v_scale[at_scale] : 0.0f};
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        top[t] = __reduce_max_sync(0xffffffffu, top[t]);
        if ((threadIdx.x & 31) == 0) warp_max[t][threadIdx.x >> 5] = top[t];
    }
    __syncthreads();
    const long long at = page * c.page_stride + head * c.head_stride + slot * c.token_stride + d0;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const int lane = threadIdx.x & 31;
        top[t] = __reduce_max_sync(0xffffffffu, lane < (int)blockDim.x / 32 ? warp_max[t][lane] : 0u);
        const float need = __fdiv_rn(kv_act<DT>((uint16_t)top[t]), kv_qmax<KT>());
        float s_new = need <= s_old[t] ? s_old[t] : need;    // a NaN on either side stays
        if (s_old[t] != s_old[t]) s_new = s_old[t];
        if (s_new < kKvScaleMin) s_new = kKvScaleMin;
        const float r = __frcp_rn(s_new);
        const bool finite = s_new < INFINITY;
        uint8_t *dst = (t ? c.v : c.k) + at;
        uint4 o;
        uint32_t *ow = &o.x;
        if (is_new) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t lo = x[t][2 * j], hi = x[t][2 * j + 1];
                ow[j] = kv_encode4<KT>(__fmul_rn(kv_act<DT>((uint16_t)lo), r), __fmul_rn(kv_act<DT>((uint16_t)(lo >> 16)), r),
                                       __fmul_rn(kv_act<DT>((uint16_t)hi), r), __fmul_rn(kv_act<DT>((uint16_t)(hi >> 16)), r));
            }
            *reinterpret_cast<uint4 *>(dst) = finite ? o : make_uint4(0, 0, 0, 0);
        } else if (slot < old && s_new != s_old[t]) {
            const uint4 q = *reinterpret_cast<const uint4 *>(dst);
            const uint32_t qw[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float v[4];
                kv_decode4<KT>(qw[j], v);
                ow[j] = kv_encode4<KT>(__fmul_rn(__fmul_rn(v[0], s_old[t]), r), __fmul_rn(__fmul_rn(v[1], s_old[t]), r),
                                       __fmul_rn(__fmul_rn(v[2], s_old[t]), r), __fmul_rn(__fmul_rn(v[3], s_old[t]), r));
            }
            *reinterpret_cast<uint4 *>(dst) = finite ? o : make_uint4(0, 0, 0, 0);
        }
        if (threadIdx.x == 0) (t ? c.v_scale : c.k_scale)[at_scale] = s_new;
    }
}

// Read: a lane takes a 16-value piece of a token's K and of its V; a warp's 32
// pieces are of one token, so that the search is the warp's.
constexpr int kReadWarps = 8;
template <int DT, int KT>
__global__ void __launch_bounds__(32 * kReadWarps)
    read_kernel(KvCache c, KvBatch b, uint16_t *k_out, uint16_t *v_out, int *status) {
    kv_begin();
    const int vecs = c.n_kv_heads * c.head_dim / 16, warps = (vecs + 31) / 32;      // of a token
    const int wid = blockIdx.x * kReadWarps + threadIdx.x / 32;
    const int t = wid / warps, e = wid % warps * 32 + (threadIdx.x & 31);
    if (t >= b.n_tokens) return;
    // the last sequence that starts at or before t
    const int i = warp_find(b.n_seqs, t, [&](int j) { return b.q_starts[j]; });
    const KvSeq s = kv_sequence(b, c.page_shift, i, status);
    const int pos = s.len - s.n + t - s.q0;
    int page = -1;
    if (t >= s.q0 && t < s.q0 + s.n && pos >= 0) page = kv_page(c, b, i, pos >> c.page_shift, status);
    const long long row = (pos & ((1 << c.page_shift) - 1)) * c.token_stride + page * c.page_stride;
    const int per_head = c.head_dim / 16;
    auto put = [&](uint16_t *dst, uint4 q, float scale) {
        const uint32_t qw[4] = {q.x, q.y, q.z, q.w};
        uint32_t o[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float v[4];
            kv_decode4<KT>(qw[j], v);
#pragma unroll
            for (int e = 0; e < 2; ++e)
                o[2 * j + e] = (uint32_t)kv_to_act<DT>(v[2 * e] * scale) |
                               (uint32_t)kv_to_act<DT>(v[2 * e + 1] * scale) << 16;
        }
        reinterpret_cast<uint4 *>(dst)[0] = make_uint4(o[0], o[1], o[2], o[3]);
        reinterpret_cast<uint4 *>(dst)[1] = make_uint4(o[4], o[5], o[6], o[7]);
    };
    if (e >= vecs) return;
    const int head = e / per_head;
    uint4 k = make_uint4(0, 0, 0, 0), v = k;
    float ks = 0.0f, vs = 0.0f;
    if (page >= 0) {
        const long long at = row + head * c.head_stride + e % per_head * 16;
        const long long sc = (long long)page * c.n_kv_heads + head;
        k = ldg_stream_v4(c.k + at), v = ldg_stream_v4(c.v + at);
        ks = __ldg(c.k_scale + sc), vs = __ldg(c.v_scale + sc);
    }
    const long long at = ((long long)t * vecs + e) * 16;
    put(k_out + at, k, ks);
    put(v_out + at, v, vs);
}

}  // namespace

cudaError_t launch_kv_append(const KvCache &c, const KvBatch &b, const void *k_new, long long k_stride,
                             const void *v_new, long long v_stride, int dtype, const DeviceInfo &dev, cudaStream_t s,
                             bool pdl) {
    const int ps = 1 << c.page_shift;
    // heads next to one another: they read neighbouring bytes of the same rows (38 us for the call above where
    // units come first)
    const int units = (b.n_tokens >> c.page_shift) + 2 * b.n_seqs;
    const dim3 grid(c.n_kv_heads, std::min(units, kRows), (units + kRows - 1) / kRows);
    const dim3 block(ps * c.head_dim / 16);
    auto kern = dtype == 0 ? (c.kv_dtype == kKvInt8 ? append_kernel<0, kKvInt8> : append_kernel<0, kKvE4m3>)
                           : (c.kv_dtype == kKvInt8 ? append_kernel<1, kKvInt8> : append_kernel<1, kKvE4m3>);
    return kv_launch(kern, grid, block, 0, s, pdl, c, b, static_cast<const uint16_t *>(k_new), k_stride,
                     static_cast<const uint16_t *>(v_new), v_stride, dev.status);
}

cudaError_t launch_kv_read(const KvCache &c, const KvBatch &b, void *k_out, void *v_out, int dtype,
                           const DeviceInfo &dev, cudaStream_t s, bool pdl) {
    auto kern = dtype == 0 ? (c.kv_dtype == kKvInt8 ? read_kernel<0, kKvInt8> : read_kernel<0, kKvE4m3>)
                           : (c.kv_dtype == kKvInt8 ? read_kernel<1, kKvInt8> : read_kernel<1, kKvE4m3>);
    const long long warps = (long long)b.n_tokens * ((c.n_kv_heads * c.head_dim / 16 + 31) / 32);
    return kv_launch(kern, dim3((unsigned)((warps + kReadWarps - 1) / kReadWarps)), dim3(32 * kReadWarps), 0, s, pdl, c, b,
                     static_cast<uint16_t *>(k_out), static_cast<uint16_t *>(v_out), dev.status);
}

}  // namespace w4a16
