// beam.cu -- beam search's selection: the best continuations of each request
// over its beams and the vocabulary.
//
// With a beam's cumulative score s_b and its logits x_b, a continuation by token t
// is worth
//     c(b, t) = s_b + x_bt - log sum_t' e^x_bt'
// and the n best of a request's beams come out in order, ties to the lower
// beam, then the lower token.  Bound by reading the logits once.
//
//  * A CTA takes a part of one beam's logits, a tile of 32 per thread at a time.
//    Each thread keeps a sum of its own, so nothing but the candidates is
//    exchanged: 2^(x log2 e - R) with R the integer next to its largest x log2 e,
//    so that sums with other references differ by a power of two, exactly.
//    log2 e is two fp32 numbers; a tile is summed in fp32, tiles in 64 bits: the
//    continuations of different beams, a few 1e-2 apart in earnest, are told
//    apart down to about 1e-8.
//  * Within a beam c rises with x: candidates are logits, kept as 64-bit keys
//    (the value's order, then the lower token).  A tile's threads whose largest
//    logit is above the n-th best key so far append theirs to a list; only when
//    it might overflow is the list cut to its n best.  How long it can get is
//    known: of the n threads with the largest maxima come at most 32 n, which is
//    also how the first tile, where all are candidates, finds its threshold.
//  * A second kernel, a CTA per request, joins the parts' sums, scores the
//    candidates in 64 bits and picks the n best by counting who is better.
//    Of sorted lists only the n with the best heads can hold any.
#include <float.h>

#include <algorithm>

#include "kv.cuh"

namespace w4a16 {
namespace {

constexpr int kThreads = 256;
constexpr int kPer = 32;                               // logits of a tile per thread, in vectors of 8
constexpr int kTile = kThreads * kPer;
constexpr int kList = (kPer + 1) * kBeamMost;          // candidates that a part may have in hand
constexpr int kMergeThreads = 512;
constexpr int kMaxLists = 1024;                        // (beam, part) pairs of a request
constexpr float kHuge = 536870912.0f;                  // 2^29: from here on logits are 32 and more apart

// The sum of a part of a beam's logits: l = sum 2^(x log2 e - reference(m)), m the
// largest x.  Where |m| >= 2^29 nothing but the logits that equal m counts, and l is their number.
struct PartSum {
    double l;
    float m;
    int pad;
};

__device__ __forceinline__ float ex2(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
constexpr float kLog2e = 1.44269502162933349609375f, kLog2eLow = 1.92596299112661746887e-8f;   // their sum is log2 e
__device__ __forceinline__ float reference(float m) { return rintf(m * kLog2e); }
// 2^k for whole k, 0 far below the range
__device__ __forceinline__ double pow2(float k) {
    return k < -1000.0f ? 0.0 : __longlong_as_double((long long)((int)k + 1023) << 52);
}
// What a sum with largest m counts for in one whose largest is `top` (>= m).
__device__ __forceinline__ double carried(float m, float top) {
    if (fabsf(top) >= kHuge) return m == top ? 1.0 : 0.0;
    if (fabsf(m) >= kHuge) return 0.0;
    return pow2(reference(m) - reference(top));
}

// Order of fp32 values as unsigned numbers (-0 as 0), and back.
__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t u = __float_as_uint(x + 0.0f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float from_ordered(uint32_t u) {
    return __uint_as_float(u & 0x80000000u ? u & 0x7fffffffu : ~u);
}
__device__ __forceinline__ unsigned long long key_of(float x, int token) {
    return (unsigned long long)ordered(x) << 32 | (uint32_t)~token;
}
__device__ __forceinline__ float key_value(unsigned long long k) { return from_ordered((uint32_t)(k >> 32)); }
__device__ __forceinline__ int key_token(unsigned long long k) { return (int)~(uint32_t)k; }

// Logits [at, at + 8) of a row, -inf from `end` on.
template <int DT>
__device__ __forceinline__ void load8(const void *row, bool wide, int at, int end, float (&x)[8]) {
    if (wide && at + 8 <= end) {
        if (DT == 2) {
            const uint4 a = ldg_stream_v4(static_cast<const float *>(row) + at);
            const uint4 b = ldg_stream_v4(static_cast<const float *>(row) + at + 4);
            const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(w[i]);
        } else {
            const uint4 a = ldg_stream_v4(static_cast<const uint16_t *>(row) + at);
            const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = kv_act<DT == 2 ? 1 : DT>((uint16_t)(w[i / 2] >> (16 * (i & 1))));
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        x[i] = -INFINITY;
        if (at + i < end)
            x[i] = DT == 2 ? static_cast<const float *>(row)[at + i]
                           : kv_act<DT == 2 ? 1 : DT>(static_cast<const uint16_t *>(row)[at + i]);
    }
}

// Whether a beam is a source of continuations by its logits.
__device__ __forceinline__ bool goes_on(const BeamArgs &a, int row) {
    return isfinite(a.scores[row]) && !(a.finished && a.finished[row]);
}

template <int DT>
__global__ void __launch_bounds__(kThreads) scan_kernel(const BeamArgs a, int parts, int part_tiles, PartSum *sums,
                                                        unsigned long long *lists) {
    kv_begin();
    __shared__ unsigned long long list[kList];
    __shared__ unsigned long long maxima[kThreads];
    __shared__ unsigned long long s_least;
    __shared__ double s_sum[kThreads / 32];
    __shared__ float s_max[kThreads / 32];
    __shared__ int s_n;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, K = a.n_out;
    const int row = blockIdx.x / parts, part = blockIdx.x % parts;
    if (!goes_on(a, row)) return;
    const void *x0 = static_cast<const char *>(a.logits) + row * a.row_stride * (DT == 2 ? 4 : 2);
    const bool wide = (reinterpret_cast<uintptr_t>(x0) & 15) == 0;
    const int begin = part * part_tiles * kTile, end = min(a.vocab, begin + part_tiles * kTile);
    float m = -INFINITY, least = -INFINITY;               // of this thread; the n-th best so far
    double l = 0.0;
    int at_most = 0;                                       // an upper bound of the list's length
    if (tid == 0) s_n = 0;

    // The list cut to its n best, in order.
    auto cut = [&]() {
        __syncthreads();
        const int n = s_n;
        unsigned long long mine[(kList + kThreads - 1) / kThreads];
        int place[(kList + kThreads - 1) / kThreads];
#pragma unroll
        for (int i = 0; i < (kList + kThreads - 1) / kThreads; ++i) {
            const int at = tid + i * kThreads;
            place[i] = K;
            if (at < n) {
                mine[i] = list[at];
                place[i] = 0;
                for (int j = 0; j < n; ++j) place[i] += list[j] > mine[i];
            }
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < (kList + kThreads - 1) / kThreads; ++i)
            if (place[i] < K) list[place[i]] = mine[i];
        if (tid == 0) s_n = min(n, K);
        __syncthreads();
        if (n >= K) least = key_value(list[K - 1]);
        at_most = min(n, K);
    };

    for (int base = begin; base < end; base += kTile) {
        float x[kPer / 8][8];
#pragma unroll
        for (int j = 0; j < kPer / 8; ++j) load8<DT>(x0, wide, base + (j * kThreads + tid) * 8, end, x[j]);
        float top = -INFINITY;
#pragma unroll
        for (int j = 0; j < kPer / 8; ++j)
#pragma unroll
            for (int e = 0; e < 8; ++e) top = fmaxf(top, x[j][e]);
        // ---- the sum
        const float to = fmaxf(m, top);
        l *= carried(m, to);
        m = to;
        float s = 0.0f;
        if (fabsf(to) < kHuge) {
            const float r = reference(to);
#pragma unroll
            for (int j = 0; j < kPer / 8; ++j)
#pragma unroll
                for (int e = 0; e < 8; ++e) s += ex2(fmaf(x[j][e], kLog2eLow, fmaf(x[j][e], kLog2e, -r)));
        } else {
#pragma unroll
            for (int j = 0; j < kPer / 8; ++j)
#pragma unroll
                for (int e = 0; e < 8; ++e)                // a NaN stays one; no logit but -inf so far: none counts
                    s += x[j][e] != x[j][e] ? x[j][e] : x[j][e] == to && to > -INFINITY ? 1.0f : 0.0f;
        }
        l += s;
        // ---- candidates
        int passing = __syncthreads_count(top > least);
        if (passing == 0) continue;
        unsigned long long from = 0;
        if (at_most + kPer * passing > kList) {
            cut();
            passing = __syncthreads_count(top > least);
            if (at_most + kPer * passing > kList) {        // more than n threads, then
                unsigned long long best = 0;
#pragma unroll
                for (int j = kPer / 8 - 1; j >= 0; --j)
#pragma unroll
                    for (int e = 7; e >= 0; --e)           // the lowest token of the largest logit
                        if (x[j][e] == top && top > least) best = key_of(top, base + (j * kThreads + tid) * 8 + e);
                maxima[tid] = best;
                __syncthreads();
                int better = 0;
                for (int j = 0; j < kThreads; ++j) better += maxima[j] > best;
                if (best != 0 && better == K - 1) s_least = best;
                __syncthreads();
                from = s_least;
                passing = K;
            }
        }
        at_most += kPer * passing;
        if (top > least) {
#pragma unroll
            for (int j = 0; j < kPer / 8; ++j)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (x[j][e] > least) {
                        const unsigned long long k = key_of(x[j][e], base + (j * kThreads + tid) * 8 + e);
                        if (k >= from) list[atomicAdd(&s_n, 1)] = k;
                    }
        }
    }
    cut();
    const int n = s_n;
    unsigned long long *out = lists + (long long)blockIdx.x * K;
    for (int i = tid; i < K; i += kThreads) out[i] = i < n ? list[i] : 0;
    // ---- the threads' sums joined
    float top = m;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    if (lane == 0) s_max[warp] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) top = fmaxf(top, s_max[w]);
    l *= carried(m, top);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
    if (lane == 0) s_sum[warp] = l;
    __syncthreads();
    if (tid == 0) {
        for (int w = 1; w < kThreads / 32; ++w) l += s_sum[w];
        sums[blockIdx.x] = PartSum{l, top, 0};
    }
}

// A CTA per request: its beams' sums, then the best of the candidates.
__global__ void __launch_bounds__(kMergeThreads) merge_kernel(const BeamArgs a, int parts, const PartSum *sums,
                                                              const unsigned long long *lists, int *status) {
    kv_begin();
    const int tid = threadIdx.x, K = a.n_out, W = a.width, n_lists = W * parts;
    // no static shared memory: raise_smem_cap
    extern __shared__ double dyn[];
    double *s_top = dyn, *s_log = s_top + kBeamMost;       // of each beam: its largest logit (NaN: none), and with x as
                                                           // x - s_top, log sum e^x
    double *s_heads = s_log + kBeamMost, *s_score = s_heads + kMaxLists;
    int *s_from = reinterpret_cast<int *>(s_score + K * K);   // list * n + place in it
    double &s_least = *reinterpret_cast<double *>(s_from + (K * K + 1) / 2 * 2);
    int &s_least_at = *reinterpret_cast<int *>(&s_least + 1), &s_n = *(&s_least_at + 1);
    const int row0 = blockIdx.x * W;
    if (tid == 0) s_n = 0, s_least = -INFINITY, s_least_at = 0x7fffffff;
    for (int b = tid; b < W; b += kMergeThreads) {
        double largest = NAN, log_sum = 0.0;
        if (goes_on(a, row0 + b)) {
            const PartSum *p = sums + (long long)(row0 + b) * parts;
            float top = -INFINITY;
            for (int i = 0; i < parts; ++i) top = fmaxf(top, p[i].m);
            double l = 0.0;
            for (int i = 0; i < parts; ++i) l += p[i].l * carried(p[i].m, top);
            // the row of a NaN or +inf has no probabilities, one without any token but -inf has no continuations
            if (top == INFINITY || l != l) {
                kv_report(status);
            } else if (top > -INFINITY) {
                largest = top;
                // relative to the largest, which may be far larger than the sum's logarithm
                log_sum = fabsf(top) >= kHuge ? log(l) : log(l) + ((double)reference(top) * 0.693147180559945309417 - largest);
            }
        }
        s_top[b] = largest, s_log[b] = log_sum;
    }
    __syncthreads();
    const unsigned long long *mine = lists + (long long)row0 * parts * K;
    // the score of a list's i-th candidate, NaN where there is none
    auto score_of = [&](int list, int i) -> double {
        const int b = list / parts, row = row0 + b;
        const double s = a.scores[row];
        if (!isfinite(s)) return NAN;
        if (a.finished && a.finished[row]) return list % parts == 0 && i == 0 ? s : (double)NAN;
        if (s_top[b] != s_top[b]) return NAN;
        const unsigned long long k = mine[(long long)list * K + i];
        return k == 0 ? (double)NAN : s + (((double)key_value(k) - s_top[b]) - s_log[b]);
    };
    // the at-th candidate of all, of score s, before the than-th of score t: equal ones by their beams, and within a beam as
    // the logits say, which may differ by less than the scores resolve
    auto better = [&](double s, int at, double t, int than) {
        if (s != t) return s > t;
        const int b = at / (parts * K), c = than / (parts * K);
        return b != c ? b < c : at != than && mine[at] > mine[than];
    };
    // of so many sorted lists only the n with the best heads matter
    if (n_lists >= K) {
        for (int i = tid; i < n_lists; i += kMergeThreads) s_heads[i] = score_of(i, 0);
        __syncthreads();
        for (int i = tid; i < n_lists; i += kMergeThreads) {
            const double s = s_heads[i];
            int place = 0;
            for (int j = 0; j < n_lists; ++j) place += better(s_heads[j], j * K, s, i * K);
            if (s == s && place == K - 1) s_least = s, s_least_at = i * K;
        }
        __syncthreads();
    }
    const double least = s_least;
    const int least_at = s_least_at;
    for (int i = tid; i < n_lists * K; i += kMergeThreads) {
        const double s = score_of(i / K, i % K);
        if (s > least || (s == least && !better(least, least_at, s, i))) {
            const int at = atomicAdd(&s_n, 1);
            s_score[at] = s;
            s_from[at] = i;
        }
    }
    __syncthreads();
    const int n = s_n;
    for (int i = tid; i < n; i += kMergeThreads) {
        const double s = s_score[i];
        const int from = s_from[i];
        int place = 0;
        for (int j = 0; j < n; ++j) place += better(s_score[j], s_from[j], s, from);
        if (place >= K) continue;
        const int list = from / K, row = row0 + list / parts;
        const bool was = a.finished && a.finished[row];
        const int token = was ? a.end_token : key_token(mine[from]);
        const long long at = (long long)blockIdx.x * K + place;
        a.out_scores[at] = (float)s;
        a.out_rows[at] = row;
        a.out_tokens[at] = token;
        if (a.out_finished) a.out_finished[at] = was || token == a.end_token;
    }
    for (int i = n + tid; i < K; i += kMergeThreads) {
        const long long at = (long long)blockIdx.x * K + i;
        a.out_scores[at] = -INFINITY;
        a.out_rows[at] = a.out_tokens[at] = -1;
        if (a.out_finished) a.out_finished[at] = 0;
    }
}

// Parts of a row and tiles of each: enough CTAs for every SM to have three.
void split_rows(int rows, int width, int vocab, int sm_count, int *parts, int *part_tiles) {
    const int tiles = std::max((vocab + kTile - 1) / kTile, 1);
    const int want = std::max(1, std::min(3 * sm_count / std::max(rows, 1), kMaxLists / width));
    *part_tiles = (tiles + want - 1) / want;
    *parts = (tiles + *part_tiles - 1) / *part_tiles;
}

}  // namespace

cudaError_t launch_beam_select(const BeamArgs &a, void *workspace, const DeviceInfo &dev, cudaStream_t s, bool pdl) {
    const int rows = a.n_groups * a.width;
    int parts, part_tiles;
    split_rows(rows, a.width, a.vocab, dev.sm_count, &parts, &part_tiles);
    PartSum *sums = static_cast<PartSum *>(workspace);
    unsigned long long *lists = reinterpret_cast<unsigned long long *>(sums + (long long)rows * parts);
    const dim3 grid((unsigned)rows * parts), block(kThreads);
    const cudaError_t e =
        a.dtype == 0   ? kv_launch(scan_kernel<0>, grid, block, 0, s, pdl, a, parts, part_tiles, sums, lists)
        : a.dtype == 1 ? kv_launch(scan_kernel<1>, grid, block, 0, s, pdl, a, parts, part_tiles, sums, lists)
                       : kv_launch(scan_kernel<2>, grid, block, 0, s, pdl, a, parts, part_tiles, sums, lists);
    if (e != cudaSuccess) return e;
    const size_t smem = (2 * kBeamMost + kMaxLists) * 8 + (size_t)a.n_out * a.n_out * 12 + 4 + 16;
    const cudaError_t f = raise_smem_cap(reinterpret_cast<const void *>(merge_kernel), smem);
    if (f != cudaSuccess) return f;
    return kv_launch(merge_kernel, dim3(a.n_groups), dim3(kMergeThreads), smem, s, pdl, a, parts, sums, lists, dev.status);
}

long long beam_select_workspace(int n_groups, int width, int vocab, int n_out, const DeviceInfo &dev) {
    int parts, part_tiles;
    split_rows(n_groups * width, width, vocab, dev.sm_count, &parts, &part_tiles);
    return (long long)n_groups * width * parts * (sizeof(PartSum) + 8LL * n_out);
}

}  // namespace w4a16
