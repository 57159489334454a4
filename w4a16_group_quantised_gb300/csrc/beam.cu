// beam.cu -- beam search's selection: the best continuations of each request
// over its beams and the vocabulary.
//
// With a beam's cumulative score s_b and its logits x_b, a continuation by token t
// is worth
//     c(b, t) = s_b + x_bt - log sum_t' e^x_bt'
// and the n best of a request's beams come out in order, ties to the lower
// beam, then the lower token.  It cannot do without reading the logits once; few
// of them take two launches' chains of loads, many what is worked out for each.
//
//  * The logits of each beam that goes on are tiles, cut into as many pieces as
//    fill the GPU; a second kernel joins a beam's pieces.  The next tile is on its
//    way while one is worked on.
//  * Each thread keeps a sum of its own, so nothing but the candidates is
//    exchanged: 2^(x log2 e - R) with R the integer next to its largest x log2 e,
//    so that sums with other references differ by a power of two, exactly.
//    log2 e is two fp32 numbers; a thread's part of a tile is summed in fp32, tiles
//    and threads in two fp32 numbers, pieces in 64 bits, and the logarithm is of the
//    sum over the largest weight as it was added up, whose error cancels: where one
//    token has all of the probability nothing is off.  Else what is: the others'
//    exponentials and the largest's, 2^-22 each, their exponents' roundings, and the
//    additions of a tile, 2^-24 each of up to 10: 2e-7 the most and 6e-8 as a root mean
//    square over 512 rows each of 30 to 131072 logits.  The continuations of different
//    beams are a few 1e-2 apart in earnest; those closer than that may change places.
//    Which thread sums what goes by the token alone, so that equal beams have equal sums.
//  * Within a beam c rises with x: candidates are logits, kept as 64-bit keys
//    (the value's order, then the lower token).  Threads note the vectors of 8 whose
//    largest logit is above the n-th best so far; every 8 tiles, and at a piece's
//    end, these are looked at again (they are in L2 still), their candidates join
//    a list, and it is cut to its n best.  A piece's first tile gets its threshold
//    from the least of the maxima of n groups of threads: n logits at least reach
//    it, a few times n in earnest.  Where more do than the list holds (many equal
//    ones), the n threads with the best maxima are found out, of which at most
//    n times a thread's share can come.
//  * The second kernel, a CTA per request, joins the pieces' sums, scores the
//    candidates in 64 bits and picks the n best by counting who is better.
//    Of sorted lists only the n with the best heads can hold any, and of these
//    lists' l-th candidates only the n / l best: 32 of 16 beams with 79 logits took
//    67 us with all candidates counted, 12 so.
//
// Measured on the GPU: 256 beams of 64 requests, a fifth of them ended, over
// 131072 bf16 logits, 54 MB: 21 us, 2.6 TB/s of logits; 40 beams over 50001 fp16
// logits 11.3 us; one beam over 32000 fp32 logits 8 us.  Of the 21, 6 are the second
// kernel; the first issues 11 instructions a logit (6 of them arithmetic of the sum)
// at 0.55 a cycle and scheduler, 2.7 CTAs an SM, each with 16 KB on their way.
#include <algorithm>
#include <type_traits>

#include "kv.cuh"

namespace w4a16 {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kPieceCost = 3;                          // tiles that a piece's start and end count for
constexpr int kBatch = 8;                              // tiles between two cuts of a list
constexpr int kList = 33 * kBeamMost;                  // its room: n candidates, and n threads' logits of a tile
constexpr int kVectors = 1024;                         // vectors with candidates between two cuts
constexpr int kSmallMerge = 256;                       // candidates for which the second kernel has 256 threads, not 1024
constexpr int kMaxLists = 1024;                        // (beam, piece) pairs of a request
constexpr int kFewCandidates = 128, kFewHeads = 128;   // so many are compared with one another at once
constexpr int kMaxRows = 2048;                         // beams among which those that go on are looked up first
constexpr float kHuge = 536870912.0f;                  // 2^29: from here on logits are 32 and more apart

// Logits of a tile per thread, in vectors of 8: as many as 16 registers hold.
template <int DT> constexpr int kPer = DT == 2 ? 16 : 32;

// The sum of a piece of a beam's logits: l = sum 2^(x log2 e - reference(m)), m the
// largest x.  Where |m| >= 2^29 nothing but the logits that equal m counts, and l is their number.
struct PartSum {
    double l;
    float m;
    int parts;                                         // pieces of the beam
};

__device__ __forceinline__ float ex2(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ uint64_t pair_of(float x, float y) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ void unpair(uint64_t v, float &x, float &y) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
constexpr float kLog2e = 1.44269502162933349609375f, kLog2eLow = 1.92596299112661746887e-8f;   // their sum is log2 e
__device__ __forceinline__ float reference(float m) { return rintf(m * kLog2e); }
// 2^k for whole k <= 127, 0 below the normal numbers
__device__ __forceinline__ float pow2(float k) {
    return k < -126.0f ? 0.0f : __uint_as_float((uint32_t)((int)k + 127) << 23);
}
// What a sum with largest m counts for in one whose largest is `top` (>= m).
__device__ __forceinline__ float carried(float m, float top) {
    if (fabsf(top) >= kHuge) return m == top ? 1.0f : 0.0f;
    if (fabsf(m) >= kHuge) return 0.0f;
    return pow2(reference(m) - reference(top));
}
// (hi, lo) += v, exactly but for the last bits of lo
__device__ __forceinline__ void add_to(float &hi, float &lo, float v) {
    const float s = __fadd_rn(hi, v), z = __fsub_rn(s, hi);
    lo = __fadd_rn(lo, __fadd_rn(__fsub_rn(hi, __fsub_rn(s, z)), __fsub_rn(v, z)));
    hi = s;
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

// The same of 64 bits; no number but a NaN's is 0.
__device__ __forceinline__ unsigned long long ordered64(double x) {
    const long long u = __double_as_longlong(x + 0.0);
    return u < 0 ? ~(unsigned long long)u : (unsigned long long)u | 1ull << 63;
}
__device__ __forceinline__ double from_ordered64(unsigned long long u) {
    return __longlong_as_double((long long)(u >> 63 ? u & ~(1ull << 63) : ~u));
}

// How many of `list`'s first n keys are above `mine`, 8 of them looked at together: one by one takes 23 cycles a key,
// 3200 of the 11000 of a piece of 2000 tokens of which 32 are kept.  The list's room is a multiple of 8, and it is 16-byte aligned.
__device__ __forceinline__ int better_than(unsigned long long mine, const unsigned long long *list, int n) {
    int better = 0, j = 0;
    auto look = [&](auto whole) {
        ulonglong2 v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = reinterpret_cast<const ulonglong2 *>(list + j)[k];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            better += v[k].x > mine && (decltype(whole)::value || j + 2 * k < n);
            better += v[k].y > mine && (decltype(whole)::value || j + 2 * k + 1 < n);
        }
    };
#pragma unroll 1
    for (; j + 8 <= n; j += 8) look(std::true_type{});
    if (j < n) look(std::false_type{});
    return better;
}

// A vector of 8 logits as it is in memory.
template <int DT>
struct Raw {
    uint32_t w[DT == 2 ? 8 : 4];
};
// A thread's vectors of a tile, at `at` and every kThreads vectors, of a row
// aligned to `align` bytes; -inf from `end` on.  Returns whether a warp's vectors
// are a half word late, the words that they begin in, where a row begins in the
// middle of one: shift_tile then.  (256 beams over 131071 bf16 logits: 52 us with
// loads of 2 bytes, 30 so; 24 over 131072 and loads of 16.)
template <int DT, int NV>
__device__ __forceinline__ bool load_tile(Raw<DT> (&x)[NV], const char *row, int align, int at, int end, bool first_row) {
    constexpr int N = DT == 2 ? 8 : 4, SIZE = DT == 2 ? 4 : 2;
    const char *p = row + (long long)at * SIZE;
    constexpr int STEP = kThreads * 8;
    if (align == 16 && at + (NV - 1) * STEP + 8 <= end) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < N; i += 4) {
                const uint4 v = ldg_stream_v4(p + j * STEP * SIZE + 4 * i);
                x[j].w[i] = v.x, x[j].w[i + 1] = v.y, x[j].w[i + 2] = v.z, x[j].w[i + 3] = v.w;
            }
        return false;
    }
    const int lane = threadIdx.x & 31;
    if (DT != 2 && align == 2 && at + (31 - lane) * 8 + (NV - 1) * STEP + 9 <= end && (at > lane * 8 || !first_row)) {
        const uint32_t *words = reinterpret_cast<const uint32_t *>(p - 2);
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < N; ++i) x[j].w[i] = __ldg(words + j * (STEP * SIZE / 4) + i);
        return true;
    }
#pragma unroll
    for (int j = 0; j < NV; ++j, p += STEP * SIZE, at += STEP) {
        const uint32_t *words = reinterpret_cast<const uint32_t *>(p);
        const uint16_t *halves = reinterpret_cast<const uint16_t *>(p);
        const uint32_t none = DT == 0 ? 0xfc00u : 0xff80u;
        if (align == 16 && at + 8 <= end) {
#pragma unroll
            for (int i = 0; i < N; i += 4) {
                const uint4 v = ldg_stream_v4(p + 4 * i);
                x[j].w[i] = v.x, x[j].w[i + 1] = v.y, x[j].w[i + 2] = v.z, x[j].w[i + 3] = v.w;
            }
            continue;
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (DT == 2)
                x[j].w[i] = at + i < end ? __ldg(words + i) : 0xff800000u;
            else if (align >= 4 && at + 2 * i + 1 < end)
                x[j].w[i] = __ldg(words + i);
            else
                x[j].w[i] = (at + 2 * i < end ? __ldg(halves + 2 * i) : none) |
                            (at + 2 * i + 1 < end ? (uint32_t)__ldg(halves + 2 * i + 1) : none) << 16;
        }
    }
    return false;
}
// What load_tile left half a word late.  A vector's last value is in the next
// thread's first word.
template <int DT, int NV>
__device__ __forceinline__ void shift_tile(Raw<DT> (&x)[NV], const char *row, int at) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        uint32_t beyond = __shfl_down_sync(0xffffffffu, x[j].w[0], 1);
        if ((threadIdx.x & 31) == 31) beyond = __ldg(reinterpret_cast<const uint32_t *>(row + 2LL * (at + j * kThreads * 8) + 14));
#pragma unroll
        for (int i = 0; i < 4; ++i) x[j].w[i] = __funnelshift_r(x[j].w[i], i < 3 ? x[j].w[(i + 1) & 3] : beyond, 16);
    }
}
template <int DT>
__device__ __forceinline__ float value_of(const Raw<DT> &r, int i) {
    if constexpr (DT == 2) return __uint_as_float(r.w[i]);
    else if constexpr (DT == 1) return __uint_as_float(i & 1 ? r.w[i / 2] & 0xffff0000u : r.w[i / 2] << 16);
    else return kv_act<0>((uint16_t)(r.w[i / 2] >> (16 * (i & 1))));
}

// Whether a beam is a source of continuations by its logits.
__device__ __forceinline__ bool goes_on(const BeamArgs &a, int row) {
    const float s = a.scores[row];
    const bool ended = a.finished && a.finished[row];
    return isfinite(s) && !ended;
}

// A beam's logits as tiles, and the pieces that they are cut into at most.
struct Cut {
    int row_tiles, slots;
};

template <int DT>
__global__ void __launch_bounds__(kThreads, 3) scan_kernel(const BeamArgs a, const Cut cut, PartSum *sums,
                                                           unsigned long long *lists) {
    constexpr int PER = kPer<DT>, NV = PER / 8, TILE = kThreads * PER;
    __shared__ __align__(16) unsigned long long list[kList];
    __shared__ __align__(16) unsigned long long s_best[kBeamMost], s_maxima[kThreads];
    __shared__ float s_group[kThreads];
    __shared__ unsigned long long s_least;
    __shared__ float s_hi[kWarps], s_lo[kWarps], s_max[kWarps];
    __shared__ int s_count[kWarps];
    __shared__ uint16_t s_rows[kMaxRows];
    __shared__ int vectors[kVectors];                      // the first tokens of vectors with candidates
    __shared__ int s_n, s_vectors;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, K = a.n_out;
    const int rows = a.n_groups * a.width;
    if (tid == 0) s_n = s_vectors = 0;
    // The next kernel is not let start early: with its CTAs waiting for room, a call of more CTAs than SMs took 24 us more.
    grid_dependency_wait();

    // ---- the beams that go on, in order (all of them where there are too many to look)
    unsigned alive = rows;
    if (rows <= kMaxRows) {
        alive = 0;
        for (int base = 0; base < rows; base += kThreads) {
            const bool on = base + tid < rows && goes_on(a, base + tid);
            const uint32_t bits = __ballot_sync(0xffffffffu, on);
            __syncthreads();
            if (lane == 0) s_count[warp] = __popc(bits);
            __syncthreads();
            int at = alive + __popc(bits & ((1u << lane) - 1));
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                at += w < warp ? s_count[w] : 0;
                alive += s_count[w];
            }
            if (on) s_rows[at] = (uint16_t)(base + tid);
        }
        __syncthreads();
    }
    if (alive == 0) return;
    // Pieces of a beam: as many as fill the grid once, twice and so on, whichever takes least with the cost of a piece's
    // start and end.  Lane i tries i + 1 rounds.
    // (32-bit numbers: 2^20 beams with 1024 / width pieces each at most, and a division of 64 bits is a hundred instructions.)
    const unsigned T = cut.row_tiles, grid = gridDim.x;
    unsigned q;
    {
        q = max(1u, min((lane + 1) * grid / alive, (unsigned)cut.slots));
        const unsigned rounds = (alive * q + grid - 1) / grid;
        const float cost = (float)rounds * (float)((T + q - 1) / q + kPieceCost);
        float least_cost = cost;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) least_cost = fminf(least_cost, __shfl_xor_sync(0xffffffffu, least_cost, d));
        q = __shfl_sync(0xffffffffu, q, __ffs(__ballot_sync(0xffffffffu, cost == least_cost)) - 1);
    }
    const unsigned units = alive * q, each = units / grid, more = units % grid;   // the first `more` CTAs have one more
    const unsigned u0 = blockIdx.x * each + min(blockIdx.x, more), u1 = u0 + each + (blockIdx.x < more);
    if (u0 == u1) return;

    float m = -INFINITY, hi = 0.0f, lo = 0.0f;             // of this thread and piece
    float least = -INFINITY;                               // the n-th best so far
    int kept = 0;                                          // candidates that the list was last cut to
    // The K best of the list's n candidates, in order; and the list cut to them.
    auto shorten = [&](int n) {
#pragma unroll 1
        for (int i = tid; i < n; i += kThreads) {
            const unsigned long long mine = list[i];
            const int better = better_than(mine, list, n);
            if (better < K) s_best[better] = mine;
        }
        __syncthreads();
    };
    auto keep_best = [&](int n) {
        if (tid < min(n, K)) list[tid] = s_best[tid];
        if (tid == 0) s_n = min(n, K);
        if (n >= K) least = key_value(s_best[K - 1]);
        __syncthreads();
    };

    auto start_of = [&](int row) {
        return static_cast<const char *>(a.logits) + row * a.row_stride * (DT == 2 ? 4 : 2);
    };
    auto logit = [&](int row, int token) {
        const char *p = start_of(row);
        if constexpr (DT == 2) return __ldg(reinterpret_cast<const float *>(p) + token);
        else return kv_act<DT>(__ldg(reinterpret_cast<const uint16_t *>(p) + token));
    };
    // A tile's candidates when there are too many of them: those of the K threads with the best maxima.
    auto careful = [&](int row, int tile) {
        const int base = tile * TILE;
        auto token_of = [&](int k) { return base + ((k >> 3) * kThreads + tid) * 8 + (k & 7); };
        unsigned long long best = 0;
#pragma unroll 4
        for (int k = 0; k < PER; ++k) {
            const int token = token_of(k);
            const float v = token < a.vocab ? logit(row, token) : -INFINITY;
            if (v > least) best = max(best, key_of(v, token));
        }
        s_maxima[tid] = best;
        if (tid == 0) s_least = 0;
        __syncthreads();
        const int better = better_than(best, s_maxima, kThreads);
        if (best != 0 && better == K - 1) s_least = best;
        __syncthreads();
        if (best >= max(s_least, 1ull))
#pragma unroll 1
            for (int k = 0; k < PER; ++k) {
                const int token = token_of(k);
                const float v = token < a.vocab ? logit(row, token) : -INFINITY;
                if (v > least && key_of(v, token) >= s_least) list[atomicAdd(&s_n, 1)] = key_of(v, token);
            }
        __syncthreads();
        const int n = s_n;
        shorten(n);
        keep_best(n);
    };

    Raw<DT> next[NV];
    bool next_late = false;
    int row = 0, piece = 0, tile = 0, last = 0;            // what is being loaded: a beam's piece, up to tile `last`
    auto open = [&](unsigned u) {
        const unsigned o = u / q;
        piece = u - o * q;
        row = rows <= kMaxRows ? (int)s_rows[o] : (int)o;
        tile = piece * T / q, last = (piece + 1) * T / q - 1;
    };
    int first = 0;                                         // of the tiles whose candidates are not in the list
    unsigned u = u0 - 1;                                   // + 1 is u0, also where that is 0
    for (bool started = false, fresh = true;;) {
        const int here = row, here_piece = piece, this_tile = tile, base = tile * TILE;
        const bool ends = !started || tile == last;
        Raw<DT> x[NV];
#pragma unroll
        for (int j = 0; j < NV; ++j) x[j] = next[j];
        if constexpr (DT != 2)
            if (next_late) shift_tile<DT>(x, start_of(here), base + tid * 8);
        if (!ends || u + 1 != u1) {
            if (ends) open(++u);
            else ++tile;
            const int end = rows <= kMaxRows || goes_on(a, row) ? a.vocab : 0;
            const char *p = start_of(row);
            const int low = (int)(reinterpret_cast<uintptr_t>(p) & 15), align = low == 0 ? 16 : low & 3 ? 2 : 4;
            next_late = load_tile<DT>(next, p, align, tile * TILE + tid * 8, end, row == 0);
        } else {
            ++u;
        }
        if (!started) {
            started = true;
            first = tile;
            continue;
        }
        float tops[NV], top = -INFINITY;                   // of each vector
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            tops[j] = -INFINITY;
#pragma unroll
            for (int e = 0; e < 8; e += 2)
                asm("max.f32 %0, %0, %1, %2;" : "+f"(tops[j]) : "f"(value_of<DT>(x[j], e)), "f"(value_of<DT>(x[j], e + 1)));
            top = fmaxf(top, tops[j]);
        }
        // ---- the sum
        const float to = fmaxf(m, top);
        if (to != m) {
            const float f = carried(m, to);
            hi *= f, lo *= f;
            m = to;
        }
        float s;
        if (fabsf(to) < kHuge) {
            const float r = -reference(to);
            const uint64_t rr = pair_of(r, r), ll = pair_of(kLog2e, kLog2e), low = pair_of(kLog2eLow, kLog2eLow);
            uint64_t sum[2] = {0, 0};
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    const uint64_t v = pair_of(value_of<DT>(x[j], e), value_of<DT>(x[j], e + 1));
                    float p, q;
                    unpair(fma2(v, low, fma2(v, ll, rr)), p, q);
                    sum[e >> 1 & 1] = add2(sum[e >> 1 & 1], pair_of(ex2(p), ex2(q)));
                }
            float p, q;
            unpair(add2(sum[0], sum[1]), p, q);
            s = p + q;
        } else {
            // a NaN stays one; no logit but -inf so far: none counts
            s = 0.0f;
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float v = value_of<DT>(x[j], e);
                    s += v != v ? v : v == to && to > -INFINITY ? 1.0f : 0.0f;
                }
        }
        add_to(hi, lo, s);
        // ---- candidates are in vectors with an x > least, in a piece's first tile an x >= bound
        float bound = -INFINITY;
        if (fresh) {
            // groups of every so-manieth thread: a last tile of few tokens is in the first threads
            const int groups = K <= 4 ? 4 : K <= 8 ? 8 : K <= 16 ? 16 : K <= 32 ? 32 : 64, across = min(groups, 32);
            float g = top;
            for (int d = 16; d >= across; d >>= 1) g = fmaxf(g, __shfl_xor_sync(0xffffffffu, g, d));
            s_group[tid] = g;
            __syncthreads();
            float even = -INFINITY, odd = -INFINITY;
#pragma unroll
            for (int w = 0; w < kWarps; w += 2) {
                even = fmaxf(even, s_group[w * 32 + lane]);
                odd = fmaxf(odd, s_group[(w + 1) * 32 + lane]);
            }
            bound = groups == 64 ? fminf(even, odd) : fmaxf(even, odd);
            for (int d = across / 2; d > 0; d >>= 1) bound = fminf(bound, __shfl_xor_sync(0xffffffffu, bound, d));
        }
        if (top > least && top >= bound) {
#pragma unroll
            for (int j = 0; j < NV; ++j)
                if (tops[j] > least && tops[j] >= bound) {
                    const int at = atomicAdd(&s_vectors, 1);
                    if (at < kVectors) vectors[at] = base + (j * kThreads + tid) * 8;
                }
        }
        if (!ends && !fresh && this_tile - first < kBatch - 1) continue;
        // ---- the candidates of the tiles since the last time
        __syncthreads();
        const int found = s_vectors;
        if (found <= kVectors)
            for (int i = tid; i < 8 * found; i += kThreads) {
                const int token = vectors[i >> 3] + (i & 7);
                const float v = token < a.vocab ? logit(here, token) : -INFINITY;
                if (v > least && v >= bound) {
                    const int at = atomicAdd(&s_n, 1);
                    if (at < kList) list[at] = key_of(v, token);
                }
            }
        __syncthreads();
        int n = s_n;
        if (found > kVectors || n > kList) {
            // too many: again, tile by tile, after what the list had been cut to before
            __syncthreads();
            if (tid == 0) s_n = kept;
#pragma unroll 1
            for (int i = first; i <= this_tile; ++i) careful(here, i);
            n = s_n;
        }
        if (tid == 0) s_vectors = 0;
        shorten(n);
        fresh = ends;
        if (!ends) {
            keep_best(n);
            kept = min(n, K);
            first = this_tile + 1;
            continue;
        }
        // ---- the piece's end: its candidates, and the threads' sums joined
        const long long slot = (long long)here * cut.slots + here_piece;
        if (tid < K) lists[slot * K + tid] = tid < n ? s_best[tid] : 0;
        float all = m;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) all = fmaxf(all, __shfl_xor_sync(0xffffffffu, all, d));
        if (lane == 0) s_max[warp] = all;
        __syncthreads();
        if (tid == 0) s_n = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) all = fmaxf(all, s_max[w]);
        const float f = carried(m, all);
        hi *= f, lo *= f;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) {
            const float h = __shfl_xor_sync(0xffffffffu, hi, d), r = __shfl_xor_sync(0xffffffffu, lo, d);
            add_to(hi, lo, h);
            lo += r;
        }
        if (lane == 0) s_hi[warp] = hi, s_lo[warp] = lo;
        __syncthreads();
        if (tid == 0) {
            hi = s_hi[0], lo = s_lo[0];
            for (int w = 1; w < kWarps; ++w) {
                add_to(hi, lo, s_hi[w]);
                lo += s_lo[w];
            }
            sums[slot] = PartSum{(double)hi + (double)lo, all, (int)q};
        }
        if (u == u1) return;
        m = -INFINITY, hi = lo = 0.0f, least = -INFINITY;
        first = tile, kept = 0;
    }
}

// The logarithm of a sum l over one of its weights w, the largest, to 2^-29: of the quotient's fraction f in
// [0.7, 1.4] as 2 atanh(q), q = (f - 1) / (f + 1), in two fp32 numbers and a
// series in q^2.  64-bit arithmetic is slow here: log() takes 1.5 us.
__device__ __forceinline__ double log_over(double l, float w) {
    const float h = (float)l, over = h / w;            // the quotient: this and `left`
    const float left = __fdividef(fmaf(-over, w, h) + (float)(l - (double)h), w);
    int e = (int)(__float_as_uint(over) >> 23) - 127;
    float scale = __uint_as_float((uint32_t)(127 - e) << 23);
    if (over * scale > 1.41421356f) scale *= 0.5f, ++e;
    const float fh = over * scale, fl = left * scale;
    const float n = fh - 1.0f, d = fh + 1.0f, dl = (fh - (d - 1.0f)) + fl;   // n exactly, d to its rounding, which dl holds
    const float q = n / d, ql = __fdividef(fmaf(-q, d, n) + fl - q * dl, d), z = q * fmaf(2.0f, ql, q);
    float s = 1.0f / 13.0f;                            // z^6 / 13 < 6e-11
    s = fmaf(s, z, 1.0f / 11.0f);
    s = fmaf(s, z, 1.0f / 9.0f);
    s = fmaf(s, z, 1.0f / 7.0f);
    s = fmaf(s, z, 1.0f / 5.0f);
    s = fmaf(s, z, 1.0f / 3.0f);
    const float rest = 2.0f * fmaf(q * z, s, ql);
    return fma((double)e, 0.693147180559945309417, (double)(2.0f * q) + (double)rest);
}
// What a beam's largest logit counts for in its sum, as scan_kernel has it, bit for bit.
__device__ __forceinline__ float largest_weight(float m) {
    return fabsf(m) >= kHuge ? 1.0f : ex2(__fmaf_rn(m, kLog2eLow, __fmaf_rn(m, kLog2e, -reference(m))));
}

// One is better than another when it is greater.  The order of its score, 0 for none; among equal ones the lower
// beam, the greater logit, the lower token.  Integers: comparing 64-bit numbers is slow here.
struct __align__(16) Candidate {
    unsigned long long score, key;                         // key: 63 - beam, the logit's order, 2^24 - 1 - token
    __device__ bool operator>(const Candidate &o) const {
        // whether o less this borrows, as 128-bit numbers: with branches a comparison takes 100 cycles, with both words'
        // comparisons 30
        uint32_t borrow;
        asm("{ .reg .u64 t; sub.cc.u64 t, %1, %2; subc.cc.u64 t, %3, %4; subc.u32 %0, 0, 0; }"
            : "=r"(borrow) : "l"(o.key), "l"(key), "l"(o.score), "l"(score));
        return borrow != 0;
    }
};
// How many of the n from `list` on are better, eight of them looked at together.
__device__ __forceinline__ int better_than(const Candidate &c, const Candidate *list, int n) {
    int better = 0, j = 0;
#pragma unroll 1
    for (; j + 8 <= n; j += 8) {
        Candidate o[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) o[k] = list[j + k];
#pragma unroll
        for (int k = 0; k < 8; ++k) better += o[k] > c;
    }
#pragma unroll 1
    for (; j < n; j += 2) {
        const Candidate o0 = list[j], o1 = list[min(j + 1, n - 1)];
        better += (o0 > c) + (j + 1 < n && o1 > c);
    }
    return better;
}

// A CTA per request: its beams' sums, then the best of the candidates.
template <int THREADS>
__global__ void __launch_bounds__(THREADS, 1) merge_kernel(const BeamArgs a, const Cut cut, const PartSum *sums,
                                                              const unsigned long long *lists, int *status) {
    // no static shared memory: raise_smem_cap
    extern __shared__ double dyn[];
    const int tid = threadIdx.x, lane = tid & 31, K = a.n_out, W = a.width, slots = cut.slots, n_lists = W * slots;
    double *s_top = dyn, *s_cum = s_top + kBeamMost;       // of each beam: its largest logit; its score less log sum
                                                           // e^(x - largest)
    Candidate *s_least = reinterpret_cast<Candidate *>(s_cum + kBeamMost);
    Candidate *s_heads = s_least + 1, *s_best = s_heads, *s_cand = s_heads + kMaxLists;
    int *s_which = reinterpret_cast<int *>(s_cand + K * K), *s_list = s_which + kMaxLists;
    int *s_parts = s_list + kBeamMost;                     // of each beam: lists it has, -1 where it has finished
    int *s_count = s_parts + kBeamMost;
    const int row0 = blockIdx.x * W;
    if (tid < 4) s_count[tid] = 0;
    if (tid == 0) *s_least = Candidate{0, 0};
    kv_begin();
    const unsigned long long *mine = lists + (long long)row0 * slots * K;
    // all loads at once: what a beam has no part for is not looked at
    unsigned long long head = 0;
    if (tid < n_lists) head = mine[(long long)tid * K];
    const float own_score = tid < W ? a.scores[row0 + tid] : 0.0f;
    // a beam's sum l and largest logit, and what they come to
    auto finish = [&](int b, float score, double l, float top, int parts, bool writes) {
        double largest = 0.0, log_sum = 0.0;
        // the row of a NaN or +inf has no probabilities, one without any token but -inf has no continuations
        if (parts > 0 && (top == INFINITY || l != l)) {
            if (writes) kv_report(status);
            parts = 0;
        } else if (parts > 0 && top == -INFINITY) {
            parts = 0;
        } else if (parts > 0) {
            largest = top;
            // relative to the largest, whose own weight as it was added up counts for 1: its exponential's error cancels, and
            // one token, or equal ones, come to their number.  No token may get more than its beam has.
            log_sum = log_over(l, largest_weight(top));
            if (__double2hiint(log_sum) < 0) log_sum = 0.0;
        }
        if (writes) s_top[b] = largest, s_cum[b] = score - log_sum, s_parts[b] = parts;
    };
    // `across` lanes a beam: as many as it may have pieces, a warp at most.  Of more than a few warps the logarithms come
    // afterwards, a lane a beam: 64-bit instructions take a warp 16 cycles and more each (16 beams of 32 pieces: 10400
    // cycles, 7900 so; 4 beams of 8 3300, 4200 so).
    const int across = slots > 16 ? 32 : slots > 8 ? 16 : slots > 4 ? 8 : slots > 2 ? 4 : slots;
    const bool afterwards = W * across > 128;
    for (int base = 0; base < W; base += THREADS / across) {
        const int b = base + tid / across, part0 = tid % across;
        const bool real = b < W;
        const PartSum *p = sums + (long long)(row0 + (real ? b : 0)) * slots;
        const float score = real ? a.scores[row0 + b] : 0.0f;
        const bool ended = real && a.finished && a.finished[row0 + b];
        PartSum part = {0.0, 0.0f, 0};
        if (part0 < slots) part = p[part0];
        int parts = __shfl_sync(0xffffffffu, part.parts, lane - part0);
        if (!real || ended || !isfinite(score)) parts = 0;
        float top = part0 < parts ? part.m : -INFINITY;
        for (int i = part0 + 32; i < parts; i += 32) top = fmaxf(top, p[i].m);
        for (int d = across / 2; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        double l = part0 < parts ? part.l * carried(part.m, top) : 0.0;
        for (int i = part0 + 32; i < parts; i += 32) l += p[i].l * carried(p[i].m, top);
        for (int d = across / 2; d > 0; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
        if (ended && isfinite(score)) parts = -1;
        const bool writes = real && part0 == 0;
        if (!afterwards) finish(b, score, l, top, parts, writes);
        else if (writes) s_top[b] = top, s_cum[b] = l, s_parts[b] = parts;
    }
    __syncthreads();
    if (afterwards) {
        if (tid < W) finish(tid, own_score, s_cum[tid], (float)s_top[tid], s_parts[tid], true);
        __syncthreads();
    }
    // a list's i-th candidate
    auto candidate = [&](int list, int i, unsigned long long key) {
        const int b = list / slots, part = list - b * slots, parts = s_parts[b];
        const unsigned long long beam = (unsigned long long)(63 - b) << 56;
        if (parts < 0)                                     // goes on as it is
            return Candidate{part == 0 && i == 0 ? ordered64(s_cum[b]) : 0ull, beam | (0xffffffu - a.end_token)};
        if (part >= parts || key == 0) return Candidate{0, 0};
        return Candidate{ordered64(s_cum[b] + ((double)key_value(key) - s_top[b])),
                         beam | key >> 32 << 24 | (0xffffffu - key_token(key))};
    };
    // places for those threads of a warp that want one
    auto place_for = [&](bool want, int *count) {
        const uint32_t bits = __ballot_sync(0xffffffffu, want);
        int at = 0;
        if (lane == 0 && bits) at = atomicAdd(count, __popc(bits));
        return __shfl_sync(0xffffffffu, at, 0) + __popc(bits & ((1u << lane) - 1));
    };
    // the lists by their heads; only the n best of them matter
    for (int base = 0; base < n_lists; base += THREADS) {
        const int i = base + tid;
        Candidate c = {0, 0};
        if (i < n_lists) c = candidate(i, 0, base == 0 ? head : mine[(long long)i * K]);
        const int at = place_for(c.score != 0, s_count);
        if (c.score != 0) s_heads[at] = c, s_which[at] = i;
    }
    __syncthreads();
    int heads = s_count[0];
    if (heads > kFewHeads) {
        // those from the n-th best score on, by the 32 bits that say most, which are found bit by bit
        Candidate c = {0, 0};
        int which = 0;
        if (tid < heads) c = s_heads[tid], which = s_which[tid];
        const uint32_t mine32 = (uint32_t)(c.score >> 32);
        uint32_t low = 0;
        for (int bit = 31; bit >= 0; --bit)
            if (__syncthreads_count(mine32 >= (low | 1u << bit)) >= K) low |= 1u << bit;
        const bool stays = tid < heads && mine32 >= low;
        const int at = place_for(stays, s_count + 3);
        if (stays) s_heads[at] = c, s_which[at] = which;
        __syncthreads();
        heads = s_count[3];
    }
    const int L = min(heads, K);
    for (int i = tid; i < heads; i += THREADS) {
        const Candidate c = s_heads[i];
        const int place = better_than(c, s_heads, heads);
        if (place < K) s_list[place] = s_which[i];
        if (place == K - 1) *s_least = c;
    }
    __syncthreads();
    // their candidates, the first ones of all lists, the second ones and so on.  The l-th of the list with the j-th best head
    // has j + l better ones, one below n heads has n.
    const Candidate least = *s_least;
    for (int base = 0; base < L * K; base += THREADS) {
        const int i = base + tid, l = i / L, j = i - l * L;
        Candidate c = {0, 0};
        if (i < L * K && j + l < K) c = candidate(s_list[j], l, mine[(long long)s_list[j] * K + l]);
        if (least > c) c = {0, 0};
        if (i < L * K) s_cand[i] = c;
        const int at = place_for(c.score != 0, s_count + 1);
        if (c.score != 0 && at < kFewCandidates) s_best[at] = c;
    }
    __syncthreads();
    int n = s_count[1];
    if (n > kFewCandidates) {
        // where b lists have a better l-th one, (b + 1) (l + 1) - 1 are better: some n log n may be among the n best
        for (int base = 0; base < L * K; base += THREADS) {
            const int i = base + tid, l = i / L;
            const Candidate c = i < L * K ? s_cand[i] : Candidate{0, 0};
            const bool may = c.score != 0 && (better_than(c, s_cand + l * L, L) + 1) * (l + 1) <= K;
            const int at = place_for(may, s_count + 2);
            if (may) s_best[at] = c;
        }
        __syncthreads();
        n = s_count[2];
    }
    for (int i = tid; i < n; i += THREADS) {
        const Candidate c = s_best[i];
        const int place = better_than(c, s_best, n);
        if (place >= K) continue;
        const int b = 63 - (int)(c.key >> 56), token = 0xffffff - (int)(c.key & 0xffffffu);
        const long long at = (long long)blockIdx.x * K + place;
        a.out_scores[at] = (float)from_ordered64(c.score);
        a.out_rows[at] = row0 + b;
        a.out_tokens[at] = token;
        if (a.out_finished) a.out_finished[at] = s_parts[b] < 0 || token == a.end_token;
    }
    for (int i = n + tid; i < K; i += THREADS) {
        const long long at = (long long)blockIdx.x * K + i;
        a.out_scores[at] = -INFINITY;
        a.out_rows[at] = a.out_tokens[at] = -1;
        if (a.out_finished) a.out_finished[at] = 0;
    }
}

// A request's beams have kMaxLists pieces at most.
Cut cut_of(int width, int vocab, int dtype) {
    const int tile = kThreads * (dtype == 2 ? kPer<2> : kPer<0>), tiles = (vocab + tile - 1) / tile;
    return Cut{tiles, std::min(tiles, kMaxLists / width)};
}

}  // namespace

cudaError_t launch_beam_select(const BeamArgs &a, void *workspace, const DeviceInfo &dev, cudaStream_t s, bool pdl) {
    const int rows = a.n_groups * a.width;
    const Cut cut = cut_of(a.width, a.vocab, a.dtype);
    PartSum *sums = static_cast<PartSum *>(workspace);
    unsigned long long *lists = reinterpret_cast<unsigned long long *>(sums + (long long)rows * cut.slots);
    const dim3 grid((unsigned)std::min<long long>((long long)rows * cut.slots, 3 * dev.sm_count));
    const dim3 block(kThreads);
    cudaError_t e = a.dtype == 0   ? kv_launch(scan_kernel<0>, grid, block, 0, s, pdl, a, cut, sums, lists)
                    : a.dtype == 1 ? kv_launch(scan_kernel<1>, grid, block, 0, s, pdl, a, cut, sums, lists)
                                   : kv_launch(scan_kernel<2>, grid, block, 0, s, pdl, a, cut, sums, lists);
    if (e != cudaSuccess) return e;
    const size_t smem = 2 * kBeamMost * 8 + (1 + kMaxLists + (size_t)a.n_out * a.n_out) * 16 + (kMaxLists + 2 * kBeamMost + 4) * 4;
    // few candidates are in order sooner in a small CTA, many in a large one
    const int n_lists = a.width * cut.slots;
    const bool large = n_lists > 256 || std::min(n_lists, a.n_out) * a.n_out > kSmallMerge;   // no more heads than threads
    const auto merge = large ? merge_kernel<1024> : merge_kernel<256>;
    e = raise_smem_cap(reinterpret_cast<const void *>(merge), smem);
    if (e != cudaSuccess) return e;
    return kv_launch(merge, dim3(a.n_groups), dim3(large ? 1024 : 256), smem, s, pdl, a, cut, sums, lists, dev.status);
}

long long beam_select_workspace(int n_groups, int width, int vocab, int n_out) {
    // of the type with the smallest tiles
    const Cut cut = cut_of(width, vocab, 2);
    return (long long)n_groups * width * cut.slots * (sizeof(PartSum) + 8LL * n_out);
}

}  // namespace w4a16
