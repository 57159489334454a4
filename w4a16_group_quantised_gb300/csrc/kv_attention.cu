// kv_attention.cu -- attention of few query rows over the paged 8-bit cache.
//
// For one kv head, with codes k_j, v_j of key j, page scales ks, vs and a
// query row q (a token and query head of the group),
//     x_j = scale log2(e) ks (q . k_j),     out = sum_j 2^x_j vs v_j / sum_j 2^x_j.
// The values' scale goes into the exponent: with e_j = x_j + log2(vs) - M the
// weights 2^e_j multiply the codes as they are, and the denominator gets
// 2^e_j / vs.  M is a running reference of each row, moved up only when some
// e_j passes 15, so that 2^e_j fits fp16 with its top 22 binades exact to
// 2^-11 and nothing above 2^-31 of the largest lost; the sums (out, the
// denominator) are fp32.
//
// Bound by the cache read: 256 B a key and kv head (head dim 128) against
// rows * 512 multiply-adds.  So the design is about bytes in flight and even
// shares, not about matrix instructions:
//  * The work is a line of steps of 16 keys: sequence by sequence, kv head by
//    kv head, row tile by row tile, every step of the keys that the sequence's
//    new tokens see.  Lengths are read here, so each CTA sums the line's
//    length up itself, takes an equal piece of it, and its warps take equal
//    pieces of that.  Ragged lengths, windows and few long sequences all
//    spread over the whole GPU alike.
//  * A warp is on its own: it owns a ring of stages, its first lane issues
//    the two TMA boxes (16 keys of K, of V) of a step into it, all lanes
//    consume.  No barrier among warps until their pieces end.  Page ids and
//    scales of 32 steps are looked up at once, one step a lane.
//  * mma.sync m16n8k16 with the keys as A (16 keys x 16 dims) and the rows as
//    B (8 rows): S^T = K Q^T, then P^T through two movmatrix transposes, then
//    out^T = V^T P^T.  The dims and keys are permuted so that every operand
//    comes from wide conflict-free shared loads (128- or 64-byte swizzled by
//    the TMA): a lane's 16 bytes of K are four k-steps of A.  Rows are at
//    most 16 here: a 128-row tcgen05 tile would be nearly empty.
//  * A tile that several warps share is summed through shared memory, one
//    that several CTAs share through the workspace, the CTA that comes last
//    summing all parts in order: the result does not depend on who that is.
//    Tickets carry the launch's number, so scratch needs no initialisation.
#include <cuda.h>

#include <algorithm>
#include <atomic>

#include "kv.cuh"
#include "skinny.cuh"

namespace w4a16 {
namespace {

constexpr int kStep = 16;                 // keys of a step
constexpr int kMaxSeqs = 1024;            // sequences of a launch
constexpr int kShort = 16;                // tiles of up to so many steps stay in one CTA
constexpr int kLeast = 4;                 // fewest steps worth a CTA
constexpr float kRefStart = -3.402823466e38f;
constexpr float kTop = 15.9f;             // weights stay below 2^kTop, inside fp16 ...
constexpr float kHead = 14.0f;            // ... and a moved reference puts the largest at 2^kHead

struct FewParams {
    KvAttentionArgs a;
    KvCache c;
    KvBatch b;
    int row_limit;                        // sequences with more rows a kv head than this are another kernel's (0: none)
    int token_first;                      // tensor map dims are (dim, head, token, page), not (dim, token, head, page)
    float *parts;                         // [grid][2][ROWS][D + 2]
    unsigned long long *tickets;          // [grid]
    unsigned long long tag;
    int *status;
};

// Steps of the keys that new tokens of a sequence see: [0, sink_steps) and
// [first_step, ...), `steps` in all, one at least.
struct Span {
    int steps, sink_steps, first_step;
};
__device__ __forceinline__ Span span_of(int n, int len, int window, int sinks) {
    Span s;
    const int lo = window > 0 ? max(0, len - n + 1 - window) : 0;
    s.first_step = lo / kStep;
    s.sink_steps = (min(sinks, lo) + kStep - 1) / kStep;
    if (s.sink_steps >= s.first_step) s.sink_steps = s.first_step;
    s.steps = max(s.sink_steps + (len + kStep - 1) / kStep - s.first_step, 1);
    return s;
}

template <int D, int NR, int NW, int NS>
struct FewSmem {
    static constexpr int kRows = 8 * NR;
    static constexpr int kStage = 2 * kStep * D;                   // K then V
    static constexpr int kPart = kRows * (D + 2);                  // floats: rows of out, then (M, l) of each row
    static constexpr int kPark = NW * NS * kStage;                 // a warp's first piece, if another began it
    static constexpr int kSeq = kPark + NW * kPart * 4;            // int4 {q0, n, len, row tiles}
    static constexpr int kPre = kSeq + kMaxSeqs * 16;              // line position of each sequence
    static constexpr int kBars = kPre + (kMaxSeqs + 1) * 8;
    static constexpr int kMisc = kBars + NW * NS * 8;
    static constexpr int kEnd = kMisc + (NW + 3) * 8 + 1024;       // 1024: slack to align the base
    static_assert(NS * kStage >= kPart * 4, "the last piece is parked in the ring");
};

__device__ __forceinline__ uint32_t movmatrix(uint32_t v) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
__device__ __forceinline__ float ex2(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t hsub2(uint32_t a, uint32_t b) {
    const __half2 r = __hsub2(*reinterpret_cast<const __half2 *>(&a), *reinterpret_cast<const __half2 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&r);
}

// Codes of a word as fp16 pairs (bytes 0, 1) and (2, 3), exactly.  int8: the
// code + 128 as the low byte of 0x6400 is 1024 + 128 + code.
template <int KT>
__device__ __forceinline__ void codes_to_half(uint32_t w, uint32_t &lo, uint32_t &hi) {
    if (KT == kKvInt8) {
        w ^= 0x80808080u;
        lo = hsub2(__byte_perm(w, 0x64646464u, 0x4140), 0x64806480u);
        hi = hsub2(__byte_perm(w, 0x64646464u, 0x4342), 0x64806480u);
    } else {
        asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t"
            "cvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
            : "=r"(lo), "=r"(hi)
            : "r"(w));
    }
}

// What a step needs, held by the lane that looked it up.
struct Meta {
    int page, where;       // page or -1; first token within the page | kv head << 8
    int pos;               // position of the first key (past every query for a page that is not there)
    int tile;              // where on the CTA's line its tile begins (below 0: in an earlier CTA)
    float ks, lv, iv;      // key scale, log2 and reciprocal of the value scale
};

template <int KT, int D, int NR, int NW, int NS>
__global__ void __launch_bounds__(32 * NW, 1)
    few_rows_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                    const FewParams p) {
    using L = FewSmem<D, NR, NW, NS>;
    constexpr int ROWS = L::kRows;
    constexpr int KS = D / 16;                                     // k-steps of S, and 16-dim tiles of out
    extern __shared__ uint8_t smem_raw[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);    // swizzled tiles need it
    // no static shared memory: the launch may ask for all of an SM's
    long long *s_scan = reinterpret_cast<long long *>(smem + L::kMisc), *s_cut = s_scan + NW;
    int &s_abort = *reinterpret_cast<int *>(s_cut + 2), &s_last = *(&s_abort + 1);
    int4 *seqs = reinterpret_cast<int4 *>(smem + L::kSeq);
    long long *pre = reinterpret_cast<long long *>(smem + L::kPre);
    const uint32_t ring = smem_u32(smem) + warp * NS * L::kStage;
    const uint32_t bars = smem_u32(smem + L::kBars) + warp * NS * 8;
    const int Hk = p.c.n_kv_heads, group = p.a.n_heads / Hk, B = p.b.n_seqs;

    if (tid == 0) {
        s_abort = 0;
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
    }
    if (lane < NS) mbar_init(bars + lane * 8, 1);
    fence_mbar_init();
    kv_begin();

    // ---- the line: each sequence's steps, summed up
    long long total = 0;
    for (int base = 0; base < B; base += 32 * NW) {
        const int i = base + tid;
        long long v = 0;
        if (i < B) {
            const KvSeq s = kv_sequence(p.b, p.c.page_shift, i, p.status);
            const int rows = s.n * group;
            const int tiles = p.row_limit > 0 && rows > p.row_limit ? 0 : (rows + ROWS - 1) / ROWS;
            seqs[i] = make_int4(s.q0, s.n, s.len, tiles);
            v = (long long)tiles * Hk * span_of(s.n, s.len, p.a.window, p.a.sinks).steps;
        }
        long long inc = v;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const long long o = __shfl_up_sync(0xffffffffu, inc, d);
            if (lane >= d) inc += o;
        }
        __syncthreads();
        if (lane == 31) s_scan[warp] = inc;
        __syncthreads();
        long long ahead = total;
        for (int w = 0; w < NW; ++w) {
            ahead += w < warp ? s_scan[w] : 0;
            total += s_scan[w];
        }
        if (i < B) pre[i] = ahead + inc - v;
    }
    if (tid == 0) pre[B] = total;
    __syncthreads();
    if (total == 0) return;

    // the sequence of a position of the line
    auto find = [&](long long at) {
        int lo = 0, hi = B - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (pre[mid] <= at) lo = mid;
            else hi = mid - 1;
        }
        return lo;
    };
    const long long ctas = min((long long)gridDim.x, (total + kLeast - 1) / kLeast);
    // where CTA i begins: an equal share, moved back to the tile's start in a short tile
    auto cut = [&](long long i) {
        const long long raw = i * total / ctas;
        if (raw <= 0 || raw >= total) return raw;
        const int b = find(raw);
        const int4 s = seqs[b];
        const int steps = span_of(s.y, s.z, p.a.window, p.a.sinks).steps;
        return steps > kShort ? raw : raw - (raw - pre[b]) % steps;
    };
    if (blockIdx.x >= ctas) return;
    if (tid < 2) s_cut[tid] = cut((long long)blockIdx.x + tid);
    __syncthreads();
    const long long c0 = s_cut[0], c1 = s_cut[1];
    if (c0 >= c1) return;
    const int mine = (int)(c1 - c0);
    const int w0 = (int)((long long)mine * warp / NW), w1 = (int)((long long)mine * (warp + 1) / NW);

    // ---- 32 steps looked up at once, one a lane
    auto look_up = [&](int at) {
        Meta m;
        m.page = -1, m.where = 0, m.pos = 0x7fffff00, m.tile = -1, m.ks = 0.0f, m.lv = 0.0f, m.iv = 0.0f;
        if (at < w1) {
            const long long line = c0 + at;
            const int b = find(line);
            const int4 s = seqs[b];
            const Span sp = span_of(s.y, s.z, p.a.window, p.a.sinks);
            const long long rem = line - pre[b];
            const int tile = (int)(rem / sp.steps), st = (int)(rem - (long long)tile * sp.steps);
            const int head = tile / s.w;
            const int blk = st < sp.sink_steps ? st : sp.first_step + st - sp.sink_steps;
            m.tile = at - st;
            m.where = (blk * kStep & ((1 << p.c.page_shift) - 1)) | head << 8;
            if (blk * kStep < s.z) m.page = kv_page(p.c, p.b, b, blk * kStep >> p.c.page_shift, p.status);
            if (m.page >= 0) {
                m.pos = blk * kStep;
                const long long i = (long long)m.page * Hk + head;
                m.ks = __ldg(p.c.k_scale + i);
                const float vs = __ldg(p.c.v_scale + i);
                m.lv = __log2f(vs);
                m.iv = 1.0f / vs;
            }
        }
        return m;
    };
    auto issue = [&](int stage, int page, int where) {
        if (lane == 0) {
            const uint32_t bar = bars + stage * 8, dst = ring + stage * L::kStage;
            mbar_arrive_expect_tx(bar, L::kStage);
            const int tok = where & 255, head = where >> 8;
            const int x = p.token_first ? head : tok, y = p.token_first ? tok : head;
            tma_load_4d(dst, &tm_k, bar, 0, x, y, page);
            tma_load_4d(dst + kStep * D, &tm_v, bar, 0, x, y, page);
        }
    };

    Meta cur = look_up(w0 + lane), nxt = cur;
    int fetched = w0;                                              // steps issued so far
    for (; fetched < min(w0 + NS, w1); ++fetched) {
        const int l = fetched - w0;
        issue(l, __shfl_sync(0xffffffffu, cur.page, l), __shfl_sync(0xffffffffu, cur.where, l));
    }
    nxt = look_up(w0 + 32 + lane);

    // ---- the running tile
    uint32_t q[NR][KS][2];
    float o[NR][KS][4], ref[NR][2], sum[NR][2], fac[NR][2];
    int row_pos[NR][2];                                            // position of each row's token; -1: no such row
    int tile = -1, tile_q0 = 0, tile_n = 0, tile_row = 0, tile_head = 0, min_pos = 0, max_pos = 0;

    auto row_of = [&](int nr, int e) { return nr * 8 + 2 * t + e; };
    // token row and query head of a row of the tile; false past the last
    auto place = [&](int row, long long &at) {
        const int r = tile_row + row;
        if (r >= tile_n * group) return false;
        at = (long long)(tile_q0 + r / group) * p.a.n_heads + tile_head * group + r % group;
        return true;
    };
    auto start_tile = [&](int at) {
        const long long line = c0 + at;
        const int b = find(line);
        const int4 s = seqs[b];
        const Span sp = span_of(s.y, s.z, p.a.window, p.a.sinks);
        const int idx = (int)((line - pre[b]) / sp.steps);
        tile_head = idx / s.w;
        tile_row = idx % s.w * ROWS;
        tile_q0 = s.x, tile_n = s.y;
        const int first = s.z - s.y;
        min_pos = first + tile_row / group;
        max_pos = first + min(tile_row + ROWS - 1, s.y * group - 1) / group;
#pragma unroll
        for (int nr = 0; nr < NR; ++nr) {
            // row g's dims as B: for a lane's chunk t (and t + 4), four words of four dims each
            float x[KS][4];
            float top = 0.0f;
            const int r = tile_row + nr * 8 + g;
            const bool has = r < s.y * group;
            const uint16_t *src = static_cast<const uint16_t *>(p.a.q) + (long long)(s.x + r / group) * p.a.q_stride +
                                  (tile_head * group + r % group) * D;
#pragma unroll
            for (int j = 0; j < KS / 4; ++j) {
                uint4 v[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
                if (has) {
                    v[0] = ldg_nc_v4(src + (t + 4 * j) * 16);
                    v[1] = ldg_nc_v4(src + (t + 4 * j) * 16 + 8);
                }
                const uint32_t w[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
#pragma unroll
                for (int i = 0; i < 8; ++i)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const uint16_t h = (uint16_t)(w[i] >> (16 * e));
                        const float f = p.a.dtype == 0 ? kv_act<0>(h) : kv_act<1>(h);
                        x[4 * j + i / 2][2 * (i & 1) + e] = f;
                        top = fmaxf(top, fabsf(f));
                    }
            }
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            // a power of two puts the row's largest value in [2^14, 2^15): exact for fp16, and for
            // bf16 down to 2^-28 of that value
            const int ex = min(max((int)(__float_as_uint(top) >> 23) - 127, -100), 127);
            const float up = __uint_as_float((uint32_t)(14 - ex + 127) << 23);
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                q[nr][k][0] = pack_half2(x[k][0] * up, x[k][1] * up);
                q[nr][k][1] = pack_half2(x[k][2] * up, x[k][3] * up);
            }
            const float back = __uint_as_float((uint32_t)(ex - 14 + 127) << 23) * p.a.scale * 1.4426950408889634f;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                fac[nr][e] = __shfl_sync(0xffffffffu, back, (2 * t + e) * 4);
                const int rr = tile_row + row_of(nr, e);
                row_pos[nr][e] = rr < s.y * group ? first + rr / group : -1;
                ref[nr][e] = kRefStart;
                sum[nr][e] = 0.0f;
            }
#pragma unroll
            for (int k = 0; k < KS; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[nr][k][i] = 0.0f;
        }
        tile = at;
    };
    // dims of out that o[.][k][0..1] (i = 0) and o[.][k][2..3] (i = 1) hold: a lane has D / 8 in a row
    // from g * D / 8 on, k and i counting them.
    auto sum_rows = [&]() {
#pragma unroll
        for (int nr = 0; nr < NR; ++nr)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                sum[nr][e] += __shfl_xor_sync(0xffffffffu, sum[nr][e], 4);
                sum[nr][e] += __shfl_xor_sync(0xffffffffu, sum[nr][e], 8);
                sum[nr][e] += __shfl_xor_sync(0xffffffffu, sum[nr][e], 16);
            }
    };
    auto store_row = [&](long long at, int d0, const float *v, int count, float l, float m) {
        const float r = l == 0.0f ? 0.0f : 1.0f / l;
        uint16_t *dst = static_cast<uint16_t *>(p.a.out) + at * D + d0;
        for (int i = 0; i < count; i += 4) {
            uint2 w;
            if (p.a.dtype == 0) {
                w.x = (uint32_t)kv_to_act<0>(v[i] * r) | (uint32_t)kv_to_act<0>(v[i + 1] * r) << 16;
                w.y = (uint32_t)kv_to_act<0>(v[i + 2] * r) | (uint32_t)kv_to_act<0>(v[i + 3] * r) << 16;
            } else {
                w.x = (uint32_t)kv_to_act<1>(v[i] * r) | (uint32_t)kv_to_act<1>(v[i + 1] * r) << 16;
                w.y = (uint32_t)kv_to_act<1>(v[i + 2] * r) | (uint32_t)kv_to_act<1>(v[i + 3] * r) << 16;
            }
            *reinterpret_cast<uint2 *>(dst + i) = w;
        }
        if (p.a.lse && d0 == 0) p.a.lse[at] = l == 0.0f ? -INFINITY : (m + __log2f(l)) * 0.6931471805599453f;
    };
    // The tile's part of this warp: to the output when `whole`, else to `park`.
    auto finish_tile = [&](bool whole, float *park) {
        sum_rows();
#pragma unroll
        for (int nr = 0; nr < NR; ++nr)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float v[2 * KS];
#pragma unroll
                for (int k = 0; k < KS; ++k) v[2 * k] = o[nr][k][e], v[2 * k + 1] = o[nr][k][2 + e];
                const int row = row_of(nr, e);
                if (whole) {
                    long long at;
                    if (place(row, at)) store_row(at, g * 2 * KS, v, 2 * KS, sum[nr][e], ref[nr][e]);
                } else {
#pragma unroll
                    for (int k = 0; k < KS; k += 2)
                        *reinterpret_cast<float4 *>(park + row * D + g * 2 * KS + 2 * k) =
                            make_float4(v[2 * k], v[2 * k + 1], v[2 * k + 2], v[2 * k + 3]);
                    if (g == 0) {
                        park[ROWS * D + 2 * row] = ref[nr][e];
                        park[ROWS * D + 2 * row + 1] = sum[nr][e];
                    }
                }
            }
    };
    float *first_part = reinterpret_cast<float *>(smem + L::kPark) + warp * L::kPart;
    float *last_part = reinterpret_cast<float *>(smem + warp * NS * L::kStage);

    // ---- steps
    // K rows as A: row g is key tau(g), row g + 8 key 8 + tau(g), an order in which eight lanes' 16-byte
    // chunks hit eight different bank groups of the swizzled tile.  P^T then has keys (tau(2t), tau(2t + 1))
    // and those plus 8 in a lane; V's chunk g of the same four keys is read in an order (`flip`) that
    // avoids conflicts, and the byte permutes undo it.
    const int tau = D == 128 ? (g >> 1 | (g & 1) << 2) : g;
    const int v_key0 = D == 128 ? t : 2 * t, v_key1 = D == 128 ? t + 4 : 2 * t + 1;
    const int flip = D == 128 ? g & 1 : (g >> 1) & 1;
    const uint32_t sel_lo = flip ? 0x1504 : 0x5140, sel_hi = flip ? 0x3726 : 0x7362;
    bool failed = false;
    int phase = 0, stage = 0;
    for (int at = w0; at < w1; ++at) {
        const int l = (at - w0) & 31;
        if (l == 0 && at != w0) {
            cur = nxt;
            nxt = look_up(at + 32 + lane);
        }
        const int m_tile = __shfl_sync(0xffffffffu, cur.tile, l);
        const int pos = __shfl_sync(0xffffffffu, cur.pos, l);
        const float ks = __shfl_sync(0xffffffffu, cur.ks, l);
        const float lv = __shfl_sync(0xffffffffu, cur.lv, l);
        const float iv = __shfl_sync(0xffffffffu, cur.iv, l);
        if (at == w0 || m_tile != tile) {
            if (at != w0) finish_tile(tile >= w0, first_part);
            start_tile(at);
            tile = m_tile;
        }
        if (!mbar_wait_bounded(bars + stage * 8, phase, p.status, &s_abort)) {
            failed = true;
            break;
        }
        const uint32_t kb = ring + stage * L::kStage, vb = kb + kStep * D;
        float s[NR][4];
#pragma unroll
        for (int nr = 0; nr < NR; ++nr)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[nr][i] = 0.0f;
#pragma unroll
        for (int j = 0; j < KS / 4; ++j) {
            const int chunk = t + 4 * j;
            const int sw = D == 128 ? chunk ^ (tau & 7) : chunk ^ ((tau >> 1) & 3);
            const uint4 a = lds128(kb + tau * D + sw * 16), b = lds128(kb + (tau + 8) * D + sw * 16);
            const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                uint32_t a0, a1, a2, a3;
                codes_to_half<KT>(aw[w], a0, a2);
                codes_to_half<KT>(bw[w], a1, a3);
#pragma unroll
                for (int nr = 0; nr < NR; ++nr)
                    mma16816<0>(s[nr], a0, a1, a2, a3, q[nr][4 * j + w][0], q[nr][4 * j + w][1]);
            }
        }
        // x_j + log2(vs); keys a row does not see get -inf
        const bool edge = pos + kStep - 1 > min_pos ||
                          (p.a.window > 0 && pos <= max_pos - p.a.window && pos + kStep > p.a.sinks);
        bool over = false;
#pragma unroll
        for (int nr = 0; nr < NR; ++nr)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int e = i & 1;
                s[nr][i] = fmaf(s[nr][i], fac[nr][e] * ks, lv);
                if (edge) {
                    const int j = pos + tau + 8 * (i >> 1), r = row_pos[nr][e];
                    const bool see = j <= r && (p.a.window == 0 || r - j < p.a.window || j < p.a.sinks);
                    if (!see) s[nr][i] = -INFINITY;
                }
                over |= s[nr][i] - ref[nr][e] > kTop;
            }
        if (__any_sync(0xffffffffu, over)) {
#pragma unroll
            for (int nr = 0; nr < NR; ++nr)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float top = fmaxf(s[nr][e], s[nr][2 + e]);
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
                    if (top - ref[nr][e] > kHead) {
                        const float f = ex2(ref[nr][e] - (top - kHead));
                        ref[nr][e] = top - kHead;
                        sum[nr][e] *= f;
#pragma unroll
                        for (int k = 0; k < KS; ++k) o[nr][k][e] *= f, o[nr][k][2 + e] *= f;
                    }
                }
        }
        uint32_t pt[NR][2];
#pragma unroll
        for (int nr = 0; nr < NR; ++nr) {
            float w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = ex2(s[nr][i] - ref[nr][i & 1]);
            sum[nr][0] = fmaf(w[0] + w[2], iv, sum[nr][0]);
            sum[nr][1] = fmaf(w[1] + w[3], iv, sum[nr][1]);
            pt[nr][0] = movmatrix(pack_half2(w[0], w[1]));
            pt[nr][1] = movmatrix(pack_half2(w[2], w[3]));
        }
        // V^T as A: byte i of a lane's chunk g is dim g * D / 8 + i
        uint32_t vw[4][D / 32];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int key = ((r & 1) != flip ? v_key1 : v_key0) + 8 * (r >> 1);
            if (D == 128) {
                const uint4 v = lds128(vb + key * D + (g ^ (key & 7)) * 16);
                vw[r][0] = v.x, vw[r][1] = v.y, vw[r][D / 32 - 2] = v.z, vw[r][D / 32 - 1] = v.w;
            } else {
                const uint2 v = lds64(vb + key * D + ((g >> 1) ^ ((key >> 1) & 3)) * 16 + (g & 1) * 8);
                vw[r][0] = v.x, vw[r][1] = v.y;
            }
        }
        if (edge && KT == kKvE4m3) {
            // bytes of keys no row sees may be NaN codes; their weight of 0 would not hide them
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int j = pos + ((r & 1) != flip ? v_key1 : v_key0) + 8 * (r >> 1);
                if (j > max_pos)
#pragma unroll
                    for (int w = 0; w < D / 32; ++w) vw[r][w] = 0;
            }
        }
#pragma unroll
        for (int w = 0; w < D / 32; ++w) {
            uint32_t a[4][2];                                      // [dim of the word][keys 0/1 or 8/9]
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t x = vw[2 * h][w], y = vw[2 * h + 1][w];
                codes_to_half<KT>(__byte_perm(x, y, sel_lo), a[0][h], a[1][h]);
                codes_to_half<KT>(__byte_perm(x, y, sel_hi), a[2][h], a[3][h]);
            }
#pragma unroll
            for (int nr = 0; nr < NR; ++nr) {
                mma16816<0>(o[nr][2 * w], a[0][0], a[1][0], a[0][1], a[1][1], pt[nr][0], pt[nr][1]);
                mma16816<0>(o[nr][2 * w + 1], a[2][0], a[3][0], a[2][1], a[3][1], pt[nr][0], pt[nr][1]);
            }
        }
        __syncwarp();
        if (fetched < w1) {
            const int f = (fetched - w0) & 31;
            const bool ahead = ((fetched - w0) ^ (at - w0)) >= 32;
            const int page = __shfl_sync(0xffffffffu, ahead ? nxt.page : cur.page, f);
            const int where = __shfl_sync(0xffffffffu, ahead ? nxt.where : cur.where, f);
            if (lane == 0) fence_proxy_async_smem();
            issue(stage, page, where);
            ++fetched;
        }
        if (++stage == NS) stage = 0, phase ^= 1;
    }
    if (failed) {
        // leave with no copy in flight
        for (int at = fetched - w0 - NS; at < fetched - w0; ++at)
            if (at >= 0) mbar_wait_bounded(bars + at % NS * 8, (at / NS) & 1, p.status, &s_abort);
    }
    // the piece still held: whole when its tile begins here and ends here
    if (w0 < w1 && !failed) {
        const long long line = c0 + w1;
        const int b = find(line - 1);
        const int4 s = seqs[b];
        const int steps = span_of(s.y, s.z, p.a.window, p.a.sinks).steps;
        const bool ends = (line - pre[b]) % steps == 0;
        if (tile >= w0 && ends) {
            finish_tile(true, nullptr);
        } else if (tile < w0) {
            finish_tile(false, first_part);                        // began before this warp: ends or goes on
        } else {
            __syncwarp();
            finish_tile(false, last_part);                         // begins here, goes on
        }
    }
    __syncthreads();
    if (s_abort) return;

    // ---- tiles that more than one warp holds a part of
    // The CTA's tiles in order: one that began earlier (or at c0), then each that a warp begins and does
    // not end.  All threads sum the parts of one tile, in warp order.
    for (int w = 0; w < NW; ++w) {
        // a tile whose first part in this CTA is warp w's
        const int a0 = (int)((long long)mine * w / NW), a1 = (int)((long long)mine * (w + 1) / NW);
        if (a0 >= a1) continue;
        for (int which = 0; which < 2; ++which) {
            // which = 0: the tile at the CTA's first step, if it began in an earlier CTA; 1: the tile at the
            // warp's last step, if it begins in this warp and goes on after it
            if (which == 0 && a0 != 0) continue;
            const int probe = which == 0 ? 0 : a1 - 1;
            const int b = find(c0 + probe);
            const int4 s = seqs[b];
            const int steps = span_of(s.y, s.z, p.a.window, p.a.sinks).steps;
            const long long begin = c0 + probe - (c0 + probe - pre[b]) % steps, end = begin + steps;
            if (which == 0 ? begin >= c0 : (begin < c0 + a0 || end <= c0 + a1)) continue;
            // its parts: warp w's, then the first parts of the warps after it up to the tile's end
            tile_q0 = s.x, tile_n = s.y;
            const int idx = (int)((begin - pre[b]) / steps);
            tile_head = idx / s.w, tile_row = idx % s.w * ROWS;
            const bool whole = begin >= c0 && end <= c1;
            const int slot = which == 0 ? 0 : 1;
            float *dst = p.parts + ((long long)blockIdx.x * 2 + slot) * L::kPart;
            const int rows = min(ROWS, s.y * group - tile_row);
            for (int i = tid; i < rows * (D / 4); i += 32 * NW) {
                const int row = i / (D / 4), d = i % (D / 4) * 4;
                float m = kRefStart;
                for (int v = w; v < NW; ++v) {
                    const long long v0 = c0 + (long long)mine * v / NW;
                    const long long v1 = c0 + (long long)mine * (v + 1) / NW;
                    if (v0 >= v1) continue;
                    if (v0 >= end) break;
                    const float *part = v == w && which == 1
                                            ? reinterpret_cast<const float *>(smem + v * NS * L::kStage)
                                            : reinterpret_cast<const float *>(smem + L::kPark) + v * L::kPart;
                    m = fmaxf(m, part[ROWS * D + 2 * row]);
                }
                float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f}, l = 0.0f;
                for (int v = w; v < NW; ++v) {
                    const long long v0 = c0 + (long long)mine * v / NW;
                    const long long v1 = c0 + (long long)mine * (v + 1) / NW;
                    if (v0 >= v1) continue;
                    if (v0 >= end) break;
                    const float *part = v == w && which == 1
                                            ? reinterpret_cast<const float *>(smem + v * NS * L::kStage)
                                            : reinterpret_cast<const float *>(smem + L::kPark) + v * L::kPart;
                    const float f = ex2(part[ROWS * D + 2 * row] - m);
                    const float4 x = *reinterpret_cast<const float4 *>(part + row * D + d);
                    l = fmaf(part[ROWS * D + 2 * row + 1], f, l);
                    acc[0] = fmaf(x.x, f, acc[0]), acc[1] = fmaf(x.y, f, acc[1]);
                    acc[2] = fmaf(x.z, f, acc[2]), acc[3] = fmaf(x.w, f, acc[3]);
                }
                if (whole) {
                    long long at;
                    if (place(row, at)) store_row(at, d, acc, 4, l, m);
                } else {
                    *reinterpret_cast<float4 *>(dst + row * D + d) = make_float4(acc[0], acc[1], acc[2], acc[3]);
                    if (d == 0) dst[ROWS * D + 2 * row] = m, dst[ROWS * D + 2 * row + 1] = l;
                }
            }
            if (whole) continue;
            // ---- a tile that CTAs from..to share: the last of them to come sums it
            const int from = (int)(((begin + 1) * ctas + total - 1) / total - 1);
            const int to = (int)((end * ctas + total - 1) / total - 1);
            __threadfence();
            __syncthreads();
            if (tid == 0) {
                unsigned long long *tk = p.tickets + from, old = *tk, seen;
                unsigned long long put;
                do {
                    seen = old;
                    const unsigned long long n = (seen >> 16) == p.tag ? (seen & 0xffff) + 1 : 1;
                    put = n == (unsigned long long)(to - from + 1) ? 0 : p.tag << 16 | n;
                    old = atomicCAS(tk, seen, put);
                } while (old != seen);
                __threadfence();
                s_last = put == 0;
            }
            __syncthreads();
            if (!s_last) continue;
            for (int i = tid; i < rows * (D / 4); i += 32 * NW) {
                const int row = i / (D / 4), d = i % (D / 4) * 4;
                float m = kRefStart;
                // CTA `from` holds its part in slot 1, the others in slot 0
                for (int c = from; c <= to; ++c)
                    m = fmaxf(m, __ldcg(p.parts + ((long long)c * 2 + (c == from)) * L::kPart + ROWS * D + 2 * row));
                float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f}, l = 0.0f;
#pragma unroll 4
                for (int c = from; c <= to; ++c) {
                    const float *part = p.parts + ((long long)c * 2 + (c == from)) * L::kPart;
                    const float f = ex2(__ldcg(part + ROWS * D + 2 * row) - m);
                    const float4 x = __ldcg(reinterpret_cast<const float4 *>(part + row * D + d));
                    l = fmaf(__ldcg(part + ROWS * D + 2 * row + 1), f, l);
                    acc[0] = fmaf(x.x, f, acc[0]), acc[1] = fmaf(x.y, f, acc[1]);
                    acc[2] = fmaf(x.z, f, acc[2]), acc[3] = fmaf(x.w, f, acc[3]);
                }
                long long at;
                if (place(row, at)) store_row(at, d, acc, 4, l, m);
            }
        }
    }
}

using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                   const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// A map of codes whose boxes are `keys` tokens of one head of one page.  The
// middle dimensions go by rising stride.
cudaError_t encode_codes(const DeviceInfo &dev, const KvCache &c, void *base, int keys, bool token_first,
                         CUtensorMap *out) {
    if (dev.encode_tiled == nullptr) return cudaErrorNotSupported;
    const cuuint64_t tokens = (cuuint64_t)1 << c.page_shift, heads = (cuuint64_t)c.n_kv_heads;
    // a dimension of one element has no stride of its own
    const cuuint64_t sh = c.n_kv_heads > 1 ? (cuuint64_t)c.head_stride : (cuuint64_t)c.token_stride << c.page_shift;
    const cuuint64_t sp = c.n_pages > 1 ? (cuuint64_t)c.page_stride : (cuuint64_t)c.token_stride << c.page_shift;
    cuuint64_t dims[4] = {(cuuint64_t)c.head_dim, tokens, heads, (cuuint64_t)c.n_pages};
    cuuint64_t strides[3] = {(cuuint64_t)c.token_stride, sh, sp};
    cuuint32_t box[4] = {(cuuint32_t)c.head_dim, (cuuint32_t)keys, 1, 1};
    const cuuint32_t one[4] = {1, 1, 1, 1};
    if (token_first) {
        std::swap(dims[1], dims[2]);
        std::swap(strides[0], strides[1]);
        std::swap(box[1], box[2]);
    }
    const CUresult r = reinterpret_cast<EncodeTiledFn>(dev.encode_tiled)(
        out, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, base, dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
        c.head_dim == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int KT, int D, int NR, int NW, int NS>
cudaError_t launch_few(const FewParams &p, const CUtensorMap &k, const CUtensorMap &v, int grid, cudaStream_t s,
                       bool pdl) {
    using L = FewSmem<D, NR, NW, NS>;
    auto kern = few_rows_kernel<KT, D, NR, NW, NS>;
    const cudaError_t e = raise_smem_cap(reinterpret_cast<const void *>(kern), L::kEnd);
    if (e != cudaSuccess) return e;
    return kv_launch(kern, dim3(grid), dim3(32 * NW), L::kEnd, s, pdl, k, v, p);
}

constexpr int kMostRows = 16;

}  // namespace

cudaError_t launch_kv_attention(const KvAttentionArgs &a, const KvCache &c, const KvBatch &batch, const DeviceInfo &dev,
                                cudaStream_t s, bool pdl) {
    const int group = a.n_heads / c.n_kv_heads;
    const bool token_first = c.n_kv_heads > 1 && c.head_stride < c.token_stride;
    CUtensorMap k, v;
    cudaError_t e = encode_codes(dev, c, c.k, kStep, token_first, &k);
    if (e == cudaSuccess) e = encode_codes(dev, c, c.v, kStep, token_first, &v);
    if (e != cudaSuccess) return e;
    static std::atomic<unsigned long long> launches{0x5ca1ab1e0000ull};
    for (int b0 = 0; b0 < batch.n_seqs; b0 += kMaxSeqs) {
        KvBatch b = batch;
        b.block_table += (long long)b0 * b.max_blocks;
        b.kv_lens += b0;
        b.q_starts += b0;
        b.n_seqs = std::min(kMaxSeqs, batch.n_seqs - b0);
        FewParams p{a, c, b, 0, token_first ? 1 : 0, nullptr, nullptr, 0, dev.status};
        p.tickets = static_cast<unsigned long long *>(a.workspace);
        p.parts = reinterpret_cast<float *>(p.tickets + ((dev.sm_count + 1) & ~1));
        p.tag = (launches.fetch_add(1) * 0x9e3779b97f4a7c15ull) >> 16;
        if (p.tag == 0) p.tag = 1;
        const int grid = dev.sm_count;
        const bool few = (long long)a.max_q_len * group <= 8;
#define W4A16_FEW(KT)                                                                          \
    e = c.head_dim == 128 ? (few ? launch_few<KT, 128, 1, 8, 5>(p, k, v, grid, s, pdl)         \
                                 : launch_few<KT, 128, 2, 8, 4>(p, k, v, grid, s, pdl))        \
                          : (few ? launch_few<KT, 64, 1, 8, 10>(p, k, v, grid, s, pdl)         \
                                 : launch_few<KT, 64, 2, 8, 8>(p, k, v, grid, s, pdl))
        if (c.kv_dtype == kKvInt8) W4A16_FEW(kKvInt8);
        else W4A16_FEW(kKvE4m3);
#undef W4A16_FEW
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

long long kv_attention_workspace(int, int, int head_dim, int, int, const DeviceInfo &dev) {
    return (long long)((dev.sm_count + 1) & ~1) * 8 + (long long)dev.sm_count * 2 * kMostRows * (head_dim + 2) * 4;
}

}  // namespace w4a16
