// kv_few_rows.cuh -- attention of few query rows over the paged 8-bit cache:
// the kernel of kv_attention.cu and kv_attention_shared.cu.
//
// For one kv head, with codes k_j, v_j of key j, page scales ks, vs and a
// query row q (a token and query head of the group),
//     x_j = scale log2(e) ks (q . k_j),     out = sum_j 2^x_j vs v_j / sum_j 2^x_j.
// The values' scale goes into the exponent: with e_j = x_j + log2(vs) - M the
// weights 2^e_j multiply the codes as they are, and the denominator gets
// 2^e_j / vs.  M is a running reference of each row, moved only when some e_j
// passes 15.9, and then so that the largest is at 2^14: the weights fit fp16,
// good to 2^-11 down to 2^-28 of the row's largest, to ever fewer bits below
// that, and zero below 2^-39; the sums (out, the denominator) are fp32.
//
// Fewer bits than 32, and why.  The weights are fp16 because the matrix
// instructions take 16-bit operands, and fp16 has three bits more than bf16;
// two halves of each weight would double the products and the registers.  It
// costs fp16 outputs 2.6e-4 to 2.8e-4 of relative error, where 32-bit weights
// rounded once give 2.1e-4; bf16 outputs have 1.7e-3 either way.  Queries in
// bf16 become fp16 after a power of two has put a row's largest value at 2^14,
// so that one conversion of the codes, to fp16, serves both types: exact down
// to 2^-28 of that value, and what is below is that much smaller than the
// scores' fp32 sums resolve.  ex2.approx and the reciprocals are good to 2^-22,
// far below a weight's 2^-11.
//
// Bound by the cache read (256 bytes a key and kv head at 128 dims) when pages
// are large, by the conversion of the codes when they hold 16 keys.  So the
// design is about bytes in flight, even shares and few instructions a key:
//  * The work is a line of steps of 16 to 64 keys: sequence by sequence, kv head
//    by kv head, row tile by row tile, every step of the keys that the
//    sequence's new tokens see.  Lengths are read here, so each CTA sums the
//    line's length up itself, takes an equal piece of it, and its warps take
//    equal pieces of that.  A tile counts for 32 keys more, its start and end.
//    Ragged lengths, windows and few long sequences all spread over the whole
//    GPU alike.
//  * A warp is on its own: it owns a ring of stages, its first lane issues a
//    TMA box (16 or 32 keys of K and of V, one page) into each, all lanes
//    consume.  No barrier among warps until their pieces end.  Page ids and
//    scales of 32 steps are looked up at once, one step a lane.
//  * mma.sync m16n8k16 with the keys as A (16 keys x 16 dims) and the rows as
//    B (8 rows): S^T = K Q^T, then P^T through two movmatrix transposes, then
//    out^T = V^T P^T.  The dims and keys are permuted so that every operand
//    comes from wide conflict-free shared loads (128- or 64-byte swizzled by
//    the TMA): a lane's 16 bytes of K are four k-steps of A.  A tile has 8 or
//    16 rows: a 128-row tcgen05 tile would be nearly empty.
//  * A tile that several warps share is summed through shared memory, one
//    that several CTAs share through the workspace, the CTA that comes last
//    summing all parts in order: the result does not depend on who that is.
//    Tickets carry the launch's number, so scratch needs no initialisation.
//
// Measured (32 query heads on 8 kv heads, 128 dims): 4 sequences of 98302 to
// 131071 keys, e4m3, pages of 64: 154 us for 1.0 GB, 6.5 TB/s, 0.96 of a copy's
// bandwidth (tokens before heads: 159 us).  64 sequences of 4 to 4096 keys,
// int8, pages of 16: 57 us for 273 MB, 4.8 TB/s (5.6 between the first key and
// the last); the arithmetic pipes are 39 % busy and 1.7 instructions a cycle go
// out, about 390 for 16 keys, most of them conversions; about 4 us go by before
// the first key and 6 after the last.  One sequence of 77 keys: 8.5 us, a chain
// of dependent loads.
#pragma once
#include <cuda.h>

#include <algorithm>
#include <atomic>

#include "kv.cuh"
#include "skinny.cuh"

namespace w4a16 {
namespace {

constexpr int kMaxSeqs = 512;             // sequences of a launch
constexpr int kMaxEntries = 640;          // entries of one (SHARED): 512 sequences and their groups
// Tiles of up to so many keys stay in one CTA.  256 / never / 1024, us, contexts of 100 to 300 keys: 256 sequences 32.7 /
// 33.4 / 31.4, 64 16.1 / 16.1 / 15.2, 8 12.2 / 11.7 / 11.6; 64 of 500 to 1000 28.5 / 28.4 / 30.5, one of 1000 14.4 / 14.4 /
// 16.0: 1024 takes too long where there are few tiles, never costs some where there are many.
constexpr int kShort = 256;
constexpr int kLeast = 2;                 // fewest steps worth a CTA
constexpr int kFewSeqs = 16;              // so many sequences may have their tiles cut alike ...
constexpr int kManyHeads = 8;             // ... of so many kv heads
constexpr int kTileCost = 32;             // keys that the start and end of a tile count for in the shares
constexpr int kFlagShift = 26;            // SHARED: an entry's flags above its first row, 2^24 at most
constexpr float kRefStart = -3.402823466e38f;
constexpr float kTop = 15.9f;             // weights stay below 2^kTop, inside fp16 ...
constexpr float kHead = 14.0f;            // ... and a moved reference puts the largest at 2^kHead

struct FewParams {
    KvAttentionArgs a;
    KvCache c;
    KvBatch b;
    int row_limit;                        // sequences with more rows a kv head than this are another kernel's (0: none)
    int token_first;                      // tensor map dims are (dim, head, token, page, K or V), not (dim, token, head, ...)
    int merged;                           // one box brings K and V; else the second map brings V
    int before, after;                    // rows before the first sequence's, after the last one's are this launch's
    int k_at, v_at;                       // where a stage holds K and V, in tiles
    float *parts;                         // [grid][2][ROWS][D + 2]
    unsigned long long *tickets;          // [grid]
    unsigned long long tag;
    int hold;                             // test hook (kv_holds)
    int *status;
    KvShare share;                        // of a call with SHARED: what its sequences are (kv_attention_shared.cu)
};

// Blocks of KB keys that new tokens of a sequence see: [0, sink) and
// [first, ...), `blocks` in all, one at least; BPS of them are a step.
struct Span {
    int blocks, sink, first, steps;
};
template <int KB, int BPS>
__device__ __forceinline__ Span span_of(int n, int len, int window, int sinks) {
    Span s;
    const int lo = window > 0 ? max(0, len - n + 1 - window) : 0;
    s.first = lo / KB;
    s.sink = min((min(sinks, lo) + KB - 1) / KB, s.first);
    s.blocks = max(s.sink + (len + KB - 1) / KB - s.first, 1);
    s.steps = (s.blocks + BPS - 1) / BPS;
    return s;
}

// a / b for a of a line's length: nearly always within 32 bits, where division is cheap
__device__ __forceinline__ int line_div(long long a, int b) {
    return a >> 32 ? (int)(a / b) : (int)((uint32_t)a / (uint32_t)b);
}

// A tile of which warps hold parts: steps [begin, end) of the CTA's line, and its rows.
struct Shared {
    int has, first_warp, begin, end, q0, n, head, row;
};

template <int D, int NR, int KB, int NW, int NS>
struct FewSmem {
    static constexpr int kRows = 8 * NR;
    static constexpr int kStage = 2 * KB * D;                      // K and V of a block
    static constexpr int kPart = kRows * (D + 2);                  // floats: rows of out, then (M, l) of each row
    static constexpr int kPark = NW * NS * kStage;                 // a warp's first piece, if another began it
    static constexpr int kSeq = kPark + NW * kPart * 4;            // int4 {q0, n, len, row tiles}
    static constexpr int kPre = kSeq + kMaxEntries * 16;              // line position of each sequence
    static constexpr int kTiles = kPre + kMaxEntries * 8;             // tiles of the sequences before each
    static constexpr int kBars = kTiles + kMaxEntries * 4;
    static constexpr int kShared = kBars + NW * NS * 8;            // tiles that warps share: the CTA's first, then by warp
    static constexpr int kMisc = kShared + (NW + 1) * 32;
    static constexpr int kEnd = kMisc + (2 * NW + 1) * 8 + 32 + (NW + 2) * 4 + 1024;       // 1024: slack to align the base
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
__device__ __forceinline__ uint32_t pack_bf162(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
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

// What a block needs, held by the lane that looked it up.
struct Meta {
    int page, where;       // page or -1; first token within the page | kv head << 8
    int pos;               // position of the first key (past every query for a block that is not there)
    float ks, vs;          // scales
};

template <bool SHARED, int KT, int D, int NR, int KB, int BPS, int NW, int NS>
__global__ void __launch_bounds__(32 * NW, 1)
    few_rows_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                    const FewParams p) {
    using L = FewSmem<D, NR, KB, NW, NS>;
    constexpr int SUB = KB / 16;                                   // 16-key tiles of a block
    constexpr int ROWS = L::kRows;
    constexpr int KS = D / 16;                                     // k-steps of S, and 16-dim tiles of out
    constexpr int LOOK = 32 / BPS;                                 // steps looked up at once, a block a lane
    extern __shared__ uint8_t smem_raw[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);    // swizzled tiles need it
    // no static shared memory: the launch may ask for all of an SM's
    long long *s_scan = reinterpret_cast<long long *>(smem + L::kMisc), *s_cut = s_scan + NW;
    int &s_abort = *reinterpret_cast<int *>(s_cut + NW + 1);
    int *s_out = &s_abort + 1, *s_from = s_out + 2, *s_to = s_from + 2;      // tiles shared with other CTAs
    int &s_alike = s_to[2], *s_seq = s_to + 3;
    int4 *seqs = reinterpret_cast<int4 *>(smem + L::kSeq);
    long long *pre = reinterpret_cast<long long *>(smem + L::kPre);
    int *tiles_before = reinterpret_cast<int *>(smem + L::kTiles);
    Shared *shared = reinterpret_cast<Shared *>(smem + L::kShared);
    const uint32_t ring = smem_u32(smem) + warp * NS * L::kStage;
    const uint32_t bars = smem_u32(smem + L::kBars) + warp * NS * 8;
    const int Hk = p.c.n_kv_heads, group = p.a.n_heads / Hk, B = p.b.n_seqs;

    if (tid == 0) {
        s_abort = 0;
        s_out[0] = s_out[1] = -1;
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
    }
    if (lane < NS) mbar_init(bars + lane * 8, 1);
    if (tid <= NW) shared[tid].has = 0;
    fence_mbar_init();
    // Beside the kernel before it, which waited for the plan before it let this one start: its end is waited for at this
    // one's, by all CTAs, so that whoever waits for this kernel has both.
    const bool beside = SHARED && p.share.beside;
    if (!beside) kv_begin();
    else __threadfence();                                          // the plan's entries, not what a call before left in L1
    auto leave = [&]() {
        if (beside) grid_dependency_wait();
    };

    // ---- the line: each sequence's steps and tiles, summed up
    constexpr int COST = (kTileCost + KB * BPS - 1) / (KB * BPS);
    auto span = [&](int n, int len) { return span_of<KB, BPS>(n, len, p.a.window, p.a.sinks); };
    long long total = 0;                                           // steps, and COST a tile
    int tiles_all = 0;
    for (int base = 0; base < B; base += 32 * NW) {
        const int i = base + tid;
        long long v = 0;
        int tiles = 0;
        if (i < B) {
            KvSeq s;
            int flags = 0;                                         // above the bits of a row
            if constexpr (SHARED) {
                const KvEntry e = kv_entry(p.share, i);
                s = KvSeq{e.q0, (e.flags & kKvBig) && kv_division(p.share, 0) ? 0 : e.n, e.len};
                flags = e.flags << kFlagShift;
            } else {
                s = kv_sequence(p.b, p.c.page_shift, i, p.status);
            }
            const int rows = s.n * group;
            const int row_tiles = p.row_limit > 0 && rows > p.row_limit ? 0 : (rows + ROWS - 1) / ROWS;
            seqs[i] = make_int4(s.q0 | flags, s.n, s.len, row_tiles);
            tiles = row_tiles * Hk;
            v = (long long)tiles * (span(s.n, s.len).steps + COST);
        }
        long long inc = v;
        int inc_tiles = tiles;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const long long x = __shfl_up_sync(0xffffffffu, inc, d);
            const int y = __shfl_up_sync(0xffffffffu, inc_tiles, d);
            if (lane >= d) inc += x, inc_tiles += y;
        }
        __syncthreads();
        if (lane == 31) s_scan[warp] = inc, s_cut[warp] = inc_tiles;
        __syncthreads();
        long long ahead = total;
        int tiles_ahead = tiles_all;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            const long long x = s_scan[w];
            const int y = (int)s_cut[w];
            ahead += w < warp ? x : 0;
            tiles_ahead += w < warp ? y : 0;
            total += x;
            tiles_all += y;
        }
        if (i < B) {
            tiles_before[i] = tiles_ahead + inc_tiles - tiles;
            pre[i] = ahead + inc - v - (long long)tiles_before[i] * COST;
        }
    }
    __syncthreads();
    kv_empty_rows(p.a, p.b, D, p.before ? seqs[0].x : 0, p.after ? seqs[B - 1].x + seqs[B - 1].y : p.b.n_tokens);
    if (total == 0) {
        leave();
        return;
    }

    // the sequence, one of lo..hi, of a position of the line: of steps alone (cost = 0), or with the tiles' cost
    auto find = [&](long long at, int cost, int lo, int hi) {
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (pre[mid] + (long long)tiles_before[mid] * cost <= at) lo = mid;
            else hi = mid - 1;
        }
        return lo;
    };
    const int grid = SHARED ? kv_division(p.share, 2) : gridDim.x;
    const long long ctas = min((long long)grid, (total + kLeast + COST - 1) / (kLeast + COST));
    if (blockIdx.x >= ctas) {
        leave();
        return;
    }
    // The step where an equal share of the work begins: `at` steps and tiles' costs into the line.  In a
    // short tile, when `snap`, the tile's first; *moved is where that is with the costs.
    auto step_of = [&](long long at, bool snap, long long &moved, int lo, int hi, int &b) {
        moved = at;
        b = find(at, COST, lo, hi);
        const int4 s = seqs[b];
        const Span sp = span(s.y, s.z);
        const int steps = sp.steps;
        const long long rem = at - pre[b] - (long long)tiles_before[b] * COST;
        const int idx = line_div(rem, steps + COST);
        int st = (int)(rem - (long long)idx * (steps + COST));
        if (snap && sp.blocks <= kShort / KB) {
            moved -= st;
            st = 0;
        }
        // past the last tile of a sequence that has any, the next one's first step
        return pre[b] + (long long)idx * steps + min(max(st - COST, 0), steps);
    };
    // Where a page's tokens hold all heads side by side, warps that go through the same keys of different heads
    // should do so at the same time, or every stretch of some heads' rows is fetched in pieces.  So with few long
    // tiles of many heads those of one sequence get the same whole number of warps' pieces, as near to equal shares as
    // that allows.  4 sequences of 98302 to 131071 keys, this / equal shares, us on two GPUs of this kind: 8 heads of
    // 128 dims 155 / 159 and 159 / 177, 8 of 64 86 / 137 and 86 / 141, 16 of 64 160 / 304 and 164 / 334.  With fewer
    // heads the whole pieces cost more than they save: 4 heads of 128 86 / 84, 2 heads 57 / 54, 9 sequences of 2 heads
    // 57 / 51 on any GPU.
    const int pieces = (int)ctas * NW;
    auto pieces_of = [&](int b, int done, long long each) {        // a tile's, of sequence b, `done` pieces before it
        const int tiles = max(seqs[b].w * Hk, 1);
        const long long end = pre[b] + (long long)tiles_before[b] * COST + seqs[b].w * Hk * each;
        return (int)min((end * pieces / total - done + tiles / 2) / tiles, (long long)(pieces - done) / tiles);
    };
    const bool alike = p.token_first && Hk >= kManyHeads && B <= kFewSeqs && tiles_all * 16 <= pieces;
    if (alike && warp == 0) {
        const int i = blockIdx.x * NW + min(lane, NW);
        long long at = total - (long long)tiles_all * COST;        // the line's end
        bool fits = true;
        int done = 0, of = B - 1;
        for (int b = 0; b < B; ++b) {
            const int tiles = seqs[b].w * Hk, steps = span(seqs[b].y, seqs[b].z).steps, each = steps + COST;
            if (tiles == 0) continue;
            const int n = pieces_of(b, done, each);
            // pieces of some length, and hardly longer than an equal share
            fits = fits && n >= 8 && each >= n * (4 + COST) && (long long)each * pieces * 25 <= n * total * 26;
            if (!fits) break;
            if (i >= done && i < done + tiles * n) {
                const int tile = (i - done) / n, k = (i - done) % n;
                at = pre[b] + (long long)tile * steps + max((int)((long long)each * k / n) - COST, 0);
                of = b;
            }
            done += tiles * n;
        }
        if (lane <= NW) s_cut[lane] = at, s_seq[lane] = of;
        if (lane == 0) s_alike = fits;
    }
    if (alike) __syncthreads();
    const bool by_tile = alike && s_alike;
    if (!by_tile && warp == 0) {
        long long v = ((long long)blockIdx.x + min(lane, 1)) * total / ctas, moved;
        int of;
        const long long end = step_of(v, true, moved, 0, B - 1, of);
        const int of0 = __shfl_sync(0xffffffffu, of, 0), of1 = __shfl_sync(0xffffffffu, of, 1);
        const long long v0 = __shfl_sync(0xffffffffu, moved, 0), v1 = __shfl_sync(0xffffffffu, moved, 1);
        const long long c0 = __shfl_sync(0xffffffffu, end, 0), c1 = __shfl_sync(0xffffffffu, end, 1);
        if (lane <= NW) {
            const long long mid = step_of(v0 + (v1 - v0) * lane / NW, false, moved, of0, of1, of);
            s_cut[lane] = lane == 0 ? c0 : lane == NW ? c1 : min(max(mid, c0), c1);
            s_seq[lane] = of;                                      // what is in a warp's piece is of s_seq[warp]..s_seq[warp + 1]
        }
    }
    __syncthreads();
    const long long c0 = s_cut[0];
    const int mine = (int)(s_cut[NW] - c0);
    if (mine <= 0) {
        leave();
        return;
    }
    auto warp_start = [&](int w) { return (int)(s_cut[w] - c0); };
    const int w0 = warp_start(warp), w1 = warp_start(warp + 1), seq_lo = s_seq[warp], seq_hi = s_seq[warp + 1];

    // ---- blocks looked up a lane each, those of LOOK steps: first the page id, then, once it is here, the scales
    auto look_up = [&](int at) {
        Meta m;
        m.page = -1, m.where = 0, m.pos = 0x7fffff00, m.ks = 0.0f, m.vs = 1.0f;
        at += lane / BPS;
        if (at < w1) {
            const long long line = c0 + at;
            const int b = find(line, 0, seq_lo, seq_hi);
            const int4 s = seqs[b];
            const Span sp = span(s.y, s.z);
            const long long rem = line - pre[b];
            const int steps = sp.steps, tile = line_div(rem, steps);
            const int nth = (int)(rem - (long long)tile * steps) * BPS + lane % BPS;
            const int head = (int)((unsigned)tile / (unsigned)s.w);
            const int blk = nth < sp.sink ? nth : sp.first + nth - sp.sink;
            m.where = (blk * KB & ((1 << p.c.page_shift) - 1)) | head << 8;
            if (blk * KB < s.z) {
                m.pos = blk * KB;
                const long long row = SHARED ? kv_entry_pages(p.share, b) : (long long)b * p.b.max_blocks;
                m.page = p.b.block_table[row + (blk * KB >> p.c.page_shift)];
            }
        }
        return m;
    };
    auto look_up_scales = [&](Meta &m) {
        if (m.pos == 0x7fffff00) return;
        if (m.page < 0 || m.page >= p.c.n_pages) {
            kv_report(p.status);
            m.page = -1, m.pos = 0x7fffff00;
            return;
        }
        const long long i = (long long)m.page * Hk + (m.where >> 8);
        m.ks = __ldg(p.c.k_scale + i);
        m.vs = __ldg(p.c.v_scale + i);
    };
    const bool holds = kv_holds(p.hold);
    auto issue = [&](int stage, int page, int where) {
        if (lane == 0 && !holds) {
            const uint32_t bar = bars + stage * 8, dst = ring + stage * L::kStage;
            mbar_arrive_expect_tx(bar, L::kStage);
            const int tok = where & 255, head = where >> 8;
            const int x = p.token_first ? head : tok, y = p.token_first ? tok : head;
            tma_load_5d(dst, &tm_k, bar, 0, x, y, page, 0);
            if (!p.merged) tma_load_5d(dst + KB * D, &tm_v, bar, 0, x, y, page, 0);
        }
    };

    // ---- the running tile
    struct Tile {
        int begin, end;                                            // on the CTA's line
        int q0, n, row, head;                                      // the sequence's rows, the tile's first row, its kv head
        int first;                                                 // position of the sequence's first new token
    };
    // an entry's flags, and the position of a tile's tok-th token
    auto flags_of = [](int q0) { return SHARED ? q0 >> kFlagShift : kKvOthers; };
    auto position = [&](const Tile &tl, int tok) { return flags_of(tl.q0) & kKvOthers ? tl.first + tok : tl.first; };
    uint32_t q[NR][KS][2];
    float o[NR][KS][4], ref[NR][2], sum[NR][2], fac[NR][2];
    int row_pos[NR][2], min_pos = 0, max_pos = 0;                  // position of each row's token; -1: no such row
    Tile tile = {}, next = {};
    uint4 raw[NR][KS / 4][2];                                      // rows of a tile to come, before conversion

    auto row_of = [&](int nr, int e) { return nr * 8 + 2 * t + e; };
    auto divide = [](int x, int y) { return (int)((unsigned)x / (unsigned)y); };
    // token row and query head of a row of a tile; false past the last
    auto place = [&](const Tile &tl, int row, long long &at) {
        const int r = tl.row + row;
        if (r >= tl.n * group) return false;
        const int tok = divide(r, group);
        const int q0 = SHARED ? tl.q0 & (1 << kFlagShift) - 1 : tl.q0;
        at = (long long)(q0 + tok) * p.a.n_heads + tl.head * group + r - tok * group;
        return true;
    };
    auto load_rows = [&](int at) {
        Tile tl;
        const long long line = c0 + at;
        const int b = find(line, 0, seq_lo, seq_hi);
        const int4 s = seqs[b];
        const int steps = span(s.y, s.z).steps;
        const long long rem = line - pre[b];
        const int idx = line_div(rem, steps);
        tl.begin = at - (int)(rem - (long long)idx * steps);
        tl.end = tl.begin + steps;
        tl.head = divide(idx, s.w);
        tl.row = (idx - tl.head * s.w) * ROWS;
        tl.q0 = s.x, tl.n = s.y;
        tl.first = flags_of(s.x) & kKvOthers ? s.z - s.y : s.z - 1;
#pragma unroll
        for (int nr = 0; nr < NR; ++nr) {
            const int r = tl.row + nr * 8 + g, tok = divide(r, group);
            const bool has = r < s.y * group;
            const int q0 = SHARED ? s.x & (1 << kFlagShift) - 1 : s.x;
            const uint16_t *src = static_cast<const uint16_t *>(p.a.q) + (long long)(q0 + tok) * p.a.q_stride +
                                  (tl.head * group + r - tok * group) * D;
#pragma unroll
            for (int j = 0; j < KS / 4; ++j)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    raw[nr][j][i] = has ? ldg_nc_v4(src + (t + 4 * j) * 16 + 8 * i) : make_uint4(0, 0, 0, 0);
        }
        return tl;
    };
    auto start_tile = [&](const Tile &tl) {
        tile = tl;
        min_pos = position(tl, divide(tl.row, group));
        max_pos = position(tl, divide(min(tl.row + ROWS, tl.n * group) - 1, group));
#pragma unroll
        for (int nr = 0; nr < NR; ++nr) {
            // row g's dims as B: for a lane's chunk t (and t + 4), four words of four dims each
            float x[KS][4];
            float top = 0.0f;
#pragma unroll
            for (int j = 0; j < KS / 4; ++j) {
                const uint4 *v = raw[nr][j];
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
            // bf16 down to 2^-28 of that value (why fp16: the file's header)
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
                const int rr = tl.row + row_of(nr, e);
                row_pos[nr][e] = rr < tl.n * group ? position(tl, divide(rr, group)) : -1;
                ref[nr][e] = kRefStart;
                sum[nr][e] = 0.0f;
            }
#pragma unroll
            for (int k = 0; k < KS; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[nr][k][i] = 0.0f;
        }
    };
    auto store_row = [&](int q0, long long at, int d0, const float *v, int count, float l, float m) {
        if constexpr (SHARED) {
            kv_store_sums<D>(p.a, p.share, flags_of(q0), at, d0, v, count, l, m);
            return;
        }
        const float r = l == 0.0f ? 0.0f : 1.0f / l;
        uint16_t *dst = static_cast<uint16_t *>(p.a.out) + at * D + d0;
#pragma unroll
        for (int i = 0; i < count; i += 4) {
            uint2 w;
            if (p.a.dtype == 0) {
                w.x = pack_half2(v[i] * r, v[i + 1] * r), w.y = pack_half2(v[i + 2] * r, v[i + 3] * r);
            } else {
                w.x = pack_bf162(v[i] * r, v[i + 1] * r), w.y = pack_bf162(v[i + 2] * r, v[i + 3] * r);
            }
            *reinterpret_cast<uint2 *>(dst + i) = w;
        }
        if (p.a.lse && d0 == 0) p.a.lse[at] = l == 0.0f ? -INFINITY : (m + __log2f(l)) * 0.6931471805599453f;
    };
    // The tile's part of this warp: to the output when `whole`, else to `park`.
    // o[.][k][0..1] and o[.][k][2..3] are dims g * D / 8 + 2 k and that plus 1.
    auto finish_tile = [&](bool whole, float *park) {
#pragma unroll
        for (int nr = 0; nr < NR; ++nr)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                sum[nr][e] += __shfl_xor_sync(0xffffffffu, sum[nr][e], 4);
                sum[nr][e] += __shfl_xor_sync(0xffffffffu, sum[nr][e], 8);
                sum[nr][e] += __shfl_xor_sync(0xffffffffu, sum[nr][e], 16);
                float v[2 * KS];
#pragma unroll
                for (int k = 0; k < KS; ++k) v[2 * k] = o[nr][k][e], v[2 * k + 1] = o[nr][k][2 + e];
                const int row = row_of(nr, e);
                long long at;
                if (!place(tile, row, at)) continue;
                if (whole) {
                    store_row(tile.q0, at, g * 2 * KS, v, 2 * KS, sum[nr][e], ref[nr][e]);
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

    // ---- first copies, first rows: every load on its way before one is waited for
    Meta cur = look_up(w0), nxt = cur;
    if (w0 < w1) next = load_rows(w0);
    look_up_scales(cur);
    const int blocks = (w1 - w0) * BPS;                            // the warp's blocks, two a step or one
    int fetched = min(NS, blocks);                                 // blocks issued so far
    for (int i = 0; i < fetched; ++i)
        issue(i, __shfl_sync(0xffffffffu, cur.page, i), __shfl_sync(0xffffffffu, cur.where, i));
    if (lane == 0 && w0 == 0 && w1 > 0 && next.begin < 0) {
        // a tile that an earlier CTA began: this warp has its first part here
        shared[0] = Shared{1, warp, next.begin, next.end, next.q0, next.n, next.head, next.row};
        s_out[0] = 0;
    }
    tile.end = w0;

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
    int phase = 0, stage = 0;                                      // of the next block to consume
    const uint32_t k_row = ring + p.k_at * KB * D + tau * D, v_ring = ring + p.v_at * KB * D;
    for (int at = w0;; ++at) {
        const int l = (at - w0) % LOOK;
        // the next blocks' page ids and scales, a few steps apart so that neither is waited for
        if (l == 0 && at != w0) cur = nxt;
        if (l == 1 && at - 1 + LOOK < w1) nxt = look_up(at - 1 + LOOK);
        if (l == LOOK / 4 && at - l + LOOK < w1) look_up_scales(nxt);
        if (at == tile.end || at == w1) {
            if (at > w0) finish_tile(tile.begin >= w0 && tile.end == at, tile.begin < w0 ? first_part : last_part);
            if (at == w1) break;
            if (NR > 1 && at > w0) next = load_rows(at);
            start_tile(next);
        }
        if (NR == 1 && at + 1 == tile.end && at + 1 < w1) next = load_rows(at + 1);
        float s[BPS][SUB][NR][4], iv[BPS];
        int pos[BPS], st[BPS];
        bool edge[BPS];
#pragma unroll
        for (int b = 0; b < BPS; ++b) {
            st[b] = stage;
            if (!mbar_wait_bounded(bars + stage * 8, phase, p.status, &s_abort)) failed = true;
            if (++stage == NS) stage = 0, phase ^= 1;
        }
        if (__any_sync(0xffffffffu, failed)) {                     // the whole warp: what follows is the warp's
            failed = true;
            break;
        }
#pragma unroll
        for (int b = 0; b < BPS; ++b)
#pragma unroll
            for (int u = 0; u < SUB; ++u) {
#pragma unroll
                for (int nr = 0; nr < NR; ++nr)
#pragma unroll
                    for (int i = 0; i < 4; ++i) s[b][u][nr][i] = 0.0f;
                const uint32_t kb = k_row + st[b] * L::kStage + u * 16 * D;
#pragma unroll
                for (int j = 0; j < KS / 4; ++j) {
                    const int chunk = t + 4 * j;
                    const int sw = D == 128 ? chunk ^ (tau & 7) : chunk ^ ((tau >> 1) & 3);
                    const uint4 x = lds128(kb + sw * 16), y = lds128(kb + 8 * D + sw * 16);
                    const uint32_t xw[4] = {x.x, x.y, x.z, x.w}, yw[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        uint32_t a0, a1, a2, a3;
                        codes_to_half<KT>(xw[w], a0, a2);
                        codes_to_half<KT>(yw[w], a1, a3);
#pragma unroll
                        for (int nr = 0; nr < NR; ++nr)
                            mma16816<0>(s[b][u][nr], a0, a1, a2, a3, q[nr][4 * j + w][0], q[nr][4 * j + w][1]);
                    }
                }
            }
        // x_j + log2(vs); keys a row does not see get -inf
        float top[NR][2];
#pragma unroll
        for (int nr = 0; nr < NR; ++nr) top[nr][0] = top[nr][1] = -INFINITY;
#pragma unroll
        for (int b = 0; b < BPS; ++b) {
            const int from = l * BPS + b;
            pos[b] = __shfl_sync(0xffffffffu, cur.pos, from);
            const float ks = __shfl_sync(0xffffffffu, cur.ks, from), vs = __shfl_sync(0xffffffffu, cur.vs, from);
            const float lv = __log2f(vs);
            iv[b] = __fdividef(1.0f, vs);
            edge[b] = pos[b] + KB - 1 > min_pos ||
                      (p.a.window > 0 && pos[b] <= max_pos - p.a.window && pos[b] + KB > p.a.sinks);
#pragma unroll
            for (int nr = 0; nr < NR; ++nr) {
                const float f0 = fac[nr][0] * ks, f1 = fac[nr][1] * ks;
#pragma unroll
                for (int u = 0; u < SUB; ++u)
#pragma unroll
                    for (int i = 0; i < 4; ++i) s[b][u][nr][i] = fmaf(s[b][u][nr][i], i & 1 ? f1 : f0, lv);
                if (edge[b])
#pragma unroll
                    for (int u = 0; u < SUB; ++u)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int j = pos[b] + u * 16 + tau + 8 * (i >> 1), r = row_pos[nr][i & 1];
                            const bool see = j <= r && (p.a.window == 0 || r - j < p.a.window || j < p.a.sinks);
                            if (!see) s[b][u][nr][i] = -INFINITY;
                        }
#pragma unroll
                for (int u = 0; u < SUB; ++u)
#pragma unroll
                    for (int i = 0; i < 4; ++i) top[nr][i & 1] = fmaxf(top[nr][i & 1], s[b][u][nr][i]);
            }
        }
        bool over = false;
#pragma unroll
        for (int nr = 0; nr < NR; ++nr)
            over |= top[nr][0] - ref[nr][0] > kTop || top[nr][1] - ref[nr][1] > kTop;
        if (__any_sync(0xffffffffu, over)) {
#pragma unroll
            for (int nr = 0; nr < NR; ++nr)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float m = top[nr][e];
                    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
                    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
                    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
                    if (m - ref[nr][e] > kHead) {
                        const float f = ex2(ref[nr][e] - (m - kHead));
                        ref[nr][e] = m - kHead;
                        sum[nr][e] *= f;
#pragma unroll
                        for (int k = 0; k < KS; ++k) o[nr][k][e] *= f, o[nr][k][2 + e] *= f;
                    }
                }
        }
#pragma unroll
        for (int b = 0; b < BPS; ++b)
#pragma unroll
            for (int u = 0; u < SUB; ++u) {
                uint32_t pt[NR][2];
#pragma unroll
                for (int nr = 0; nr < NR; ++nr) {
                    float w[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) w[i] = ex2(s[b][u][nr][i] - ref[nr][i & 1]);
                    // a block that the row does not see adds nothing, whatever its scale
                    if (w[0] + w[2] != 0.0f) sum[nr][0] = fmaf(w[0] + w[2], iv[b], sum[nr][0]);
                    if (w[1] + w[3] != 0.0f) sum[nr][1] = fmaf(w[1] + w[3], iv[b], sum[nr][1]);
                    pt[nr][0] = movmatrix(pack_half2(w[0], w[1]));
                    pt[nr][1] = movmatrix(pack_half2(w[2], w[3]));
                }
                // V^T as A: byte i of a lane's chunk g is dim g * D / 8 + i
                const uint32_t vb = v_ring + st[b] * L::kStage + u * 16 * D;
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
                if (KT == kKvE4m3 && edge[b]) {
                    // bytes of keys no row sees may be NaN codes; their weight of 0 would not hide them
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int j = pos[b] + u * 16 + ((r & 1) != flip ? v_key1 : v_key0) + 8 * (r >> 1);
                        if (j > max_pos)
#pragma unroll
                            for (int w = 0; w < D / 32; ++w) vw[r][w] = 0;
                    }
                }
#pragma unroll
                for (int w = 0; w < D / 32; ++w) {
                    uint32_t a[4][2];                              // [dim of the word][keys 2t, 2t + 1 or those + 8]
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
            }
        __syncwarp();
        if (fetched < blocks) {
            if (lane == 0) fence_proxy_async_smem();
            // the blocks just freed: `fetched` counts blocks, LOOK * BPS = 32 of them a look-up
            const bool ahead = fetched / 32 != (at - w0) / LOOK;
#pragma unroll
            for (int b = 0; b < BPS; ++b) {
                // with an odd ring the two blocks of a step may belong to different look-ups
                const int f = fetched + b;
                const bool far = BPS == 1 ? ahead : f / 32 != (at - w0) / LOOK;
                const int page = __shfl_sync(0xffffffffu, far ? nxt.page : cur.page, f & 31);
                const int where = __shfl_sync(0xffffffffu, far ? nxt.where : cur.where, f & 31);
                if (f < blocks) issue(st[b], page, where);
            }
            fetched += BPS;
        }
    }
    if (failed) {
        // leave with no copy in flight
        for (int i = max(0, min(fetched, blocks) - NS); i < min(fetched, blocks); ++i)
            mbar_wait_bounded(bars + i % NS * 8, (i / NS) & 1, p.status, &s_abort);
    } else if (lane == 0 && w0 < w1 && tile.begin >= w0 && tile.end > w1) {
        // the warp that holds a tile's first part in this CTA says so
        shared[1 + warp] = Shared{1, warp, tile.begin, tile.end, tile.q0, tile.n, tile.head, tile.row};
        if (tile.end > mine) s_out[1] = 1 + warp;
    }
    __syncthreads();
    // A CTA that gave a wait up has no results, but its tickets are counted: they are back at 0 after every launch,
    // also for a replay, whose tag is the same.
    const bool gave_up = s_abort != 0;

    // ---- tiles that more than one warp holds a part of, summed in warp order
    // Parts of a shared tile: the first warp's (its last piece when the tile begins there), then the first
    // pieces of the warps after it up to the tile's end.  Row `row`, dims d..d + 3.
    auto sum_parts = [&](const Shared &sh, bool leads, int row, int d, float (&acc)[4], float &l, float &m) {
        const float *part = leads ? reinterpret_cast<const float *>(smem + sh.first_warp * NS * L::kStage)
                                  : reinterpret_cast<const float *>(smem + L::kPark) + sh.first_warp * L::kPart;
        m = kRefStart, l = 0.0f;
        acc[0] = acc[1] = acc[2] = acc[3] = 0.0f;
        for (int v = sh.first_warp; v < NW; ++v) {
            const int v0 = warp_start(v), v1 = warp_start(v + 1);
            if (v0 >= sh.end) break;
            if (v > sh.first_warp) part = reinterpret_cast<const float *>(smem + L::kPark) + v * L::kPart;
            if (v0 >= v1) continue;
            const float2 ml = *reinterpret_cast<const float2 *>(part + ROWS * D + 2 * row);
            const float4 x = *reinterpret_cast<const float4 *>(part + row * D + d);
            const float to = fmaxf(m, ml.x), f = ex2(m - to), w = ex2(ml.x - to);
            m = to;
            l = fmaf(ml.y, w, l * f);
            acc[0] = fmaf(x.x, w, acc[0] * f), acc[1] = fmaf(x.y, w, acc[1] * f);
            acc[2] = fmaf(x.z, w, acc[2] * f), acc[3] = fmaf(x.w, w, acc[3] * f);
        }
    };
    // Those that leave the CTA first: at its start and at its end, into slots 0 and 1 of the workspace, by all threads.
    bool out[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        out[i] = s_out[i] >= 0;
        if (!out[i] || gave_up) continue;
        const Shared sh = shared[s_out[i]];
        const int rows = min(ROWS, sh.n * group - sh.row);
        float *dst = p.parts + ((long long)blockIdx.x * 2 + i) * L::kPart;
        for (int k = tid; k < rows * (D / 4); k += 32 * NW) {
            const int row = k / (D / 4), d = k % (D / 4) * 4;
            float acc[4], l, m;
            sum_parts(sh, i == 1, row, d, acc, l, m);
            __stcg(reinterpret_cast<float4 *>(dst + row * D + d), make_float4(acc[0], acc[1], acc[2], acc[3]));
            if (d == 0) __stcg(reinterpret_cast<float2 *>(dst + ROWS * D + 2 * row), make_float2(m, l));
        }
    }
    const bool defer = SHARED && p.share.defer;                    // whoever reads the rows sums the parts
    if (!defer && (out[0] || out[1] || gave_up)) {
        // tickets: which CTAs share the tile follows from where it begins and ends (a warp that has hardly had
        // anything to sum: eight rows are 256 pieces at most)
        const int nth = tid - 32 * (NW - 1);
        bool asks = nth >= 0 && nth < 2 && (out[nth & 1] || gave_up);
        int from = 0, to = 0;
        if (asks) {
            // the tile of the CTA's first step or of its last
            const long long line = c0 + (nth ? mine - 1 : 0);
            const int b = find(line, 0, s_seq[0], s_seq[NW]), steps = span(seqs[b].y, seqs[b].z).steps;
            const int idx = line_div(line - pre[b], steps);
            const long long first = pre[b] + (long long)idx * steps;
            if (gave_up) asks = nth ? first >= c0 && first + steps > c0 + mine : first < c0;
            // with the costs, the tile begins and ends at
            const long long begin = first + (long long)(tiles_before[b] + idx) * COST;
            const long long end = begin + steps + COST;
            // the last CTA whose share begins by the tile's first step, and by its last
            from = (int)(((begin + COST + 1) * ctas + total - 1) / total - 1);
            to = (int)((end * ctas + total - 1) / total - 1);
            if (by_tile) {
                int done = 0, n = 0;
                for (int i = 0; i <= b; ++i) {
                    if (seqs[i].w == 0) continue;
                    n = pieces_of(i, done, span(seqs[i].y, seqs[i].z).steps + COST);
                    if (i < b) done += n * seqs[i].w * Hk;
                }
                from = (done + idx * n) / NW;
                to = (done + idx * n + n - 1) / NW;
            }
        }
        __syncthreads();
        if (asks) {
            __threadfence();                                       // after the barrier: for the whole CTA's parts
            // the guess that all others have come: right for the last, for whom it counts
            unsigned long long *tk = p.tickets + from, seen = p.tag << 16 | (unsigned long long)(to - from), put = 0;
            for (;;) {
                const unsigned long long old = atomicCAS(tk, seen, put);
                if (old == seen) break;
                seen = old;
                const unsigned long long n = (seen >> 16) == p.tag ? (seen & 0xffff) + 1 : 1;
                put = n == (unsigned long long)(to - from + 1) ? 0 : p.tag << 16 | n;
            }
            __threadfence();
            s_from[nth] = put == 0 ? from : -1;
            s_to[nth] = to;
        }
    }
    if (gave_up) {
        leave();
        return;
    }
    if (defer && out[1] && warp == NW - 1) {
        // the tile that begins here: the last CTA whose share begins by its last step
        const Shared sh = shared[s_out[1]];
        const long long line = c0 + mine - 1;
        const int b = find(line, 0, s_seq[0], s_seq[NW]), steps = span(seqs[b].y, seqs[b].z).steps;
        const int idx = line_div(line - pre[b], steps);
        const long long end = pre[b] + (long long)idx * steps + (long long)(tiles_before[b] + idx) * COST + steps + COST;
        int to = (int)((end * ctas + total - 1) / total - 1);
        if (by_tile) {
            int done = 0, n = 0;
            for (int i = 0; i <= b; ++i) {
                if (seqs[i].w == 0) continue;
                n = pieces_of(i, done, span(seqs[i].y, seqs[i].z).steps + COST);
                if (i < b) done += n * seqs[i].w * Hk;
            }
            to = (done + idx * n + n - 1) / NW;
        }
        const Tile tl = {sh.begin, sh.end, sh.q0, sh.n, sh.row, sh.head, 0};
        for (int row = lane; row < ROWS; row += 32) {
            long long at;
            if (place(tl, row, at)) p.share.where[flags_of(tl.q0) & kKvOthers][at] = kv_where(kKvFewParts, row, blockIdx.x, to);
        }
    }
    // those within the CTA: each by the warp that holds the first part
    {
        const Shared sh = shared[1 + warp];
        if (sh.has && sh.end <= mine) {
            const int rows = min(ROWS, sh.n * group - sh.row);
            for (int k = lane; k < rows * (D / 4); k += 32) {
                const int row = k / (D / 4), d = k % (D / 4) * 4;
                float acc[4], l, m;
                sum_parts(sh, true, row, d, acc, l, m);
                long long at;
                if (place(tile, row, at)) store_row(tile.q0, at, d, acc, 4, l, m);
            }
        }
    }
    if (defer || (!out[0] && !out[1])) {
        leave();
        return;
    }
    __syncthreads();
    // ---- a tile that CTAs from..to share: the last of them to come sums it
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        if (!out[i] || s_from[i] < 0) continue;
        const int from = s_from[i], to = s_to[i];
        const Shared sh = shared[s_out[i]];
        const Tile tl = {sh.begin, sh.end, sh.q0, sh.n, sh.row, sh.head, 0};
        const int rows = min(ROWS, sh.n * group - sh.row);
        // CTA `from` holds its part in slot 1, the others in slot 0
        auto slot = [&](int c) { return p.parts + ((long long)c * 2 + (c == from)) * L::kPart; };
        for (int k = tid; k < rows * (D / 4); k += 32 * NW) {
            const int row = k / (D / 4), d = k % (D / 4) * 4;
            float m = kRefStart, acc[4] = {0.0f, 0.0f, 0.0f, 0.0f}, l = 0.0f;
            // eight parts at a time: their loads are on their way together
            for (int c = from; c <= to; c += 8) {
                float2 ml[8];
                float4 x[8];
                float top = m;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float *part = slot(min(c + j, to));
                    ml[j] = __ldcg(reinterpret_cast<const float2 *>(part + ROWS * D + 2 * row));
                    x[j] = __ldcg(reinterpret_cast<const float4 *>(part + row * D + d));
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) top = fmaxf(top, ml[j].x);
                const float f = ex2(m - top);
                m = top;
                l *= f;
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[j] *= f;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float w = c + j <= to ? ex2(ml[j].x - m) : 0.0f;
                    l = fmaf(ml[j].y, w, l);
                    acc[0] = fmaf(x[j].x, w, acc[0]), acc[1] = fmaf(x[j].y, w, acc[1]);
                    acc[2] = fmaf(x[j].z, w, acc[2]), acc[3] = fmaf(x[j].w, w, acc[3]);
                }
            }
            long long at;
            if (place(tl, row, at)) store_row(tl.q0, at, d, acc, 4, l, m);
        }
    }
    leave();
}

using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                   const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// A map of codes whose boxes are `keys` tokens of one head of one page, of one
// tensor or (apart > 0: the bytes from it to the other) of K and V.  The
// dimensions after the first go by rising stride.
cudaError_t encode_codes(const DeviceInfo &dev, const KvCache &c, void *base, long long apart, int keys,
                         bool token_first, CUtensorMap *out) {
    if (dev.encode_tiled == nullptr) return cudaErrorNotSupported;
    const cuuint64_t tokens = (cuuint64_t)1 << c.page_shift, heads = (cuuint64_t)c.n_kv_heads;
    // a dimension of one element has no stride of its own
    const cuuint64_t sh = c.n_kv_heads > 1 ? (cuuint64_t)c.head_stride : (cuuint64_t)c.token_stride << c.page_shift;
    const cuuint64_t sp = c.n_pages > 1 ? (cuuint64_t)c.page_stride : (cuuint64_t)c.token_stride << c.page_shift;
    const cuuint32_t both = apart > 0 ? 2 : 1;
    cuuint64_t dims[5] = {(cuuint64_t)c.head_dim, tokens, heads, (cuuint64_t)c.n_pages, both};
    cuuint64_t strides[4] = {(cuuint64_t)c.token_stride, sh, sp, apart > 0 ? (cuuint64_t)apart : sp};
    cuuint32_t box[5] = {(cuuint32_t)c.head_dim, (cuuint32_t)keys, 1, 1, both};
    const cuuint32_t one[5] = {1, 1, 1, 1, 1};
    if (token_first) {
        std::swap(dims[1], dims[2]);
        std::swap(strides[0], strides[1]);
        std::swap(box[1], box[2]);
    }
    const CUresult r = reinterpret_cast<EncodeTiledFn>(dev.encode_tiled)(
        out, CU_TENSOR_MAP_DATA_TYPE_UINT8, 5, base, dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
        c.head_dim == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <bool SHARED, int KT, int D, int NR, int KB, int BPS, int NW, int NS>
cudaError_t launch_few(const FewParams &p, const CUtensorMap &k, const CUtensorMap &v, int grid, cudaStream_t s,
                       bool pdl) {
    using L = FewSmem<D, NR, KB, NW, NS>;
    auto kern = few_rows_kernel<SHARED, KT, D, NR, KB, BPS, NW, NS>;
    const cudaError_t e = raise_smem_cap(reinterpret_cast<const void *>(kern), L::kEnd);
    if (e != cudaSuccess) return e;
    return kv_launch(kern, dim3(grid), dim3(32 * NW), L::kEnd, s, pdl, k, v, p);
}

constexpr int kTileRows = 16;             // the most rows of a tile here

// Rows of a tile for a batch whose sequences have up to so many tokens.
inline int few_tile_rows(int max_q_len, int group) { return (long long)max_q_len * group <= 8 ? 8 : kTileRows; }

// All sequences of the batch, or those of up to row_limit rows a kv head (0: all).
template <bool SHARED>
cudaError_t launch_few_rows(const KvAttentionArgs &a, const KvCache &c, const KvBatch &batch, int row_limit,
                            KvShare share, const DeviceInfo &dev, cudaStream_t s, bool pdl) {
    const int group = a.n_heads / c.n_kv_heads;
    const KvEntry *entries = share.entries;
    const bool token_first = c.n_kv_heads > 1 && c.head_stride < c.token_stride;
    // blocks of 32 keys where a page holds them: half the boxes and look-ups
    const int keys = c.page_shift >= 5 ? 32 : 16;
    // one map over both tensors, from the lower one up, where their distance fits a stride
    const long long apart = c.v - c.k, distance = apart < 0 ? -apart : apart;
    const bool merged = distance > 0 && distance < 1LL << 40;
    CUtensorMap k, v;
    cudaError_t e = encode_codes(dev, c, merged && apart < 0 ? c.v : c.k, merged ? distance : 0, keys, token_first, &k);
    if (e == cudaSuccess && !merged) e = encode_codes(dev, c, c.v, 0, keys, token_first, &v);
    if (e != cudaSuccess) return e;
    if (merged) v = k;
    static std::atomic<unsigned long long> launches{SHARED ? 0x5ca1ab1f0000ull : 0x5ca1ab1e0000ull};
    constexpr int kMost = SHARED ? kMaxEntries : kMaxSeqs;
    for (int b0 = 0; b0 < batch.n_seqs; b0 += kMost) {
        KvBatch b = batch;
        if constexpr (SHARED) {
            share.entries = entries + b0;
        } else {
            b.block_table += (long long)b0 * b.max_blocks;
            b.kv_lens += b0;
            b.q_starts += b0;
        }
        b.n_seqs = std::min(kMost, batch.n_seqs - b0);
        const bool owns = !SHARED;                              // rows that are no sequence's
        FewParams p{a, c, b, row_limit, token_first ? 1 : 0, merged ? 1 : 0, owns && b0 == 0,
                    owns && b0 + b.n_seqs == batch.n_seqs, merged && apart < 0 ? 1 : 0, merged && apart < 0 ? 0 : 1,
                    nullptr, nullptr, 0, hold_copies(), dev.status, share};
        p.tickets = static_cast<unsigned long long *>(a.workspace);
        p.parts = reinterpret_cast<float *>(p.tickets + ((dev.sm_count + 1) & ~1));
        p.tag = (launches.fetch_add(1) * 0x9e3779b97f4a7c15ull) >> 16;
        if (p.tag == 0) p.tag = 1;
        const int grid = dev.sm_count;
        const bool few = few_tile_rows(a.max_q_len, group) == 8;
        // <codes, dims, 8-row tiles, keys a block, blocks a step, warps, ring stages>
        // Two blocks a step where the registers allow it: one costs 68 us instead of 57 (64 ragged contexts, pages of
        // 16), 55 instead of 44 (the same at 64 dims), 41 instead of 34 (64 dims, pages of 64), 61 instead of 52 (24 x 5
        // tokens, 64 dims, pages of 16).  Rings of 128 to 160 KB, what fits beside the parts: a stage or two more or
        // less changes up to 2 %, but for 16-row tiles of 128 dims and 16 keys, where three stages take 60.5 us for 24 x
        // 4 tokens and these four 65.4.
#define W4A16_FEW(KT)                                                                                              \
    if (keys == 32)                                                                                                \
        e = c.head_dim == 128 ? (few ? launch_few<SHARED, KT, 128, 1, 32, 1, 8, 2>(p, k, v, grid, s, pdl)          \
                                     : launch_few<SHARED, KT, 128, 2, 32, 1, 8, 2>(p, k, v, grid, s, pdl))         \
                              : (few ? launch_few<SHARED, KT, 64, 1, 32, 2, 8, 5>(p, k, v, grid, s, pdl)           \
                                     : launch_few<SHARED, KT, 64, 2, 32, 1, 8, 4>(p, k, v, grid, s, pdl));         \
    else                                                                                                           \
        e = c.head_dim == 128 ? (few ? launch_few<SHARED, KT, 128, 1, 16, 2, 8, 5>(p, k, v, grid, s, pdl)          \
                                     : launch_few<SHARED, KT, 128, 2, 16, 1, 8, 4>(p, k, v, grid, s, pdl))         \
                              : (few ? launch_few<SHARED, KT, 64, 1, 16, 2, 8, 10>(p, k, v, grid, s, pdl)          \
                                     : launch_few<SHARED, KT, 64, 2, 16, 2, 8, 8>(p, k, v, grid, s, pdl))
        if (c.kv_dtype == kKvInt8) {
            W4A16_FEW(kKvInt8);
        } else {
            W4A16_FEW(kKvE4m3);
        }
#undef W4A16_FEW
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace
}  // namespace w4a16
