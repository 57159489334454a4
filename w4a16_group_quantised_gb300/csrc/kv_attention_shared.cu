// kv_attention_shared.cu -- attention over the paged 8-bit cache of a batch whose
// sequences share pages: samples and beams of a prompt, users of one system
// prompt.
//
// A softmax over two sets of keys splits: with sums o_i = sum_j 2^(x_j - m_i) v_j
// and l_i = sum_j 2^(x_j - m_i) over each, and m the larger of m_1 and m_2,
//     out = (2^(m_1 - m) o_1 + 2^(m_2 - m) o_2) / (2^(m_1 - m) l_1 + 2^(m_2 - m) l_2).
// So the keys that a group's sequences have in common are read once, for the
// tokens of all of them as the rows of one problem, and joined with every row's
// sum over its own keys at the end.
//  * The plan: what a group shares (whole pages that lie before all of its new
//    tokens), as an entry of rows, keys and a place in the block table for
//    each group and for the rest of each sequence.
//  * The kernels of kv_few_rows.cuh and, where it may pay, kv_attention_tc.cu,
//    with entries in place of sequences: shared keys, which every row of a
//    group sees, and the others at once.
//  * The join, a warp or half of one a row.  A group's tile is long and there are
//    few of them, so that each is cut over many CTAs: the parts that these
//    leave are read here, by all SMs, where in kv_attention the last CTA to come
//    sums them alone.
//
// Measured on the GPU (32 query heads of 128 dims; w4a16_kv_attention in
// brackets): 64 sequences on a system prompt of 8192 tokens with 1 to 2000 of
// their own, e4m3, 164 MB: 62 us (154), 2.6 TB/s; 31 and 40 sequences of 1 to 5
// tokens on documents of 32 thousand, 109 GFLOP: 211 us (759), 515
// TFLOP/s; 16 prompts of 100 to 1920 tokens in 3 to 8 samples: 52 us (52).  Bound
// by the two kernels' own ways: what they take to start and end (the plan 5 us,
// the join 4 to 8 beside), their tiles' chains, and the codes' conversion, which
// comes again for every 8 or 256 rows.
#include <algorithm>
#include <cstdio>

#include "kv_few_rows.cuh"

namespace w4a16 {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kLeastShared = 64;          // positions that are worth an entry of their own
constexpr int kBigRows = 16;              // more rows a kv head may be kv_attention_tc.cu's

// What entries take, in ns on kCostSms SMs with 128 dims: kv_few_rows.cuh 16 keys of
// a tile of 8 rows, with pages of 16 or of more tokens, or of 16 rows (a tile's start
// and end count for 192 or 288 keys); kv_attention_tc.cu 128 keys of a tile of 256 (384
// keys); and what each kernel takes to start and end.  Fitted to 170 calls of 8 to 256
// sequences in 1 to 16 groups that read 190 to 840 MB unshared: all 170 take 10.2 ms
// so, 9.9 with the better choice for each, 11.1 with starts of 10 and 45 us and 80 keys
// a tile, and 64 sequences on a prompt of 8192 tokens 64 us (73 with 1.5 of the
// others' time, which most like as well).
// Few rows / tensor cores for the shared keys, us a call with 8 heads to each of 4 kv
// heads, 64 keys of each sequence's own: one group of 8 sequences over 25000 keys
// 47 / 42, over 51000 82 / 53; of 32 over 6000 48 / 40, over 13000 83 / 46; 16 groups of
// 16 over 700 keys 57 / 61, over 1500 89 / 65; 4 groups of 4 over 12000 48 / 49.
constexpr float kFewNs8 = 0.75f, kFewNs8Wide = 0.66f, kFewNs16 = 1.05f, kManyNs = 16.0f, kOf64Dims = 0.55f;
constexpr float kFewStartNs = 16000.0f, kManyStartNs = 40000.0f;
constexpr int kCostSms = 152;
__host__ __device__ inline unsigned long long few_steps(long long rows, int tile_shift, int keys) {
    const unsigned ends = tile_shift == 3 ? 12 : 18;
    return (unsigned long long)((rows + (1 << tile_shift) - 1) >> tile_shift) * (((keys + 15) >> 4) + ends);
}
__host__ __device__ inline unsigned long long many_steps(long long rows, int keys) {
    return (unsigned long long)((rows + kManyTileRows - 1) / kManyTileRows) * (unsigned)(((keys + 127) >> 7) + 3);
}

struct PlanParams {
    KvBatch b;
    KvGroups g;
    int page_shift, group, tile_shift;
    float few_ns, many_ns;                // of a step, all kv heads
    KvEntry *entries;                     // of groups, then of sequences
    int *shared;                          // positions that each group shares
    int *use_many;                        // KvShare
    int choice;                           // w4a16_debug_set_config(10)
    int sms, may_many, beside;
    uint4 *where;                         // of both kinds, to be cleared
    long long where_vecs;
    int *status;
};

// The first CTA: groups, a warp each, then sequences.  The others: no row has a sum yet.
__global__ void __launch_bounds__(kPlanThreads) plan_shared_kernel(const PlanParams p) {
    kv_begin();
    if (blockIdx.x > 0) {
        for (long long i = (long long)(blockIdx.x - 1) * kPlanThreads + threadIdx.x; i < p.where_vecs;
             i += (long long)(gridDim.x - 1) * kPlanThreads)
            p.where[i] = make_uint4(0, 0, 0, 0);
        return;
    }
    // steps of the big entries by either kernel, of the others; the best division of the SMs
    __shared__ unsigned long long s_few, s_many, s_rest;
    __shared__ unsigned s_best;
    if (threadIdx.x == 0) s_few = s_many = s_rest = 0, s_best = 0xffffffffu;
    __syncthreads();
    unsigned long long few = 0, many = 0, rest = 0;       // of this thread
    auto big = [&](int n, int keys) {
        const long long rows = (long long)n * p.group;
        const unsigned long long steps = few_steps(rows, p.tile_shift, max(keys, 0));
        if (rows <= kBigRows) {
            rest += steps;
            return 0;
        }
        few += steps;
        many += many_steps(rows, max(keys, 0));
        return kKvBig;
    };
    const int lane = threadIdx.x & 31, n_seqs = p.b.n_seqs, n_groups = p.g.n_groups;
    for (int g = threadIdx.x >> 5; g < n_groups; g += kPlanThreads / 32) {
        const int s0 = p.g.group_starts[g], s1 = p.g.group_starts[g + 1], said = p.g.prefix_lens[g];
        const int lo = min(max(s0, 0), n_seqs), hi = min(max(s1, lo), n_seqs);
        if (lane == 0 && (lo != s0 || hi != s1 || said < 0)) kv_report(p.status);
        // of the sequences that bring tokens: how many, the first, the rows of all, the shortest past
        int count = 0, first = n_seqs, q0 = p.b.n_tokens, q1 = 0, past = 0x7fffffff;
        for (int i = lo + lane; i < hi; i += 32) {
            const KvSeq s = kv_sequence(p.b, p.page_shift, i, p.status);
            if (s.n == 0) continue;
            ++count;
            first = min(first, i);
            q0 = min(q0, s.q0), q1 = max(q1, s.q0 + s.n);
            past = min(past, max(s.len - s.n, 0));
        }
        count = __reduce_add_sync(0xffffffffu, count);
        first = __reduce_min_sync(0xffffffffu, first);
        q0 = __reduce_min_sync(0xffffffffu, q0), q1 = __reduce_max_sync(0xffffffffu, q1);
        past = __reduce_min_sync(0xffffffffu, past);
        int n = count > 1 ? min(max(said, 0), past) >> p.page_shift << p.page_shift : 0;
        if (n < kLeastShared) n = 0;
        if (lane == 0) {
            p.shared[g] = n;
            p.entries[g] = n > 0 ? KvEntry{q0, q1 - q0, n, big(q1 - q0, n), (long long)first * p.b.max_blocks, 0} : KvEntry{};
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n_seqs; i += kPlanThreads) {
        const KvSeq s = kv_sequence(p.b, p.page_shift, i, p.status);
        // the last group that begins at or before the sequence, if it is one of its
        int lo = 0, hi = n_groups;
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (p.g.group_starts[mid] <= i) lo = mid + 1;
            else hi = mid;
        }
        const bool member = lo > 0 && p.g.group_starts[lo] > i;
        // starts that fall may find a sequence in a group that it was not counted with: never more than its past
        const int past = max(s.len - s.n, 0) >> p.page_shift << p.page_shift;
        const int skip = member && s.n > 0 ? min(p.shared[lo - 1], past) : 0;
        const int flags = kKvOthers | (skip == 0 ? kKvAlone : 0) | big(s.n, s.len - skip);
        p.entries[n_groups + i] =
            KvEntry{s.q0, s.n, s.len - skip, flags, (long long)i * p.b.max_blocks + (skip >> p.page_shift), 0};
    }
    auto sum = [&](unsigned long long v, unsigned long long &to) {
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
        if (lane == 0 && v > 0) atomicAdd(&to, v);
    };
    sum(few, s_few), sum(many, s_many), sum(rest, s_rest);
    __syncthreads();
    // Both kernels side by side, on some SMs each, or one after the other on all; or the few-rows kernel alone.
    const float few_ns = p.few_ns * kCostSms, on_many = (float)s_many * p.many_ns * kCostSms, on_rest = (float)s_rest * few_ns;
    const bool some_rest = s_rest > 0;
    // The least time t and its k in one word: t is above 0, so that its bits are in its order, and of the 23 of its fraction
    // 13 do; the 10 below them are k.  (A cut t would be the same for every k from the cut on, and k = 1 the least.)
    if (p.may_many && p.choice != 1 && s_few > 0) {
        for (int k = threadIdx.x + 1; k <= p.sms; k += kPlanThreads) {
            float t;
            if (k == p.sms) {
                t = kManyStartNs + on_many / p.sms + (some_rest ? kFewStartNs + on_rest / p.sms : 0.0f);
            } else {
                if (!p.beside || !some_rest) continue;
                t = fmaxf(kManyStartNs + on_many / k, kFewStartNs + on_rest / (p.sms - k));
            }
            atomicMin(&s_best, (__float_as_uint(t) & ~1023u) | (unsigned)k);
        }
        __syncthreads();
    }
    if (threadIdx.x == 0) {
        const float alone = kFewStartNs + (on_rest + (float)s_few * few_ns) / p.sms;
        const bool use = s_best != 0xffffffffu && (p.choice == 2 || __uint_as_float(s_best & ~1023u) < alone);
        const int k = use ? (int)(s_best & 1023) : 0;
        p.use_many[0] = use;
        p.use_many[1] = k;
        p.use_many[2] = k == p.sms ? k : p.sms - k;
    }
}

struct JoinParams {
    KvAttentionArgs a;
    KvShare share;
    const float *few, *many;              // parts
    int few_rows;                         // of a tile of kv_few_rows.cuh
    int rows;
};

// A row's sums of both kinds, D / 4 lanes a row, four dims each.
template <int D>
__global__ void __launch_bounds__(256) join_kernel(const JoinParams p) {
    kv_begin();
    constexpr int LANES = D / 4;
    const long long row = ((long long)blockIdx.x * 256 + threadIdx.x) / LANES;
    const int d = threadIdx.x % LANES * 4;
    if (row >= p.rows) return;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    float m = kRefStart, l = 0.0f;
    auto add = [&](float2 ml, float4 x) {
        const float top = fmaxf(m, ml.x), f = ex2(m - top), w = ex2(ml.x - top);
        m = top;
        l = fmaf(ml.y, w, l * f);
        o = make_float4(fmaf(x.x, w, o.x * f), fmaf(x.y, w, o.y * f), fmaf(x.z, w, o.z * f), fmaf(x.w, w, o.w * f));
    };
    unsigned long long where[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) where[i] = p.share.where[i][row];
    if ((where[1] & 7) == kKvDone) return;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int kind = (int)(where[i] & 7), r = (int)(where[i] >> 3 & 511);
        const int from = (int)(where[i] >> 16 & 0xffff), to = (int)(where[i] >> 32 & 0xffff);
        if (kind == kKvNone) continue;
        if (kind == kKvInArrays) {
            add(reinterpret_cast<const float2 *>(p.share.ml[i])[row],
                *reinterpret_cast<const float4 *>(p.share.out[i] + row * D + d));
            continue;
        }
        const bool few = kind == kKvFewParts;
        const int tile = few ? p.few_rows : kManyTileRows, part = tile * (D + 2);
        // where a part has the row's four dims, and its (m, l)
        const float *base = few ? p.few : p.many;
        const int at = few ? r * D + d : d * tile + 4 * r, ml_at = tile * D + 2 * r;
        constexpr int N = 8;                               // parts whose loads are on their way together
        for (int c = from; c <= to; c += N) {
            float2 ml[N];
            float4 x[N];
#pragma unroll
            for (int k = 0; k < N; ++k) {
                const int cta = min(c + k, to);
                const float *src = base + (2LL * cta + (cta == from)) * part;
                ml[k] = *reinterpret_cast<const float2 *>(src + ml_at);
                x[k] = *reinterpret_cast<const float4 *>(src + at);
            }
#pragma unroll
            for (int k = 0; k < N; ++k)
                if (c + k <= to) add(ml[k], x[k]);
        }
    }
    const float r = l == 0.0f ? 0.0f : 1.0f / l;
    uint2 w;
    if (p.a.dtype == 0) w.x = pack_half2(o.x * r, o.y * r), w.y = pack_half2(o.z * r, o.w * r);
    else w.x = pack_bf162(o.x * r, o.y * r), w.y = pack_bf162(o.z * r, o.w * r);
    *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.a.out) + row * D + d) = w;
    if (p.a.lse && d == 0) p.a.lse[row] = l == 0.0f ? -INFINITY : (m + __log2f(l)) * 0.6931471805599453f;
}

struct Scratch {
    void *few, *many;                     // of the two kernels: tickets, parts
    KvEntry *entries;
    int *shared, *use_many;
    unsigned long long *where[2];
    float *ml[2], *out[2];
    long long bytes;
};

long long tickets_bytes(const DeviceInfo &dev) { return (long long)((dev.sm_count + 1) & ~1) * 8; }

Scratch scratch_of(void *ws, int n_heads, int n_kv_heads, int head_dim, int n_seqs, int n_groups, int n_tokens,
                   const DeviceInfo &dev) {
    char *p = static_cast<char *>(ws);
    auto take = [&](long long bytes) {
        char *q = p;
        p += (bytes + 15) & ~15LL;
        return q;
    };
    Scratch s;
    const long long rows = (long long)n_tokens * n_heads;
    s.entries = reinterpret_cast<KvEntry *>(take(((long long)n_groups + n_seqs) * sizeof(KvEntry)));
    s.shared = reinterpret_cast<int *>(take((long long)n_groups * 4));
    s.use_many = reinterpret_cast<int *>(take(12));
    s.where[0] = reinterpret_cast<unsigned long long *>(take((rows + 1) / 2 * 32));
    s.where[1] = s.where[0] + (rows + 1) / 2 * 2;
    s.few = take(tickets_bytes(dev) + (long long)dev.sm_count * 2 * kTileRows * (head_dim + 2) * 4);
    s.many = (long long)n_tokens * (n_heads / n_kv_heads) > kBigRows ? take(kv_attention_many_workspace(head_dim, dev)) : nullptr;
    for (int i = 0; i < 2; ++i) {
        s.ml[i] = reinterpret_cast<float *>(take(rows * 8));
        s.out[i] = reinterpret_cast<float *>(take(rows * head_dim * 4));
    }
    s.bytes = p - static_cast<char *>(ws);
    return s;
}

// Whether kv_attention is called instead, by what there is at most: sequences as long as the table is wide, the lengths
// being on the device (in a table of 2048 columns four beams of 901 tokens take 16.7 us, in one of 61 12.8).  Its one launch
// is the faster one for few bytes of cache, and where sequences fill tiles by themselves: what sharing saves are tiles, of 8
// rows (which one sequence with 8 rows fills), or of the 256 of kv_attention_tc.cu, which take as long as some 3.6 of 8.
// This / that in us, bytes as all sequences read them:
//    1 row a sequence (query heads of a kv head, times tokens): 48 MB 16 / 18, 96 MB 17 to 27 / 24, 192 MB 19 to 36 / 38
//    4 rows: 48 MB 18 to 26 / 18, 96 MB 25 to 33 / 25, 192 MB 33 to 41 / 38, 400 MB 50 to 62 / 67
//    8 rows: 96 MB 32 to 40 / 26 to 29, 192 MB 42 to 59 / 40, 400 MB 45 to 68 / 67 (16 sequences in 4 groups 86)
//    16 rows: 62 MB 43 / 30, 125 MB 50 / 52, 188 MB 43 / 53.  32 rows: 31 MB 37 / 30, 62 MB 45 / 52, 94 MB 40 / 52
//    64 rows: 62 MB 56 / 45, 94 MB 47 / 66, 125 MB 82 / 81, 188 MB 65 / 101
//    128 rows: 62 MB 75 / 45, 125 MB 122 / 82, 188 MB 91 / 102, 375 MB 156 / 196.  256 rows: 375 MB 303 / 226
bool kv_attention_instead(double bytes, int rows) {
    const double tiles = std::min((double)((rows + 7) / 8), 3.6);
    return rows > 96 || bytes * tiles <= (40 << 20) * (double)std::min(std::max(rows, 2), 8);
}

}  // namespace

cudaError_t launch_kv_attention_shared(const KvAttentionArgs &a, const KvCache &c, const KvBatch &b, const KvGroups &g,
                                       const DeviceInfo &dev, cudaStream_t s, bool pdl) {
    const int group = a.n_heads / c.n_kv_heads, rows = b.n_tokens * a.n_heads;
    const long long longest = (long long)b.max_blocks << c.page_shift;
    const int forced = shared_kernels();
    const int seqs = std::min(b.n_seqs, b.n_tokens);          // that bring tokens, at most
    const int seq_rows = (int)(((long long)b.n_tokens * group + seqs - 1) / seqs);
    const bool plain = g.n_groups == 0 ||
                       (!forced && kv_attention_instead(2.0 * longest * seqs * c.n_kv_heads * c.head_dim, seq_rows));
    // the tensor-core kernel is launched where the plan might ask for it
    const int tile_rows = few_tile_rows(a.max_q_len, group), tile_shift = tile_rows == 16 ? 4 : 3;
    const long long all = (long long)b.n_tokens * group, entries = (long long)g.n_groups + b.n_seqs;
    const float scale = c.n_kv_heads * (c.head_dim == 64 ? kOf64Dims : 1.0f);
    const float few_ns = scale * (tile_rows == 16 ? kFewNs16 : c.page_shift > 4 ? kFewNs8Wide : kFewNs8);
    const float most = (float)few_steps(2 * (all + entries * tile_rows), tile_shift, (int)longest) * few_ns;
    const bool may_many = all > kBigRows && forced != 1 && (forced == 2 || most > kManyStartNs);
    if (kernel_log_on()) {
        char line[256];
        std::snprintf(line, sizeof line,
                      "kv_attention_shared tokens=%d seqs=%d groups=%d longest=%d heads=%d/%d D=%d page=%d %s %s kernel=%s "
                      "rows=%d grid=%d pdl=%d",
                      b.n_tokens, b.n_seqs, g.n_groups, a.max_q_len, a.n_heads, c.n_kv_heads, c.head_dim, 1 << c.page_shift,
                      c.kv_dtype == kKvInt8 ? "int8" : "e4m3", a.dtype == 0 ? "fp16" : "bf16",
                      plain ? "kv_attention" : may_many ? "few_rows+many_rows" : "few_rows", tile_rows, dev.sm_count, pdl ? 1 : 0);
        log_kernel_selection(line);
    }
    if (plain) return launch_kv_attention(a, c, b, dev, s, pdl);
    const Scratch w = scratch_of(a.workspace, a.n_heads, c.n_kv_heads, c.head_dim, b.n_seqs, g.n_groups, b.n_tokens, dev);
    const long long vecs = ((long long)rows + 1) / 2 * 2;
    const PlanParams plan{b, g, c.page_shift, group, tile_shift, few_ns, scale * kManyNs, w.entries, w.shared, w.use_many, forced,
                          dev.sm_count, may_many, pdl, reinterpret_cast<uint4 *>(w.where[0]), vecs, dev.status};
    const int fill = (int)std::min<long long>((vecs + 4 * kPlanThreads - 1) / (4 * kPlanThreads), dev.sm_count);
    cudaError_t e = kv_launch(plan_shared_kernel, dim3(1 + fill), dim3(kPlanThreads), 0, s, pdl, plan);
    if (e != cudaSuccess) return e;
    KvBatch batch = b;
    batch.n_seqs = (int)entries;
    KvAttentionArgs args = a;
    KvShare share{w.entries, w.use_many, 0, 0, {w.out[0], w.out[1]}, {w.ml[0], w.ml[1]}, {w.where[0], w.where[1]}};
    if (may_many) {
        args.workspace = w.many;
        share.defer = kv_attention_many_at_once(batch, group);
        e = launch_kv_attention_many(args, c, batch, 0, dev, s, pdl, &share);
        if (e != cudaSuccess) return e;
    }
    args.workspace = w.few;
    share.defer = entries <= kMaxEntries;                     // one launch: its parts stay until the join
    share.beside = may_many && pdl;
    e = launch_few_rows<true>(args, c, batch, 0, share, dev, s, pdl);
    if (e != cudaSuccess) return e;
    auto parts = [&](void *ws) { return reinterpret_cast<const float *>(static_cast<char *>(ws) + tickets_bytes(dev)); };
    const JoinParams join{a, share, parts(w.few), may_many ? parts(w.many) : nullptr, tile_rows, rows};
    const dim3 grid((unsigned)(((long long)rows * (c.head_dim / 4) + 255) / 256));
    return c.head_dim == 128 ? kv_launch(join_kernel<128>, grid, dim3(256), 0, s, pdl, join)
                             : kv_launch(join_kernel<64>, grid, dim3(256), 0, s, pdl, join);
}

long long kv_attention_shared_workspace(int n_heads, int n_kv_heads, int head_dim, int n_seqs, int n_groups,
                                        int n_tokens, const DeviceInfo &dev) {
    // what kv_attention needs where that is called
    return std::max(scratch_of(nullptr, n_heads, n_kv_heads, head_dim, n_seqs, n_groups, n_tokens, dev).bytes,
                    kv_attention_workspace(n_heads, n_kv_heads, head_dim, n_seqs, n_tokens, dev));
}

}  // namespace w4a16
