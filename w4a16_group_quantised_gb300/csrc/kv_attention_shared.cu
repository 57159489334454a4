// kv_attention_shared.cu -- attention over the paged 8-bit cache of a batch whose
// sequences share pages: samples and beams of a prompt, users of one system
// prompt.
//
// A softmax over two sets of keys splits: with sums o_i = sum_j 2^(x_j - m_i) v_j
// and l_i = sum_j 2^(x_j - m_i) over each, and m the larger of m_1 and m_2,
//     out = (2^(m_1 - m) o_1 + 2^(m_2 - m) o_2) / (2^(m_1 - m) l_1 + 2^(m_2 - m) l_2).
// So the keys that a group's sequences have in common are read once, for the
// tokens of all of them as the rows of one problem, and joined with every row's
// sum over its own keys at the end.  Four kernels:
//  * the plan: what a group shares (whole pages that lie before all of its new
//    tokens), as an entry of rows, keys and a place in the block table for
//    each group and for the rest of each sequence;
//  * the shared keys, all rows of a group seeing all of them;
//  * the others;
//  * the join, a warp or half of one a row.
// The middle two are the kernels of kv_few_rows.cuh and kv_attention_tc.cu with
// entries in place of sequences; which of them follows from the rows.  A group's
// tile is long, and there are few of them, so that each is cut over many CTAs:
// the parts that these leave are read by the join, by all SMs, where in
// kv_attention the last CTA to come sums them alone.
#include <algorithm>
#include <cstdio>

#include "kv_few_rows.cuh"

namespace w4a16 {
namespace {

constexpr int kPlanThreads = 1024;

struct PlanParams {
    KvBatch b;
    KvGroups g;
    int page_shift;
    KvEntry *groups, *seqs;
    int *shared;                          // positions that each group shares
    uint4 *where;                         // of both passes, to be cleared
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
        const int n = count > 1 ? min(max(said, 0), past) >> p.page_shift << p.page_shift : 0;
        if (lane == 0) {
            p.shared[g] = n;
            p.groups[g] = n > 0 ? KvEntry{q0, q1 - q0, n, 0, (long long)first * p.b.max_blocks, 0} : KvEntry{};
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
        p.seqs[i] = KvEntry{s.q0, s.n, s.len - skip, 0, (long long)i * p.b.max_blocks + (skip >> p.page_shift), 0};
    }
}

// What the join reads of a pass.
struct PassSums {
    const unsigned long long *where;
    const float *out, *ml;
    const float *few, *many;              // parts
    int few_rows;                         // of a tile of kv_few_rows.cuh
};
struct JoinParams {
    KvAttentionArgs a;
    PassSums pass[2];
    int rows;
};

// A row's sums of both passes, D / 4 lanes a row, four dims each.
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
    for (int i = 0; i < 2; ++i) where[i] = p.pass[i].where[row];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const PassSums &s = p.pass[i];
        const int kind = (int)(where[i] & 3), r = (int)(where[i] >> 2 & 511);
        const int from = (int)(where[i] >> 16 & 0xffff), to = (int)(where[i] >> 32 & 0xffff);
        if (kind == kKvNone) continue;
        if (kind == kKvInArrays) {
            add(reinterpret_cast<const float2 *>(s.ml)[row], *reinterpret_cast<const float4 *>(s.out + row * D + d));
            continue;
        }
        const bool few = kind == kKvFewParts;
        const int tile = few ? s.few_rows : kManyTileRows, part = tile * (D + 2);
        // where a part has the row's four dims, and its (m, l)
        const float *base = few ? s.few : s.many;
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
    void *few[2], *many[2];               // of the passes' kernels: tickets, parts
    KvEntry *groups, *seqs;
    int *shared;
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
    const bool many = (long long)n_tokens * (n_heads / n_kv_heads) > kTileRows;
    s.groups = reinterpret_cast<KvEntry *>(take((long long)n_groups * sizeof(KvEntry)));
    s.seqs = reinterpret_cast<KvEntry *>(take((long long)n_seqs * sizeof(KvEntry)));
    s.shared = reinterpret_cast<int *>(take((long long)n_groups * 4));
    s.where[0] = reinterpret_cast<unsigned long long *>(take(2 * ((rows * 8 + 15) & ~15LL)));
    s.where[1] = s.where[0] + ((rows + 1) & ~1LL);
    for (int i = 0; i < 2; ++i) {
        s.few[i] = take(tickets_bytes(dev) + (long long)dev.sm_count * 2 * kTileRows * (head_dim + 2) * 4);
        s.many[i] = many ? take(kv_attention_many_workspace(head_dim, dev)) : nullptr;
        s.ml[i] = reinterpret_cast<float *>(take(rows * 8));
        s.out[i] = reinterpret_cast<float *>(take(rows * head_dim * 4));
    }
    s.bytes = p - static_cast<char *>(ws);
    return s;
}

}  // namespace

cudaError_t launch_kv_attention_shared(const KvAttentionArgs &a, const KvCache &c, const KvBatch &b, const KvGroups &g,
                                       const DeviceInfo &dev, cudaStream_t s, bool pdl) {
    const Scratch w = scratch_of(a.workspace, a.n_heads, c.n_kv_heads, c.head_dim, b.n_seqs, g.n_groups, b.n_tokens, dev);
    const int group = a.n_heads / c.n_kv_heads, most = kv_few_rows_most(c), rows = b.n_tokens * a.n_heads;
    const long long vecs = ((long long)rows + 1) / 2 * 2;
    const PlanParams plan{b, g, c.page_shift, w.groups, w.seqs, w.shared, reinterpret_cast<uint4 *>(w.where[0]), vecs,
                          dev.status};
    const int fill = (int)std::min<long long>((vecs + 4 * kPlanThreads - 1) / (4 * kPlanThreads), dev.sm_count);
    cudaError_t e = kv_launch(plan_shared_kernel, dim3(1 + fill), dim3(kPlanThreads), 0, s, pdl, plan);
    if (e != cudaSuccess) return e;
    // Shared keys: by the tokens that a group has in the mean when that decides, else each kernel those it is for.
    const long long all = (long long)b.n_tokens * group;
    const bool many_shared = all > most, all_many_shared = many_shared && all > (long long)most * g.n_groups;
    // The others as in kv_attention.cu.
    const bool many = (long long)a.max_q_len * group > most;
    const bool all_many = many && (long long)a.max_q_len * b.n_seqs == b.n_tokens;
    if (kernel_log_on()) {
        char line[256];
        std::snprintf(line, sizeof line,
                      "kv_attention_shared tokens=%d seqs=%d groups=%d longest=%d heads=%d/%d D=%d page=%d %s %s shared=%s "
                      "others=%s rows<=%d grid=%d pdl=%d",
                      b.n_tokens, b.n_seqs, g.n_groups, a.max_q_len, a.n_heads, c.n_kv_heads, c.head_dim, 1 << c.page_shift,
                      c.kv_dtype == kKvInt8 ? "int8" : "e4m3", a.dtype == 0 ? "fp16" : "bf16",
                      all_many_shared ? "many_rows" : many_shared ? "few_rows+many_rows" : "few_rows",
                      all_many ? "many_rows" : many ? "few_rows+many_rows" : "few_rows", most, dev.sm_count, pdl ? 1 : 0);
        log_kernel_selection(line);
    }
    JoinParams join{a, {}, rows};
    for (int i = 0; i < 2; ++i) {
        KvBatch batch = b;
        batch.n_seqs = i ? b.n_seqs : g.n_groups;
        KvAttentionArgs args = a;
        if (i == 0) args.max_q_len = b.n_tokens;           // picks tiles of 8 or 16 rows
        const bool some_many = i ? many : many_shared, only_many = i ? all_many : all_many_shared;
        KvShare share{i ? w.seqs : w.groups, i, 0, w.out[i], w.ml[i], w.where[i]};
        if (!only_many) {
            args.workspace = w.few[i];
            share.defer = batch.n_seqs <= kMaxSeqs;        // one launch: its parts stay until the join
            e = launch_few_rows<true>(args, c, batch, some_many ? most : 0, share, dev, s, pdl);
            if (e != cudaSuccess) return e;
        }
        if (some_many) {
            args.workspace = w.many[i];
            share.defer = kv_attention_many_launches(batch, group) == 1;
            e = launch_kv_attention_many(args, c, batch, only_many ? 0 : most, dev, s, pdl, &share);
            if (e != cudaSuccess) return e;
        }
        auto parts = [&](void *ws) { return reinterpret_cast<const float *>(static_cast<char *>(ws) + tickets_bytes(dev)); };
        join.pass[i] = PassSums{w.where[i], w.out[i], w.ml[i], parts(w.few[i]), w.many[i] ? parts(w.many[i]) : nullptr,
                                few_tile_rows(args.max_q_len, group)};
    }
    const dim3 grid((unsigned)(((long long)rows * (c.head_dim / 4) + 255) / 256));
    return c.head_dim == 128 ? kv_launch(join_kernel<128>, grid, dim3(256), 0, s, pdl, join)
                             : kv_launch(join_kernel<64>, grid, dim3(256), 0, s, pdl, join);
}

long long kv_attention_shared_workspace(int n_heads, int n_kv_heads, int head_dim, int n_seqs, int n_groups,
                                        int n_tokens, const DeviceInfo &dev) {
    return scratch_of(nullptr, n_heads, n_kv_heads, head_dim, n_seqs, n_groups, n_tokens, dev).bytes;
}

}  // namespace w4a16
