// kv_attention_shared.cu -- attention over the paged 8-bit cache of a batch whose
// sequences share pages: samples and beams of a prompt, users of one system
// prompt.
//
// A softmax over two sets of keys splits: with sums o_i = sum_j 2^(x_j - m_i) v_j
// and l_i = sum_j 2^(x_j - m_i) over each, and m the larger of m_1 and m_2,
//     out = (2^(m_1 - m) o_1 + 2^(m_2 - m) o_2) / (2^(m_1 - m) l_1 + 2^(m_2 - m) l_2).
// So the keys that a group's sequences have in common are read once, for the
// tokens of all of them as the rows of one problem, and every row's sum over
// its own keys is joined with that where the row is written.  Three kernels:
//  * the plan: what a group shares (whole pages that lie before all of its new
//    tokens), as an entry of rows, keys and a place in the block table for
//    each group and for the rest of each sequence;
//  * the shared keys, all rows of a group seeing all of them: sums in fp32 with
//    reference and denominator to scratch;
//  * the others, joined on the way out.
// The last two are the kernels of kv_few_rows.cuh and kv_attention_tc.cu with
// entries in place of sequences; which of them follows from the rows.
#include <algorithm>
#include <cstdio>

#include "kv_few_rows.cuh"

namespace w4a16 {
namespace {

constexpr int kPlanThreads = 1024;

struct PlanParams {
    KvBatch b;
    KvGroups g;
    int page_shift, rows;                 // rows: n_tokens * n_heads
    KvEntry *groups, *seqs;
    int *shared;                          // positions that each group shares
    float *ml;
    int *status;
};

// The first CTA: groups, a warp each, then sequences.  The others: no row has a sum over shared keys yet.
__global__ void __launch_bounds__(kPlanThreads) plan_shared_kernel(const PlanParams p) {
    kv_begin();
    if (blockIdx.x > 0) {
        for (int i = (blockIdx.x - 1) * kPlanThreads + threadIdx.x; i < p.rows; i += (gridDim.x - 1) * kPlanThreads)
            reinterpret_cast<float2 *>(p.ml)[i] = make_float2(kRefStart, 0.0f);
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

struct Scratch {
    void *attention;                      // of the two passes, one after the other
    KvEntry *groups, *seqs;
    int *shared;
    float *ml, *out;
    long long bytes;
};

Scratch scratch_of(void *ws, int n_heads, int n_kv_heads, int head_dim, int n_seqs, int n_groups, int n_tokens,
                   const DeviceInfo &dev) {
    char *p = static_cast<char *>(ws);
    auto take = [&](long long bytes) {
        char *q = p;
        p += (bytes + 15) & ~15LL;
        return q;
    };
    Scratch s;
    s.attention = take(kv_attention_workspace(n_heads, n_kv_heads, head_dim, n_seqs, n_tokens, dev));
    s.groups = reinterpret_cast<KvEntry *>(take((long long)n_groups * sizeof(KvEntry)));
    s.seqs = reinterpret_cast<KvEntry *>(take((long long)n_seqs * sizeof(KvEntry)));
    s.shared = reinterpret_cast<int *>(take((long long)n_groups * 4));
    const long long rows = (long long)n_tokens * n_heads;
    s.ml = reinterpret_cast<float *>(take(rows * 8));
    s.out = reinterpret_cast<float *>(take(rows * head_dim * 4));
    s.bytes = p - static_cast<char *>(ws);
    return s;
}

}  // namespace

cudaError_t launch_kv_attention_shared(const KvAttentionArgs &a, const KvCache &c, const KvBatch &b, const KvGroups &g,
                                       const DeviceInfo &dev, cudaStream_t s, bool pdl) {
    const Scratch w = scratch_of(a.workspace, a.n_heads, c.n_kv_heads, c.head_dim, b.n_seqs, g.n_groups, b.n_tokens, dev);
    const int group = a.n_heads / c.n_kv_heads, most = kv_few_rows_most(c), rows = b.n_tokens * a.n_heads;
    const PlanParams plan{b, g, c.page_shift, rows, w.groups, w.seqs, w.shared, w.ml, dev.status};
    const int fill = std::min((rows + 4 * kPlanThreads - 1) / (4 * kPlanThreads), dev.sm_count);
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
    KvAttentionArgs args = a;
    args.workspace = w.attention;
    KvBatch batch = b;
    if (g.n_groups > 0) {
        const KvShare share{w.groups, 0, w.out, w.ml};
        batch.n_seqs = g.n_groups;
        args.max_q_len = b.n_tokens;                       // picks tiles of 8 or 16 rows
        if (!all_many_shared) e = launch_few_rows<true>(args, c, batch, many_shared ? most : 0, share, dev, s, pdl);
        if (e == cudaSuccess && many_shared)
            e = launch_kv_attention_many(args, c, batch, all_many_shared ? 0 : most, dev, s, pdl, &share);
        if (e != cudaSuccess) return e;
    }
    const KvShare share{w.seqs, 1, w.out, w.ml};
    batch.n_seqs = b.n_seqs;
    args.max_q_len = a.max_q_len;
    if (!all_many) e = launch_few_rows<true>(args, c, batch, many ? most : 0, share, dev, s, pdl);
    if (e == cudaSuccess && many) e = launch_kv_attention_many(args, c, batch, all_many ? 0 : most, dev, s, pdl, &share);
    return e;
}

long long kv_attention_shared_workspace(int n_heads, int n_kv_heads, int head_dim, int n_seqs, int n_groups,
                                        int n_tokens, const DeviceInfo &dev) {
    return scratch_of(nullptr, n_heads, n_kv_heads, head_dim, n_seqs, n_groups, n_tokens, dev).bytes;
}

}  // namespace w4a16
