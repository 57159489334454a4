// kv_attention.cu -- attention over the paged 8-bit cache: the choice between the
// kernels of kv_few_rows.cuh and kv_attention_tc.cu.
#include <cstdio>

#include "kv_few_rows.cuh"

namespace w4a16 {

// Rows a kv head up to which a sequence is this kernel's.  A second tile reads
// the keys again, out of L2; with 32 keys a block or 64 dims that still costs
// less than a mostly empty 128-row tile, with 16 keys of 128 dims it need not.
// Measured, this kernel / the other, in us, at 32 rows of 24 sequences of 128
// to 4001 tokens: pages of 64 75 / 80, 64 dims 49 / 59, pages of 16 100 / 84; at
// 40 rows (three tiles) 99 / 81, 66 / 59 and 131 / 84; at 16 rows 65 / 85.
int kv_few_rows_most(const KvCache &c) { return c.page_shift >= 5 || c.head_dim == 64 ? 2 * kTileRows : kTileRows; }

cudaError_t launch_kv_attention(const KvAttentionArgs &a, const KvCache &c, const KvBatch &batch, const DeviceInfo &dev,
                                cudaStream_t s, bool pdl) {
    const int group = a.n_heads / c.n_kv_heads, most = kv_few_rows_most(c);
    // Sequences with more rows go to the tensor-core kernel.  When every sequence brings max_q_len tokens all of
    // them do, and this kernel, which would find nothing to do (about 4 us), is left out; should max_q_len not be
    // the longest, that kernel has them all the same.
    const bool many = (long long)a.max_q_len * group > most;
    const bool all_many = many && (long long)a.max_q_len * batch.n_seqs == batch.n_tokens;
    if (kernel_log_on()) {
        char line[256];
        std::snprintf(line, sizeof line,
                      "kv_attention tokens=%d seqs=%d longest=%d heads=%d/%d D=%d page=%d %s %s kernel=%s rows<=%d grid=%d pdl=%d",
                      batch.n_tokens, batch.n_seqs, a.max_q_len, a.n_heads, c.n_kv_heads, c.head_dim, 1 << c.page_shift,
                      c.kv_dtype == kKvInt8 ? "int8" : "e4m3", a.dtype == 0 ? "fp16" : "bf16",
                      all_many ? "many_rows" : many ? "few_rows+many_rows" : "few_rows", most, dev.sm_count, pdl ? 1 : 0);
        log_kernel_selection(line);
    }
    if (all_many)
        return launch_kv_attention_many(a, c, batch, 0, dev, s, pdl);
    const cudaError_t e = launch_few_rows<false>(a, c, batch, many ? most : 0, KvShare{}, dev, s, pdl);
    if (e != cudaSuccess) return e;
    return many ? launch_kv_attention_many(a, c, batch, most, dev, s, pdl) : cudaSuccess;
}

long long kv_attention_workspace(int n_heads, int n_kv_heads, int head_dim, int, int n_tokens, const DeviceInfo &dev) {
    if ((long long)n_tokens * (n_heads / n_kv_heads) > kTileRows) return kv_attention_many_workspace(head_dim, dev);
    return (long long)((dev.sm_count + 1) & ~1) * 8 + (long long)dev.sm_count * 2 * kTileRows * (head_dim + 2) * 4;
}

}  // namespace w4a16
