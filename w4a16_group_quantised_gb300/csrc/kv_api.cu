// kv_api.cu -- C ABI of the paged 8-bit key/value cache: host-side validation
// and dispatch to kv_append.cu, kv_attention.cu and kv_pages.cu.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdlib>

#include "kernels.h"
#include "w4a16.h"

namespace w4a16 {
namespace {

bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int shift_of(int page_size) {
    for (int s = 4; s <= 7; ++s)
        if (page_size == 1 << s) return s;
    return -1;
}

int check_dtype(int dtype) { return dtype == W4A16_F16 || dtype == W4A16_BF16 ? W4A16_OK : W4A16_ERR_DTYPE; }

// Whether no two rows of head_dim bytes, of all pages, heads and tokens, overlap.
bool rows_apart(const w4a16_kv_cache_t *c) {
    struct { long long n, stride; } dims[3] = {
        {c->page_size, c->token_stride}, {c->n_kv_heads, c->head_stride}, {c->n_pages, c->page_stride}};
    std::sort(dims, dims + 3, [](const auto &a, const auto &b) { return a.stride < b.stride; });
    // one dimension within the next: every ordinary layout
    long long extent = c->head_dim;
    bool nested = true;
    for (const auto &d : dims) {
        if (d.n == 1) continue;
        nested = nested && d.stride >= extent;
        extent += (d.n - 1) * d.stride;
    }
    if (nested) return true;
    // else every distance in tokens and heads against the nearest one in pages
    const long long pages = c->n_pages - 1, sp = c->page_stride;
    for (int t = 0; t < c->page_size; ++t)
        for (int h = 1 - c->n_kv_heads; h < c->n_kv_heads; ++h) {
            const long long at = t * c->token_stride + h * c->head_stride;
            const long long near = sp > 0 ? -at / sp : 0;
            for (long long p = std::max(near - 1, -pages); p <= std::min(near + 1, pages); ++p)
                if ((t != 0 || h != 0 || p != 0) && std::llabs(at + p * sp) < c->head_dim) return false;
        }
    return true;
}

int check_cache(const w4a16_kv_cache_t *c, KvCache *out) {
    if (c == nullptr) return W4A16_ERR_NULL;
    if (c->kv_dtype != W4A16_KV_INT8 && c->kv_dtype != W4A16_KV_E4M3) return W4A16_ERR_DTYPE;
    const int shift = shift_of(c->page_size);
    if (shift < 0 || (c->head_dim != 64 && c->head_dim != 128)) return W4A16_ERR_SHAPE;
    if (c->n_pages <= 0 || c->n_pages > (1 << 28) || c->n_kv_heads <= 0 || c->n_kv_heads > 1024) return W4A16_ERR_SHAPE;
    if (c->k == nullptr || c->v == nullptr || c->k_scale == nullptr || c->v_scale == nullptr) return W4A16_ERR_NULL;
    const long long strides[3] = {c->page_stride, c->head_stride, c->token_stride};
    for (long long s : strides) {
        if (s < 0 || s >= (1LL << 40)) return W4A16_ERR_SHAPE;
        if (s % 16 != 0) return W4A16_ERR_ALIGN;
    }
    if (c->token_stride < c->head_dim || (c->n_kv_heads > 1 && c->head_stride < c->head_dim) ||
        (c->n_pages > 1 && c->page_stride < c->head_dim))
        return W4A16_ERR_SHAPE;
    if (!rows_apart(c)) return W4A16_ERR_SHAPE;
    if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4))
        return W4A16_ERR_ALIGN;
    *out = KvCache{static_cast<uint8_t *>(c->k), static_cast<uint8_t *>(c->v), c->k_scale, c->v_scale,
                   c->page_stride, c->head_stride, c->token_stride, c->n_pages, shift, c->n_kv_heads, c->head_dim,
                   c->kv_dtype};
    return W4A16_OK;
}

// Positions of a sequence: a step's keys more than the last, or a window and a call's tokens less than the first, are
// still 32-bit numbers.
constexpr long long kMaxPositions = (1LL << 31) - (1LL << 25);

int check_table(const void *table, const void *lens, int n_seqs, int max_blocks, int page_size) {
    if (n_seqs < 0 || n_seqs > (1 << 20) || max_blocks <= 0 || (long long)max_blocks * page_size > kMaxPositions)
        return W4A16_ERR_SHAPE;
    if (n_seqs > 0 && (table == nullptr || lens == nullptr)) return W4A16_ERR_NULL;
    if (!aligned(table, 4) || !aligned(lens, 4)) return W4A16_ERR_ALIGN;
    return W4A16_OK;
}

int check_batch(const w4a16_kv_batch_t *b, int page_size, KvBatch *out) {
    if (b == nullptr) return W4A16_ERR_NULL;
    const int rc = check_table(b->block_table, b->kv_lens, b->n_seqs, b->max_blocks, page_size);
    if (rc != W4A16_OK) return rc;
    if (b->n_tokens < 0 || b->n_tokens > (1 << 24) || (b->n_seqs == 0 && b->n_tokens > 0)) return W4A16_ERR_SHAPE;
    if (b->n_seqs > 0 && b->q_starts == nullptr) return W4A16_ERR_NULL;
    if (!aligned(b->q_starts, 4)) return W4A16_ERR_ALIGN;
    *out = KvBatch{b->block_table, b->kv_lens, b->q_starts, b->n_seqs, b->max_blocks, b->n_tokens};
    return W4A16_OK;
}

// Rows of token tensors: 16-byte aligned, `width` elements or more apart.
int check_rows(const void *p, long long stride, long long width) {
    if (stride < width || stride >= (1LL << 32)) return W4A16_ERR_SHAPE;
    if (stride % 8 != 0 || !aligned(p, 16)) return W4A16_ERR_ALIGN;
    return W4A16_OK;
}

int check_pool(const void *refcount, int n_pages, const void *workspace, long long bytes) {
    if (refcount == nullptr || workspace == nullptr) return W4A16_ERR_NULL;
    if (!aligned(refcount, 4) || !aligned(workspace, 16)) return W4A16_ERR_ALIGN;
    return bytes < kv_pool_workspace(n_pages) ? W4A16_ERR_ARG : W4A16_OK;
}

int done(cudaError_t e) { return e == cudaSuccess ? W4A16_OK : W4A16_ERR_CUDA; }
cudaStream_t str(w4a16_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

}  // namespace
}  // namespace w4a16

using namespace w4a16;

#define W4A16_TRY(x)                     \
    do {                                 \
        const int rc_ = (x);             \
        if (rc_ != W4A16_OK) return rc_; \
    } while (0)

extern "C" {

int w4a16_kv_append(const w4a16_kv_cache_t *cache, const void *k_new, long long k_stride, const void *v_new,
                    long long v_stride, const w4a16_kv_batch_t *batch, w4a16_dtype_t dtype, w4a16_stream_t stream) {
    KvCache c;
    KvBatch b;
    W4A16_TRY(check_dtype((int)dtype));
    W4A16_TRY(check_cache(cache, &c));
    W4A16_TRY(check_batch(batch, cache->page_size, &b));
    if (b.n_tokens == 0) return W4A16_OK;
    if (k_new == nullptr || v_new == nullptr) return W4A16_ERR_NULL;
    W4A16_TRY(check_rows(k_new, k_stride, (long long)c.n_kv_heads * c.head_dim));
    W4A16_TRY(check_rows(v_new, v_stride, (long long)c.n_kv_heads * c.head_dim));
    const DeviceInfo *dev = nullptr;
    W4A16_TRY(device_info(&dev));
    return done(launch_kv_append(c, b, k_new, k_stride, v_new, v_stride, (int)dtype, *dev, str(stream), pdl_enabled()));
}

int w4a16_kv_read(const w4a16_kv_cache_t *cache, const w4a16_kv_batch_t *batch, void *k_out, void *v_out,
                  w4a16_dtype_t dtype, w4a16_stream_t stream) {
    KvCache c;
    KvBatch b;
    W4A16_TRY(check_dtype((int)dtype));
    W4A16_TRY(check_cache(cache, &c));
    W4A16_TRY(check_batch(batch, cache->page_size, &b));
    if (b.n_tokens == 0) return W4A16_OK;
    if (k_out == nullptr || v_out == nullptr) return W4A16_ERR_NULL;
    if (!aligned(k_out, 16) || !aligned(v_out, 16)) return W4A16_ERR_ALIGN;
    const DeviceInfo *dev = nullptr;
    W4A16_TRY(device_info(&dev));
    return done(launch_kv_read(c, b, k_out, v_out, (int)dtype, *dev, str(stream), pdl_enabled()));
}

int w4a16_kv_attention(const void *q, long long q_stride, int n_heads, const w4a16_kv_cache_t *cache,
                       const w4a16_kv_batch_t *batch, int max_q_len, float scale, int window, int sinks, void *out,
                       float *lse_or_null, w4a16_dtype_t dtype, void *workspace, long long workspace_bytes,
                       w4a16_stream_t stream) {
    KvCache c;
    KvBatch b;
    W4A16_TRY(check_dtype((int)dtype));
    W4A16_TRY(check_cache(cache, &c));
    W4A16_TRY(check_batch(batch, cache->page_size, &b));
    if (n_heads <= 0 || n_heads % c.n_kv_heads != 0 || n_heads / c.n_kv_heads > 128 || n_heads > 4096)
        return W4A16_ERR_SHAPE;
    if ((long long)b.n_tokens * n_heads >= (1LL << 31)) return W4A16_ERR_SHAPE;
    if (max_q_len < 0 || window < 0 || sinks < 0 || !(scale == scale)) return W4A16_ERR_ARG;
    if (b.n_tokens == 0) return W4A16_OK;
    if (q == nullptr || out == nullptr) return W4A16_ERR_NULL;
    W4A16_TRY(check_rows(q, q_stride, (long long)n_heads * c.head_dim));
    if (!aligned(out, 16) || !aligned(lse_or_null, 4)) return W4A16_ERR_ALIGN;
    const DeviceInfo *dev = nullptr;
    W4A16_TRY(device_info(&dev));
    const long long need = kv_attention_workspace(n_heads, c.n_kv_heads, c.head_dim, b.n_seqs, b.n_tokens, *dev);
    if (need > 0 && workspace == nullptr) return W4A16_ERR_NULL;
    if (!aligned(workspace, 16)) return W4A16_ERR_ALIGN;
    if (workspace_bytes < need) return W4A16_ERR_ARG;
    // no sequence is as long as the table is wide and a window: every token sees all keys before it
    if (window >= b.max_blocks * cache->page_size) window = 0;
    KvAttentionArgs a{q, q_stride, n_heads, max_q_len, window, sinks, scale, out, lse_or_null, (int)dtype, workspace};
    return done(launch_kv_attention(a, c, b, *dev, str(stream), pdl_enabled()));
}

int w4a16_kv_attention_workspace(int n_heads, int n_kv_heads, int head_dim, int n_seqs, int n_tokens,
                                 long long *bytes) {
    if (bytes == nullptr) return W4A16_ERR_NULL;
    if (n_heads <= 0 || n_kv_heads <= 0 || n_heads % n_kv_heads != 0 || n_heads / n_kv_heads > 128 || n_heads > 4096 ||
        (head_dim != 64 && head_dim != 128) || n_seqs < 0 || n_tokens < 0)
        return W4A16_ERR_SHAPE;
    const DeviceInfo *dev = nullptr;
    W4A16_TRY(device_info(&dev));
    *bytes = kv_attention_workspace(n_heads, n_kv_heads, head_dim, n_seqs, n_tokens, *dev);
    return W4A16_OK;
}

int w4a16_kv_copy_pages(const w4a16_kv_cache_t *cache, const int32_t *src, const int32_t *dst, int n,
                        w4a16_stream_t stream) {
    KvCache c;
    W4A16_TRY(check_cache(cache, &c));
    if (n < 0 || (long long)n * c.n_kv_heads >= (1LL << 31)) return W4A16_ERR_SHAPE;
    if (n == 0) return W4A16_OK;
    if (src == nullptr || dst == nullptr) return W4A16_ERR_NULL;
    if (!aligned(src, 4) || !aligned(dst, 4)) return W4A16_ERR_ALIGN;
    const DeviceInfo *dev = nullptr;
    W4A16_TRY(device_info(&dev));
    return done(launch_kv_copy_pages(c, src, dst, n, *dev, str(stream), pdl_enabled()));
}

int w4a16_kv_fork(const w4a16_kv_cache_t *cache, int32_t *block_table, int32_t *kv_lens, int n_seqs, int max_blocks,
                  int32_t *refcount, const int32_t *parents, const int32_t *children, int n, void *workspace,
                  long long workspace_bytes, w4a16_stream_t stream) {
    KvCache c;
    W4A16_TRY(check_cache(cache, &c));
    W4A16_TRY(check_table(block_table, kv_lens, n_seqs, max_blocks, cache->page_size));
    if (n < 0 || n > n_seqs) return W4A16_ERR_SHAPE;
    if (n == 0) return W4A16_OK;
    if (parents == nullptr || children == nullptr) return W4A16_ERR_NULL;
    if (!aligned(parents, 4) || !aligned(children, 4)) return W4A16_ERR_ALIGN;
    W4A16_TRY(check_pool(refcount, c.n_pages, workspace, workspace_bytes));
    const DeviceInfo *dev = nullptr;
    W4A16_TRY(device_info(&dev));
    return done(launch_kv_fork(c, block_table, kv_lens, n_seqs, max_blocks, refcount, parents, children, n, workspace,
                               *dev, str(stream), pdl_enabled()));
}

int w4a16_kv_free(int32_t *block_table, int32_t *kv_lens, int n_seqs, int max_blocks, int32_t *refcount, int n_pages,
                  const int32_t *seqs, int n, w4a16_stream_t stream) {
    W4A16_TRY(check_table(block_table, kv_lens, n_seqs, max_blocks, 1));
    if (n < 0 || n > n_seqs || n_pages <= 0) return W4A16_ERR_SHAPE;
    if (n == 0) return W4A16_OK;
    if (refcount == nullptr || seqs == nullptr) return W4A16_ERR_NULL;
    if (!aligned(refcount, 4) || !aligned(seqs, 4)) return W4A16_ERR_ALIGN;
    const DeviceInfo *dev = nullptr;
    W4A16_TRY(device_info(&dev));
    return done(launch_kv_free(block_table, kv_lens, n_seqs, max_blocks, refcount, n_pages, seqs, n, *dev, str(stream),
                               pdl_enabled()));
}

int w4a16_kv_trim(int32_t *block_table, const int32_t *kv_lens, int n_seqs, int max_blocks, int32_t *refcount,
                  int n_pages, int page_size, int window, int sinks, w4a16_stream_t stream) {
    if (shift_of(page_size) < 0 || n_pages <= 0) return W4A16_ERR_SHAPE;
    W4A16_TRY(check_table(block_table, kv_lens, n_seqs, max_blocks, page_size));
    if (window < 0 || sinks < 0) return W4A16_ERR_ARG;
    if (n_seqs == 0 || window == 0) return W4A16_OK;
    if (refcount == nullptr) return W4A16_ERR_NULL;
    if (!aligned(refcount, 4)) return W4A16_ERR_ALIGN;
    const DeviceInfo *dev = nullptr;
    W4A16_TRY(device_info(&dev));
    return done(launch_kv_trim(block_table, kv_lens, n_seqs, max_blocks, refcount, n_pages, page_size, window, sinks,
                               *dev, str(stream), pdl_enabled()));
}

int w4a16_kv_compact(const w4a16_kv_cache_t *cache, int32_t *block_table, int n_seqs, int max_blocks,
                     int32_t *refcount, int32_t *n_live_or_null, void *workspace, long long workspace_bytes,
                     w4a16_stream_t stream) {
    KvCache c;
    W4A16_TRY(check_cache(cache, &c));
    W4A16_TRY(check_table(block_table, block_table, n_seqs, max_blocks, cache->page_size));
    if (!aligned(n_live_or_null, 4)) return W4A16_ERR_ALIGN;
    W4A16_TRY(check_pool(refcount, c.n_pages, workspace, workspace_bytes));
    const DeviceInfo *dev = nullptr;
    W4A16_TRY(device_info(&dev));
    return done(launch_kv_compact(c, block_table, n_seqs, max_blocks, refcount, n_live_or_null, workspace, *dev,
                                  str(stream), pdl_enabled()));
}

int w4a16_kv_pool_workspace(int n_pages, long long *bytes) {
    if (bytes == nullptr) return W4A16_ERR_NULL;
    if (n_pages <= 0 || n_pages > (1 << 28)) return W4A16_ERR_SHAPE;
    *bytes = kv_pool_workspace(n_pages);
    return W4A16_OK;
}

}  // extern "C"
