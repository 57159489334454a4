// kv_pages.cu -- page pool of the paged cache: copy, fork, free, trim, compact.
//
// All of it is integer bookkeeping on the device (no count reaches the host),
// plus page copies, which are bound by memory: 2 bytes of traffic per byte of
// page.  Which free page goes to whom is fixed by rank (the r-th free page in
// ascending order), so results do not depend on the order of CTAs; counts
// change by integer atomics, whose order does not show.
//
// Measured (8 kv heads, 128 dims): 3001 pages of 16 copied in 32 us, 0.90 of a
// copy's bandwidth.  16 prompts forked to 8 sequences each: 6.5 us, two short
// launches.  Freeing 40 of 96 sequences, trimming the rest to a window and
// compacting: 68 us, of them 49 the moves (44 at a copy's bandwidth), the rest
// four short launches.
#include "kv.cuh"

#include <algorithm>

namespace w4a16 {
namespace {

constexpr int kChunk = 1024;     // pages of a bitmap chunk
constexpr int kCopyThreads = 256;

// Copy part `part` of `parts` of page src to page dst, both codes and (part
// 0) scales.  16-byte pieces, head by head; four of K and four of V in flight
// per thread.
__device__ __forceinline__ void copy_page(const KvCache &c, int src, int dst, int part, int parts) {
    const int vecs = c.head_dim / 16, per_head = vecs << c.page_shift;
    const int pieces = c.n_kv_heads * per_head;
    const uint8_t *ks = c.k + src * c.page_stride, *vs = c.v + src * c.page_stride;
    uint8_t *kd = c.k + dst * c.page_stride, *vd = c.v + dst * c.page_stride;
    const bool by_head = c.head_stride >= c.token_stride;
    const int hi = by_head ? per_head : c.n_kv_heads * vecs;
    for (int base = part * 4 * (int)blockDim.x; base < pieces; base += parts * 4 * (int)blockDim.x) {
        long long off[4];
        uint4 a[4], b[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int i = base + j * (int)blockDim.x + (int)threadIdx.x;
            off[j] = -1;
            if (i < pieces) {
                const int outer = i / hi, mid = i % hi / vecs;
                off[j] = (by_head ? outer : mid) * c.head_stride + (by_head ? mid : outer) * c.token_stride +
                         i % vecs * 16;
                a[j] = *reinterpret_cast<const uint4 *>(ks + off[j]);
                b[j] = *reinterpret_cast<const uint4 *>(vs + off[j]);
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (off[j] >= 0) {
                *reinterpret_cast<uint4 *>(kd + off[j]) = a[j];
                *reinterpret_cast<uint4 *>(vd + off[j]) = b[j];
            }
    }
    if (part == 0)
        for (int h = threadIdx.x; h < c.n_kv_heads; h += blockDim.x) {
            const long long s = (long long)src * c.n_kv_heads + h, d = (long long)dst * c.n_kv_heads + h;
            c.k_scale[d] = c.k_scale[s];
            c.v_scale[d] = c.v_scale[s];
        }
}

// CTAs that share one page's copy: each moves a few thousand pieces.
int copy_parts(const KvCache &c) {
    const long long pieces = (long long)c.n_kv_heads * (c.head_dim / 16) << c.page_shift;
    const long long parts = (pieces + 4 * kCopyThreads - 1) / (4 * kCopyThreads);
    return (int)(parts < 1 ? 1 : parts);
}

__global__ void copy_kernel(KvCache c, const int *src, const int *dst, int n, int parts, int *status) {
    kv_begin();
    const int i = blockIdx.x / parts, part = blockIdx.x % parts;
    const int s = src[i], d = dst[i];
    if (s < 0 || d < 0) return;
    if (s >= c.n_pages || d >= c.n_pages) {
        if (threadIdx.x == 0) kv_report(status);
        return;
    }
    if (s != d) copy_page(c, s, d, part, parts);
}

// Bitmap of the pages whose count is (not) zero, and its population by chunk.
// One CTA of 1024 threads per chunk.
__global__ void bitmap_kernel(const int *refcount, int n_pages, int want_free, uint32_t *bits, int *counts) {
    kv_begin();
    __shared__ int s_count[32];
    const int p = blockIdx.x * kChunk + threadIdx.x;
    const bool set = p < n_pages && ((refcount[p] == 0) == (want_free != 0));
    const uint32_t w = __ballot_sync(0xffffffffu, set);
    if ((threadIdx.x & 31) == 0) {
        bits[p >> 5] = w;
        s_count[threadIdx.x >> 5] = __popc(w);
    }
    __syncthreads();
    if (threadIdx.x < 32) {
        const int t = __reduce_add_sync(0xffffffffu, s_count[threadIdx.x]);
        if (threadIdx.x == 0) counts[blockIdx.x] = t;
    }
}

// Sum over the CTA (every thread gets it).
__device__ __forceinline__ int block_sum(int v, int *scratch) {
    v = __reduce_add_sync(0xffffffffu, v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
    __syncthreads();
    int t = 0;
    for (int w = 0; w < (int)blockDim.x / 32; ++w) t += scratch[w];
    return t;
}

// Sum of the threads before this one; *total gets the CTA's sum.
__device__ __forceinline__ int block_before(int v, int *scratch, int *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int inc = v;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const int o = __shfl_up_sync(0xffffffffu, inc, d);
        if (lane >= d) inc += o;
    }
    __syncthreads();
    if (lane == 31) scratch[warp] = inc;
    __syncthreads();
    int ahead = 0, all = 0;
    for (int w = 0; w < (int)blockDim.x / 32; ++w) {
        const int t = scratch[w];
        all += t;
        ahead += w < warp ? t : 0;
    }
    *total = all;
    return ahead + inc - v;
}

// The r-th set bit (from 0) of the bitmap, or -1: every thread of the CTA
// calls.  The chunk that holds it, then its word, then the bit: at each level
// the one thread whose range of ranks contains r goes on.
__device__ int select_bit(const uint32_t *bits, const int *counts, int n_chunks, int r, int *scratch) {
    __shared__ int s_chunk, s_rank, s_at;
    if (threadIdx.x == 0) s_chunk = -1;
    for (int base = 0; base < n_chunks; base += blockDim.x) {
        const int i = base + threadIdx.x;
        const int v = i < n_chunks ? counts[i] : 0;
        int total;
        const int before = block_before(v, scratch, &total);
        if (r >= before && r < before + v) {
            s_chunk = i;
            s_rank = r - before;
        }
        if (r < total) break;
        r -= total;
    }
    __syncthreads();
    if (s_chunk < 0) return -1;
    const uint32_t word = threadIdx.x < kChunk / 32 ? bits[s_chunk * (kChunk / 32) + threadIdx.x] : 0;
    int total;
    const int before = block_before(__popc(word), scratch, &total);
    int left = s_rank - before;
    if (left >= 0 && left < __popc(word)) {
        uint32_t m = word;
        for (; left > 0; --left) m &= m - 1;
        s_at = s_chunk * kChunk + (int)threadIdx.x * 32 + __ffs(m) - 1;
    }
    __syncthreads();
    return s_at;
}

// `parts` CTAs per child: each finds the child's page, the first of them also
// writes the tables and counts, and each copies its part of the page.
__global__ void fork_kernel(KvCache c, int *table, int *lens, int n_seqs, int max_blocks, int *refcount,
                            const int *parents, const int *children, int n, int parts,
                            const uint32_t *free_bits, const int *free_counts, int *status) {
    kv_begin();
    __shared__ int scratch[32];
    const int shift = c.page_shift, part_mask = (1 << shift) - 1;
    const int me = blockIdx.x / parts, part = blockIdx.x % parts;
    const int par = parents[me], chi = children[me];
    if (par < 0 || par >= n_seqs || chi < 0 || chi >= n_seqs) {
        if (threadIdx.x == 0) kv_report(status);
        return;
    }
    const int cap = max_blocks << shift;
    const int said = lens[par], len = min(max(said, 0), cap);
    const int full = len >> shift;
    const int *from = table + (long long)par * max_blocks;
    // a partly filled last page is copied; where the parent's is not there, the child has none either
    const bool tail = (len & part_mask) != 0;
    const int src = tail ? from[full] : -1;
    const bool takes = src >= 0 && src < c.n_pages;
    int fresh = -1;
    if (takes) {
        int before = 0;                                  // children ahead of this one that take a page
        for (int j = threadIdx.x; j < me; j += blockDim.x) {
            const int p = parents[j], ch = children[j];
            if (p < 0 || p >= n_seqs || ch < 0 || ch >= n_seqs) continue;
            const int l = min(max(lens[p], 0), cap);
            if ((l & part_mask) == 0) continue;
            const int last = table[(long long)p * max_blocks + (l >> shift)];
            before += last >= 0 && last < c.n_pages;
        }
        before = block_sum(before, scratch);
        fresh = select_bit(free_bits, free_counts, (c.n_pages + kChunk - 1) / kChunk, before, scratch);
    }
    const bool ok = !takes || fresh >= 0;
    int *to = table + (long long)chi * max_blocks;
    for (int k = threadIdx.x; part == 0 && k < max_blocks; k += blockDim.x) {
        int p = -1;
        if (ok && k < full) {
            p = from[k];
            if (p >= c.n_pages) {
                kv_report(status);
                p = -1;
            }
            if (p >= 0) atomicAdd(refcount + p, 1);      // a trimmed entry (-1) stays one
        } else if (k == full) {
            p = fresh;
        }
        to[k] = p;
    }
    if (part == 0 && threadIdx.x == 0) {
        lens[chi] = ok ? len : 0;
        if (!ok || (tail && !takes) || len != said) kv_report(status);
        if (fresh >= 0) refcount[fresh] = 1;
    }
    if (fresh >= 0) copy_page(c, src, fresh, part, parts);
}

// A table entry that named page p is gone: its count goes down.
__device__ __forceinline__ void drop_page(int p, int *refcount, int n_pages, int *status) {
    if (p < 0) return;
    if (p >= n_pages) {
        kv_report(status);
    } else if (atomicSub(refcount + p, 1) <= 0) {        // was free already
        atomicAdd(refcount + p, 1);
        kv_report(status);
    }
}

__global__ void free_kernel(int *table, int *lens, int n_seqs, int max_blocks, int *refcount, int n_pages,
                            const int *seqs, int *status) {
    kv_begin();
    const int i = seqs[blockIdx.x];
    if (i < 0 || i >= n_seqs) {
        if (threadIdx.x == 0) kv_report(status);
        return;
    }
    // a sequence listed twice: whoever takes the page id out of an entry lowers the count
    for (int k = threadIdx.x; k < max_blocks; k += blockDim.x)
        drop_page(atomicExch(table + (long long)i * max_blocks + k, -1), refcount, n_pages, status);
    if (threadIdx.x == 0) lens[i] = 0;
}

__global__ void trim_kernel(int *table, const int *lens, int max_blocks, int *refcount, int n_pages, int shift,
                            int window, int sinks, int *status) {
    kv_begin();
    const int i = blockIdx.x, ps = 1 << shift;
    const int said = lens[i], len = min(max(said, 0), max_blocks << shift);
    if (len != said && threadIdx.x == 0) kv_report(status);
    // blocks [lo, hi) lie whole in positions [sinks, len - window + 1)
    const int lo = (int)(((long long)sinks + ps - 1) >> shift);
    const int hi = max(len - window + 1, 0) >> shift;
    for (int k = lo + threadIdx.x; k < hi; k += blockDim.x) {
        int *e = table + (long long)i * max_blocks + k;
        const int p = *e;
        if (p >= 0) *e = -1;
        drop_page(p, refcount, n_pages, status);
    }
}

struct CompactScratch {
    uint32_t *bits;      // pages in use
    int *counts;         // of each chunk
    int *src, *dst;      // the moves, by rank
    int *rank;           // of each page that moves, among those
    int *n_moves;
};

__host__ __device__ inline long long round16(long long v) { return (v + 15) & ~15LL; }

CompactScratch compact_scratch(void *ws, int n_pages) {
    const long long chunks = (n_pages + kChunk - 1) / kChunk;
    char *p = static_cast<char *>(ws);
    CompactScratch s;
    auto take = [&](long long bytes) {
        char *q = p;
        p += round16(bytes);
        return q;
    };
    s.n_moves = reinterpret_cast<int *>(take(16));
    s.counts = reinterpret_cast<int *>(take(chunks * 4));
    s.bits = reinterpret_cast<uint32_t *>(take(chunks * kChunk / 8));
    s.src = reinterpret_cast<int *>(take((long long)n_pages * 4));
    s.dst = reinterpret_cast<int *>(take((long long)n_pages * 4));
    s.rank = reinterpret_cast<int *>(take((long long)n_pages * 4));
    return s;
}

// With m pages in use: the in-use pages at m and above by rank, and the free
// pages below m by rank.  Both lists have the same length.
__global__ void plan_kernel(CompactScratch w, int n_pages, int *n_live) {
    kv_begin();
    __shared__ int scratch[32];
    __shared__ int s_words[kChunk / 32];
    const int n_chunks = (n_pages + kChunk - 1) / kChunk;
    int before = 0, all = 0;
    for (int i = threadIdx.x; i < n_chunks; i += blockDim.x) {
        const int v = w.counts[i];
        all += v;
        before += i < (int)blockIdx.x ? v : 0;
    }
    before = block_sum(before, scratch);
    const int m = block_sum(all, scratch);
    // in-use pages below m: whole chunks, then the words of the chunk that holds m (none when m is all chunks' end; a
    // full pool's m is in its last chunk unless that is full too)
    int below = 0;
    for (int i = threadIdx.x; i < min(m / kChunk, n_chunks); i += blockDim.x) below += w.counts[i];
    const int w0 = m / kChunk * (kChunk / 32), wm = m >> 5;
    if (m < n_chunks * kChunk) {
        for (int i = w0 + threadIdx.x; i < wm; i += blockDim.x) below += __popc(w.bits[i]);
        if (threadIdx.x == 0) below += __popc(w.bits[wm] & ((1u << (m & 31)) - 1));
    }
    below = block_sum(below, scratch);
    const int p = blockIdx.x * kChunk + threadIdx.x;
    const uint32_t word = w.bits[p >> 5];
    if ((threadIdx.x & 31) == 0) s_words[threadIdx.x >> 5] = __popc(word);
    __syncthreads();
    int live = before;                                   // in-use pages before p
    for (int i = 0; i < (int)threadIdx.x / 32; ++i) live += s_words[i];
    live += __popc(word & ((1u << (threadIdx.x & 31)) - 1));
    if (p < n_pages) {
        const bool in_use = (word >> (threadIdx.x & 31)) & 1;
        if (in_use && p >= m) {
            w.src[live - below] = p;
            w.rank[p] = live - below;
        } else if (!in_use && p < m) {
            w.dst[p - live] = p;
        }
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        *w.n_moves = m - below;
        if (n_live) *n_live = m;
    }
}

// The first `movers` CTAs copy pages and their counts, the others rename
// table entries.  m (the pages in use) = below + moves is not needed: an
// entry moves iff its page is in the list under its own rank.
__global__ void move_kernel(KvCache c, CompactScratch w, int *table, long long entries, int *refcount, int movers,
                            int parts, int *status) {
    kv_begin();
    const int moves = *w.n_moves;
    if ((int)blockIdx.x < movers) {
        for (long long i = blockIdx.x; i < (long long)moves * parts; i += movers) {
            const int r = (int)(i / parts), part = (int)(i % parts);
            const int s = w.src[r], d = w.dst[r];
            copy_page(c, s, d, part, parts);
            if (part == 0 && threadIdx.x == 0) {
                refcount[d] = refcount[s];
                refcount[s] = 0;
            }
        }
        return;
    }
    const long long stride = (long long)(gridDim.x - movers) * blockDim.x;
    for (long long i = (long long)(blockIdx.x - movers) * blockDim.x + threadIdx.x; i < entries; i += stride) {
        const int p = table[i];
        if (p < 0) continue;
        if (p >= c.n_pages) {
            kv_report(status);
            continue;
        }
        // rank[] is written only for pages that move; elsewhere it holds anything
        const int r = w.rank[p];
        if (r >= 0 && r < moves && w.src[r] == p) table[i] = w.dst[r];
    }
}

}  // namespace

cudaError_t launch_kv_copy_pages(const KvCache &c, const int *src, const int *dst, int n, const DeviceInfo &dev,
                                 cudaStream_t s, bool pdl) {
    const int parts = copy_parts(c);
    return kv_launch(copy_kernel, dim3((unsigned)n * parts), dim3(kCopyThreads), 0, s, pdl, c, src, dst, n, parts,
                     dev.status);
}

cudaError_t launch_kv_fork(const KvCache &c, int *table, int *lens, int n_seqs, int max_blocks, int *refcount,
                           const int *parents, const int *children, int n, void *workspace, const DeviceInfo &dev,
                           cudaStream_t s, bool pdl) {
    const CompactScratch w = compact_scratch(workspace, c.n_pages);
    const cudaError_t e = kv_launch(bitmap_kernel, dim3((c.n_pages + kChunk - 1) / kChunk), dim3(kChunk), 0, s, pdl,
                                    refcount, c.n_pages, 1, w.bits, w.counts);
    if (e != cudaSuccess) return e;
    const int parts = std::min(copy_parts(c), 4);
    return kv_launch(fork_kernel, dim3((unsigned)n * parts), dim3(kCopyThreads), 0, s, pdl, c, table, lens, n_seqs,
                     max_blocks, refcount, parents, children, n, parts, w.bits, w.counts, dev.status);
}

cudaError_t launch_kv_free(int *table, int *lens, int n_seqs, int max_blocks, int *refcount, int n_pages,
                           const int *seqs, int n, const DeviceInfo &dev, cudaStream_t s, bool pdl) {
    return kv_launch(free_kernel, dim3(n), dim3(512), 0, s, pdl, table, lens, n_seqs, max_blocks, refcount, n_pages,
                     seqs, dev.status);
}

cudaError_t launch_kv_trim(int *table, const int *lens, int n_seqs, int max_blocks, int *refcount, int n_pages,
                           int page_size, int window, int sinks, const DeviceInfo &dev, cudaStream_t s, bool pdl) {
    return kv_launch(trim_kernel, dim3(n_seqs), dim3(512), 0, s, pdl, table, lens, max_blocks, refcount, n_pages,
                     kv_log2(page_size), window, sinks, dev.status);
}

cudaError_t launch_kv_compact(const KvCache &c, int *table, int n_seqs, int max_blocks, int *refcount, int *n_live,
                              void *workspace, const DeviceInfo &dev, cudaStream_t s, bool pdl) {
    const CompactScratch w = compact_scratch(workspace, c.n_pages);
    const int chunks = (c.n_pages + kChunk - 1) / kChunk;
    cudaError_t e = kv_launch(bitmap_kernel, dim3(chunks), dim3(kChunk), 0, s, pdl, refcount, c.n_pages, 0, w.bits,
                              w.counts);
    if (e != cudaSuccess) return e;
    e = kv_launch(plan_kernel, dim3(chunks), dim3(kChunk), 0, s, pdl, w, c.n_pages, n_live);
    if (e != cudaSuccess) return e;
    const int parts = copy_parts(c);
    const long long entries = (long long)n_seqs * max_blocks;
    const long long most = ((long long)c.n_pages + 1) / 2 * parts;
    const int movers = (int)std::min<long long>(most, (long long)dev.sm_count * 8);
    const int renamers = (int)std::min<long long>((entries + kCopyThreads - 1) / kCopyThreads, dev.sm_count);
    return kv_launch(move_kernel, dim3(movers + renamers), dim3(kCopyThreads), 0, s, pdl, c, w, table, entries,
                     refcount, movers, parts, dev.status);
}

long long kv_pool_workspace(int n_pages) {
    const long long chunks = (n_pages + kChunk - 1) / kChunk;
    return 16 + round16(chunks * 4) + round16(chunks * kChunk / 8) + 3 * round16((long long)n_pages * 4);
}

}  // namespace w4a16
