"""The attention block of a decoder layer on 4-bit weights and an 8-bit cache.

Per step, for a batch of sequences: the qkv projection (w4a16_gemm), the new
keys and values quantised into the cache's pages (w4a16_kv_append), attention
over the cache with a sliding window and sink tokens (w4a16_kv_attention), the
output projection (w4a16_gemm).  Between steps, the pages: a prompt continued
in several sequences (w4a16_kv_fork), pages that left the window given back
(w4a16_kv_trim), finished sequences freed (w4a16_kv_free) and the pool closed
up (w4a16_kv_compact).

    python examples/decoder_attention.py

runs prompts, forks them, decodes, and prints the time of a step.  Positions
are not encoded here: a rotary embedding would go between the projection and
the append.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import w4a16_group_quantised_gb300 as w  # noqa: E402


class Block:
    """Weights of one attention block: merged qkv and output projections, 4 bits with a scale per group."""

    def __init__(self, hidden=4096, heads=32, kv_heads=8, dim=128, G=128, dtype=torch.bfloat16, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.hidden, self.heads, self.kv_heads, self.dim, self.G = hidden, heads, kv_heads, dim, G

        def weight(n, k):
            q = torch.randint(0, 16, (n, k), generator=g, device="cuda", dtype=torch.uint8)
            s = torch.empty((n, k // G), device="cuda").uniform_(0.5, 1.5, generator=g) * (k ** -0.5 / 4.6)
            return q, w.w4a16_pack(q), s.to(dtype)

        self.qkv_codes, self.qkv, self.qkv_scales = weight((heads + 2 * kv_heads) * dim, hidden)
        self.out_codes, self.out, self.out_scales = weight(hidden, heads * dim)


class Sequences:
    """A page pool and the sequences in it.  The host keeps lengths and hands out pages; the rest is on the device."""

    def __init__(self, block, rows, pages, width, page=16, store=torch.int8):
        codes = [torch.empty((pages, block.kv_heads, page, block.dim), dtype=store, device="cuda") for _ in range(2)]
        scales = [torch.empty((pages, block.kv_heads), device="cuda") for _ in range(2)]
        self.cache, self.page = w.KVCache(*codes, *scales), page
        self.table = torch.full((rows, width), -1, dtype=torch.int32, device="cuda")
        self.refcount = torch.zeros(pages, dtype=torch.int32, device="cuda")
        self.lens = [0] * rows

    def device_lens(self):
        return torch.tensor(self.lens, dtype=torch.int32, device="cuda")

    def extend(self, new):
        """Room for new[b] more tokens of each sequence: pages from the free ones, lowest first."""
        free = torch.nonzero(self.refcount == 0)[:, 0].int()
        at = 0
        for b, n in enumerate(new):
            first, last = -(-self.lens[b] // self.page), -(-(self.lens[b] + n) // self.page)
            take = free[at:at + last - first]
            if len(take) < last - first:
                raise RuntimeError("the pool is out of pages")
            self.table[b, first:last] = take
            self.refcount[take.long()] = 1
            at += last - first
            self.lens[b] += n

    def fork(self, parent, children):
        """Rows `children` continue row `parent`, which they share all full pages with."""
        lens = self.device_lens()
        w.w4a16_kv_fork(self.cache, self.table, lens, self.refcount,
                        torch.full((len(children),), parent, dtype=torch.int32, device="cuda"),
                        torch.tensor(children, dtype=torch.int32, device="cuda"))
        for c in children:
            self.lens[c] = self.lens[parent]

    def free(self, rows):
        w.w4a16_kv_free(self.table, self.device_lens(), self.refcount, torch.tensor(rows, dtype=torch.int32, device="cuda"))
        for r in rows:
            self.lens[r] = 0

    def close_up(self, window, sinks):
        """Give back what no later token sees, and move the pages in use to the front of the pool."""
        w.w4a16_kv_trim(self.table, self.device_lens(), self.refcount, self.page, window=window, sinks=sinks)
        w.w4a16_kv_compact(self.cache, self.table, self.refcount)


def step(block, seqs, x, new, window=0, sinks=0):
    """One pass of the block: x holds new[b] tokens of each sequence b, one after another; the same rows come back."""
    seqs.extend(new)
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    lens = seqs.device_lens()
    starts = torch.tensor(starts, dtype=torch.int32, device="cuda")
    qkv = w.w4a16_gemm(x, block.qkv, block.qkv_scales, None, block.G)
    q, k, v = qkv.split([block.heads * block.dim, block.kv_heads * block.dim, block.kv_heads * block.dim], 1)
    k, v = k.unflatten(1, (block.kv_heads, block.dim)), v.unflatten(1, (block.kv_heads, block.dim))
    w.w4a16_kv_append(seqs.cache, k, v, seqs.table, lens, starts)
    o = w.w4a16_kv_attention(q.unflatten(1, (block.heads, block.dim)), seqs.cache, seqs.table, lens, starts, max(new),
                             window=window, sinks=sinks)
    return w.w4a16_gemm(o.flatten(1), block.out, block.out_scales, None, block.G), o


def normed(x):
    """Rows of unit mean square: what a layer's norm would hand on."""
    return (x.float() * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + 1e-6)).to(x.dtype)


def main():
    block = Block()
    prompts, samples, window, sinks = 4, 4, 1024, 4
    seqs = Sequences(block, rows=prompts * samples, pages=4096, width=256)
    g = torch.Generator(device="cuda").manual_seed(1)

    def tokens(n):
        return torch.randn((n, block.hidden), generator=g, device="cuda").to(torch.bfloat16)

    new = [1920, 128, 777, 1500] + [0] * (prompts * samples - prompts)
    step(block, seqs, tokens(sum(new)), new, window, sinks)
    for p in range(prompts):
        seqs.fork(p, [prompts + p * (samples - 1) + i for i in range(samples - 1)])
    ones = [1] * (prompts * samples)
    x = tokens(len(ones))
    for _ in range(8):
        x = normed(step(block, seqs, x, ones, window, sinks)[0])
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    for _ in range(32):
        x = normed(step(block, seqs, x, ones, window, sinks)[0])
    b.record()
    torch.cuda.synchronize()
    used = int((seqs.refcount > 0).sum())
    seqs.free(list(range(prompts, prompts * samples)))
    seqs.close_up(window, sinks)
    left = int((seqs.refcount > 0).sum())
    if w.w4a16_last_device_error() != 0:
        raise RuntimeError(f"device status {w.w4a16_last_device_error()}")
    print(f"{len(ones)} sequences, a step of the block {a.elapsed_time(b) / 32 * 1e3:.0f} us with its host work; "
          f"pages in use {used}, after the samples ended {left}, output finite: {bool(torch.isfinite(x.float()).all())}")


if __name__ == "__main__":
    main()
