"""Beam search over an attention block on 4-bit weights and an 8-bit cache, all of it on the device.

The prompts enter the cache (w4a16_kv_grow, w4a16_kv_append, w4a16_kv_attention) and every beam of a request takes over its
prompt's pages (w4a16_kv_reorder).  A step selects the best continuations (w4a16_beam_select), lets the cache's rows follow
them (w4a16_kv_reorder), makes room for a token of each beam, which copies the last pages that beams share (w4a16_kv_grow),
and runs the block on the tokens, the prompt's keys read once for all beams of a request (w4a16_kv_attention_shared), to the
next logits (w4a16_gemm).  Nothing of it comes to the host, so that a step is captured in a CUDA graph and replayed.

    python examples/beam_search.py

runs a few requests and prints the time of a step.  The block has random weights, one attention layer and no positions: the
tokens it finds mean nothing.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import w4a16_group_quantised_gb300 as w  # noqa: E402

INT = torch.int32


class Model:
    """Embeddings, the attention block's merged qkv and output projections and the head; 4 bits with a scale per group."""

    def __init__(self, hidden=2048, heads=16, kv_heads=4, dim=128, vocab=32000, G=128, dtype=torch.bfloat16, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.hidden, self.heads, self.kv_heads, self.dim, self.vocab, self.G = hidden, heads, kv_heads, dim, vocab, G

        def weight(n, k, gain=1.0):
            q = torch.randint(0, 16, (n, k), generator=g, device="cuda", dtype=torch.uint8)
            s = torch.empty((n, k // G), device="cuda").uniform_(0.5, 1.5, generator=g) * (gain * k ** -0.5 / 4.6)
            return w.w4a16_pack(q), s.to(dtype)

        self.embed = torch.randn((vocab, hidden), generator=g, device="cuda").to(dtype)
        self.qkv, self.out = weight((heads + 2 * kv_heads) * dim, hidden), weight(hidden, heads * dim)
        self.head = weight(vocab, hidden, 3.0)

    def linear(self, x, weight):
        return w.w4a16_gemm(x, *weight, None, self.G)

    def logits(self, x):
        """Of hidden rows, normed as a last layer's are."""
        x = x.float()
        return self.linear((x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)).to(self.embed.dtype), self.head)


class Search:
    """Requests with `width` beams each: rows [g * width, (g + 1) * width) of the tables are request g's."""

    def __init__(self, model, requests, width, pages, columns, page=16, store=torch.int8, end_token=2):
        m, rows = model, requests * width
        self.model, self.requests, self.width, self.rows, self.end_token = m, requests, width, rows, end_token
        codes = [torch.empty((pages, m.kv_heads, page, m.dim), dtype=store, device="cuda") for _ in range(2)]
        scales = [torch.empty((pages, m.kv_heads), device="cuda") for _ in range(2)]
        self.cache = w.KVCache(*codes, *scales)
        self.table = torch.full((rows, columns), -1, dtype=INT, device="cuda")
        self.lens, self.refcount = torch.zeros(rows, dtype=INT, device="cuda"), torch.zeros(pages, dtype=INT, device="cuda")
        self.ones = torch.ones(rows, dtype=INT, device="cuda")
        self.groups = torch.arange(0, rows + 1, width, dtype=INT, device="cuda")
        self.prefix = torch.zeros(requests, dtype=INT, device="cuda")

    def attend(self, x, starts, longest, groups=None):
        m = self.model
        q, k, v = m.linear(x, m.qkv).split([m.heads * m.dim, m.kv_heads * m.dim, m.kv_heads * m.dim], 1)
        k, v, q = (t.unflatten(1, (-1, m.dim)) for t in (k, v, q))
        w.w4a16_kv_append(self.cache, k, v, self.table, self.lens, starts)
        if groups is None:
            o = w.w4a16_kv_attention(q, self.cache, self.table, self.lens, starts, longest)
        else:
            o = w.w4a16_kv_attention_shared(q, self.cache, self.table, self.lens, starts, longest, groups, self.prefix)
        return x + m.linear(o.flatten(1), m.out)

    def begin(self, prompts):
        """The prompts (int64 tensors of tokens) through the block, each into its request's first row; then a beam that is
        alive and width - 1 that are not yet, on the prompt's pages."""
        new = torch.zeros(self.rows, dtype=INT)
        new[::self.width] = torch.tensor([len(p) for p in prompts], dtype=INT)
        tokens = torch.cat(prompts)
        starts, _, _ = w.w4a16_kv_grow(self.cache, self.table, self.lens, self.refcount, new.cuda(), len(tokens))
        x = self.attend(self.model.embed[tokens], starts, max(len(p) for p in prompts))
        last = starts[1::self.width].long() - 1
        self.logits = self.model.logits(x[last]).repeat_interleave(self.width, 0)
        self.prefix.copy_(self.lens[::self.width])
        src = torch.arange(0, self.rows, self.width, dtype=INT, device="cuda").repeat_interleave(self.width)
        w.w4a16_kv_reorder(self.table, self.lens, self.refcount, src)
        self.scores = torch.full((self.requests, self.width), -float("inf"), device="cuda")
        self.scores[:, 0] = 0.0
        self.scores = self.scores.flatten()
        self.finished = torch.zeros(self.rows, dtype=torch.bool, device="cuda")

    def step(self):
        """One token of every beam; returns (rows that the beams continue, tokens), [requests, width]."""
        scores, src, tokens, finished = w.w4a16_beam_select(self.logits, self.scores, self.width, self.width,
                                                            finished=self.finished, end_token=self.end_token)
        w.w4a16_kv_reorder(self.table, self.lens, self.refcount, src.flatten())
        starts, _, _ = w.w4a16_kv_grow(self.cache, self.table, self.lens, self.refcount, self.ones, self.rows)
        x = self.attend(self.model.embed[tokens.flatten().clamp(min=0).long()], starts, 1, self.groups)
        self.logits.copy_(self.model.logits(x))
        self.scores.copy_(scores.flatten())
        self.finished.copy_(finished.flatten())
        return src, tokens


def best(steps, scores, width):
    """The best beam's tokens of each request, from what the steps returned (rows and tokens, on the host)."""
    out = []
    for g in range(scores.shape[0] // width):
        row, tokens = g * width + int(scores[g * width:(g + 1) * width].argmax()), []
        for src, tok in reversed(steps):
            tokens.append(int(tok.flatten()[row]))
            row = int(src.flatten()[row])
        out.append(tokens[::-1])
    return out


def main():
    model = Model()
    search = Search(model, requests=4, width=4, pages=2048, columns=160)
    g = torch.Generator(device="cuda").manual_seed(1)
    prompts = [torch.randint(0, model.vocab, (n,), generator=g, device="cuda") for n in (1920, 128, 777, 1500)]
    search.begin(prompts)
    steps = [tuple(t.clone() for t in search.step()) for _ in range(3)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = search.step()
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    for _ in range(32):
        graph.replay()
        steps.append(tuple(t.clone() for t in captured))
    b.record()
    torch.cuda.synchronize()
    if w.w4a16_last_device_error() != 0:
        raise RuntimeError(f"device status {w.w4a16_last_device_error()}")
    found = best([(s.cpu(), t.cpu()) for s, t in steps], search.scores.cpu(), search.width)
    print(f"{search.rows} beams, a step {a.elapsed_time(b) / 32 * 1e3:.0f} us; pages in use {int((search.refcount > 0).sum())}, "
          f"best scores {[round(float(x), 2) for x in search.scores.view(-1, search.width).max(1).values]}, "
          f"tokens of the first {found[0][:8]} ...")


if __name__ == "__main__":
    main()
