"""Cases of the operators for batches that share what they have cached: parallel
samples and beams of a prompt, users of one system prompt.

  attention  attention of each sequence's newest tokens over the paged 8-bit
             cache, where groups of sequences have their first pages in common
  grow       room for new tokens: block tables, row starts, positions and slots
             of the tokens, from how many each sequence brings; a partly filled
             last page that several sequences name is copied for all but one
  select     beam search's selection: the best continuations of each request
             over its beams and the vocabulary
  reorder    the cache's sequences follow the selection

The cache: codes in 8 bits (int8, or e4m3) of shape [pages, kv heads, tokens of
a page, head dim], and one fp32 scale for each page and kv head; a value is
code * scale.  `own` false computes the plain form (elementary torch operations
in 32 bits, the selection in 64, rounded once); `own` true calls the framework.
"""
import math
import random

import torch

own = False

ACT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
STORE = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}


# ------------------------------------------------------------------ cases
def _attn(name, **kw):
    c = {"name": name, "op": "attention", "groups": 1, "members_lo": 4, "members_hi": 4, "prefix_lo": 0, "prefix_hi": 0,
         "past_lo": 0, "past_hi": 0, "new_lo": 1, "new_hi": 1, "heads": 32, "kv_heads": 8, "dim": 128, "page": 16,
         "act": "bf16", "store": "int8", "layout": "heads", "mix": 1}
    c.update(kw)
    return c


def _grow(name, **kw):
    c = {"name": name, "op": "grow", "groups": 1, "members": 1, "past_lo": 0, "past_hi": 0, "new_lo": 1, "new_hi": 1,
         "kv_heads": 8, "dim": 128, "page": 16, "store": "int8", "layout": "heads", "mix": 1}
    c.update(kw)
    return c


def _select(name, **kw):
    c = {"name": name, "op": "select", "groups": 1, "width": 4, "n_out": 4, "vocab": 32000, "act": "f32", "first": False,
         "ended": 0.0, "end": 2, "pad": 0, "mix": 1}
    c.update(kw)
    return c


def _reorder(name, **kw):
    c = {"name": name, "op": "reorder", "groups": 1, "width": 4, "prefix_lo": 0, "prefix_hi": 0, "past_lo": 0, "past_hi": 0,
         "page": 16, "dead": 0.0, "mix": 1}
    c.update(kw)
    return c


def listed():
    return [
        # four beams of one request, a short prompt: the call's latency is all there is
        _attn("shared_1x4_beams", prefix_lo=901, prefix_hi=901, past_lo=5, past_hi=60, mix=1),
        # parallel samples of prompts of the prefill workload's lengths, some way into their answers
        _attn("shared_16x8_samples", groups=16, members_lo=3, members_hi=8, prefix_lo=100, prefix_hi=1920, past_lo=3,
              past_hi=500, mix=2),
        # a serving batch whose users all have one long system prompt; pages laid out token first
        _attn("shared_64_system_prompt", members_lo=64, members_hi=64, prefix_lo=8192, prefix_hi=8192, past_lo=1, past_hi=2000,
              page=64, act="f16", store="e4m3", layout="tokens", mix=3),
        # questions on two long documents, a few drafted tokens of each verified at a time, eight heads to a kv head
        _attn("shared_2x40_documents", groups=2, members_lo=24, members_hi=40, prefix_lo=20011, prefix_hi=32768, past_lo=20,
              past_hi=900, new_lo=1, new_hi=5, kv_heads=4, act="f16", page=32, mix=4),
        # the next token of one request's beams
        _grow("grow_1x4_beams", members=4, past_lo=950, past_hi=950, mix=5),
        # the next token of a serving batch, every request in four samples that share their last page
        _grow("grow_64x4_tokens", groups=64, members=4, past_lo=3, past_hi=4095, mix=6),
        # prompts of the prefill workload's lengths that enter the cache; pages laid out token first
        _grow("grow_64_prompts", groups=64, new_lo=17, new_hi=1920, page=64, store="e4m3", layout="tokens", mix=7),
        # the first step of one request: a single beam is alive
        _select("select_1x4_first", first=True, mix=8),
        # a batch of requests, twice as many continuations as beams, a vocabulary of odd size in rows that are padded
        _select("select_8x5_odd", groups=8, width=5, n_out=10, vocab=50001, act="f16", pad=15, mix=9),
        # a large batch and vocabulary, some beams have ended
        _select("select_64x4_large", groups=64, width=4, n_out=4, vocab=131072, act="bf16", ended=0.2, mix=10),
        # one request's beams
        _reorder("reorder_1x4", prefix_lo=901, prefix_hi=901, past_lo=5, past_hi=60, mix=11),
        # a large batch of wide beams over long prompts, some slots without a continuation
        _reorder("reorder_64x16", groups=64, width=16, prefix_lo=100, prefix_hi=8192, past_lo=1, past_hi=600, dead=0.05,
                 mix=12),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["samples", "samples", "system", "documents", "grow", "grow", "select", "select", "reorder"])
    mix = rng.randrange(1 << 30)
    page = rng.choice([16, 32, 64, 128])
    store, layout = rng.choice(["int8", "e4m3"]), rng.choice(["heads", "tokens"])
    heads, kv_heads = rng.choice([(32, 8), (32, 8), (32, 4), (28, 4), (32, 32), (8, 1)])
    dim = rng.choice([64, 128, 128])
    if op in ("samples", "system", "documents"):
        c = {"op": "attention", "heads": heads, "kv_heads": kv_heads, "dim": dim, "page": page, "act": rng.choice(["bf16", "f16"]),
             "store": store, "layout": layout, "mix": mix, "new_lo": 1, "new_hi": 1}
        if op == "samples":
            most = rng.randrange(2, 17)
            c.update(groups=_log(rng, 1, 16), members_lo=rng.choice([1, 2, most]), members_hi=most)
            prefix, past = _log(rng, 5, 8192), _log(rng, 1, 1000)
        elif op == "system":
            most = _log(rng, 2, 128)
            c.update(groups=1, members_lo=most, members_hi=most)
            prefix, past = _log(rng, 64, 32768), _log(rng, 1, 2000)
        else:
            most, new = _log(rng, 2, 40), rng.randrange(1, 40)
            c.update(groups=rng.randrange(1, 4), members_lo=max(1, most // 2), members_hi=most, new_lo=rng.choice([0, 1, new]),
                     new_hi=new)
            prefix, past = _log(rng, 1000, 32768), _log(rng, 1, 1000)
        # no more scores and no more cached values than the largest listed cases have
        while (c["groups"] * c["members_hi"] * c["new_hi"] * heads * (prefix + past) > 2 * 32 * 3 * 32 * 27000
               or (c["groups"] * (prefix + c["members_hi"] * (past + c["new_hi"]))) * kv_heads * dim > 160000 * 8 * 128):
            prefix, past = max(4, prefix * 3 // 4), max(1, past * 3 // 4)
            c["new_hi"] = max(1, c["new_hi"] * 3 // 4)
        c["members_lo"], c["new_lo"] = min(c["members_lo"], c["members_hi"]), min(c["new_lo"], c["new_hi"])
        c.update(prefix_lo=rng.choice([prefix // 4, prefix]), prefix_hi=prefix, past_lo=rng.choice([0, past // 2, past]),
                 past_hi=past)
        return c
    if op == "grow":
        new = rng.choice([1, rng.randrange(1, 9), _log(rng, 1, 1920)])
        past = rng.choice([0, _log(rng, 1, 4095)])
        c = {"op": "grow", "groups": _log(rng, 1, 64), "members": rng.choice([1, 1, 2, 4, 8]), "past_lo": rng.choice([0, past // 2]),
             "past_hi": past, "new_lo": rng.choice([0, 1, new]), "new_hi": new, "kv_heads": min(kv_heads, 8), "dim": dim,
             "page": page, "store": store, "layout": layout, "mix": mix}
        while c["groups"] * (c["past_hi"] + c["members"] * c["new_hi"]) > 64 * 4096:
            c["groups"] = max(1, c["groups"] * 2 // 3)
            c["past_hi"], c["new_hi"] = max(0, c["past_hi"] * 3 // 4), max(1, c["new_hi"] * 3 // 4)
        c["past_lo"], c["new_lo"] = min(c["past_lo"], c["past_hi"]), min(c["new_lo"], c["new_hi"])
        return c
    if op == "select":
        width = rng.choice([1, 2, 3, 4, 5, 8, 16])
        vocab = _log(rng, 30, 131072)
        c = {"op": "select", "groups": _log(rng, 1, 64), "width": width, "n_out": rng.choice([width, 2 * width, 1]),
             "vocab": vocab, "act": rng.choice(["bf16", "f16", "f32"]), "first": rng.random() < 0.15,
             "ended": rng.choice([0.0, 0.0, 0.3]), "end": rng.randrange(0, vocab), "pad": rng.choice([0, 0, 1, 64]), "mix": mix}
        size = 2 if c["act"] == "f32" else 1
        while c["groups"] * width * vocab * size > 64 * 4 * 131072:
            c["groups"] = max(1, c["groups"] // 2)
        return c
    width = _log(rng, 1, 16)
    prefix, past = _log(rng, 1, 8192), _log(rng, 1, 600)
    return {"op": "reorder", "groups": _log(rng, 1, 64), "width": width, "prefix_lo": prefix // 4, "prefix_hi": prefix,
            "past_lo": rng.choice([0, past]), "past_hi": past, "page": page, "dead": rng.choice([0.0, 0.1, 1.0]), "mix": mix}


# ------------------------------------------------------------------ lengths
class _Plan:
    """What the case alone fixes: members of each group, lengths, new tokens (plain lists)."""

    def __init__(self, c):
        r = random.Random(c["mix"])
        G = c["groups"]
        if c["op"] == "attention":
            count = [r.randint(c["members_lo"], c["members_hi"]) for _ in range(G)]
            count[-1] = c["members_hi"]
        else:
            count = [c["width"] if c["op"] == "reorder" else c["members"]] * G
        # a grown batch shares all that is cached, its partly filled last page included
        self.prefix = [r.randint(c["prefix_lo"], c["prefix_hi"]) if "prefix_lo" in c else r.randint(c["past_lo"], c["past_hi"])
                       for _ in range(G)]
        self.prefix[0] = c["prefix_hi"] if "prefix_hi" in c else c["past_hi"]
        self.first = [0]
        for n in count:
            self.first.append(self.first[-1] + n)
        self.group = [g for g, n in enumerate(count) for _ in range(n)]
        B = len(self.group)
        self.seqs = B
        past = [0] * B if c["op"] == "grow" else [r.randint(c["past_lo"], c["past_hi"]) for _ in range(B)]
        self.new = [r.randint(c["new_lo"], c["new_hi"]) if "new_lo" in c else 0 for _ in range(B)]
        if "new_hi" in c:
            self.new[-1] = c["new_hi"]
        self.past = [self.prefix[g] + p for g, p in zip(self.group, past)]
        ps = c["page"]
        # pages in common: full ones; for growth the last one too
        up = ps - 1 if c["op"] == "grow" else 0
        self.common = [(p + up) // ps for p in self.prefix]

    def shared(self, ps):
        """Positions that a group's sequences have in common and read together: whole pages before every new token, where
        two sequences or more bring any."""
        out = []
        for g, p in enumerate(self.prefix):
            past = [self.past[b] for b in range(self.first[g], self.first[g + 1]) if self.new[b] > 0]
            out.append(min([p] + past) // ps * ps if len(past) > 1 else 0)
        return out


def _starts(counts):
    s = [0]
    for n in counts:
        s.append(s[-1] + n)
    return s


def work(case):
    if case["op"] == "select":
        rows = case["groups"] * case["width"]
        if case["first"]:
            rows = case["groups"]
        rows -= int(rows * case["ended"])
        size = 4 if case["act"] == "f32" else 2
        return {"bytes": rows * case["vocab"] * size + case["groups"] * case["n_out"] * 13, "flops": 4 * rows * case["vocab"]}
    p, ps = _Plan(case), case["page"]
    if case["op"] == "attention":
        H, Hk, D = case["heads"], case["kv_heads"], case["dim"]
        shared = p.shared(ps)
        keys = sum(shared) + sum(a + n - shared[g] for a, n, g in zip(p.past, p.new, p.group) if n)
        pairs = sum(n * a + n * (n + 1) // 2 for a, n in zip(p.past, p.new))
        return {"bytes": 4 * sum(p.new) * H * D + keys * Hk * D * 2 + keys / ps * (8 * Hk + 4), "flops": 4 * pairs * H * D}
    if case["op"] == "grow":
        page_bytes = 2 * case["kv_heads"] * (ps * case["dim"] + 4)
        added = sum(-(-(a + n) // ps) - -(-a // ps) for a, n in zip(p.past, p.new))
        copied = shared = 0
        for g in range(case["groups"]):
            grows = sum(1 for b in range(p.first[g], p.first[g + 1]) if p.new[b] > 0)
            if p.prefix[g] % ps and grows:
                n = min(grows, p.first[g + 1] - p.first[g] - 1)
                copied, shared = copied + n, shared + (n > 0)
        # counts read, entries, lengths, starts, positions and slots written, shared last pages copied
        return {"bytes": (copied + shared) * page_bytes + 4 * _pool(p, case) + 8 * added + 16 * p.seqs + 12 * sum(p.new),
                "flops": 0}
    return {"bytes": 8 * sum(-(-a // ps) for a in p.past) + 12 * p.seqs, "flops": 0}


def _pool(p, c):
    """Pages of the pool: what the sequences hold, what growth adds, and some that are free."""
    ps = c["page"]
    own_pages = sum(-(-(a + n) // ps) - p.common[g] for a, n, g in zip(p.past, p.new, p.group))
    held = sum(p.common) + own_pages + (p.seqs if c["op"] == "grow" else 0)
    return held + max(4, held // 8)


# ------------------------------------------------------------------ inputs
def _rand_codes(shape, store, g):
    """Codes of roughly normal values, the largest of a block near the end of the range."""
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.float16)
    if store == "int8":
        return x.mul_(38.0).round_().clamp_(-127, 127).to(torch.int8)
    return x.mul_(120.0).clamp_(-448, 448).to(torch.float8_e4m3fn)


def _cache(case, pages, g):
    """Pages of codes with scales, as [pages, kv heads, tokens, dim] in memory order or with tokens outermost."""
    Hk, ps, D = case["kv_heads"], case["page"], case["dim"]
    unit = 1.0 / (38.0 if case["store"] == "int8" else 120.0)
    out = []
    for _ in range(2):
        if case["layout"] == "heads":
            out.append(_rand_codes((pages, Hk, ps, D), case["store"], g))
        else:
            out.append(_rand_codes((pages, ps, Hk, D), case["store"], g).permute(0, 2, 1, 3))
    for _ in range(2):
        out.append(torch.empty((pages, Hk), device="cuda").uniform_(0.6, 1.5, generator=g) * unit)
    return out


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _tables(p, c, pages, blocks, width, g):
    """Block table [sequences, width] of `blocks` pages a row, the groups' common ones first, drawn from all over the pool."""
    perm = torch.randperm(pages, generator=g, device="cuda", dtype=torch.int32)
    common, group = _ints(p.common).long(), _ints(p.group).long()
    first = torch.cumsum(common, 0) - common
    have = torch.minimum(common[group], _ints(blocks).long())
    rest = _ints(blocks).long() - have
    begin = common.sum() + torch.cumsum(rest, 0) - rest
    col = torch.arange(width, device="cuda")
    at = torch.where(col < have[:, None], first[group][:, None] + col, begin[:, None] + col - have[:, None])
    table = perm[at.clamp(max=pages - 1)]
    return torch.where(col < _ints(blocks)[:, None], table, torch.full_like(table, -1)).contiguous()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 1000003 + 29)
    s = {"case": case}
    if case["op"] == "select":
        return _prepare_select(s, case, g)
    p, ps = _Plan(case), case["page"]
    s["plan"] = p
    pages = _pool(p, case)
    if case["op"] == "attention":
        lens = [a + n for a, n in zip(p.past, p.new)]
        blocks = [-(-n // ps) for n in lens]
        s["k"], s["v"], s["ks"], s["vs"] = _cache(case, pages, g)
        s["table"] = _tables(p, case, pages, blocks, max(1, max(blocks)), g)
        s["lens"], s["starts"] = _ints(lens), _ints(_starts(p.new))
        s["groups"], s["prefix"], s["max_new"] = _ints(p.first), _ints(p.prefix), max(p.new)
        H, Hk, D = case["heads"], case["kv_heads"], case["dim"]
        # the rows of a merged qkv projection's output, of which q is a view
        qkv = torch.randn((sum(p.new), (H + 2 * Hk) * D), generator=g, device="cuda").to(ACT[case["act"]])
        s["q"] = qkv[:, :H * D].unflatten(1, (H, D))
        return s
    blocks = [-(-n // ps) for n in p.past]
    width = max(1, max(-(-(a + n) // ps) for a, n in zip(p.past, p.new)))
    table = _tables(p, case, pages, blocks, width, g)
    ref = torch.zeros(pages, dtype=torch.int32, device="cuda")
    named = table[table >= 0].long()
    ref.index_add_(0, named, torch.ones_like(named, dtype=torch.int32))
    # tables, lengths and counts as they are before a pass, and what a pass works on
    s["before"] = torch.cat([table.flatten(), _ints(p.past), ref])
    s["at"] = torch.empty_like(s["before"])
    n = table.numel()
    s["table"], s["lens"], s["ref"] = s["at"][:n].view(table.shape), s["at"][n:n + p.seqs], s["at"][n + p.seqs:]
    if case["op"] == "grow":
        s["k"], s["v"], s["ks"], s["vs"] = _cache(case, pages, g)
        s["new"], s["tokens"] = _ints(p.new), sum(p.new)
        return s
    # each slot continues some beam of its request, the better ones more often; some have none
    u = torch.rand((p.seqs,), generator=g, device="cuda")
    src = (u * u * case["width"]).int() + _ints([p.first[x] for x in p.group])
    dead = torch.rand((p.seqs,), generator=g, device="cuda") < case["dead"]
    s["src"] = torch.where(dead, torch.full_like(src, -1), src)
    return s


def _prepare_select(s, c, g):
    rows, V = c["groups"] * c["width"], c["vocab"]
    # logits of a language model: a broad bulk, a few tokens far above it, some tokens not allowed
    x = torch.randn((rows, V + c["pad"]), generator=g, device="cuda").mul_(2.3)
    some = torch.randint(0, V, (rows, 24), generator=g, device="cuda")
    x.scatter_add_(1, some, torch.empty((rows, 24), device="cuda").uniform_(2.0, 11.0, generator=g))
    banned = torch.randint(0, V, (rows, max(1, V // 50)), generator=g, device="cuda")
    x.scatter_(1, banned, -math.inf)
    if c["act"] != "f32":
        x = x.to(ACT[c["act"]])
    s["logits"] = x[:, :V]
    # cumulative log-probabilities, the best beam first
    steps = torch.empty((c["groups"], c["width"]), device="cuda").uniform_(0.0, 1.5, generator=g)
    score = -torch.empty((c["groups"], 1), device="cuda").uniform_(1.0, 40.0, generator=g) - torch.cumsum(steps, 1)
    if c["first"]:
        score[:, 0] = 0.0
        score[:, 1:] = -math.inf
    s["scores"] = score.flatten()
    s["finished"] = torch.rand((rows,), generator=g, device="cuda") < c["ended"]
    return s


# ------------------------------------------------------------------ one pass
def run(state):
    case = state["case"]
    form = _FRAMEWORK if own else _PLAIN
    return form[case["op"]](state, case)


def _codes(s):
    """The cache's buffers: page operators move codes and scales as they are."""
    return {"k": s["k"], "v": s["v"], "ks": s["ks"], "vs": s["vs"]}


def _own_attention(s, c):
    import w4a16_group_quantised_gb300 as w
    return w.w4a16_kv_attention_shared(s["q"], w.KVCache(s["k"], s["v"], s["ks"], s["vs"]), s["table"], s["lens"], s["starts"],
                                       s["max_new"], s["groups"], s["prefix"])


def _own_grow(s, c):
    import w4a16_group_quantised_gb300 as w
    s["at"].copy_(s["before"])
    starts, positions, slots = w.w4a16_kv_grow(w.KVCache(s["k"], s["v"], s["ks"], s["vs"]), s["table"], s["lens"], s["ref"],
                                               s["new"], s["tokens"])
    return {"table": s["table"], "lens": s["lens"], "ref": s["ref"], "starts": starts, "positions": positions, "slots": slots,
            **_codes(s)}


def _own_select(s, c):
    import w4a16_group_quantised_gb300 as w
    scores, rows, tokens, finished = w.w4a16_beam_select(s["logits"], s["scores"], c["width"], c["n_out"],
                                                         finished=s["finished"], end_token=c["end"])
    return {"scores": scores, "rows": rows, "tokens": tokens, "finished": finished}


def _own_reorder(s, c):
    import w4a16_group_quantised_gb300 as w
    s["at"].copy_(s["before"])
    w.w4a16_kv_reorder(s["table"], s["lens"], s["ref"], s["src"])
    return {"table": s["table"], "lens": s["lens"], "ref": s["ref"]}


_FRAMEWORK = {"attention": _own_attention, "grow": _own_grow, "select": _own_select, "reorder": _own_reorder}


# ------------------------------------------------------------------ the plain forms
def _bytes(t):
    return t.view(torch.int8)


def _values(codes, scales, pages):
    """fp32 values [..., kv heads, positions, dim] of the pages [..., blocks]."""
    x = _bytes(codes)[pages].view(codes.dtype).float() * scales[pages][..., None, None]
    return x.transpose(-4, -3).flatten(-3, -2)


def _places(starts, T):
    """Sequence of each token of the batch, and its number within the sequence."""
    tok = torch.arange(T, device="cuda")
    seq = torch.searchsorted(starts[1:].long(), tok, right=True)
    return seq, tok - starts.long()[seq]


def _plain_attention(s, c):
    H, Hk, D, ps, p = c["heads"], c["kv_heads"], c["dim"], c["page"], s["plan"]
    B, T, nq, G = p.seqs, s["q"].shape[0], s["max_new"], H // Hk
    seq, t = _places(s["starts"], T)
    q = torch.zeros((B, nq, H, D), device="cuda")
    q[seq, t] = s["q"].float()
    q = q.view(B, nq, Hk, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hk, G * nq, D)
    scale = 1.0 / math.sqrt(D)
    top = torch.full((B, Hk, G * nq, 1), -3.0e38, device="cuda")
    total, out = torch.zeros_like(top), torch.zeros_like(q)
    # the common pages, group by group: all of the group's rows at once
    shared = p.shared(ps)
    for g, n in enumerate(shared):
        if n == 0:
            continue
        lo, hi = p.first[g], p.first[g + 1]
        pages = s["table"][next(b for b in range(lo, hi) if p.new[b] > 0), :n // ps].long()
        k, v = _values(s["k"], s["ks"], pages), _values(s["v"], s["vs"], pages)
        rows = q[lo:hi].transpose(0, 1).reshape(Hk, (hi - lo) * G * nq, D)
        x = torch.matmul(rows, k.transpose(1, 2)).mul_(scale)
        m = x.amax(-1, keepdim=True)
        x = x.sub_(m).exp_()
        back = [y.view(Hk, hi - lo, G * nq, -1).transpose(0, 1) for y in (m, x.sum(-1, keepdim=True), torch.matmul(x, v))]
        top[lo:hi], total[lo:hi], out[lo:hi] = back
    # what is each sequence's own
    skip = _ints([shared[g] for g in p.group])
    rest = s["lens"] - skip
    n = max(1, max(a + m - shared[g] for a, m, g in zip(p.past, p.new, p.group)))
    col = (skip // ps).long()[:, None] + torch.arange(-(-n // ps), device="cuda")
    pages = s["table"].long().gather(1, col.clamp(max=s["table"].shape[1] - 1)).clamp(min=0)
    k = _values(s["k"], s["ks"], pages)
    j = torch.arange(k.shape[2], device="cuda")
    new = s["starts"][1:] - s["starts"][:-1]
    pos = (rest - new)[:, None] + torch.arange(nq, device="cuda")
    x = torch.matmul(q, k.transpose(2, 3)).mul_(scale).view(B, Hk, G, nq, -1)
    x = x.masked_fill_((j > pos[..., None])[:, None, None], -math.inf).view(B, Hk, G * nq, -1)
    del k
    m = torch.maximum(x.amax(-1, keepdim=True), top)
    x = x.sub_(m).exp_()
    v = _values(s["v"], s["vs"], pages).masked_fill((j >= rest[:, None])[:, None, :, None], 0.0)
    f = torch.exp(top - m)
    out = (out * f + torch.matmul(x, v)) / (total * f + x.sum(-1, keepdim=True)).clamp(min=1e-37)
    return out.view(B, Hk, G, nq, D).permute(0, 3, 1, 2, 4).reshape(B, nq, H, D)[seq, t].to(s["q"].dtype)


def _plain_grow(s, c):
    s["at"].copy_(s["before"])
    table, lens, ref, new, ps = s["table"], s["lens"], s["ref"], s["new"].long(), c["page"]
    B, before = table.shape[0], lens.long()
    after = before + new
    have, want = (before + ps - 1) // ps, (after + ps - 1) // ps
    # a partly filled last page: whoever grows while others name it too takes a copy, in the order of rows
    row = torch.arange(B, device="cuda")
    last = table[row, (before // ps).clamp(max=table.shape[1] - 1)].long()
    partial = (before % ps != 0) & (new > 0)
    same = partial[:, None] & partial[None] & (last[:, None] == last[None])
    rank = (same & (row[None] < row[:, None])).sum(1)
    copies = partial & (ref[last.clamp(min=0)] - rank > 1)
    need = want - have + copies
    ends = torch.cumsum(need, 0)
    free = torch.nonzero(ref == 0)[:, 0]
    col = torch.arange(table.shape[1], device="cuda")
    start = have - copies.long()
    takes = (col >= start[:, None]) & (col < want[:, None])
    fresh = free[((ends - need)[:, None] + col - start[:, None]).clamp(0, free.shape[0] - 1)]
    src, dst = last[copies], fresh[row[copies], start[copies]]
    table.copy_(torch.where(takes, fresh.int(), table))
    ref.index_add_(0, src, torch.full_like(src, -1, dtype=torch.int32))
    ref[fresh[takes]] = 1
    lens.copy_(after)
    for name in ("k", "v"):
        _bytes(s[name])[dst] = _bytes(s[name])[src]
        s[name + "s"][dst] = s[name + "s"][src]
    starts = torch.cat([torch.zeros(1, dtype=torch.long, device="cuda"), torch.cumsum(new, 0)])
    seq, t = _places(starts, s["tokens"])
    positions = before[seq] + t
    slots = table[seq, positions // ps].long() * ps + positions % ps
    return {"table": table, "lens": lens, "ref": ref, "starts": starts.int(), "positions": positions.int(), "slots": slots,
            **_codes(s)}


def _plain_select(s, c):
    G, W, V, K = c["groups"], c["width"], c["vocab"], c["n_out"]
    # candidates next to one another differ by less than 32 bits resolve: in 64
    x = s["logits"].double()
    x = x.sub_(x.amax(-1, keepdim=True).clamp(min=-3.5e38))
    x = x.sub_(torch.log(x.exp().sum(-1, keepdim=True).clamp(min=1e-300)))
    x = x.add_(s["scores"].double()[:, None])
    # a beam that has ended goes on as it is
    only = torch.full_like(x[:1], -math.inf)
    ended = torch.where(torch.arange(V, device="cuda") == c["end"], s["scores"].double()[:, None], only)
    x = torch.where(s["finished"][:, None], ended, x).view(G, W * V)
    K_have = min(K, W * V)
    least = x.topk(K_have, 1).values[:, -1:]
    # all that reach the last place, by their index; then by their value, the order among equals kept
    g, at = torch.nonzero((x >= least) & (x > -math.inf), as_tuple=True)
    value, order = torch.sort(x[g, at], descending=True, stable=True)
    g, at = g[order], at[order]
    g, order = torch.sort(g, stable=True)
    value, at = value[order], at[order]
    place = torch.arange(g.shape[0], device="cuda") - torch.searchsorted(g, g)
    keep = place < K
    g, at, value, place = g[keep], at[keep], value[keep], place[keep]
    scores = torch.full((G, K), -math.inf, dtype=torch.float32, device="cuda")
    rows, tokens = (torch.full((G, K), -1, dtype=torch.int32, device="cuda") for _ in range(2))
    finished = torch.zeros((G, K), dtype=torch.bool, device="cuda")
    scores[g, place] = value.float()
    rows[g, place] = (g * W + at // V).int()
    tokens[g, place] = (at % V).int()
    finished[g, place] = s["finished"][g * W + at // V] | (at % V == c["end"])
    return {"scores": scores, "rows": rows, "tokens": tokens, "finished": finished}


def _plain_reorder(s, c):
    s["at"].copy_(s["before"])
    table, lens, ref, src = s["table"], s["lens"], s["ref"], s["src"].long()
    lost = table[table >= 0].long()
    there = src >= 0
    rows = torch.where(there[:, None], table[src.clamp(min=0)], torch.full_like(table, -1))
    gained = rows[rows >= 0].long()
    ref.index_add_(0, lost, torch.full_like(lost, -1, dtype=torch.int32))
    ref.index_add_(0, gained, torch.ones_like(gained, dtype=torch.int32))
    lens.copy_(torch.where(there, lens[src.clamp(min=0)], torch.zeros_like(lens)))
    table.copy_(rows)
    return {"table": table, "lens": lens, "ref": ref}


_PLAIN = {"attention": _plain_attention, "grow": _plain_grow, "select": _plain_select, "reorder": _plain_reorder}


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    """The definitions in 64 bits, sequence by sequence and request by request; growth and reordering compute no numbers."""
    if case["op"] not in ("attention", "select"):
        return None
    s = prepare(case, seed)
    return _exact_attention(s, case) if case["op"] == "attention" else _exact_select(s, case)


def _exact_attention(s, c):
    H, Hk, D, ps = c["heads"], c["kv_heads"], c["dim"], c["page"]
    G = H // Hk
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lens, starts = s["lens"].tolist(), s["starts"].tolist()
    for b, n in enumerate(lens):
        a, z = starts[b], starts[b + 1]
        if a == z:
            continue
        pages = s["table"][b, :-(-n // ps)].long()
        hidden = torch.arange(n, device="cuda") > torch.arange(n - (z - a), n, device="cuda")[:, None]
        k, v = (s[x].view(torch.int8)[pages].view(s[x].dtype).double() * s[x + "s"][pages].double()[:, :, None, None]
                for x in ("k", "v"))
        for h in range(Hk):
            x = torch.einsum("tgd,nd->gtn", s["q"][a:z, h * G:(h + 1) * G].double(), k[:, h].reshape(-1, D)[:n]) / math.sqrt(D)
            x = torch.softmax(x.masked_fill(hidden, -math.inf), -1)
            out[a:z, h * G:(h + 1) * G] = torch.einsum("gtn,nd->tgd", x, v[:, h].reshape(-1, D)[:n])
    return out


def _exact_select(s, c):
    G, W, K = c["groups"], c["width"], c["n_out"]
    got = {"scores": [], "rows": [], "tokens": [], "finished": []}
    scores, finished = s["scores"].double(), s["finished"]
    alive, ended = torch.isfinite(scores).tolist(), finished.tolist()
    for g in range(G):
        values, rows, tokens = [], [], []
        for r in range(g * W, (g + 1) * W):
            if not alive[r]:
                continue
            if ended[r]:
                v, t = scores[r:r + 1], torch.tensor([c["end"]], device="cuda")
            else:
                v, t = torch.sort(torch.log_softmax(s["logits"][r].double(), 0), descending=True, stable=True)
                v, t = v[:K] + scores[r], t[:K]
                v, t = v[v > -math.inf], t[v > -math.inf]
            values.append(v)
            tokens.append(t)
            rows.append(torch.full_like(t, r))
        fill = K
        if values:
            v, order = torch.sort(torch.cat(values), descending=True, stable=True)
            v, order = v[:K], order[:K]
            r, t = torch.cat(rows)[order], torch.cat(tokens)[order]
            fill = K - v.shape[0]
        else:
            v, r, t = (torch.zeros(0, dtype=d, device="cuda") for d in (torch.float64, torch.long, torch.long))
        pad = torch.full((fill,), -1, device="cuda")
        got["scores"].append(torch.cat([v, torch.full((fill,), -math.inf, dtype=torch.float64, device="cuda")]))
        got["rows"].append(torch.cat([r, pad]).int())
        got["tokens"].append(torch.cat([t, pad]).int())
        got["finished"].append(torch.cat([finished[r] | (t == c["end"]), torch.zeros(fill, dtype=torch.bool, device="cuda")]))
    return {k: torch.stack(v) for k, v in got.items()}
