"""Cases of the paged 8-bit key/value cache operators: what a decoder layer
runs between its qkv and its output projection, and what a scheduler runs on
the cache's pages between steps.

  attention  attention of each sequence's newest tokens over its cache, causal,
             optionally with a sliding window and sink tokens
  append     quantise new keys and values into the cache's pages, then read
             the touched blocks back
  fork, retire, copy
             sequences that share pages; finished sequences freed, pages that
             left the window trimmed and the pool compacted; page copies

The cache: codes in 8 bits (int8, or e4m3) of shape [pages, kv heads, tokens of
a page, head dim], and one fp32 scale for each page and kv head; a value is
code * scale.  `own` false computes the plain form (elementary torch operations
in 32 bits, rounded once); `own` true calls the framework.
"""
import math
import random

import torch

own = False

ACT = {"bf16": torch.bfloat16, "f16": torch.float16}
STORE = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}
QMAX = {"int8": 127.0, "e4m3": 448.0}
SCALE_MIN = 2.0 ** -60        # the scale of a block of zeros


# ------------------------------------------------------------------ cases
def _attn(name, **kw):
    c = {"name": name, "op": "attention", "seqs": 1, "new_lo": 1, "new_hi": 1, "past_lo": 0, "past_hi": 0,
         "heads": 32, "kv_heads": 8, "dim": 128, "page": 16, "window": 0, "sinks": 0, "act": "bf16",
         "store": "int8", "layout": "heads", "mix": 1}
    c.update(kw)
    return c


def listed():
    return [
        # one chat user, a short context: the call's latency is all there is
        _attn("attn_decode_1x77", past_lo=76, past_hi=76),
        # a serving batch, contexts from a few tokens to past the prompt lengths of the prefill workload
        _attn("attn_decode_64_ragged", seqs=64, past_lo=3, past_hi=4095, mix=2),
        # few sequences, very long contexts (the cache read is the whole cost); pages laid out token first
        _attn("attn_decode_4_long", seqs=4, past_lo=98301, past_hi=131070, page=64, act="f16", store="e4m3",
              layout="tokens", mix=3),
        # a model with a sliding window and sinks, one kv head per head, small heads
        _attn("attn_decode_48_window", seqs=48, past_lo=900, past_hi=16383, heads=32, kv_heads=32, dim=64, page=32,
              window=1024, sinks=4, mix=4),
        # verification of a few drafted tokens per sequence, eight heads to a kv head
        _attn("attn_verify_24x5", seqs=24, new_lo=5, new_hi=5, past_lo=128, past_hi=4001, heads=32, kv_heads=4,
              act="f16", mix=5),
        # a prompt of the prefill workload's length
        _attn("attn_prefill_1920", new_lo=1920, new_hi=1920, page=16, mix=6),
        # chunks of long prompts over what is already cached, with a window and sinks
        _attn("attn_chunks_window", seqs=4, new_lo=700, new_hi=2048, past_lo=2047, past_hi=6144, page=64, window=4096,
              sinks=4, act="f16", store="e4m3", mix=7),
        # the token of each sequence of a serving batch
        {"name": "append_decode_64", "op": "append", "seqs": 64, "new_lo": 1, "new_hi": 1, "past_lo": 0,
         "past_hi": 4095, "heads": 32, "kv_heads": 8, "dim": 128, "page": 16, "act": "bf16", "store": "int8",
         "layout": "heads", "mix": 8},
        # prompts entering the cache, the first page of some already begun
        {"name": "append_prompts_8x1920", "op": "append", "seqs": 8, "new_lo": 1857, "new_hi": 1920, "past_lo": 0,
         "past_hi": 131, "heads": 32, "kv_heads": 8, "dim": 128, "page": 64, "act": "f16", "store": "e4m3",
         "layout": "tokens", "mix": 9},
        # parallel sampling: every prompt continues in several sequences that share its full pages
        {"name": "fork_16x8", "op": "fork", "seqs": 16, "copies": 8, "past_lo": 100, "past_hi": 1920, "kv_heads": 8,
         "dim": 128, "page": 32, "store": "int8", "layout": "heads", "mix": 10},
        # a scheduler's clean-up: a share of the sequences ends, the others lose what left their window, the pool closes up
        {"name": "retire_96", "op": "retire", "seqs": 96, "ended": 40, "past_lo": 60, "past_hi": 8191, "kv_heads": 8,
         "dim": 128, "page": 16, "window": 2048, "sinks": 4, "store": "int8", "layout": "heads", "mix": 11},
        # pages moved on a list, e.g. to make room for a pinned prefix
        {"name": "copy_3001_pages", "op": "copy", "pages": 8192, "moved": 3001, "kv_heads": 8, "dim": 128,
         "page": 16, "store": "e4m3", "layout": "tokens", "mix": 12},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["decode", "decode", "verify", "prefill", "chunks", "append", "fork", "retire", "copy"])
    mix = rng.randrange(1 << 30)
    store = rng.choice(["int8", "e4m3"])
    layout = rng.choice(["heads", "tokens"])
    page = rng.choice([16, 32, 64, 128])
    heads, kv_heads = rng.choice([(32, 8), (32, 8), (32, 4), (28, 4), (32, 32), (8, 1)])
    dim = rng.choice([64, 128, 128])
    act = rng.choice(["bf16", "f16"])
    if op in ("decode", "verify", "prefill", "chunks"):
        c = {"op": "attention", "heads": heads, "kv_heads": kv_heads, "dim": dim, "page": page, "act": act,
             "store": store, "layout": layout, "mix": mix}
        if rng.random() < 0.4:
            c.update(window=_log(rng, 1, 4096), sinks=rng.choice([0, 1, 4, 17]))
        else:
            c.update(window=0, sinks=0)
        if op == "decode":
            c.update(seqs=_log(rng, 1, 64), new_lo=1, new_hi=1)
            past = _log(rng, 1, 131000)
        elif op == "verify":
            new = rng.randrange(2, 17)
            c.update(seqs=_log(rng, 1, 24), new_lo=rng.choice([0, 1, new]), new_hi=new)
            past = _log(rng, 1, 16000)
        elif op == "prefill":
            new = _log(rng, 17, 4096)
            c.update(seqs=_log(rng, 1, 8), new_lo=rng.choice([1, new]), new_hi=new)
            past = 0
        else:
            new = _log(rng, 64, 2048)
            c.update(seqs=_log(rng, 1, 4), new_lo=rng.choice([1, new // 2, new]), new_hi=new)
            past = _log(rng, 16, 16000)
        # no more cached values and no more scores than the largest listed cases have
        while c["seqs"] * (past + c["new_hi"]) * kv_heads * dim > 4 * 131071 * 8 * 128:
            c["seqs"], past = max(1, c["seqs"] * 2 // 3), max(1, past * 2 // 3)
        while c["seqs"] * heads * c["new_hi"] * (past + c["new_hi"]) > 4 * 32 * 2048 * 8192:
            c["seqs"], past, c["new_hi"] = max(1, c["seqs"] // 2), past * 2 // 3, max(2, c["new_hi"] * 3 // 4)
        c["new_lo"] = min(c["new_lo"], c["new_hi"])
        c.update(past_lo=rng.choice([past // 8, past // 2, past]), past_hi=past)
        return c
    base = {"kv_heads": kv_heads, "dim": dim, "page": page, "store": store, "layout": layout, "mix": mix}
    if op == "append":
        new = rng.choice([1, _log(rng, 1, 1920)])
        past = _log(rng, 1, 4096)
        return {"op": "append", "seqs": _log(rng, 1, 64 if new == 1 else 8), "new_lo": rng.choice([1, new]),
                "new_hi": new, "past_lo": rng.choice([0, past // 2]), "past_hi": past, "heads": heads, "act": act, **base,
                "kv_heads": min(kv_heads, 8)}
    base["kv_heads"] = min(kv_heads, 8)
    past = _log(rng, 8, 4096)
    if op == "fork":
        return {"op": "fork", "seqs": _log(rng, 1, 16), "copies": rng.randrange(1, 9), "past_lo": past // 8,
                "past_hi": past, **base}
    if op == "retire":
        seqs = _log(rng, 2, 96)
        return {"op": "retire", "seqs": seqs, "ended": rng.randrange(0, seqs), "past_lo": past // 8, "past_hi": past,
                "window": rng.choice([0, _log(rng, 1, 4096)]), "sinks": rng.choice([0, 4, 33]), **base}
    pages = _log(rng, 16, 8192 * 16 // page)
    return {"op": "copy", "pages": pages, "moved": max(1, int(pages * rng.uniform(0.05, 0.45))), **base}


# ------------------------------------------------------------------ lengths
def _lengths(case):
    """Past and new tokens of each sequence: plain lists, from the case alone."""
    r = random.Random(case["mix"])
    past = [r.randint(case["past_lo"], case["past_hi"]) for _ in range(case["seqs"])]
    new = [r.randint(case["new_lo"], case["new_hi"]) if "new_lo" in case else 0 for _ in range(case["seqs"])]
    if "new_hi" in case and max(new) < case["new_hi"]:
        new[-1] = case["new_hi"]
    past[0] = case["past_hi"]
    return past, new


def _starts(counts):
    s = [0]
    for n in counts:
        s.append(s[-1] + n)
    return s


def _visible(i, window, sinks):
    """How many of the positions 0..i a query at position i sees."""
    if window <= 0 or i + 1 <= window:
        return i + 1
    return window + min(sinks, i + 1 - window)


def _seen_by_any(past, new, window, sinks):
    """How many positions at least one of a sequence's new tokens sees."""
    n = past + new
    if new == 0:
        return 0
    lo = max(0, past + 1 - window) if window > 0 else 0
    return n - lo + min(sinks, lo)


def work(case):
    D, Hk, ps = case["dim"], case["kv_heads"], case["page"]
    page_bytes = 2 * Hk * (ps * D + 4)
    if case["op"] == "attention":
        past, new = _lengths(case)
        w, s, H = case["window"], case["sinks"], case["heads"]
        tokens = sum(new)
        kv = sum(_seen_by_any(p, n, w, s) for p, n in zip(past, new))
        pairs = sum(_visible(p + t, w, s) for p, n in zip(past, new) for t in range(n))
        return {"bytes": 2 * tokens * H * D * 2 + kv * Hk * D * 2 + kv / ps * (8 * Hk + 4), "flops": 4 * pairs * H * D}
    if case["op"] == "append":
        past, new = _lengths(case)
        touched = sum(p + n - p // ps * ps for p, n in zip(past, new))
        # new keys and values read, codes and scales written; the read-back's codes and scales read, values written
        return {"bytes": sum(new) * Hk * D * (4 + 2) + touched * Hk * D * (2 + 4) + touched / ps * Hk * 24,
                "flops": 8 * sum(new) * Hk * D}
    if case["op"] == "copy":
        return {"bytes": case["moved"] * (2 * page_bytes + 8), "flops": 0}
    past, _ = _lengths(case)
    blocks = [-(-p // ps) for p in past]
    if case["op"] == "fork":
        tails = sum(1 for p in past if p % ps) * case["copies"]
        full = sum(p // ps for p in past) * case["copies"]
        read_tails = sum(1 for p in past if p % ps)
        return {"bytes": (tails + read_tails) * page_bytes + full * 8 + 4 * _pool(blocks, case), "flops": 0}
    kept, moved = _retired(case, past)
    return {"bytes": moved * 2 * page_bytes + 4 * sum(blocks) * 2 + 4 * _pool(blocks, case), "flops": 0}


def _pool(blocks, case):
    """Pages of the pool: what the sequences hold, what forks add, and some that are free."""
    return sum(blocks) + case["seqs"] * case.get("copies", 0) + max(4, sum(blocks) // 8)


def _retired(case, past):
    """How many pages stay after the clean-up, and how many of them have to move (an even spread assumed)."""
    ps, w, s = case["page"], case["window"], case["sinks"]
    kept = 0
    for p in past[case["ended"]:]:
        for b in range(-(-p // ps)):
            kept += not (w > 0 and b * ps >= s and b * ps + ps <= p - w + 1)
    pool = _pool([-(-p // ps) for p in past], case)
    return kept, int(kept * (1 - kept / pool))


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


def _table(blocks, pages, g, rows=None):
    """Block table [rows, widest]: the sequences' pages drawn from all over the pool; -1 where there is none."""
    rows = rows or len(blocks)
    width = max(1, max(blocks))
    perm = torch.randperm(pages, generator=g, device="cuda", dtype=torch.int32)
    has = torch.tensor(list(blocks) + [0] * (rows - len(blocks)), device="cuda")
    first = torch.cumsum(has, 0) - has
    col = torch.arange(width, device="cuda")
    idx = (first[:, None] + col[None]).clamp_(max=pages - 1)
    return torch.where(col[None] < has[:, None], perm[idx.long()], torch.full_like(perm[idx.long()], -1)).contiguous()


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 1000003 + 17)
    Hk, ps, D = case["kv_heads"], case["page"], case["dim"]
    s = {"case": case}
    if case["op"] == "copy":
        s["k"], s["v"], s["ks"], s["vs"] = _cache(case, case["pages"], g)
        perm = torch.randperm(case["pages"], generator=g, device="cuda", dtype=torch.int32)
        s["src"], s["dst"] = perm[:case["moved"]].contiguous(), perm[case["moved"]:2 * case["moved"]].contiguous()
        return s
    past, new = _lengths(case)
    if case["op"] in ("attention", "append"):
        lens = [p + n for p, n in zip(past, new)]
        blocks = [-(-n // ps) for n in lens]
        pages = sum(blocks) + max(1, sum(blocks) // 16)
        s["k"], s["v"], s["ks"], s["vs"] = _cache(case, pages, g)
        s["table"], s["lens"], s["starts"] = _table(blocks, pages, g), _ints(lens), _ints(_starts(new))
        s["max_new"] = max(new)
        T, dt = sum(new), ACT[case["act"]]
        H = case["heads"]
        # the rows of a merged qkv projection's output: q, k and v are views of it
        qkv = torch.randn((T, (H + 2 * Hk) * D), generator=g, device="cuda", dtype=torch.float32).to(dt)
        if case["op"] == "attention":
            s["q"] = qkv[:, :H * D].unflatten(1, (H, D))
        else:
            s["k_new"] = qkv[:, H * D:(H + Hk) * D].unflatten(1, (Hk, D))
            s["v_new"] = qkv[:, (H + Hk) * D:].unflatten(1, (Hk, D))
            # the read-back: from the start of the first page that the new tokens touch
            back = [n - p // ps * ps for n, p in zip(lens, past)]
            s["back"], s["n_back"] = _ints(_starts(back)), sum(back)
        return s
    blocks = [-(-p // ps) for p in past]
    pages = _pool(blocks, case)
    rows = case["seqs"] * (1 + case.get("copies", 0))
    s["k"], s["v"], s["ks"], s["vs"] = _cache(case, pages, g)
    s["table"] = _table(blocks, pages, g, rows)
    s["lens"] = _ints(past + [0] * (rows - len(past)))
    s["ref"] = torch.zeros(pages, dtype=torch.int32, device="cuda")
    s["ref"][s["table"][s["table"] >= 0].long()] = 1
    if case["op"] == "fork":
        n = case["seqs"]
        s["parents"] = _ints([b for b in range(n) for _ in range(case["copies"])])
        s["children"] = _ints(list(range(n, rows)))
    else:
        s["ended"] = _ints(list(range(case["ended"])))
    return s


# ------------------------------------------------------------------ one pass
def run(state):
    case = state["case"]
    form = _FRAMEWORK if own else _PLAIN
    return form[case["op"]](state, case)


def _own_cache(w, s):
    return w.KVCache(s["k"], s["v"], s["ks"], s["vs"])


def _own_attention(s, c):
    import w4a16_group_quantised_gb300 as w
    return w.w4a16_kv_attention(s["q"], _own_cache(w, s), s["table"], s["lens"], s["starts"], s["max_new"],
                                window=c["window"], sinks=c["sinks"])


def _own_append(s, c):
    import w4a16_group_quantised_gb300 as w
    cache = _own_cache(w, s)
    w.w4a16_kv_append(cache, s["k_new"], s["v_new"], s["table"], s["lens"], s["starts"])
    k, v = w.w4a16_kv_read(cache, s["table"], s["lens"], s["back"], s["n_back"], ACT[c["act"]])
    return {"k": k, "v": v, "ks": s["ks"], "vs": s["vs"]}


def _own_fork(s, c):
    import w4a16_group_quantised_gb300 as w
    table, lens, ref = s["table"].clone(), s["lens"].clone(), s["ref"].clone()
    w.w4a16_kv_fork(_own_cache(w, s), table, lens, ref, s["parents"], s["children"])
    return {"table": table, "lens": lens, "ref": ref, **_codes(s)}


def _own_retire(s, c):
    import w4a16_group_quantised_gb300 as w
    table, lens, ref = s["table"].clone(), s["lens"].clone(), s["ref"].clone()
    w.w4a16_kv_free(table, lens, ref, s["ended"])
    w.w4a16_kv_trim(table, lens, ref, c["page"], window=c["window"], sinks=c["sinks"])
    w.w4a16_kv_compact(_own_cache(w, s), table, ref)
    return {"table": table, "lens": lens, "ref": ref, **_codes(s)}


def _own_copy(s, c):
    import w4a16_group_quantised_gb300 as w
    w.w4a16_kv_copy_pages(_own_cache(w, s), s["src"], s["dst"])
    return _codes(s)


def _codes(s):
    """The cache's buffers: page operators move codes and scales as they are."""
    return {"k": s["k"], "v": s["v"], "ks": s["ks"], "vs": s["vs"]}


_FRAMEWORK = {"attention": _own_attention, "append": _own_append, "fork": _own_fork, "retire": _own_retire,
              "copy": _own_copy}


# ------------------------------------------------------------------ the plain forms
def _bytes(t):
    return t.view(torch.int8)


def _gather(codes, scales, table, n):
    """fp32 values [sequences, n, kv heads, dim] of the first n cached positions."""
    ps = codes.shape[2]
    t = table[:, :-(-n // ps)].long().clamp(min=0)
    x = _bytes(codes)[t].view(codes.dtype).float() * scales[t][..., None, None]
    return x.transpose(2, 3).flatten(1, 2)[:, :n]


def _places(starts, T):
    """Sequence of each token of the batch, and its number within the sequence."""
    tok = torch.arange(T, device="cuda")
    seq = torch.searchsorted(starts[1:].long(), tok, right=True)
    return seq, tok - starts.long()[seq]


def _plain_attention(s, c):
    H, Hk, D = c["heads"], c["kv_heads"], c["dim"]
    B, T, nq = s["lens"].shape[0], s["q"].shape[0], s["max_new"]
    n = s["table"].shape[1] * c["page"]
    seq, t = _places(s["starts"], T)
    q = torch.zeros((B, nq, H, D), device="cuda")
    q[seq, t] = s["q"].float()
    q = q.view(B, nq, Hk, H // Hk, D).permute(0, 2, 3, 1, 4).reshape(B, Hk, H // Hk * nq, D)
    k = _gather(s["k"], s["ks"], s["table"], n).transpose(1, 2)
    new = s["starts"][1:] - s["starts"][:-1]
    pos = (s["lens"] - new)[:, None] + torch.arange(nq, device="cuda")
    j = torch.arange(n, device="cuda")
    seen = j <= pos[..., None]
    if c["window"] > 0:
        seen &= (pos[..., None] - j < c["window"]) | (j < c["sinks"])
    x = torch.matmul(q, k.transpose(2, 3)).view(B, Hk, H // Hk, nq, n)
    del k
    x = x.mul_(1.0 / math.sqrt(D)).masked_fill_(~seen[:, None, None], -math.inf)
    x = x.sub_(x.amax(-1, keepdim=True).clamp(min=-3.0e38)).exp_()
    x = x.div_(x.sum(-1, keepdim=True).clamp(min=1e-37))
    v = _gather(s["v"], s["vs"], s["table"], n).transpose(1, 2)
    v = v.masked_fill((j >= s["lens"][:, None])[:, None, :, None], 0.0)
    o = torch.matmul(x.view(B, Hk, H // Hk * nq, n), v).view(B, H, nq, D)
    return o.transpose(1, 2)[seq, t].to(s["q"].dtype)


def _round_codes(x, store):
    if store == "int8":
        return x.round().clamp(-127, 127).to(torch.int8)
    return x.clamp(-448, 448).to(torch.float8_e4m3fn)


def _plain_append_one(codes, scales, x, s, c, plan):
    seq, pos, page, slot, old = plan
    Hk, ps = c["kv_heads"], c["page"]
    x = x.float()
    # each touched page's largest new value, against the scale its older tokens have
    top = torch.zeros(scales.shape, device="cuda").index_reduce_(0, page, x.abs().amax(-1), "amax")
    touched = torch.zeros(scales.shape[0], dtype=torch.bool, device="cuda")
    touched[page] = True
    before = torch.where((old > 0)[:, None], scales, torch.zeros_like(scales))
    scale = torch.maximum(torch.maximum(before, top / QMAX[c["store"]]), torch.full_like(scales, SCALE_MIN))
    scale = torch.where(touched[:, None], scale, scales)
    p = torch.nonzero(touched & (old > 0))[:, 0]
    # older tokens of a page whose scale grew are rounded again; where it did not, they stay as they are
    kept = _bytes(codes)[p].view(codes.dtype).float()
    again = _round_codes(kept * scales[p][..., None, None] * (1.0 / scale[p])[..., None, None], c["store"])
    grew = ((scale[p] != scales[p])[..., None, None]
            & (torch.arange(ps, device="cuda")[None, :] < old[p][:, None])[:, None, :, None])
    _bytes(codes)[p] = torch.where(grew, _bytes(again), _bytes(codes)[p])
    _bytes(codes)[page, :, slot] = _bytes(_round_codes(x * (1.0 / scale[page])[..., None], c["store"]))
    scales.copy_(scale)


def _plain_read(codes, scales, seq, pos, table, dt):
    ps = codes.shape[2]
    page = table[seq, pos // ps].long()
    return (_bytes(codes)[page, :, pos % ps].view(codes.dtype).float() * scales[page][..., None]).to(dt)


def _plain_append(s, c):
    ps, table = c["page"], s["table"]
    seq, t = _places(s["starts"], s["k_new"].shape[0])
    first = s["lens"].long() - (s["starts"][1:] - s["starts"][:-1]).long()
    pos = first[seq] + t
    page = table[seq, pos // ps].long()
    # tokens that a page held before: all slots below the first new one
    old = torch.zeros(s["k"].shape[0], dtype=torch.long, device="cuda")
    old[page] = (first[seq] - pos // ps * ps).clamp(min=0)
    plan = seq, pos, page, pos % ps, old
    _plain_append_one(s["k"], s["ks"], s["k_new"], s, c, plan)
    _plain_append_one(s["v"], s["vs"], s["v_new"], s, c, plan)
    seq, t = _places(s["back"], s["n_back"])
    pos = s["lens"].long()[seq] - (s["back"][1:] - s["back"][:-1]).long()[seq] + t
    dt = ACT[c["act"]]
    return {"k": _plain_read(s["k"], s["ks"], seq, pos, table, dt), "v": _plain_read(s["v"], s["vs"], seq, pos, table, dt),
            "ks": s["ks"], "vs": s["vs"]}


def _copy_pages(s, src, dst):
    src, dst = src.long(), dst.long()
    _bytes(s["k"])[dst] = _bytes(s["k"])[src]
    _bytes(s["v"])[dst] = _bytes(s["v"])[src]
    s["ks"][dst] = s["ks"][src]
    s["vs"][dst] = s["vs"][src]


def _plain_copy(s, c):
    _copy_pages(s, s["src"], s["dst"])
    return _codes(s)


def _plain_fork(s, c):
    table, lens, ref = s["table"].clone(), s["lens"].clone(), s["ref"].clone()
    par, chi, ps = s["parents"].long(), s["children"].long(), c["page"]
    n = lens[par].long()
    free = torch.nonzero(ref == 0)[:, 0]
    # a child whose parent's last page is not full gets the lowest free page, in the children's order
    tail = n % ps != 0
    fresh = free[(torch.cumsum(tail, 0) - 1)[tail]]
    source = table[par[tail], n[tail] // ps]
    rows = table[par]
    shared = rows[torch.arange(rows.shape[1], device="cuda") < (n // ps)[:, None]]
    ref.index_add_(0, shared.long(), torch.ones_like(shared))
    ref[fresh] = 1
    rows = torch.where(torch.arange(rows.shape[1], device="cuda") < (-(-n // ps))[:, None], rows, torch.full_like(rows, -1))
    table[chi] = rows
    table[chi[tail], n[tail] // ps] = fresh.int()
    lens[chi] = lens[par]
    _copy_pages(s, source, fresh)
    return {"table": table, "lens": lens, "ref": ref, **_codes(s)}


def _plain_retire(s, c):
    table, lens, ref = s["table"].clone(), s["lens"].clone(), s["ref"].clone()
    ps, w, sinks, pages = c["page"], c["window"], c["sinks"], s["ref"].shape[0]
    ended = s["ended"].long()
    col = torch.arange(table.shape[1], device="cuda")
    gone = torch.zeros_like(table, dtype=torch.bool)
    gone[ended] = True
    if w > 0:
        # no later token sees positions from `sinks` to len - window
        gone |= (col * ps >= sinks) & (col * ps + ps <= lens[:, None] - w + 1)
    gone &= table >= 0
    ref.index_add_(0, table[gone].long(), torch.full_like(table[gone], -1))
    table[gone] = -1
    lens[ended] = 0
    live = ref > 0
    m = live.sum()
    at = torch.arange(pages, device="cuda")
    src = torch.nonzero(live & (at >= m))[:, 0]
    dst = torch.nonzero(~live & (at < m))[:, 0]
    to = torch.arange(pages, device="cuda", dtype=torch.int32)
    to[src] = dst.int()
    table = torch.where(table >= 0, to[table.long().clamp(min=0)], table)
    ref[dst] = ref[src]
    ref[src] = 0
    _copy_pages(s, src, dst)
    return {"table": table, "lens": lens, "ref": ref, **_codes(s)}


_PLAIN = {"attention": _plain_attention, "append": _plain_append, "fork": _plain_fork, "retire": _plain_retire,
          "copy": _plain_copy}


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    """The definitions in 64 bits, sequence by sequence; the page operators compute no numbers."""
    if case["op"] not in ("attention", "append"):
        return None
    s = prepare(case, seed)
    past, new = _lengths(case)
    one = _exact_attention if case["op"] == "attention" else _exact_append
    return one(s, case, past, new)


def _sequence(codes, scales, pages, n, h):
    """Values [n, dim] in 64 bits of one sequence and kv head."""
    x = codes.view(torch.int8)[pages, h].view(codes.dtype).double() * scales[pages, h].double()[:, None, None]
    return x.reshape(-1, x.shape[-1])[:n]


def _exact_attention(s, c, past, new):
    H, Hk, D = c["heads"], c["kv_heads"], c["dim"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    at = 0
    for b, (p, m) in enumerate(zip(past, new)):
        pages = s["table"][b, :-(-(p + m) // c["page"])].long()
        for h in range(Hk if m else 0):
            k, v = (_sequence(s[x], s[x + "s"], pages, p + m, h) for x in ("k", "v"))
            for t0 in range(0, m, 512):
                i = torch.arange(p + t0, p + min(m, t0 + 512), device="cuda")[:, None]
                j = torch.arange(p + m, device="cuda")[None, :]
                hidden = j > i
                if c["window"] > 0:
                    hidden |= (i - j >= c["window"]) & (j >= c["sinks"])
                for g in range(H // Hk):
                    a = h * (H // Hk) + g
                    x = s["q"][at + t0:at + min(m, t0 + 512), a].double() @ k.T / math.sqrt(D)
                    x[hidden] = -math.inf
                    out[at + t0:at + min(m, t0 + 512), a] = torch.softmax(x, -1) @ v
        at += m
    return out


def _exact_round(x, store):
    if store == "int8":
        return torch.clamp(torch.round(x), -127, 127)
    # e4m3: 3 fraction bits, the smallest normal 2^-6, the largest value 448
    a = x.abs().clamp(max=448.0)
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3)
    return torch.sign(x) * (torch.round(a / step) * step).clamp(max=448.0)


def _exact_append(s, c, past, new):
    ps, Hk, D, store = c["page"], c["kv_heads"], c["dim"], c["store"]
    got = {}
    for name in ("k", "v"):
        codes, scales = s[name], s[name + "s"].double()
        rows, at = [], 0
        for b, (p, m) in enumerate(zip(past, new)):
            x = s[name + "_new"][at:at + m].double()
            at += m
            lo = p // ps * ps
            if m == 0:
                pages = s["table"][b, p // ps:-(-p // ps)].long()
                rows.append((codes.view(torch.int8)[pages].view(codes.dtype).double() * scales[pages][..., None, None])
                            .transpose(1, 2).reshape(-1, Hk, D)[:p - lo])
                continue
            n_pages = -(-(p + m) // ps) - p // ps
            pages = s["table"][b, p // ps:p // ps + n_pages].long()
            full = torch.zeros((n_pages * ps, Hk, D), dtype=torch.float64, device="cuda")
            full[p - lo:p - lo + m] = x
            full = full.view(n_pages, ps, Hk, D)
            scale = full.abs().amax((1, 3)) / QMAX[store]
            if p > lo:
                scale[0] = torch.maximum(scale[0], scales[pages[0]])
            scale = scale.clamp(min=SCALE_MIN)
            if p > lo:
                old = codes.view(torch.int8)[pages[0]].view(codes.dtype).double().transpose(0, 1)[:p - lo]
                full[0, :p - lo] = old * scales[pages[0]][:, None]
            q = _exact_round(full / scale[:, None, :, None], store)
            rows.append((q * scale[:, None, :, None]).reshape(-1, Hk, D)[:p - lo + m])
            scales[pages] = scale
        got[name], got[name + "s"] = torch.cat(rows), scales
    return got
