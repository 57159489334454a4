"""Plain 64-bit definitions of the paged-cache operators on the CPU, and the
inputs their tests share.  Nothing here calls the library."""
import math

import torch

ACT = {"f16": torch.float16, "bf16": torch.bfloat16}
STORE = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}
QMAX = {"int8": 127.0, "e4m3": 448.0}
SCALE_MIN = 2.0 ** -60
# unit roundoff of the output type: half a unit in the last place, relative
ROUND = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}
# half the spacing of its subnormal numbers
TINY = {"f16": 2.0 ** -25, "bf16": 2.0 ** -134}


class Problem:
    """A cache, its tables and the sequences of one call (CPU tensors)."""

    def __init__(self, lens, new, heads=8, kv_heads=2, dim=128, page=16, store="int8", layout="heads", act="bf16",
                 seed=0, spare=3, blocks=None, wide=0):
        g = torch.Generator().manual_seed(seed)
        self.heads, self.kv_heads, self.dim, self.page = heads, kv_heads, dim, page
        self.store, self.layout, self.act = store, layout, act
        self.lens, self.new = list(lens), list(new)
        need = [-(-n // page) for n in lens]
        self.n_pages = sum(need) + spare
        # codes: normal values; slots past a sequence's length and spare pages keep hostile bytes
        unit = 1.0 / (38.0 if store == "int8" else 120.0)
        shape = (self.n_pages, kv_heads, page, dim)
        self.k, self.v = (self._codes(torch.randn(shape, generator=g)) for _ in range(2))
        self.ks, self.vs = (torch.empty(self.n_pages, kv_heads).uniform_(0.5, 1.5, generator=g) * unit for _ in range(2))
        perm = torch.randperm(self.n_pages, generator=g, dtype=torch.int32)
        self.table = torch.full((len(lens), max([1] + need) + wide), -1, dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = perm[at:at + n]
            at += n
        used = torch.zeros(self.n_pages, dtype=torch.bool)
        used[perm[:at].long()] = True
        for t in (self.k, self.v):
            raw = t.view(torch.int8)
            raw[~used] = 127                      # NaN as e4m3
            for b, n in enumerate(lens):
                if n % page:
                    raw[self.table[b, n // page].long(), :, n % page:] = 127
        self.ks[~used] = float("nan")
        self.vs[~used] = float("inf")
        T = sum(new)
        self.starts = torch.tensor([0] + list(torch.tensor(new).cumsum(0)) if new else [0], dtype=torch.int32)
        self.T = T
        rows = torch.randn((T, (heads + 2 * kv_heads) * dim), generator=g)
        self.rows = rows.to(ACT[act])

    def _codes(self, x):
        if self.store == "int8":
            return (x * 38).round().clamp(-127, 127).to(torch.int8)
        return (x * 120).clamp(-448, 448).to(torch.float8_e4m3fn)

    @property
    def q(self):
        return self.rows[:, :self.heads * self.dim].unflatten(1, (self.heads, self.dim))

    @property
    def k_new(self):
        return self.rows[:, self.heads * self.dim:(self.heads + self.kv_heads) * self.dim].unflatten(1, (self.kv_heads, self.dim))

    @property
    def v_new(self):
        return self.rows[:, (self.heads + self.kv_heads) * self.dim:].unflatten(1, (self.kv_heads, self.dim))

    def to_cuda(self, w):
        """(cache, table, lens, starts, rows) on the GPU, in the layout asked for."""
        def put(t):
            t = t.view(torch.int8).cuda()
            if self.layout == "tokens":
                t = t.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3)
            elif self.layout == "padded":         # rows further apart than they are long
                big = torch.full((t.shape[0], t.shape[1], t.shape[2] + 1, t.shape[3] + 16), 127, dtype=torch.int8, device="cuda")
                big[:, :, :-1, :-16] = t
                t = big[:, :, :-1, :-16]
            return t.view(STORE[self.store])
        if self.layout == "pairs":                # K and V of a page next to each other in one tensor
            both = torch.stack([self.k.view(torch.int8), self.v.view(torch.int8)], 1).cuda()
            cache = w.KVCache(both[:, 0].view(STORE[self.store]), both[:, 1].view(STORE[self.store]), self.ks.cuda(), self.vs.cuda())
        else:
            cache = w.KVCache(put(self.k), put(self.v), self.ks.cuda(), self.vs.cuda())
        return (cache, self.table.cuda(), torch.tensor(self.lens, dtype=torch.int32).cuda(), self.starts.cuda(),
                self.rows.cuda())

    def values(self, codes, scales, b, n):
        """[n, kv_heads, dim] in 64 bits."""
        ps = self.page
        pages = self.table[b, :-(-n // ps)].long().clamp(min=0)
        x = codes.view(torch.int8)[pages].view(codes.dtype).double() * scales[pages].double()[..., None, None]
        return x.transpose(1, 2).reshape(-1, self.kv_heads, self.dim)[:n]


def visible(i, n, window, sinks):
    j = torch.arange(n)
    see = j <= i
    if window > 0:
        see &= (i - j < window) | (j < sinks)
    return see


def attention(p, scale=None, window=0, sinks=0):
    """(out, lse, spread) in 64 bits; spread = sum_j p_j |v_j|, what a relative error of the weights is worth."""
    scale = p.dim ** -0.5 if scale is None else scale
    out = torch.zeros(p.T, p.heads, p.dim, dtype=torch.float64)
    spread = torch.zeros_like(out)
    lse = torch.full((p.T, p.heads), -math.inf, dtype=torch.float64)
    g = p.heads // p.kv_heads
    at = 0
    for b, (n, m) in enumerate(zip(p.lens, p.new)):
        if m == 0:
            continue
        k, v = p.values(p.k, p.ks, b, n), p.values(p.v, p.vs, b, n)
        pos = torch.arange(n - m, n)
        j = torch.arange(n)
        see = j[None, :] <= pos[:, None]
        if window > 0:
            see = see & ((pos[:, None] - j[None, :] < window) | (j[None, :] < sinks))
        hidden_rows = ~see.any(0) if n else see
        v = torch.where(hidden_rows[:, None, None], torch.zeros_like(v), v)
        for a in range(p.heads):
            s = p.q[at:at + m, a].double() @ k[:, a // g].T * scale
            s = torch.where(see, s, torch.full_like(s, -math.inf))
            rows = see.any(1)
            w = torch.softmax(s[rows], -1)
            idx = at + torch.nonzero(rows)[:, 0]
            out[idx, a] = w @ v[:, a // g]
            spread[idx, a] = w @ v[:, a // g].abs()
            lse[idx, a] = torch.logsumexp(s[rows], -1)
        at += m
    return out, lse, spread


def attention_tolerance(p, out, spread):
    """Elementwise bound on the kernels' error.  The output is rounded once
    (unit roundoff of its type, or half its smallest spacing).  Softmax weights meet the values as fp16 at
    worst: 2^-11 of each weight, so of `spread`.  Scores are fp32 sums of at
    most 128 exact products of moderate size, and exp2 is good to 2^-22: together below
    2^-12 of a weight at the scores these tests draw."""
    return ROUND[p.act] * out.abs() + (2.0 ** -11 + 2.0 ** -12) * spread + TINY[p.act]


def round_code(x, store):
    """Nearest code's value (ties to even, saturated) of values in 64 bits."""
    if store == "int8":
        return torch.clamp(torch.round(x), -127, 127)
    return x.float().clamp(-448, 448).to(torch.float8_e4m3fn).double()


def append(p):
    """(k codes, v codes, k scales, v scales) after the append, in the fp32
    arithmetic that the definition fixes; p's own tensors stay."""
    out = []
    for codes, scales, x in ((p.k, p.ks, p.k_new), (p.v, p.vs, p.v_new)):
        val, scales = codes.float(), scales.clone()
        at = 0
        for b, (n, m) in enumerate(zip(p.lens, p.new)):
            first = n - m
            for blk in range(first // p.page, -(-n // p.page) if m else 0):
                page = int(p.table[b, blk])
                lo, hi = max(first, blk * p.page), min(n, blk * p.page + p.page)
                old = lo - blk * p.page
                new = x[at + lo - first:at + hi - first].float()           # [tokens, heads, dim]
                s_old = scales[page] if old else torch.zeros(p.kv_heads)
                amax = new.abs().amax((0, 2))
                s = torch.maximum(torch.maximum(s_old, amax / torch.tensor(QMAX[p.store])), torch.tensor(SCALE_MIN))
                r = (1.0 / s)[:, None, None]
                if old:
                    again = _round32(val[page, :, :old] * s_old[:, None, None] * r, p.store)
                    val[page, :, :old] = torch.where((s != s_old)[:, None, None], again, val[page, :, :old])
                val[page, :, old:old + hi - lo] = _round32(new.transpose(0, 1) * r, p.store)
                scales[page] = s
            at += m
        stay = codes.view(torch.int8)
        new_codes = val.to(codes.dtype).view(torch.int8)
        same = (val == codes.float()) | codes.float().isnan()
        out.append((torch.where(same, stay, new_codes), scales))
    return out[0][0], out[1][0], out[0][1], out[1][1]


def _round32(x, store):
    if store == "int8":
        return x.round().clamp(-127, 127)
    return x.clamp(-448, 448).to(torch.float8_e4m3fn).float()
