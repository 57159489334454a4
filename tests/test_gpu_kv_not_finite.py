"""A value that is not finite, appended: its block's scale says so, its codes
are zeros, and attention gives NaN to the tokens that see the block and the
right answer to all others."""
import pytest
import torch

from kv_reference import Problem, attention, attention_tolerance, visible

pytestmark = pytest.mark.gpu


def appended(w, p, bad, where, head=0, dim=5):
    """The cache of p after its append, `bad` planted in K or V of the new token `where`."""
    at = (p.heads + (0 if "k" in bad[0] else p.kv_heads) + head) * p.dim + dim
    p.rows[where, at] = bad[1]
    cache, table, lens, starts, rows = p.to_cuda(w)
    a, b = p.heads * p.dim, (p.heads + p.kv_heads) * p.dim
    w.w4a16_kv_append(cache, rows[:, a:b].unflatten(1, (p.kv_heads, p.dim)), rows[:, b:].unflatten(1, (p.kv_heads, p.dim)),
                      table, lens, starts)
    torch.cuda.synchronize()
    return cache, table, lens, starts, rows


@pytest.mark.parametrize("store", ["int8", "e4m3"])
@pytest.mark.parametrize("bad", [("k", float("inf")), ("k", float("nan")), ("v", -float("inf")), ("v", float("nan"))])
@pytest.mark.parametrize("new, where, window, sinks", [(2, 1, 0, 0), (2, 1, 30, 4), (140, 139, 0, 0), (140, 139, 60, 3),
                                                       (140, 12, 20, 0), (140, 12, 20, 40), (20, 0, 2, 0)])
def test_only_who_sees_it(cuda_lib, store, bad, new, where, window, sinks):
    w = cuda_lib
    past = 64 + (-where) % 16                        # the bad token is the first of a page
    p = Problem([past + new, 40], [new, 0], heads=8, kv_heads=2, page=16, store=store, act="f16", seed=new + where)
    cache, table, lens, starts, rows = appended(w, p, bad, where)
    q = rows[:, :p.heads * p.dim].unflatten(1, (p.heads, p.dim))
    out = w.w4a16_kv_attention(q, cache, table, lens, starts, new, window=window, sinks=sinks)
    torch.cuda.synchronize()
    blk = (past + where) // 16
    sees = torch.tensor([bool(visible(past + t, past + new, window, sinks)[blk * 16:blk * 16 + 16].any()) for t in range(new)])
    assert bool(sees.any()) and not bool(sees.all())
    got = out.cpu()
    assert bool(torch.isnan(got[sees][:, :4].float()).all())
    # everyone else: the definition, over a cache whose bad block, which they do not see, is all zeros
    p.k, p.v, p.ks, p.vs = (t.cpu() for t in cache)
    for t in (p.ks, p.vs):
        t[p.table[0, blk].long(), 0] = 1.0 if not bool(torch.isfinite(t[p.table[0, blk].long(), 0])) else t[p.table[0, blk].long(), 0]
    want, _, spread = attention(p, None, window, sinks)
    near = (got.double() - want).abs() <= attention_tolerance(p, want, spread)
    assert bool(near[~sees].all()) and bool(near[:, 4:].all())
    assert w.w4a16_last_device_error() == 0


@pytest.mark.parametrize("store", ["int8", "e4m3"])
@pytest.mark.parametrize("bad", [("k", float("inf")), ("k", float("nan")), ("v", float("inf")), ("v", float("nan"))])
def test_codes_of_a_bad_block_are_zeros(cuda_lib, store, bad):
    w = cuda_lib
    p = Problem([40, 40], [3, 3], kv_heads=2, act="f16", store=store, seed=3)
    before = (p.k.view(torch.int8).clone(), p.v.view(torch.int8).clone())
    cache, table, lens, starts, rows = appended(w, p, bad, 1)
    which = 0 if bad[0] == "k" else 1
    page = int(p.table[0, 2])                        # positions 32..39, five of them there before
    codes = cache[which].view(torch.int8).cpu()
    assert bool((codes[page, 0, :8] == 0).all())     # the new tokens' and the older ones'
    assert not bool((codes[page, 1, :8] == 0).all())
    assert torch.equal(codes[page, 0, 8:], before[which][page, 0, 8:])
    scale = cache[2 + which][page, 0].clone()
    assert not bool(torch.isfinite(scale))
    # a later token: the block stays what it is
    lens += torch.tensor([1, 0], dtype=torch.int32, device="cuda")
    one = torch.tensor([0, 1, 1], dtype=torch.int32, device="cuda")
    x = torch.ones((1, 2, p.dim), dtype=torch.float16, device="cuda")
    w.w4a16_kv_append(cache, x, x, table, lens, one)
    torch.cuda.synchronize()
    assert bool((cache[which].view(torch.int8)[page, 0, :9] == 0).all())
    assert torch.equal(cache[2 + which][page, 0].view(torch.int32), scale.view(torch.int32))
    assert w.w4a16_last_device_error() == 0
