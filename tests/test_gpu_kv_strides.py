"""Strides of dimensions of one element say nothing: they may be anything."""
import pytest
import torch

from kv_reference import Problem, append, attention, attention_tolerance

pytestmark = pytest.mark.gpu


def restrided(t, dim, stride):
    """t, whose dimension `dim` has one element, with another stride there."""
    strides = list(t.stride())
    strides[dim] = stride
    return torch.as_strided(t, t.shape, strides)


@pytest.mark.parametrize("new", [1, 60])
@pytest.mark.parametrize("stride", [0, 24, 64, 1 << 45])
def test_one_kv_head(cuda_lib, new, stride):
    w = cuda_lib
    p = Problem([new + 90, new], [new, new], heads=4, kv_heads=1, dim=64, seed=new)
    cache, table, lens, starts, rows = p.to_cuda(w)
    cache = cache._replace(v=restrided(cache.v, 1, stride))
    q = rows[:, :4 * 64].unflatten(1, (4, 64))
    out = w.w4a16_kv_attention(q, cache, table, lens, starts, new)
    want, _, spread = attention(p)
    assert bool(((out.cpu().double() - want).abs() <= attention_tolerance(p, want, spread)).all())
    both = w.KVCache(restrided(cache.k, 1, stride), cache.v, cache.k_scale, cache.v_scale)
    assert torch.equal(out, w.w4a16_kv_attention(q, both, table, lens, starts, new))
    assert w.w4a16_last_device_error() == 0


@pytest.mark.parametrize("stride", [0, 16, 72])
def test_one_page(cuda_lib, stride):
    w = cuda_lib
    p = Problem([9], [4], seed=2, spare=0)
    cache, table, lens, starts, rows = p.to_cuda(w)
    assert cache.k.shape[0] == 1
    want = append(p)
    a, b = p.heads * p.dim, (p.heads + p.kv_heads) * p.dim
    odd = cache._replace(k=restrided(cache.k, 0, stride), v=restrided(cache.v, 0, 5 * stride))
    w.w4a16_kv_append(odd, rows[:, a:b].unflatten(1, (p.kv_heads, p.dim)), rows[:, b:].unflatten(1, (p.kv_heads, p.dim)),
                      table, lens, starts)
    torch.cuda.synchronize()
    for got, ref in zip(cache, want):
        assert torch.equal(got.cpu().view(torch.uint8), ref.view(torch.uint8))
    p.k, p.v, p.ks, p.vs = want[0].view(p.k.dtype), want[1].view(p.v.dtype), want[2], want[3]
    out = w.w4a16_kv_attention(rows[:, :a].unflatten(1, (p.heads, p.dim)), odd, table, lens, starts, 4)
    ref, _, spread = attention(p)
    assert bool(((out.cpu().double() - ref).abs() <= attention_tolerance(p, ref, spread)).all())
    assert w.w4a16_last_device_error() == 0


def test_one_token_of_rows_of_an_odd_width(cuda_lib):
    """One row has no next one: its stride need not be a multiple of eight."""
    w = cuda_lib
    p = Problem([70], [1], seed=3)
    want = append(p)
    cache, table, lens, starts, rows = p.to_cuda(w)
    a, b = p.heads * p.dim, (p.heads + p.kv_heads) * p.dim
    q, k_new, v_new = (restrided(rows[:, x:y].unflatten(1, (-1, p.dim)), 0, rows.shape[1] + 3) for x, y in ((0, a), (a, b), (b, None)))
    assert q.stride(0) % 8 and q.stride(0) > a
    w.w4a16_kv_append(cache, k_new, v_new, table, lens, starts)
    torch.cuda.synchronize()
    for got, ref in zip(cache, want):
        assert torch.equal(got.cpu().view(torch.uint8), ref.view(torch.uint8))
    p.k, p.v, p.ks, p.vs = want[0].view(p.k.dtype), want[1].view(p.v.dtype), want[2], want[3]
    out = w.w4a16_kv_attention(q, cache, table, lens, starts, 1)
    ref, _, spread = attention(p)
    assert bool(((out.cpu().double() - ref).abs() <= attention_tolerance(p, ref, spread)).all())
    assert w.w4a16_last_device_error() == 0
