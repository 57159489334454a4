"""Appending to and reading from the paged 8-bit cache, bit for bit against the
definition, whose arithmetic is fp32."""
import pytest
import torch

from kv_reference import ACT, Problem, append

pytestmark = pytest.mark.gpu


def views(p, rows):
    a, b = p.heads * p.dim, (p.heads + p.kv_heads) * p.dim
    return (rows[:, a:b].unflatten(1, (p.kv_heads, p.dim)), rows[:, b:].unflatten(1, (p.kv_heads, p.dim)))


def same(got, want):
    got, want = got.cpu(), want.cpu()
    if got.dtype == torch.float32:
        return torch.equal(got.view(torch.int32), want.view(torch.int32))
    return torch.equal(got.view(torch.int8), want.view(torch.int8))


def check(w, p):
    want = append(p)
    cache, table, lens, starts, rows = p.to_cuda(w)
    k_new, v_new = views(p, rows)
    for _ in range(2):                               # the second time changes nothing
        w.w4a16_kv_append(cache, k_new, v_new, table, lens, starts)
        torch.cuda.synchronize()
        for name, got, ref in zip(("k", "v", "k_scale", "v_scale"), cache, want):
            assert same(got, ref), name
    assert w.w4a16_last_device_error() == 0
    p.k, p.v, p.ks, p.vs = want[0].view(p.k.dtype), want[1].view(p.v.dtype), want[2], want[3]
    return cache, table, lens, starts


@pytest.mark.parametrize("store", ["int8", "e4m3"])
@pytest.mark.parametrize("act", ["f16", "bf16"])
@pytest.mark.parametrize("dim, page, layout", [(128, 16, "heads"), (64, 16, "tokens"), (128, 64, "padded"), (64, 128, "heads"),
                                               (128, 128, "tokens"), (64, 32, "padded")])
def test_append(cuda_lib, store, act, dim, page, layout):
    new = [1, 0, 1, 40, 129, 7, 300, 1]
    lens = [1, 50, 64, 40, 150, 16, 311, 200]
    check(cuda_lib, Problem(lens, new, 4, 3, dim, page, store, layout, act, seed=dim + page))


@pytest.mark.parametrize("store", ["int8", "e4m3"])
def test_values_of_any_size(cuda_lib, store):
    """Zeros, tiny and large values, and blocks that grow a lot or not at all."""
    p = Problem([20, 33, 3, 90, 17], [4, 20, 3, 30, 1], store=store, seed=1)
    _, k, v = p.rows.split([p.heads * p.dim, p.kv_heads * p.dim, p.kv_heads * p.dim], 1)
    k[:4] = 0
    v[:4] *= 1e-30
    k[4:24] *= 1e30
    v[24:27] = 0
    k[24:27] *= 1e-6
    check(cuda_lib, p)


@pytest.mark.parametrize("store", ["int8", "e4m3"])
def test_ties_round_to_even(cuda_lib, store):
    """amax = qmax makes the scale exactly 1, so half-way values are ties."""
    p = Problem([16], [16], act="bf16", store=store, kv_heads=1, heads=1)
    x = torch.arange(16 * p.dim).float() % 128 - 63.5
    rows = p.rows.view(-1)
    flat = x.view(16, p.dim)
    flat[:, 0] = 127.0 if store == "int8" else 448.0
    p.rows[:, p.dim:2 * p.dim] = flat.to(ACT["bf16"])
    p.rows[:, 2 * p.dim:] = (flat / 2).to(ACT["bf16"])
    assert rows.numel() == 16 * 3 * p.dim
    check(cuda_lib, p)


def test_not_finite_values_make_the_scale_not_finite(cuda_lib):
    w = cuda_lib
    p = Problem([20, 20], [3, 3], kv_heads=2, act="f16")
    p.rows[0, p.heads * p.dim + 5] = float("nan")
    p.rows[1, (p.heads + 2 * p.kv_heads) * p.dim - 1] = float("inf")
    cache, table, lens, starts, rows = p.to_cuda(w)
    w.w4a16_kv_append(cache, *views(p, rows), table, lens, starts)
    torch.cuda.synchronize()
    page = int(p.table[0, 1])
    assert torch.isnan(cache.k_scale[page, 0]) and torch.isfinite(cache.k_scale[page, 1])
    assert torch.isinf(cache.v_scale[page, 1]) and torch.isfinite(cache.v_scale[page, 0])
    assert bool(torch.isfinite(cache.k_scale[p.table[1].long().cuda()]).all())


@pytest.mark.parametrize("store", ["int8", "e4m3"])
@pytest.mark.parametrize("act", ["f16", "bf16"])
@pytest.mark.parametrize("dim, page, layout", [(128, 16, "heads"), (64, 64, "tokens"), (128, 32, "padded")])
def test_read(cuda_lib, store, act, dim, page, layout):
    w = cuda_lib
    new = [5, 0, 1, 200, 33]
    p = Problem([5, 8, 77, 260, 33], new, 4, 3, dim, page, store, layout, act, seed=dim)
    cache, table, lens, starts, _ = p.to_cuda(w)
    k, v = w.w4a16_kv_read(cache, table, lens, starts, p.T, ACT[act])
    torch.cuda.synchronize()
    for got, codes, scales in ((k, p.k, p.ks), (v, p.v, p.vs)):
        want = torch.cat([p.values(codes, scales, b, n)[n - m:] for b, (n, m) in enumerate(zip(p.lens, p.new))])
        # one fp32 product of a code and a scale, rounded to the type: never further than one rounding of each
        assert torch.equal(got.cpu(), (want.float()).to(ACT[act]))
    assert w.w4a16_last_device_error() == 0


def test_token_by_token_is_a_cache(cuda_lib):
    """A sequence appended one token at a time stays within the rounding its growing scales allow."""
    w = cuda_lib
    p = Problem([48], [48], heads=1, kv_heads=2, store="int8", act="bf16", seed=3)
    cache, table, lens, starts, rows = p.to_cuda(w)
    k_new, v_new = views(p, rows)
    one = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    for t in range(48):
        lens.fill_(t + 1)
        w.w4a16_kv_append(cache, k_new[t:t + 1], v_new[t:t + 1], table, lens, one)
    k, _ = w.w4a16_kv_read(cache, table, lens, starts, 48, torch.bfloat16)
    torch.cuda.synchronize()
    scale = cache.k_scale[p.table[0].long().cuda()].repeat_interleave(16, 0)[..., None].double()
    # each rounding is off by half a step of its time, and steps only grow: 15 roundings at most in a page of 16
    assert bool(((k.double() - k_new.double()).abs() <= 8.0 * scale + 2.0 ** -8 * k_new.double().abs()).all())


def test_bad_device_arguments_touch_nothing(cuda_lib):
    w = cuda_lib
    p = Problem([40, 20], [2, 2])
    cache, table, lens, starts, rows = p.to_cuda(w)
    before = [t.clone() for t in cache]

    def reported():
        torch.cuda.synchronize()
        got = w.w4a16_last_device_error()
        w.w4a16_clear_device_error()
        return got == -9 and all(same(a, b) for a, b in zip(cache, before))

    bad = table.clone()
    bad[0, 2], bad[1, 1] = p.n_pages, -5
    w.w4a16_kv_append(cache, *views(p, rows), bad, lens, starts)
    assert reported()
    short = torch.ones_like(lens)                    # tokens before position 0 are dropped; no page but the first is touched
    short[:] = 0
    w.w4a16_kv_append(cache, *views(p, rows), table, short, starts)
    assert reported()
    k, v = w.w4a16_kv_read(cache, bad, lens, starts, 4, torch.float16)
    assert reported()
    assert bool((k[0] == 0).all()) or bool((k[1] == 0).all())


def test_more_units_than_a_grid_has_rows(cuda_lib):
    """70000 sequences of one token: the kernel's pages go on in a second plane of its grid."""
    w, n = cuda_lib, 70000
    g = torch.Generator().manual_seed(5)
    x = torch.randn((n, 2, 64), generator=g).half()
    k = torch.zeros((n, 1, 16, 64), dtype=torch.int8, device="cuda")
    v, ks, vs = torch.zeros_like(k), torch.zeros((n, 1), device="cuda"), torch.zeros((n, 1), device="cuda")
    cache = w.KVCache(k, v, ks, vs)
    table = torch.arange(n, dtype=torch.int32, device="cuda").flip(0).unsqueeze(1).contiguous()
    lens = torch.ones(n, dtype=torch.int32, device="cuda")
    starts = torch.arange(n + 1, dtype=torch.int32, device="cuda")
    rows = x.cuda()
    w.w4a16_kv_append(cache, rows[:, :1], rows[:, 1:], table, lens, starts)
    got = w.w4a16_kv_read(cache, table, lens, starts, n, torch.float16)
    for have, want in zip(got, (x[:, :1].double(), x[:, 1:].double())):
        step = want.abs().amax(dim=-1, keepdim=True) / 127
        # half a step, a little more for the two roundings before the code's, and the output's own
        assert bool(((have.cpu().double() - want).abs() <= step * (0.5 + 2.0 ** -14) + want.abs() * 2.0 ** -10).all())
    assert w.w4a16_last_device_error() == 0
