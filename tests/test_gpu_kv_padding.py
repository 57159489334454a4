"""Rows of a batch that no sequence owns: a captured call of a fixed number of
rows may be replayed with fewer live ones."""
import pytest
import torch

from kv_reference import ACT, Problem, attention, attention_tolerance

pytestmark = pytest.mark.gpu


def padded(p, w, front, back):
    """p's batch in a larger one: `front` rows before the first sequence's, `back` after the last one's."""
    cache, table, lens, starts, rows = p.to_cuda(w)
    wide = torch.full((front + p.T + back, rows.shape[1]), float("nan"), dtype=rows.dtype, device="cuda")
    wide[front:front + p.T] = rows
    return cache, table, lens, starts + front, wide


@pytest.mark.parametrize("front, back", [(0, 1), (0, 37), (3, 0), (5, 300)])
@pytest.mark.parametrize("new, dim, kv_heads", [([1, 1, 1], 128, 2), ([1], 64, 8), ([5, 0, 2], 128, 2), ([140, 200], 128, 2),
                                                ([150], 64, 2), ([1, 140, 0, 3], 128, 2), ([0, 0], 64, 2)])
@pytest.mark.parametrize("said", ["longest", "more"])
def test_attention(cuda_lib, front, back, new, dim, kv_heads, said):
    w = cuda_lib
    p = Problem([n + 50 for n in new], new, 8, kv_heads, dim, seed=sum(new) + front)
    cache, table, lens, starts, rows = padded(p, w, front, back)
    q = rows[:, :8 * dim].unflatten(1, (8, dim))
    out = torch.full(q.shape, float("nan"), dtype=q.dtype, device="cuda")
    lse = torch.full(q.shape[:2], float("nan"), device="cuda")
    w.w4a16_kv_attention(q, cache, table, lens, starts, max(new) if said == "longest" else 1000, out=out, lse=lse)
    torch.cuda.synchronize()
    own = slice(front, front + p.T)
    want, want_lse, spread = attention(p)
    assert bool(((out[own].cpu().double() - want).abs() <= attention_tolerance(p, want, spread)).all())
    assert bool(torch.isfinite(lse[own]).all())
    for rest in (slice(0, front), slice(front + p.T, None)):
        assert bool((out[rest] == 0).all())
        assert bool((lse[rest] == -float("inf")).all())
    assert w.w4a16_last_device_error() == 0


def test_attention_of_more_sequences_than_a_launch_takes(cuda_lib):
    w = cuda_lib
    for new in ([1] * 1030, [30] * 520):
        p = Problem([n + 3 for n in new], new, 8, 2, 64, seed=4)
        cache, table, lens, starts, rows = padded(p, w, 7, 9)
        q = rows[:, :8 * 64].unflatten(1, (8, 64))
        out = torch.full(q.shape, float("nan"), dtype=q.dtype, device="cuda")
        w.w4a16_kv_attention(q, cache, table, lens, starts, max(new), out=out)
        torch.cuda.synchronize()
        want, _, spread = attention(p)
        assert bool(((out[7:-9].cpu().double() - want).abs() <= attention_tolerance(p, want, spread)).all())
        assert bool((out[:7] == 0).all()) and bool((out[-9:] == 0).all())
        assert w.w4a16_last_device_error() == 0


@pytest.mark.parametrize("front, back", [(0, 40), (3, 2)])
def test_append_and_read(cuda_lib, front, back):
    w = cuda_lib
    p = Problem([20, 70, 33], [3, 0, 33], seed=front)
    cache, table, lens, starts, rows = p.to_cuda(w)
    a, b = p.heads * p.dim, (p.heads + p.kv_heads) * p.dim

    def views(x):
        return x[:, a:b].unflatten(1, (p.kv_heads, p.dim)), x[:, b:].unflatten(1, (p.kv_heads, p.dim))

    w.w4a16_kv_append(cache, *views(rows), table, lens, starts)
    k, v = w.w4a16_kv_read(cache, table, lens, starts, p.T, ACT[p.act])
    cache2, table, lens, starts, wide = padded(p, w, front, back)
    w.w4a16_kv_append(cache2, *views(wide), table, lens, starts)
    k2, v2 = (torch.full((front + p.T + back, p.kv_heads, p.dim), float("nan"), dtype=ACT[p.act], device="cuda") for _ in range(2))
    w.w4a16_kv_read(cache2, table, lens, starts, front + p.T + back, ACT[p.act], k_out=k2, v_out=v2)
    torch.cuda.synchronize()
    for x, y in zip(cache, cache2):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    for x, y in ((k, k2), (v, v2)):
        assert torch.equal(x, y[front:front + p.T])
        assert bool((y[:front] == 0).all()) and bool((y[front + p.T:] == 0).all())
    assert w.w4a16_last_device_error() == 0
