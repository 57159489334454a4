"""The bounded waits of the attention over the 8-bit cache, made to run out on purpose without a fault: with the test hook on, all
CTAs or every second one issue no copies.  The kernels leave, the status word reads W4A16_ERR_TIMEOUT, and the next call
is right again."""
import pytest
import torch

from kv_reference import Problem, attention, attention_tolerance

pytestmark = pytest.mark.gpu

W4A16_ERR_TIMEOUT = -8
# few rows; many rows dealt out whole; many rows in shares; both kernels
CASES = [([1, 1], [9000, 5000]), ([300], [400]), ([9] * 12, [3000 + 400 * i for i in range(12)]), ([1, 9, 30], [7000, 4000, 3000])]


def held(w, hold, call):
    w.w4a16_clear_device_error()
    w.w4a16_debug_set_config(7, [hold])
    try:
        call()
        torch.cuda.synchronize()
    finally:
        w.w4a16_debug_set_config(7, None)
    assert w.w4a16_last_device_error() == W4A16_ERR_TIMEOUT
    w.w4a16_clear_device_error()


@pytest.mark.parametrize("new, lens", CASES)
@pytest.mark.parametrize("dim, page, layout", [(128, 16, "heads"), (64, 64, "tokens")])
@pytest.mark.parametrize("hold", [1, 2])
def test_waits_run_out_and_the_next_call_is_right(cuda_lib, new, lens, dim, page, layout, hold):
    w = cuda_lib
    p = Problem(lens, new, heads=8, kv_heads=2, dim=dim, page=page, layout=layout, seed=len(new))
    cache, table, n, starts, rows = p.to_cuda(w)
    q = rows[:, :8 * dim].unflatten(1, (8, dim))
    held(w, hold, lambda: w.w4a16_kv_attention(q, cache, table, n, starts, max(new)))
    out = w.w4a16_kv_attention(q, cache, table, n, starts, max(new))
    torch.cuda.synchronize()
    want, _, spread = attention(p)
    assert bool(((out.cpu().double() - want).abs() <= attention_tolerance(p, want, spread)).all())
    assert w.w4a16_last_device_error() == 0


@pytest.mark.parametrize("new, lens", CASES)
@pytest.mark.parametrize("dim, page, layout", [(128, 16, "heads"), (64, 64, "tokens")])
@pytest.mark.parametrize("hold", [2, 3])
def test_tickets_are_back_at_zero(cuda_lib, new, lens, dim, page, layout, hold):
    """A replay of the same launch counts on from what it finds: every ticket taken has to be given back."""
    w = cuda_lib
    p = Problem(lens, new, heads=8, kv_heads=2, dim=dim, page=page, layout=layout, seed=len(new))
    cache, table, n, starts, rows = p.to_cuda(w)
    q = rows[:, :8 * dim].unflatten(1, (8, dim))
    ws = torch.zeros(w.w4a16_kv_attention_workspace(8, 2, dim, len(new), p.T), dtype=torch.uint8, device="cuda")
    tickets = ws.view(torch.int64)[:torch.cuda.get_device_properties(0).multi_processor_count]

    def call():
        return w.w4a16_kv_attention(q, cache, table, n, starts, max(new), workspace=ws)

    call()
    torch.cuda.synchronize()
    assert not bool(tickets.any())
    held(w, hold, call)
    assert not bool(tickets.any())
    out = call()
    torch.cuda.synchronize()
    want, _, spread = attention(p)
    assert bool(((out.cpu().double() - want).abs() <= attention_tolerance(p, want, spread)).all())
    assert not bool(tickets.any())
    assert w.w4a16_last_device_error() == 0
