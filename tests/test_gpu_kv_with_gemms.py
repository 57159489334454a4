"""Attention of many rows and GEMMs of many rows one after the other on a stream, each starting while the one before it
drains: both take tensor memory."""
import pytest
import torch

from kv_reference import Problem, attention, attention_tolerance

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("new", [[300], [140, 900, 200]])
def test_in_turn(cuda_lib, dim, new):
    w = cuda_lib
    p = Problem([n + 200 for n in new], new, heads=8, kv_heads=2, dim=dim, act="bf16", seed=dim)
    cache, table, lens, starts, rows = p.to_cuda(w)
    q = rows[:, :8 * dim].unflatten(1, (8, dim))
    g = torch.Generator(device="cuda").manual_seed(0)
    codes = torch.randint(0, 16, (2048, 8 * dim), generator=g, device="cuda", dtype=torch.uint8)
    packed = w.w4a16_pack(codes)
    scales = torch.full((2048, 8 * dim // 128), 0.01, device="cuda", dtype=torch.bfloat16)
    x = q.reshape(p.T, -1).contiguous()
    alone = w.w4a16_gemm(x, packed, scales, None, 128)
    torch.cuda.synchronize()
    outs, ys = [], []
    for _ in range(30):
        outs.append(w.w4a16_kv_attention(q, cache, table, lens, starts, max(new)))
        ys.append(w.w4a16_gemm(x, packed, scales, None, 128))
    chained = w.w4a16_gemm(outs[-1].flatten(1), packed, scales, None, 128)
    torch.cuda.synchronize()
    want, _, spread = attention(p)
    assert bool(((outs[0].cpu().double() - want).abs() <= attention_tolerance(p, want, spread)).all())
    assert all(torch.equal(o, outs[0]) for o in outs) and all(torch.equal(y, alone) for y in ys)
    assert torch.equal(chained, w.w4a16_gemm(outs[0].flatten(1).clone(), packed, scales, None, 128))
    assert w.w4a16_last_device_error() == 0
