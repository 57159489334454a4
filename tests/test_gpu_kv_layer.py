"""The example's attention block end to end: 4-bit projections, the 8-bit
cache, forks, trims and compaction, against 64-bit products of the block's own
stages."""
import importlib.util
import os

import pytest
import torch

from kv_reference import ROUND

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example(cuda_lib):
    spec = importlib.util.spec_from_file_location("decoder_attention", os.path.join(ROOT, "examples", "decoder_attention.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def values(cache, table, b, n):
    pages = table[b, :-(-n // cache.k.shape[2])].long().clamp(min=0)
    return [(c[pages].double() * s[pages].double()[..., None, None]).transpose(1, 2).flatten(0, 1)[:n]
            for c, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale))]


def check_step(ex, block, seqs, x, new, window, sinks):
    """One step, its attention against the definition over the cache that the step left behind."""
    w = ex.w
    y, o = ex.step(block, seqs, x, new, window, sinks)
    qkv = w.w4a16_gemm(x, block.qkv, block.qkv_scales, None, block.G)
    q = qkv[:, :block.heads * block.dim].unflatten(1, (block.heads, block.dim)).double()
    at, group = 0, block.heads // block.kv_heads
    for b, m in enumerate(new):
        n = seqs.lens[b]
        if m == 0:
            continue
        k, v = values(seqs.cache, seqs.table, b, n)
        i = torch.arange(n - m, n, device="cuda")[:, None]
        j = torch.arange(n, device="cuda")[None]
        see = (j <= i) & ((i - j < window) | (j < sinks)) if window else j <= i
        for a in range(block.heads):
            s = (q[at:at + m, a] @ k[:, a // group].T * block.dim ** -0.5).masked_fill(~see, -float("inf"))
            p = torch.softmax(s, -1)
            want, spread = p @ v[:, a // group], p @ v[:, a // group].abs()
            # one rounding of the output and fp16 weights, as for the attention's own tests
            tol = ROUND["bf16"] * want.abs() + (2.0 ** -11 + 2.0 ** -12) * spread + 2.0 ** -134
            assert bool(((o[at:at + m, a].double() - want).abs() <= tol).all())
        at += m
    assert w.w4a16_last_device_error() == 0
    return y


def test_block(example):
    ex = example
    block = ex.Block(hidden=512, heads=8, kv_heads=2, dim=64, G=64)
    seqs = ex.Sequences(block, rows=6, pages=80, width=20)
    g = torch.Generator(device="cuda").manual_seed(0)

    def tokens(n):
        return torch.randn((n, 512), generator=g, device="cuda").to(torch.bfloat16)

    check_step(ex, block, seqs, tokens(150 + 33 + 5), [150, 33, 5, 0, 0, 0], 0, 0)
    before = seqs.cache.k[seqs.table[0, :9].long()].clone()
    seqs.fork(0, [3, 4])
    seqs.fork(2, [5])
    assert torch.equal(seqs.table[3, :9], seqs.table[0, :9]) and int(seqs.table[3, 9]) != int(seqs.table[0, 9])
    # each of the forks goes its own way; what they share stays as it was
    for _ in range(3):
        check_step(ex, block, seqs, tokens(6), [1] * 6, 0, 0)
    check_step(ex, block, seqs, tokens(30), [5] * 6, 40, 4)
    assert torch.equal(before, seqs.cache.k[seqs.table[0, :9].long()])
    seqs.free([0, 2])
    seqs.close_up(40, 4)
    torch.cuda.synchronize()
    live = int((seqs.refcount > 0).sum())
    assert bool((seqs.refcount[:live] > 0).all()) and live < 30
    x = check_step(ex, block, seqs, tokens(4), [0, 1, 0, 1, 1, 1], 40, 4)
    assert x.shape == (4, 512) and bool(torch.isfinite(x.float()).all())


def test_projection_matches_the_codes(example):
    """The block's first projection is the product with its own codes: the layer is wired as it says."""
    ex = example
    block = ex.Block(hidden=512, heads=4, kv_heads=2, dim=64, G=64, seed=3)
    x = torch.randn((3, 512), device="cuda").to(torch.bfloat16)
    y = ex.w.w4a16_gemm(x, block.qkv, block.qkv_scales, None, 64)
    s = block.qkv_scales.double().repeat_interleave(64, 1)
    wd = ((block.qkv_codes.double() - 8) * s).to(torch.bfloat16).double()
    want = x.double() @ wd.T
    assert bool(((y.double() - want).abs() <= 2.0 ** -8 * want.abs() + 512 * 2.0 ** -23 * (x.double().abs() @ wd.abs().T)).all())


def test_main_runs(example, capsys):
    example.main()
    assert "output finite: True" in capsys.readouterr().out
