"""What attention over a common prefix, growth, reordering and beam selection refuse on the
host, before any device is touched, and what the binding refuses before the C call."""
import pytest
import torch

from test_kv_refusals_cpu import (ERR_ALIGN, ERR_ARG, ERR_DTYPE, ERR_NULL, ERR_SHAPE, NULL, OK, batch, cache,  # noqa: F401
                                  lib)


def grow(lib, c=None, table=OK, lens=OK, seqs=2, blocks=4, ref=OK, new=OK, tokens=3, starts=OK, pos=OK, slots=OK, ws=OK,
         size=1 << 40):
    return lib.w4a16_kv_grow(c or cache(), table, lens, seqs, blocks, ref, new, tokens, starts, pos, slots, ws, size, None)


def reorder(lib, table=OK, lens=OK, seqs=4, blocks=4, ref=OK, pages=8, dst=NULL, src=OK, n=2):
    return lib.w4a16_kv_reorder(table, lens, seqs, blocks, ref, pages, dst, src, n, None)


def select(lib, logits=OK, stride=100, dtype=0, scores=OK, finished=NULL, groups=2, width=4, vocab=100, end=-1, n=4, os=OK,
           rows=OK, tokens=OK, fin=OK, ws=OK, size=1 << 40):
    return lib.w4a16_beam_select(logits, stride, dtype, scores, finished, groups, width, vocab, end, n, os, rows, tokens, fin,
                                 ws, size, None)


def shared(lib, c=None, b=None, q=OK, qs=1024, heads=8, most=1, starts=OK, prefix=OK, groups=1, scale=0.1, out=OK, lse=None,
           dt=0, ws=OK, size=1 << 40):
    return lib.w4a16_kv_attention_shared(q, qs, heads, c or cache(), b or batch(), most, starts, prefix, groups, scale, out, lse,
                                         dt, ws, size, None)


def test_attention_shared(lib):  # noqa: F811
    assert shared(lib, dt=2) == ERR_DTYPE and shared(lib, c=cache(kv_dtype=2)) == ERR_DTYPE
    for bad in (dict(heads=0), dict(heads=7), dict(heads=2 * 129), dict(groups=-1), dict(groups=3), dict(qs=1000),
                dict(c=cache(page_size=8)), dict(b=batch(n_seqs=-1)), dict(b=batch(n_tokens=1 << 24), heads=256, qs=1 << 15)):
        assert shared(lib, **bad) == ERR_SHAPE, bad
    for bad in (dict(q=NULL), dict(out=NULL), dict(ws=NULL), dict(starts=NULL), dict(prefix=NULL),
                dict(b=batch(kv_lens=NULL))):
        assert shared(lib, **bad) == ERR_NULL, bad
    for bad in (dict(q=OK + 8), dict(out=OK + 4), dict(lse=OK + 2), dict(ws=OK + 8), dict(starts=OK + 2), dict(prefix=OK + 1),
                dict(qs=1028)):
        assert shared(lib, **bad) == ERR_ALIGN, bad
    assert shared(lib, most=-1) == ERR_ARG and shared(lib, scale=float("nan")) == ERR_ARG
    assert shared(lib, b=batch(n_tokens=0), q=NULL, out=NULL, ws=NULL, starts=NULL) == 0


def test_attention_shared_workspace(lib):  # noqa: F811
    import ctypes
    need = ctypes.c_longlong(0)
    assert lib.w4a16_kv_attention_shared_workspace(8, 2, 128, 4, 1, 4, None) == ERR_NULL
    for bad in ((0, 2, 128, 4, 1, 4), (8, 3, 128, 4, 1, 4), (8, 2, 96, 4, 1, 4), (8, 2, 128, -1, 0, 4), (8, 2, 128, 4, 5, 4),
                (8, 2, 128, 4, -1, 4), (8, 2, 128, 4, 1, -1)):
        assert lib.w4a16_kv_attention_shared_workspace(*bad, ctypes.byref(need)) == ERR_SHAPE, bad


def test_grow(lib):  # noqa: F811
    assert grow(lib, c=cache(kv_dtype=3)) == ERR_DTYPE
    for bad in (dict(c=cache(page_size=24)), dict(seqs=-1), dict(seqs=8193), dict(blocks=0), dict(blocks=1 << 28),
                dict(tokens=-1), dict(tokens=(1 << 24) + 1)):
        assert grow(lib, **bad) == ERR_SHAPE, bad
    for bad in ("table", "lens", "ref", "new", "starts", "pos", "slots", "ws"):
        assert grow(lib, **{bad: NULL}) == ERR_NULL, bad
    for bad in (dict(table=OK + 2), dict(lens=OK + 1), dict(ref=OK + 2), dict(new=OK + 3), dict(starts=OK + 2),
                dict(pos=OK + 2), dict(slots=OK + 4), dict(ws=OK + 8)):
        assert grow(lib, **bad) == ERR_ALIGN, bad
    assert grow(lib, size=100) == ERR_ARG


def test_grow_workspace(lib):  # noqa: F811
    import ctypes
    need = ctypes.c_longlong(0)
    assert lib.w4a16_kv_grow_workspace(8, 2, None) == ERR_NULL
    for bad in ((0, 2), ((1 << 28) + 1, 2), (8, -1), (8, 8193)):
        assert lib.w4a16_kv_grow_workspace(*bad, ctypes.byref(need)) == ERR_SHAPE
    assert lib.w4a16_kv_grow_workspace(8, 2, ctypes.byref(need)) == 0
    # a bit a page, a count a chunk, 32 bytes a row
    assert need.value >= 4 + 128 + 2 * 32
    assert grow(lib, size=need.value - 1) == ERR_ARG


def test_reorder(lib):  # noqa: F811
    for bad in (dict(seqs=-1), dict(blocks=0), dict(pages=0), dict(n=-1), dict(n=5), dict(seqs=20000, n=16385)):
        assert reorder(lib, **bad) == ERR_SHAPE, bad
    for bad in ("table", "lens", "ref", "src"):
        assert reorder(lib, **{bad: NULL}) == ERR_NULL, bad
    for bad in (dict(table=OK + 2), dict(lens=OK + 1), dict(ref=OK + 2), dict(src=OK + 3), dict(dst=OK + 1)):
        assert reorder(lib, **bad) == ERR_ALIGN, bad
    assert reorder(lib, n=0) == 0


def test_select(lib):  # noqa: F811
    assert select(lib, dtype=3) == ERR_DTYPE and select(lib, dtype=-1) == ERR_DTYPE
    for bad in (dict(groups=-1), dict(width=0), dict(width=65), dict(n=0), dict(n=65), dict(vocab=0), dict(stride=99),
                dict(vocab=(1 << 24) + 1, stride=1 << 25), dict(groups=1 << 19, width=4), dict(stride=1 << 32)):
        assert select(lib, **bad) == ERR_SHAPE, bad
    for bad in ("logits", "scores", "os", "rows", "tokens", "ws"):
        assert select(lib, **{bad: NULL}) == ERR_NULL, bad
    for bad in (dict(logits=OK + 1), dict(logits=OK + 2, dtype=2), dict(scores=OK + 2), dict(os=OK + 1), dict(rows=OK + 2),
                dict(tokens=OK + 3), dict(ws=OK + 8)):
        assert select(lib, **bad) == ERR_ALIGN, bad
    assert select(lib, finished=OK, end=-1) == ERR_ARG and select(lib, finished=OK, end=100) == ERR_ARG
    assert select(lib, groups=0) == 0


def test_gemm_takes_no_fp32(lib):  # noqa: F811
    assert lib.w4a16_gemm(OK, 1, 128, OK, OK, None, 32, 64, OK, None, 2) == ERR_DTYPE


def test_binding():
    """CPU tensors are refused by name, whatever else is right."""
    import w4a16_group_quantised_gb300 as w
    i = torch.zeros(4, dtype=torch.int32)
    kv = w.KVCache(torch.zeros((4, 1, 16, 64), dtype=torch.int8), torch.zeros((4, 1, 16, 64), dtype=torch.int8),
                   torch.zeros((4, 1)), torch.zeros((4, 1)))
    with pytest.raises(ValueError, match="cache.k"):
        w.w4a16_kv_grow(kv, i.view(2, 2), i[:2], i, i[:2], 3)
    with pytest.raises(ValueError, match="cache.k"):
        w.w4a16_kv_attention_shared(torch.zeros((2, 4, 64)), kv, i.view(2, 2), i[:2], i[:3], 1, i[:2], i[:1])
    with pytest.raises(ValueError, match="block_table"):
        w.w4a16_kv_reorder(i.view(2, 2), i[:2], i, i[:2])
    with pytest.raises(ValueError, match="logits"):
        w.w4a16_beam_select(torch.zeros((4, 10)), torch.zeros(4), 2, 2)
    with pytest.raises(TypeError, match="logits"):
        w.w4a16_beam_select([1.0], torch.zeros(4), 2, 2)
