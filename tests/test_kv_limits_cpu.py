"""Sizes at the edge of what the paged-cache entry points take, checked on the host."""
import pytest

from test_kv_refusals_cpu import ERR_SHAPE, OK, append, attend, batch, cache, lib, read  # noqa: F401


@pytest.mark.parametrize("call", [append, read, attend])
@pytest.mark.parametrize("page_size", [16, 128])
def test_positions_of_a_row(lib, call, page_size):  # noqa: F811
    """A row of the table holds positions that stay 32-bit numbers with a step's keys added or a window taken off."""
    most = ((1 << 31) - (1 << 25)) // page_size
    c = cache(page_size=page_size, head_stride=page_size * 128, page_stride=2 * page_size * 128)
    assert call(lib, c=c, b=batch(max_blocks=most, n_tokens=0)) == 0
    assert call(lib, c=c, b=batch(max_blocks=most + 1, n_tokens=0)) == ERR_SHAPE
    assert call(lib, c=c, b=batch(max_blocks=(1 << 31) // page_size - 1, n_tokens=0)) == ERR_SHAPE


def test_positions_of_the_page_operators(lib):  # noqa: F811
    most = ((1 << 31) - (1 << 25)) // 16
    for blocks, want in ((most, 0), (most + 1, ERR_SHAPE)):
        assert lib.w4a16_kv_trim(OK, OK, 2, blocks, OK, 8, 16, 0, 0, None) == want
        assert lib.w4a16_kv_fork(cache(), OK, OK, 4, blocks, OK, OK, OK, 0, OK, 1 << 20, None) == want


def reference_overlap(n_pages, heads, page, dim, sp, sh, st):
    at = sorted(p * sp + h * sh + t * st for p in range(n_pages) for h in range(heads) for t in range(page))
    return any(b - a < dim for a, b in zip(at, at[1:]))


@pytest.mark.parametrize("n_pages, heads, sp, sh, st", [
    (8, 2, 2048, 128, 128), (8, 2, 4096, 1024, 128), (8, 2, 4096 - 16, 2048, 128), (8, 2, 128, 128, 256), (8, 4, 4096, 128, 256),
    (8, 3, 128, 1024, 3072 - 16),
    # apart: heads or pages outermost or innermost, padded, K and V in turn, and dimensions that interleave
    (8, 2, 4096, 2048, 128), (8, 2, 4096, 128, 256), (8, 2, 2048, 16384, 128), (8, 2, 128, 1024, 2048), (8, 2, 8192, 2176, 144 - 16),
    (8, 2, 8192, 2176, 136 + 8), (1, 2, 0, 2048, 128), (8, 1, 2048, 0, 128), (1, 1, 0, 0, 128), (4, 2, 8192, 640, 256),
    (2, 3, 384, 128, 768), (2, 2, 4096 + 128, 2 * 4096 + 2 * 128, 256)])
def test_rows_that_overlap(lib, n_pages, heads, sp, sh, st):  # noqa: F811
    c = cache(n_pages=n_pages, n_kv_heads=heads, page_stride=sp, head_stride=sh, token_stride=st)
    want = ERR_SHAPE if reference_overlap(n_pages, heads, 16, 128, sp, sh, st) else 0
    assert attend(lib, c=c, b=batch(n_tokens=0), heads=2 * heads) == want
    assert lib.w4a16_kv_copy_pages(c, OK, OK, 0, None) == want
    assert lib.w4a16_kv_fork(c, OK, OK, 4, 4, OK, OK, OK, 0, OK, 1 << 20, None) == want


def test_rows_that_overlap_at_random(lib):  # noqa: F811
    import random
    rng = random.Random(0)
    apart = 0
    for _ in range(3000):
        n_pages, heads = rng.randrange(1, 5), rng.randrange(1, 5)
        sp, sh, st = (16 * rng.randrange(8, rng.choice([12, 40, 200])) for _ in range(3))
        over = reference_overlap(n_pages, heads, 16, 128, sp if n_pages > 1 else 0, sh if heads > 1 else 0, st)
        apart += not over
        c = cache(n_pages=n_pages, n_kv_heads=heads, page_stride=sp, head_stride=sh, token_stride=st)
        assert lib.w4a16_kv_copy_pages(c, OK, OK, 0, None) == (ERR_SHAPE if over else 0), (n_pages, heads, sp, sh, st)
    assert apart > 100
