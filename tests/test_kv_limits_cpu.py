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
