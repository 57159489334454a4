"""Growth by many tokens of a row whose partly filled last page other rows name too: as many of its blocks as a CTA has
threads, one more and one less, shares of several CTAs."""
import pytest
import torch

from test_gpu_kv_grow import check, shared
from test_gpu_kv_pages import counts, pool

pytestmark = pytest.mark.gpu
LENGTH = 905                                                           # 9 tokens in the last page, whatever its size


def grow(w, new, page, kv_heads=8, store="int8", layout="heads", length=LENGTH):
    """Rows of `length` tokens that share all their pages grow by `new`; the pages hold random codes and scales."""
    blocks = -(-length // page)
    need = sum(-(-(length + n) // page) - blocks + 1 for n in new)
    cache, table, n, ref = pool(w, [length], len(new), page, layout, store, kv_heads=kv_heads, spare=need + 5)
    wide = -(-(length + max(new)) // page) - table.shape[1] + 1
    table = torch.cat([table, torch.full((len(new), wide), -1, dtype=torch.int32, device="cuda")], 1).contiguous()
    shared(table, n, ref, [list(range(len(new)))])
    check(w, cache, table, n, ref, new, page=page)
    assert counts(table, ref.shape[0]) == ref.tolist()


@pytest.mark.parametrize("others", [0, 1, 2, 63])
@pytest.mark.parametrize("long", [4071, 4072, 4096, 8192, 70000])
def test_pages_of_16(cuda_lib, long, others):
    grow(cuda_lib, [long] + [i % 3 % 2 for i in range(1, others + 1)], 16)


@pytest.mark.parametrize("others", [2, 15])
@pytest.mark.parametrize("page, long", [(32, 4096), (32, 16312), (32, 70000), (64, 4096), (64, 65272), (64, 70000)])
def test_larger_pages(cuda_lib, page, long, others):
    """A copy that several CTAs have a hand in."""
    grow(cuda_lib, [long] + [1] * others, page)


@pytest.mark.parametrize("at", [0, 1, 2, 3])
@pytest.mark.parametrize("rest", [0, 1])
@pytest.mark.parametrize("store, layout", [("int8", "tokens"), ("e4m3", "heads")])
def test_places(cuda_lib, at, rest, store, layout):
    """Of four rows that share a last page; the last one keeps it where all grow."""
    new = [rest] * 4
    new[at] = 4096
    grow(cuda_lib, new, 16, kv_heads=2, store=store, layout=layout)


@pytest.mark.parametrize("tokens", [255 * 16 - 9, 256 * 16 - 9, 257 * 16 - 9, 511 * 16, 512 * 16 - 9, 513 * 16])
@pytest.mark.parametrize("length", [9, 16, 16 * 300 + 1])
def test_whole_batches_of_blocks(cuda_lib, tokens, length):
    """A row that shares its last page with one that stays as it is, and the same without a partly filled one."""
    grow(cuda_lib, [tokens, 0, 1, 0], 16, kv_heads=1, length=length)
