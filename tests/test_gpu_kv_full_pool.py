"""Compacting a pool whose every page is in use: nothing moves, whatever the number of pages."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("pages", [1, 31, 32, 33, 100, 1023, 1024, 1025, 2048, 3001])
@pytest.mark.parametrize("stale", [0, 255])
def test_compact_a_full_pool(cuda_lib, pages, stale):
    w = cuda_lib
    g = torch.Generator(device="cuda").manual_seed(pages)
    k, v = (torch.randint(-128, 128, (pages, 1, 16, 64), generator=g, device="cuda", dtype=torch.int8) for _ in range(2))
    ks, vs = (torch.empty((pages, 1), device="cuda").uniform_(0.5, 2.0, generator=g) for _ in range(2))
    cache = w.KVCache(k, v, ks, vs)
    before = [t.clone() for t in cache]
    table = torch.randperm(pages, generator=g, device="cuda").int().unsqueeze(0)
    ref = torch.ones(pages, dtype=torch.int32, device="cuda")
    ref[0] = 3
    rows, counts = table.clone(), ref.clone()
    n_live = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.full((w.w4a16_kv_pool_workspace(pages),), stale, dtype=torch.uint8, device="cuda")
    w.w4a16_kv_compact(cache, table, ref, n_live=n_live, workspace=ws)
    torch.cuda.synchronize()
    assert int(n_live) == pages
    assert torch.equal(table, rows) and torch.equal(ref, counts)
    assert all(torch.equal(a, b) for a, b in zip(cache, before))
    assert w.w4a16_last_device_error() == 0


@pytest.mark.parametrize("pages", [33, 1025])
def test_one_page_free(cuda_lib, pages):
    """The neighbour of the full pool: the last page moves into the only hole, or the hole is the last page."""
    w = cuda_lib
    for hole in (0, pages // 2, pages - 1):
        k = torch.arange(pages, device="cuda").remainder(127).to(torch.int8)[:, None, None, None].expand(pages, 1, 16, 64).contiguous()
        cache = w.KVCache(k, k.clone(), torch.ones((pages, 1), device="cuda"), torch.ones((pages, 1), device="cuda"))
        table = torch.tensor([[p for p in range(pages) if p != hole]], dtype=torch.int32, device="cuda")
        ref = torch.ones(pages, dtype=torch.int32, device="cuda")
        ref[hole] = 0
        w.w4a16_kv_compact(cache, table, ref)
        torch.cuda.synchronize()
        want = [p if p != pages - 1 else hole for p in range(pages) if p != hole]
        assert table[0].tolist() == want
        assert ref.tolist() == [1] * (pages - 1) + [0]
        if hole != pages - 1:
            assert int(cache.k[hole, 0, 0, 0]) == (pages - 1) % 127 and int(cache.v[hole, 0, 15, 63]) == (pages - 1) % 127
        assert w.w4a16_last_device_error() == 0
