"""Rows of the tables that become other rows: entries, lengths and counts."""
import pytest
import torch

from test_gpu_kv_pages import counts

pytestmark = pytest.mark.gpu


def tables(rows, width, pages, seed=0, full=0.7):
    """Random rows over pages; some entries are trimmed, many pages are in several rows."""
    g = torch.Generator().manual_seed(seed)
    table = torch.randint(0, pages, (rows, width), generator=g, dtype=torch.int32)
    table[torch.rand((rows, width), generator=g) > full] = -1
    lens = torch.randint(0, 16 * width + 1, (rows,), generator=g, dtype=torch.int32)
    ref = torch.tensor(counts(table, pages), dtype=torch.int32)
    return table.cuda(), lens.cuda(), ref.cuda(), g


def want(table, lens, src, dst):
    t, n = table.clone(), lens.clone()
    for i, s in enumerate(src):
        d = i if dst is None else dst[i]
        if s >= table.shape[0] or not 0 <= d < table.shape[0]:
            continue
        t[d] = table[s] if s >= 0 else -1
        n[d] = lens[s] if s >= 0 else 0
    return t, n


def check(w, table, lens, ref, src, dst=None, error=0, stream=None):
    t, n = want(table.cpu(), lens.cpu(), src, dst)
    put = lambda v: torch.tensor(v, dtype=torch.int32).cuda()
    a, b = put(src), None if dst is None else put(dst)
    torch.cuda.synchronize()
    w.w4a16_kv_reorder(table, lens, ref, a, b, stream=stream)
    torch.cuda.synchronize()
    assert torch.equal(table.cpu(), t) and torch.equal(lens.cpu(), n)
    assert ref.tolist() == counts(t, ref.shape[0])
    assert w.w4a16_last_device_error() == error
    w.w4a16_clear_device_error()


@pytest.mark.parametrize("rows, width", [(1, 1), (2, 1), (4, 60), (7, 8), (33, 65), (256, 31), (1024, 9)])
def test_rows(cuda_lib, rows, width):
    table, lens, ref, g = tables(rows, width, 3 * rows + 5, seed=rows + width)
    for _ in range(3):
        src = torch.randint(-1, rows, (rows,), generator=g).tolist()
        check(cuda_lib, table, lens, ref, src)


@pytest.mark.parametrize("src", [[1, 2, 3, 0], [3, 2, 1, 0], [0, 1, 2, 3], [2, 2, 2, 2], [-1, 0, -1, 1], [-1, -1, -1, -1]])
def test_cycles_copies_and_ends(cuda_lib, src):
    table, lens, ref, _ = tables(6, 20, 30, seed=3)
    check(cuda_lib, table, lens, ref, src)                  # the other two rows stay


def test_listed_rows(cuda_lib):
    table, lens, ref, g = tables(40, 17, 90, seed=5)
    dst = torch.randperm(40, generator=g)[:23].tolist()
    src = torch.randint(-2, 40, (23,), generator=g).tolist()
    check(cuda_lib, table, lens, ref, src, dst)
    check(cuda_lib, table, lens, ref, [], [])


def test_ids_out_of_range(cuda_lib):
    table, lens, ref, _ = tables(5, 9, 20, seed=6)
    check(cuda_lib, table, lens, ref, [4, 5, 0, 2**31 - 1], error=-9)
    check(cuda_lib, table, lens, ref, [4, 3, 0], [-1, 5, 2], error=-9)


def test_pages_out_of_range(cuda_lib):
    """An entry that names no page goes on as none; a count that is 0 already stays."""
    w = cuda_lib
    table = torch.tensor([[0, 7, -5], [1, 2, 3]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([40, 41], dtype=torch.int32, device="cuda")
    ref = torch.tensor([1, 0, 1, 1], dtype=torch.int32, device="cuda")
    w.w4a16_kv_reorder(table, lens, ref, torch.tensor([0, 0], dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert table[1].tolist() == [0, -1, -1] and lens.tolist() == [40, 40]
    assert ref.tolist() == [2, 0, 0, 0]
    assert w.w4a16_last_device_error() == -9
    w.w4a16_clear_device_error()


@pytest.mark.parametrize("rows, width", [(4096, 5), (16384, 3)])
def test_many_rows(cuda_lib, rows, width):
    table, lens, ref, g = tables(rows, width, rows, seed=7)
    check(cuda_lib, table, lens, ref, torch.randint(-1, rows, (rows,), generator=g).tolist())
    dst = torch.randperm(rows, generator=g)[:rows // 2 + 1].tolist()
    check(cuda_lib, table, lens, ref, torch.randint(-1, rows, (len(dst),), generator=g).tolist(), dst)


def test_other_stream(cuda_lib):
    table, lens, ref, _ = tables(12, 30, 50, seed=8)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    check(cuda_lib, table, lens, ref, [3, 3, 1, 11, 0, 5], stream=s)


def test_captured(cuda_lib):
    w = cuda_lib
    table, lens, ref, g = tables(9, 21, 40, seed=9)
    src = torch.arange(9, dtype=torch.int32, device="cuda")
    w.w4a16_kv_reorder(table, lens, ref, src)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w.w4a16_kv_reorder(table, lens, ref, src)
    for _ in range(4):
        src.copy_(torch.randint(-1, 9, (9,), generator=g, dtype=torch.int32))
        t, n = want(table.cpu(), lens.cpu(), src.tolist(), None)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(table.cpu(), t) and torch.equal(lens.cpu(), n) and ref.tolist() == counts(t, 40)
    assert w.w4a16_last_device_error() == 0
