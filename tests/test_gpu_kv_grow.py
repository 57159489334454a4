"""Growth of sequences: tables, counts, copies, starts, positions and slots,
against a model that serves the rows one after the other."""
import pytest
import torch

from test_gpu_kv_pages import counts, pool, snapshot

pytestmark = pytest.mark.gpu


def model(table, lens, ref, new, page, n_tokens):
    """(tables after the call, copies (src, dst), anything wrong) of lists, in the order of rows."""
    table, lens, ref = [list(r) for r in table], list(lens), list(ref)
    n_pages, cap = len(ref), len(table[0]) * page if table else 0
    free = [p for p in range(n_pages) if ref[p] == 0]
    # who may keep a last page: the last of its growing rows, when they are all that name it
    named, wrong, plan = {}, False, []
    for b, n in enumerate(new):
        ok = 0 <= lens[b] <= cap and n >= 0 and lens[b] + n <= cap
        last = table[b][lens[b] // page] if ok and n > 0 and lens[b] % page else None
        if last is not None and not 0 <= last < n_pages:
            ok = False
        wrong |= not ok
        plan.append((n if ok else 0, last if ok else None))
    left = dict()
    starts, positions, slots, copies, stopped, at = [0], [], [], [], False, 0
    for b, (n, last) in enumerate(plan):
        copy = last is not None and ref[last] - left.get(last, 0) > 1
        need = -(-(lens[b] + n) // page) - -(-lens[b] // page) + copy
        if stopped or at + need > len(free) or starts[-1] + n > n_tokens:
            stopped = True
            starts.append(starts[-1])
            continue
        pages, at = free[at:at + need], at + need
        if copy:
            left[last] = left.get(last, 0) + 1
            copies.append((last, pages[0]))
        first = -(-lens[b] // page) - copy
        for i, p in enumerate(pages):
            table[b][first + i] = p
        for i in range(n):
            positions.append(lens[b] + i)
            slots.append(table[b][(lens[b] + i) // page] * page + (lens[b] + i) % page)
        for p in pages:
            ref[p] = 1
        lens[b] += n
        starts.append(starts[-1] + n)
    for p, n in left.items():
        ref[p] -= n
    rest = n_tokens - len(positions)
    return table, lens, ref, starts, positions + [-1] * rest, slots + [-1] * rest, copies, wrong or stopped


def check(w, cache, table, lens, ref, new, n_tokens=None, page=16, stream=None):
    before = snapshot(*cache)
    n_tokens = sum(max(n, 0) for n in new) if n_tokens is None else n_tokens
    want = model(table.tolist(), lens.tolist(), ref.tolist(), new, page, n_tokens)
    got = w.w4a16_kv_grow(cache, table, lens, ref, torch.tensor(new, dtype=torch.int32).cuda(), n_tokens, stream=stream)
    torch.cuda.synchronize()
    assert table.tolist() == want[0]
    assert lens.tolist() == want[1]
    assert ref.tolist() == want[2]
    assert [t.tolist() for t in got] == list(want[3:6])
    assert [t.dtype for t in got] == [torch.int32, torch.int32, torch.int64]
    for src, dst in want[6]:
        for t in before:
            t[dst] = t[src]
    for t, old in zip(snapshot(*cache), before):
        assert torch.equal(t, old)
    assert w.w4a16_last_device_error() == (-9 if want[7] else 0)
    w.w4a16_clear_device_error()
    return want


def shared(table, lens, ref, groups):
    """Rows that name the pages of the first row of their group, its partly filled last page too."""
    for g in groups:
        for b in g[1:]:
            table[b], lens[b] = table[g[0]], lens[g[0]]
    ref.copy_(torch.tensor(counts(table, ref.shape[0]), dtype=torch.int32))


@pytest.mark.parametrize("page, layout, store, dim", [(16, "heads", "int8", 128), (32, "tokens", "e4m3", 64),
                                                       (64, "padded", "int8", 64), (128, "tokens", "int8", 128)])
@pytest.mark.parametrize("new", [1, 16, 300])
def test_growth(cuda_lib, page, layout, store, dim, new):
    """Lengths of nothing, full pages and parts of pages; no page in common."""
    lens = [1, 15, 16, 17, 31, 32, 100, 128, 129, 300, 0, 0]
    cache, table, n, ref = pool(cuda_lib, lens, len(lens), page, layout, store, dim, kv_heads=3, spare=60 + 12 * new // 16)
    table = torch.cat([table, torch.full((len(lens), new // page + 1), -1, dtype=torch.int32, device="cuda")], 1).contiguous()
    check(cuda_lib, cache, table, n, ref, [new - i % 2 for i in range(len(lens))], page=page)
    check(cuda_lib, cache, table, n, ref, [0, 1] * 6, n_tokens=9, page=page)


@pytest.mark.parametrize("grows", [[1, 1, 1, 1], [1, 0, 1, 0], [0, 0, 0, 1], [0, 0, 0, 0], [20, 1, 17, 3]])
@pytest.mark.parametrize("length", [48, 50, 5])
def test_shared_last_pages(cuda_lib, grows, length):
    """All but one of the rows that share a last page get a copy; all that grow when some do not."""
    lens = [length, 0, 0, 0, 77, 0, 9]
    cache, table, n, ref = pool(cuda_lib, lens, 7, spare=40)
    table = torch.cat([table, torch.full((7, 3), -1, dtype=torch.int32, device="cuda")], 1).contiguous()
    shared(table, n, ref, [[0, 1, 2, 3], [4, 5]])
    check(cuda_lib, cache, table, n, ref, grows + [2, 2, 40])
    assert counts(table, ref.shape[0]) == ref.tolist()
    check(cuda_lib, cache, table, n, ref, [1] * 7)
    assert counts(table, ref.shape[0]) == ref.tolist()


@pytest.mark.parametrize("spare", [0, 1, 2, 3, 4, 7])
def test_too_few_pages(cuda_lib, spare):
    """From the first row on that does not get its pages none grows, the ones that need no page included."""
    lens = [16, 20, 0, 5, 32, 7]
    cache, table, n, ref = pool(cuda_lib, lens, 6, spare=spare)
    table = torch.cat([table, torch.full((6, 4), -1, dtype=torch.int32, device="cuda")], 1).contiguous()
    shared(table, n, ref, [[1, 2]])
    check(cuda_lib, cache, table, n, ref, [1, 3, 1, 1, 17, 2])


@pytest.mark.parametrize("rows, spare", [(1024, 100), (1024, 511), (1100, 0), (1100, 550), (1100, 2000)])
def test_many_rows_and_too_few_pages(cuda_lib, rows, spare):
    """Where rows or pages are too many for one launch, and just before."""
    lens = [16 * (1 + b % 3) + (b % 5) for b in range(rows)]
    cache, table, n, ref = pool(cuda_lib, lens, rows, kv_heads=1, dim=64, spare=spare)
    table = torch.cat([table, torch.full((rows, 1), -1, dtype=torch.int32, device="cuda")], 1).contiguous()
    shared(table, n, ref, [[b, b + 1, b + 2] for b in range(0, rows - 3, 7)])
    check(cuda_lib, cache, table, n, ref, [b % 4 for b in range(rows)])


@pytest.mark.parametrize("pages", [32768, 32769])
def test_pool_of_one_launch_and_one_more(cuda_lib, pages):
    w = cuda_lib
    g = torch.Generator().manual_seed(pages)
    codes = [torch.randint(-127, 128, (pages, 1, 16, 64), generator=g, dtype=torch.int8).cuda() for _ in range(2)]
    cache = w.KVCache(*codes, torch.ones((pages, 1), device="cuda"), torch.ones((pages, 1), device="cuda"))
    ref = torch.randint(0, 2, (pages,), generator=g, dtype=torch.int32)
    ref[-1], ref[:64] = 0, 1
    table = torch.full((40, 700), -1, dtype=torch.int32)
    table[:, 0] = torch.arange(40) // 2
    ref[:20] = 2
    lens = torch.full((40,), 5, dtype=torch.int32)
    new = [7000 if b % 2 else 6500 for b in range(40)]                  # more than half of the pages: not enough
    check(w, cache, table.cuda(), lens.cuda(), ref.cuda(), new)


@pytest.mark.parametrize("n_tokens", [0, 1, 5, 11, 12, 40])
def test_too_few_rows(cuda_lib, n_tokens):
    cache, table, n, ref = pool(cuda_lib, [16, 20, 3], 3, spare=9)
    table = torch.cat([table, torch.full((3, 2), -1, dtype=torch.int32, device="cuda")], 1).contiguous()
    check(cuda_lib, cache, table, n, ref, [1, 4, 7], n_tokens=n_tokens)


def test_what_cannot_be(cuda_lib):
    """Rows that ask for it do not grow, others do."""
    lens = [20, 20, 20, 20, 20, 32, 40]
    cache, table, n, ref = pool(cuda_lib, lens, 7, spare=30)           # three columns
    n[1], n[2] = -4, 49
    table[3, 1], table[4, 1] = -1, ref.shape[0]
    check(cuda_lib, cache, table, n, ref, [28, 1, 1, 1, 1, 17, -2], n_tokens=64)
    n[1], n[2] = 48, 0
    check(cuda_lib, cache, table, n, ref, [1, 0, 48, 0, 0, 16, 2**31 - 1], n_tokens=64)


def test_nothing(cuda_lib):
    cache, table, n, ref = pool(cuda_lib, [5], 1)
    check(cuda_lib, cache, table[:0], n[:0], ref, [], n_tokens=3)
    check(cuda_lib, cache, table, n, ref, [0], n_tokens=0)


@pytest.mark.parametrize("rows", [1025, 8192])
def test_many_rows(cuda_lib, rows):
    """Groups of rows that share a last page, of all sizes, over several widths of a CTA."""
    g = torch.Generator().manual_seed(rows)
    pages = 3 * rows
    cache, _, _, _ = pool(cuda_lib, [16 * pages - 640], 1, kv_heads=1, dim=64, spare=40)
    pages = cache.k.shape[0]
    perm = torch.randperm(pages, generator=g, dtype=torch.int32)
    size = torch.randint(1, 9, (rows,), generator=g)
    group = torch.repeat_interleave(torch.arange(rows), size)[:rows]
    lens = torch.randint(0, 31, (rows,), generator=g, dtype=torch.int32)[group]
    table = torch.full((rows, 4), -1, dtype=torch.int32)
    # groups lie far apart in the rows
    order = torch.randperm(rows, generator=g)
    for k in range(2):
        table[:, k] = torch.where(lens > 16 * k, perm[2 * group + k], table[:, k])
    table, lens = table[order].contiguous(), lens[order].contiguous()
    ref = torch.tensor(counts(table, pages), dtype=torch.int32)
    new = torch.randint(0, 3, (rows,), generator=g).tolist()
    check(cuda_lib, cache, table.cuda(), lens.cuda(), ref.cuda(), new)


def test_large_pool(cuda_lib):
    """Free pages far apart, over many chunks of the bitmap."""
    w = cuda_lib
    pages = 150001
    codes = [torch.zeros((pages, 1, 16, 64), dtype=torch.int8, device="cuda") for _ in range(2)]
    cache = w.KVCache(*codes, torch.ones((pages, 1), device="cuda"), torch.ones((pages, 1), device="cuda"))
    ref = torch.ones(pages, dtype=torch.int32, device="cuda")
    ref[[3, 1023, 1024, 5000, 77777, 149999, 150000]] = 0
    table = torch.full((3, 4), -1, dtype=torch.int32, device="cuda")
    table[1, 0] = 7
    lens = torch.tensor([0, 9, 0], dtype=torch.int32, device="cuda")
    ref[7] = 2
    check(w, cache, table, lens, ref, [33, 1, 40])


def test_pool_of_more_than_a_million_pages(cuda_lib):
    """Counts of more chunks than are looked at together, codes past 2^31 bytes."""
    w = cuda_lib
    pages = 2_200_001
    codes = [torch.zeros((pages, 1, 16, 64), dtype=torch.int8, device="cuda") for _ in range(2)]
    cache = w.KVCache(*codes, torch.ones((pages, 1), device="cuda"), torch.ones((pages, 1), device="cuda"))
    ref = torch.ones(pages, dtype=torch.int32, device="cuda")
    free = [70, 1_048_575, 1_048_576, 1_500_000, 2_097_151, 2_097_152, 2_200_000]
    ref[free] = 0
    table = torch.full((3, 4), -1, dtype=torch.int32, device="cuda")
    table[1, 0], table[2, 0] = 2_199_998, 2_199_998
    ref[2_199_998] = 2
    codes[0][2_199_998], codes[1][2_199_998] = 5, -7
    lens = torch.tensor([0, 9, 9], dtype=torch.int32, device="cuda")
    new = torch.tensor([48, 24, 8], dtype=torch.int32, device="cuda")
    starts, positions, slots = w.w4a16_kv_grow(cache, table, lens, ref, new, 80)
    torch.cuda.synchronize()
    # three blocks; a copy and two blocks; the last row that names it keeps its page, and begins a block
    assert table.tolist() == [free[:3] + [-1], free[3:6] + [-1], [2_199_998, free[6], -1, -1]]
    assert lens.tolist() == [48, 33, 17] and starts.tolist() == [0, 48, 72, 80]
    assert bool((ref == 1).all()) and w.w4a16_last_device_error() == 0
    want = [16 * p + i for p in free[:3] for i in range(16)]
    want += [16 * free[3] + i for i in range(9, 16)] + [16 * free[4] + i for i in range(16)] + [16 * free[5]]
    want += [16 * 2_199_998 + i for i in range(9, 16)] + [16 * free[6]]
    assert slots.tolist() == want
    for c, v in zip(codes, (5, -7)):
        assert bool((c[free[3]] == v).all()) and int((c != 0).any(-1).any(-1).sum()) == 2


def test_other_stream_outputs_and_workspace(cuda_lib):
    w = cuda_lib
    cache, table, n, ref = pool(w, [20, 31, 0], 3, spare=20)
    table = torch.cat([table, torch.full((3, 2), -1, dtype=torch.int32, device="cuda")], 1).contiguous()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    check(w, cache, table, n, ref, [3, 2, 20], stream=s)
    new = torch.tensor([1, 1, 1], dtype=torch.int32, device="cuda")
    out = (torch.empty(4, dtype=torch.int32, device="cuda"), torch.empty(3, dtype=torch.int32, device="cuda"),
           torch.empty(3, dtype=torch.int64, device="cuda"))
    ws = torch.empty(w.w4a16_kv_grow_workspace(ref.shape[0], 3), dtype=torch.uint8, device="cuda")
    got = w.w4a16_kv_grow(cache, table, n, ref, new, 3, *out, workspace=ws)
    assert all(a is b for a, b in zip(got, out))
    assert out[1].tolist() == [23, 33, 20]


def test_captured(cuda_lib):
    """One captured call, replayed with other requests and less than it was captured for."""
    w = cuda_lib
    cache, table, n, ref = pool(w, [20, 0, 31, 16], 4, spare=60)
    table = torch.cat([table, torch.full((4, 3), -1, dtype=torch.int32, device="cuda")], 1).contiguous()
    shared(table, n, ref, [[0, 1]])
    new = torch.zeros(4, dtype=torch.int32, device="cuda")
    w.w4a16_kv_grow(cache, table, n, ref, new, 12)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = w.w4a16_kv_grow(cache, table, n, ref, new, 12)
    for ask in ([1, 1, 1, 1], [0, 3, 1, 8], [2, 0, 0, 0], [5, 5, 5, 0]):
        want = model(table.tolist(), n.tolist(), ref.tolist(), ask, 16, 12)
        new.copy_(torch.tensor(ask, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        assert (table.tolist(), n.tolist(), ref.tolist()) == want[:3]
        assert [t.tolist() for t in got] == list(want[3:6])
    assert w.w4a16_last_device_error() == -9                # 15 tokens for 12 rows
    w.w4a16_clear_device_error()
