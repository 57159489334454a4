"""Page operators of the cache: tables, counts and page contents, exactly."""
import pytest
import torch

from kv_reference import Problem

pytestmark = pytest.mark.gpu


def pool(w, lens, rows, page=16, layout="heads", store="int8", dim=128, kv_heads=2, spare=40, seed=0):
    """(cache, table with `rows` rows, lens, refcount)"""
    p = Problem(lens, [0] * len(lens), 4, kv_heads, dim, page, store, layout, seed=seed, spare=spare)
    cache, table, n, _, _ = p.to_cuda(w)
    g = torch.Generator(device="cuda").manual_seed(seed)
    for t in cache[:2]:
        raw = t.view(torch.int8)
        raw.copy_(torch.randint(-128, 128, raw.shape, generator=g, device="cuda", dtype=torch.int8))
    for t in cache[2:]:
        t.uniform_(0.5, 2.0, generator=g)
    extra = rows - len(lens)
    table = torch.cat([table, torch.full((extra, table.shape[1]), -1, dtype=torch.int32, device="cuda")])
    n = torch.cat([n, torch.zeros(extra, dtype=torch.int32, device="cuda")])
    ref = torch.zeros(p.n_pages, dtype=torch.int32, device="cuda")
    ref[table[table >= 0].long()] = 1
    return cache, table, n, ref


def snapshot(*ts):
    return [t.view(torch.int8).cpu().clone() if t.element_size() == 1 else t.cpu().clone() for t in ts]


def counts(table, n_pages):
    ref = [0] * n_pages
    for p in table.flatten().tolist():
        if p >= 0:
            ref[p] += 1
    return ref


@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("layout", ["heads", "tokens", "padded"])
@pytest.mark.parametrize("store, dim", [("int8", 128), ("e4m3", 64)])
def test_copy(cuda_lib, page, layout, store, dim):
    w = cuda_lib
    cache, *_ = pool(w, [300], 1, page, layout, store, dim, kv_heads=3)
    before = snapshot(*cache)
    n = cache.k.shape[0]
    perm = torch.randperm(n, generator=torch.Generator().manual_seed(1))
    src, dst = perm[:17].clone(), perm[17:34].clone()
    src[3], dst[5] = -1, -1
    w.w4a16_kv_copy_pages(cache, src.int().cuda(), dst.int().cuda())
    torch.cuda.synchronize()
    for got, old in zip(snapshot(*cache), before):
        for s, d in zip(src.tolist(), dst.tolist()):
            if s >= 0 and d >= 0:
                old[d] = old[s]
        assert torch.equal(got, old)
    assert w.w4a16_last_device_error() == 0
    src[0] = n
    w.w4a16_kv_copy_pages(cache, src[:1].int().cuda(), dst[:1].int().cuda())
    torch.cuda.synchronize()
    assert w.w4a16_last_device_error() == -9
    w.w4a16_clear_device_error()


@pytest.mark.parametrize("page, layout", [(16, "heads"), (64, "tokens"), (32, "padded")])
@pytest.mark.parametrize("copies", [1, 3, 8])
def test_fork(cuda_lib, page, layout, copies):
    w = cuda_lib
    lens = [1, page, page + 1, 5 * page - 1, 0, 200]
    cache, table, n, ref = pool(w, lens, len(lens) * (copies + 1), page, layout, spare=60)
    par = [b for b in range(len(lens)) for _ in range(copies)]
    chi = list(range(len(lens), len(lens) * (copies + 1)))
    table[chi[0]] = 7                                 # a child's old row is overwritten, not freed
    before = snapshot(*cache)
    t, ln, free = table.cpu(), n.cpu(), [p for p, c in enumerate(ref.tolist()) if c == 0]
    want_ref = ref.tolist()
    for a, b in zip(par, chi):
        full, tail = lens[a] // page, lens[a] % page
        t[b] = -1
        t[b, :full] = t[a, :full]
        for q in t[a, :full].tolist():
            want_ref[q] += 1
        ln[b] = lens[a]
        if tail:
            f = free.pop(0)
            t[b, full] = f
            want_ref[f] = 1
            for x in before:
                x[f] = x[int(t[a, full])]
    w.w4a16_kv_fork(cache, table, n, ref, torch.tensor(par, dtype=torch.int32).cuda(), torch.tensor(chi, dtype=torch.int32).cuda())
    torch.cuda.synchronize()
    assert torch.equal(table.cpu(), t) and torch.equal(n.cpu(), ln) and ref.tolist() == want_ref
    for got, want in zip(snapshot(*cache), before):
        assert torch.equal(got, want)
    assert w.w4a16_last_device_error() == 0


def test_fork_without_enough_pages(cuda_lib):
    w = cuda_lib
    cache, table, n, ref = pool(w, [20, 16], 6, spare=2)
    free = [p for p, c in enumerate(ref.tolist()) if c == 0]
    par, chi = torch.tensor([0, 0, 1, 0], dtype=torch.int32).cuda(), torch.tensor([2, 3, 4, 5], dtype=torch.int32).cuda()
    w.w4a16_kv_fork(cache, table, n, ref, par, chi)
    torch.cuda.synchronize()
    assert n.tolist() == [20, 16, 20, 20, 16, 0]
    assert [int(table[2, 1]), int(table[3, 1])] == free
    assert bool((table[5] == -1).all())
    assert ref.tolist() == counts(table, len(ref))
    assert w.w4a16_last_device_error() == -9
    w.w4a16_clear_device_error()


def test_fork_from_a_large_pool(cuda_lib):
    """Free pages far apart: over many chunks of the bitmap, in ascending order."""
    w = cuda_lib
    cache, table, n, ref = pool(w, [5] * 40, 80, dim=64, kv_heads=1, spare=700000, seed=3)
    ref.fill_(1)
    free = torch.randperm(ref.shape[0], generator=torch.Generator().manual_seed(0))[:40].sort().values
    ref[free.cuda()] = 0
    ids = torch.arange(80, dtype=torch.int32, device="cuda")
    w.w4a16_kv_fork(cache, table, n, ref, ids[:40], ids[40:])
    torch.cuda.synchronize()
    assert torch.equal(table[40:, 0].cpu(), free.int())
    assert w.w4a16_last_device_error() == 0


def test_free(cuda_lib):
    w = cuda_lib
    cache, table, n, ref = pool(w, [100, 0, 33, 400], 8)
    ids = torch.tensor([0, 3], dtype=torch.int32).cuda()
    w.w4a16_kv_fork(cache, table, n, ref, ids, torch.tensor([4, 5], dtype=torch.int32).cuda())
    w.w4a16_kv_free(table, n, ref, torch.tensor([3, 1, 4, 3], dtype=torch.int32).cuda())     # 3 twice: once
    torch.cuda.synchronize()
    assert n.tolist() == [100, 0, 33, 0, 0, 400, 0, 0]
    assert bool((table[3] == -1).all()) and bool((table[4] == -1).all())
    assert ref.tolist() == counts(table, len(ref))
    assert w.w4a16_last_device_error() == 0
    w.w4a16_kv_free(table, n, ref, torch.tensor([99], dtype=torch.int32).cuda())
    torch.cuda.synchronize()
    assert w.w4a16_last_device_error() == -9
    w.w4a16_clear_device_error()
    ref[table[0, 0].long()] = 0                       # a count that is already 0 stays, and is reported
    w.w4a16_kv_free(table, n, ref, ids[:1])
    torch.cuda.synchronize()
    assert w.w4a16_last_device_error() == -9 and int(ref.min()) == 0
    w.w4a16_clear_device_error()


@pytest.mark.parametrize("window, sinks", [(1, 0), (16, 0), (17, 1), (100, 16), (100, 17), (1, 1000), (5000, 4), (0, 4)])
def test_trim(cuda_lib, window, sinks):
    w = cuda_lib
    lens = [0, 1, 16, 17, 200, 333]
    _, table, n, ref = pool(w, lens, 6)
    t = table.cpu().clone()
    for b, ln in enumerate(lens):
        for blk in range(t.shape[1]):
            # a later token, at position ln or more, sees none of the block's positions
            if window and all(j >= sinks and ln - j >= window for j in range(blk * 16, blk * 16 + 16)):
                t[b, blk] = -1
    w.w4a16_kv_trim(table, n, ref, 16, window, sinks)
    torch.cuda.synchronize()
    assert torch.equal(table.cpu(), t) and n.tolist() == lens
    assert ref.tolist() == counts(table, len(ref))
    assert w.w4a16_last_device_error() == 0


@pytest.mark.parametrize("page, layout", [(16, "heads"), (128, "tokens"), (32, "padded")])
@pytest.mark.parametrize("gone", [[], [0], [1, 2, 5], [0, 1, 2, 3, 4, 5], [3]])
def test_compact(cuda_lib, page, layout, gone):
    w = cuda_lib
    cache, table, n, ref = pool(w, [1, 700, 33, 90, 0, 512], 7, page, layout, seed=len(gone))
    w.w4a16_kv_fork(cache, table, n, ref, torch.tensor([3], dtype=torch.int32).cuda(), torch.tensor([6], dtype=torch.int32).cuda())
    w.w4a16_kv_free(table, n, ref, torch.tensor(gone, dtype=torch.int32).cuda())
    torch.cuda.synchronize()
    before, t0, r0 = snapshot(*cache), table.cpu().clone(), ref.tolist()
    live = [p for p, c in enumerate(r0) if c]
    m = len(live)
    to = dict(zip([p for p in live if p >= m], [p for p in range(m) if not r0[p]]))
    n_live = torch.zeros(1, dtype=torch.int32, device="cuda")
    w.w4a16_kv_compact(cache, table, ref, n_live=n_live)
    torch.cuda.synchronize()
    assert int(n_live) == m
    assert table.cpu().tolist() == [[to.get(p, p) for p in row] for row in t0.tolist()]
    assert ref.tolist() == [r0[{v: k for k, v in to.items()}.get(p, p)] if p < m else 0 for p in range(len(r0))]
    for got, old in zip(snapshot(*cache), before):
        for s, d in to.items():
            old[d] = old[s]
        assert torch.equal(got, old)
    assert w.w4a16_last_device_error() == 0


def test_compact_a_large_pool(cuda_lib):
    """Many chunks of the bitmap, some empty, some full; stale scratch."""
    w = cuda_lib
    cache, table, n, ref = pool(w, [3000 * 16], 1, dim=64, kv_heads=1, spare=60000, seed=5)
    before = cache.k.clone()
    old = table.clone()
    ws = torch.full((w.w4a16_kv_pool_workspace(ref.shape[0]),), 255, dtype=torch.uint8, device="cuda")
    w.w4a16_kv_compact(cache, table, ref, workspace=ws)
    torch.cuda.synchronize()
    assert int(ref[:3000].sum()) == 3000 and int(ref.sum()) == 3000
    assert torch.equal(cache.k[table[0].long()], before[old[0].long()])
    assert sorted(table[0].tolist()) == list(range(3000))
    w.w4a16_kv_compact(cache, table, ref, workspace=ws)          # nothing left to move
    torch.cuda.synchronize()
    assert sorted(table[0].tolist()) == list(range(3000))
