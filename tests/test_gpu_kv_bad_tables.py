"""Tables and starts that are wrong on the device: exactly what they name wrongly is left out."""
import pytest
import torch

from kv_reference import ACT, Problem, attention, attention_tolerance

pytestmark = pytest.mark.gpu


def reported(w):
    torch.cuda.synchronize()
    got = w.w4a16_last_device_error()
    w.w4a16_clear_device_error()
    return got == -9


def without(p, blocks):
    """(out, spread) in 64 bits of p's only sequence, the keys of `blocks` left out."""
    n, m = p.lens[0], p.new[0]
    k, v = p.values(p.k, p.ks, 0, n), p.values(p.v, p.vs, 0, n)
    pos, j = torch.arange(n - m, n)[:, None], torch.arange(n)[None]
    see = (j <= pos) & ~torch.isin(j // p.page, torch.tensor(blocks))
    g = p.heads // p.kv_heads
    out, spread = (torch.zeros(m, p.heads, p.dim, dtype=torch.float64) for _ in range(2))
    for a in range(p.heads):
        s = (p.q[:, a].double() @ k[:, a // g].T * p.dim ** -0.5).masked_fill(~see, -float("inf"))
        x = torch.where(see.any(1, keepdim=True), torch.softmax(s, -1), torch.zeros_like(s))
        out[:, a], spread[:, a] = x @ v[:, a // g], x @ v[:, a // g].abs()
    return out, spread


@pytest.mark.parametrize("new", [1, 5, 70, 300])
@pytest.mark.parametrize("store, dim, page", [("int8", 128, 16), ("e4m3", 64, 32)])
@pytest.mark.parametrize("wrong", [-1, -7, "n_pages", 1 << 30])
def test_attention_leaves_the_page_out(cuda_lib, new, store, dim, page, wrong):
    w = cuda_lib
    p = Problem([200 + new], [new], store=store, dim=dim, page=page, seed=new)
    cache, table, lens, starts, rows = p.to_cuda(w)
    blocks = [0, 2, (199 + new) // page]
    for b in blocks:
        table[0, b] = p.n_pages if wrong == "n_pages" else wrong
    q = rows[:, :p.heads * dim].unflatten(1, (p.heads, dim))
    out = w.w4a16_kv_attention(q, cache, table, lens, starts, new)
    assert reported(w)
    want, spread = without(p, blocks)
    assert bool(((out.cpu().double() - want).abs() <= attention_tolerance(p, want, spread)).all())


@pytest.mark.parametrize("new", [1, 40])
def test_all_pages_wrong_is_an_empty_row(cuda_lib, new):
    w = cuda_lib
    p = Problem([90 + new, 33 + new], [new, new], seed=2)
    cache, table, lens, starts, rows = p.to_cuda(w)
    table[0] = -1
    q = rows[:, :p.heads * p.dim].unflatten(1, (p.heads, p.dim))
    lse = torch.zeros((p.T, p.heads), device="cuda")
    out = w.w4a16_kv_attention(q, cache, table, lens, starts, new, lse=lse)
    assert reported(w)
    want, _, spread = attention(p)
    assert bool((out[:new] == 0).all()) and bool((lse[:new] == -float("inf")).all())
    assert bool(((out[new:].cpu().double() - want[new:]).abs() <= attention_tolerance(p, want, spread)[new:]).all())


@pytest.mark.parametrize("new", [3, 200])
@pytest.mark.parametrize("window", [0, 5, 2 ** 31 - 1])
def test_more_new_tokens_than_the_sequence_is_long(cuda_lib, new, window):
    """Tokens at negative positions are empty rows; those at positions from 0 on get their answer."""
    w = cuda_lib
    p = Problem([new], [new], seed=new)
    cache, table, lens, starts, rows = p.to_cuda(w)
    gone = new // 2
    lens -= gone
    q = rows[:, :p.heads * p.dim].unflatten(1, (p.heads, p.dim))
    out = w.w4a16_kv_attention(q, cache, table, lens, starts, new, window=window)
    assert reported(w)
    p.lens = [new - gone]
    p.new, p.rows, p.T = [new - gone], p.rows[gone:], new - gone
    want, _, spread = attention(p, None, window)
    assert bool((out[:gone] == 0).all())
    assert bool(((out[gone:].cpu().double() - want).abs() <= attention_tolerance(p, want, spread)).all())


def test_read_gives_zeros_for_the_rows_of_a_wrong_page(cuda_lib):
    w = cuda_lib
    p = Problem([40, 20], [20, 10], act="f16", seed=1)
    cache, table, lens, starts, _ = p.to_cuda(w)
    table[0, 1], table[1, 1] = p.n_pages, -3              # positions 16..31 of both
    k, v = w.w4a16_kv_read(cache, table, lens, starts, p.T, torch.float16)
    assert reported(w)
    for got, codes, scales in ((k, p.k, p.ks), (v, p.v, p.vs)):
        want = torch.cat([p.values(codes, scales, b, n)[n - m:] for b, (n, m) in enumerate(zip(p.lens, p.new))]).float()
        want = want.to(ACT[p.act])
        want[:12] = 0                                     # positions 20..31 of the first sequence
        want[20 + 6:] = 0                                 # positions 16..19 of the second, of 10..19
        assert torch.equal(got.cpu(), want)


def test_append_leaves_out_the_tokens_of_a_wrong_page(cuda_lib):
    w = cuda_lib
    p = Problem([40, 20], [20, 10], act="f16", seed=2)
    cache, table, lens, starts, rows = p.to_cuda(w)
    a, b = p.heads * p.dim, (p.heads + p.kv_heads) * p.dim
    new = rows[:, a:b].unflatten(1, (p.kv_heads, p.dim)), rows[:, b:].unflatten(1, (p.kv_heads, p.dim))
    before = [t.view(torch.uint8).clone() for t in cache]
    good = [t.clone() for t in cache]
    w.w4a16_kv_append(w.KVCache(*good), *new, table, lens, starts)
    wrong = table.clone()
    wrong[0, 1] = 1 << 29
    w.w4a16_kv_append(cache, *new, wrong, lens, starts)
    assert reported(w)
    page = int(table[0, 1])
    for got, old, want in zip(cache, before, good):
        got, want = got.view(torch.uint8), want.view(torch.uint8)
        assert torch.equal(got[page], old[page])
        rest = torch.arange(p.n_pages, device="cuda") != page
        assert torch.equal(got[rest], want[rest])


def test_fork_of_a_last_page_that_is_not_there(cuda_lib):
    """The child of a parent whose partly filled last page is unknown gets no page for it, and its keys are left out there too."""
    w = cuda_lib
    p = Problem([40, 35, 20], [0, 0, 0], seed=3, spare=6)
    cache, table, lens, _, _ = p.to_cuda(w)
    table = torch.cat([table, torch.full((3, table.shape[1]), 5, dtype=torch.int32, device="cuda")])
    lens = torch.cat([lens, torch.zeros(3, dtype=torch.int32, device="cuda")])
    ref = torch.zeros(p.n_pages, dtype=torch.int32, device="cuda")
    ref[table[:3][table[:3] >= 0].long()] = 1
    last = int(table[1, 2])
    table[1, 2] = -1
    ref[last] = 0
    free = torch.nonzero(ref == 0)[:, 0].tolist()
    t = table.cpu()
    w.w4a16_kv_fork(cache, table, lens, ref, torch.tensor([0, 1, 2], dtype=torch.int32).cuda(),
                    torch.tensor([3, 4, 5], dtype=torch.int32).cuda())
    assert reported(w)
    assert lens.tolist() == [40, 35, 20, 40, 35, 20]
    assert table[3].tolist() == t[0, :2].tolist() + [free[0]]
    assert table[4].tolist() == t[1, :2].tolist() + [-1]
    assert table[5].tolist() == t[2, :1].tolist() + [free[1], -1]
    named = [0] * p.n_pages
    for q in table.flatten().tolist():
        if q >= 0:
            named[q] += 1
    assert ref.tolist() == named


def test_lengths_past_the_table(cuda_lib):
    """Fork and trim take what the table holds, and report."""
    w = cuda_lib
    p = Problem([48, 40], [0, 0], seed=5)
    cache, table, lens, _, _ = p.to_cuda(w)
    ref = torch.zeros(p.n_pages, dtype=torch.int32, device="cuda")
    ref[table[table >= 0].long()] = 1
    lens[0] = 1000                                        # the table has three blocks
    t = table.clone()
    w.w4a16_kv_trim(table, lens, ref, 16, 17, 0)
    assert reported(w)
    assert table[0].tolist() == [-1, -1, int(t[0, 2])] and table[1].tolist() == [-1] + t[1, 1:].tolist()
    rows = torch.cat([t, torch.full_like(t[:1], -1)])
    lens = torch.tensor([1000, 40, 0], dtype=torch.int32, device="cuda")
    w.w4a16_kv_fork(cache, rows, lens, ref, torch.tensor([0], dtype=torch.int32).cuda(), torch.tensor([2], dtype=torch.int32).cuda())
    assert reported(w)
    assert rows[2].tolist() == t[0].tolist() and lens.tolist() == [1000, 40, 48]
