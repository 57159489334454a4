"""Attention over the paged 8-bit cache against its definition in 64 bits, at
the lengths, masks and layouts where it can go wrong."""
import pytest
import torch

from kv_reference import Problem, attention, attention_tolerance

pytestmark = pytest.mark.gpu


def run(w, p, window=0, sinks=0, scale=None, max_new=None, lse=True, stream=None):
    cache, table, lens, starts, rows = p.to_cuda(w)
    q = rows[:, :p.heads * p.dim].unflatten(1, (p.heads, p.dim))
    out_lse = torch.full((p.T, p.heads), 7.0, device="cuda") if lse else None
    out = w.w4a16_kv_attention(q, cache, table, lens, starts, max(p.new) if max_new is None else max_new, scale=scale,
                               window=window, sinks=sinks, lse=out_lse)
    torch.cuda.synchronize()
    return out, out_lse


def check(w, p, window=0, sinks=0, scale=None, max_new=None):
    out, lse = run(w, p, window, sinks, scale, max_new)
    want, want_lse, spread = attention(p, scale, window, sinks)
    err = (out.cpu().double() - want).abs()
    tol = attention_tolerance(p, want, spread)
    assert bool((err <= tol).all()), f"max excess {(err - tol).max().item():.3e}, max error {err.max().item():.3e}"
    empty = want_lse == -float("inf")
    assert torch.equal(lse.cpu() == -float("inf"), empty)
    # fp32 sums of weights that are each good to 2^-12, at scores of some tens
    assert bool(((lse.cpu().double() - want_lse)[~empty].abs() <= 2.0 ** -11 + 2.0 ** -18 * want_lse[~empty].abs()).all())
    assert w.w4a16_last_device_error() == 0
    return out


@pytest.mark.parametrize("store", ["int8", "e4m3"])
@pytest.mark.parametrize("act", ["f16", "bf16"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("heads, kv_heads", [(4, 4), (8, 2), (14, 2), (8, 1), (40, 2)])
def test_single_tokens(cuda_lib, store, act, dim, heads, kv_heads):
    lens = [1, 2, 15, 16, 17, 31, 100, 257, 1000]
    check(cuda_lib, Problem(lens, [1] * len(lens), heads, kv_heads, dim, 16, store, "heads", act, seed=heads + dim))


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("layout", ["heads", "tokens", "padded", "pairs"])
def test_pages_and_layouts(cuda_lib, page, layout):
    check(cuda_lib, Problem([5, 130, 300, 129], [1, 2, 1, 5], page=page, layout=layout, store="int8", seed=page))
    check(cuda_lib, Problem([50, 130, 300], [50, 2, 130], page=page, layout=layout, store="e4m3", seed=page))
    check(cuda_lib, Problem([5, 130, 300, 129], [1, 2, 1, 5], page=page, layout=layout, store="e4m3", dim=64, act="f16",
                            seed=page + 1))


@pytest.mark.parametrize("window, sinks", [(1, 0), (1, 4), (16, 0), (17, 3), (64, 16), (100, 17), (33, 500), (5000, 4)])
@pytest.mark.parametrize("new", [1, 5, 40])
def test_window_and_sinks(cuda_lib, window, sinks, new):
    lens = [new, new + 3, 64 + new, 301 + new, 700 + new]
    check(cuda_lib, Problem(lens, [new] * len(lens), seed=window + sinks + new), window, sinks)


@pytest.mark.parametrize("lens", [[30000], [20011, 9999], [17000, 0, 17777, 16000], [40000, 12]])
@pytest.mark.parametrize("heads, kv_heads, new", [(8, 2, 1), (4, 1, 1), (8, 8, 1), (16, 2, 2)])
def test_few_long_sequences_token_first(cuda_lib, lens, heads, kv_heads, new):
    """Tiles of one sequence cut into the same number of pieces, or not where that would be uneven."""
    news = [min(new, n) for n in lens]
    check(cuda_lib, Problem(lens, news, heads, kv_heads, 128, 64, "e4m3", "tokens", "f16", seed=len(lens)))
    check(cuda_lib, Problem(lens, news, heads, kv_heads, 64, 16, "int8", "tokens", "bf16", seed=kv_heads))


@pytest.mark.parametrize("page", [16, 32])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("new", [[4, 4], [5, 5], [8, 8], [9, 9], [1, 4, 5, 8, 9, 0, 40]])
def test_rows_around_the_kernels_limits(cuda_lib, new, dim, page):
    """16, 20, 32 and 36 rows a kv head: one tile or two of the few-rows kernel, or the other kernel's."""
    lens = [n + past for n, past in zip(new, [300, 0, 77, 1000, 15, 60, 129])]
    check(cuda_lib, Problem(lens, new, 8, 2, dim, page, "int8", "heads", "bf16", seed=sum(new) + dim))
    check(cuda_lib, Problem(lens, new, 8, 2, dim, page, "e4m3", "tokens", "f16", seed=sum(new) + page), 50, 3)


@pytest.mark.parametrize("new", [[2], [3, 0, 1], [16, 17], [0, 33, 0], [64, 1, 65], [1, 200, 7]])
@pytest.mark.parametrize("heads, kv_heads, dim", [(8, 2, 128), (2, 2, 64), (14, 2, 128), (16, 1, 64)])
def test_several_tokens(cuda_lib, new, heads, kv_heads, dim):
    lens = [n + past for n, past in zip(new, (90, 0, 1000))]
    check(cuda_lib, Problem(lens, new, heads, kv_heads, dim, act="f16", store="e4m3", seed=sum(new)))


@pytest.mark.parametrize("heads, kv_heads, dim, store, act, window, sinks", [
    (8, 2, 128, "int8", "bf16", 0, 0), (8, 2, 128, "e4m3", "f16", 0, 0), (4, 4, 64, "int8", "f16", 0, 0),
    (7, 1, 128, "int8", "bf16", 0, 0), (8, 1, 64, "e4m3", "bf16", 0, 0),
    (8, 2, 128, "int8", "bf16", 200, 4), (4, 4, 64, "e4m3", "f16", 129, 0), (14, 2, 128, "int8", "bf16", 1, 1)])
def test_prompts(cuda_lib, heads, kv_heads, dim, store, act, window, sinks):
    new = [300, 1, 513, 0, 128]
    lens = [300, 70, 1200, 33, 129]
    check(cuda_lib, Problem(lens, new, heads, kv_heads, dim, 32, store, "tokens", act, seed=dim), window, sinks)


def test_lengths_of_zero(cuda_lib):
    # no cached token at all, no new token, and tokens whose cache is shorter than they are many
    w = cuda_lib
    p = Problem([0, 40, 0], [0, 2, 0])
    check(w, p)
    cache, table, lens, starts, rows = p.to_cuda(w)
    lens.zero_()
    out = w.w4a16_kv_attention(rows[:, :p.heads * p.dim].unflatten(1, (p.heads, p.dim)), cache, table, lens, starts, 2)
    torch.cuda.synchronize()
    assert bool((out == 0).all())
    assert w.w4a16_last_device_error() == -9           # more new tokens than the sequence is long
    w.w4a16_clear_device_error()


def test_no_sequences(cuda_lib):
    w = cuda_lib
    p = Problem([4], [1])
    cache, table, lens, starts, rows = p.to_cuda(w)
    q = rows[:0, :p.heads * p.dim].unflatten(1, (p.heads, p.dim))
    assert w.w4a16_kv_attention(q, cache, table[:0], lens[:0], starts[:1], 0).shape == (0, p.heads, p.dim)
    torch.cuda.synchronize()


@pytest.mark.parametrize("new", [1, 3, 150])
def test_pages_out_of_the_window_are_not_read(cuda_lib, new):
    p = Problem([900 + new, 77 + new], [new, new], seed=new)
    window, sinks = 100, 20
    want = check(cuda_lib, p, window, sinks)
    for b, n in enumerate(p.lens):
        first = n - new
        for blk in range(p.table.shape[1]):
            if blk * 16 >= sinks and blk * 16 + 16 <= first + 1 - window:
                p.table[b, blk] = -1
    assert bool((p.table[0] == -1).sum() > 40)
    assert torch.equal(want, run(cuda_lib, p, window, sinks)[0])
    assert cuda_lib.w4a16_last_device_error() == 0


@pytest.mark.parametrize("new", [1, 6, 130])
def test_what_is_not_visible_does_not_matter(cuda_lib, new):
    """Scales of unseen pages and codes of unseen slots may be anything, NaN included (Problem plants them)."""
    p = Problem([37 + new, 200 + new], [new, new], store="e4m3", wide=3, seed=new)
    a = check(cuda_lib, p)
    cache, table, lens, starts, rows = p.to_cuda(cuda_lib)
    table[table < 0] = 1 << 30
    q = rows[:, :p.heads * p.dim].unflatten(1, (p.heads, p.dim))
    assert torch.equal(a, cuda_lib.w4a16_kv_attention(q, cache, table, lens, starts, new))
    torch.cuda.synchronize()
    assert cuda_lib.w4a16_last_device_error() == 0


@pytest.mark.parametrize("new", [1, 70])
def test_bad_page_is_left_out_and_reported(cuda_lib, new):
    w = cuda_lib
    p = Problem([100 + new], [new])
    cache, table, lens, starts, rows = p.to_cuda(w)
    table[0, 2] = p.n_pages
    q = rows[:, :p.heads * p.dim].unflatten(1, (p.heads, p.dim))
    out = w.w4a16_kv_attention(q, cache, table, lens, starts, new)
    torch.cuda.synchronize()
    assert w.w4a16_last_device_error() == -9
    w.w4a16_clear_device_error()
    # as if the page's sixteen keys were not there: the same answer with their weight driven to nothing
    assert bool(torch.isfinite(out.float()).all())


@pytest.mark.parametrize("new", [1, 4, 140])
def test_large_scores(cuda_lib, new):
    """Scores of hundreds: the softmax is all but one-hot, and exponents far apart do not overflow."""
    p = Problem([500 + new, new], [new, new], act="f16", seed=9)
    p.rows[:, :p.heads * p.dim] *= 30
    check(cuda_lib, p)


@pytest.mark.parametrize("new", [1, 130])
@pytest.mark.parametrize("act", ["f16", "bf16"])
def test_rows_of_any_magnitude(cuda_lib, new, act):
    """Queries past fp16's range as bf16, tiny ones, and zero rows; values whose scales differ by 2^40 between blocks."""
    p = Problem([300 + new], [new], act=act, seed=4)
    p.rows[:, :p.dim] = 0
    p.rows[:, p.dim:2 * p.dim] *= 2.0 ** -20 if act == "bf16" else 2.0 ** -10
    if act == "bf16":
        p.rows[:, 2 * p.dim:3 * p.dim] *= 1e6
        p.ks *= 1e-5
    p.vs[p.table[0, ::3].long()] *= 2.0 ** -40
    check(cuda_lib, p)


def test_first_token_holds_the_weight(cuda_lib):
    """One key takes nearly all of the softmax and its value is zero: the rest, thousands of small weights, is the output."""
    p = Problem([6001], [1], heads=4, kv_heads=1, act="f16", seed=2)
    page = int(p.table[0, 0])
    raw = p.k.view(torch.int8)
    q = p.q[0, 0].float()
    raw[page, 0, 0] = (q.sign() * 127).to(torch.int8)
    p.v.view(torch.int8)[page, 0, 0] = 0
    check(cuda_lib, p)


@pytest.mark.parametrize("new", [1, 130])
def test_not_finite_values_show(cuda_lib, new):
    w = cuda_lib
    p = Problem([64 + new, 64 + new], [new, new])
    p.vs[p.table[0, 1].long(), 0] = float("nan")
    p.ks[p.table[0, 0].long(), 1] = float("inf")
    out, _ = run(w, p)
    assert bool(torch.isnan(out[:new].float()).all())
    assert bool(torch.isfinite(out[new:].float()).all())


def test_any_max_q_len_gives_the_answer(cuda_lib):
    p = Problem([200, 40, 333], [150, 1, 6], seed=3)
    for said in (0, 1, 6, 150, 4000):
        check(cuda_lib, p, max_new=said)


def test_other_stream_and_graph_replay_with_other_lengths(cuda_lib):
    w = cuda_lib
    p = Problem([513, 90, 256, 17], [1, 1, 1, 1], seed=5)
    cache, table, lens, starts, rows = p.to_cuda(w)
    q = rows[:, :p.heads * p.dim].unflatten(1, (p.heads, p.dim))
    out = torch.empty(q.shape, dtype=q.dtype, device="cuda")
    need = w.w4a16_kv_attention_workspace(p.heads, p.kv_heads, p.dim, 4, 4)
    ws = torch.full((max(16, need),), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        w.w4a16_kv_attention(q, cache, table, lens, starts, 1, out=out, workspace=ws)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        w.w4a16_kv_attention(q, cache, table, lens, starts, 1, out=out, workspace=ws)
    for lengths in ([513, 90, 256, 17], [1, 33, 2, 16], [400, 1, 1, 5]):
        lens.copy_(torch.tensor(lengths, dtype=torch.int32))
        ws.fill_(255)
        out.fill_(-1)
        graph.replay()
        torch.cuda.synchronize()
        p.lens = lengths
        want, _, spread = attention(p)
        assert bool(((out.cpu().double() - want).abs() <= attention_tolerance(p, want, spread)).all())


@pytest.mark.parametrize("new", [1, 5, 300])
def test_repeatable(cuda_lib, new):
    """The order of CTAs does not show: the same call gives the same bits."""
    p = Problem([3000 + new] * 3, [new] * 3, seed=6)
    first = run(cuda_lib, p)[0]
    for _ in range(5):
        assert torch.equal(first, run(cuda_lib, p)[0])


@pytest.mark.parametrize("new", [1, 140])
def test_offsets_past_32_bits(cuda_lib, new):
    """The same pages at the far end of a pool of over 8 GB."""
    w = cuda_lib
    p = Problem([400 + new], [new], heads=8, kv_heads=8, page=16, seed=8)
    want = check(w, p)
    cache, table, lens, starts, rows = p.to_cuda(w)
    n = (1 << 33) // (8 * 16 * 128) // 2 + p.n_pages      # K and V: 4 GB and a bit each
    big = [torch.empty((n, 8, 16, 128), dtype=torch.int8, device="cuda") for _ in range(2)]
    scales = [torch.empty((n, 8), device="cuda") for _ in range(2)]
    for dst, src in zip(big + scales, cache):
        dst[n - p.n_pages:] = src
    far = w.KVCache(*big, *scales)
    table[table >= 0] += n - p.n_pages
    q = rows[:, :p.heads * p.dim].unflatten(1, (p.heads, p.dim))
    assert torch.equal(want, w.w4a16_kv_attention(q, far, table, lens, starts, new))
    # an append there, too, and a copy back to the start of the pool
    k_new = rows[:, p.heads * p.dim:2 * p.heads * p.dim].unflatten(1, (8, 128))
    w.w4a16_kv_append(far, k_new, k_new, table, lens, starts)
    w.w4a16_kv_append(cache, k_new, k_new, p.table.cuda(), lens, starts)
    ids = torch.arange(p.n_pages, dtype=torch.int32, device="cuda")
    w.w4a16_kv_copy_pages(far, ids + (n - p.n_pages), ids)
    torch.cuda.synchronize()
    for a, b in zip(far, cache):
        assert torch.equal(a[:p.n_pages].nan_to_num(3), b.nan_to_num(3)) if a.is_floating_point() else torch.equal(a[:p.n_pages], b)


def test_long_context(cuda_lib):
    """A context long enough for every processor to share each head's keys."""
    p = Problem([40001, 3], [1, 1], heads=8, kv_heads=2, page=64, act="f16", seed=11)
    check(cuda_lib, p)
    check(cuda_lib, p, window=20000, sinks=4)


def test_binding_refusals(cuda_lib):
    w = cuda_lib
    p = Problem([20], [2])
    cache, table, lens, starts, rows = p.to_cuda(w)
    q = rows[:, :p.heads * p.dim].unflatten(1, (p.heads, p.dim))
    args = (table, lens, starts, 2)
    for bad, kind in [((q.float(), cache) + args, TypeError), ((q[..., :64], cache) + args, ValueError),
                      ((q.transpose(0, 1), cache) + args, ValueError),
                      ((q, cache._replace(v=cache.v[:1])) + args, ValueError),
                      ((q, cache._replace(k=cache.k.short(), v=cache.v.short())) + args, TypeError),
                      ((q, cache._replace(k_scale=cache.k_scale.half())) + args, TypeError),
                      ((q, cache._replace(k_scale=cache.k_scale[:1])) + args, ValueError),
                      ((q, cache, table.long(), lens, starts, 2), TypeError),
                      ((q, cache, table, lens, starts[:1], 2), ValueError),
                      ((q, cache, table[:, :1].t().contiguous()[:0], lens, starts, 2), ValueError)]:
        with pytest.raises(kind):
            w.w4a16_kv_attention(*bad)
    with pytest.raises(ValueError):
        w.w4a16_kv_attention(q, cache, *args, out=torch.empty_like(q.contiguous()[:1]))
    with pytest.raises(TypeError):
        w.w4a16_kv_attention(q, cache, *args, lse=torch.empty((2, p.heads), device="cuda", dtype=torch.float64))
    with pytest.raises(w.W4A16Error):
        w.w4a16_kv_attention(q, cache, *args, window=-1)
    with pytest.raises(w.W4A16Error):
        w.w4a16_kv_attention(q[:, :7], cache, *args)
    torch.cuda.synchronize()
    assert w.w4a16_last_device_error() == 0


@pytest.mark.parametrize("new", [1, 3, 200])
@pytest.mark.parametrize("act, store", [("f16", "int8"), ("bf16", "e4m3"), ("bf16", "int8")])
@pytest.mark.parametrize("scale", [-0.1, 0.0, 0.5])
def test_scales(cuda_lib, request, new, act, store, scale):
    """Negative and zero score scales: the largest weight is then the smallest score's, or everyone's."""
    if (new, act, store, scale) == (200, "bf16", "int8", 0.5):
        # One key holds a row's weight and its code is 0 in one dim; all other weights are below 2^-39 of that one,
        # where fp16 weights end, so the output is 0 there and not 5e-12.  The bound has no term for that.
        request.applymarker(pytest.mark.xfail(strict=True, reason="weights below 2^-39 of a row's largest count as 0"))
    check(cuda_lib, Problem([300 + new, new, 77 + new], [new, new, new], act=act, store=store, seed=7), scale=scale)


@pytest.mark.parametrize("heads, kv_heads", [(14, 2), (7, 1), (10, 2), (96, 1), (6, 2), (128, 1)])
@pytest.mark.parametrize("new", [[40, 9, 70], [300, 1, 30]])
def test_groups_that_do_not_divide_a_tile(cuda_lib, heads, kv_heads, new):
    lens = [n + past for n, past in zip(new, (100, 0, 600))]
    check(cuda_lib, Problem(lens, new, heads, kv_heads, 64, 32, seed=heads))


@pytest.mark.parametrize("new", [2, 140])
def test_values_before_a_bad_block_stay_finite(cuda_lib, new):
    """A block with a scale that is not finite shows in the tokens that see it, and in no other."""
    w = cuda_lib
    p = Problem([48 + new], [new], page=16, seed=12)
    last = (48 + new - 1) // 16
    p.vs[p.table[0, last].long(), 0] = float("nan")
    p.ks[p.table[0, last].long(), 1] = float("nan")
    out, _ = run(w, p)
    sees = torch.arange(48, 48 + new) >= last * 16
    bad = torch.isnan(out.float()).any(-1).any(-1).cpu()
    assert torch.equal(bad, sees)


@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("order", ["values first", "the same tensor"])
def test_where_k_and_v_lie(cuda_lib, new, order):
    """V below K in memory, and one tensor as both."""
    w = cuda_lib
    p = Problem([200 + new, new], [new, new], seed=13)
    if order == "the same tensor":
        p.v, p.vs = p.k, p.ks
    cache, table, lens, starts, rows = p.to_cuda(w)
    if order == "the same tensor":
        cache = w.KVCache(cache.k, cache.k, cache.k_scale, cache.k_scale)
    else:
        both = torch.stack([cache.v, cache.k])
        cache = w.KVCache(both[1], both[0], cache.k_scale, cache.v_scale)
    q = rows[:, :p.heads * p.dim].unflatten(1, (p.heads, p.dim))
    out = w.w4a16_kv_attention(q, cache, table, lens, starts, new)
    want, _, spread = attention(p)
    assert bool(((out.cpu().double() - want).abs() <= attention_tolerance(p, want, spread)).all())
    assert w.w4a16_last_device_error() == 0


def test_many_sequences(cuda_lib):
    """More sequences, and more row tiles, than one launch takes."""
    new = [(i * 7) % 4 if i % 3 else 80 for i in range(600)]
    lens = [n + (i * 13) % 50 for i, n in enumerate(new)]
    check(cuda_lib, Problem(lens, new, heads=16, kv_heads=1, dim=64, act="f16", seed=14))
    new = [1 + i % 2 for i in range(1100)]
    check(cuda_lib, Problem([n + i % 70 for i, n in enumerate(new)], new, heads=2, kv_heads=1, dim=64, seed=15))
