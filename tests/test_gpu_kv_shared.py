"""Attention of a batch whose sequences share their first pages, against the
definition in 64 bits over each sequence's own table."""
import math

import pytest
import torch

from kv_reference import Problem, attention, attention_tolerance

pytestmark = pytest.mark.gpu


@pytest.fixture(params=["few", "many"])
def shared_kernels(request, cuda_lib):
    """Those that look at the groups."""
    cuda_lib.w4a16_debug_set_config(10, [1 if request.param == "few" else 2])
    yield cuda_lib
    cuda_lib.w4a16_debug_set_config(10, None)


@pytest.fixture(params=["few", "many", "chosen"])
def kernels(request, cuda_lib):
    """The few-rows kernel alone, the tensor-core kernel where there are rows for it, or whichever the sizes call for
    (with these small ones w4a16_kv_attention itself)."""
    if request.param != "chosen":
        cuda_lib.w4a16_debug_set_config(10, [1 if request.param == "few" else 2])
    yield cuda_lib
    cuda_lib.w4a16_debug_set_config(10, None)


def grouped(groups, heads=8, kv_heads=2, dim=128, page=16, store="int8", layout="heads", act="bf16", seed=0, loose=()):
    """(problem, group starts, prefix lengths): groups of (prefix, [(past beyond the prefix, new tokens), ...]); `loose`
    sequences (past, new) come after them and are in no group."""
    lens, new, starts, prefix = [], [], [0], []
    for p, members in groups:
        lens += [p + past + n for past, n in members]
        new += [n for _, n in members]
        starts.append(starts[-1] + len(members))
        prefix.append(p)
    lens, new = lens + [p + n for p, n in loose], new + [n for _, n in loose]
    prob = Problem(lens, new, heads, kv_heads, dim, page, store, layout, act, seed=seed)
    for g, p in enumerate(prefix):
        for b in range(starts[g] + 1, starts[g + 1]):
            prob.table[b, :p // page] = prob.table[starts[g], :p // page]
    return prob, starts, prefix


def run(w, p, starts, prefix, max_new=None, lse=True, scale=None, stream=None, workspace=None):
    cache, table, lens, q_starts, rows = p.to_cuda(w)
    q = rows[:, :p.heads * p.dim].unflatten(1, (p.heads, p.dim))
    out_lse = torch.full((p.T, p.heads), 7.0, device="cuda") if lse else None
    put = lambda v: torch.tensor(v, dtype=torch.int32).cuda()
    a, b = put(starts), put(prefix)
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    out = w.w4a16_kv_attention_shared(q, cache, table, lens, q_starts, max(p.new) if max_new is None else max_new, a, b,
                                      scale=scale, lse=out_lse, stream=stream, workspace=workspace)
    torch.cuda.synchronize()
    return out, out_lse


def weights_floor(p):
    """What the spacing of the smallest weights is worth.  A set of keys' largest weight, its value scale included, is
    at 2^14 or above in fp16, whose subnormal numbers are rounded by up to 2^-25: 2^-39 of the largest for each key.
    With value scales that differ by up to 3 and weights that sum to the denominator that is at most 3 * 2^-39 sum |v|.
    It shows where the keys that count have a value of 0 in a dim."""
    top = float((p.v.float().abs().nan_to_num(0) * p.vs.nan_to_num(0, 0, 0)[..., None, None]).max())
    return 3 * 2.0 ** -39 * max(p.lens) * top


def compare(p, out, lse, scale=None):
    want, want_lse, spread = attention(p, scale)
    err, tol = (out.cpu().double() - want).abs(), attention_tolerance(p, want, spread) + weights_floor(p)
    assert bool((err <= tol).all()), f"max excess {(err - tol).max().item():.3e}, max error {err.max().item():.3e}"
    empty = want_lse == -math.inf
    assert torch.equal(lse.cpu() == -math.inf, empty)
    # fp32 sums of weights that are each good to 2^-12, at scores of some tens
    assert bool(((lse.cpu().double() - want_lse)[~empty].abs() <= 2.0 ** -11 + 2.0 ** -18 * want_lse[~empty].abs()).all())


def check(w, p, starts, prefix, **kw):
    out, lse = run(w, p, starts, prefix, **kw)
    compare(p, out, lse, kw.get("scale"))
    assert w.w4a16_last_device_error() == 0
    return out


@pytest.mark.parametrize("store, act", [("int8", "bf16"), ("e4m3", "f16"), ("int8", "f16"), ("e4m3", "bf16")])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("heads, kv_heads", [(4, 4), (8, 2), (14, 2), (8, 1), (40, 2)])
def test_single_tokens(kernels, store, act, dim, heads, kv_heads):
    groups = [(100, [(0, 1), (3, 1), (40, 1)]), (16, [(0, 1), (200, 1)]), (333, [(5, 1)] * 4), (64, [(9, 1)])]
    check(kernels, *grouped(groups, heads, kv_heads, dim, 16, store, "heads", act, seed=heads + dim))


@pytest.mark.parametrize("heads, kv_heads, dim", [(128, 1, 128), (256, 2, 64), (64, 64, 64), (33, 11, 128)])
def test_many_heads(kernels, heads, kv_heads, dim):
    groups = [(150, [(0, 1), (3, 1), (40, 2)]), (16, [(0, 1), (100, 3)]), (90, [(9, 1)])]
    check(kernels, *grouped(groups, heads, kv_heads, dim, seed=heads))


@pytest.mark.parametrize("members", [4, 40])
def test_tokens_without_keys(kernels, members):
    """Lengths of zero, and shorter than the tokens that the sequence brings: these see nothing, and nothing is shared."""
    w = kernels
    p, starts, prefix = grouped([(100, [(7, 3)] * members), (100, [(7, 3)] * members)], seed=3)
    p.lens[1], p.lens[members], p.lens[members + 1] = 0, 2, 1
    out, lse = run(w, p, starts, prefix)
    assert int((lse == -math.inf).sum()) == (3 + 1 + 2) * p.heads
    assert w.w4a16_last_device_error() == -9             # a sequence shorter than what it brings, as everywhere
    w.w4a16_clear_device_error()
    # the definition wants a key at least: with one the second sequence's last token has it
    assert bool((out[5] == 0).all())
    p.lens[1] = 1
    want, want_lse, _ = attention(p)
    out[5], lse[5] = want[5].to(out), want_lse[5].to(lse)
    compare(p, out, lse)


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("layout", ["heads", "tokens", "padded", "pairs"])
@pytest.mark.parametrize("members", [2, 9, 40, 70])
def test_pages_layouts_and_rows(kernels, page, layout, members):
    """Rows a group and kv head from 8 to 280: both kernels, one and two halves of the large tile, several tiles."""
    groups = [(300, [(i * 7 % 50, 1) for i in range(members)]), (128, [(3, 1)] * 3)]
    check(kernels, *grouped(groups, page=page, layout=layout, seed=page + members))
    check(kernels, *grouped(groups, page=page, layout=layout, store="e4m3", dim=64, act="f16", seed=members))


@pytest.mark.parametrize("prefix", [0, 1, 15, 16, 17, 127, 128, 129, 255, 256, 1000])
@pytest.mark.parametrize("members", [3, 40])
def test_prefix_lengths(kernels, prefix, members):
    check(kernels, *grouped([(prefix, [(i % 5, 1 + i % 2) for i in range(members)])], seed=prefix))


@pytest.mark.parametrize("new", [1, 2, 5, 40, 200])
@pytest.mark.parametrize("page", [16, 64])
def test_several_tokens(kernels, new, page):
    """Sequences with many tokens, few and none; the rest of a sequence is causal."""
    groups = [(257, [(0, new), (30, 1), (0, 0), (7, new)]), (90, [(1, 3), (100, new)]), (50, [(2, 0), (3, 0)])]
    check(kernels, *grouped(groups, page=page, seed=new + page, loose=[(33, new), (0, 2)]))


def test_mixed_groups(kernels):
    """Groups for either kernel and sequences for either kernel in one call."""
    groups = [(200, [(4, 1)] * 60), (500, [(1, 1), (2, 1)]), (77, [(9, 50), (8, 1)])] + [(64, [(3, 1)] * 2)] * 20
    check(kernels, *grouped(groups, page=32, seed=8, loose=[(400, 90)]))
    check(kernels, *grouped(groups, page=16, heads=16, kv_heads=2, seed=9, loose=[(5, 1)] * 3))


def test_no_groups(kernels):
    p, _, _ = grouped([], loose=[(100, 1), (0, 1), (40, 60)])
    check(kernels, p, [0], [])
    check(kernels, p, [1, 1, 3, 3], [10, 0, 20])                     # nothing in common that is a page
    check(kernels, p, [3, 3], [50])


@pytest.mark.parametrize("prefix", [96, 97, 112, 400])
def test_prefix_past_the_past(kernels, prefix):
    """A prefix that reaches into the new tokens counts as far as the shortest past of those that bring any."""
    p, starts, _ = grouped([(96, [(0, 3), (20, 1), (0, 0)])], seed=2)
    p.table[2, :6] = -1                                               # brings nothing: its row is not read
    check(kernels, p, starts, [prefix])


def test_pages_of_the_first_row_that_brings_tokens(shared_kernels):
    """Whatever the others' rows say for the shared part is not looked at."""
    w = shared_kernels
    for members in (4, 50):
        p, starts, prefix = grouped([(130, [(5, 0)] + [(7, 1)] * members)], seed=members)
        want = attention(p)
        p.table[0] = -1
        p.table[2:, :8] = 2**31 - 1
        out, lse = run(w, p, starts, prefix)
        err, tol = (out.cpu().double() - want[0]).abs(), attention_tolerance(p, want[0], want[2])
        assert bool((err <= tol).all())
        assert w.w4a16_last_device_error() == 0


@pytest.mark.parametrize("scale", [0.0, -0.125, 1.5])
@pytest.mark.parametrize("members", [3, 40])
def test_scales(kernels, scale, members):
    check(kernels, *grouped([(150, [(9, 1)] * members)], seed=4), scale=scale)


@pytest.mark.parametrize("members, max_new", [(5, 0), (5, 4), (40, 0), (40, 1), (5, 1000)])
def test_any_longest(kernels, members, max_new):
    check(kernels, *grouped([(150, [(9, 1 + i % 4) for i in range(members)])], seed=5), max_new=max_new)


def test_long_prefix(kernels):
    groups = [(20000, [(3, 1), (700, 1), (20, 2)]), (9000, [(100, 1)] * 33)]
    check(kernels, *grouped(groups, kv_heads=2, page=64, store="e4m3", layout="tokens", seed=6))
    check(kernels, *grouped(groups, kv_heads=1, dim=64, page=16, seed=7))


@pytest.mark.parametrize("groups", [[(12000, [(9000, 1), (11000, 1)])], [(30000, [(3, 1)] * 2)],
                                    [(12000, [(9000, 1), (11000, 1)]), (10000, [(8000, 2), (9000, 1)])]])
@pytest.mark.parametrize("dim, page", [(128, 64), (64, 16)])
def test_few_long_tiles_token_first(kernels, groups, dim, page):
    """Tiles of one entry cut into the same number of pieces, or not where that would be uneven."""
    check(kernels, *grouped(groups, heads=16, kv_heads=8, dim=dim, page=page, store="e4m3", layout="tokens", act="f16", seed=dim))


@pytest.mark.parametrize("members", [3, 60])
def test_without_early_start(kernels, members):
    """One kernel after the other, each waiting for the one before it."""
    kernels.w4a16_debug_set_config(3, [0])
    try:
        check(kernels, *grouped([(500, [(i % 9, 1) for i in range(members)]), (80, [(1, 40), (2, 1)])], seed=21))
    finally:
        kernels.w4a16_debug_set_config(3, [1])


@pytest.mark.parametrize("members, prefix", [(160, 4000), (64, 6000)])
@pytest.mark.parametrize("heads, kv_heads", [(32, 8), (32, 4)])
def test_as_the_sizes_call_for(cuda_lib, members, prefix, heads, kv_heads):
    """Large enough for the tensor-core kernel to be chosen, with the other beside it."""
    groups = [(prefix, [(i * 37 % 300, 1) for i in range(members)]), (60, [(1000, 1)] * 3)]
    check(cuda_lib, *grouped(groups, heads=heads, kv_heads=kv_heads, seed=members))


@pytest.mark.parametrize("count", [513, 1100])
def test_many_sequences_and_groups(kernels, count):
    """More of them than one launch takes."""
    groups = [(33, [(i % 3, 1), (1, 1)]) for i in range(count // 2)]
    check(kernels, *grouped(groups, heads=2, kv_heads=1, dim=64, seed=9))
    check(kernels, *grouped([(40, [(i % 3, 1) for i in range(count)])], heads=2, kv_heads=1, dim=64, seed=10))


def test_rows_of_no_sequence(kernels):
    """Rows before the first start and after the last: zeros and -inf."""
    w = kernels
    p, starts, prefix = grouped([(100, [(2, 1)] * 3), (40, [(1, 2)] * 2)], seed=11)
    cache, table, lens, q_starts, rows = p.to_cuda(w)
    rows = torch.cat([rows.new_full((2, rows.shape[1]), 9.0), rows, rows.new_full((3, rows.shape[1]), 9.0)])
    q = rows[:, :p.heads * p.dim].unflatten(1, (p.heads, p.dim))
    lse = torch.full((p.T + 5, p.heads), 7.0, device="cuda")
    put = lambda v: torch.tensor(v, dtype=torch.int32).cuda()
    out = w.w4a16_kv_attention_shared(q, cache, table, lens, q_starts + 2, 2, put(starts), put(prefix), lse=lse)
    torch.cuda.synchronize()
    compare(p, out[2:-3], lse[2:-3])
    for part, part_lse in ((out[:2], lse[:2]), (out[-3:], lse[-3:])):
        assert not bool(part.any()) and bool((part_lse == -math.inf).all())
    assert w.w4a16_last_device_error() == 0


@pytest.mark.parametrize("starts, prefix", [([0, 3, 2, 5], [64, 64, 64]), ([-1, 2, 5], [64, 64]), ([0, 2, 6], [64, 64]),
                                             ([0, 2, 5], [64, -1]), ([4, 1, 2**31 - 1], [64, 64]), ([5, 0], [64])])
def test_groups_that_cannot_be(shared_kernels, starts, prefix):
    """Reported; sequences of groups that are right are right, nothing out of range is read."""
    w = shared_kernels
    p, _, _ = grouped([(64, [(5, 1)] * 5)], seed=12)
    run(w, p, starts, prefix)
    assert w.w4a16_last_device_error() == -9
    w.w4a16_clear_device_error()
    check(w, p, [0, 5], [64])


def test_bad_pages(kernels):
    """A page id out of range among the shared ones: its keys are left out for all of the group, and it is reported."""
    w = kernels
    for members in (3, 45):
        p, starts, prefix = grouped([(96, [(5, 1)] * members)], seed=13)
        p.table[0, 2], p.table[1:, 2] = p.n_pages, -1
        out, _ = run(w, p, starts, prefix)
        assert w.w4a16_last_device_error() == -9
        w.w4a16_clear_device_error()
        assert bool(out.isfinite().all())
        # the same without these 16 keys: the page in front of it twice at half the weight is another problem, so by hand
        for b in (0, members - 1):
            n = p.lens[b]
            keep = [i for i in range(n) if i // 16 != 2]
            p.table[:, 2] = 0
            k, v = p.values(p.k, p.ks, b, n)[keep], p.values(p.v, p.vs, b, n)[keep]
            for a in range(p.heads):
                x = torch.softmax(p.q[b, a].double() @ k[:, a // 4].T * p.dim ** -0.5, 0)
                want, spread = x @ v[:, a // 4], x @ v[:, a // 4].abs()
                assert bool(((out[b, a].cpu().double() - want).abs() <= attention_tolerance(p, want, spread)).all())


def test_blocks_that_are_not_finite(kernels):
    """Seen by the group: NaN for the group, nothing for the others."""
    w = kernels
    p, starts, prefix = grouped([(64, [(5, 1)] * 3), (64, [(5, 1)] * 40)], seed=14)
    p.vs[p.table[0, 1].long()] = math.inf
    p.v.view(torch.int8)[p.table[0, 1].long()] = 0
    out, _ = run(w, p, starts, prefix)
    assert bool(out[:3].isnan().all()) and bool(out[3:].isfinite().all())


@pytest.mark.parametrize("members", [4, 40])
def test_captured(kernels, members):
    """One captured call, replayed with other lengths, groups and prefixes."""
    w = kernels
    p, starts, prefix = grouped([(200, [(9, 1)] * members), (200, [(3, 1)] * members)], seed=15)
    cache, table, lens, q_starts, rows = p.to_cuda(w)
    q = rows[:, :p.heads * p.dim].unflatten(1, (p.heads, p.dim))
    put = lambda v: torch.tensor(v, dtype=torch.int32).cuda()
    a, b, lse = put(starts), put(prefix), torch.empty((p.T, p.heads), device="cuda")
    call = lambda: w.w4a16_kv_attention_shared(q, cache, table, lens, q_starts, 1, a, b, lse=lse)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    for short, s, pre in ((0, starts, [200, 200]), (3, starts, [100, 0]), (60, [0, 2, 2 * members], [64, 17]),
                          (5, [0, 0, members], [50, 190])):
        p.lens = [n - short for n in p.lens]
        lens.copy_(put(p.lens)), a.copy_(put(s)), b.copy_(put(pre))
        # a group over both halves has nothing in common: make it so that it has
        t = p.table.clone()
        for g in range(2):
            for i in range(s[g], s[g + 1]):
                t[i, :pre[g] // 16] = t[s[g], :pre[g] // 16]
        p.table, keep = t, p.table
        table.copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        compare(p, out, lse)
        p.lens, p.table = [n + short for n in p.lens], keep
    assert w.w4a16_last_device_error() == 0


def test_other_stream_and_workspace(kernels):
    """A workspace of its own, used by one call after the other, with other sizes and with the plain attention."""
    w = kernels
    ws = torch.full((160 << 20,), 0xff, dtype=torch.uint8, device="cuda")
    for i, members in enumerate((3, 40, 5, 70)):
        p, starts, prefix = grouped([(300, [(9, 1 + i)] * members)], seed=16 + i)
        check(w, p, starts, prefix, workspace=ws)
        check(w, p, starts, prefix, stream=torch.cuda.Stream())
        cache, table, lens, q_starts, rows = p.to_cuda(w)
        q = rows[:, :p.heads * p.dim].unflatten(1, (p.heads, p.dim))
        lse = torch.empty((p.T, p.heads), device="cuda")
        compare(p, w.w4a16_kv_attention(q, cache, table, lens, q_starts, 1 + i, lse=lse, workspace=ws), lse)
    need = w.w4a16_kv_attention_shared_workspace(8, 2, 128, 70, 1, 280)
    assert need < ws.numel()
    with pytest.raises(w.W4A16Error):
        run(w, p, starts, prefix, workspace=ws[:need - 16])


@pytest.mark.parametrize("groups", [[(9000, [(5, 1)] * 3)], [(3000, [(500, 1)] * 50)], [(400, [(0, 300)] * 2)]])
@pytest.mark.parametrize("hold", [1, 2])
def test_waits_run_out_and_the_next_call_is_right(kernels, groups, hold):
    w = kernels
    p, starts, prefix = grouped(groups, seed=17)
    w.w4a16_clear_device_error()
    w.w4a16_debug_set_config(7, [hold])
    try:
        run(w, p, starts, prefix)
    finally:
        w.w4a16_debug_set_config(7, None)
    assert w.w4a16_last_device_error() == -8
    w.w4a16_clear_device_error()
    check(w, p, starts, prefix)
