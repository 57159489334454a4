"""Beam search's selection against its definition in 64 bits."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

ACT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
# An error bound of a score before it is rounded.  The sum's weights: 2^-22 each from the exponential, 2^-24 of an
# exponent of up to 32 from the products; a tile's 32 weights added in fp32 in any order, 31 * 2^-24.  The sum of
# these, as a relative error of the sum, is the error of its logarithm.
BOUND = 2.0 ** -22 + 2.0 ** -19 + 31 * 2.0 ** -24


def reference(logits, scores, width, n_out, finished=None, end=-1):
    """Lists of (score, row, token, finished) for each request, and the candidate after the last."""
    x, out = logits.double(), []
    for g in range(x.shape[0] // width):
        cand = []
        for r in range(g * width, (g + 1) * width):
            s = float(scores[r])
            if not math.isfinite(s):
                continue
            if finished is not None and bool(finished[r]):
                cand.append((s, r, end, True))
                continue
            if bool(x[r].isnan().any()) or bool((x[r] == math.inf).any()) or not bool((x[r] > -math.inf).any()):
                continue
            c = (x[r] - x[r].max()) - torch.log(torch.exp(x[r] - x[r].max()).sum()) + s
            # in the order of the logits: c rises with them, also where 64 bits of c no longer show it
            for t in torch.sort(x[r], descending=True, stable=True).indices[:n_out + 1].tolist():
                if c[t] > -math.inf:
                    cand.append((float(c[t]), r, t, t == end))
        cand.sort(key=lambda z: (-z[0], z[1]))                         # stable: a beam's own order stays
        out.append(cand[:n_out + 1])
    return out


def check(w, logits, scores, width, n_out, finished=None, end=-1, error=0, stream=None):
    put = lambda t: None if t is None else t.cuda()
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    args = logits if logits.is_cuda else put(logits), put(scores), put(finished)
    torch.cuda.synchronize()
    got = w.w4a16_beam_select(args[0], args[1], width, n_out, finished=args[2], end_token=end, stream=stream)
    torch.cuda.synchronize()
    assert [t.dtype for t in got] == [torch.float32, torch.int32, torch.int32, torch.bool]
    assert w.w4a16_last_device_error() == error
    w.w4a16_clear_device_error()
    got = [t.tolist() for t in got]
    for g, want in enumerate(reference(logits.cpu(), scores, width, n_out, finished, end)):
        for i in range(n_out):
            mine = tuple(t[g][i] for t in got)
            if i >= len(want):
                assert mine == (-math.inf, -1, -1, False), (g, i, mine)
                continue
            v = want[i][0]
            assert mine[0] == v or abs(mine[0] - v) <= BOUND + 2.0 ** -24 * abs(v) + 2.0 ** -149, (g, i, mine, want[i])
            # neighbours closer than both may be off, but not equal, can come in either order
            near = [want[j][0] for j in (i - 1, i + 1) if 0 <= j < len(want)]
            if all(u == v or abs(u - v) > 2 * BOUND for u in near):
                assert mine[1:] == want[i][1:], (g, i, mine, want[i])
    return got


def problem(rows, vocab, act, seed, pad=0, spread=3.0):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn((rows, vocab + pad), generator=g) * spread).to(ACT[act])[:, :vocab]
    scores = -torch.rand((rows,), generator=g) * 4 - 10
    return x, scores, g


@pytest.mark.parametrize("act", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("vocab, pad", [(1, 0), (2, 3), (7, 0), (31, 1), (257, 0), (8191, 0), (8192, 0), (8193, 7), (50001, 0),
                                         (50001, 15)])
def test_sizes(cuda_lib, act, vocab, pad):
    x, s, _ = problem(12, vocab, act, vocab + pad, pad)
    check(cuda_lib, x, s, 4, 4)
    check(cuda_lib, x, s, 3, 6)
    check(cuda_lib, x, s, 12, 1)


def on_gpu(x):
    """The same values with the same strides (rows that are views stay views)."""
    big = torch.full((x.shape[0] * x.stride(0),), 9.0, dtype=x.dtype).as_strided(x.shape, x.stride())
    big.copy_(x)
    flat = torch.full((x.shape[0] * x.stride(0) + 3,), 9.0, dtype=x.dtype, device="cuda")
    view = flat[3:].as_strided(x.shape, x.stride(), 3)
    view.copy_(big)
    return view


@pytest.mark.parametrize("act", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("vocab, pad", [(5, 2), (129, 0), (8200, 1), (33001, 4), (16384, 0)])
def test_rows_of_any_alignment(cuda_lib, act, vocab, pad):
    x, s, _ = problem(6, vocab, act, vocab, pad)
    check(cuda_lib, on_gpu(x), s, 2, 4)


@pytest.mark.parametrize("width, n_out", [(1, 1), (1, 64), (2, 3), (5, 10), (16, 16), (33, 64), (64, 64), (64, 1)])
@pytest.mark.parametrize("groups", [1, 3])
def test_widths(cuda_lib, width, n_out, groups):
    x, s, _ = problem(groups * width, 20000, "f32", width + n_out)
    check(cuda_lib, x, s, width, n_out)


@pytest.mark.parametrize("width, n_out, vocab, act", [(64, 64, 70001, "f32"), (16, 32, 131072, "bf16"), (40, 64, 66001, "f16"),
                                                      (16, 1, 131071, "f32"), (16, 32, 60, "f32"), (3, 64, 9000, "bf16")])
def test_many_candidates(cuda_lib, width, n_out, vocab, act):
    """More pieces, and more candidates of the best ones, than are compared with one another at once."""
    x, s, _ = problem(width, vocab, act, width + vocab)
    check(cuda_lib, x, s, width, n_out)
    check(cuda_lib, x, s * 0.001, width, n_out)                        # nearly even


@pytest.mark.parametrize("width, n_out", [(64, 64), (16, 32), (64, 1), (5, 64)])
def test_ties_of_many_beams(cuda_lib, width, n_out):
    """All beams alike, the pieces of each too."""
    x, s, g = problem(2 * width, 70000, "f32", width)
    x[:] = torch.arange(70000).remainder(7).float()
    s[:] = -2.0
    check(cuda_lib, x, s, width, n_out)
    x[:] = 0.0
    check(cuda_lib, x, s, width, n_out)
    x[:] = torch.randn(70000, generator=g)
    got = check(cuda_lib, x, s, width, n_out)
    # the best token of every beam, then the second
    rows = [i % width for i in range(n_out)]
    assert got[1] == [rows, [width + i for i in rows]]


@pytest.mark.parametrize("groups", [40, 200])
def test_many_requests(cuda_lib, groups):
    x, s, _ = problem(groups * 4, 9000, "bf16", groups)
    check(cuda_lib, x, s, 4, 8)


@pytest.mark.parametrize("rows, width", [(2048, 4), (2052, 4), (5000, 1), (3200, 64)])
def test_very_many_beams(cuda_lib, rows, width):
    """Up to 2048 those that go on are looked up first; of more, the others are passed over one by one."""
    x, s, g = problem(rows, 300, "bf16", rows)
    done = torch.rand(rows, generator=g) < 0.3
    s[torch.rand(rows, generator=g) < 0.2] = -math.inf
    x[done] = math.nan                                                 # never read
    check(cuda_lib, x, s, width, 4, finished=done, end=299)


@pytest.mark.parametrize("act", ["f16", "f32"])
def test_the_largest_vocabulary(cuda_lib, act):
    x, s, _ = problem(2, 1 << 24, act, 12, spread=2.0)
    check(cuda_lib, x, s, 2, 5)


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("n_out", [1, 5, 64])
def test_ties(cuda_lib, act, n_out):
    """Equal logits: the lower beam, then the lower token; more of them than any list holds."""
    x, s, g = problem(6, 40000, act, n_out)
    x.copy_(torch.randint(-2, 3, x.shape, generator=g))               # five values
    check(cuda_lib, x, s, 3, n_out)
    x.fill_(1.5)
    check(cuda_lib, x, s, 3, n_out)
    x.copy_(torch.where(torch.rand(x.shape, generator=g) < 0.5, 0.0, -0.0))
    check(cuda_lib, x, s, 2, n_out)


@pytest.mark.parametrize("vocab", [50001, 32000])
def test_equal_beams(cuda_lib, vocab):
    """Beams with the same logits and scores, at rows of different alignment."""
    x, s, _ = problem(8, vocab, "f16", 5)
    x[:], s[:] = x[0].clone(), -3.0
    got = check(cuda_lib, x, s, 4, 8)
    assert got[1][0] == [0, 1, 2, 3] * 2 and got[1][1] == [4, 5, 6, 7] * 2


@pytest.mark.parametrize("rising", [True, False])
@pytest.mark.parametrize("n_out", [4, 64])
def test_sorted_logits(cuda_lib, rising, n_out):
    """Rising logits: every tile's are better than all before it."""
    x, s, _ = problem(4, 100000, "f32", 1)
    x = torch.sort(x, 1, descending=not rising).values
    check(cuda_lib, x, s, 2, n_out)


@pytest.mark.parametrize("act", ["f16", "bf16", "f32"])
def test_masked(cuda_lib, act):
    """Tokens of -inf or the type's lowest value; beams of nothing else."""
    low = torch.finfo(ACT[act]).min
    x, s, g = problem(12, 20000, act, 2)
    for r, keep in enumerate([0, 1, 2, 5, 20000, 3, 0, 1, 2, 5, 0, 0]):
        gone = torch.ones(20000, dtype=torch.bool)
        gone[torch.randperm(20000, generator=g)[:keep]] = False
        x[r][gone] = -math.inf if r < 6 else low
    x[11, 10000:] = -math.inf                                          # half lowest, half -inf
    for width, n_out in ((6, 8), (3, 8), (1, 8), (12, 16)):
        check(cuda_lib, x, s, width, n_out)


@pytest.mark.parametrize("top", [1e4, 6e4, 1e9, 1e30, 3e38])
def test_large_logits(cuda_lib, top):
    x, s, g = problem(4, 9000, "f32", 3)
    x[:, 4000] = top
    x[1, 4000:4007] = top
    x[2] = -top
    x[3] = x[3] * (top / 16)                                           # 4000 becomes +inf from 1e30 on: reported
    error = -9 if bool((x == math.inf).any()) else 0
    assert (error != 0) == (top >= 1e30)
    check(cuda_lib, x, s, 2, 4, error=error)
    check(cuda_lib, x, s, 1, 4, error=error)


def test_not_numbers(cuda_lib):
    """A beam with NaN or +inf gives nothing, others are not touched by it."""
    x, s, _ = problem(8, 30000, "f32", 4)
    x[1, 29999] = math.nan
    x[4, 3] = math.inf
    x[6] = math.nan
    check(cuda_lib, x, s, 4, 8, error=-9)
    check(cuda_lib, x, s, 1, 8, error=-9)


def test_dead_and_finished_beams(cuda_lib):
    x, s, g = problem(16, 30000, "bf16", 6)
    s[1:4] = -math.inf
    s[5], s[6] = math.nan, math.inf
    s[8:12] = -math.inf
    x[0, 17] = 30.0
    done = torch.tensor([0, 1, 0, 0, 1, 0, 1, 0, 1, 0, 0, 0, 1, 1, 1, 1], dtype=torch.bool)
    x[done] = math.nan                                                 # never read
    got = check(cuda_lib, x, s, 4, 6, finished=done, end=17)
    assert got[3][0][0] and got[2][0][0] == 17
    check(cuda_lib, x, s, 8, 6, finished=done, end=29999)
    check(cuda_lib, x, s, 16, 20, finished=done, end=0)
    # no beam had finished: the end token alone ends them
    check(cuda_lib, x[:1], s[:1], 1, 3, end=17)


def test_outputs_workspace_and_stream(cuda_lib):
    w = cuda_lib
    x, s, _ = problem(8, 12345, "f16", 7)
    check(w, x, s, 4, 4, stream=torch.cuda.Stream())
    out = [torch.empty((2, 4), dtype=d, device="cuda") for d in (torch.float32, torch.int32, torch.int32, torch.bool)]
    ws = torch.empty(w.w4a16_beam_select_workspace(2, 4, 12345, 4), dtype=torch.uint8, device="cuda")
    a = w.w4a16_beam_select(x.cuda(), s.cuda(), 4, 4, out_scores=out[0], out_rows=out[1], out_tokens=out[2],
                            out_finished=out[3], workspace=ws)
    b = w.w4a16_beam_select(x.cuda(), s.cuda(), 4, 4)
    assert all(p is q for p, q in zip(a, out)) and all(torch.equal(p, q) for p, q in zip(a, b))
    empty = w.w4a16_beam_select(x.cuda()[:0], s.cuda()[:0], 4, 4)
    assert [tuple(t.shape) for t in empty] == [(0, 4)] * 4


def test_captured(cuda_lib):
    w = cuda_lib
    x, s, _ = problem(8, 30000, "bf16", 8)
    xd, sd, done = x.cuda(), s.cuda(), torch.zeros(8, dtype=torch.bool, device="cuda")
    w.w4a16_beam_select(xd, sd, 4, 4, finished=done, end_token=5)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = w.w4a16_beam_select(xd, sd, 4, 4, finished=done, end_token=5)
    for seed in (9, 10, 11):
        x, s, g = problem(8, 30000, "bf16", seed)
        fin = torch.rand(8, generator=g) < 0.3
        s[seed - 8] = -math.inf
        xd.copy_(x), sd.copy_(s), done.copy_(fin)
        graph.replay()
        torch.cuda.synchronize()
        again = w.w4a16_beam_select(xd, sd, 4, 4, finished=done, end_token=5)
        assert all(torch.equal(p, q) for p, q in zip(got, again))
        check(w, x, s, 4, 4, finished=fin, end=5)
