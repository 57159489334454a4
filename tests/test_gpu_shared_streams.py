"""The operators for batches that share what they have cached on streams: results of a call on another stream, calls at the
same time, calls one after the other without a wait."""
import pytest
import torch

from test_gpu_beam import problem
from test_gpu_kv_shared import compare, grouped

pytestmark = pytest.mark.gpu
BUSY = 20_000_000                                    # clock cycles: some 10 ms


def put(v):
    return torch.tensor(v, dtype=torch.int32).cuda()


def attention(w, seed, members):
    p, starts, prefix = grouped([(300 + seed, [(i % 30, 1) for i in range(members)])] * 2, seed=seed)
    cache, table, lens, q_starts, rows = p.to_cuda(w)
    q, a, b = rows[:, :p.heads * p.dim].unflatten(1, (p.heads, p.dim)), put(starts), put(prefix)
    return p, lambda stream=None, lse=None: w.w4a16_kv_attention_shared(q, cache, table, lens, q_starts, 1, a, b, lse=lse,
                                                                        stream=stream)


def select(w, seed, rows):
    x, s, _ = problem(rows, 30000 + seed, "bf16", seed)
    x, s = x.cuda(), s.cuda()
    return lambda stream=None: list(w.w4a16_beam_select(x, s, 4, 4, stream=stream))


@pytest.fixture(params=[1, 2, None])
def kernels(request, cuda_lib):
    cuda_lib.w4a16_debug_set_config(10, request.param and [request.param])
    yield cuda_lib
    cuda_lib.w4a16_debug_set_config(10, None)


def test_attention_on_two_streams_at_once(kernels):
    w = kernels
    both = [attention(w, seed, members) for seed, members in ((1, 40), (2, 9))]
    lse = [torch.empty((p.T, p.heads), device="cuda") for p, _ in both]
    streams = [torch.cuda.Stream() for _ in both]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(12):
        for i, (_, call) in enumerate(both):
            outs[i].append(call(streams[i], lse[i]))
    torch.cuda.synchronize()
    for i, (p, _) in enumerate(both):
        compare(p, outs[i][0], lse[i])
        assert all(torch.equal(o, outs[i][0]) for o in outs[i])
    assert w.w4a16_last_device_error() == 0


def test_attention_beside_other_kernels(kernels):
    """Calls one after another with a tensor-core GEMM and a plain attention between them: each has the SMs and the tensor
    memory to itself in its turn."""
    w = kernels
    p, call = attention(w, 3, 50)
    lse = torch.empty((p.T, p.heads), device="cuda")
    x = torch.randn((512, 512), device="cuda").to(torch.bfloat16)
    qw = w.w4a16_pack(torch.randint(0, 16, (1024, 512), dtype=torch.uint8, device="cuda"))
    sc = torch.rand((1024, 4), device="cuda").to(torch.bfloat16)
    torch.cuda.synchronize()
    first = w.w4a16_gemm(x, qw, sc, None, 128)
    for _ in range(20):
        out = call(None, lse)
        y = w.w4a16_gemm(x, qw, sc, None, 128)
    torch.cuda.synchronize()
    compare(p, out, lse)
    assert torch.equal(first, y) and w.w4a16_last_device_error() == 0


def test_selection_on_two_streams_at_once(cuda_lib):
    w = cuda_lib
    both = [select(w, 1, 8), select(w, 2, 400)]
    want = [call() for call in both]
    streams = [torch.cuda.Stream() for _ in both]
    torch.cuda.synchronize()
    got = [[call(streams[i]) for call in [both[i]] for _ in range(10)] for i in range(2)]
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(a, b) for g in got[i] for a, b in zip(g, want[i]))


def test_growth_on_two_streams_at_once(cuda_lib):
    """Two pools: neither call is in the other's way."""
    from test_gpu_kv_pages import pool
    w, state = cuda_lib, []
    for seed in (1, 2):
        cache, table, lens, ref = pool(w, [20 + seed, 31, 0], 3, spare=60, seed=seed)
        table = torch.cat([table, torch.full((3, 20), -1, dtype=torch.int32, device="cuda")], 1).contiguous()
        state.append((cache, table, lens, ref, put([3, 1, 17]), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(4):
        for cache, table, lens, ref, new, s in state:
            w.w4a16_kv_grow(cache, table, lens, ref, new, 21, stream=s)
            w.w4a16_kv_reorder(table, lens, ref, put([0, 1, 2]), stream=s)
    torch.cuda.synchronize()
    for i, (cache, table, lens, ref, new, s) in enumerate(state):
        assert lens.tolist() == [33 + i, 35, 68]
        used = table[table >= 0]
        assert used.numel() == used.unique().numel() == int((ref == 1).sum()) == -(-(33 + i) // 16) + 3 + 5
    assert w.w4a16_last_device_error() == 0


def test_two_graphs_share_a_workspace(kernels):
    """Captured calls of different sizes with one workspace between them, replayed in turn on a stream."""
    w = kernels
    ws = torch.full((160 << 20,), 0xff, dtype=torch.uint8, device="cuda")
    calls, check = [], []
    for seed, members in ((4, 40), (5, 7)):
        p, starts, prefix = grouped([(300 + seed, [(i % 30, 1) for i in range(members)])] * 2, seed=seed)
        cache, table, lens, q_starts, rows = p.to_cuda(w)
        q, a, b = rows[:, :p.heads * p.dim].unflatten(1, (p.heads, p.dim)), put(starts), put(prefix)
        lse = torch.empty((p.T, p.heads), device="cuda")
        calls.append(lambda args=(q, cache, table, lens, q_starts, 1, a, b), lse=lse: w.w4a16_kv_attention_shared(
            *args, lse=lse, workspace=ws))
        check.append(lambda out, p=p, lse=lse: compare(p, out, lse))
    for seed, rows in ((1, 8), (2, 300)):
        x, s, _ = problem(rows, 20000 + seed, "f16", seed)
        x, s = x.cuda(), s.cuda()
        want = w.w4a16_beam_select(x, s, 4, 4)
        calls.append(lambda x=x, s=s: w.w4a16_beam_select(x, s, 4, 4, workspace=ws))
        check.append(lambda out, want=want: [torch.testing.assert_close(o, v, rtol=0, atol=0) for o, v in zip(out, want)])
    for call in calls:
        call()
    torch.cuda.synchronize()
    graphs, outs = [torch.cuda.CUDAGraph() for _ in calls], []
    for g, call in zip(graphs, calls):
        with torch.cuda.graph(g):
            outs.append(call())
    for out in outs:
        for o in out if isinstance(out, tuple) else [out]:
            o.fill_(1)
    for _ in range(5):
        for i in (0, 2, 1, 3, 0, 1, 2, 3):
            graphs[i].replay()
    torch.cuda.synchronize()
    for c, out in zip(check, outs):
        c(out)
    assert w.w4a16_last_device_error() == 0


@pytest.mark.parametrize("name", ["shared", "select", "grow"])
def test_a_dropped_result_is_not_handed_out_while_its_stream_works(cuda_lib, name):
    from test_gpu_kv_pages import pool
    w = cuda_lib
    if name == "shared":
        run = attention(w, 4, 5)[1]
        call = lambda s: [run(s)]
    elif name == "select":
        call = select(w, 3, 8)
    else:
        cache, table, lens, ref = pool(w, [20, 31], 2, spare=20)
        new = put([0, 0])
        call = lambda s: list(w.w4a16_kv_grow(cache, table, lens, ref, new, 8, stream=s))
    for s in (None, torch.cuda.current_stream()):
        [t.float().sum() + torch.empty_like(t).fill_(1).sum() for t in call(s)]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(BUSY)
    results = call(s)
    at = {t.data_ptr() for t in results}
    kinds = {(t.shape, t.dtype) for t in results}
    del results
    later = [torch.empty(shape, dtype=dtype, device="cuda") for shape, dtype in kinds for _ in range(64)]
    assert not s.query()                             # the call has not run yet
    assert not at & {t.data_ptr() for t in later}
    torch.cuda.synchronize()


LOG = r"""
import sys
sys.path[:0] = [%r, %r]
import w4a16_group_quantised_gb300 as w
from test_gpu_kv_shared import grouped, run
w.load_library()
p = grouped([(300, [(9, 1)] * 40)], seed=1)
run(w, *p)
w.w4a16_debug_set_config(10, [1])
run(w, *p), run(w, *p)
w.w4a16_debug_set_config(10, [2])
run(w, *p)
"""


def test_kernel_log(cuda_lib):
    import os
    import subprocess
    import sys
    here = os.path.dirname(os.path.abspath(__file__))
    r = subprocess.run([sys.executable, "-c", LOG % (os.path.dirname(here), here)], env=dict(os.environ, W4A16_LOG="1"),
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-2000:]
    lines = [line for line in r.stderr.splitlines() if line.startswith("w4a16: kv_attention_shared ")]
    assert [line.split("kernel=")[1].split()[0] for line in lines] == ["kv_attention", "few_rows", "few_rows+many_rows"]
    assert "tokens=40 seqs=40 groups=1 longest=1 heads=8/2 D=128 page=16 int8 bf16" in lines[0]
