"""Calls on a stream that is not the current one: whose memory the results are, and calls at the same time."""
import pytest
import torch

from kv_reference import ACT, Problem, attention, attention_tolerance

pytestmark = pytest.mark.gpu
BUSY = 20_000_000                                    # clock cycles: some 10 ms


def calls(w, p, put):
    cache, table, lens, starts, rows = put
    q = rows[:, :p.heads * p.dim].unflatten(1, (p.heads, p.dim))
    found = {"attention": lambda s: [w.w4a16_kv_attention(q, cache, table, lens, starts, max(p.new), stream=s)],
            "read": lambda s: list(w.w4a16_kv_read(cache, table, lens, starts, p.T, ACT[p.act], stream=s))}
    for call in found.values():                      # a kernel's first call loads it, which takes its time
        [t.float().sum() + torch.empty_like(t).fill_(1).sum() for t in call(None) + call(torch.cuda.current_stream())]
    torch.cuda.synchronize()
    return found


@pytest.mark.parametrize("name", ["attention", "read"])
@pytest.mark.parametrize("wrap", [lambda s: s, lambda s: type("Handle", (), {"cuda_stream": s.cuda_stream})()])
def test_a_dropped_result_is_not_handed_out_while_its_stream_works(cuda_lib, name, wrap):
    p = Problem([70, 33], [1, 1], seed=1)
    put = p.to_cuda(cuda_lib)
    call = calls(cuda_lib, p, put)[name]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(BUSY)
    results = call(wrap(s))
    at = {t.data_ptr() for t in results}
    shape, dtype = results[0].shape, results[0].dtype
    del results
    later = [torch.empty(shape, dtype=dtype, device="cuda") for _ in range(64)]
    assert not s.query()                             # the call has not run yet
    assert not at & {t.data_ptr() for t in later}
    torch.cuda.synchronize()


@pytest.mark.parametrize("name", ["attention", "read"])
def test_a_result_is_not_where_the_current_stream_still_works(cuda_lib, name):
    p = Problem([70, 33], [1, 1], seed=1)
    put = p.to_cuda(cuda_lib)
    call = calls(cuda_lib, p, put)[name]
    s = torch.cuda.Stream()
    shape, dtype = call(None)[0].shape, ACT[p.act]
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    held = [torch.empty(shape, dtype=dtype, device="cuda").fill_(1) for _ in range(8)]
    at = {t.data_ptr() for t in held}
    del held
    results = call(s)
    assert not torch.cuda.current_stream().query()
    assert not at & {t.data_ptr() for t in results}
    torch.cuda.synchronize()


@pytest.mark.parametrize("name", ["attention", "read"])
def test_a_result_is_kept_for_the_current_stream(cuda_lib, name):
    """Used on the current stream and dropped: the next call on the other stream does not write over it."""
    p = Problem([70, 33], [1, 1], seed=1)
    put = p.to_cuda(cuda_lib)
    call = calls(cuda_lib, p, put)[name]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    results = call(s)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda._sleep(BUSY)
    sums = [t.float().sum() for t in results]
    at = {t.data_ptr() for t in results}
    del results
    again = call(s)
    assert not torch.cuda.current_stream().query()
    assert not at & {t.data_ptr() for t in again}
    torch.cuda.synchronize()
    assert all(bool(torch.isfinite(x)) for x in sums)


@pytest.mark.parametrize("new", [[1] * 20, [40, 300], [1, 200, 5]])
def test_two_streams_at_once(cuda_lib, new):
    w = cuda_lib
    problems = [Problem([n + 900 + 77 * i for i, n in enumerate(new)], new, seed=seed, store=store)
                for seed, store in ((1, "int8"), (2, "e4m3"))]
    puts = [p.to_cuda(w) for p in problems]
    wants = [attention(p) for p in problems]
    streams = [torch.cuda.Stream() for _ in problems]
    torch.cuda.synchronize()
    found = [calls(w, p, put)["attention"] for p, put in zip(problems, puts)]
    got = []
    for _ in range(20):
        for call, s in zip(found, streams):
            got.append(call(s)[0])
    torch.cuda.synchronize()
    for i, p in enumerate(problems):
        want, _, spread = wants[i]
        for out in got[i::2]:
            assert torch.equal(out, got[i])
        assert bool(((got[i].cpu().double() - want).abs() <= attention_tolerance(p, want, spread)).all())
    assert w.w4a16_last_device_error() == 0


def test_stream_is_the_current_one(cuda_lib):
    p = Problem([70, 33], [1, 1], seed=1)
    put = p.to_cuda(cuda_lib)
    for name, call in calls(cuda_lib, p, put).items():
        for a, b in zip(call(None), call(torch.cuda.current_stream())):
            torch.cuda.synchronize()
            assert torch.equal(a, b)
