"""Captured calls replayed with other lengths, their scratch left as each replay leaves it."""
import pytest
import torch

from kv_reference import ACT, Problem, append, attention, attention_tolerance

pytestmark = pytest.mark.gpu


def captured(call):
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        call()
    return graph


@pytest.mark.parametrize("scratch", ["own", "the call's"])
@pytest.mark.parametrize("heads, kv_heads, dim, page, layout, store", [(8, 2, 128, 16, "heads", "int8"),
                                                                      (4, 1, 64, 64, "tokens", "e4m3")])
@pytest.mark.parametrize("longest, batches", [
    # few rows: (new, lens), where the cuts between CTAs move from one replay to the next
    (1, [([1, 1, 1], [9000, 40, 7000]), ([1, 1, 1], [300, 16000, 1]), ([1, 1, 1], [1, 1, 1]), ([1, 1, 1], [16000, 16000, 16000]),
         ([1, 1, 1], [4000, 15000, 800])]),
    # many rows, whole tiles dealt out or in shares
    (300, [([300, 300, 300], [300, 3000, 9000]), ([300, 300, 300], [16000, 300, 300]), ([300, 300, 300], [9000, 9000, 9000]),
           ([300, 300, 300], [320, 400, 300])]),
    # both kernels in one call
    (290, [([290, 1, 9], [8000, 16000, 500]), ([9, 290, 1], [9000, 290, 12000]), ([1, 9, 290], [1, 700, 16000]),
           ([290, 9, 1], [290, 15000, 16000])]),
])
def test_attention(cuda_lib, scratch, heads, kv_heads, dim, page, layout, store, longest, batches):
    w = cuda_lib
    p = Problem([16000] * 3, batches[0][0], heads, kv_heads, dim, page, store, layout, act="f16", seed=longest)
    cache, table, lens, starts, rows = p.to_cuda(w)
    q = rows[:, :heads * dim].unflatten(1, (heads, dim))
    out = torch.empty(q.shape, dtype=q.dtype, device="cuda")
    lse = torch.empty(q.shape[:2], device="cuda")
    ws = None
    if scratch == "own":
        need = w.w4a16_kv_attention_workspace(heads, kv_heads, dim, 3, p.T)
        ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    graph = captured(lambda: w.w4a16_kv_attention(q, cache, table, lens, starts, longest, out=out, lse=lse, workspace=ws))
    for new, lengths in batches + batches[::-1]:
        assert sum(new) == p.T
        lens.copy_(torch.tensor(lengths, dtype=torch.int32))
        p.lens, p.new = lengths, new
        p.starts = torch.tensor([0, new[0], new[0] + new[1], p.T], dtype=torch.int32)
        starts.copy_(p.starts)
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        want, _, spread = attention(p)
        assert bool(((out.cpu().double() - want).abs() <= attention_tolerance(p, want, spread)).all())
    assert w.w4a16_last_device_error() == 0


def test_append_and_read(cuda_lib):
    w = cuda_lib
    p = Problem([70, 70, 70], [40, 0, 7], store="e4m3", seed=1)
    cache, table, lens, starts, rows = p.to_cuda(w)
    begin = [t.clone() for t in cache]
    a, b = p.heads * p.dim, (p.heads + p.kv_heads) * p.dim
    k, v = (torch.empty((p.T, p.kv_heads, p.dim), dtype=ACT[p.act], device="cuda") for _ in range(2))

    def call():
        w.w4a16_kv_append(cache, rows[:, a:b].unflatten(1, (p.kv_heads, p.dim)), rows[:, b:].unflatten(1, (p.kv_heads, p.dim)),
                          table, lens, starts)
        w.w4a16_kv_read(cache, table, lens, starts, p.T, ACT[p.act], k_out=k, v_out=v)

    graph = captured(call)
    codes = p.k, p.v, p.ks, p.vs
    for new, lengths in (([40, 0, 7], [70, 70, 70]), ([1, 45, 1], [1, 64, 17]), ([0, 0, 47], [5, 5, 47]), ([16, 16, 15], [16, 33, 70])):
        for t, old in zip(cache, begin):
            t.copy_(old)
        lens.copy_(torch.tensor(lengths, dtype=torch.int32))
        p.lens, p.new, (p.k, p.v, p.ks, p.vs) = lengths, new, codes
        starts.copy_(torch.tensor([0, new[0], new[0] + new[1], p.T], dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        want = append(p)
        for got, ref in zip(cache, want):
            assert torch.equal(got.cpu().view(torch.uint8), ref.view(torch.uint8))
        at = 0
        p.k, p.v, p.ks, p.vs = want[0].view(codes[0].dtype), want[1].view(codes[1].dtype), want[2], want[3]
        for i, (n, m) in enumerate(zip(lengths, new)):
            for got, c, s in ((k, p.k, p.ks), (v, p.v, p.vs)):
                assert torch.equal(got[at:at + m].cpu(), p.values(c, s, i, n)[n - m:].float().to(ACT[p.act]))
            at += m
    assert w.w4a16_last_device_error() == 0


def test_fork_free_trim_and_compact(cuda_lib):
    """One captured round of a scheduler's page work, replayed on other tables: as the calls one by one."""
    w = cuda_lib

    def pool(seed):
        g = torch.Generator().manual_seed(seed)
        lens = torch.randint(1, 300, (4,), generator=g).tolist()
        p = Problem(lens, [0] * 4, 4, 2, 64, 16, seed=seed, spare=110 - sum(-(-n // 16) for n in lens))
        cache, table, n, _, _ = p.to_cuda(w)
        full = torch.full((8, 19), -1, dtype=torch.int32, device="cuda")
        full[:4, :table.shape[1]] = table
        ref = torch.zeros(p.n_pages, dtype=torch.int32, device="cuda")
        ref[table[table >= 0].long()] = 1
        return list(cache) + [full, torch.cat([n, torch.zeros_like(n)]), ref]

    ids = torch.arange(8, dtype=torch.int32, device="cuda")
    live = torch.zeros(1, dtype=torch.int32, device="cuda")

    def work(s):
        cache, (table, lens, ref) = w.KVCache(*s[:4]), s[4:]
        w.w4a16_kv_fork(cache, table, lens, ref, ids[:4], ids[4:])
        w.w4a16_kv_free(table, lens, ref, ids[1:3])
        w.w4a16_kv_trim(table, lens, ref, 16, 100, 4)
        w.w4a16_kv_compact(cache, table, ref, n_live=live)

    state = pool(0)
    assert state[0].shape[0] == 110
    graph = captured(lambda: work(state))
    for seed in (0, 1, 2, 3):
        for t, x in zip(state, pool(seed)):
            t.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        m = int(live)
        one = pool(seed)
        work(one)
        torch.cuda.synchronize()
        assert int(live) == m and bool((state[6][:m] > 0).all()) and not bool(state[6][m:].any())
        for a, b in zip(state, one):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert w.w4a16_last_device_error() == 0
