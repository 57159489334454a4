"""The operators for batches that share what they have cached, run together as a beam search: each stage of each step
against its definition, captured steps against eager ones."""
import importlib.util
import os

import pytest
import torch

from kv_reference import ROUND
from test_gpu_beam import reference
from test_gpu_kv_grow import model as grown
from test_gpu_kv_pages import counts
from test_gpu_kv_reorder import want as reordered

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example(cuda_lib):
    spec = importlib.util.spec_from_file_location("beam_search", os.path.join(ROOT, "examples", "beam_search.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def small(ex, requests=3, width=4, page=16, store=torch.int8, **kw):
    model = ex.Model(hidden=512, heads=8, kv_heads=2, dim=64, vocab=1000, G=64, **kw)
    return ex.Search(model, requests, width, pages=200, columns=40, page=page, store=store)


def prompts(search, lens, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randint(0, search.model.vocab, (n,), generator=g, device="cuda") for n in lens]


class Recorded:
    """The example's calls of the library, with their arguments before and after."""

    def __init__(self, ex, monkeypatch):
        self.calls = []
        for name in ("w4a16_beam_select", "w4a16_kv_reorder", "w4a16_kv_grow", "w4a16_kv_attention_shared"):
            monkeypatch.setattr(ex.w, name, self.wrap(name, getattr(ex.w, name)), raising=False)

    def wrap(self, name, call):
        keep = lambda t: t.clone() if isinstance(t, torch.Tensor) else t

        def run(*args, **kw):
            before = [keep(a) for a in args], {k: keep(v) for k, v in kw.items()}
            out = call(*args, **kw)
            self.calls.append((name, before, [keep(a) for a in args], out if isinstance(out, tuple) else (out,)))
            return out
        return run


def check_attention(search, args, out):
    q, cache, table, lens, starts = args[:5]
    m = search.model
    for b, n in enumerate(lens.tolist()):
        pages = table[b, :-(-n // cache.k.shape[2])].long()
        k, v = ((c[pages].double() * s[pages].double()[..., None, None]).transpose(1, 2).flatten(0, 1)[:n]
                for c, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)))
        for a in range(m.heads):
            p = torch.softmax(q[b, a].double() @ k[:, a * m.kv_heads // m.heads].T * m.dim ** -0.5, -1)
            val = v[:, a * m.kv_heads // m.heads]
            # one rounding of the output and fp16 weights, as for the attention's own tests
            tol = ROUND["bf16"] * (p @ val).abs() + (2.0 ** -11 + 2.0 ** -12) * (p @ val.abs()) + 2.0 ** -134
            assert bool(((out[b, a].double() - p @ val).abs() <= tol).all())


@pytest.mark.parametrize("kernels", [None, 1, 2])
@pytest.mark.parametrize("page, store", [(16, torch.int8), (32, torch.float8_e4m3fn)])
def test_stages(example, monkeypatch, kernels, page, store):
    ex, w = example, example.w
    if kernels:
        w.w4a16_debug_set_config(10, [kernels])
    try:
        search = small(ex, page=page, store=store)
        search.begin(prompts(search, [100, 16, 77]))
        seen = Recorded(ex, monkeypatch)
        for _ in range(6):
            search.step()
        torch.cuda.synchronize()
    finally:
        w.w4a16_debug_set_config(10, None)
    assert w.w4a16_last_device_error() == 0
    for name, (args, kw), after, out in seen.calls:
        if name == "w4a16_beam_select":
            best = reference(args[0].cpu(), args[1].cpu(), search.width, search.width, kw["finished"].cpu(), search.end_token)
            for g, cand in enumerate(best):
                for i, (score, row, token, end) in enumerate(cand[:search.width]):
                    assert abs(float(out[0][g, i]) - score) < 1e-4
                    near = [c[0] for j, c in enumerate(cand) if abs(j - i) == 1]
                    if all(abs(c - score) > 1e-4 for c in near):
                        assert (int(out[1][g, i]), int(out[2][g, i]), bool(out[3][g, i])) == (row, token, end)
        elif name == "w4a16_kv_reorder":
            t, n = reordered(args[0].cpu(), args[1].cpu(), args[3].tolist(), None)
            assert torch.equal(after[0].cpu(), t) and torch.equal(after[1].cpu(), n)
            assert after[2].tolist() == counts(t, after[2].shape[0])
        elif name == "w4a16_kv_grow":
            t, n, ref, starts, pos, slots, _, wrong = grown(args[1].tolist(), args[2].tolist(), args[3].tolist(),
                                                            args[4].tolist(), page, args[5])
            assert not wrong and (after[1].tolist(), after[2].tolist(), after[3].tolist()) == (t, n, ref)
            assert [x.tolist() for x in out] == [starts, pos, slots]
            # whoever appends has its last page for itself
            last = [t[b][(n[b] - 1) // page] for b in range(len(n))]
            assert len(set(last)) == len(last)
    # a later append may scale a page's codes again: the cache as the last step left it
    name, _, after, out = [c for c in seen.calls if c[0] == "w4a16_kv_attention_shared"][-1]
    check_attention(search, after, out[0])


def test_beams_that_end_and_pages_that_come_back(example):
    """An end token that is always likely: beams finish and keep their places; counts stay those of the tables."""
    search = small(example, requests=2, width=3)
    search.begin(prompts(search, [40, 31], seed=3))
    search.model.head[1][search.end_token] *= 0
    for _ in range(10):
        search.step()
        assert search.refcount.tolist() == counts(search.table, search.refcount.shape[0])
    torch.cuda.synchronize()
    assert bool(torch.isfinite(search.scores).all()) and example.w.w4a16_last_device_error() == 0


def test_captured_steps(example):
    """A captured step, replayed, finds what eager steps find."""
    found = []
    for captured in (False, True):
        search = small(example, seed=5)
        search.begin(prompts(search, [50, 90, 33], seed=4))
        steps = [tuple(t.clone() for t in search.step()) for _ in range(2)]
        torch.cuda.synchronize()
        if captured:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                out = search.step()
        for _ in range(12):
            if captured:
                graph.replay()
            else:
                out = search.step()
            steps.append(tuple(t.clone() for t in out))
        torch.cuda.synchronize()
        found.append((torch.stack([s for s, _ in steps]), torch.stack([t for _, t in steps]), search.scores, search.table,
                      search.refcount))
    assert all(torch.equal(a, b) for a, b in zip(*found))
    assert example.w.w4a16_last_device_error() == 0


def test_the_example_runs(example, capsys):
    example.main()
    assert "beams, a step" in capsys.readouterr().out
