"""Beam search's selection where one token has nearly all of a beam's probability, as a language model's rows often do:
how far the scores are off, and in what order beams come that are close to one another."""
import pytest
import torch

pytestmark = pytest.mark.gpu

ACT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
# Relative error of a sum, and so the error of its logarithm, where all but 2^-6 of it is one weight: 2^-22 from the
# exponential; two roundings of an exponent of at most 1/2, 2^-26 each, times ln 2; 10 additions in fp32 of a thread's 32
# logits in four sums, 2^-24 each; the others' weights, as far off as 2^-18 of themselves, 2^-24.  15.4 * 2^-24 together.
PEAKED = 2.0 ** -20


def rows_of(n, vocab, act, peak, seed):
    """Rows of spread 2.3 with one token some `peak` above the others."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((n, vocab), generator=g) * 2.3
    top = x.amax(1) + peak + 3 * torch.rand((n,), generator=g)
    x[torch.arange(n), torch.randint(0, vocab, (n,), generator=g)] = top
    return x.to(ACT[act])


def exact(x):
    """The largest log-probability of each row, in 64 bits."""
    d = x.double()
    return -torch.log(torch.exp(d - d.amax(1, keepdim=True)).sum(1))


def others(x):
    """Weight of all tokens but the largest, of the largest's."""
    return torch.expm1(-exact(x))


@pytest.mark.parametrize("act", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("vocab", [2, 30, 1000, 32000, 70001])
@pytest.mark.parametrize("peak", [15, 20, 30])
def test_error(cuda_lib, act, vocab, peak):
    """With a score that takes a row's log-probability to about 0, its rounding hides nothing."""
    x = rows_of(200, vocab, act, peak, vocab + peak)
    assert float(others(x).max()) < 2.0 ** -6
    want = exact(x)
    scores = (2.0 ** -10 - want).float()
    got = cuda_lib.w4a16_beam_select(x.cuda(), scores.cuda(), 1, 1)
    assert torch.equal(got[2].cpu()[:, 0].long(), x.float().argmax(1))
    off = got[0].cpu()[:, 0].double() - (want + scores.double())
    assert float(off.abs().max()) <= PEAKED + 2.0 ** -24 * 2.0 ** -9


@pytest.mark.parametrize("act", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("vocab, peak", [(1, 0), (2, 20), (30, 15), (30, 25), (32000, 25), (70001, 40)])
@pytest.mark.parametrize("score", [0.0, -7.25, 3.0e-5])
def test_no_better_than_the_beam(cuda_lib, act, vocab, peak, score):
    """A token's probability is 1 at most."""
    x = rows_of(400, vocab, act, peak, vocab + peak)
    scores = torch.full((400,), score)
    got = cuda_lib.w4a16_beam_select(x.cuda(), scores.cuda(), 1, 1)[0].cpu()[:, 0]
    assert bool((got <= scores).all())
    assert bool(((got.double() - exact(x) - scores.double()).abs() <= PEAKED + 2.0 ** -24 * abs(score)).all())


@pytest.mark.parametrize("act", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("vocab", [30, 32000])
@pytest.mark.parametrize("width", [4, 16])
def test_order_of_beams(cuda_lib, act, vocab, width):
    """Beams whose best continuations are 2.5 * 2^-20 apart, as their scores make them, come in that order."""
    groups = 40
    x = rows_of(groups * width, vocab, act, 20, vocab + width)
    g = torch.Generator().manual_seed(width)
    place = torch.stack([torch.randperm(width, generator=g) for _ in range(groups)]).flatten()
    scores = (-exact(x) - 2.5 * 2.0 ** -20 * place).float()             # around 0: rounded by less than 2^-38
    got = cuda_lib.w4a16_beam_select(x.cuda(), scores.cuda(), width, width)
    rows = torch.arange(groups).repeat_interleave(width) * width + 0
    want = torch.empty(groups * width, dtype=torch.int32)
    want[(rows + place).long()] = torch.arange(groups * width, dtype=torch.int32)
    assert torch.equal(got[1].cpu().flatten(), want)
    assert torch.equal(got[2].cpu().flatten().long(), x.float().argmax(1)[want.long()])
