"""Beam search's selection where a beam's probabilities are plain numbers: one token that may follow, or equal ones."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

ACT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


@pytest.mark.parametrize("act", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("vocab", [1, 2, 33, 9001, 70001])
@pytest.mark.parametrize("others", [-math.inf, -200.0])
def test_one_token(cuda_lib, act, vocab, others):
    """All the others are masked, or worth 0 in 32 bits: the beam's score is what it was."""
    g = torch.Generator().manual_seed(vocab)
    x = torch.full((120, vocab), others)
    token = torch.randint(0, vocab, (120,), generator=g)
    x[torch.arange(120), token] = torch.randn((120,), generator=g) * 20
    scores = -torch.rand((120,), generator=g) * 30
    got = cuda_lib.w4a16_beam_select(x.to(ACT[act]).cuda(), scores.cuda(), 1, 1)
    assert torch.equal(got[0].cpu()[:, 0], scores) and torch.equal(got[2].cpu()[:, 0].long(), token)


@pytest.mark.parametrize("act", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("vocab, n_out", [(2, 1), (4, 4), (100, 3), (1024, 1), (16384, 5), (60000, 64)])
def test_equal_tokens(cuda_lib, act, vocab, n_out):
    """The logarithm of their number, good to 2^-29.  A thread adds 2 of a vector's 8 weights a in each of four sums, then
    these: a + a, 2a + 2a, 4a + 4a are exact in fp32.  So is everything for a power of two of up to 2048 tokens, a vector a
    thread (or less).  Of more vectors the sums pass 3a, 5a, 6a and 7a, which may not be: 10 additions, 2^-24 each."""
    g = torch.Generator().manual_seed(vocab)
    x = (torch.randn((100, 1), generator=g) * 9).to(ACT[act]).expand(-1, vocab).contiguous()
    scores = torch.full((100,), math.log(vocab))
    got = cuda_lib.w4a16_beam_select(x.cuda(), scores.cuda(), 1, n_out)
    off = got[0].cpu().double() - (scores.double() - math.log(vocab))[:, None]
    assert float(off.abs().max()) <= (0 if vocab & (vocab - 1) == 0 and vocab <= 2048 else 10 * 2.0 ** -24) + 2.0 ** -29
    assert torch.equal(got[2].cpu(), torch.arange(n_out, dtype=torch.int32).expand(100, -1))


@pytest.mark.parametrize("act", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("first", ["ended", "certain"])
def test_beams_that_tie(cuda_lib, act, first):
    """A beam that has ended and one that can go on in one way only, with the same score: the lower one comes first."""
    g = torch.Generator().manual_seed(3)
    requests, vocab = 50, 5000
    x = torch.full((2 * requests, vocab), -math.inf)
    x[:, 77] = torch.randn((2 * requests,), generator=g) * 15
    finished = torch.tensor([first == "ended", first != "ended"] * requests)
    scores = (-torch.rand((requests, 1), generator=g) * 20).expand(-1, 2).flatten().contiguous()
    got = cuda_lib.w4a16_beam_select(x.to(ACT[act]).cuda(), scores.cuda(), 2, 2, finished=finished.cuda(), end_token=9)
    assert torch.equal(got[0].cpu().flatten(), scores)
    assert got[1].cpu().flatten().tolist() == list(range(2 * requests))
    assert got[2].cpu().tolist() == [[9, 77] if first == "ended" else [77, 9]] * requests
