"""Tokens appended one at a time to a page whose scale grows with nearly every one of them: what the repeated rounding adds up
to stays within the bound that the header states, at every page size."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("store", [torch.int8, torch.float8_e4m3fn])
@pytest.mark.parametrize("rate", [1.004, 1.03, 1.3])
def test_error_of_a_growing_page(cuda_lib, page, store, rate):
    w = cuda_lib
    g = torch.Generator().manual_seed(page)
    x = (torch.randn((page, 2, 64), generator=g) * 0.3).clamp(-1, 1)
    x[:, :, 0] = 1.0                                  # the largest of each token, a little larger every time
    x = (x * rate ** torch.arange(page)[:, None, None]).to(torch.bfloat16).cuda()
    k = torch.zeros((1, 2, page, 64), device="cuda").to(store)
    cache = w.KVCache(k, k.clone(), torch.zeros((1, 2), device="cuda"), torch.zeros((1, 2), device="cuda"))
    table = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    starts = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    scales = []
    for t in range(page):
        w.w4a16_kv_append(cache, x[t:t + 1], x[t:t + 1], table, torch.tensor([t + 1], dtype=torch.int32, device="cuda"), starts)
        scales.append(cache.k_scale[0].clone())
    s = torch.stack(scales).cpu().double()            # [token, head]
    grew = (s[1:] > s[:-1]).double().flip(0).cumsum(0).flip(0)
    grew = torch.cat([grew, torch.zeros_like(grew[:1])])          # how often after each token
    assert float(grew[0].max()) > page / 4
    got = cache.k[0].float().cpu().double() * s[-1][:, None, None]
    err = (got.transpose(0, 1) - x.cpu().double()).abs()
    # the fp32 products move a value by 2^-22 of the largest at most, far below 2^-10 of a spacing
    if store is torch.int8:
        bound = ((grew + 1) / 2 * s[-1])[..., None].expand_as(err)
    else:
        # relative for normal codes, half of 2^-9 s for subnormal ones
        bound = x.cpu().double().abs() * ((1 + 2.0 ** -4) ** (grew + 1) - 1)[..., None] + ((grew + 1) * 2.0 ** -10 * s[-1])[..., None]
    assert bool((err <= bound * (1 + 2.0 ** -10)).all())
    assert w.w4a16_last_device_error() == 0
