"""Attention over the quantised cache, code by code: sequences of a single token,
whose weight is one, give back their values without any rounding."""
import pytest
import torch

import latent_cache_ref as cref
from test_gpu_latent_cache import ints
from test_gpu_operators import BF16, kda, normal  # noqa: F401
from test_gpu_latent_cache_edges import FORMS

pytestmark = pytest.mark.gpu


def one_token_each(kda, codes, exponents, page, g):  # noqa: F811
    """A cache of sequences of one token with these codes [n, 512] (bytes), each on a page of its own, and its table."""
    n = codes.shape[0]
    cache = torch.zeros(n, kda.latent_cache_page_bytes(page), dtype=torch.uint8, device="cuda")
    c, r, s = cref.views(cache, page, 512, 64)
    c.view(torch.uint8)[:, 0] = codes.cuda()
    r[:, 0] = normal(g, n, 64, dtype=BF16).cuda()
    s[:, 0] = (exponents + 127).to(torch.uint8).cuda()
    return cache, torch.arange(n, dtype=torch.int32, device="cuda")[:, None]


@pytest.mark.parametrize("dtype,simt", FORMS)
@pytest.mark.parametrize("page", [64, 6, 1])
def test_every_code_is_worth_its_value(kda, dtype, simt, page):  # noqa: F811
    g = torch.Generator().manual_seed(71)
    codes = torch.stack([(torch.arange(512) * 5 + n) % 256 for n in range(24)] + [torch.randint(0, 256, (512,), generator=g) for _ in range(8)])
    codes = torch.where((codes & 127) == 127, 0, codes).to(torch.uint8)
    e = torch.arange(32) - 16
    cache, table = one_token_each(kda, codes, e, page, 72)
    want = codes.view(cref.E4M3).float() * torch.exp2(e.float())[:, None]
    q = torch.zeros(32, 3, 576, dtype=dtype, device="cuda")
    out, lse = kda.latent_decode(q, cache, table, ints(*[1] * 32), scale=0.1, page_size=page,
                                 flags=kda.KDA_FLAG_CUDA_CORE_PREFILL if simt else 0)
    assert torch.equal(out.float().cpu(), want[:, None].expand(32, 3, 512))
    assert float(lse.abs().max()) < 1e-5


@pytest.mark.parametrize("dtype,simt", FORMS)
def test_a_code_that_is_nan_is_found_in_every_channel(kda, dtype, simt):  # noqa: F811
    g = torch.Generator().manual_seed(73)
    codes = torch.randint(0, 127, (513, 512), generator=g)
    codes += 128 * torch.randint(0, 2, codes.shape, generator=g)               # (126: the largest value, both signs)
    at = torch.arange(512)
    codes[at, at] = torch.where(at % 3 == 0, 255, 127)
    cache, table = one_token_each(kda, codes.to(torch.uint8), torch.zeros(513, dtype=torch.int64), 64, 74)
    q = normal(75, 513, 2, 576, dtype=dtype).cuda()
    out, lse = kda.latent_decode(q, cache, table, ints(*[1] * 513), scale=0.01, page_size=64,
                                 flags=kda.KDA_FLAG_CUDA_CORE_PREFILL if simt else 0)
    assert torch.isnan(out[:512]).all() and torch.isnan(lse[:512]).all()
    assert torch.isfinite(out[512]).all() and torch.isfinite(lse[512]).all()
