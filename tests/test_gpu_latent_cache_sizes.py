"""Attention over pages and lengths near the ends of their ranges."""
import pytest
import torch

from test_gpu_latent_cache import ints
from test_gpu_operators import BF16, kda, normal  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("length", [2 ** 22, 3355444 + 129])
def test_one_page_of_millions_of_tokens(kda, length):  # noqa: F811
    """Offsets within a page above 31 bits: the same tokens in one page of 2.7 GB and in pages of 128."""
    page, small, step = 2 ** 22, 128, 2 ** 16
    one = torch.empty(1, kda.latent_cache_page_bytes(page), dtype=torch.uint8, device="cuda")
    many = torch.empty(page // small, kda.latent_cache_page_bytes(small), dtype=torch.uint8, device="cuda")
    zero, table = ints(0).view(1, 1), torch.arange(page // small, dtype=torch.int32, device="cuda").view(1, -1)
    g = torch.Generator(device="cuda").manual_seed(1)
    for at in range(0, length, step):
        rows = torch.randn(min(step, length - at), 576, generator=g, device="cuda").to(BF16)
        for cache, t, size in ((one, zero, page), (many, table, small)):
            kda.latent_cache_write(rows[:, :512], rows[:, 512:], cache, t, ints(at + rows.shape[0]), page_size=size)
    q = normal(2, 1, 16, 576, dtype=BF16).cuda()
    ws = torch.empty(kda.latent_decode_workspace_bytes(1, 1, 16, 512, 64, BF16, page, 1, quantized=True), dtype=torch.uint8, device="cuda")
    a = kda.latent_decode(q, one, zero, ints(length), scale=0.02, page_size=page, workspace=ws)
    assert kda.latent_status(ws) == kda.KDA_OK
    b = kda.latent_decode(q, many, table, ints(length), scale=0.02, page_size=small)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and torch.isfinite(a[0].float()).all()
    x, r = kda.latent_cache_read(one, zero, ints(length), total_tokens=300, page_size=page)
    y, w = kda.latent_cache_read(many, table, ints(length), total_tokens=300, page_size=small)
    assert torch.equal(x, y) and torch.equal(r, w) and torch.equal(r, rows[-300:, 512:])
