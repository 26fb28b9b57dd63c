"""Attention over a quantised cache in memory that nothing has cleared: what lies in
places that were never written, codes, rotary channels and scale bytes, changes no
bit."""
import pytest
import torch

from test_gpu_latent_cache import cached, ints
from test_gpu_latent_cache_edges import FORMS
from test_gpu_operators import BF16, kda, normal  # noqa: F401

pytestmark = pytest.mark.gpu


def written(cache, table, lens, page):
    """Which bytes of the pages belong to cached tokens."""
    mask = torch.zeros(cache.shape, dtype=torch.bool)
    for n, length in enumerate(lens):
        for t in range(length):
            p, i = int(table[n, t // page]), t % page
            mask[p, i * 640:(i + 1) * 640] = True
            mask[p, page * 640 + i] = True
    return mask.cuda()


@pytest.mark.parametrize("dtype,simt", FORMS)
@pytest.mark.parametrize("lens,lq,h,page", [
    ([1, 2, 3, 4, 5, 6, 7, 8], 1, 16, 64), ([129, 130, 131, 0, 127], 3, 16, 16), ([9, 1030, 33], 4, 4, 8), ([61, 254], 2, 100, 128),
    ([701], 1, 32, 64), ([5001, 2, 2047, 3002], 1, 32, 64), ([6003], 3, 16, 32)])
def test_unwritten_places_change_no_bit(kda, dtype, simt, lens, lq, h, page):  # noqa: F811
    cache, table, _ = cached(kda, lens, page, 512, 64, 81)
    mask = written(cache, table.cpu(), lens, page)
    q = normal(82, len(lens), lq, h, 576, dtype=dtype).cuda()
    g = torch.Generator(device="cuda").manual_seed(83)
    ws = torch.empty(kda.latent_decode_workspace_bytes(len(lens), lq, h, 512, 64, dtype, page, table.shape[1], quantized=True),
                     dtype=torch.uint8, device="cuda")

    def go(other):
        o, l = kda.latent_decode(q, torch.where(mask, cache, other), table, ints(*lens), scale=0.07, page_size=page, workspace=ws,
                                 flags=kda.KDA_FLAG_CUDA_CORE_PREFILL if simt else 0)
        assert kda.latent_status(ws) == kda.KDA_OK
        return o, l
    out, lse = go(torch.zeros_like(cache))
    assert torch.isfinite(out.float()).all() and not torch.isnan(lse).any()
    others = [torch.full_like(cache, b) for b in (0xFF, 0xFE, 0x7F, 0x80)]
    others += [torch.randint(0, 256, cache.shape, generator=g, dtype=torch.uint8, device="cuda") for _ in range(3)]
    for other in others:
        o, l = go(other)
        assert torch.equal(o, out) and torch.equal(l, lse), int(other[0, 0])


@pytest.mark.parametrize("new", [1, 2, 3, 4, 5])
def test_a_cache_of_memory_that_held_something_else(kda, new):  # noqa: F811
    """Tokens written into pages full of 0xFF, as integers of -1 leave them, and read by the decode."""
    rows = normal(84, new, 576, dtype=BF16).cuda()
    q = normal(85, 1, 16, 576, dtype=BF16).cuda()
    got = []
    for fill in (0, 0xFF):
        cache = torch.full((2, kda.latent_cache_page_bytes(64)), fill, dtype=torch.uint8, device="cuda")
        kda.latent_cache_write(rows[:, :512], rows[:, 512:], cache, ints(1).view(1, 1), ints(new), page_size=64)
        got.append(kda.latent_decode(q, cache, ints(1).view(1, 1), ints(new), scale=0.07, page_size=64))
    assert torch.isfinite(got[0][0].float()).all() and torch.isfinite(got[0][1]).all()
    assert all(torch.equal(a, b) for a, b in zip(*got))


@pytest.mark.parametrize("dtype,simt", FORMS)
@pytest.mark.parametrize("lens,lq,h,page", [([1, 1, 64], 1, 16, 64), ([700, 2], 3, 32, 16), ([9000], 1, 100, 64)])
def test_a_cleared_cache_holds_tokens_of_zeros(kda, dtype, simt, lens, lq, h, page):  # noqa: F811
    """Pages of zeros, as batches are padded with: all scores are 0, so lse is the logarithm of the tokens seen."""
    _, table, _ = cached(kda, lens, page, 512, 64, 86)
    pages = sum(-(-n // page) for n in lens) + 2
    cache = torch.zeros(pages, kda.latent_cache_page_bytes(page), dtype=torch.uint8, device="cuda")
    q = normal(87, len(lens), lq, h, 576, dtype=dtype).cuda()
    out, lse = kda.latent_decode(q, cache, table, ints(*lens), scale=0.07, page_size=page, flags=kda.KDA_FLAG_CUDA_CORE_PREFILL if simt else 0)
    assert (out == 0).all()
    seen = torch.tensor([[max(0, n - lq + 1 + i) for i in range(lq)] for n in lens], dtype=torch.float64)
    # the exponent of a scale stands in the sum's logarithm: 2^-24 of 130 four times, and the sum's own additions
    assert float((lse.cpu().double() - seen.log()[:, :, None]).abs().nan_to_num().max()) < 4 * 2.0 ** -24 * 140 + 9000 * 2.0 ** -23
    assert torch.equal(torch.isinf(lse.cpu()), (seen == 0)[:, :, None].expand(lse.shape))
