"""Attention over pages and lengths near the ends of their ranges."""
import math

import pytest
import torch

import latent_cache_ref as cref
from operators_ref import ADD, F, HALF
from test_gpu_latent_cache import ints, latents
from test_gpu_operators import BF16, kda, normal, within  # noqa: F401

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


def repeated(kda, quantized):  # noqa: F811
    """A page of 64 tokens and its keys in 64 bits."""
    rows = latents(5, 64, 576, dtype=BF16)
    if not quantized:
        return rows.cuda()[None], rows.to(F)
    cache = torch.zeros(1, kda.latent_cache_page_bytes(64), dtype=torch.uint8, device="cuda")
    kda.latent_cache_write(rows[:, :512].cuda(), rows[:, 512:].cuda(), cache, ints(0).view(1, 1), ints(64), page_size=64)
    v, r = cref.values(cache.cpu(), 64, 512, 64)
    return cache, torch.cat([v[0], r[0]], 1)


@pytest.mark.parametrize("quantized", [True, False])
def test_the_longest_sequences(kda, quantized):  # noqa: F811
    """2^31 - 64 tokens, one page over and over, beside a short sequence: the weights are those of the page's 64 tokens,
    the sum is as many times theirs.  A thread block adds up 2^24 / 152 tiles one after another, a product of 128 tokens in
    eight steps at most."""
    cache, keys = repeated(kda, quantized)
    pages = 2 ** 25 - 1
    table = torch.zeros(2, pages, dtype=torch.int32, device="cuda")
    lens, h = ints(64 * pages, 64), 16
    q = normal(6, 2, h, 576, dtype=BF16, scale=0.2)
    q[1] = q[0]
    kw = dict(page_size=64) if quantized else {}
    size = kda.latent_decode_workspace_bytes(2, 1, h, 512, 64, BF16, 64, pages, quantized=quantized)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    out, lse = kda.latent_decode(q.cuda(), cache, table, lens, scale=0.07, workspace=ws, **kw)
    assert kda.latent_status(ws) == kda.KDA_OK
    tiles = 2 ** 24 // 152 + 1
    sums, products = tiles * 2.0 ** -24 + 152 * 2.0 ** -24, 8 * tiles * ADD
    for i, reps in ((0, pages), (1, 1)):
        for c in (0, 7, 15):
            s = (keys @ q[i, c].to(F)) * 0.07
            p = torch.softmax(s, 0)
            size = float((keys.abs() @ q[i, c].to(F).abs()).max()) * 0.07
            scores = 640 * ADD * size                                  # the scores' own additions
            rel = 2 * scores + 2.0 ** -8 + (sums + products if i == 0 else 0) + 2.0 ** -18
            bound = 1.1 * rel * (p @ keys[:, :512].abs()) + HALF[BF16] * (p @ keys[:, :512]).abs()
            within(out[i, c], p @ keys[:, :512], bound, (i, c))
            assert abs(float(lse[i, c]) - float(torch.logsumexp(s, 0)) - math.log(reps)) < 1.1 * (scores + (sums if i == 0 else 0)) + 1e-4


@pytest.mark.parametrize("quantized", [True, False])
def test_a_sequence_that_takes_a_thread_block_seconds(kda, quantized):  # noqa: F811
    """2^28 tokens, one page over and over, by 4096 query rows: a thread block has all tiles of a group (over the cache in
    16 bits half of them), and the queries of the short sequence behind them wait for seconds."""
    cache, _ = repeated(kda, quantized)
    kw = dict(page_size=64) if quantized else {}
    lq, h, pages = 32, 128, 2 ** 22
    table = torch.zeros(2, pages, dtype=torch.int32, device="cuda")
    q = normal(7, 2, lq, h, 576, dtype=BF16, scale=0.2).cuda()
    size = kda.latent_decode_workspace_bytes(2, lq, h, 512, 64, BF16, 64, pages, quantized=quantized)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    out, lse = kda.latent_decode(q, cache, table, ints(64 * pages, 64), scale=0.07, workspace=ws, **kw)
    assert kda.latent_status(ws) == kda.KDA_OK
    want, wl = kda.latent_decode(q[1:], cache, table[1:], ints(64), scale=0.07, **kw)
    assert torch.equal(out[1:], want) and torch.equal(lse[1:], wl) and torch.isfinite(out.float()).all() and torch.isfinite(lse).all()
