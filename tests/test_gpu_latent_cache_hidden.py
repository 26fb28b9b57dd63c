"""Attention over the quantised cache with several queries a sequence: a latent that is
no number reaches the queries that see its token, and no others."""
import pytest
import torch

import latent_cache_ref as cref
import operators_ref as ref
from test_gpu_latent_cache import cached, ints, place
from test_gpu_latent_cache_edges import FORMS
from test_gpu_operators import BF16, kda, normal, within  # noqa: F401

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("dtype,simt", FORMS)
@pytest.mark.parametrize("length,lq,h,page,tokens,channels", [
    (300, 3, 16, 64, [299], [0]), (300, 3, 16, 64, [298], [511]), (257, 4, 32, 16, [254, 256], [130, 300]), (129, 4, 8, 64, [126], [383]),
    (2, 4, 4, 64, [0, 1], [200]), (128, 2, 64, 128, [127], range(512)), (5000, 3, 16, 64, [4999], [7, 400]), (1, 2, 1, 8, [0], [128]),
    (131, 3, 2, 8, [128, 129, 130], [255]), (140, 16, 8, 32, list(range(125, 139, 2)), [64, 256])])
def test_latents_that_are_no_numbers_reach_the_queries_that_see_them(kda, dtype, simt, length, lq, h, page, tokens, channels):  # noqa: F811
    cache, table, seqs = cached(kda, [length, 70], page, 512, 64, 91)
    lens, q = [length, 70], normal(92, 2, lq, h, 576, dtype=dtype)
    codes = cref.views(cache, page, 512, 64)[0].view(torch.uint8)
    for k, t in enumerate(tokens):
        for c in channels:
            codes[(*place(table.cpu(), page, 0, t), c)] = 0xFF if (k + c) % 2 else 0x7F
    out, lse = kda.latent_decode(q.cuda(), cache, table, ints(*lens), scale=0.07, page_size=page,
                                 flags=kda.KDA_FLAG_CUDA_CORE_PREFILL if simt else 0)
    tensor = dtype == BF16 and not simt
    for n in range(2):
        for i in range(lq):
            end = max(0, lens[n] - lq + i + 1)
            if n == 0 and end > min(tokens):
                assert torch.isnan(out[n, i]).all() and torch.isnan(lse[n, i]).all(), i
                continue
            for hh in {0, h // 2, h - 1}:
                k = seqs[n][:end]
                want, wl, weight, ds = ref.attend(q[n, i, hh], k, k[:, :512], 0.07)
                bo, bl = cref.attention_bounds(q[n, i, hh], k, 512, want, wl, weight, ds, 0.07, dtype, tensor)
                within(out[n, i, hh], want, bo, ("out", n, i, hh))
                within(lse[n, i, hh], torch.tensor(wl), bl, ("lse", n, i, hh))


@pytest.mark.parametrize("value", [NAN, INF, -INF])
def test_a_drafted_token_that_is_no_number(kda, value):  # noqa: F811
    """Written by the package: of four tokens verified together the third has such a channel; the first two come out as
    they would without it."""
    rows = normal(93, 90, 576, dtype=BF16).cuda()
    q = normal(94, 1, 4, 16, 576, dtype=BF16).cuda()
    got = []
    for bad in (False, True):
        if bad:
            rows[88, 77] = value
        cache = torch.empty(2, kda.latent_cache_page_bytes(64), dtype=torch.uint8, device="cuda")
        kda.latent_cache_write(rows[:, :512], rows[:, 512:], cache, ints(0, 1).view(1, 2), ints(90), page_size=64)
        got.append(kda.latent_decode(q, cache, ints(0, 1).view(1, 2), ints(90), scale=0.07, page_size=64))
    (out, lse), (o, l) = got
    assert torch.equal(o[:, :2], out[:, :2]) and torch.equal(l[:, :2], lse[:, :2]) and torch.isfinite(out.float()).all()
    assert torch.isnan(o[:, 2:]).all() and torch.isnan(l[:, 2:]).all()
