"""Attention over the quantised cache where tokens' scales lie very far apart: a weight
counts in its row's sum whatever its token's latents are."""
import pytest
import torch

import operators_ref as ref
from operators_ref import F, HALF
from test_gpu_latent_cache import ints
from test_gpu_latent_cache_edges import by_hand
from test_gpu_operators import BF16, kda, normal, within  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("simt", [False, True])
@pytest.mark.parametrize("n,h", [(200, 16), (3000, 32)])
@pytest.mark.parametrize("small,large", [(None, 0), (None, 30), (None, 60), (None, 100), (-90, 30), (-60, 60), (-20, 60)])
def test_weights_of_tokens_with_small_latents_count(kda, simt, n, h, small, large):  # noqa: F811
    """Half of the tokens have latents of about 2^small (None: zero), the others of 2^large.  The queries' latent channels
    are zero, so the rotary ones alone make the scores, both halves have a good part of every weight, and there is no
    rounding of queries.  The rest of the bound: the scale's exponent added to a score (2^-24 of both); on the tensor cores
    a weight's 2^-8.6, or 2^-26 of the largest product of weight and value for each token."""
    c = normal(1, n, 512).clamp(-3, 3) * 2.0 ** large
    c[::2] = 0 if small is None else c[::2] * 2.0 ** (small - large)
    r = normal(2, n, 64, dtype=BF16)
    cache, table, keys = by_hand(kda, c.to(BF16), r)
    q = normal(3, 1, 1, h, 576, dtype=BF16)
    q[..., :512] = 0
    out, lse = kda.latent_decode(q.cuda(), cache, table, ints(n), scale=0.07, page_size=64, flags=kda.KDA_FLAG_CUDA_CORE_PREFILL if simt else 0)
    for hh in (0, 7, h - 1):
        want, wl, weight, ds = ref.attend(q[0, 0, hh], keys, keys[:, :512], 0.07)
        bo, bl = ref.attention_bounds(want, wl, weight, ds, n, BF16, False)
        if not simt:
            more = 4 * 2.0 ** -24 * (130 + abs(wl))
            p = torch.exp((keys @ q[0, 0, hh].to(F)) * 0.07 - wl)
            floor = n * 2.0 ** -26 * float((p * keys[:, :512].abs().amax(1)).max()) * 2
            bo, bl = bo + (2 * more + 2.0 ** -8.6) * weight * (1 + HALF[BF16]) + floor, bl + more
        within(out[0, 0, hh], want, bo, ("out", hh))
        within(lse[0, 0, hh], torch.tensor(wl), bl, ("lse", hh))
