"""Rotary positions where a call is unusual."""
import pytest
import torch

from test_gpu_operators import BF16, F32, kda, normal  # noqa: F401
from test_gpu_rotary import places

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("heads,width,dim", [(3, 80, 48), (2, 33, 18), (1, 1024, 1024)])
def test_frequencies_that_are_no_numbers_make_their_pairs_nan(kda, dtype, interleaved, heads, width, dim):  # noqa: F811
    x, f, pos = normal(1, 70, heads, width, dtype=dtype).cuda(), kda.rotary_frequencies(dim), places(2, 70, 5000)
    pos[3] = 0
    want = kda.rotary(x, pos, f, offset=1 if width > dim else 0, interleaved=interleaved)[0]
    bad = f.clone()
    at = [0, 5, dim // 2 - 1]
    bad[at[0]], bad[at[1]], bad[at[2]] = INF, NAN, -INF
    offset = 1 if width > dim else 0
    for inverse in (False, True):
        y = kda.rotary(x, pos, bad, offset=offset, interleaved=interleaved, inverse=inverse)[0]
        if inverse:
            want = kda.rotary(x, pos, f, offset=offset, interleaved=interleaved, inverse=True)[0]
        none = torch.zeros(width, dtype=torch.bool, device="cuda")
        for i in at:
            for c in ((2 * i, 2 * i + 1) if interleaved else (i, i + dim // 2)):
                none[offset + c] = True
        assert torch.isnan(y[..., none]).all() and torch.equal(y[..., ~none], want[..., ~none])
