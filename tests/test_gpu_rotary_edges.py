"""Rotary positions where a call is unusual: frequencies that are no numbers, and queries
and keys that lie side by side within each head."""
import pytest
import torch

from test_gpu_operators import BF16, F32, kda, normal  # noqa: F401
from test_gpu_rotary import check, places

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


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("t,h,a,b,gap,outside", [(50, 4, 64, 64, 0, False), (7, 3, 96, 64, 8, False), (1, 5, 64, 70, 2, False),
                                                 (40, 4, 64, 64, 0, True), (33, 1, 64, 128, 4, True), (9, 6, 66, 64, 6, True)])
def test_rotary_in_place_of_queries_and_keys_side_by_side_in_each_head(kda, dtype, interleaved, t, h, a, b, gap, outside):  # noqa: F811
    """[tokens, heads, (query | key)], or with the heads outermost: they are turned as apart from one another."""
    both = normal(3, *((h, t) if outside else (t, h)), a + b + gap, dtype=dtype).cuda()
    view = both.transpose(0, 1) if outside else both
    q, k = view[..., :a], view[..., a:a + b]
    f, pos = kda.rotary_frequencies(64), places(4, t, 40000)
    want = kda.rotary(q.contiguous(), pos, f, key=k.contiguous(), interleaved=interleaved, scale=1.2)
    rest = view[..., a + b:].clone()
    check(kda, q, pos, f, key=k, interleaved=interleaved, scale=1.2, out=q, key_out=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(view[..., a + b:], rest)


def test_rotary_of_rows_that_overlap_within_heads_is_refused(kda):  # noqa: F811
    both = normal(5, 50, 4, 136, dtype=BF16).cuda()
    f, pos = kda.rotary_frequencies(64), places(6, 50, 100)
    keep = both.clone()
    for q, k in ((both[..., :64], both[..., 63:127]), (both[..., :66], both[..., 64:128]), (both[..., 70:], both[:, :2, 8:72]),
                 (both.view(50, 2, 272)[..., :64], both[:, :3, 60:126]), (both[..., :64], both.view(100, 272)[:50, 10:74])):
        with pytest.raises(kda.KdaError):
            kda.rotary(q, pos, f, key=k, out=q, key_out=k)
    assert torch.equal(both, keep)
