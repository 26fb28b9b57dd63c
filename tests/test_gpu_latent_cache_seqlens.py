"""Writing and reading the quantised cache with cu_seqlens that are none: the rows of the
sequences concerned are left out, those of the others are as ever."""
import pytest
import torch

from test_gpu_latent_cache import ints, latents, tables
from test_gpu_operators import BF16, F32, kda  # noqa: F401

pytestmark = pytest.mark.gpu

MOST = 2 ** 31 - 1


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("status", [False, True])
@pytest.mark.parametrize("cu,left", [
    ([1, 40, 100, 102], range(40, 102)), ([-1, 40, 100, 102], range(40, 102)), ([0, 40, 100, 103], range(100)),
    ([0, -5, 100, 102], [100, 101]), ([0, MOST, 100, 102], [100, 101]), ([0, 40, MOST, MOST], range(40)), ([0, 40, 100, -1], range(100)),
    ([-2 ** 31, 40, 100, 102], range(40, 102)), ([0, 40, 39, 102], range(39))])
def test_rows_of_malformed_sequences_are_left_out(kda, dtype, status, cu, left):  # noqa: F811
    lens, page, left = [100, 90, 80], 16, list(left)
    table, pages = tables(lens, page, 3)
    table = table.cuda()
    size = kda.latent_cache_page_bytes(page)
    rows = latents(4, 102, 576, dtype=dtype).cuda()
    ws = torch.full((256,), 9, dtype=torch.uint8, device="cuda") if status else None

    def both(q):
        cache = torch.zeros(pages, size, dtype=torch.uint8, device="cuda")
        kda.latent_cache_write(rows[:, :512], rows[:, 512:], cache, table, ints(*lens), q, page_size=page, workspace=ws)
        return cache, (kda.latent_status(ws) if status else None)

    def back(cache, q):
        x, y = (torch.full((102, w), 7.0, dtype=dtype, device="cuda") for w in (512, 64))
        kda.latent_cache_read(cache, table, ints(*lens), q, total_tokens=102, page_size=page, latents=x, rope=y, workspace=ws)
        return torch.cat([x, y], 1), (kda.latent_status(ws) if status else None)
    good = ints(0, 40, 100, 102)
    full, rc = both(good)
    assert rc in (None, kda.KDA_OK)
    want = back(full, good)[0]
    cache, rc = both(ints(*cu))
    assert rc in (None, kda.KDA_ERR_BAD_SEQLENS)
    x, rc = back(full, ints(*cu))
    assert rc in (None, kda.KDA_ERR_BAD_SEQLENS)
    # Rows of the sequences whose bounds are right (and, with bounds that overlap, those that no other claims)
    claimed = set(left) | set(range(39, 102) if cu[2] == 39 else [])
    there = torch.zeros(102, dtype=torch.bool, device="cuda")
    there[left] = True
    assert torch.equal(x[there], want[there])
    for i in set(range(102)) - claimed:
        assert (x[i] == 7).all(), i
    if cu[2] == 39:
        return
    # In the cache, what the same rows alone write
    ends = [0, 40, 100, 102]
    only = torch.zeros_like(cache)
    for n in range(3):
        if ends[n] in left:
            part = rows[ends[n]:ends[n + 1]]
            kda.latent_cache_write(part[:, :512], part[:, 512:], only, table[n:n + 1], ints(lens[n]), page_size=page)
    assert torch.equal(cache, only)
