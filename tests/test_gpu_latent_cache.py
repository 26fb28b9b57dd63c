"""The quantised cache of latents on the GPU: writing and reading back bit for bit
against a plain form, attention over it within bounds that count the roundings."""
import math

import pytest
import torch

import latent_cache_ref as cref
import operators_ref as ref
from operators_ref import F
from test_gpu_operators import BF16, F32, kda, normal, within  # noqa: F401

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")


def ints(*l):
    return torch.tensor(l, dtype=torch.int32, device="cuda")


def tables(lens, page, seed, spare=2):
    """A page table with pages in a shuffled order (and what is never read behind a length), and the pages there are."""
    need = [-(-n // page) for n in lens]
    total, cols = sum(need) + spare, max(1, max(need, default=1))
    order = torch.randperm(total, generator=torch.Generator().manual_seed(seed)).tolist()
    table = torch.full((len(lens), cols), 12345678, dtype=torch.int32)
    for n, p in enumerate(need):
        table[n, :p] = torch.tensor([order.pop() for _ in range(p)], dtype=torch.int32)
    return table, total


def latents(seed, *shape, dtype):
    """Tokens and channels of different size."""
    c = normal(seed, *shape) * torch.exp(normal(seed + 1, shape[-1], scale=0.7)) * torch.exp(normal(seed + 2, *shape[:-1], 1, scale=2.0))
    return c.to(dtype)


def place(table, page, n, t):
    return int(table[n, t // page]), t % page


# ------------------------------------------------------------------ writing and reading
def check_write(kda, lens, new, page, dtype, rank=512, rope=64, seed=0, packed=True, pad=0, lead=0, stride=0):  # noqa: F811
    """Writes `new` tokens of each sequence; every byte of the cache against the plain form, then reads them back."""
    table, pages = tables(lens, page, seed)
    size = kda.latent_cache_page_bytes(page, rank, rope)
    assert size == cref.page_bytes(page, rank, rope)
    pool = torch.randint(0, 256, (pages, size + stride), generator=torch.Generator().manual_seed(seed), dtype=torch.uint8)
    want = pool.clone()
    t = sum(new)
    rows = latents(seed + 3, t + pad, lead + rank + rope, dtype=dtype)
    c, r = rows[:, lead:lead + rank], rows[:, lead + rank:]
    v, e = cref.quantise(c)
    codes, rot, scales = cref.views(want[:, :size], page, rank, rope)
    at, cu = 0, [0]
    for n, k in enumerate(new):
        for i in range(k):
            p = lens[n] - k + i
            if p >= 0:
                w = place(table, page, n, p)
                codes[w], scales[w] = v[at].float().to(cref.E4M3), int(e[at]) + 127
                if rope:
                    rot[w] = r[at].to(BF16)
            at += 1
        cu.append(at)
    dev = pool.cuda()
    d = rows.cuda()
    ws = torch.full((256,), 9, dtype=torch.uint8, device="cuda")
    args = (dev[:, :size], table.cuda(), ints(*lens), ints(*cu) if packed else None)
    kda.latent_cache_write(d[:, lead:lead + rank], d[:, lead + rank:] if rope else None, *args, page_size=page, workspace=ws)
    assert kda.latent_status(ws) == kda.KDA_OK
    got = dev.cpu()
    if not torch.equal(got, want):
        off = (got != want).nonzero()
        raise AssertionError((len(off), off[:5].tolist(), got[got != want][:5], want[got != want][:5]))
    # back, in both types, beside whatever was there
    for dt in (BF16, F32):
        wide = torch.full((t + pad, rank + rope + 8), 5.0, dtype=dt, device="cuda")
        x, y = kda.latent_cache_read(*args, total_tokens=t + pad, page_size=page, rank=rank, d_rope=rope,
                                     latents=wide[:, :rank], rope=wide[:, rank:rank + rope] if rope else None, workspace=ws)
        assert kda.latent_status(ws) == kda.KDA_OK
        there = torch.zeros(t + pad, dtype=torch.bool)
        at = 0
        for n, k in enumerate(new):
            there[at:at + k] = torch.arange(lens[n] - k, lens[n]) >= 0
            at += k
        full = torch.full((t + pad, rank), 5.0, dtype=F)
        full[there] = (v * torch.exp2(e.to(F))[:, None])[there]
        assert torch.equal(x.cpu().to(F), full)
        if rope:
            fr = torch.full((t + pad, rope), 5.0, dtype=F)
            fr[there] = r.to(BF16).to(F)[there]
            assert torch.equal(y.cpu().to(F), fr)
        assert (wide[:, rank + rope:] == 5).all()
    return dev, table, args


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("lens,new,page", [
    ([1], [1], 64), ([700], [700], 16), ([5, 64, 65, 128], [5, 64, 65, 128], 64), ([300, 17, 0, 90], [3, 17, 0, 1], 16),
    ([1000, 33, 8], [600, 1, 8], 128), ([40] * 70, [2] * 70, 32), ([0, 0, 3], [0, 0, 3], 8), ([7, 9], [7, 9], 1), ([100, 99], [50, 99], 5)])
def test_write_and_read(kda, dtype, lens, new, page):  # noqa: F811
    check_write(kda, lens, new, page, dtype)


@pytest.mark.parametrize("lens,each,page", [([1, 2, 300, 64], 1, 64), ([90] * 40, 3, 16), ([5000], 4900, 64), ([0, 3, 1], 2, 32)])
def test_write_without_cu_seqlens(kda, lens, each, page):  # noqa: F811
    """As many tokens for each; those of sequences padded into a batch (length 0) and of places below 0 are left out."""
    check_write(kda, lens, [each] * len(lens), page, BF16, packed=False)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rank,rope,lead,stride,pad", [(512, 64, 0, 0, 3), (512, 64, 1, 16, 0), (256, 0, 0, 0, 0), (16, 8, 3, 128, 1),
                                                       (496, 128, 0, 0, 0), (128, 40, 8, 0, 70), (512, 0, 4, 0, 0)])
def test_write_other_sizes_strides_and_padding(kda, dtype, rank, rope, lead, stride, pad):  # noqa: F811
    check_write(kda, [130, 0, 77, 20], [100, 0, 77, 1], 32, dtype, rank, rope, lead=lead, stride=stride, pad=pad)
    check_write(kda, [4000, 2000], [3900, 2000], 64, dtype, rank, rope, lead=lead, stride=stride, pad=pad)


def test_write_many_sequences(kda):  # noqa: F811
    """More than one look of 32 for a token's sequence, empty ones between."""
    new = [n % 4 for n in range(1100)]
    check_write(kda, [k + n % 50 for n, k in enumerate(new)], new, 16, BF16)
    new = [0] * 40 + [5000] + [0] * 1030 + [900, 0, 1]
    check_write(kda, [k + 3 for k in new], new, 64, BF16)


def test_write_extremes(kda):  # noqa: F811
    """Zero rows, the borders of the scale's steps, the smallest and largest numbers, infinities and NaN."""
    c = torch.zeros(16, 512, dtype=F32)
    c[1] = 448
    c[2] = 448 * (1 + 2.0 ** -20)
    c[3] = 2.0 ** -140
    c[4], c[4, 7] = 1.0, 3e38
    c[5], c[5, 0] = 0.001, 448 * 2.0 ** -100
    c[6] = 449 * 2.0 ** -101
    c[7], c[7, 3], c[7, 4], c[7, 5] = 3.0, NAN, INF, -INF
    c[8], c[8, 1] = NAN, -2.5
    c[9] = INF
    c[10] = torch.linspace(-448, 448, 512)
    c[11] = torch.exp2(torch.linspace(-30, 8, 512))
    c[12] = 464.0                                                       # a tie of 448 and 480 under the scale below
    c[13], c[13, 0] = 17.0, 224.0                                       # ties between codes
    c[14, 0] = -1.0
    c[15] = -448 * 2.0 ** 3
    pages = torch.zeros(2, kda.latent_cache_page_bytes(16), dtype=torch.uint8, device="cuda")
    kda.latent_cache_write(c.cuda(), normal(1, 16, 64).cuda(), pages, ints(1).view(1, 1), ints(16), page_size=16)
    codes, _, scales = cref.views(pages[1:].cpu(), 16, 512, 64)
    v, e = cref.quantise(c)
    assert torch.equal(scales[0].long() - 127, e)
    got = codes[0].to(F)
    assert torch.equal(torch.isnan(got), ~torch.isfinite(c)) and torch.equal(torch.nan_to_num(got), torch.nan_to_num(v))
    assert (pages[0] == 0).all()


def test_write_reports_and_leaves_out_what_is_wrong(kda):  # noqa: F811
    lens, new, page = [100, 60, 30], [40, 60, 2], 16
    table, pages = tables(lens, page, 3)
    size = kda.latent_cache_page_bytes(page)
    rows = latents(4, sum(new), 576, dtype=BF16).cuda()
    ws = torch.full((256,), 9, dtype=torch.uint8, device="cuda")
    cu = ints(0, 40, 100, 102)

    def both(l, t, q, rows_=rows):
        cache = torch.zeros(pages, size, dtype=torch.uint8, device="cuda")
        kda.latent_cache_write(rows_[:, :512], rows_[:, 512:], cache, t.cuda(), ints(*l), q, page_size=page, workspace=ws)
        rc = kda.latent_status(ws)
        x, y = kda.latent_cache_read(cache, t.cuda(), ints(*l), q, total_tokens=rows_.shape[0], page_size=page, workspace=ws,
                                     latents=torch.zeros(rows_.shape[0], 512, dtype=BF16, device="cuda"))
        assert kda.latent_status(ws) == rc
        return rc, cache, x
    rc, good, back = both(lens, table, cu)
    assert rc == kda.KDA_OK
    for bad in (-1, pages, 2 ** 31 - 1, -2 ** 31):
        t = table.clone()
        t[0, 5] = bad                                                    # tokens 80 .. 95 of the first
        rc, cache, x = both(lens, t, cu)
        assert rc == kda.KDA_ERR_BAD_PAGE and torch.equal(x[40:], back[40:]) and torch.equal(x[:20], back[:20])
        assert (x[20:36] == 0).all() and (cache[int(table[0, 5])] == 0).all()
        t = table.clone()
        t[0, 0] = bad                                                    # not of the new tokens
        assert both(lens, t, cu)[0] == kda.KDA_OK
    for length in (-1, table.shape[1] * page + 1, 2 ** 31 - 1, -2 ** 31):
        rc, cache, x = both([100, length, 30], table, cu)
        assert rc == kda.KDA_ERR_BAD_SEQLENS and (x[40:100] == 0).all()
        assert torch.equal(x[:40], back[:40]) and torch.equal(x[100:], back[100:])
    for q in (ints(1, 40, 100, 102), ints(0, 50, 40, 102), ints(0, 40, 100, 103), ints(0, -5, 100, 102), ints(0, 2 ** 31 - 1, 100, 102)):
        assert both(lens, table, q)[0] == kda.KDA_ERR_BAD_SEQLENS
    rc, _, x = both(lens, table, ints(0, 40, 100, 100))                  # two rows behind the last sequence
    assert rc == kda.KDA_OK and torch.equal(x[:100], back[:100]) and (x[100:] == 0).all()
    # nothing to write: a status all the same
    assert both(lens, table, ints(0, 0, 0, 0), rows[:0])[0] == kda.KDA_OK
    assert both(lens, table, ints(0, 0, 1, 0), rows[:0])[0] == kda.KDA_ERR_BAD_SEQLENS
    assert both([], table[:0], ints(0), rows)[0] == kda.KDA_OK


def test_cache_at_the_end_of_a_large_pool(kda):  # noqa: F811
    """Offsets above 32 bits."""
    page = 64
    size = kda.latent_cache_page_bytes(page)
    pool = torch.empty(130_000, size, dtype=torch.uint8, device="cuda")                # 5.3 GB
    table = ints(*range(130_000 - 5, 130_000)).view(1, 5)
    small = torch.empty(5, size, dtype=torch.uint8, device="cuda")
    rows = latents(5, 300, 576, dtype=BF16).cuda()
    q = normal(6, 1, 1, 16, 576, dtype=BF16).cuda()
    for c, t in ((pool, table), (small, ints(*range(5)).view(1, 5))):
        kda.latent_cache_write(rows[:, :512], rows[:, 512:], c, t, ints(300), page_size=page)
    assert torch.equal(pool[-5:-1, :page * 640], small[:-1, :page * 640])               # (four whole pages)
    for flags in (0, kda.KDA_FLAG_CUDA_CORE_PREFILL):
        a, b = (kda.latent_decode(q, c, t, ints(300), scale=0.07, page_size=page, flags=flags)
                for c, t in ((pool, table), (small, ints(*range(5)).view(1, 5))))
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    x, y = kda.latent_cache_read(pool, table, ints(300), total_tokens=300, page_size=page)
    z, w = kda.latent_cache_read(small, ints(*range(5)).view(1, 5), ints(300), total_tokens=300, page_size=page)
    assert torch.equal(x, z) and torch.equal(y, w)


# ------------------------------------------------------------------ attention
def cached(kda, lens, page, rank, rope, seed, stride=0, nan=True):  # noqa: F811
    """(cache, table, [keys of each sequence in 64 bits]); NaN codes and infinities behind the lengths and in spare pages."""
    table, pages = tables(lens, page, seed)
    size = kda.latent_cache_page_bytes(page, rank, rope)
    pool = torch.full((pages, size + stride), 0x7F, dtype=torch.uint8)
    cache = pool[:, :size]
    codes, rot, scales = cref.views(cache, page, rank, rope)
    seqs = []
    for n, length in enumerate(lens):
        c = latents(seed + 10 * n + 1, length, rank, dtype=F32)
        c = c / c.abs().amax(-1, keepdim=True).clamp_min(1e-30) * torch.exp(normal(seed + n, length, 1, scale=0.8)) * 4
        v, e = cref.quantise(c) if length else (torch.zeros(0, rank, dtype=F), torch.zeros(0, dtype=torch.long))
        r = normal(seed + 10 * n + 5, length, rope, dtype=BF16)
        where = [place(table, page, n, t) for t in range(length)]
        if length:
            i, j = torch.tensor(where).T
            codes[i, j] = v.float().to(cref.E4M3)
            scales[i, j] = (e + 127).to(torch.uint8)
            if rope:
                rot[i, j] = r
        seqs.append(torch.cat([v * torch.exp2(e.to(F))[:, None], r.to(F)], 1))
    if not nan:
        cache[(torch.arange(pages)[:, None] < 0).expand_as(cache)] = 0
    return pool.cuda()[:, :size], table.cuda(), seqs


def check_decode(kda, lens, lq, h, page, rank=512, rope=64, dtype=BF16, simt=False, seed=0, rows=None, stride=0, gain=1.0,  # noqa: F811
                 scale=192 ** -0.5, seqs_at=None, **kw):
    cache, table, seqs = cached(kda, lens, page, rank, rope, seed, stride)
    q = normal(seed + 9, len(lens), lq, h, rank + rope, dtype=dtype, scale=gain)
    ws = torch.empty(kda.latent_decode_workspace_bytes(len(lens), lq, h, rank, rope, dtype, page, table.shape[1], quantized=True),
                     dtype=torch.uint8, device="cuda")
    out, lse = kda.latent_decode(q.cuda(), cache, table, ints(*lens), scale=scale, rank=rank, page_size=page, workspace=ws,
                                 flags=kda.KDA_FLAG_CUDA_CORE_PREFILL if simt else 0, **kw)
    assert kda.latent_status(ws) == kda.KDA_OK
    tensor = dtype == BF16 and not simt
    compare(q, seqs, out, lse, lens, lq, h, rank, scale, dtype, tensor, rows, seqs_at)
    return out, lse


def compare(q, seqs, out, lse, lens, lq, h, rank, scale, dtype, tensor, rows=None, seqs_at=None):
    o, l = out.cpu(), lse.cpu()
    for n, k in enumerate(seqs):
        if seqs_at is not None and n not in seqs_at:
            continue
        for i in range(lq):
            end = max(0, lens[n] - lq + i + 1)
            for hh in range(h) if rows is None else [r for r in rows if r < h]:
                want, wl, weight, ds = ref.attend(q[n, i, hh], k[:end], k[:end, :rank], scale)
                bo, bl = cref.attention_bounds(q[n, i, hh], k[:end], rank, want, wl, weight, ds, scale, dtype, tensor)
                within(o[n, i, hh], want, bo, ("out", n, i, hh))
                within(l[n, i, hh], torch.tensor(wl), bl, ("lse", n, i, hh))


HEADS = [0, 1, 7, 15, 16, 31, 32, 33, 63, 64, 127]


@pytest.mark.parametrize("simt", [False, True])
@pytest.mark.parametrize("lens,lq,h,page", [
    ([1], 1, 16, 64), ([0, 1, 2, 700], 1, 32, 64), ([127, 128, 129], 1, 16, 16), ([300, 5, 64], 3, 16, 32), ([2, 0, 1, 4], 4, 8, 16),
    ([513, 90], 1, 128, 128), ([200], 2, 20, 64), ([1000, 33], 4, 64, 16), ([600], 1, 1, 8), ([700, 800], 1, 33, 256)])
def test_decode(kda, simt, lens, lq, h, page):  # noqa: F811
    check_decode(kda, lens, lq, h, page, simt=simt, rows=HEADS)


@pytest.mark.parametrize("rank,rope,dtype,page", [(512, 64, F32, 64), (512, 64, BF16, 48), (256, 32, BF16, 64), (112, 8, F32, 5), (512, 0, BF16, 1),
                                                  (512, 64, BF16, 4)])
def test_decode_other_sizes_types_and_pages(kda, rank, rope, dtype, page):  # noqa: F811
    check_decode(kda, [130, 0, 77], 2, 3, page, rank, rope, dtype, simt=True)
    # these run on CUDA cores whatever the flags
    check_decode(kda, [130, 0, 77], 2, 3, page, rank, rope, dtype, simt=False)


@pytest.mark.parametrize("lens,lq,h", [([9000], 1, 16), ([5000, 17, 0, 3001], 2, 32), ([40] * 300, 1, 16), ([0] * 5, 1, 16)])
def test_decode_split_over_the_cache(kda, lens, lq, h):  # noqa: F811
    check_decode(kda, lens, lq, h, 64, rows=[0, 9, h - 1], seqs_at={0, 1, 2, 3, 299})


def test_decode_large_scores(kda):  # noqa: F811
    check_decode(kda, [400, 1500], 1, 32, 64, gain=25.0, rows=[0, 5, 31])


@pytest.mark.parametrize("simt", [False, True])
def test_decode_layouts(kda, simt):  # noqa: F811
    """Pages apart in a larger pool, one query given without its dimension, strided query heads."""
    lens, h, kw = [300, 61], 16, dict(page_size=32, scale=0.07, flags=kda.KDA_FLAG_CUDA_CORE_PREFILL if simt else 0)
    check_decode(kda, lens, 1, h, 32, stride=48, simt=simt)
    cache, table, _ = cached(kda, lens, 32, 512, 64, 3)
    q = normal(4, 2, 1, h, 576, dtype=BF16).cuda()
    o, l = kda.latent_decode(q, cache, table, ints(*lens), **kw)
    o1, l1 = kda.latent_decode(q[:, 0], cache, table, ints(*lens), **kw)
    assert o1.shape == (2, h, 512) and torch.equal(o[:, 0], o1) and torch.equal(l[:, 0], l1)
    wide = torch.zeros(2, h, 640, dtype=BF16, device="cuda")
    for lo in (0, 64, 3):
        wide[..., lo:lo + 576] = q[:, 0]
        o2, l2 = kda.latent_decode(wide[..., lo:lo + 576], cache, table, ints(*lens), **kw)
        assert torch.allclose(o2.float(), o1.float(), rtol=2.0 ** -6, atol=2.0 ** -6)
        if lo != 3 or simt:
            assert torch.equal(o2, o1) and torch.equal(l2, l1)


@pytest.mark.parametrize("simt", [False, True])
def test_decode_over_written_tokens(kda, simt):  # noqa: F811
    """Written token by token and all at once: the same bytes, and attention over them is that over what is read back."""
    page, h, rank = 32, 16, 512
    rows = latents(7, 150, 576, dtype=BF16).cuda()
    table, pages = tables([100, 50], page, 8)
    table = table.cuda()
    whole, steps = (torch.zeros(pages, kda.latent_cache_page_bytes(page), dtype=torch.uint8, device="cuda") for _ in range(2))
    cu, lens = ints(0, 100, 150), ints(100, 50)
    kda.latent_cache_write(rows[:, :512], rows[:, 512:], whole, table, lens, cu, page_size=page)
    for t in range(100):
        now = torch.stack([rows[t], rows[100 + min(t, 49)]])
        kda.latent_cache_write(now[:, :512], now[:, 512:], steps, table, ints(t + 1, min(t, 49) + 1), page_size=page)
    assert torch.equal(whole, steps)
    x, r = kda.latent_cache_read(whole, table, lens, cu, total_tokens=150, page_size=page, dtype=F32)
    q = normal(9, 2, 1, h, 576, dtype=BF16)
    out, lse = kda.latent_decode(q.cuda(), whole, table, lens, scale=0.07, page_size=page, flags=kda.KDA_FLAG_CUDA_CORE_PREFILL if simt else 0)
    keys = torch.cat([x, r], 1).cpu().to(F)
    compare(q, [keys[:100], keys[100:]], out, lse, [100, 50], 1, h, rank, 0.07, BF16, not simt)


@pytest.mark.parametrize("simt", [False, True])
def test_decode_reports_bad_pages_and_lengths(kda, simt):  # noqa: F811
    cache, table, _ = cached(kda, [300, 200], 64, 512, 64, 3)
    q = normal(4, 2, 1, 16, 576, dtype=BF16).cuda()
    ws = torch.empty(kda.latent_decode_workspace_bytes(2, 1, 16, 512, 64, BF16, 64, table.shape[1], quantized=True), dtype=torch.uint8, device="cuda")

    def call(lens, t):
        o, _ = kda.latent_decode(q, cache, t, ints(*lens), scale=0.07, page_size=64, workspace=ws, flags=kda.KDA_FLAG_CUDA_CORE_PREFILL if simt else 0)
        return o, kda.latent_status(ws)
    good, rc = call([300, 200], table)
    assert rc == kda.KDA_OK
    for page in (-1, cache.shape[0], 2 ** 31 - 1, -2 ** 31):
        bad = table.clone()
        bad[0, 2] = page
        o, rc = call([300, 200], bad)
        assert rc == kda.KDA_ERR_BAD_PAGE and torch.equal(o[1], good[1])
        assert call([128, 200], bad)[1] == kda.KDA_OK          # behind the length: not read
    for length in (-1, table.shape[1] * 64 + 1, 2 ** 31 - 1):
        o, rc = call([length, 200], table)
        assert rc == kda.KDA_ERR_BAD_SEQLENS and torch.equal(o[1], good[1])


# ------------------------------------------------------------------ refusals
def test_cache_refusals(kda):  # noqa: F811
    size = kda.latent_cache_page_bytes(64)
    cache, table, lens = torch.zeros(4, size, dtype=torch.uint8, device="cuda"), ints(0, 1).view(1, 2), ints(100)
    x, r, q = normal(1, 3, 512, dtype=BF16).cuda(), normal(2, 3, 64, dtype=BF16).cuda(), normal(3, 1, 4, 576, dtype=BF16).cuda()
    w = lambda **k: kda.latent_cache_write(*[k.pop(n, v) for n, v in dict(x=x, r=r, c=cache, t=table, l=lens).items()], **{"page_size": 64, **k})  # noqa: E731
    g = lambda **k: kda.latent_cache_read(*[k.pop(n, v) for n, v in dict(c=cache, t=table, l=lens).items()],  # noqa: E731
                                          **{"page_size": 64, "total_tokens": 3, **k})
    d = lambda **k: kda.latent_decode(*[k.pop(n, v) for n, v in dict(q=q, c=cache, t=table, l=lens).items()], scale=0.1, **{"page_size": 64, **k})  # noqa: E731
    w(), g(), d()
    bad_cache = [cache[:, :-1], cache.view(torch.int8), cache.cpu(), cache[0], cache.t()]
    for c in bad_cache:
        for call in (w, g):
            with pytest.raises(ValueError):
                call(c=c)
    for c in (cache[:, :-1], cache.view(torch.int8), cache[0]):
        with pytest.raises(ValueError):
            d(c=c)
    for call in (w, g, d):
        for k in (dict(page_size=63), dict(page_size=0), dict(page_size=None), dict(t=table[0]), dict(t=table.long()), dict(l=lens.long()),
                  dict(l=ints(1, 2)), dict(page_size=2 ** 40), dict(workspace=torch.zeros(256, dtype=torch.uint8))):
            with pytest.raises(ValueError):
                call(**k)
    for k in (dict(x=x.half()), dict(r=r[:2]), dict(r=r.float()), dict(r=None), dict(x=x[:, :500]), dict(x=x[:, ::2]), dict(cu_seqlens=ints(0, 1, 3)),
              dict(t=ints(0, 1).view(2, 1), l=ints(1, 2))):
        with pytest.raises(ValueError):
            w(**k)
    for k in (dict(rank=500), dict(rank=256), dict(d_rope=0), dict(dtype=torch.float16), dict(total_tokens=-1), dict(latents=x[:2]),
              dict(rope=r.float(), latents=x), dict(latents=x[:, :256])):
        with pytest.raises(ValueError):
            g(**k)
    for k in (dict(rank=500), dict(flags=kda.KDA_FLAG_CACHE_8, c=torch.zeros(2, 64, 576, dtype=BF16, device="cuda"))):
        with pytest.raises(ValueError):
            d(**k)
    for bad in (dict(workspace=torch.zeros(8, dtype=torch.uint8, device="cuda")), dict(workspace=torch.zeros(520, dtype=torch.uint8, device="cuda")[8:])):
        for call in (w, g, d):
            with pytest.raises(kda.KdaError):
                call(**bad)
    with pytest.raises(kda.KdaError):
        w(x=x[:1].expand(3, 512))
    with pytest.raises(kda.KdaError):                                      # pages off 16 bytes
        w(c=torch.zeros(4 * size + 8, dtype=torch.uint8, device="cuda")[8:].view(4, size))
    with pytest.raises(ValueError):
        kda.latent_cache_page_bytes(64, 500, 64)
