"""Norm, scaled 8-bit product and latent attention on the GPU against plain
forms in 64 bits, element by element within bounds that count the roundings
(tests/operators_ref.py)."""
import math

import pytest
import torch

import operators_ref as ref
from operators_ref import ADD, F, HALF

pytestmark = pytest.mark.gpu

BF16, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def kda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import kda_gated_delta_chunked_gb300 as m
    return m


def normal(seed, *shape, dtype=F32, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g, dtype=F32) * scale).to(dtype)


def within(x, want, bound, what):
    x, want = x.detach().cpu().to(F), want.to(F)
    assert x.shape == want.shape, (what, x.shape, want.shape)
    bad = ~((x - want).abs() <= bound)
    same = torch.isinf(want) & (x == want)
    bad &= ~same
    assert not bad.any(), (what, int(bad.sum()), float((x - want).abs()[bad].max()), torch.nonzero(bad)[:4].tolist())


# ------------------------------------------------------------------ norm
def check_norm(kda, x, w, r, normed, quantize, eps=1e-6, **kw):
    y, q, s, h = kda.rms_norm(x, w, r, eps=eps, normed=normed, quantize=quantize, **kw)
    torch.cuda.synchronize()
    c = lambda t: None if t is None else t.detach().cpu().reshape(-1, t.shape[-1])  # noqa: E731
    wc = None if w is None else w.cpu()
    hr, yr = ref.rms_norm(c(x), wc, c(r), eps)
    d, half = x.shape[-1], HALF[x.dtype]
    fp = (64 + 8) * 2.0 ** -24              # at most 64 additions deep, 8 roundings behind
    if r is not None:
        within(c(h), hr, (half + 2.0 ** -24) * hr.abs() * (1 + half), "h")
    else:
        assert h is None
    if normed:
        within(c(y), yr, (half + fp * (1 + half)) * yr.abs(), "y")
    else:
        assert y is None
    if quantize:
        sr = ref.scales(yr)
        assert s.shape == (*x.shape[:-1], (d + 127) // 128) and q.dtype == F8
        within(c(s), sr, (fp + 2.0 ** -23) * sr, "scales")
        each = c(s).to(F).repeat_interleave(128, 1)[:, :d]
        # half a step of e4m3: 2^-4 of the value, 2^-10 below its smallest normal
        within(c(q).to(F) * each, yr, (HALF[F8] * yr.abs() + 2.0 ** -10 * each) * (1 + 2.0 ** -18) + fp * yr.abs(), "q")
    return y, q, s, h


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("tokens,dim", [(1, 1), (3, 7), (1, 4096), (5, 128), (7, 200), (130, 2051), (33, 1024), (2, 8192),
                                        (2, 16384), (3, 20001)])
def test_norm(kda, dtype, tokens, dim):
    x = normal(1, tokens, dim, dtype=dtype).cuda()
    r = normal(2, tokens, dim, dtype=dtype, scale=3).cuda()
    w = (1 + normal(3, dim, scale=0.2)).to(dtype).cuda()
    check_norm(kda, x, w, r, True, True)
    check_norm(kda, x, None, None, False, True)
    check_norm(kda, x, w, None, True, False)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("tokens,dim", [(40, 1100), (40, 2560), (17, 4305), (21, 6592), (500, 8200), (700, 9001), (500, 16384)])
def test_norm_of_rows_between_powers_of_two_and_blocks_with_several_rows(kda, dtype, tokens, dim):
    x = normal(31, tokens, dim, dtype=dtype).cuda()
    r = normal(32, tokens, dim, dtype=dtype, scale=3).cuda()
    w = (1 + normal(33, dim, scale=0.2)).to(dtype).cuda()
    y, q, s, h = check_norm(kda, x, w, r, True, True)
    check_norm(kda, x, None, None, False, True)
    again = kda.rms_norm(x, w, r, quantize=True, residual_out=x)          # in place of its own input
    assert torch.equal(again[0], y) and torch.equal(again[1].view(torch.uint8), q.view(torch.uint8))
    assert torch.equal(again[2], s) and torch.equal(x, h)


def test_norm_shapes_strides_and_updates_in_place(kda):
    wide = normal(4, 9, 1000, dtype=BF16).cuda()
    x, r = wide[:, 8:520], wide[:, 488:1000]              # 16-byte rows that are not dense
    w = normal(5, 512, dtype=BF16).cuda()
    check_norm(kda, x, w, r, True, True)
    check_norm(kda, wide[:, 3:515], w, wide[:, 484:996], True, True)         # rows off every vector's boundary
    x3 = normal(6, 2, 3, 256, dtype=F32).cuda()
    y, q, s, h = check_norm(kda, x3, None, x3.clone(), True, True)
    assert y.shape == q.shape == h.shape == (2, 3, 256) and s.shape == (2, 3, 2)
    for dim in (512, 18000):                                # registers, and the second read
        x, r = normal(7, 6, dim, dtype=BF16).cuda(), normal(8, 6, dim, dtype=BF16).cuda()
        want = kda.rms_norm(x, None, r, quantize=True)
        keep = r.clone()
        got = kda.rms_norm(x, None, r, quantize=True, residual_out=r)
        assert got[3] is r and torch.equal(r, want[3]) and torch.equal(got[0], want[0])
        got = kda.rms_norm(x, None, keep, quantize=True, residual_out=x)
        assert torch.equal(x, want[3]) and torch.equal(got[0], want[0]) and torch.equal(got[2], want[2])


def test_norm_zero_rows_extremes_and_neighbours(kda):
    x = normal(9, 4, 300, dtype=BF16)
    x[1] = 0
    x[2, 5] = float("inf")
    x = x.cuda()
    y, q, s, _ = kda.rms_norm(x, quantize=True)
    torch.cuda.synchronize()
    assert torch.equal(y[1].float(), torch.zeros(300, device="cuda")) and (q[1].float() == 0).all()
    assert torch.allclose(s[1], torch.full((3,), 1e-12 / 448, device="cuda"), rtol=1e-6)
    check_norm(kda, x[[0, 1, 3]].contiguous(), None, None, True, True)
    for i in (0, 3):                                        # the row with an infinity moves no other
        alone = kda.rms_norm(x[i:i + 1], quantize=True)
        assert torch.equal(alone[0], y[i:i + 1]) and torch.equal(alone[2], s[i:i + 1])
    check_norm(kda, (normal(10, 3, 256) * 1e15).cuda(), None, None, True, True)
    assert [t is None for t in kda.rms_norm(x[:0], quantize=True)] == [False, False, False, True]


# ------------------------------------------------------------------ scaled 8-bit product
def e4m3(seed, r, k):
    return (normal(seed, r, k) * 112).clamp(-448, 448).to(F8)


def check_matmul(kda, a, sa, b, sb, **kw):
    c = kda.matmul_fp8(a, sa, b, sb, **kw)
    torch.cuda.synchronize()
    want, size = ref.matmul_fp8(a.cpu(), sa.cpu(), b.cpu(), sb.cpu())
    kb = sa.shape[1]
    acc = ((128 + kb) * ADD + 4 * 2.0 ** -24) * size
    half = HALF[c.dtype]
    within(c, want, half * want.abs() + (1 + half) * acc, "c")
    return c


def operands(m, n, k, seed=0):
    kb = (k + 127) // 128
    sa = torch.exp(0.5 * normal(seed + 3, m, kb)) / 112
    sb = torch.exp(0.3 * normal(seed + 4, (n + 127) // 128, kb)) / 112
    return e4m3(seed + 1, m, k).cuda(), sa.cuda(), e4m3(seed + 2, n, k).cuda(), sb.cuda()


@pytest.mark.parametrize("simt", [False, True])
@pytest.mark.parametrize("m,n,k", [
    (1, 1, 16), (1, 128, 128), (1, 4096, 512), (2, 300, 1040), (8, 129, 2000), (17, 1000, 640), (33, 64, 256),
    (64, 255, 4096), (65, 513, 144), (100, 1001, 2000), (128, 128, 128), (129, 257, 272), (256, 256, 1024),
    (300, 700, 384), (513, 1300, 528), (1025, 260, 128)])
def test_matmul(kda, simt, m, n, k):
    a, sa, b, sb = operands(m, n, k)
    flags = kda.KDA_FLAG_CUDA_CORE_PREFILL if simt else 0
    check_matmul(kda, a, sa, b, sb, out_dtype=F32, flags=flags)
    check_matmul(kda, a, sa, b, sb, flags=flags)


@pytest.mark.parametrize("m,n,k", [(5, 200, 96 * 128 + 16), (90, 4000, 1008), (256, 2000, 2064), (700, 10000, 272), (1500, 1026, 400),
                                   (2000, 3001, 160)])
def test_matmul_shapes_on_both_sides_of_the_choices(kda, m, n, k):
    a, sa, b, sb = operands(m, n, k)
    check_matmul(kda, a, sa, b, sb, out_dtype=F32)
    check_matmul(kda, a, sa, b, sb)


@pytest.mark.parametrize("m,n,k", [(3, 5, 1), (20, 130, 77), (130, 200, 333)])
def test_matmul_rows_off_every_boundary(kda, m, n, k):
    a, sa, b, sb = operands(m, n, k)
    check_matmul(kda, a, sa, b, sb, out_dtype=F32)


@pytest.mark.parametrize("m", [5, 200, 600])
def test_matmul_strided_rows_and_output(kda, m):
    n, k = 210, 384
    a, sa, b, sb = operands(m, n, 2 * k)
    sa, sb = sa[:, :3].contiguous(), sb[:, :3].contiguous()
    for lo in (0, 128, 5):                  # 5: rows off the 16-byte boundary
        x, y = a[:, lo:lo + k], b[:, lo:lo + k]
        for dt in (F32, BF16):
            wide = torch.full((m, n + 30), 7.0, dtype=dt, device="cuda")
            out = check_matmul(kda, x, sa, y, sb, out=wide[:, 9:9 + n])
            assert out.data_ptr() == wide.data_ptr() + 9 * wide.element_size()
            assert (wide[:, :9] == 7).all() and (wide[:, 9 + n:] == 7).all()


@pytest.mark.parametrize("m", [4, 300])
def test_matmul_nan_and_far_scales_stay_in_their_rows(kda, m):
    a, sa, b, sb = operands(m, 140, 256)
    base = kda.matmul_fp8(a, sa, b, sb, out_dtype=F32).clone()
    a2, sa2 = a.clone(), sa.clone()
    a2.view(torch.uint8)[1, 7] = 0x7F                       # NaN
    sa2[2, 1] = float("inf")
    c = kda.matmul_fp8(a2, sa2, b, sb, out_dtype=F32)
    assert torch.isnan(c[1]).all() and not torch.isfinite(c[2]).any()
    rest = [i for i in range(m) if i not in (1, 2)]
    assert torch.equal(c[rest], base[rest])
    check_matmul(kda, a, sa * 1e-18, b, sb * 1e-12, out_dtype=F32)


def test_norm_feeds_matmul(kda):
    x, r = normal(11, 37, 640, dtype=BF16).cuda(), normal(12, 37, 640, dtype=BF16).cuda()
    _, q, s, _ = kda.rms_norm(x, None, r, normed=False, quantize=True)
    _, _, b, sb = operands(1, 500, 640)
    check_matmul(kda, q, s, b, sb)


# ------------------------------------------------------------------ latent attention, expanded
def check_prefill(kda, q, kn, kr, v, lq=None, lk=None, causal=True, scale=None, simt=False, rows=None, **kw):
    scale = scale or 1 / math.sqrt(q.shape[2])
    cu = lambda l: None if l is None else torch.tensor([0] + list(torch.tensor(l).cumsum(0)), dtype=torch.int32).cuda()  # noqa: E731
    dev = [t if t is None or t.is_cuda else t.cuda() for t in (q, kn, kr, v)]
    ws = torch.empty(kda.latent_prefill_workspace_bytes(len(lq or [0]), q.shape[1], q.dtype), dtype=torch.uint8, device="cuda")
    out, lse = kda.latent_prefill(*dev, cu(lq), cu(lk), scale=scale, causal=causal, workspace=ws,
                                  flags=kda.KDA_FLAG_CUDA_CORE_PREFILL if simt else 0, **kw)
    assert kda.latent_status(ws) == kda.KDA_OK
    q, kn, v = q.cpu(), kn.cpu(), v.cpu()
    kr = None if kr is None else kr.cpu()
    o, l = out.cpu(), lse.cpu()
    tc = q.dtype == BF16 and not simt
    i0 = k0 = 0
    for a, b in zip(lq or [q.shape[0]], lk or [kn.shape[0]]):
        for i in (range(a) if rows is None else [r for r in rows if r < a]):
            end = max(0, min(b, b - a + i + 1)) if causal else b
            for h in range(q.shape[1]):
                k = kn[k0:k0 + end, h]
                k = k if kr is None else torch.cat([k, kr[k0:k0 + end]], 1)
                want, wl, weight, ds = ref.attend(q[i0 + i, h], k, v[k0:k0 + end, h], scale)
                bo, bl = ref.attention_bounds(want, wl, weight, ds, end, q.dtype, tc)
                within(o[i0 + i, h], want, bo, ("out", i0 + i, h))
                within(l[i0 + i, h], torch.tensor(wl), bl, ("lse", i0 + i, h))
        i0, k0 = i0 + a, k0 + b
    return out, lse


def expanded(tq, tk, h, dk=128, dr=64, dv=128, dtype=BF16, seed=0):
    kv = normal(seed + 2, tk, h, dk + dv, dtype=dtype)
    return (normal(seed + 1, tq, h, dk + dr, dtype=dtype), kv[..., :dk], normal(seed + 3, tk, dr, dtype=dtype) if dr else None,
            kv[..., dk:])


@pytest.mark.parametrize("simt", [False, True])
@pytest.mark.parametrize("lq,lk", [([1], [1]), ([1], [300]), ([129], [129]), ([5, 0, 1, 130, 64], [5, 3, 1, 260, 64]),
                                   ([40, 7], [10, 0]), ([260], [257])])
@pytest.mark.parametrize("causal", [True, False])
def test_prefill(kda, simt, lq, lk, causal):
    check_prefill(kda, *expanded(sum(lq), sum(lk), 2), lq, lk, causal, simt=simt, rows=[0, 1, 2, 3, 4, 63, 64, 127, 128, 129, 200, 255, 256, 259])


def test_prefill_long_rows(kda):
    x = expanded(1500, 1500, 3)
    check_prefill(kda, *x, rows=[0, 127, 128, 511, 512, 767, 768, 1300, 1499])
    check_prefill(kda, *x, causal=False, rows=[0, 700, 1499])
    check_prefill(kda, *expanded(300, 2222, 2), rows=[0, 1, 255, 256, 299])


@pytest.mark.parametrize("lq,lk,h", [([256], [5000], 2), ([256], [5000], 33), ([1], [2000], 2), ([300], [1999], 1), ([129, 0, 40], [2100, 500, 1900], 2),
                                     ([1500], [1100], 1), ([7000], [6999], 1), ([200], [130], 1)])
@pytest.mark.parametrize("causal", [True, False])
def test_prefill_few_rows_of_many_keys(kda, lq, lk, h, causal):
    """Where several blocks share the keys of the same rows, some of them without a key that the rows see."""
    x = expanded(sum(lq) + 3, sum(lk) + 9, h, seed=11)
    q, kn, kr, v = x[0][:sum(lq)], x[1], x[2], x[3]
    kn, kr, v = kn.clone(), kr.clone(), v.clone()
    kn[sum(lk):], kr[sum(lk):], v[sum(lk):] = float("nan"), float("nan"), float("inf")
    check_prefill(kda, q, kn[:sum(lk)], kr[:sum(lk)], v[:sum(lk)], lq, lk, causal, rows=[0, 63, 64, 128, 255, 256, 399, 400, 1499, 6999])


@pytest.mark.parametrize("lq,lk,h", [([37 * i % 301 for i in range(70)], [53 * i % 407 for i in range(70)], 9), ([0] * 200 + [5], [3] * 201, 2),
                                     ([600] * 12, [700] * 12, 16)])
@pytest.mark.parametrize("causal", [True, False])
def test_prefill_more_rows_than_the_gpu_holds(kda, lq, lk, h, causal):
    """Blocks take over the rows of others: every row once, whoever computes it, and the same bits each time."""
    q, kn, kr, v = (t.cuda() for t in expanded(sum(lq), sum(lk), h, seed=21))
    o, l = check_prefill(kda, q, kn, kr, v, lq, lk, causal, rows=[0, 127, 128, 300, 599])
    cu = lambda x: torch.tensor([0] + list(torch.tensor(x).cumsum(0)), dtype=torch.int32).cuda()  # noqa: E731
    for _ in range(3):
        out = torch.full_like(o, 7.0)
        o2, l2 = kda.latent_prefill(q, kn, kr, v, cu(lq), cu(lk), scale=1 / math.sqrt(192), causal=causal, out=out)
        assert torch.equal(o, o2) and torch.equal(l, l2)


@pytest.mark.parametrize("dk,dr,dv,dtype", [(128, 64, 128, F32), (96, 32, 64, BF16), (40, 0, 33, BF16), (192, 64, 256, F32)])
def test_prefill_other_sizes_and_types(kda, dk, dr, dv, dtype):
    check_prefill(kda, *expanded(50, 70, 3, dk, dr, dv, dtype), simt=True)
    check_prefill(kda, *expanded(50, 70, 3, dk, dr, dv, dtype), [20, 30], [41, 29], simt=(dk, dr, dv) != (128, 64, 128) or dtype == F32)


def test_prefill_strides(kda):
    """Heads outside tokens, rows inside wider ones, and rows off the 16-byte boundary give what dense ones give."""
    q, kn, kr, v = expanded(140, 150, 3)
    o, l = check_prefill(kda, q.contiguous(), kn.contiguous(), kr, v.contiguous(), rows=[0, 139])
    perm = lambda t: t.cuda().transpose(0, 1).contiguous().transpose(0, 1)  # noqa: E731
    o2, l2 = kda.latent_prefill(perm(q), perm(kn), kr.cuda(), perm(v), scale=1 / math.sqrt(192))
    assert torch.equal(o, o2) and torch.equal(l, l2)
    wide = torch.zeros(150, 80, dtype=BF16, device="cuda")
    wide[:, 8:72] = kr.cuda()
    o2, l2 = kda.latent_prefill(q.cuda(), kn.cuda(), wide[:, 8:72], v.cuda(), scale=1 / math.sqrt(192))
    assert torch.equal(o, o2) and torch.equal(l, l2)
    wide[:, 3:67] = kr.cuda()
    check_prefill(kda, q, kn, wide[:, 3:67], v, rows=[0, 1, 70, 139])


def test_prefill_large_scores_and_infinities(kda):
    q, kn, kr, v = expanded(200, 200, 2, seed=5)
    q = (q.float() * 30).to(BF16)
    check_prefill(kda, q, kn, kr, v, rows=[0, 1, 64, 150, 199])
    # scores of -infinity hide a key; values there do not count unless all are hidden
    q, kn = q.abs(), kn.clone()
    kn[::3] = -float("inf")
    out, lse = kda.latent_prefill(q.cuda(), kn.cuda(), kr.cuda(), v.cuda(), scale=0.01)
    k = torch.cat([kn, kr[:, None].expand(-1, 2, -1)], 2)
    for i in (1, 130, 199):
        seen = [j for j in range(i + 1) if j % 3]
        want, wl, weight, ds = ref.attend(q[i, 1], k[seen, 1], v[seen, 1], 0.01)
        bo, bl = ref.attention_bounds(want, wl, weight, ds, i + 1, BF16, True)
        within(out[i, 1], want, bo, i)
        within(lse[i, 1], torch.tensor(wl), bl, i)
    assert (out[0] == 0).all() and (lse[0] == -float("inf")).all()


def test_prefill_nan_behind_a_sequence_stays_there(kda):
    """Keys and values of the next sequence (here NaN and infinities) never enter a sequence's last tile."""
    lq, lk = [130, 40, 70], [150, 40, 70]
    q, kn, kr, v = expanded(sum(lq), sum(lk), 2, seed=8)
    want, wl = check_prefill(kda, q, kn, kr, v, lq, lk, rows=[0, 129])
    kn, kr, v = kn.clone(), kr.clone(), v.clone()
    kn[150:190], kr[150:190], v[150:190] = float("nan"), float("inf"), float("nan")
    for causal in (True, False):
        cu = lambda l: torch.tensor([0] + list(torch.tensor(l).cumsum(0)), dtype=torch.int32).cuda()  # noqa: E731
        good, _ = kda.latent_prefill(*(t.cuda() for t in expanded(sum(lq), sum(lk), 2, seed=8)), cu(lq), cu(lk), scale=192 ** -0.5, causal=causal)
        out, lse = kda.latent_prefill(q.cuda(), kn.cuda(), kr.cuda(), v.cuda(), cu(lq), cu(lk), scale=192 ** -0.5, causal=causal)
        assert torch.equal(out[:130], good[:130]) and torch.equal(out[170:], good[170:])
        assert torch.isnan(out[130:170].float()).all()


def test_prefill_reports_bad_lengths(kda):
    q, kn, kr, v = (t.cuda() for t in expanded(100, 100, 2))
    ws = torch.empty(kda.latent_prefill_workspace_bytes(2, 2, BF16), dtype=torch.uint8, device="cuda")
    for a, b in (([0, 60, 90], [0, 60, 100]), ([0, 120, 100], [0, 50, 100]), ([0, 50, 100], [0, 130, 100]), ([1, 50, 100], [0, 50, 100])):
        for flags in (0, kda.KDA_FLAG_CUDA_CORE_PREFILL):
            t = lambda c: torch.tensor(c, dtype=torch.int32, device="cuda")  # noqa: E731
            kda.latent_prefill(q, kn, kr, v, t(a), t(b), scale=0.1, workspace=ws, flags=flags)
            assert kda.latent_status(ws) == kda.KDA_ERR_BAD_SEQLENS, (a, b, flags)


# ------------------------------------------------------------------ latent attention, absorbed
def paged(lens, page, width, dtype, seed, spare=2, stride=None):
    """(cache, table, [latents of each sequence]) with pages in a shuffled order."""
    need = [-(-n // page) for n in lens]
    total, cols = sum(need) + spare, max(1, max(need, default=1))
    order = torch.randperm(total, generator=torch.Generator().manual_seed(seed)).tolist()
    rows = normal(seed + 1, total, stride or page, width, dtype=dtype)
    cache = rows[:, :page]
    table = torch.full((len(lens), cols), -1 if spare == 0 else 12345678, dtype=torch.int32)   # never read behind a length
    seqs = []
    for n, (length, p) in enumerate(zip(lens, need)):
        mine = [order.pop() for _ in range(p)]
        table[n, :p] = torch.tensor(mine, dtype=torch.int32)
        seqs.append(cache[mine].reshape(-1, width)[:length])
    return rows.cuda()[:, :page], table.cuda(), seqs


def check_decode(kda, lens, lq, h, page, rank=512, rope=64, dtype=BF16, simt=False, scale=None, seed=0, rows=None, stride=None, gain=1.0):
    w = rank + rope
    scale = scale or 1 / math.sqrt(192)
    cache, table, seqs = paged(lens, page, w, dtype, seed, stride=stride)
    q = normal(seed + 9, len(lens), lq, h, w, dtype=dtype, scale=gain)
    ws = torch.empty(kda.latent_decode_workspace_bytes(len(lens), lq, h, rank, rope, dtype, page, table.shape[1]), dtype=torch.uint8, device="cuda")
    out, lse = kda.latent_decode(q.cuda(), cache, table, torch.tensor(lens, dtype=torch.int32).cuda(), scale=scale, rank=rank,
                                 workspace=ws, flags=kda.KDA_FLAG_CUDA_CORE_PREFILL if simt else 0)
    assert kda.latent_status(ws) == kda.KDA_OK
    o, l = out.cpu(), lse.cpu()
    for n, c in enumerate(seqs):
        for i in range(lq):
            end = max(0, lens[n] - lq + i + 1)
            for hh in range(h) if rows is None else [r for r in rows if r < h]:
                want, wl, weight, ds = ref.attend(q[n, i, hh], c[:end], c[:end, :rank], scale)
                bo, bl = ref.attention_bounds(want, wl, weight, ds, end, dtype, dtype == BF16 and not simt)
                within(o[n, i, hh], want, bo, ("out", n, i, hh))
                within(l[n, i, hh], torch.tensor(wl), bl, ("lse", n, i, hh))
    return out, lse


@pytest.mark.parametrize("simt", [False, True])
@pytest.mark.parametrize("lens,lq,h,page", [
    ([1], 1, 16, 64), ([0, 1, 2, 700], 1, 32, 64), ([127, 128, 129], 1, 16, 16), ([300, 5, 64], 3, 16, 32), ([2, 0, 1, 4], 4, 8, 16),
    ([513, 90], 1, 128, 128), ([200], 2, 20, 64), ([1000, 33], 4, 64, 16), ([600], 1, 1, 8), ([700, 800], 1, 33, 256)])
def test_decode(kda, simt, lens, lq, h, page):
    check_decode(kda, lens, lq, h, page, simt=simt, rows=[0, 1, 7, 15, 16, 31, 32, 33, 63, 64, 127])


@pytest.mark.parametrize("lens,lq,h", [([9000], 1, 16), ([5000, 17, 0, 3001], 2, 32), ([40] * 300, 1, 16), ([0] * 5, 1, 16)])
def test_decode_split_over_the_cache(kda, lens, lq, h):
    check_decode(kda, lens, lq, h, 64, rows=[0, 9, h - 1])


@pytest.mark.parametrize("lens,lq,h,page", [([45000], 1, 32, 64), ([1500] * 70, 1, 16, 64), ([2100, 0, 1, 3333] * 14, 1, 32, 16),
                                            ([1900] * 40, 3, 16, 32), ([2500] * 30, 1, 100, 64)])
def test_decode_many_tiles_a_block_and_nan_behind_the_lengths(kda, lens, lq, h, page):
    """Several tiles and sequences a thread block; pages hold NaN and infinities behind each sequence's length."""
    cache, table, seqs = paged(lens, page, 576, BF16, 31)
    seqs = [c.clone() for c in seqs]
    host = cache.cpu()
    for n, length in enumerate(lens):
        if length % page:
            last = int(table[n, length // page])
            host[last, length % page:] = float("nan")
            host[last, -1] = float("inf")
    for spare in set(range(cache.shape[0])) - set(table.flatten().tolist()):
        host[spare] = float("nan")
    q = normal(32, len(lens), lq, h, 576, dtype=BF16)
    L = torch.tensor(lens, dtype=torch.int32).cuda()
    ws = torch.empty(kda.latent_decode_workspace_bytes(len(lens), lq, h, 512, 64, BF16, page, table.shape[1]), dtype=torch.uint8, device="cuda")
    out, lse = kda.latent_decode(q.cuda(), host.cuda(), table, L, scale=0.0722, workspace=ws)
    assert kda.latent_status(ws) == kda.KDA_OK
    again, lse2 = kda.latent_decode(q.cuda(), host.cuda(), table, L, scale=0.0722)
    assert torch.equal(out, again) and torch.equal(lse, lse2) and torch.isfinite(out.float()).all()
    simt, slse = kda.latent_decode(q.cuda(), cache, table, L, scale=0.0722, flags=kda.KDA_FLAG_CUDA_CORE_PREFILL)
    o, l = out.cpu(), lse.cpu()
    for n in sorted({0, 1, len(lens) // 2, len(lens) - 1} & set(range(len(lens)))):
        for i in range(lq):
            end = max(0, lens[n] - lq + i + 1)
            for hh in (0, h - 1):
                want, wl, weight, ds = ref.attend(q[n, i, hh], seqs[n][:end], seqs[n][:end, :512], 0.0722)
                bo, bl = ref.attention_bounds(want, wl, weight, ds, end, BF16, True)
                within(o[n, i, hh], want, bo, ("out", n, i, hh))
                within(l[n, i, hh], torch.tensor(wl), bl, ("lse", n, i, hh))
    # every row against the CUDA cores' form: both round the output, one its weights
    off = (out.float() - simt.float()).norm(dim=-1) / simt.float().norm(dim=-1).clamp_min(1e-20)
    assert float(off.max()) < 3 * 2.0 ** -8, float(off.max())
    some = torch.isfinite(slse)
    assert torch.equal(torch.isfinite(lse), some) and float((lse - slse)[some].abs().max()) < 1e-4


@pytest.mark.parametrize("rank,rope,dtype,page", [(512, 64, F32, 64), (512, 64, BF16, 48), (256, 32, BF16, 64), (100, 7, F32, 5), (512, 0, BF16, 1)])
def test_decode_other_sizes_types_and_pages(kda, rank, rope, dtype, page):
    check_decode(kda, [130, 0, 77], 2, 3, page, rank, rope, dtype, simt=True)
    check_decode(kda, [130, 0, 77], 2, 3, page, rank, rope, dtype, simt=(rank, rope, dtype) != (512, 64, BF16))


def test_decode_layouts(kda):
    """Pages apart in a larger pool, one query given without its dimension, strided query heads."""
    lens, h = [300, 61], 16
    check_decode(kda, lens, 1, h, 32, stride=40)
    cache, table, _ = paged(lens, 32, 576, BF16, 3)
    q = normal(4, 2, 1, h, 576, dtype=BF16).cuda()
    L = torch.tensor(lens, dtype=torch.int32).cuda()
    o, l = kda.latent_decode(q, cache, table, L, scale=0.07)
    o1, l1 = kda.latent_decode(q[:, 0], cache, table, L, scale=0.07)
    assert o1.shape == (2, h, 512) and torch.equal(o[:, 0], o1) and torch.equal(l[:, 0], l1)
    wide = torch.zeros(2, h, 640, dtype=BF16, device="cuda")
    for lo in (0, 64, 3):
        wide[..., lo:lo + 576] = q[:, 0]
        o2, l2 = kda.latent_decode(wide[..., lo:lo + 576], cache, table, L, scale=0.07)
        if lo != 3:
            assert torch.equal(o2, o1) and torch.equal(l2, l1)
        else:
            assert torch.allclose(o2.float(), o1.float(), rtol=2.0 ** -6, atol=2.0 ** -6)


def test_decode_large_scores(kda):
    check_decode(kda, [400, 1500], 1, 32, 64, gain=25.0, rows=[0, 5, 31])


def test_decode_last_rows_follow_the_query(kda):
    """The last of Lq queries over a cache of L tokens is the single query over it; the first sees Lq - 1 fewer."""
    cache, table, _ = paged([500], 64, 576, BF16, 3)
    q = normal(4, 1, 3, 16, 576, dtype=BF16).cuda()
    at = lambda n: torch.tensor([n], dtype=torch.int32, device="cuda")  # noqa: E731
    o, l = kda.latent_decode(q, cache, table, at(500), scale=0.07)
    for i in range(3):
        o1, l1 = kda.latent_decode(q[:, i], cache, table, at(498 + i), scale=0.07)
        assert torch.allclose(l[:, i], l1, rtol=0, atol=1e-5)
        assert torch.allclose(o[:, i].float(), o1.float(), rtol=2.0 ** -6, atol=2.0 ** -7)


def test_decode_reports_bad_pages_and_lengths(kda):
    """Page numbers outside the cache and lengths outside the table are reported, not followed."""
    for flags in (0, kda.KDA_FLAG_CUDA_CORE_PREFILL):
        cache, table, seqs = paged([300, 200], 64, 576, BF16, 3)
        q = normal(4, 2, 1, 16, 576, dtype=BF16).cuda()
        ws = torch.empty(kda.latent_decode_workspace_bytes(2, 1, 16, 512, 64, BF16, 64, table.shape[1]), dtype=torch.uint8, device="cuda")

        def call(lens, t):
            o, _ = kda.latent_decode(q, cache, t, torch.tensor(lens, dtype=torch.int32, device="cuda"), scale=0.07, workspace=ws, flags=flags)
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


# ------------------------------------------------------------------ together, streams, graphs, repeats
def _all(kda, stream=None):
    x, r = normal(20, 70, 512, dtype=BF16).cuda(), normal(21, 70, 512, dtype=BF16).cuda()
    a, sa, b, sb = operands(70, 300, 512, 22)
    q, kn, kr, v = (t.cuda() for t in expanded(200, 200, 2, seed=23))
    cache, table, _ = paged([700, 9], 64, 576, BF16, 24)
    qd, L = normal(25, 2, 1, 16, 576, dtype=BF16).cuda(), torch.tensor([700, 9], dtype=torch.int32).cuda()
    torch.cuda.synchronize()

    def go():
        out = [t for t in kda.rms_norm(x, None, r, quantize=True, stream=stream)]
        out.append(kda.matmul_fp8(a, sa, b, sb, stream=stream))
        out.append(kda.matmul_fp8(out[1], out[2], b, sb, stream=stream))
        out += kda.latent_prefill(q, kn, kr, v, scale=0.07, stream=stream)
        out += kda.latent_decode(qd, cache, table, L, scale=0.07, stream=stream)
        return out
    return go


def same(a, b):
    return all(torch.equal(x.view(torch.uint8) if x.dtype == F8 else x, y.view(torch.uint8) if y.dtype == F8 else y) for x, y in zip(a, b))


def test_repeats_streams_and_graphs_give_the_same_bits(kda):
    go = _all(kda)
    want = go()
    torch.cuda.synchronize()
    for _ in range(5):
        assert same(go(), want)
    for other in (torch.cuda.Stream(), torch.cuda.Stream().cuda_stream):
        got = _all(kda, other)()
        torch.cuda.synchronize()
        assert same(got, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = go()
    for t in got:
        t.view(torch.uint8).zero_()
    g.replay()
    g.replay()
    torch.cuda.synchronize()
    assert same(got, want)


def test_nothing_is_written_outside_the_outputs(kda):
    def guarded(*shape, dtype):
        n = math.prod(shape) * torch.empty((), dtype=dtype).element_size()
        whole = torch.full((n + 512,), 0xA5, dtype=torch.uint8, device="cuda")
        return whole, whole[256:256 + n].view(dtype).view(*shape)

    def check(*wholes):
        torch.cuda.synchronize()
        for w in wholes:
            assert (w[:256] == 0xA5).all() and (w[-256:] == 0xA5).all()
    for m, n, k in ((3, 77, 64), (200, 333, 256), (700, 600, 144)):
        for dt in (BF16, F32):
            w, c = guarded(m, n, dtype=dt)
            kda.matmul_fp8(*operands(m, n, k), out=c)
            check(w)
    for lq, lk in (([3], [3]), ([130, 1, 257], [150, 1, 257])):
        (w1, o), (w2, l) = guarded(sum(lq), 2, 128, dtype=BF16), guarded(sum(lq), 2, dtype=F32)
        check_prefill(kda, *expanded(sum(lq), sum(lk), 2), lq, lk, rows=[0], out=o, lse=l)
        check(w1, w2)
    for h, lq in ((16, 1), (20, 3), (100, 1)):
        cache, table, _ = paged([700, 9, 0], 64, 576, BF16, 24)
        q = normal(25, 3, lq, h, 576, dtype=BF16).cuda()
        (w1, o), (w2, l) = guarded(3, lq, h, 512, dtype=BF16), guarded(3, lq, h, dtype=F32)
        w3, ws = guarded(kda.latent_decode_workspace_bytes(3, lq, h, 512, 64, BF16, 64, table.shape[1]), dtype=torch.uint8)
        kda.latent_decode(q, cache, table, torch.tensor([700, 9, 0], dtype=torch.int32).cuda(), scale=0.07, out=o, lse=l, workspace=ws)
        check(w1, w2, w3)
