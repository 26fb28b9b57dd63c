"""Rotary positions on the GPU against 64-bit forms, element by element."""
import math

import pytest
import torch

import latent_cache_ref as cref
from operators_ref import F, HALF
from test_gpu_operators import BF16, F32, kda, normal, within  # noqa: F401

pytestmark = pytest.mark.gpu


def check(kda, x, pos, f, *, key=None, offset=None, key_offset=None, interleaved=False, inverse=False, scale=1.0, **kw):  # noqa: F811
    dim = 2 * f.numel()
    xc, kc = x.detach().cpu().clone(), None if key is None else key.detach().cpu().clone()
    y, ky = kda.rotary(x, pos, f, key=key, offset=offset, key_offset=key_offset, interleaved=interleaved, inverse=inverse,
                       scale=scale, **kw)
    torch.cuda.synchronize()
    for what, got, src, at in (("x", y, xc, offset), ("key", ky, kc, key_offset)):
        if src is None:
            assert got is None
            continue
        assert got.shape == src.shape and got.dtype == src.dtype
        rows = src if src.dim() == 3 else src[:, None]
        want, size = cref.rotary(rows, pos.cpu(), f.cpu(), dim, rows.shape[-1] - dim if at is None else at, interleaved, inverse, scale)
        bound = cref.rotary_bound(want, size, pos.cpu(), f.cpu(), src.dtype)
        within(got.cpu().view_as(rows) if got.dim() == 3 else got.cpu()[:, None], want, bound, what)
    return y, ky


def places(seed, t, far, wide=False):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(0, far, (t,), generator=g).to("cuda", torch.int64 if wide else torch.int32)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("t,heads,width,dim,offset", [
    (1, 1, 2, 2, 0), (1, 32, 192, 64, 128), (5, 3, 64, 64, 0), (777, 7, 80, 48, 0), (33, 5, 100, 36, 7), (130, 1, 64, 64, None),
    (3, 130, 40, 14, 26), (70, 2, 1024, 1024, 0), (9, 1, 4096, 2, 4093), (4, 65, 256, 128, 64), (1000, 4, 24, 8, None), (300, 1, 6, 6, 0)])
def test_rotary(kda, dtype, interleaved, t, heads, width, dim, offset):  # noqa: F811
    x, f = normal(t, t, heads, width, dtype=dtype).cuda(), kda.rotary_frequencies(dim)
    check(kda, x, places(1, t, 100000), f, offset=offset, interleaved=interleaved)
    check(kda, x, places(2, t, 3000, True), f, offset=offset, interleaved=interleaved, inverse=True, scale=1.3466)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("t,heads,width,keys,kwidth,dim", [(1, 32, 192, 1, 64, 64), (300, 16, 128, 2, 128, 128), (65, 3, 64, 5, 200, 62),
                                                           (2, 1, 64, 64, 64, 64), (7, 128, 192, 1, 64, 64)])
def test_rotary_of_queries_and_keys(kda, dtype, interleaved, t, heads, width, keys, kwidth, dim):  # noqa: F811
    x, k = normal(1, t, heads, width, dtype=dtype).cuda(), normal(2, t, keys, kwidth, dtype=dtype).cuda()
    f, pos = kda.rotary_frequencies(dim, base=500000.0), places(3, t, 1000000)
    y, ky = check(kda, x, pos, f, key=k, interleaved=interleaved, scale=0.9)
    assert torch.equal(y, kda.rotary(x, pos, f, interleaved=interleaved, scale=0.9)[0])        # alone, and together
    assert torch.equal(ky, kda.rotary(k, pos, f, interleaved=interleaved, scale=0.9)[0])
    check(kda, x, pos, f, key=k, interleaved=interleaved, offset=0, key_offset=0)
    if keys == 1:
        y2, ky2 = check(kda, x, pos, f, key=k[:, 0], interleaved=interleaved, scale=0.9)
        assert torch.equal(y2, y) and torch.equal(ky2, ky[:, 0])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("lead,gap", [(0, 0), (8, 16), (1, 3), (2, 2)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_in_place_of_parts_of_one_projection(kda, dtype, lead, gap, interleaved):  # noqa: F811
    """Queries and the shared key as views of one buffer, whatever their alignment: only the turned channels change."""
    t, h, w, d = 50, 4, 192, 64
    both = normal(4, t, lead + h * w + gap + d, dtype=dtype).cuda()
    q, k = both[:, lead:lead + h * w].unflatten(1, (h, w)), both[:, lead + h * w + gap:]
    f, pos = kda.rotary_frequencies(d), places(5, t, 40000)
    want = kda.rotary(q.contiguous(), pos, f, key=k.contiguous(), interleaved=interleaved)
    keep = both.clone()
    got = check(kda, q, pos, f, key=k, interleaved=interleaved, out=q, key_out=k)
    assert got[0].data_ptr() == q.data_ptr() and torch.equal(q, want[0]) and torch.equal(k, want[1])
    turned = torch.zeros_like(both, dtype=torch.bool)
    turned[:, lead:lead + h * w].unflatten(1, (h, w))[..., w - d:] = True
    turned[:, lead + h * w + gap:] = True
    assert torch.equal(both[~turned], keep[~turned])


def test_rotary_layouts(kda):  # noqa: F811
    """Heads outside tokens, expanded inputs, outputs with strides, a sequence padded with zeros."""
    f, pos = kda.rotary_frequencies(32), places(6, 40, 5000)
    x = normal(7, 6, 40, 64, dtype=BF16).cuda().transpose(0, 1)                     # [40, 6, 64], heads outermost
    want = check(kda, x, pos, f)[0]
    out = torch.full((6, 41, 72), 7.0, dtype=BF16, device="cuda")
    got = kda.rotary(x, pos, f, out=out[:, :40, :64].transpose(0, 1))[0]
    assert torch.equal(got, want) and (out[:, 40:] == 7).all() and (out[:, :, 64:] == 7).all()
    one = normal(8, 1, 1, 64, dtype=F32).cuda()
    check(kda, one.expand(40, 3, 64), pos, f, interleaved=True)                      # every row the same one
    e, ek = kda.rotary(x[:0], pos[:0], f, key=x[:0])
    assert e.shape == (0, 6, 64) and ek.shape == (0, 6, 64)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_far_positions(kda, interleaved):  # noqa: F811
    """Positions up to 2^31 and 2^40 and negative ones: the angle is right to 2^-52 of position times frequency."""
    f = kda.rotary_frequencies(64)
    x = normal(9, 9, 2, 64, dtype=F32).cuda()
    far = torch.tensor([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 10 ** 6, 10 ** 7 + 1, -12345, 4096], device="cuda")
    a = check(kda, x, far.int(), f, interleaved=interleaved)[0]
    b = check(kda, x, far, f, interleaved=interleaved)[0]
    assert torch.equal(a, b)
    slow = f * 2.0 ** -9
    check(kda, x, far * 512, slow, interleaved=interleaved)
    fast = f * 100                                                                    # more than a turn a position
    check(kda, x, far.clamp(-10 ** 6, 10 ** 6), fast, interleaved=interleaved)


def test_rotary_turns_back(kda):  # noqa: F811
    """The inverse of a turn, and the gradient: against differences of a sum over the outputs."""
    f, pos = kda.rotary_frequencies(24), places(10, 11, 900)
    x, g = normal(11, 11, 3, 40, dtype=F32).cuda(), normal(12, 11, 3, 40, dtype=F32).cuda()
    for interleaved in (False, True):
        y = kda.rotary(x, pos, f, interleaved=interleaved)[0]
        back = kda.rotary(y, pos, f, interleaved=interleaved, inverse=True)[0]
        assert float((back - x).abs().max()) < 4 * (cref.ROTARY + HALF[F32]) * float(x.abs().max()) * 2
        grad = kda.rotary(g, pos, f, interleaved=interleaved, inverse=True, scale=1.25)[0].double()
        for at in ((0, 0, 0), (3, 1, 17), (10, 2, 39), (5, 0, 28)):
            e = torch.zeros_like(x)
            e[at] = 0.5
            up, down = (kda.rotary(x + s * e, pos, f, interleaved=interleaved, scale=1.25)[0].double() for s in (1, -1))
            part = slice(16, 40)
            # linear: the difference is exact but for the roundings of both outputs
            if at[2] >= 16:
                d = float(((up - down)[..., part] * g.double()[..., part]).sum())
                room = 2 * (cref.ROTARY + HALF[F32]) * 2.5 * (float(x.abs().max()) + 1) * float(g.abs().sum(-1).max())
                assert abs(d - float(grad[at])) < room, (at, d, float(grad[at]))
            else:
                assert torch.equal((up - down).nonzero(), torch.tensor([at], device="cuda"))


def test_rotary_scores_depend_on_distances_alone(kda):  # noqa: F811
    """What the operator is for: q.k of turned rows is a function of the positions' difference."""
    f = kda.rotary_frequencies(64)
    q, k = normal(13, 1, 1, 64, dtype=F32).cuda(), normal(14, 1, 1, 64, dtype=F32).cuda()

    def score(m, n):
        at = lambda p: torch.tensor([p], dtype=torch.int64, device="cuda")  # noqa: E731
        return float((kda.rotary(q, at(m), f)[0].double() * kda.rotary(k, at(n), f)[0].double()).sum())
    room = 64 * 4 * (cref.ROTARY + HALF[F32]) * float(q.abs().max() * k.abs().max())
    for m, n in ((5, 3), (1000, 998), (10 ** 6, 10 ** 6 - 2), (0, -2)):
        assert abs(score(m, n) - score(2, 0)) < room, (m, n)


def test_rotary_frequencies_on_the_device(kda):  # noqa: F811
    f = kda.rotary_frequencies(64, method=kda.KDA_ROTARY_BY_PARTS, factor=32.0, original_length=4096)
    assert f.is_cuda and f.dtype == F and f.shape == (32,)
    x = normal(15, 20, 4, 192, dtype=BF16).cuda()
    check(kda, x, places(16, 20, 131072), f, interleaved=True, scale=0.1 * math.log(32) + 1)


def test_rotary_of_rows_far_apart(kda):  # noqa: F811
    """Offsets above 32 bits."""
    x = normal(17, 300, 2, 64, dtype=BF16).cuda()
    f, pos = kda.rotary_frequencies(64), places(18, 300, 5000)
    want = kda.rotary(x, pos, f)[0]
    step = 1 << 24
    wide = torch.empty(300 * step, dtype=BF16, device="cuda").as_strided(x.shape, (step, 64, 1))
    wide.copy_(x)
    assert torch.equal(kda.rotary(wide, pos, f)[0], want)
    assert torch.equal(kda.rotary(wide, pos, f, out=wide)[0], want)


def test_rotary_refusals(kda):  # noqa: F811
    x, f, pos = normal(19, 4, 2, 64, dtype=BF16).cuda(), kda.rotary_frequencies(64), places(20, 4, 50)
    bad = [dict(x=x.half()), dict(x=x[:3]), dict(x=x[..., :32]), dict(x=x.cpu()), dict(x=x[..., ::2]), dict(x=x[:, :0]), dict(x=x[None]),
           dict(positions=pos.float()), dict(positions=pos[:, None]), dict(positions=pos.cpu()), dict(frequencies=f.float()),
           dict(frequencies=f[:0]), dict(frequencies=f.cpu()), dict(offset=1), dict(offset=-1), dict(out=x[:3]), dict(out=x.float()),
           dict(key_out=x), dict(key=x.float()), dict(key=x[:2]), dict(key=x, key_offset=4), dict(key=x[..., :32]), dict(scale="a"),
           dict(offset=0.5)]
    for kw in bad:
        args = dict(x=x, positions=pos, frequencies=f)
        args.update(kw)
        with pytest.raises(ValueError):
            kda.rotary(args.pop("x"), args.pop("positions"), args.pop("frequencies"), **args)
    flat = normal(21, 4 * 2 * 64 + 64, dtype=BF16).cuda()
    for kw in (dict(out=flat[64:].view(4, 2, 64)), dict(key=x, key_out=flat[:512].view(4, 2, 64)), dict(scale=float("nan")),
               dict(out=x[:1].expand(4, 2, 64))):
        with pytest.raises(kda.KdaError):
            kda.rotary(flat[:512].view(4, 2, 64), pos, f, **kw)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("lead,row", [(8, 104), (4, 104), (4, 100), (2, 106), (1, 100), (0, 97)])
def test_rotary_of_every_alignment_gives_the_same_bits(kda, dtype, interleaved, lead, row):  # noqa: F811
    """Rows of 96 channels, 64 turned, that start on 16, 8, 4 or 2 bytes; what lies between them stays."""
    x = normal(19, 130, 5, 96, dtype=dtype).cuda()
    f, pos = kda.rotary_frequencies(64), places(20, 130, 70000)
    want = check(kda, x, pos, f, offset=16, interleaved=interleaved)[0]
    wide = lambda: torch.full((lead + 130 * 5 * row,), 5.0, dtype=dtype, device="cuda")  # noqa: E731
    of = lambda b: b[lead:].view(130, 5, row)[..., :96]  # noqa: E731
    a, b = wide(), wide()
    of(a).copy_(x)
    kda.rotary(of(a), pos, f, offset=16, interleaved=interleaved, out=of(b))
    assert torch.equal(of(b), want)
    assert (b[:lead] == 5).all() and (b[lead:].view(130, 5, row)[..., 96:] == 5).all()
    kda.rotary(of(a), pos, f, offset=16, interleaved=interleaved, out=of(a))
    assert torch.equal(a, b)
