"""The quantised cache of latents and the rotary positions in plain 64-bit forms,
and the bounds their tests use (beside those of operators_ref.py)."""
import math

import torch

import operators_ref as ref
from operators_ref import F, HALF

E4M3 = torch.float8_e4m3fn


def exponent(c):
    """The smallest integer e with max |finite c| <= 448 2^e, within -100 .. 120, of each row."""
    top = torch.where(torch.isfinite(c), c.to(F).abs(), torch.zeros((), dtype=F)).amax(-1)
    e = torch.full(top.shape, -100, dtype=torch.int64)
    for k in range(-100, 120):
        e = torch.where(top > 448 * 2.0 ** k, torch.full_like(e, k + 1), e)
    return e


def nearest_e4m3(x):
    """The nearest multiple of the step (3 bits behind the leading one, 2^-9 below 2^-6), ties to even; at most 448."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp_min(2.0 ** -6))) - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)


def quantise(c):
    """(values of the codes in 64 bits, e) of rows c."""
    e = exponent(c)
    v = nearest_e4m3(c.to(F) / torch.exp2(e.to(F))[..., None])
    return torch.where(torch.isfinite(c), v, torch.full_like(v, math.nan)), e


def page_bytes(page, rank, rope):
    return -(-page * (rank + 2 * rope + 1) // 128) * 128


def views(cache, page, rank, rope):
    """Codes (e4m3), rotary channels (bf16) and scale bytes of a cache [pages, bytes], as views."""
    row = rank + 2 * rope
    rows = cache[:, :page * row].unflatten(1, (page, row))
    return rows[..., :rank].view(E4M3), rows[..., rank:].view(torch.bfloat16), cache[:, page * row:page * (row + 1)]


def fill(cache, page, rank, rope, latents, rotary):
    """Quantises latents [pages, page, rank] and rotary [pages, page, rope] into the whole cache."""
    codes, r, s = views(cache, page, rank, rope)
    v, e = quantise(latents)
    codes.copy_(v.float().to(E4M3))
    r.copy_(rotary.to(torch.bfloat16))
    s.copy_((e + 127).to(torch.uint8))


def values(cache, page, rank, rope):
    """(2^e code [pages, page, rank], rotary channels) in 64 bits."""
    codes, r, s = views(cache, page, rank, rope)
    return codes.to(F) * torch.exp2(s.to(F) - 127)[..., None], r.to(F)


def attention_bounds(q, keys, rank, want, lse, weight, ds, scale, dtype, tensor_cores):
    """Bounds of (out, lse) of one query row over keys [n, rank + rope] of the quantised cache.

    On CUDA cores those of fp32.  On the tensor cores:
    - a query's channel is the sum of two e4m3 values under a power of two that
      puts its row's largest within 224 .. 448: exact for the 8 bits of bf16,
      below that half of e4m3's smallest step, 2^-10 / 16, so 2^-14 / 224 of the
      largest channel;
    - a weight is rounded to half precision (2^-11) and then the sum of three e5m2
      values, each the rest of the one before (2^-3 of it), so off by 2^-8.6, or by
      half of the third one's smallest step, 2^-23, where the reference keeps the
      largest weight at 2^3 or more.
    - the exponent of a token's scale is added to its score: 2^-24 of both."""
    n = keys.shape[0]
    bo, bl = ref.attention_bounds(want, lse, weight, ds, n, dtype, False)
    if not tensor_cores or n == 0:
        return bo, bl
    more = scale * 2.0 ** -21.8 * float(q.abs().to(F).max()) * float(keys[:, :rank].abs().sum(1).max())
    more += 4 * 2.0 ** -24 * (130 + abs(lse))
    p = torch.exp((keys.to(F) @ q.to(F)) * scale - lse)
    floor = n * 2.0 ** -26 * float((p * keys[:, :rank].abs().amax(1)).max()) * 2
    return bo + (2 * more + 2.0 ** -8.6) * weight * (1 + HALF[dtype]) + floor, bl + more


def rotary(x, positions, frequencies, dim, offset, interleaved, inverse, scale):
    """(result, sum of |terms|) in 64 bits of x [t, heads, width]."""
    theta = positions.to(F)[:, None] * frequencies
    c, s = torch.cos(theta)[:, None] * scale, torch.sin(theta)[:, None] * scale * (-1 if inverse else 1)
    part = x[..., offset:offset + dim].to(F)
    at = (slice(0, dim, 2), slice(1, dim, 2)) if interleaved else (slice(0, dim // 2), slice(dim // 2, dim))
    a, b = part[..., at[0]], part[..., at[1]]
    y, size = x.to(F).clone(), torch.zeros(x.shape, dtype=F)
    out, terms = torch.empty_like(part), torch.empty_like(part)
    out[..., at[0]], out[..., at[1]] = a * c - b * s, b * c + a * s
    terms[..., at[0]] = terms[..., at[1]] = (a.abs() + b.abs()) * abs(scale)
    y[..., offset:offset + dim], size[..., offset:offset + dim] = out, terms
    return y, size


# cos and sin: the angle in half turns is rounded to 24 bits (pi 2^-25), sincospi is off by 2 ulp (2^-23), then the
# scale, the product and the sum are rounded (3 2^-24)
ROTARY = math.pi * 2.0 ** -25 + 2.0 ** -23 + 3 * 2.0 ** -24


def rotary_bound(y, size, positions, frequencies, dtype):
    """Element-wise bound; the turn fraction of a position is off by 2^-52 of position times frequency."""
    angle = 2 * float(positions.abs().max() if positions.numel() else 0) * float(frequencies.abs().max()) * 2.0 ** -52
    rel = ROTARY * 1.01 + angle
    return rel * size + HALF[dtype] * (y.abs() + rel * size) * (size > 0)
