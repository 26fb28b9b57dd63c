"""Plain 64-bit forms of the operators around the recurrent layers, one row at a
time, and the element-wise error bounds their tests use.

A rounding to a type is off by at most HALF[type] relative to the value.  Sums
of n fp32 terms are off by at most n * 2^-23 times the sum of the terms' sizes
(2^-23, not 2^-24, an addition: the tensor cores align and cut their addends).
"""
import math

import torch

F = torch.float64
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float8_e4m3fn: 2.0 ** -4}
ADD = 2.0 ** -23


def rms_norm(x, weight, residual, eps):
    """(h, y) in 64 bits."""
    h = x.to(F) + (residual.to(F) if residual is not None else 0)
    y = h / torch.sqrt((h * h).mean(-1, keepdim=True) + eps)
    return h, y * weight.to(F) if weight is not None else y


def scales(y):
    """Per block of 128 of a row: max(max |y|, 1e-12) / 448."""
    t, d = y.shape
    cols = [y[:, b:b + 128].abs().amax(1) for b in range(0, d, 128)]
    return torch.stack(cols, 1).clamp_min(1e-12) / 448


def matmul_fp8(a, sa, b, sb):
    """(c, sum of |terms|) in 64 bits."""
    k, n = a.shape[1], b.shape[0]
    x = a.to(F) * sa.to(F).repeat_interleave(128, 1)[:, :k]
    y = b.to(F) * sb.to(F).repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)[:, :k]
    return x @ y.t(), x.abs() @ y.abs().t()


def attend(q, k, v, scale):
    """One query row over the keys it sees: (out, lse, sum p |v|, bound of the scores' absolute error)."""
    if k.shape[0] == 0:
        z = torch.zeros(v.shape[1], dtype=F)
        return z, -math.inf, z, 0.0
    q, k, v = q.to(F), k.to(F), v.to(F)
    s = (k @ q) * scale
    lse = torch.logsumexp(s, 0)
    p = torch.exp(s - lse)
    size = float((k.abs() @ q.abs()).max()) * scale
    # the dot product's additions, and the factor's and the exponent's roundings
    return p @ v, float(lse), p @ v.abs(), k.shape[1] * ADD * size + 4 * 2.0 ** -24 * (size + abs(float(lse)))


def attention_bounds(ref, lse, weight, ds, keys, dtype, tensor_cores):
    """Element-wise bounds of (out, lse): scores off by ds move every weight by
    2 ds at most; exp2 by 2^-22; the sum over the keys; weights rounded to bf16
    once on the tensor cores; partial results joined in fp32; the output rounded
    once."""
    rel = 2 * ds + 4 * 2.0 ** -22 + keys * ADD + (HALF[torch.bfloat16] if tensor_cores else 0.0)
    return rel * weight + HALF[dtype] * (ref.abs() + rel * weight) + 1e-30, ds + 2.0 ** -21 + keys * ADD + 4 * 2.0 ** -24 * abs(lse)
