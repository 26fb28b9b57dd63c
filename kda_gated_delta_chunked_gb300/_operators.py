"""Norm, 8-bit products and latent attention: the operators around the recurrent
layers (argument marshalling only; see include/kda.h for what each computes)."""
from __future__ import annotations

import contextlib
import ctypes
from typing import Optional

import torch

from . import _binding as B
from ._binding import KDA_ERR_UNSUPPORTED, KDA_OK, KdaError, lib

KDA_FLAG_NO_CAUSAL = 4


class KdaNormDesc(ctypes.Structure):
    """Mirror of ``kda_norm_desc`` in include/kda.h."""
    _fields_ = [("rows", ctypes.c_int64), ("dim", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("x_stride", ctypes.c_int64), ("residual_stride", ctypes.c_int64), ("eps", ctypes.c_float)]


class KdaMatmulDesc(ctypes.Structure):
    """Mirror of ``kda_matmul_desc`` in include/kda.h."""
    _fields_ = [("m", ctypes.c_int64), ("n", ctypes.c_int32), ("k", ctypes.c_int32), ("a_stride", ctypes.c_int64),
                ("b_stride", ctypes.c_int64), ("c_stride", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("flags", ctypes.c_int32)]


class KdaLatentDesc(ctypes.Structure):
    """Mirror of ``kda_latent_desc`` in include/kda.h."""
    _fields_ = [("num_seqs", ctypes.c_int32), ("num_heads", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("flags", ctypes.c_int32), ("scale", ctypes.c_float), ("d_k", ctypes.c_int32),
                ("d_rope", ctypes.c_int32), ("d_v", ctypes.c_int32), ("total_q", ctypes.c_int64),
                ("total_k", ctypes.c_int64), ("q_token_stride", ctypes.c_int64), ("q_head_stride", ctypes.c_int64),
                ("k_token_stride", ctypes.c_int64), ("k_head_stride", ctypes.c_int64),
                ("v_token_stride", ctypes.c_int64), ("v_head_stride", ctypes.c_int64),
                ("rope_token_stride", ctypes.c_int64), ("num_queries", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("num_pages", ctypes.c_int32), ("max_pages", ctypes.c_int32),
                ("page_stride", ctypes.c_int64), ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t)]


def _declare():
    vp, ref = ctypes.c_void_p, ctypes.POINTER
    for name, args, res in (
            ("kda_rms_norm", [ref(KdaNormDesc)] + [vp] * 8, ctypes.c_int),
            ("kda_matmul_fp8", [ref(KdaMatmulDesc)] + [vp] * 6, ctypes.c_int),
            ("kda_latent_prefill_workspace_bytes", [ref(KdaLatentDesc)], ctypes.c_size_t),
            ("kda_latent_decode_workspace_bytes", [ref(KdaLatentDesc)], ctypes.c_size_t),
            ("kda_latent_prefill", [ref(KdaLatentDesc)] + [vp] * 9, ctypes.c_int),
            ("kda_latent_decode", [ref(KdaLatentDesc)] + [vp] * 7, ctypes.c_int),
            ("kda_latent_status", [ref(KdaLatentDesc), vp], ctypes.c_int)):
        f = getattr(lib, name)
        f.argtypes, f.restype = args, res


_declare()
_byref = ctypes.byref
_current_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice
_F8, _F32, _I32 = torch.float8_e4m3fn, torch.float32, torch.int32


def kda_rms_norm(desc: KdaNormDesc, x, weight, residual, residual_out, normed, quantized, scales, stream=None) -> int:
    """Raw C call: every tensor argument is passed as its data pointer (or NULL)."""
    p = B._p
    return lib.kda_rms_norm(_byref(desc), p(x), p(weight), p(residual), p(residual_out), p(normed), p(quantized),
                            p(scales), B._stream(stream))


def kda_matmul_fp8(desc: KdaMatmulDesc, a, a_scale, b, b_scale, c, stream=None) -> int:
    """Raw C call of the scaled e4m3 product."""
    p = B._p
    return lib.kda_matmul_fp8(_byref(desc), p(a), p(a_scale), p(b), p(b_scale), p(c), B._stream(stream))


def kda_latent_prefill_workspace_bytes(desc: KdaLatentDesc) -> int:
    return lib.kda_latent_prefill_workspace_bytes(_byref(desc))


def kda_latent_decode_workspace_bytes(desc: KdaLatentDesc) -> int:
    return lib.kda_latent_decode_workspace_bytes(_byref(desc))


def kda_latent_prefill(desc: KdaLatentDesc, q, k_nope, k_rope, v, cu_seqlens_q, cu_seqlens_k, out, lse,
                       stream=None) -> int:
    """Raw C call of the expanded form."""
    p = B._p
    return lib.kda_latent_prefill(_byref(desc), p(q), p(k_nope), p(k_rope), p(v), p(cu_seqlens_q), p(cu_seqlens_k),
                                  p(out), p(lse), B._stream(stream))


def kda_latent_decode(desc: KdaLatentDesc, q, cache, page_table, lengths, out, lse, stream=None) -> int:
    """Raw C call of the absorbed form."""
    p = B._p
    return lib.kda_latent_decode(_byref(desc), p(q), p(cache), p(page_table), p(lengths), p(out), p(lse),
                                 B._stream(stream))


def kda_latent_status(desc: KdaLatentDesc, stream=None) -> int:
    """Device status word of the last latent call on the desc's workspace (synchronises the stream)."""
    return lib.kda_latent_status(_byref(desc), B._stream(stream))


# ------------------------------------------------------------------ checks
def _tensor(t, name: str, dtype, dim: int, device):
    """A tensor of `dim` dimensions on `device` whose last one is dense."""
    if t.dtype != dtype or t.dim() != dim or t.device != device or (t.stride(-1) != 1 and t.shape[-1] > 1):
        raise ValueError(f"{name} must be a {dim}-D {dtype} tensor on {device} with a dense last dimension: got "
                         f"{tuple(t.shape)}, {t.dtype}, {t.device}, strides {t.stride()}")


def _dense(t, name: str, dtype, shape, device):
    if t.dtype != dtype or t.shape != shape or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {tuple(shape)} {dtype} tensor on {device}: got "
                         f"{tuple(t.shape)}, {t.dtype}, {t.device}, strides {t.stride()}")


def _device(t, name: str):
    if not t.is_cuda or t.get_device() != _current_device():
        raise ValueError(f"{name} must be on the current CUDA device: got {t.device}")
    return t.device


def _row_stride(t, width: int) -> int:
    """Elements between rows of a 2-D tensor (a single row may carry any stride)."""
    return t.stride(0) if t.shape[0] > 1 else width


_NULL = contextlib.nullcontext()


def _on(stream, device):
    """(raw stream, context in which buffers are allocated so that they belong to it)."""
    if stream is None:
        return _current_raw_stream(device.index), _NULL
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    return stream.cuda_stream, torch.cuda.stream(stream)


# ------------------------------------------------------------------ operators
def rms_norm(x, weight=None, residual=None, *, eps: float = 1e-6, normed: bool = True, quantize: bool = False,
             residual_out: Optional[torch.Tensor] = None, stream=None):
    """y = h / sqrt(mean(h^2) + eps) * weight over the last dimension, h = x + residual.

    x, residual ``[..., D]`` (fp32 or bf16; 2-D ones may have strided rows),
    weight ``[D]``.  Returns (y, quantized, scales, h): y in x's dtype if
    ``normed``; e4m3 values and their fp32 scales ``[..., ceil(D / 128)]`` if
    ``quantize``; h in x's dtype if a residual is given, written to
    ``residual_out`` (which may be x or residual) or to a new tensor.  What is
    not asked for is None."""
    dev = _device(x, "x")
    dt = B._DTYPES.get(x.dtype)
    if dt is None or x.dim() < 1:
        raise ValueError(f"x must be float32 or bfloat16 rows: got {x.dtype}, {tuple(x.shape)}")
    if not (normed or quantize or residual is not None):
        raise ValueError("nothing to compute: normed, quantize or a residual")
    shape, dim = x.shape, x.shape[-1]
    if dim < 1:
        raise ValueError("rows must have an element")
    if x.dim() != 2:
        if not x.is_contiguous():
            raise ValueError("x must be contiguous unless it is 2-D")
        x2 = x.view(-1, dim)
    else:
        _tensor(x, "x", x.dtype, 2, dev)
        x2 = x
    rows = x2.shape[0]
    r_stride = dim
    if weight is not None:
        _dense(weight, "weight", x.dtype, (dim,), dev)
    if residual is not None:
        if residual.shape != shape:
            raise ValueError(f"residual must have x's shape {tuple(shape)}: got {tuple(residual.shape)}")
        if residual.dim() == 2:
            _tensor(residual, "residual", x.dtype, 2, dev)
            r_stride = _row_stride(residual, dim)
        else:
            _dense(residual, "residual", x.dtype, shape, dev)
    y = q = s = None
    raw, where = _on(stream, dev)
    with where:
        if residual is not None and residual_out is None:
            residual_out = torch.empty(shape, dtype=x.dtype, device=dev)
        elif residual_out is not None:
            if residual is None:
                raise ValueError("residual_out without a residual")
            _dense(residual_out, "residual_out", x.dtype, shape, dev)
        if normed:
            y = torch.empty(shape, dtype=x.dtype, device=dev)
        if quantize:
            q = torch.empty(shape, dtype=_F8, device=dev)
            s = torch.empty((*shape[:-1], (dim + 127) // 128), dtype=_F32, device=dev)
    if rows:
        rc = lib.kda_rms_norm(
            _byref(KdaNormDesc(rows, dim, dt, _row_stride(x2, dim), r_stride, eps)), x.data_ptr(),
            None if weight is None else weight.data_ptr(), None if residual is None else residual.data_ptr(),
            None if residual_out is None else residual_out.data_ptr(), y.data_ptr() if normed else None,
            q.data_ptr() if quantize else None, s.data_ptr() if quantize else None, raw)
        if rc != KDA_OK:
            raise KdaError("kda_rms_norm", rc)
    return y, q, s, residual_out


def matmul_fp8(a, a_scale, b, b_scale, *, out: Optional[torch.Tensor] = None, out_dtype=torch.bfloat16, stream=None,
               flags: int = 0):
    """c[m, n] = sum_k a[m, k] a_scale[m, k // 128] b[n, k] b_scale[n // 128, k // 128].

    a ``[M, K]``, b ``[N, K]`` e4m3 (rows may be strided), a_scale ``[M,
    ceil(K / 128)]``, b_scale ``[ceil(N / 128), ceil(K / 128)]`` fp32.  Returns c
    ``[M, N]`` in ``out_dtype`` (bf16 or fp32), or ``out`` (rows may be strided)."""
    dev = _device(a, "a")
    _tensor(a, "a", _F8, 2, dev)
    _tensor(b, "b", _F8, 2, dev)
    (m, k), (n, kb_) = a.shape, b.shape
    if kb_ != k or k < 1:
        raise ValueError(f"a and b must have rows of the same length: got {k} and {kb_}")
    kb = (k + 127) // 128
    _dense(a_scale, "a_scale", _F32, (m, kb), dev)
    _dense(b_scale, "b_scale", _F32, ((n + 127) // 128, kb), dev)
    raw, where = _on(stream, dev)
    if out is None:
        with where:
            out = torch.empty((m, n), dtype=out_dtype, device=dev)
        ldc = n
    else:
        _tensor(out, "out", out.dtype, 2, dev)
        if out.shape != (m, n):
            raise ValueError(f"out must be {(m, n)}: got {tuple(out.shape)}")
        ldc = _row_stride(out, n)
    dt = B._DTYPES.get(out.dtype)
    if dt is None:
        raise ValueError(f"the output must be float32 or bfloat16: got {out.dtype}")
    if m and n:
        rc = lib.kda_matmul_fp8(_byref(KdaMatmulDesc(m, n, k, _row_stride(a, k), _row_stride(b, k), ldc, dt, flags)),
                                a.data_ptr(), a_scale.data_ptr(), b.data_ptr(), b_scale.data_ptr(), out.data_ptr(),
                                raw)
        if rc != KDA_OK:
            raise KdaError("kda_matmul_fp8", rc)
    return out


def _latent_workspace(desc, bytes_of, name, workspace, dev):
    if workspace is None:
        n = bytes_of(_byref(desc))
        if n == 0:
            raise KdaError(name, KDA_ERR_UNSUPPORTED)
        workspace = torch.empty(n, dtype=torch.uint8, device=dev)
    desc.workspace = workspace.data_ptr()
    desc.workspace_bytes = workspace.numel() * workspace.element_size()
    return workspace


def latent_prefill(q, k_nope, k_rope, v, cu_seqlens_q=None, cu_seqlens_k=None, *, scale: float, causal: bool = True,
                   out=None, lse=None, workspace=None, stream=None, flags: int = 0):
    """Attention of packed prompts in the expanded form (kda_latent_prefill).

    q ``[Tq, H, d_k + d_rope]``, k_nope ``[Tk, H, d_k]``, k_rope ``[Tk,
    d_rope]`` shared by the heads (or None), v ``[Tk, H, d_v]``; rows and heads
    may be strided (k_nope and v may be views of one projection's output).
    Query i of a sequence sees keys 0 .. Lk - Lq + i, all without ``causal``.
    Returns (out ``[Tq, H, d_v]``, lse fp32 ``[Tq, H]``).  A caller that passes
    a ``workspace`` (uint8) can read the call's device status from it with
    ``latent_status``."""
    dev = _device(q, "q")
    dt = B._DTYPES.get(q.dtype)
    if dt is None:
        raise ValueError(f"q must be float32 or bfloat16: got {q.dtype}")
    for t, name in ((q, "q"), (k_nope, "k_nope"), (v, "v")):
        _tensor(t, name, q.dtype, 3, dev)
    tq, h, dqk = q.shape
    tk, hk, dk = k_nope.shape
    dv = v.shape[2]
    dr = 0
    if k_rope is not None:
        _tensor(k_rope, "k_rope", q.dtype, 2, dev)
        dr = k_rope.shape[1]
        if k_rope.shape[0] != tk:
            raise ValueError("k_rope must have k_nope's tokens")
    if hk != h or v.shape[0] != tk or v.shape[1] != h or dk + dr != dqk:
        raise ValueError(f"shapes do not fit: q {tuple(q.shape)}, k_nope {tuple(k_nope.shape)}, v {tuple(v.shape)}, d_rope {dr}")
    n = 1
    if (cu_seqlens_q is None) != (cu_seqlens_k is None):
        raise ValueError("both cu_seqlens or neither")
    if cu_seqlens_q is not None:
        n = cu_seqlens_q.shape[0] - 1
        _dense(cu_seqlens_q, "cu_seqlens_q", _I32, (n + 1,), dev)
        _dense(cu_seqlens_k, "cu_seqlens_k", _I32, (n + 1,), dev)
    desc = KdaLatentDesc(n, h, dt, flags if causal else flags | KDA_FLAG_NO_CAUSAL, scale, dk, dr, dv, tq, tk,
                         q.stride(0), q.stride(1), k_nope.stride(0), k_nope.stride(1), v.stride(0), v.stride(1),
                         k_rope.stride(0) if dr else 0)
    raw, where = _on(stream, dev)
    with where:
        if out is None:
            out = torch.empty((tq, h, dv), dtype=q.dtype, device=dev)
        else:
            _dense(out, "out", q.dtype, (tq, h, dv), dev)
        if lse is None:
            lse = torch.empty((tq, h), dtype=_F32, device=dev)
        else:
            _dense(lse, "lse", _F32, (tq, h), dev)
        workspace = _latent_workspace(desc, lib.kda_latent_prefill_workspace_bytes, "kda_latent_prefill", workspace,
                                      dev)
    rc = lib.kda_latent_prefill(_byref(desc), q.data_ptr(), k_nope.data_ptr(),
                                k_rope.data_ptr() if dr else None, v.data_ptr(),
                                None if cu_seqlens_q is None else cu_seqlens_q.data_ptr(),
                                None if cu_seqlens_k is None else cu_seqlens_k.data_ptr(), out.data_ptr(),
                                lse.data_ptr(), raw)
    if rc != KDA_OK:
        raise KdaError("kda_latent_prefill", rc)
    return out, lse


def latent_decode(q, cache, page_table, lengths, *, scale: float, rank: Optional[int] = None, out=None, lse=None,
                  workspace=None, stream=None, flags: int = 0):
    """Attention of the last tokens of each sequence over a paged cache of
    latents, in the absorbed form (kda_latent_decode).

    q ``[N, Lq, H, rank + d_rope]`` (or ``[N, H, rank + d_rope]`` for one query
    a sequence), cache ``[pages, page_size, rank + d_rope]`` (pages may be
    strided), page_table int32 ``[N, max_pages]``, lengths int32 ``[N]``: tokens
    of each sequence in the cache, its queries' own among them.  ``rank`` is the
    values' width, by default all but the last 64.  Returns (out ``[N, (Lq,) H,
    rank]``, lse fp32 ``[N, (Lq,) H]``)."""
    dev = _device(q, "q")
    dt = B._DTYPES.get(q.dtype)
    if dt is None:
        raise ValueError(f"q must be float32 or bfloat16: got {q.dtype}")
    single = q.dim() == 3
    _tensor(q, "q", q.dtype, 3 if single else 4, dev)
    if single:
        n, h, w = q.shape
        lq, q_ts, q_hs = 1, q.stride(0), q.stride(1)
    else:
        n, lq, h, w = q.shape
        q_ts, q_hs = q.stride(1), q.stride(2)
        if lq == 1:
            q_ts = q.stride(0)
        else:
            if n > 1 and q.stride(0) != lq * q_ts:
                raise ValueError("q's sequences and queries must form one strided dimension")
    if not (cache.dim() == 3 and cache.dtype == q.dtype and cache.device == dev and cache.shape[2] == w and cache.stride(2) == 1 and cache.stride(1) == w):
        raise ValueError(f"cache must be a [pages, page_size, {w}] {q.dtype} tensor on {dev} with dense pages")
    rank = w - 64 if rank is None else rank
    if not 1 <= rank <= w:
        raise ValueError(f"rank must be within 1 .. {w}: got {rank}")
    if page_table.dim() != 2 or page_table.shape[0] != n:
        raise ValueError(f"page_table must be [{n}, max_pages]")
    _dense(page_table, "page_table", _I32, page_table.shape, dev)
    _dense(lengths, "lengths", _I32, (n,), dev)
    pages, size = cache.shape[0], cache.shape[1]
    desc = KdaLatentDesc(n, h, dt, flags, scale, rank, w - rank, rank, 0, 0, q_ts, q_hs, 0, 0, 0, 0, 0, lq, size,
                         pages, page_table.shape[1], cache.stride(0) if pages > 1 else size * w)
    lead = (n, h) if single else (n, lq, h)
    raw, where = _on(stream, dev)
    with where:
        if out is None:
            out = torch.empty((*lead, rank), dtype=q.dtype, device=dev)
        else:
            _dense(out, "out", q.dtype, (*lead, rank), dev)
        if lse is None:
            lse = torch.empty(lead, dtype=_F32, device=dev)
        else:
            _dense(lse, "lse", _F32, lead, dev)
        workspace = _latent_workspace(desc, lib.kda_latent_decode_workspace_bytes, "kda_latent_decode", workspace,
                                      dev)
    rc = lib.kda_latent_decode(_byref(desc), q.data_ptr(), cache.data_ptr(), page_table.data_ptr(),
                               lengths.data_ptr(), out.data_ptr(), lse.data_ptr(), raw)
    if rc != KDA_OK:
        raise KdaError("kda_latent_decode", rc)
    return out, lse


def latent_status(workspace, stream=None) -> int:
    """Device status (KDA_OK, KDA_ERR_BAD_SEQLENS, KDA_ERR_BAD_PAGE, KDA_ERR_TIMEOUT) that the last
    latent_prefill or latent_decode on this workspace recorded; synchronises the stream."""
    desc = KdaLatentDesc()
    desc.workspace = workspace.data_ptr()
    desc.workspace_bytes = workspace.numel() * workspace.element_size()
    return kda_latent_status(desc, stream)


def latent_prefill_workspace_bytes(num_seqs: int, num_heads: int, dtype) -> int:
    """Bytes of a latent_prefill workspace."""
    return kda_latent_prefill_workspace_bytes(KdaLatentDesc(num_seqs, num_heads, B._DTYPES[dtype], 0, 1.0, 1, 0, 1))


def latent_decode_workspace_bytes(num_seqs: int, num_queries: int, num_heads: int, rank: int, d_rope: int, dtype,
                                  page_size: int, max_pages: int) -> int:
    """Bytes of a latent_decode workspace for these sizes (whatever the lengths)."""
    return kda_latent_decode_workspace_bytes(KdaLatentDesc(
        num_seqs, num_heads, B._DTYPES[dtype], 0, 1.0, rank, d_rope, rank, 0, 0, 0, 0, 0, 0, 0, 0, 0, num_queries,
        page_size, 1, max_pages, page_size * (rank + d_rope)))
