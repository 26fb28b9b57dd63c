"""Norm, 8-bit products and latent attention: the operators around the recurrent
layers (argument marshalling only; see include/kda.h for what each computes).

Work goes to the current stream, or to a given ``stream`` (a torch stream or a
handle), where it is ordered behind that stream's work alone: the caller lets
that stream wait for whatever wrote the inputs, and the reader of the outputs
wait for it.  The memory of the inputs is kept until the stream has read them,
also if the caller drops them at once; the outputs are allocated on it."""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os
import threading
from typing import Optional

import torch

from . import _binding as B
from ._binding import KdaError, lib, library_path

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
            ("kda_latent_status", [ref(KdaLatentDesc), vp], ctypes.c_int),
            ("kda_selftest_drop_arrival", [ctypes.c_int32], ctypes.c_int)):
        f = getattr(lib, name)
        f.argtypes, f.restype = args, res


_declare()
_byref = ctypes.byref


_native = None
_native_lock = threading.Lock()


def _load_native():
    """The compiled marshalling (csrc/kda_torch.cpp), bound to the entry points of the loaded library; from beside that
    library, or from this package.  It is loaded by the first operator that is called: it belongs to one Python and one
    torch, which the other calls of the package do not need."""
    global _native
    with _native_lock:
        if _native is not None:
            return _native
        places = [os.path.dirname(os.path.abspath(library_path())), os.path.join(os.path.dirname(os.path.abspath(__file__)), "_build")]
        paths = [os.path.join(p, "_kda_torch.so") for p in places]
        path = next((p for p in paths if os.path.exists(p)), None)
        if path is None:
            raise ImportError(f"_kda_torch.so not built at {paths[-1]}: run "
                              f"`python -c 'import __graft_entry__ as g; g.build()'` first")
        loader = importlib.machinery.ExtensionFileLoader("_kda_torch", path)
        module = importlib.util.module_from_spec(importlib.util.spec_from_loader("_kda_torch", loader))
        loader.exec_module(module)
        module.bind(*(ctypes.cast(getattr(lib, name), ctypes.c_void_p).value for name in (
            "kda_rms_norm", "kda_matmul_fp8", "kda_latent_prefill_workspace_bytes", "kda_latent_decode_workspace_bytes",
            "kda_latent_prefill", "kda_latent_decode")))
        _native = module
        return module


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


def kda_selftest_drop_arrival(which: int) -> int:
    """Lets waits of later calls run out (1 .. 5, see include/kda.h); 0 ends it."""
    return lib.kda_selftest_drop_arrival(which)


# ------------------------------------------------------------------ operators
def _call(name: str, stream, *args):
    """The native call on the current stream or on ``stream``, see above."""
    native = _native or _load_native()
    if stream is None:
        r = getattr(native, name)(*args)
    else:
        if not hasattr(stream, "cuda_stream"):
            stream = torch.cuda.ExternalStream(int(stream))
        with torch.cuda.stream(stream):
            r = getattr(native, name)(*args)
        for t in args:                                    # the allocator gives none of them away before the stream is there
            if isinstance(t, torch.Tensor):
                t.record_stream(stream)
    if type(r) is int:
        raise KdaError(f"kda_{name}", r)
    return r


def rms_norm(x, weight=None, residual=None, *, eps: float = 1e-6, normed: bool = True, quantize: bool = False,
             residual_out: Optional[torch.Tensor] = None, stream=None):
    """y = h / sqrt(mean(h^2) + eps) * weight over the last dimension, h = x + residual.

    x, residual ``[..., D]`` (fp32 or bf16; 2-D ones may have strided rows),
    weight ``[D]``.  Returns (y, quantized, scales, h): y in x's dtype if
    ``normed``; e4m3 values and their fp32 scales ``[..., ceil(D / 128)]`` if
    ``quantize``; h in x's dtype if a residual is given, written to
    ``residual_out`` (which may be x or residual) or to a new tensor.  What is
    not asked for is None."""
    return _call("rms_norm", stream, x, weight, residual, eps, normed, quantize, residual_out)


def matmul_fp8(a, a_scale, b, b_scale, *, out: Optional[torch.Tensor] = None, out_dtype=torch.bfloat16, stream=None,
               flags: int = 0):
    """c[m, n] = sum_k a[m, k] a_scale[m, k // 128] b[n, k] b_scale[n // 128, k // 128].

    a ``[M, K]``, b ``[N, K]`` e4m3 (rows may be strided), a_scale ``[M,
    ceil(K / 128)]``, b_scale ``[ceil(N / 128), ceil(K / 128)]`` fp32.  Returns c
    ``[M, N]`` in ``out_dtype`` (bf16 or fp32), or ``out`` (rows may be strided)."""
    if out_dtype is not torch.bfloat16 and out_dtype is not torch.float32:
        raise ValueError(f"the output must be float32 or bfloat16: got {out_dtype}")
    return _call("matmul_fp8", stream, a, a_scale, b, b_scale, out, out_dtype is torch.bfloat16, flags)


def latent_prefill(q, k_nope, k_rope, v, cu_seqlens_q=None, cu_seqlens_k=None, *, scale: float, causal: bool = True,
                   out=None, lse=None, workspace=None, stream=None, flags: int = 0):
    """Attention of packed prompts in the expanded form (kda_latent_prefill).

    q ``[Tq, H, d_k + d_rope]``, k_nope ``[Tk, H, d_k]``, k_rope ``[Tk,
    d_rope]`` shared by the heads (or None), v ``[Tk, H, d_v]``; rows and heads
    may be strided (k_nope and v may be views of one projection's output).
    Query i of a sequence sees keys 0 .. Lk - Lq + i, all without ``causal``.
    Returns (out ``[Tq, H, d_v]``, lse fp32 ``[Tq, H]``).  A caller that passes
    a ``workspace`` (uint8) can read the call's device status from it with
    ``latent_status``.  In bf16 the softmax weights are rounded to bf16 before
    they meet the values, fp32 inputs keep them in fp32 (include/kda.h)."""
    return _call("latent_prefill", stream, q, k_nope, k_rope, v, cu_seqlens_q, cu_seqlens_k, scale,
                 flags if causal else flags | KDA_FLAG_NO_CAUSAL, out, lse, workspace)


def latent_decode(q, cache, page_table, lengths, *, scale: float, rank: Optional[int] = None, out=None, lse=None,
                  workspace=None, stream=None, flags: int = 0):
    """Attention of the last tokens of each sequence over a paged cache of
    latents, in the absorbed form (kda_latent_decode).

    q ``[N, Lq, H, rank + d_rope]`` (or ``[N, H, rank + d_rope]`` for one query
    a sequence), cache ``[pages, page_size, rank + d_rope]`` (pages may be
    strided), page_table int32 ``[N, max_pages]``, lengths int32 ``[N]``: tokens
    of each sequence in the cache, its queries' own among them.  ``rank`` is the
    values' width, by default all but the last 64.  Returns (out ``[N, (Lq,) H,
    rank]``, lse fp32 ``[N, (Lq,) H]``).  The softmax weights are held as in
    ``latent_prefill``."""
    return _call("latent_decode", stream, q, cache, page_table, lengths, scale, -1 if rank is None else rank, flags, out,
                 lse, workspace)


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
