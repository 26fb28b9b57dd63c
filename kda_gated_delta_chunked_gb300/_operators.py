"""Norm, 8-bit products, rotary positions, latent attention and its quantised
cache: the operators around the recurrent layers (argument marshalling only; see
include/kda.h for what each computes).

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
KDA_FLAG_INTERLEAVED, KDA_FLAG_INVERSE, KDA_FLAG_POSITIONS_64 = 8, 16, 32
KDA_FLAG_CACHE_8 = 64
KDA_ROTARY_PLAIN, KDA_ROTARY_LINEAR, KDA_ROTARY_BASE, KDA_ROTARY_BY_PARTS = 0, 1, 2, 3


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


class KdaLatentCacheDesc(ctypes.Structure):
    """Mirror of ``kda_latent_cache_desc`` in include/kda.h."""
    _fields_ = [("num_seqs", ctypes.c_int32), ("dtype", ctypes.c_int32), ("total_tokens", ctypes.c_int64),
                ("rank", ctypes.c_int32), ("d_rope", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("num_pages", ctypes.c_int32), ("max_pages", ctypes.c_int32), ("flags", ctypes.c_int32),
                ("page_stride", ctypes.c_int64), ("latent_stride", ctypes.c_int64), ("rope_stride", ctypes.c_int64),
                ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t)]


class KdaRotaryPart(ctypes.Structure):
    """Mirror of ``kda_rotary_part`` in include/kda.h."""
    _fields_ = [("heads", ctypes.c_int32), ("width", ctypes.c_int32), ("offset", ctypes.c_int32),
                ("reserved", ctypes.c_int32), ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64),
                ("out_token_stride", ctypes.c_int64), ("out_head_stride", ctypes.c_int64)]


class KdaRotaryDesc(ctypes.Structure):
    """Mirror of ``kda_rotary_desc`` in include/kda.h."""
    _fields_ = [("tokens", ctypes.c_int64), ("dim", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("flags", ctypes.c_int32), ("scale", ctypes.c_float), ("x", KdaRotaryPart), ("key", KdaRotaryPart)]


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
            ("kda_selftest_drop_arrival", [ctypes.c_int32], ctypes.c_int),
            ("kda_latent_cache_page_bytes", [ctypes.c_int32] * 3, ctypes.c_size_t),
            ("kda_latent_cache_write", [ref(KdaLatentCacheDesc)] + [vp] * 7, ctypes.c_int),
            ("kda_latent_cache_read", [ref(KdaLatentCacheDesc)] + [vp] * 7, ctypes.c_int),
            ("kda_rotary", [ref(KdaRotaryDesc)] + [vp] * 7, ctypes.c_int),
            ("kda_rotary_frequencies", [ctypes.c_int32, ctypes.c_double, ctypes.c_int32] + [ctypes.c_double] * 4 + [vp],
             ctypes.c_int)):
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
            "kda_latent_prefill", "kda_latent_decode", "kda_latent_cache_page_bytes", "kda_latent_cache_write",
            "kda_latent_cache_read", "kda_rotary")))
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


def kda_latent_cache_page_bytes(page_size: int, rank: int, d_rope: int) -> int:
    return lib.kda_latent_cache_page_bytes(page_size, rank, d_rope)


def kda_latent_cache_write(desc: KdaLatentCacheDesc, latents, rope, cu_seqlens, page_table, lengths, cache,
                           stream=None) -> int:
    """Raw C call that quantises rows into the pages of a cache."""
    p = B._p
    return lib.kda_latent_cache_write(_byref(desc), p(latents), p(rope), p(cu_seqlens), p(page_table), p(lengths),
                                      p(cache), B._stream(stream))


def kda_latent_cache_read(desc: KdaLatentCacheDesc, cache, page_table, lengths, cu_seqlens, latents, rope,
                          stream=None) -> int:
    """Raw C call that reads rows out of the pages of a cache."""
    p = B._p
    return lib.kda_latent_cache_read(_byref(desc), p(cache), p(page_table), p(lengths), p(cu_seqlens), p(latents),
                                     p(rope), B._stream(stream))


def kda_rotary(desc: KdaRotaryDesc, x, key, positions, frequencies, out, key_out, stream=None) -> int:
    """Raw C call of the rotary positions."""
    p = B._p
    return lib.kda_rotary(_byref(desc), p(x), p(key), p(positions), p(frequencies), p(out), p(key_out),
                          B._stream(stream))


def kda_rotary_frequencies(dim: int, base: float, method: int, factor: float, original_length: float, slow: float,
                           fast: float, frequencies) -> int:
    """Raw C call; frequencies: a ctypes array of dim / 2 doubles (host memory)."""
    return lib.kda_rotary_frequencies(dim, base, method, factor, original_length, slow, fast,
                                      None if frequencies is None else ctypes.cast(frequencies, ctypes.c_void_p))


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


def latent_decode(q, cache, page_table, lengths, *, scale: float, rank: Optional[int] = None,
                  page_size: Optional[int] = None, out=None, lse=None, workspace=None, stream=None, flags: int = 0):
    """Attention of the last tokens of each sequence over a paged cache of
    latents, in the absorbed form (kda_latent_decode).

    q ``[N, Lq, H, rank + d_rope]`` (or ``[N, H, rank + d_rope]`` for one query
    a sequence), cache ``[pages, page_size, rank + d_rope]`` (pages may be
    strided), page_table int32 ``[N, max_pages]``, lengths int32 ``[N]``: tokens
    of each sequence in the cache, its queries' own among them.  ``rank`` is the
    values' width, by default all but the last 64.  Returns (out ``[N, (Lq,) H,
    rank]``, lse fp32 ``[N, (Lq,) H]``).  The softmax weights are held as in
    ``latent_prefill``.

    A uint8 cache ``[pages, latent_cache_page_bytes(...)]`` with its
    ``page_size`` is a quantised one (``latent_cache_write``).  In bf16, queries
    and softmax weights then meet its codes as sums of two and three 8-bit
    values (include/kda.h); fp32 queries stay in fp32."""
    return _call("latent_decode", stream, q, cache, page_table, lengths, scale, -1 if rank is None else rank, flags, out,
                 lse, workspace, page_size)


def latent_cache_page_bytes(page_size: int, rank: int = 512, d_rope: int = 64) -> int:
    """Bytes of a page of the quantised cache: a cache is ``torch.empty(pages, these bytes, dtype=torch.uint8)``."""
    n = kda_latent_cache_page_bytes(page_size, rank, d_rope)
    if n == 0:
        raise ValueError(f"a quantised cache has pages of at least one token, ranks that are multiples of 16 up to 512 and "
                         f"d_rope of 8 up to 128: got {page_size}, {rank}, {d_rope}")
    return n


def latent_cache_write(latents, rope, cache, page_table, lengths, cu_seqlens=None, *, page_size: int, workspace=None,
                       stream=None) -> None:
    """Quantises the last tokens of each sequence into the pages of ``cache``:
    e4m3 codes under a power of two for each token (kda_latent_cache_write).

    latents ``[T, rank]``, rope ``[T, d_rope]`` or None (fp32 or bf16; rows may
    be strided): sequence n's are rows cu_seqlens[n] .. cu_seqlens[n + 1] - 1,
    or T / N rows each.  cache uint8 ``[pages, latent_cache_page_bytes(...)]``
    (pages may be strided), page_table and lengths as for ``latent_decode``:
    lengths count the new tokens.  A caller that passes a ``workspace`` (uint8,
    256 bytes) can read the call's device status from it with
    ``latent_status``."""
    _call("latent_cache_write", stream, latents, rope, cache, page_table, lengths, cu_seqlens, page_size, workspace)


def latent_cache_read(cache, page_table, lengths, cu_seqlens=None, *, total_tokens: int, page_size: int, rank: int = 512,
                      d_rope: int = 64, dtype=torch.bfloat16, latents=None, rope=None, workspace=None, stream=None):
    """Reads the last tokens of each sequence back out of a quantised cache
    (kda_latent_cache_read): the ones that ``latent_cache_write`` with the same
    lengths and cu_seqlens would write.  With cu_seqlens made of the lengths,
    the whole sequences.

    Returns (latents ``[total_tokens, rank]``, rope ``[total_tokens, d_rope]`` or
    None) in ``dtype`` (exact in fp32 and bf16), or in the tensors given (rows
    may be strided).  Rows of no sequence are left as they were."""
    if dtype is not torch.bfloat16 and dtype is not torch.float32:
        raise ValueError(f"the output must be float32 or bfloat16: got {dtype}")
    return _call("latent_cache_read", stream, cache, page_table, lengths, cu_seqlens, total_tokens, page_size, rank,
                 d_rope, dtype is torch.bfloat16, latents, rope, workspace)


def rotary_frequencies(dim: int, *, base: float = 10000.0, method: int = KDA_ROTARY_PLAIN, factor: float = 1.0,
                       original_length: float = 4096, slow: float = 1.0, fast: float = 32.0, device=None) -> torch.Tensor:
    """Frequencies fp64 ``[dim / 2]`` for ``rotary``, in radians a position:
    base^(-2 i / dim), scaled for contexts ``factor`` times as long as
    ``original_length`` by a KDA_ROTARY_* method (kda_rotary_frequencies).
    KDA_ROTARY_BY_PARTS blends by the turns that a pair made in training, not by
    its index: frequencies of models that do so are the caller's to make."""
    host = (ctypes.c_double * max(1, dim // 2))()
    status = kda_rotary_frequencies(dim, base, method, factor, original_length, slow, fast, host)
    if status != B.KDA_OK:
        raise KdaError("kda_rotary_frequencies", status)
    return torch.tensor(list(host), dtype=torch.float64, device="cuda" if device is None else device)


def rotary(x, positions, frequencies, *, key=None, offset: Optional[int] = None, key_offset: Optional[int] = None,
           interleaved: bool = False, inverse: bool = False, scale: float = 1.0, out=None, key_out=None, stream=None):
    """Turns pairs of channels by position * frequency (kda_rotary).

    x ``[T, heads, channels]`` or ``[T, channels]`` (fp32 or bf16; tokens and
    heads may be strided), positions int32 or int64 ``[T]``, frequencies fp64
    ``[dim / 2]`` (``rotary_frequencies``).  The dim channels from ``offset`` on
    are turned, by default the last ones, the others copied; pairs are
    neighbours if ``interleaved``, else half of dim apart.  ``key`` (its own
    heads and channels, from ``key_offset`` on) goes along in the same launch.
    ``inverse`` turns the other way: the gradient of x from that of the output.
    Results are ``scale`` times the turned channels.  ``out`` may be x, and
    ``key_out`` key.  Returns (out, key_out)."""
    flags = (KDA_FLAG_INTERLEAVED if interleaved else 0) | (KDA_FLAG_INVERSE if inverse else 0)
    return _call("rotary", stream, x, positions, frequencies, key, offset, key_offset, scale, flags, out, key_out)


def latent_status(workspace, stream=None) -> int:
    """Device status (KDA_OK, KDA_ERR_BAD_SEQLENS, KDA_ERR_BAD_PAGE, KDA_ERR_TIMEOUT) that the last
    latent_* call on this workspace recorded; synchronises the stream."""
    desc = KdaLatentDesc()
    desc.workspace = workspace.data_ptr()
    desc.workspace_bytes = workspace.numel() * workspace.element_size()
    return kda_latent_status(desc, stream)


def latent_prefill_workspace_bytes(num_seqs: int, num_heads: int, dtype) -> int:
    """Bytes of a latent_prefill workspace."""
    return kda_latent_prefill_workspace_bytes(KdaLatentDesc(num_seqs, num_heads, B._DTYPES[dtype], 0, 1.0, 1, 0, 1))


def latent_decode_workspace_bytes(num_seqs: int, num_queries: int, num_heads: int, rank: int, d_rope: int, dtype,
                                  page_size: int, max_pages: int, quantized: bool = False) -> int:
    """Bytes of a latent_decode workspace for these sizes (whatever the lengths); quantized: over a quantised cache."""
    pages = kda_latent_cache_page_bytes(page_size, rank, d_rope) if quantized else page_size * (rank + d_rope)
    return kda_latent_decode_workspace_bytes(KdaLatentDesc(
        num_seqs, num_heads, B._DTYPES[dtype], KDA_FLAG_CACHE_8 if quantized else 0, 1.0, rank, d_rope, rank, 0, 0, 0, 0,
        0, 0, 0, 0, 0, num_queries, page_size, 1, max_pages, pages))
