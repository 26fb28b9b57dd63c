"""Refusals of the quantised cache and the rotary positions by the C entries,
before any CUDA work, and the frequencies, which are host work."""
import ctypes
import math
import os
import subprocess

import pytest
import torch

kda = pytest.importorskip("kda_gated_delta_chunked_gb300", reason="libkda.so not built (run __graft_entry__.build())")
from test_operators_host import BAD, P, UNSUP, WS, Ptr, latent  # noqa: E402

OK = kda.KDA_OK


def test_struct_sizes_match_the_header(tmp_path):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    c = tmp_path / "s.c"
    c.write_text('#include <stdio.h>\n#include "kda.h"\nint main(void){printf("%zu %zu %zu %zu %zu", sizeof(kda_latent_cache_desc),'
                 'offsetof(kda_latent_cache_desc, workspace), sizeof(kda_rotary_part), sizeof(kda_rotary_desc), offsetof(kda_rotary_desc, key));'
                 'return 0;}\n')
    subprocess.run(["gcc", "-I", os.path.join(root, "include"), str(c), "-o", str(tmp_path / "s")], check=True)
    got = [int(x) for x in subprocess.run([str(tmp_path / "s")], capture_output=True, text=True, check=True).stdout.split()]
    C, R = kda.KdaLatentCacheDesc, kda.KdaRotaryDesc
    assert got == [ctypes.sizeof(C), C.workspace.offset, ctypes.sizeof(kda.KdaRotaryPart), ctypes.sizeof(R), R.key.offset]


def test_page_bytes():
    assert kda.latent_cache_page_bytes(64) == 64 * 640 + 128 and kda.latent_cache_page_bytes(1, 16, 0) == 128
    assert kda.latent_cache_page_bytes(1 << 24, 512, 128) == (1 << 24) * 769
    for bad in ((0, 512, 64), (64, 500, 64), (64, 528, 64), (64, 0, 64), (64, 512, 4), (64, 512, 136), (64, 512, -8), (-1, 512, 64)):
        assert kda.kda_latent_cache_page_bytes(*bad) == 0
        with pytest.raises(ValueError):
            kda.latent_cache_page_bytes(*bad)


def cache_call(write, lat=P[0], rope=P[1], cu=P[2], table=P[3], lens=P[4], cache=P[5], **kw):
    f = dict(num_seqs=2, dtype=kda.KDA_BF16, total_tokens=10, rank=512, d_rope=64, page_size=64, num_pages=10, max_pages=5, flags=0,
             page_stride=41088, latent_stride=576, rope_stride=576, workspace=None, workspace_bytes=0)
    f.update(kw)
    d = kda.KdaLatentCacheDesc(**f)
    return (kda.kda_latent_cache_write(d, lat, rope, cu, table, lens, cache, 0) if write
            else kda.kda_latent_cache_read(d, cache, table, lens, cu, lat, rope, 0))


@pytest.mark.parametrize("write", [False, True])
def test_cache_refusals(write):
    def call(**kw):
        return cache_call(write, **kw)
    assert call(num_seqs=-1) == BAD and call(dtype=2) == BAD and call(total_tokens=-1) == BAD and call(flags=1) == BAD
    assert call(page_size=0) == BAD and call(num_pages=-1) == BAD and call(max_pages=0) == BAD and call(rank=0) == BAD and call(d_rope=-8) == BAD
    assert call(rank=500) == UNSUP and call(rank=528, latent_stride=528) == UNSUP and call(d_rope=4) == UNSUP and call(d_rope=136, rope_stride=136) == UNSUP
    assert call(max_pages=1 << 30) == UNSUP and call(total_tokens=1 << 31) == UNSUP
    assert call(page_stride=41087) == BAD and call(page_stride=41088 + 8) == BAD and call(page_stride=-41088) == BAD
    assert call(latent_stride=511) == BAD and call(rope_stride=63) == BAD
    assert call(cu=None, total_tokens=11) == BAD and call(cu=None, num_seqs=0) == BAD
    assert call(lat=None) == BAD and call(rope=None) == BAD and call(table=None) == BAD and call(lens=None) == BAD and call(cache=None) == BAD
    assert call(d_rope=0, rope_stride=0, page_stride=32896) == BAD                       # rotary rows without channels
    assert call(lat=P[0] + 1) == BAD and call(rope=P[1] + 1) == BAD and call(cu=P[2] + 2) == BAD and call(table=P[3] + 1) == BAD
    assert call(cache=P[5] + 8) == BAD and call(lens=P[4] + 2) == BAD
    assert call(lat=P[5] + 1024) == BAD and call(rope=P[5]) == BAD                        # rows inside the cache
    assert call(workspace=P[9].addr, workspace_bytes=8) == WS and call(workspace=P[9].addr + 8, workspace_bytes=512) == WS
    for over in (P[0], P[3], P[4], P[5]):
        assert call(workspace=over.addr, workspace_bytes=256) == BAD
    assert call(num_seqs=0) == OK and call(total_tokens=0, lat=None, rope=None) == OK and call(cu=None, total_tokens=0) == OK
    if write:
        assert call(cu=P[5] + 64) == BAD and call(lens=P[5] + 64) == BAD and call(table=P[5]) == BAD
    else:
        assert call(cu=P[0] + 64) == BAD and call(lens=P[1]) == BAD
        assert call(rope=P[0] + 2 * 511) == BAD                                          # the two outputs overlap


def test_decode_refusals_over_the_quantised_cache():
    def call(q=P[0], cache=P[1], table=P[2], lens=P[3], out=P[4], lse=P[5], **kw):
        f = dict(d_k=512, d_rope=64, d_v=512, q_token_stride=4 * 576, q_head_stride=576, num_queries=1, page_size=64, num_pages=10,
                 max_pages=5, page_stride=41088, flags=kda.KDA_FLAG_CACHE_8)
        f.update(kw)
        return kda.kda_latent_decode(latent(**f), q, cache, table, lens, out, lse, 0)
    assert call(page_stride=41072) == BAD and call(page_stride=41089) == BAD and call(cache=P[1] + 8) == BAD
    assert call(d_k=500, d_v=500) == UNSUP and call(d_rope=4) == UNSUP and call(d_v=256) == BAD
    assert call(flags=kda.KDA_FLAG_CACHE_8 | kda.KDA_FLAG_NO_CAUSAL) == BAD and call(flags=128) == BAD
    assert call(out=P[1] + 64) == BAD and call(out=P[1] + 9 * 41088 + 41080) == BAD and call(workspace=None) == WS and call(workspace_bytes=8) == WS
    assert call(num_seqs=0) == OK
    # prompts have no such cache
    assert kda.kda_latent_prefill(latent(flags=kda.KDA_FLAG_CACHE_8), *P[:8], 0) == BAD


def rot(x=P[0], key=P[1], pos=P[2], f=P[3], out=P[4], key_out=P[5], part=None, key_part=None, **kw):
    one = dict(heads=4, width=192, offset=128, reserved=0, token_stride=768, head_stride=192, out_token_stride=768, out_head_stride=192)
    two = dict(heads=1, width=64, offset=0, reserved=0, token_stride=64, head_stride=64, out_token_stride=64, out_head_stride=64)
    one.update(part or {})
    two.update(key_part or {})
    d = dict(tokens=10, dim=64, dtype=kda.KDA_BF16, flags=0, scale=1.0, x=kda.KdaRotaryPart(**one), key=kda.KdaRotaryPart(**two))
    d.update(kw)
    return kda.kda_rotary(kda.KdaRotaryDesc(**d), x, key, pos, f, out, key_out, 0)


def test_rotary_refusals():
    assert rot(tokens=-1) == BAD and rot(dim=0) == BAD and rot(dim=63) == BAD and rot(dtype=2) == BAD and rot(flags=1) == BAD and rot(flags=64) == BAD
    assert rot(scale=float("nan")) == BAD and rot(scale=float("inf")) == BAD
    for p in (dict(heads=0), dict(reserved=1), dict(offset=-1), dict(offset=129), dict(width=63, offset=0), dict(token_stride=-1), dict(head_stride=-1),
              dict(out_token_stride=767), dict(out_head_stride=191), dict(out_head_stride=0), dict(out_token_stride=0), dict(offset=2 ** 31 - 1)):
        assert rot(part=p) == BAD, p
    assert rot(key_part=dict(width=32)) == BAD and rot(key_part=dict(out_token_stride=63)) == BAD
    assert rot(part=dict(heads=65536, token_stride=1 << 24, out_token_stride=1 << 24)) == UNSUP and rot(part=dict(width=4097, out_head_stride=4097, out_token_stride=20000)) == UNSUP
    assert rot(dim=1026, part=dict(width=1026, offset=0, out_head_stride=1026, out_token_stride=5000), key_part=dict(width=1026, out_token_stride=1026)) == UNSUP
    assert rot(tokens=1 << 31) == UNSUP and rot(part=dict(token_stride=1 << 60)) == UNSUP
    assert rot(x=None) == BAD and rot(out=None) == BAD and rot(pos=None) == BAD and rot(f=None) == BAD and rot(key=None) == BAD and rot(key_out=None) == BAD
    assert rot(x=P[0] + 1) == BAD and rot(pos=P[2] + 2) == BAD and rot(f=P[3] + 4) == BAD and rot(pos=P[2] + 4, flags=kda.KDA_FLAG_POSITIONS_64) == BAD
    assert rot(out=P[0] + 64) == BAD and rot(out=P[1]) == BAD and rot(key_out=P[0]) == BAD and rot(key_out=P[4] + 128) == BAD
    assert rot(out=P[0], part=dict(out_token_stride=800)) == BAD                        # its own input, with other strides
    assert rot(out=P[2]) == BAD and rot(key_out=P[3]) == BAD
    assert rot(tokens=0, x=None, key=None, pos=None, f=None, out=None, key_out=None) == OK
    # queries and key of one projection, 832 channels a token, do not meet (tests on the GPU); a channel to either side they do
    wide = dict(token_stride=832, out_token_stride=832)
    over = lambda at: rot(out=P[0], key_out=P[0] + 2 * at, key=P[0] + 2 * at, part=wide, key_part=wide)  # noqa: E731
    assert over(767) == BAD and over(769) == BAD


def frequencies(dim, **kw):
    a = dict(base=10000.0, method=kda.KDA_ROTARY_PLAIN, factor=1.0, original_length=4096.0, slow=1.0, fast=32.0)
    a.update(kw)
    out = (ctypes.c_double * max(1, dim // 2))()
    rc = kda.kda_rotary_frequencies(dim, a["base"], a["method"], a["factor"], a["original_length"], a["slow"], a["fast"], out)
    return rc, list(out)


@pytest.mark.parametrize("dim", [2, 16, 64, 128, 1024])
def test_frequencies(dim):
    """pow and a few operations of 64 bits: 8 roundings at most."""
    near = lambda a, b: all(abs(x - y) <= 8 * 2.0 ** -53 * abs(y) for x, y in zip(a, b)) and len(a) == len(b) == dim // 2  # noqa: E731
    plain = [10000.0 ** (-2 * i / dim) for i in range(dim // 2)]
    assert frequencies(dim)[0] == OK and near(frequencies(dim)[1], plain)
    assert near(frequencies(dim, method=kda.KDA_ROTARY_LINEAR, factor=8.0)[1], [f / 8 for f in plain])
    rc, got = frequencies(dim, method=kda.KDA_ROTARY_BASE, factor=8.0)
    if dim == 2:
        assert rc == BAD
    else:
        assert got[0] == 1.0 and abs(got[-1] - plain[-1] / 8) <= 200 * 2.0 ** -53 * got[-1]       # (the exponent's rounding, times log)
        assert all(x <= y for x, y in zip(got, plain))
    rc, got = frequencies(dim, method=kda.KDA_ROTARY_BY_PARTS, factor=32.0)
    for f, x in zip(plain, got):
        turns = 4096 * f / (2 * math.pi)
        w = min(1.0, max(0.0, (turns - 1) / 31))
        assert abs(x - f * (w + (1 - w) / 32)) <= 2.0 ** -45 * f
        assert x == f or turns < 32 + 1e-9
    assert torch.equal(kda.rotary_frequencies(dim, device="cpu"), torch.tensor(frequencies(dim)[1], dtype=torch.float64))


def test_frequency_refusals():
    for kw in (dict(dim=0), dict(dim=7), dict(dim=-2), dict(base=0.0), dict(base=-1.0), dict(base=math.nan), dict(base=math.inf), dict(method=-1),
               dict(method=4), dict(method=1, factor=0.0), dict(method=2, factor=math.inf), dict(method=3, factor=2.0, original_length=0.0),
               dict(method=3, factor=2.0, slow=32.0), dict(method=3, factor=2.0, fast=math.inf), dict(method=3, slow=-1.0)):
        kw = dict(kw)
        assert frequencies(kw.pop("dim", 64), **kw)[0] == BAD, kw
    assert frequencies(1026)[0] == UNSUP
    assert kda.kda_rotary_frequencies(64, 1e4, 0, 1.0, 1.0, 1.0, 2.0, None) == BAD
    with pytest.raises(kda.KdaError):
        kda.rotary_frequencies(7, device="cpu")


def test_python_refusals():
    """What the torch layer turns back: here, anything that is not on a CUDA device."""
    x = torch.zeros(4, 512)
    for call in (lambda: kda.rotary(x, x, x), lambda: kda.latent_cache_write(x, x, x, x, x, page_size=64),
                 lambda: kda.latent_cache_read(x, x, x, total_tokens=1, page_size=64)):
        with pytest.raises(ValueError):
            call()


def test_nothing_of_a_device_is_kept_for_the_process():
    """Functions' plain statics would be the first device's: attributes of kernels, blocks that run at once."""
    import re
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    for name in ("kda_latent_decode8_tc.cu", "kda_latent_cache.cu", "kda_rotary.cu", "kda_launch.cuh", "kda_latent_decode.cuh"):
        text = open(os.path.join(root, "kda_gated_delta_chunked_gb300", "csrc", name)).read()
        found = re.findall(r"^ {4,}static (?!constexpr|__device__)(\w+)", text, re.M)
        assert set(found) <= {"PerDevice"}, (name, found)
