"""The quantised cache and attention over it where a call is unusual: values that
are no numbers, scales far apart, waits that run out, workspaces, streams, graphs,
contexts, and what lies beside the outputs."""
import math
import os
import subprocess
import sys

import pytest
import torch

import latent_cache_ref as cref
import operators_ref as ref
from operators_ref import F
from test_gpu_latent_cache import cached, compare, ints, latents, place, tables
from test_gpu_operators import BF16, F32, kda, normal, within  # noqa: F401
from test_gpu_operators_edges import dropped, runs_out  # noqa: F401

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NAN, INF = float("nan"), float("inf")
FORMS = [(BF16, False), (BF16, True), (F32, True)]          # tensor cores, CUDA cores, CUDA cores


def workspace(kda, n, lq, h, page, table, fill=0):  # noqa: F811
    size = kda.latent_decode_workspace_bytes(n, lq, h, 512, 64, BF16, page, table.shape[1], quantized=True)
    return torch.full((size,), fill, dtype=torch.uint8, device="cuda")


# ------------------------------------------------------------------ many tiles
@pytest.mark.parametrize("lens,lq,h,page", [([45000], 1, 32, 64), ([1500] * 70, 1, 16, 64), ([2100, 0, 1, 3333] * 14, 1, 32, 16),
                                            ([1900] * 40, 3, 16, 32), ([2500] * 30, 1, 100, 64), ([128] * 400, 1, 20, 128), ([129, 127] * 200, 1, 4, 8)])
def test_decode_many_tiles_a_block(kda, lens, lq, h, page):  # noqa: F811
    """Several tiles and sequences a thread block; pages hold NaN codes behind each sequence's length."""
    cache, table, seqs = cached(kda, lens, page, 512, 64, 31)
    q = normal(32, len(lens), lq, h, 576, dtype=BF16)
    L, ws = ints(*lens), workspace(kda, len(lens), lq, h, page, table)
    go = lambda **kw: kda.latent_decode(q.cuda(), cache, table, L, scale=0.0722, page_size=page, **kw)  # noqa: E731
    out, lse = go(workspace=ws)
    assert kda.latent_status(ws) == kda.KDA_OK
    again, lse2 = go()
    assert torch.equal(out, again) and torch.equal(lse, lse2) and torch.isfinite(out.float()).all()
    simt, slse = go(flags=kda.KDA_FLAG_CUDA_CORE_PREFILL)
    compare(q, seqs, out, lse, lens, lq, h, 512, 0.0722, BF16, True, rows=[0, h - 1], seqs_at={0, 1, len(lens) // 2, len(lens) - 1})
    # every row against the CUDA cores' form: both round the output, one its weights
    off = (out.float() - simt.float()).norm(dim=-1) / simt.float().norm(dim=-1).clamp_min(1e-20)
    assert float(off.max()) < 3 * 2.0 ** -8, float(off.max())
    some = torch.isfinite(slse)
    assert torch.equal(torch.isfinite(lse), some) and float((lse - slse)[some].abs().max()) < 1e-4


# ------------------------------------------------------------------ scales far apart, small weights
def by_hand(kda, c, r, page=64):  # noqa: F811
    """A cache of one sequence written from latents and rotary channels, its table, and its keys in 64 bits."""
    n = c.shape[0]
    table, pages = tables([n], page, 1)
    cache = torch.zeros(pages, kda.latent_cache_page_bytes(page), dtype=torch.uint8, device="cuda")
    kda.latent_cache_write(c.cuda(), r.cuda(), cache, table.cuda(), ints(n), page_size=page)
    v, e = cref.quantise(c)
    return cache, table.cuda(), torch.cat([v * torch.exp2(e.to(F))[:, None], r.to(BF16).to(F)], 1)


@pytest.mark.parametrize("simt", [False, True])
@pytest.mark.parametrize("spread", [3, 20, 30])
def test_decode_of_tokens_of_different_size(kda, simt, spread):  # noqa: F811
    """Latents from 2^-spread to 2^spread: a token's weight meets its scale, the largest product sets the reference."""
    n, h = 500, 16
    size = torch.exp2(torch.linspace(-spread, spread, n)[torch.randperm(n, generator=torch.Generator().manual_seed(2))])
    c = (normal(1, n, 512) * size[:, None]).to(BF16)
    r = normal(3, n, 64, dtype=BF16)
    cache, table, keys = by_hand(kda, c, r)
    q = normal(4, 1, 1, h, 576, dtype=BF16)
    q[..., :512] *= 2.0 ** -spread
    out, lse = kda.latent_decode(q.cuda(), cache, table, ints(n), scale=0.07, page_size=64, flags=kda.KDA_FLAG_CUDA_CORE_PREFILL if simt else 0)
    compare(q, [keys], out, lse, [n], 1, h, 512, 0.07, BF16, not simt)


@pytest.mark.parametrize("simt", [False, True])
def test_decode_of_zeros_and_of_the_smallest_and_largest_latents(kda, simt):  # noqa: F811
    for c in (torch.zeros(200, 512), torch.full((200, 512), 2.0 ** -120), torch.full((200, 512), 2.0 ** 100),
              torch.cat([torch.zeros(100, 512), torch.ones(100, 512)])):
        c = c.to(BF16)
        r = normal(3, 200, 64, dtype=BF16)
        cache, table, keys = by_hand(kda, c, r)
        q = normal(4, 1, 1, 16, 576, dtype=BF16)
        q[..., :512] = 0
        out, lse = kda.latent_decode(q.cuda(), cache, table, ints(200), scale=0.07, page_size=64, flags=kda.KDA_FLAG_CUDA_CORE_PREFILL if simt else 0)
        compare(q, [keys], out, lse, [200], 1, 16, 512, 0.07, BF16, not simt)


@pytest.mark.parametrize("n,below", [(60000, 10.0), (60000, 13.3), (20000, 17.7)])
def test_decode_many_small_weights_behind_a_dominant_one(kda, n, below):  # noqa: F811
    """A first token with 2^below times every other's weight: together the others are a good part of the sum, and equal
    weights are rounded the same way.  An exponent of the bound: 2^-8.6 of each."""
    c = torch.ones(n, 512) * 0.37
    c[0] = -1.3
    r = torch.zeros(n, 64)
    r[0, 0] = 1.0
    cache, table, keys = by_hand(kda, c.to(BF16), r.to(BF16))
    q = torch.zeros(1, 1, 16, 576)
    q[..., 512] = below * math.log(2) / 0.125
    q = (q + normal(5, 1, 1, 16, 576, scale=0.01)).to(BF16)
    out, lse = kda.latent_decode(q.cuda(), cache, table, ints(n), scale=0.125, page_size=64)
    compare(q, [keys], out, lse, [n], 1, 16, 512, 0.125, BF16, True, rows=[0, 7, 15])


def test_decode_references_that_keep_growing(kda):  # noqa: F811
    """Scores that rise from tile to tile by more than the references' slack, in some rows, and fall in others."""
    n, h = 2000, 32
    c, r = normal(1, n, 512, dtype=BF16), torch.zeros(n, 64)
    r[:, 0] = torch.arange(n) / 128
    r[:, 1] = 1 - torch.arange(n) / 128
    cache, table, keys = by_hand(kda, c, r.to(BF16))
    q = normal(4, 1, 1, h, 576, dtype=BF16, scale=0.05)
    q[:, :, ::3, 512] = 100
    q[:, :, 1::3, 513] = 100
    out, lse = kda.latent_decode(q.cuda(), cache, table, ints(n), scale=0.125, page_size=64)
    compare(q, [keys], out, lse, [n], 1, h, 512, 0.125, BF16, True)


# ------------------------------------------------------------------ values that are no numbers
@pytest.mark.parametrize("dtype,simt", FORMS)
@pytest.mark.parametrize("length,at", [(1, 0), (300, 0), (300, 2), (300, 130), (300, 299)])
def test_nan_scores_reach_the_rows_that_see_them(kda, dtype, simt, length, at):  # noqa: F811
    flags = kda.KDA_FLAG_CUDA_CORE_PREFILL if simt else 0
    cache, table, _ = cached(kda, [length, 70], 64, 512, 64, 43)
    q = normal(44, 2, 1, 16, 576, dtype=dtype).cuda()
    go = lambda: kda.latent_decode(q, cache, table, ints(length, 70), scale=192 ** -0.5, page_size=64, flags=flags)  # noqa: E731
    out, lse = go()
    assert torch.isfinite(out.float()).all()
    keep = cache.clone()
    cref.views(cache, 64, 512, 64)[1][int(table[0, at // 64]), at % 64, 58] = NAN       # a rotary channel: no value has it
    o, l = go()
    assert torch.isnan(o[0]).all() and torch.isnan(l[0]).all()
    assert torch.equal(o[1], out[1]) and torch.equal(l[1], lse[1])
    cache.copy_(keep)
    for channel, value in ((0, NAN), (511, INF), (300, -INF), (575, NAN)):
        q2 = q.clone()
        q2[0, 0, 7, channel] = value
        o, l = kda.latent_decode(q2, cache, table, ints(length, 70), scale=192 ** -0.5, page_size=64, flags=flags)
        if value is NAN or not simt:                       # (on CUDA cores an infinite channel's scores have signs)
            assert torch.isnan(o[0, 0, 7]).all() and torch.isnan(l[0, 0, 7]), (channel, value)
        o[0, 0, 7], l[0, 0, 7] = out[0, 0, 7], lse[0, 0, 7]
        assert torch.equal(o, out) and torch.equal(l, lse)


@pytest.mark.parametrize("dtype,simt", FORMS)
def test_scores_of_minus_infinity_hide_and_of_plus_infinity_spoil(kda, dtype, simt):  # noqa: F811
    flags = kda.KDA_FLAG_CUDA_CORE_PREFILL if simt else 0
    n = 200
    r = torch.zeros(n, 64)
    r[::3, 5] = -INF
    cache, table, keys = by_hand(kda, normal(1, n, 512, dtype=BF16), r.to(BF16))
    q = normal(2, 1, 1, 16, 576, dtype=dtype)
    q[..., 517] = 1.0
    out, lse = kda.latent_decode(q.cuda(), cache, table, ints(n), scale=0.05, page_size=64, flags=flags)
    seen = [t for t in range(n) if t % 3]
    for h in (0, 15):
        want, wl, weight, ds = ref.attend(q[0, 0, h], keys[seen], keys[seen, :512], 0.05)
        bo, bl = cref.attention_bounds(q[0, 0, h], keys[seen], 512, want, wl, weight, ds, 0.05, dtype, not simt)
        within(out[0, 0, h], want, bo, h)
        within(lse[0, 0, h], torch.tensor(wl), bl, h)
    cref.views(cache, 64, 512, 64)[1][int(table[0, 1]), 3, 9] = INF
    q[..., 521] = 1.0
    q[0, 0, 4, 521] = -1.0
    out, lse = kda.latent_decode(q.cuda(), cache, table, ints(n), scale=0.05, page_size=64, flags=flags)
    assert torch.isnan(out[0, 0, :4]).all() and torch.isnan(out[0, 0, 5:]).all() and torch.isfinite(out[0, 0, 4].float()).all()
    only = ints(0)
    o, l = kda.latent_decode(q.cuda(), cache, table, only, scale=0.05, page_size=64, flags=flags)
    assert (o == 0).all() and (l == -INF).all()


# ------------------------------------------------------------------ workspaces, waits that run out
@pytest.mark.parametrize("lens,lq,h", [([5000], 1, 16), ([0, 0, 9000, 0, 1, 20000, 0], 2, 16), ([n % 3 * 70 for n in range(1001)], 1, 16),
                                       ([0] * 500 + [40000] + [0] * 500 + [1], 1, 32), ([0] * 70, 1, 16), ([3000, 129, 5000], 1, 100)])
def test_decode_does_not_depend_on_what_its_workspace_held(kda, lens, lq, h):  # noqa: F811
    cache, table, _ = cached(kda, lens, 64, 512, 64, 61)
    q = normal(62, len(lens), lq, h, 576, dtype=BF16).cuda()
    go = lambda fill: kda.latent_decode(q, cache, table, ints(*lens), scale=0.07, page_size=64,  # noqa: E731
                                        workspace=workspace(kda, len(lens), lq, h, 64, table, fill))
    out, lse = go(0)
    for fill in (0x7F, 0xFF):
        o, l = go(fill)
        assert torch.equal(o, out) and torch.equal(l, lse)


COPIES, PRODUCTS, SECOND, WEIGHTS, ROWS = 1, 2, 3, 4, 5


@pytest.mark.parametrize("lens,h,which", [([5000, 700] * 20 + [1], 16, COPIES), ([5000, 700] * 20 + [1], 32, SECOND), ([700, 1300], 32, PRODUCTS),
                                          ([700, 1300], 64, WEIGHTS), ([20000, 1300], 16, SECOND), ([700, 1300], 100, ROWS)])
def test_decode_waits_that_run_out_are_reported(kda, dropped, lens, h, which):  # noqa: F811
    """With a workspace of bytes that make no sense as indices: what the join reads was all written."""
    cache, table, _ = cached(kda, lens, 64, 512, 64, 73)
    q = normal(74, len(lens), 1, h, 576, dtype=BF16).cuda()
    ws = workspace(kda, len(lens), 1, h, 64, table)

    def go():
        ws.fill_(0x7F)
        return kda.latent_decode(q, cache, table, ints(*lens), scale=0.07, page_size=64, workspace=ws)
    states = [kda.latent_status(ws) for _ in runs_out(dropped, which, go)]
    assert states == [kda.KDA_ERR_TIMEOUT, kda.KDA_OK]


@pytest.mark.parametrize("simt", [False, True])
def test_decode_reports_one_of_several_faults(kda, simt):  # noqa: F811
    cache, table, _ = cached(kda, [300, 200, 70], 64, 512, 64, 63)
    q = normal(64, 3, 1, 16, 576, dtype=BF16).cuda()
    ws = workspace(kda, 3, 1, 16, 64, table)
    go = lambda t, l: kda.latent_decode(q, cache, t, l, scale=0.07, page_size=64, workspace=ws,  # noqa: E731
                                        flags=kda.KDA_FLAG_CUDA_CORE_PREFILL if simt else 0)[0]
    want = go(table, ints(300, 200, 70))
    bad = table.clone()
    bad[0, 1] = cache.shape[0]
    out = go(bad, ints(300, -5, 70))
    assert kda.latent_status(ws) in (kda.KDA_ERR_BAD_PAGE, kda.KDA_ERR_BAD_SEQLENS)
    assert torch.equal(out[2], want[2])
    assert torch.equal(go(table, ints(300, 200, 70)), want) and kda.latent_status(ws) == kda.KDA_OK
    empty = kda.latent_decode(q[:0], cache, table[:0], ints(), scale=0.07, page_size=64, workspace=ws)
    assert empty[0].shape == (0, 1, 16, 512) and kda.latent_status(ws) == kda.KDA_OK
    none = torch.zeros(0, cache.shape[1], dtype=torch.uint8, device="cuda")                 # a cache without pages
    out = kda.latent_decode(q, none, table, ints(0, 0, 0), scale=0.07, page_size=64, workspace=ws)[0]
    assert (out == 0).all() and kda.latent_status(ws) == kda.KDA_OK


# ------------------------------------------------------------------ together: streams, graphs, repeats
class Serving:
    """A step of a layer over the quantised cache: turn, write, attend; and the cached tokens read back."""

    def __init__(self, kda, lens, h, page=64, seed=5):  # noqa: F811
        self.kda, self.page = kda, page
        self.cache, table, _ = cached(kda, [n + 8 for n in lens], page, 512, 64, seed)
        self.table, self.lens = table, ints(*lens)
        n = len(lens)
        self.q, self.down = normal(seed + 1, n, h, 576, dtype=BF16).cuda(), normal(seed + 2, n, 576, dtype=BF16).cuda()
        self.cu = torch.tensor([0] + lens).cumsum(0).to("cuda", torch.int32)
        self.total, self.f = sum(lens), kda.rotary_frequencies(64)
        torch.cuda.synchronize()

    def go(self, stream=None):
        k = self.kda
        q, rope = k.rotary(self.q, self.lens, self.f, key=self.down[:, 512:], interleaved=True, stream=stream)
        k.latent_cache_write(self.down[:, :512], rope, self.cache, self.table, self.lens, page_size=self.page, stream=stream)
        out, lse = k.latent_decode(q, self.cache, self.table, self.lens, scale=0.07, page_size=self.page, stream=stream)
        c, r = k.latent_cache_read(self.cache, self.table, self.lens, self.cu, total_tokens=self.total, page_size=self.page, stream=stream)
        return [q, rope, out, lse, c, r]


def same(a, b):
    return all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))


def test_repeats_streams_and_graphs_give_the_same_bits(kda):  # noqa: F811
    s = Serving(kda, [700, 9, 64, 5000], 16)
    want = s.go()
    torch.cuda.synchronize()
    for _ in range(4):
        assert same(s.go(), want)
    for other in (torch.cuda.Stream(), torch.cuda.Stream().cuda_stream):
        got = s.go(other)
        torch.cuda.synchronize()
        assert same(got, want)
    for stream in (None, torch.cuda.Stream()):
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=stream):
            got = s.go(stream)
        for t in got:
            t.view(torch.uint8).zero_()
        g.replay()
        g.replay()
        torch.cuda.synchronize()
        assert same(got, want)
    # the same graph for the next tokens: lengths and inputs of a replay are those in memory then
    s.lens += 1
    s.q.neg_()
    g.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in got[:4]]
    assert same(got, s.go()[:4])


def test_calls_on_several_streams_at_once_give_the_same_bits(kda):  # noqa: F811
    layers = [Serving(kda, [5000, 60, 900] * 4, h, page, seed) for h, page, seed in ((16, 64, 11), (32, 16, 12), (100, 128, 13), (128, 64, 14))]
    want = [x.go() for x in layers]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in layers]
    got = []
    for turn in range(8):
        for i, x in enumerate(layers):
            got.append((i, x.go(streams[i])))
    torch.cuda.synchronize()
    for i, outs in got:
        assert same(outs, want[i]), i


def test_a_batch_padded_with_empty_sequences(kda):  # noqa: F811
    """Sequences of length 0 behind the real ones, their table rows and inputs whatever they are."""
    s = Serving(kda, [300, 65, 7], 16)
    want = s.go()
    n, k = 3, 5
    p = Serving(kda, [300, 65, 7], 16)
    p.q = torch.cat([p.q, torch.full((k, 16, 576), NAN, dtype=BF16, device="cuda")])
    p.down = torch.cat([p.down, torch.full((k, 576), NAN, dtype=BF16, device="cuda")])
    p.table = torch.cat([p.table, torch.full((k, p.table.shape[1]), -7, dtype=torch.int32, device="cuda")])
    p.lens = torch.cat([p.lens, ints(*[0] * k)])
    p.cu = torch.cat([p.cu, p.cu[-1:].repeat(k)])
    got = p.go()
    assert same([got[0][:n], got[1][:n], got[2][:n], got[3][:n], got[4], got[5]], want) and torch.equal(p.cache, s.cache)
    assert (got[2][n:] == 0).all() and (got[3][n:] == -INF).all()


# ------------------------------------------------------------------ what lies beside the outputs
def test_nothing_is_written_outside_the_outputs(kda):  # noqa: F811
    def guarded(*shape, dtype):
        n = math.prod(shape) * torch.empty((), dtype=dtype).element_size()
        whole = torch.full((n + 512,), 0xA5, dtype=torch.uint8, device="cuda")
        return whole, whole[256:256 + n].view(dtype).view(*shape)

    def check(*wholes):
        torch.cuda.synchronize()
        for w in wholes:
            assert (w[:256] == 0xA5).all() and (w[-256:] == 0xA5).all()
    for h, lq in ((16, 1), (20, 3), (100, 1), (32, 1)):
        cache, table, _ = cached(kda, [700, 9, 0], 64, 512, 64, 24)
        q = normal(25, 3, lq, h, 576, dtype=BF16).cuda()
        (w1, o), (w2, l) = guarded(3, lq, h, 512, dtype=BF16), guarded(3, lq, h, dtype=F32)
        size = kda.latent_decode_workspace_bytes(3, lq, h, 512, 64, BF16, 64, table.shape[1], quantized=True)
        w3, ws = guarded(size, dtype=torch.uint8)
        kda.latent_decode(q, cache, table, ints(700, 9, 0), scale=0.07, page_size=64, out=o, lse=l, workspace=ws)
        check(w1, w2, w3)
        assert torch.equal(o, kda.latent_decode(q, cache, table, ints(700, 9, 0), scale=0.07, page_size=64)[0])
    for dt in (BF16, F32):
        cache, table, _ = cached(kda, [700, 9, 0], 16, 512, 64, 24)
        (w1, c), (w2, r) = guarded(709, 512, dtype=dt), guarded(709, 64, dtype=dt)
        kda.latent_cache_read(cache, table, ints(700, 9, 0), ints(0, 700, 709, 709), total_tokens=709, page_size=16, latents=c, rope=r)
        check(w1, w2)
        f = kda.rotary_frequencies(64)
        pos = torch.arange(709, device="cuda", dtype=torch.int32)
        w3, x = guarded(709, 3, 80, dtype=dt)
        w4, y = guarded(709, 64, dtype=dt)
        kda.rotary(normal(1, 709, 3, 80, dtype=dt).cuda(), pos, f, key=r, out=x, key_out=y)
        check(w3, w4)
    w5, pages = guarded(6, kda.latent_cache_page_bytes(16), dtype=torch.uint8)
    pages.zero_()
    x = latents(3, 96, 576, dtype=BF16).cuda()
    kda.latent_cache_write(x[:, :512], x[:, 512:], pages, ints(5, 0, 1, 3, 4, 2).view(1, 6), ints(96), page_size=16)
    check(w5)
    assert (pages[:, 16 * 641:] == 0).all()                                          # the padding of a page


def test_inputs_of_another_stream_live_until_it_has_read_them(kda):  # noqa: F811
    s = Serving(kda, [300, 65], 16)
    want = s.go()
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(other):
        torch.cuda._sleep(400_000_000)                     # some 0.2 s before the calls' kernels start
    q, down, table, cu = s.q.clone(), s.down.clone(), s.table.clone(), s.cu.clone()
    torch.cuda.current_stream().synchronize()
    s.q, s.down, s.table, s.cu = q, down, table, cu
    got = s.go(other)
    sizes = [(t.shape, t.dtype) for t in (q, down, table, cu)]
    del q, down, table, cu
    s.q = s.down = s.table = s.cu = None
    others = [torch.zeros(shape, dtype=dtype, device="cuda") for shape, dtype in sizes for _ in range(4)]
    torch.cuda.synchronize()
    assert same(got, want) and len(others) == 16


# ------------------------------------------------------------------ contexts
CONTEXTS = '''
import ctypes, re, sys
sys.path.insert(0, sys.argv[1])
import kda_gated_delta_chunked_gb300 as kda                 # (torch is imported, and makes no context)
rt = ctypes.CDLL(re.search(r"\\S*libcudart\\.so\\S*", open("/proc/self/maps").read()).group(0))

class Ptr:
    def __init__(self, n, words=None):
        p = ctypes.c_void_p()
        assert rt.cudaMalloc(ctypes.byref(p), ctypes.c_size_t(n)) == 0
        assert rt.cudaMemset(p, 0, ctypes.c_size_t(n)) == 0
        if words is not None:
            a = (ctypes.c_int32 * len(words))(*words)
            assert rt.cudaMemcpy(p, a, ctypes.c_size_t(4 * len(words)), 1) == 0
        self.p = p.value
    def data_ptr(self):
        return self.p

def all_calls():
    x, y = Ptr(1 << 24), [Ptr(1 << 24) for _ in range(5)]
    table, lens, pos, f = Ptr(1 << 12, list(range(16))), Ptr(1 << 12, [700]), Ptr(1 << 14, list(range(700))), Ptr(1 << 12)
    part = kda.KdaRotaryPart(4, 192, 128, 0, 768, 192, 768, 192)
    rc = [kda.kda_rotary(kda.KdaRotaryDesc(700, 64, kda.KDA_BF16, 0, 1.0, part, part), x, None, pos, f, y[0], None, 0)]
    d = kda.KdaLatentCacheDesc(1, kda.KDA_BF16, 700, 512, 64, 64, 16, 16, 0, 41088, 576, 576, y[3].p, 256)
    rc += [kda.kda_latent_cache_write(d, x, y[0], None, table, lens, y[1], 0), kda.kda_latent_cache_read(d, y[1], table, lens, None, y[2], y[0], 0)]
    for h in (16, 64):
        d = kda.KdaLatentDesc(1, h, kda.KDA_BF16, kda.KDA_FLAG_CACHE_8, 0.1, d_k=512, d_rope=64, d_v=512, q_token_stride=h * 576, q_head_stride=576,
                              num_queries=1, page_size=64, num_pages=16, max_pages=16, page_stride=41088, workspace=y[3].p, workspace_bytes=1 << 24)
        rc += [kda.kda_latent_decode(d, x, y[1], table, lens, y[2], y[4], 0), kda.kda_latent_status(d, 0)]
    return rc + [rt.cudaDeviceSynchronize()]

def check(what):
    rc = all_calls()
    print(what, rc, kda.lib.kda_last_cuda_error())
    assert not any(rc)

check("first")
cu, context = ctypes.CDLL("libcuda.so.1"), ctypes.c_void_p()
assert cu.cuCtxCreate_v2(ctypes.byref(context), 0, 0) == 0   # current from here on
check("another context of the device")
assert cu.cuCtxDestroy_v2(context) == 0
assert rt.cudaDeviceReset() == 0
check("after a reset")
'''


def test_a_new_context_of_the_device_is_as_good_as_the_first(kda):  # noqa: F811
    r = subprocess.run([sys.executable, "-c", CONTEXTS, ROOT], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-1500:] + r.stderr[-1500:]
