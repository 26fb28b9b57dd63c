"""Norm, scaled 8-bit product and latent attention where a call is unusual: values
that are no numbers, waits that run out, calls without work, other contexts and
streams."""
import os
import subprocess
import sys
import time

import pytest
import torch

from test_gpu_operators import BF16, F32, check_matmul, expanded, kda, normal, operands, paged  # noqa: F401

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NAN, INF = float("nan"), float("inf")


def lengths(*l):
    return torch.tensor(l, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ values that are no numbers
# Nothing here is a question of rounding: a row with a score that is no number has no numbers in it, every other row
# keeps its bits.
FORMS = [(BF16, False), (BF16, True), (F32, True)]          # tensor cores, CUDA cores, CUDA cores


@pytest.mark.parametrize("dtype,simt", FORMS)
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("at", [0, 1, 5, 63, 99])
def test_prefill_nan_scores_reach_the_rows_that_see_them(kda, dtype, simt, causal, at):  # noqa: F811
    n, flags = 100, kda.KDA_FLAG_CUDA_CORE_PREFILL if simt else 0
    q, kn, kr, v = (t.cuda() for t in expanded(n, n, 2, dtype=dtype, seed=41))
    go = lambda: kda.latent_prefill(q, kn, kr, v, scale=192 ** -0.5, causal=causal, flags=flags)  # noqa: E731
    out, lse = go()
    keep = kn.clone()
    kn = kn.clone()
    kn[at, 1] = NAN                                          # a key of one head
    o, l = go()
    seen = torch.arange(n, device="cuda") >= (at if causal else 0)
    assert torch.isnan(o[seen, 1]).all() and torch.isnan(l[seen, 1]).all()
    assert torch.equal(o[~seen], out[~seen]) and torch.equal(l[~seen], lse[~seen])
    assert torch.equal(o[:, 0], out[:, 0]) and torch.equal(l[:, 0], lse[:, 0])
    kn, q = keep, q.clone()
    q[at, 0, 3] = NAN                                        # a query: all its scores
    o, l = go()
    assert torch.isnan(o[at, 0]).all() and torch.isnan(l[at, 0])
    o[at, 0], l[at, 0] = out[at, 0], lse[at, 0]
    assert torch.equal(o, out) and torch.equal(l, lse)


@pytest.mark.parametrize("dtype,simt", FORMS)
@pytest.mark.parametrize("length,at", [(1, 0), (300, 0), (300, 1), (300, 2), (300, 3), (300, 130), (300, 299)])
def test_decode_nan_scores_reach_the_rows_that_see_them(kda, dtype, simt, length, at):  # noqa: F811
    flags = kda.KDA_FLAG_CUDA_CORE_PREFILL if simt else 0
    cache, table, _ = paged([length, 70], 64, 576, dtype, 43)
    q = normal(44, 2, 1, 16, 576, dtype=dtype).cuda()
    go = lambda: kda.latent_decode(q, cache, table, lengths(length, 70), scale=192 ** -0.5, flags=flags)  # noqa: E731
    out, lse = go()
    keep = cache.clone()
    cache[int(table[0, at // 64]), at % 64, 570] = NAN       # a rotary channel: no value has it
    o, l = go()
    assert torch.isnan(o[0]).all() and torch.isnan(l[0]).all()
    assert torch.equal(o[1], out[1]) and torch.equal(l[1], lse[1])
    cache, q = keep, q.clone()
    q[0, 0, 7, 0] = NAN
    o, l = go()
    assert torch.isnan(o[0, 0, 7]).all() and torch.isnan(l[0, 0, 7])
    o[0, 0, 7], l[0, 0, 7] = out[0, 0, 7], lse[0, 0, 7]
    assert torch.equal(o, out) and torch.equal(l, lse)


@pytest.mark.parametrize("dtype,simt", FORMS)
def test_scores_of_minus_infinity_hide_and_of_plus_infinity_spoil(kda, dtype, simt):  # noqa: F811
    flags = kda.KDA_FLAG_CUDA_CORE_PREFILL if simt else 0
    q, kn, kr, v = (t.cuda() for t in expanded(40, 40, 1, dtype=dtype, seed=45))
    q, kr = q.abs() + 0.01, torch.zeros_like(kr)
    kn = torch.zeros_like(kn)
    kn[:3] = -INF
    out, lse = kda.latent_prefill(q, kn, kr, v, scale=0.1, flags=flags)
    assert (out[:3] == 0).all() and (lse[:3] == -INF).all() and torch.isfinite(out[3:].float()).all()
    # the scores behind are zeros: equal weights, and the log of their number to fp32's rounding of one logarithm
    want = torch.log(torch.arange(1, 38, device="cuda", dtype=torch.float64))
    assert float((lse[3:, 0].double() - want).abs().max()) < 2.0 ** -20
    kn[10] = INF
    out, lse = kda.latent_prefill(q, kn, kr, v, scale=0.1, flags=flags)
    assert (out[:3] == 0).all() and torch.isfinite(out[3:10].float()).all() and torch.isnan(out[10:].float()).all()


# ------------------------------------------------------------------ what a workspace held, waits that run out
@pytest.mark.parametrize("lens,lq,h", [([5000], 1, 16), ([0, 0, 9000, 0, 1, 20000, 0], 2, 16), ([n % 3 * 70 for n in range(3001)], 1, 16),
                                       ([0] * 500 + [40000] + [0] * 500 + [1], 1, 32), ([0] * 70, 1, 16), ([3000, 129, 5000], 1, 100)])
def test_decode_does_not_depend_on_what_its_workspace_held(kda, lens, lq, h):  # noqa: F811
    cache, table, _ = paged(lens, 64, 576, BF16, 61)
    q = normal(62, len(lens), lq, h, 576, dtype=BF16).cuda()
    n = kda.latent_decode_workspace_bytes(len(lens), lq, h, 512, 64, BF16, 64, table.shape[1])
    go = lambda fill: kda.latent_decode(q, cache, table, lengths(*lens), scale=0.07,  # noqa: E731
                                        workspace=torch.full((n,), fill, dtype=torch.uint8, device="cuda"))
    out, lse = go(0)
    for fill in (0x7F, 0xFF):
        o, l = go(fill)
        assert torch.equal(o, out) and torch.equal(l, lse)
    simt, slse = kda.latent_decode(q, cache, table, lengths(*lens), scale=0.07, flags=kda.KDA_FLAG_CUDA_CORE_PREFILL)
    some = torch.isfinite(slse)
    assert torch.equal(torch.isfinite(lse), some) and (not some.any() or float((lse - slse)[some].abs().max()) < 1e-4)


@pytest.mark.parametrize("simt", [False, True])
def test_decode_reports_one_of_several_faults(kda, simt):  # noqa: F811
    """A bad page and a bad length in one call: one of the two, and the sequences without a fault keep their bits."""
    cache, table, _ = paged([300, 200, 70], 64, 576, BF16, 63)
    q = normal(64, 3, 1, 16, 576, dtype=BF16).cuda()
    ws = torch.zeros(kda.latent_decode_workspace_bytes(3, 1, 16, 512, 64, BF16, 64, table.shape[1]), dtype=torch.uint8, device="cuda")
    go = lambda t, l: kda.latent_decode(q, cache, t, l, scale=0.07, workspace=ws, flags=kda.KDA_FLAG_CUDA_CORE_PREFILL if simt else 0)[0]  # noqa: E731
    want = go(table, lengths(300, 200, 70))
    bad = table.clone()
    bad[0, 1] = cache.shape[0]
    out = go(bad, lengths(300, -5, 70))
    assert kda.latent_status(ws) in (kda.KDA_ERR_BAD_PAGE, kda.KDA_ERR_BAD_SEQLENS)
    assert torch.equal(out[2], want[2])
    assert torch.equal(go(table, lengths(300, 200, 70)), want) and kda.latent_status(ws) == kda.KDA_OK


# Each wait of the kernels runs out after 2 s; a call's follow one another a few times at most.
COPIES, PRODUCTS, SECOND, WEIGHTS, ROWS = 1, 2, 3, 4, 5


@pytest.fixture
def dropped(kda):  # noqa: F811
    yield kda.kda_selftest_drop_arrival
    torch.cuda.synchronize()
    assert kda.kda_selftest_drop_arrival(0) == kda.KDA_OK


def runs_out(dropped, which, call):
    """`call` with an arrival missing ends by itself; after it the same call gives what it gave before."""
    want = [t.clone() for t in call()]
    torch.cuda.synchronize()
    assert dropped(which) == 0
    t = time.perf_counter()
    late = call()
    torch.cuda.synchronize()
    assert 1.5 < time.perf_counter() - t < 30
    yield late
    assert dropped(0) == 0
    got = call()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    yield got


def test_dropped_arrivals_have_numbers(kda, dropped):  # noqa: F811
    assert [dropped(w) for w in (-1, 6, 100)] == [kda.KDA_ERR_INVALID_ARGUMENT] * 3 and dropped(5) == kda.KDA_OK


@pytest.mark.parametrize("m,n,k,which", [(3, 700, 1024, COPIES), (3, 700, 1024, PRODUCTS), (300, 500, 2000, COPIES), (300, 500, 2000, PRODUCTS),
                                         (2000, 3001, 1040, COPIES), (2000, 3001, 1040, PRODUCTS)])
def test_matmul_waits_that_run_out_give_nan(kda, dropped, m, n, k, which):  # noqa: F811
    a, sa, b, sb = operands(m, n, k, 71)
    late = [bool(torch.isnan(c).all()) for c, in runs_out(dropped, which, lambda: (kda.matmul_fp8(a, sa, b, sb, out_dtype=F32),))]
    assert late == [True, False]


@pytest.mark.parametrize("tq,tk,h,which", [(300, 2000, 2, COPIES), (300, 2000, 2, SECOND), (300, 2000, 2, ROWS), (2000, 2000, 16, PRODUCTS),
                                           (2000, 2000, 16, WEIGHTS), (2000, 2000, 16, ROWS)])
def test_prefill_waits_that_run_out_are_reported(kda, dropped, tq, tk, h, which):  # noqa: F811
    q, kn, kr, v = (t.cuda() for t in expanded(tq, tk, h, seed=72))
    ws = torch.zeros(kda.latent_prefill_workspace_bytes(1, h, BF16), dtype=torch.uint8, device="cuda")
    states = [kda.latent_status(ws) for _ in runs_out(dropped, which, lambda: kda.latent_prefill(q, kn, kr, v, scale=0.07, workspace=ws))]
    assert states == [kda.KDA_ERR_TIMEOUT, kda.KDA_OK]


@pytest.mark.parametrize("lens,h,which", [([5000, 700] * 20 + [1], 16, COPIES), ([5000, 700] * 20 + [1], 16, SECOND), ([700, 1300], 32, PRODUCTS),
                                          ([700, 1300], 64, WEIGHTS), ([700, 1300], 64, SECOND), ([700, 1300], 100, ROWS)])
def test_decode_waits_that_run_out_are_reported(kda, dropped, lens, h, which):  # noqa: F811
    """With a workspace of bytes that make no sense as indices: what the join reads was all written."""
    cache, table, _ = paged(lens, 64, 576, BF16, 73)
    q = normal(74, len(lens), 1, h, 576, dtype=BF16).cuda()
    ws = torch.full((kda.latent_decode_workspace_bytes(len(lens), 1, h, 512, 64, BF16, 64, table.shape[1]),), 0x7F, dtype=torch.uint8, device="cuda")

    def go():
        ws.fill_(0x7F)
        return kda.latent_decode(q, cache, table, lengths(*lens), scale=0.07, workspace=ws)
    states = [kda.latent_status(ws) for _ in runs_out(dropped, which, go)]
    assert states == [kda.KDA_ERR_TIMEOUT, kda.KDA_OK]


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
    x, y = Ptr(1 << 24), [Ptr(1 << 24) for _ in range(8)]
    sc = Ptr(1 << 20)
    rc = [kda.kda_rms_norm(kda.KdaNormDesc(4, 16384, kda.KDA_BF16, 16384, 16384, 1e-6), x, None, None, None, y[0], None, None, 0)]
    for m, n in ((1, 128), (20, 128), (60, 128), (300, 512), (3000, 2000)):
        for dt in (kda.KDA_BF16, kda.KDA_F32):
            rc.append(kda.kda_matmul_fp8(kda.KdaMatmulDesc(m, n, 256, 256, 256, n, dt, 0), x, sc, y[0], sc, y[1 + (dt == 0)], 0))
    def latent(h, rows, **kw):
        d = kda.KdaLatentDesc(1, h, kda.KDA_BF16, 0, 0.1)
        for k, v in kw.items():
            setattr(d, k, v)
        d.workspace, d.workspace_bytes = y[7].p, 1 << 24
        return d
    for h, t in ((2, 100), (8, 300)):                        # keys shared by a cluster, and not
        d = latent(h, t, d_k=128, d_rope=64, d_v=128, total_q=t, total_k=t * 4, q_token_stride=h * 192, q_head_stride=192,
                   k_token_stride=h * 128, k_head_stride=128, v_token_stride=h * 128, v_head_stride=128, rope_token_stride=64)
        rc += [kda.kda_latent_prefill(d, x, y[0], y[1], y[2], None, None, y[3], y[4], 0), kda.kda_latent_status(d, 0)]
    table, lens = Ptr(1 << 12, list(range(16))), Ptr(1 << 12, [700])
    for h in (16, 32, 64):
        d = latent(h, 1, d_k=512, d_rope=64, d_v=512, q_token_stride=h * 576, q_head_stride=576, num_queries=1, page_size=64,
                   num_pages=16, max_pages=16, page_stride=64 * 576)
        rc += [kda.kda_latent_decode(d, x, y[0], table, lens, y[3], y[4], 0), kda.kda_latent_status(d, 0)]
    return rc + [rt.cudaDeviceSynchronize()]

def check(what):
    rc = all_calls()
    print(what, rc, kda.lib.kda_last_cuda_error())
    assert not any(rc)

check("first")
check("again")
cu, context = ctypes.CDLL("libcuda.so.1"), ctypes.c_void_p()
assert cu.cuCtxCreate_v2(ctypes.byref(context), 0, 0) == 0   # current from here on
check("another context of the device")
assert cu.cuCtxDestroy_v2(context) == 0
assert rt.cudaDeviceReset() == 0
check("after a reset")
'''


def test_a_new_context_of_the_device_is_as_good_as_the_first(kda):  # noqa: F811
    """What was set for kernels in one context (more shared memory than they have by default) is not taken for set in the next."""
    r = subprocess.run([sys.executable, "-c", CONTEXTS, ROOT], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-1500:] + r.stderr[-1500:]


# ------------------------------------------------------------------ calls without work
def test_status_of_calls_without_work(kda):  # noqa: F811
    """They leave a status as others do, whatever the workspace held."""
    stale = lambda: torch.full((1 << 20,), 5, dtype=torch.uint8, device="cuda")  # noqa: E731
    q, kn, kr, v = (t.cuda() for t in expanded(5, 5, 2))
    for flags in (0, kda.KDA_FLAG_CUDA_CORE_PREFILL):
        def prefill(tq, cq, ck):
            ws = stale()
            o, l = kda.latent_prefill(q[:tq], kn, kr, v, cq, ck, scale=0.1, workspace=ws, flags=flags)
            assert o.shape == (tq, 2, 128) and l.shape == (tq, 2)
            return kda.latent_status(ws)
        assert prefill(0, None, None) == kda.KDA_OK
        assert prefill(0, lengths(0, 0, 0), lengths(0, 2, 5)) == kda.KDA_OK
        assert prefill(0, lengths(0, 0, 0), lengths(0, 6, 5)) == kda.KDA_ERR_BAD_SEQLENS
        assert prefill(0, lengths(0, 3, 0), lengths(0, 2, 5)) == kda.KDA_ERR_BAD_SEQLENS
        assert prefill(0, lengths(0, 0), lengths(1, 5)) == kda.KDA_ERR_BAD_SEQLENS
        assert prefill(5, lengths(0, 5), lengths(0, 5)) == kda.KDA_OK
        cache, table, _ = paged([70], 64, 576, BF16, 3)
        ws = stale()
        o, l = kda.latent_decode(normal(1, 0, 1, 16, 576, dtype=BF16).cuda(), cache, table[:0], lengths(), scale=0.1, workspace=ws, flags=flags)
        assert o.shape == (0, 1, 16, 512) and kda.latent_status(ws) == kda.KDA_OK
    empty = [t[:0].contiguous() for t in (q, kn, kr, v)]
    ws = stale()
    kda.latent_prefill(*empty, lengths(0), lengths(0), scale=0.1, workspace=ws)
    assert kda.latent_status(ws) == kda.KDA_OK
    kda.latent_prefill(*empty, lengths(3), lengths(0), scale=0.1, workspace=ws)
    assert kda.latent_status(ws) == kda.KDA_ERR_BAD_SEQLENS


def test_rows_without_a_sequence_are_refused(kda):  # noqa: F811
    q, kn, kr, v = (t.cuda() for t in expanded(5, 5, 2))
    for args in ((q, kn, kr, v), (q[:0], kn, kr, v), (q, kn[:0].contiguous(), kr[:0].contiguous(), v[:0].contiguous())):
        with pytest.raises(ValueError):
            kda.latent_prefill(*args, lengths(0), lengths(0), scale=0.1)


def test_calls_without_work_are_captured(kda):  # noqa: F811
    q, kn, kr, v = (t.cuda() for t in expanded(5, 5, 2))
    good, bad = lengths(0, 0), lengths(0, 4)
    ws = torch.full((512,), 5, dtype=torch.uint8, device="cuda")
    for lk, want in ((lengths(0, 5), kda.KDA_OK), (bad, kda.KDA_ERR_BAD_SEQLENS)):
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            kda.latent_prefill(q[:0], kn, kr, v, good, lk, scale=0.1, workspace=ws)
        g.replay()
        assert kda.latent_status(ws) == want


# ------------------------------------------------------------------ streams
def test_inputs_of_another_stream_live_until_it_has_read_them(kda):  # noqa: F811
    """A caller may drop its inputs once a call has returned, also a call on a stream that is not the current one."""
    other = torch.cuda.Stream()
    x = normal(51, 64, 512, dtype=BF16).cuda()
    want = kda.rms_norm(x)[0].clone()
    raw = torch.cuda.Stream().cuda_stream
    for stream in (other, raw):
        torch.cuda.synchronize()
        s = stream if stream is other else torch.cuda.ExternalStream(stream)
        with torch.cuda.stream(s):
            torch.cuda._sleep(400_000_000)                     # some 0.2 s before the call's kernel starts
        copy = x.clone()
        torch.cuda.current_stream().synchronize()
        at = copy.data_ptr()
        y = kda.rms_norm(copy, stream=stream)[0]
        del copy
        others = [torch.zeros_like(x) for _ in range(8)]
        assert not s.query()                                   # still asleep: the input must be there
        assert at not in [t.data_ptr() for t in others]
        torch.cuda.synchronize()
        assert torch.equal(y, want)


def test_arguments_that_are_no_truth_value_or_too_large_are_refused(kda):  # noqa: F811
    x = normal(52, 4, 128, dtype=BF16).cuda()
    for kw in (dict(normed=torch.ones(2)), dict(quantize=torch.ones(2))):
        with pytest.raises(ValueError):
            kda.rms_norm(x, **kw)
    with pytest.raises(ValueError):
        kda.matmul_fp8(x.to(torch.float8_e4m3fn), torch.ones(4, 1, device="cuda"), x.to(torch.float8_e4m3fn), torch.ones(1, 1, device="cuda"),
                       flags=1 << 32)


# ------------------------------------------------------------------ long sums
@pytest.mark.parametrize("m,n,k", [(1, 300, 12304), (16, 129, 18432), (33, 256, 14352), (64, 128, 20000), (200, 500, 18448), (1, 16, 2300000),
                                   (64, 8, 540000), (300, 200, 100000)])
def test_matmul_of_few_rows_and_long_sums(kda, m, n, k):  # noqa: F811
    """Rows whose blocks' scales lie in shared memory, one CTA's share of them, and rows too long for that."""
    a, sa, b, sb = operands(m, n, k, 81)
    check_matmul(kda, a, sa, b, sb, out_dtype=F32)
    check_matmul(kda, a, sa, b, sb)


# ------------------------------------------------------------------ what lies beside the outputs
@pytest.mark.parametrize("rows,dim", [(1, 1), (3, 7), (5, 128), (130, 2051), (33, 4096), (7, 200), (3, 16384), (700, 9001), (2, 40000)])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("shift", [0, 1])
def test_norm_writes_nothing_outside_its_outputs(kda, rows, dim, dtype, shift):  # noqa: F811
    """Outputs that start on 16 bytes, and outputs that start an element (of 8 bits: a byte) behind."""
    esz = torch.empty((), dtype=dtype).element_size()

    def guarded(n, width):
        whole = torch.full((n * width + 512 + width,), 0xA5, dtype=torch.uint8, device="cuda")
        return whole, 256 + shift * width, n * width
    x, r = normal(91, rows, dim, dtype=dtype).cuda(), normal(92, rows, dim, dtype=dtype).cuda()
    w = (1 + normal(93, dim, scale=0.2)).to(dtype).cuda()
    y, q, s, h = kda.rms_norm(x, w, r, quantize=True)
    outs = [guarded(rows * dim, esz), guarded(rows * dim, esz), guarded(rows * dim, 1), guarded(s.numel(), 4)]
    d = kda.KdaNormDesc(rows, dim, kda.KDA_BF16 if dtype == BF16 else kda.KDA_F32, dim, dim, 1e-6)
    ho, yo, qo, so = (t[at:at + n] for t, at, n in outs)
    assert kda.kda_rms_norm(d, x, w, r, ho, yo, qo, so) == kda.KDA_OK
    torch.cuda.synchronize()
    for t, at, n in outs:
        assert (t[:at] == 0xA5).all() and (t[at + n:] == 0xA5).all()
    assert torch.equal(ho, h.view(torch.uint8).flatten())      # one addition and its rounding, whoever does it
    if not shift:
        assert torch.equal(yo, y.view(torch.uint8).flatten()) and torch.equal(qo, q.view(torch.uint8).flatten())
        assert torch.equal(so, s.view(torch.uint8).flatten())
    else:                                                      # sums in another order: 72 roundings of 2^-24 on either side
        assert torch.allclose(so.clone().view(F32), s.flatten(), rtol=2 * 72 * 2.0 ** -24, atol=0)


# ------------------------------------------------------------------ offsets above 32 bits
FAR = 1 << 24                                                # elements between rows: 300 of them span 5e9


def far(t, lead=0):
    """The same values in rows FAR elements apart."""
    wide = torch.empty(t.shape[0] * FAR, dtype=t.dtype, device="cuda")
    view = wide.as_strided(t.shape, (FAR, *t.contiguous().stride()[1:]), lead)
    view.copy_(t)
    return view


@pytest.mark.parametrize("simt", [False, True])
def test_decode_from_pages_at_the_end_of_a_large_pool(kda, simt):  # noqa: F811
    cache, table, _ = paged([300, 1, 700], 64, 576, BF16, 95)
    q = normal(96, 3, 1, 16, 576, dtype=BF16).cuda()
    go = lambda c, t: kda.latent_decode(q, c, t, lengths(300, 1, 700), scale=0.07, flags=kda.KDA_FLAG_CUDA_CORE_PREFILL if simt else 0)  # noqa: E731
    want = go(cache, table)
    pool = torch.empty(120_000, 64, 576, dtype=BF16, device="cuda")
    first = pool.shape[0] - cache.shape[0]
    pool[first:] = cache
    got = go(pool, torch.where(table < cache.shape[0], table + first, table))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("simt", [False, True])
def test_prefill_of_rows_far_apart(kda, simt):  # noqa: F811
    q, kn, kr, v = (t.cuda() for t in expanded(300, 300, 2, seed=97))
    go = lambda *x: kda.latent_prefill(*x, scale=0.07, flags=kda.KDA_FLAG_CUDA_CORE_PREFILL if simt else 0)  # noqa: E731
    want = go(q, kn, kr, v)
    for i in range(4):
        x = [q, kn, kr, v]
        x[i] = far(x[i])
        got = go(*x)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("simt,m", [(False, 300), (True, 300), (False, 40)])
def test_matmul_of_rows_far_apart(kda, simt, m):  # noqa: F811
    a, sa, b, sb = operands(m, 300, 400, 98)
    flags = kda.KDA_FLAG_CUDA_CORE_PREFILL if simt else 0
    want = kda.matmul_fp8(a, sa, b, sb, flags=flags)
    bytes_ = lambda t: far(t.view(torch.uint8)).view(t.dtype)  # noqa: E731
    assert torch.equal(kda.matmul_fp8(bytes_(a), sa, b, sb, flags=flags), want)
    assert torch.equal(kda.matmul_fp8(a, sa, bytes_(b), sb, flags=flags), want)
    for lead in (0, 1):
        out = far(torch.zeros_like(want), lead)
        assert torch.equal(kda.matmul_fp8(a, sa, b, sb, out=out, flags=flags), want)


@pytest.mark.parametrize("dim", [512, 515, 16384])
def test_norm_of_rows_far_apart(kda, dim):  # noqa: F811
    x, r = normal(99, 300, dim, dtype=BF16).cuda(), normal(100, 300, dim, dtype=BF16).cuda()
    want = kda.rms_norm(x, None, r, quantize=True)
    for y, s in ((far(x), r), (x, far(r))):
        got = kda.rms_norm(y, None, s, quantize=True)
        assert all(torch.equal(g.view(torch.uint8), w.view(torch.uint8)) for g, w in zip(got, want))


def test_calls_on_several_streams_at_once_give_the_same_bits(kda):  # noqa: F811
    """Kernels of all operators beside one another, each with its own workspace."""
    a, sa, b, sb = operands(700, 1300, 1024, 101)
    x = normal(102, 900, 4096, dtype=BF16).cuda()
    few = [t.cuda() for t in expanded(300, 2500, 2, seed=103)]
    many = [t.cuda() for t in expanded(1500, 1500, 8, seed=104)]
    cache, table, _ = paged([5000, 60, 0, 900] * 6, 64, 576, BF16, 105)
    L = lengths(*([5000, 60, 0, 900] * 6))
    q16, q48 = normal(106, 24, 1, 16, 576, dtype=BF16).cuda(), normal(107, 24, 3, 16, 576, dtype=BF16).cuda()
    calls = [lambda s: kda.rms_norm(x, quantize=True, stream=s)[:3], lambda s: [kda.matmul_fp8(a, sa, b, sb, stream=s)],
             lambda s: [kda.matmul_fp8(a[:9], sa[:9].contiguous(), b, sb, stream=s)],
             lambda s: kda.latent_prefill(*few, scale=0.07, stream=s), lambda s: kda.latent_prefill(*many, scale=0.07, stream=s),
             lambda s: kda.latent_decode(q16, cache, table, L, scale=0.07, stream=s),
             lambda s: kda.latent_decode(q48, cache, table, L, scale=0.07, stream=s)]
    want = [c(None) for c in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    got = []
    for turn in range(12):
        for i in range(len(calls)):
            got.append((i, calls[i](streams[(i + turn) % len(streams)])))
    torch.cuda.synchronize()
    for i, outs in got:
        assert all(torch.equal(o.view(torch.uint8), w.view(torch.uint8)) for o, w in zip(outs, want[i])), i


def test_calls_on_a_given_stream_are_captured(kda):  # noqa: F811
    """The stream that is captured named in the call, with inputs from outside and from inside the capture."""
    x, w = normal(111, 64, 512, dtype=BF16).cuda(), normal(112, 512, dtype=BF16).cuda()
    a, sa, b, sb = operands(64, 300, 512, 113)
    want = [kda.rms_norm(x * 2, w)[0], kda.matmul_fp8(a, sa, b, sb)]
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=s):
        inside = x * 2
        got = [kda.rms_norm(inside, w, stream=s)[0], kda.matmul_fp8(a, sa, b, sb, stream=s)]
        del inside
        torch.zeros(64, 512, dtype=BF16, device="cuda")
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, want))
