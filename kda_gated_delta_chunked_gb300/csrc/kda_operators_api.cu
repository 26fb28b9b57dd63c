// kda_operators_api.cu -- C entries of the operators around the recurrent
// layers: argument checks, choice of path, workspaces.
#include <math.h>

#include <atomic>
#include <stdint.h>
#include <string.h>

#include "kda_common.cuh"
#include "kda_paths.h"

namespace kda {

int cuda_fail(cudaError_t e);

static size_t esize(int dtype) { return dtype == KDA_BF16 ? 2 : 4; }
static bool dtype_ok(int dtype) { return dtype == KDA_F32 || dtype == KDA_BF16; }
static bool misaligned(const void* p, size_t a) { return ((uintptr_t)p & (a - 1)) != 0; }

// Bytes that `rows` rows of `width` elements, `stride` apart, span.
static size_t span(int64_t rows, int64_t stride, int64_t width, size_t esz) {
    return rows > 0 && width > 0 ? ((size_t)(rows - 1) * (size_t)stride + (size_t)width) * esz : 0;
}

struct Range { const void* p; size_t n; };
static bool overlap(const Range& a, const Range& b) {
    if (!a.p || !b.p || !a.n || !b.n) return false;
    const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
    return x < y + b.n && y < x + a.n;
}
// Whether some output meets an input or another output.
static bool any_overlap(const Range* outs, int no, const Range* ins, int ni) {
    for (int i = 0; i < no; ++i) {
        for (int j = 0; j < ni; ++j)
            if (overlap(outs[i], ins[j])) return true;
        for (int j = i + 1; j < no; ++j)
            if (overlap(outs[i], outs[j])) return true;
    }
    return false;
}

constexpr size_t kStatusBytes = sizeof(DeviceHeader);

static std::atomic<int> g_drop{kDropNone};              // kda_selftest_drop_arrival

static int latent_common(const kda_latent_desc* d) {
    if (!d || d->num_seqs < 0 || d->num_heads < 1 || !dtype_ok(d->dtype)) return KDA_ERR_INVALID_ARGUMENT;
    if (d->flags & ~(KDA_FLAG_CUDA_CORE_PREFILL | KDA_FLAG_NO_CAUSAL)) return KDA_ERR_INVALID_ARGUMENT;
    if (!(d->scale > 0.f) || !isfinite(d->scale)) return KDA_ERR_INVALID_ARGUMENT;
    if (d->d_k < 1 || d->d_rope < 0 || d->d_v < 1) return KDA_ERR_INVALID_ARGUMENT;
    if (d->num_heads > 65535) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}
static int prefill_desc(const kda_latent_desc* d) {
    if (int rc = latent_common(d)) return rc;
    if (d->total_q < 0 || d->total_k < 0 || d->total_q > 0x7fffffffLL || d->total_k > 0x7fffffffLL)
        return KDA_ERR_INVALID_ARGUMENT;
    if (d->d_k + d->d_rope > 256 || d->d_v > 256) return KDA_ERR_UNSUPPORTED;
    const int64_t st[7] = {d->q_token_stride, d->q_head_stride, d->k_token_stride, d->k_head_stride,
                           d->v_token_stride, d->v_head_stride, d->rope_token_stride};
    for (int i = 0; i < 7; ++i)
        if (st[i] < 0) return KDA_ERR_INVALID_ARGUMENT;
    return KDA_OK;
}
static int decode_desc(const kda_latent_desc* d) {
    if (int rc = latent_common(d)) return rc;
    if (d->flags & KDA_FLAG_NO_CAUSAL) return KDA_ERR_INVALID_ARGUMENT;
    if (d->num_queries < 1 || d->page_size < 1 || d->num_pages < 0 || d->max_pages < 1 || d->d_v != d->d_k)
        return KDA_ERR_INVALID_ARGUMENT;
    if (d->q_token_stride < 0 || d->q_head_stride < 0) return KDA_ERR_INVALID_ARGUMENT;
    if (d->page_stride < (int64_t)d->page_size * (d->d_k + d->d_rope)) return KDA_ERR_INVALID_ARGUMENT;
    if (d->d_k > 512 || d->d_k + d->d_rope > 640) return KDA_ERR_UNSUPPORTED;
    if ((int64_t)d->max_pages * d->page_size > 0x7fffffffLL) return KDA_ERR_UNSUPPORTED;
    if ((int64_t)d->num_seqs * d->num_queries > 0x7fffffffLL) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}
static bool decode_tc(const kda_latent_desc* d) {
    return (d->flags & KDA_FLAG_CUDA_CORE_PREFILL) == 0 &&
           latent_decode_tc_takes(d->dtype, d->d_k, d->d_rope, d->num_heads, d->num_queries, d->page_size);
}
static int workspace_fault(const kda_latent_desc* d, size_t need) {
    return !d->workspace || d->workspace_bytes < need || misaligned(d->workspace, 256);
}

// Status of a call that computes nothing.  It needs no workspace; one that is not device memory is left alone.
static int nothing_to_compute(const kda_latent_desc* d, const int32_t* cu_q, const int32_t* cu_k, kda_stream_t stream) {
    if (workspace_fault(d, kStatusBytes) || misaligned(cu_q, 4) || misaligned(cu_k, 4)) return KDA_OK;
    cudaPointerAttributes at = {};
    if (cudaPointerGetAttributes(&at, d->workspace) != cudaSuccess) {
        cudaGetLastError();
        return KDA_OK;
    }
    if (at.type != cudaMemoryTypeDevice && at.type != cudaMemoryTypeManaged) return KDA_OK;
    const cudaError_t err = latent_status_launch(cu_q, cu_k, d->num_seqs, d->total_q, d->total_k, (int32_t*)d->workspace,
                                                 (cudaStream_t)stream);
    return err == cudaSuccess ? KDA_OK : cuda_fail(err);
}

}  // namespace kda

using namespace kda;

extern "C" {

int kda_rms_norm(const kda_norm_desc* d, const void* x, const void* weight, const void* residual,
                 void* residual_out, void* normed, uint8_t* quantized, float* scales, kda_stream_t stream) {
    if (!d || d->rows < 0 || d->dim < 1 || !dtype_ok(d->dtype)) return KDA_ERR_INVALID_ARGUMENT;
    if (!(d->eps >= 0.f) || !isfinite(d->eps)) return KDA_ERR_INVALID_ARGUMENT;
    if (d->x_stride < d->dim || (residual && d->residual_stride < d->dim)) return KDA_ERR_INVALID_ARGUMENT;
    if ((quantized == nullptr) != (scales == nullptr)) return KDA_ERR_INVALID_ARGUMENT;
    if (d->rows > 0x7fffffffLL || d->dim > (1 << 30)) return KDA_ERR_UNSUPPORTED;
    if (d->rows == 0) return KDA_OK;
    if (!x || (!residual_out && !normed && !quantized)) return KDA_ERR_INVALID_ARGUMENT;
    const size_t e = esize(d->dtype);
    if (misaligned(x, e) || misaligned(weight, e) || misaligned(residual, e) || misaligned(residual_out, e) ||
        misaligned(normed, e) || misaligned(scales, 4)) return KDA_ERR_INVALID_ARGUMENT;
    const size_t dense = (size_t)d->rows * d->dim;
    const Range xr = {x, span(d->rows, d->x_stride, d->dim, e)};
    const Range rr = {residual, span(d->rows, d->residual_stride, d->dim, e)};
    // h over x or over the residual, exactly, is an update in place
    const bool over_x = residual_out == x && d->x_stride == d->dim;
    const bool over_r = residual_out == residual && d->residual_stride == d->dim;
    const Range h = {residual_out, dense * e};
    const Range hin[3] = {over_x ? Range{nullptr, 0} : xr, over_r ? Range{nullptr, 0} : rr, {weight, d->dim * e}};
    if (any_overlap(&h, 1, hin, 3)) return KDA_ERR_INVALID_ARGUMENT;
    const size_t blocks = (d->dim + 127) / 128;
    const Range outs[3] = {{normed, dense * e}, {quantized, dense}, {scales, (size_t)d->rows * blocks * 4}};
    const Range ins[4] = {xr, rr, {weight, d->dim * e}, h};
    if (any_overlap(outs, 3, ins, 4)) return KDA_ERR_INVALID_ARGUMENT;
    const cudaError_t err = rms_norm_launch(*d, x, weight, residual, residual_out, normed, quantized, scales,
                                            (cudaStream_t)stream);
    return err == cudaSuccess ? KDA_OK : cuda_fail(err);
}

int kda_matmul_fp8(const kda_matmul_desc* d, const uint8_t* a, const float* a_scale, const uint8_t* b,
                   const float* b_scale, void* c, kda_stream_t stream) {
    if (!d || d->m < 0 || d->n < 0 || d->k < 1 || !dtype_ok(d->dtype)) return KDA_ERR_INVALID_ARGUMENT;
    if (d->flags & ~KDA_FLAG_CUDA_CORE_PREFILL) return KDA_ERR_INVALID_ARGUMENT;
    if (d->a_stride < d->k || d->b_stride < d->k || d->c_stride < d->n) return KDA_ERR_INVALID_ARGUMENT;
    if (d->m > 0x7fffffffLL || d->n > 65535 * 64) return KDA_ERR_UNSUPPORTED;
    if (d->m == 0 || d->n == 0) return KDA_OK;
    if (!a || !a_scale || !b || !b_scale || !c) return KDA_ERR_INVALID_ARGUMENT;
    const size_t e = esize(d->dtype), kb = ((size_t)d->k + 127) / 128, nb = ((size_t)d->n + 127) / 128;
    if (misaligned(a_scale, 4) || misaligned(b_scale, 4) || misaligned(c, e)) return KDA_ERR_INVALID_ARGUMENT;
    const Range out = {c, span(d->m, d->c_stride, d->n, e)};
    const Range ins[4] = {{a, span(d->m, d->a_stride, d->k, 1)}, {a_scale, (size_t)d->m * kb * 4},
                          {b, span(d->n, d->b_stride, d->k, 1)}, {b_scale, nb * kb * 4}};
    if (any_overlap(&out, 1, ins, 4)) return KDA_ERR_INVALID_ARGUMENT;
    MatmulArgs m;
    m.m = d->m; m.lda = d->a_stride; m.ldb = d->b_stride; m.ldc = d->c_stride;
    m.n = d->n; m.k = d->k; m.dtype = d->dtype; m.drop = g_drop.load(std::memory_order_relaxed);
    m.a = a; m.b = b; m.sa = a_scale; m.sb = b_scale; m.c = c;
    const bool tc = (d->flags & KDA_FLAG_CUDA_CORE_PREFILL) == 0 && matmul_tc_takes(m);
    const cudaError_t err = tc ? matmul_tc_launch(m, (cudaStream_t)stream) : matmul_simt_launch(m, (cudaStream_t)stream);
    return err == cudaSuccess ? KDA_OK : cuda_fail(err);
}

size_t kda_latent_prefill_workspace_bytes(const kda_latent_desc* d) {
    return prefill_desc(d) ? 0 : kStatusBytes;
}

size_t kda_latent_decode_workspace_bytes(const kda_latent_desc* d) {
    if (decode_desc(d)) return 0;
    const bool tc = decode_tc(d);
    return kStatusBytes + (tc ? latent_decode_tc_bytes(d->num_seqs, d->num_queries, d->num_heads, d->page_size, d->max_pages) : 0);
}

int kda_latent_prefill(const kda_latent_desc* d, const void* q, const void* k_nope, const void* k_rope,
                       const void* v, const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k, void* out,
                       float* lse, kda_stream_t stream) {
    if (int rc = prefill_desc(d)) return rc;
    if ((cu_seqlens_q == nullptr) != (cu_seqlens_k == nullptr)) return KDA_ERR_INVALID_ARGUMENT;
    if (!cu_seqlens_q && d->num_seqs != 1) return KDA_ERR_INVALID_ARGUMENT;
    if (d->num_seqs == 0 || d->total_q == 0) return nothing_to_compute(d, cu_seqlens_q, cu_seqlens_k, stream);
    if (!q || !out) return KDA_ERR_INVALID_ARGUMENT;
    if (d->total_k > 0 && (!k_nope || !v || (d->d_rope > 0) != (k_rope != nullptr))) return KDA_ERR_INVALID_ARGUMENT;
    const size_t e = esize(d->dtype);
    if (misaligned(q, e) || misaligned(k_nope, e) || misaligned(k_rope, e) || misaligned(v, e) ||
        misaligned(out, e) || misaligned(lse, 4) || misaligned(cu_seqlens_q, 4) || misaligned(cu_seqlens_k, 4))
        return KDA_ERR_INVALID_ARGUMENT;
    const int64_t H = d->num_heads, tq = d->total_q, tk = d->total_k;
    auto rows = [&](int64_t t, int64_t ts, int64_t hs, int64_t w) {
        return t > 0 ? ((size_t)(t - 1) * ts + (size_t)(H - 1) * hs + (size_t)w) * e : (size_t)0;
    };
    const size_t ncu = ((size_t)d->num_seqs + 1) * 4;
    const Range outs[3] = {{out, (size_t)tq * H * d->d_v * e}, {lse, (size_t)tq * H * 4},
                           {d->workspace, d->workspace_bytes}};
    const Range ins[6] = {{q, rows(tq, d->q_token_stride, d->q_head_stride, d->d_k + d->d_rope)},
                          {k_nope, rows(tk, d->k_token_stride, d->k_head_stride, d->d_k)},
                          {k_rope, span(tk, d->rope_token_stride, d->d_rope, e)},
                          {v, rows(tk, d->v_token_stride, d->v_head_stride, d->d_v)},
                          {cu_seqlens_q, ncu}, {cu_seqlens_k, ncu}};
    if (any_overlap(outs, 3, ins, 6)) return KDA_ERR_INVALID_ARGUMENT;
    if (workspace_fault(d, kStatusBytes)) return KDA_ERR_WORKSPACE;
    LatentPrefillArgs a;
    a.dtype = d->dtype; a.N = d->num_seqs; a.H = d->num_heads; a.dk = d->d_k; a.dr = d->d_rope; a.dv = d->d_v;
    a.causal = (d->flags & KDA_FLAG_NO_CAUSAL) == 0; a.drop = g_drop.load(std::memory_order_relaxed); a.scale = d->scale; a.tq = tq; a.tk = tk;
    a.q_ts = d->q_token_stride; a.q_hs = d->q_head_stride; a.k_ts = d->k_token_stride; a.k_hs = d->k_head_stride;
    a.v_ts = d->v_token_stride; a.v_hs = d->v_head_stride; a.r_ts = d->rope_token_stride;
    a.q = q; a.k = k_nope; a.r = k_rope; a.v = v; a.cu_q = cu_seqlens_q; a.cu_k = cu_seqlens_k;
    a.out = out; a.lse = lse; a.status = (int32_t*)d->workspace;
    cudaStream_t s = (cudaStream_t)stream;
    const bool tc = (d->flags & KDA_FLAG_CUDA_CORE_PREFILL) == 0 && latent_prefill_tc_takes(a);
    const cudaError_t err = tc ? latent_prefill_tc_launch(a, s) : latent_prefill_simt_launch(a, s);
    return err == cudaSuccess ? KDA_OK : cuda_fail(err);
}

int kda_latent_decode(const kda_latent_desc* d, const void* q, const void* cache, const int32_t* page_table,
                      const int32_t* lengths, void* out, float* lse, kda_stream_t stream) {
    if (int rc = decode_desc(d)) return rc;
    if (d->num_seqs == 0) return nothing_to_compute(d, nullptr, nullptr, stream);
    if (!q || !out || !page_table || !lengths || (d->num_pages > 0 && !cache)) return KDA_ERR_INVALID_ARGUMENT;
    const size_t e = esize(d->dtype);
    if (misaligned(q, e) || misaligned(cache, e) || misaligned(out, e) || misaligned(lse, 4) ||
        misaligned(page_table, 4) || misaligned(lengths, 4)) return KDA_ERR_INVALID_ARGUMENT;
    const int64_t rows = (int64_t)d->num_seqs * d->num_queries, H = d->num_heads, w = d->d_k + d->d_rope;
    const Range outs[3] = {{out, (size_t)rows * H * d->d_k * e}, {lse, (size_t)rows * H * 4},
                           {d->workspace, d->workspace_bytes}};
    const Range ins[4] = {{q, ((size_t)(rows - 1) * d->q_token_stride + (size_t)(H - 1) * d->q_head_stride + w) * e},
                          {cache, span(d->num_pages, d->page_stride, (int64_t)d->page_size * w, e)},
                          {page_table, (size_t)d->num_seqs * d->max_pages * 4}, {lengths, (size_t)d->num_seqs * 4}};
    if (any_overlap(outs, 3, ins, 4)) return KDA_ERR_INVALID_ARGUMENT;
    if (workspace_fault(d, kda_latent_decode_workspace_bytes(d))) return KDA_ERR_WORKSPACE;
    LatentDecodeArgs a;
    a.dtype = d->dtype; a.N = d->num_seqs; a.H = d->num_heads; a.Lq = d->num_queries; a.dk = d->d_k; a.dr = d->d_rope;
    a.drop = g_drop.load(std::memory_order_relaxed);
    a.scale = d->scale; a.q_ts = d->q_token_stride; a.q_hs = d->q_head_stride; a.page_stride = d->page_stride;
    a.page_size = d->page_size; a.num_pages = d->num_pages; a.max_pages = d->max_pages;
    a.q = q; a.cache = cache; a.table = page_table; a.lens = lengths; a.out = out; a.lse = lse;
    a.status = (int32_t*)d->workspace; a.scratch = (char*)d->workspace + kStatusBytes;
    cudaStream_t s = (cudaStream_t)stream;
    cudaError_t err;
    if (decode_tc(d) && latent_decode_tc_aligned(a)) {
        err = latent_decode_tc_launch(a, s);
    } else {
        err = cudaMemsetAsync(a.status, 0, sizeof(int32_t), s);
        if (err == cudaSuccess) err = latent_decode_simt_launch(a, s);
    }
    return err == cudaSuccess ? KDA_OK : cuda_fail(err);
}

int kda_selftest_drop_arrival(int32_t which) {
    if (which < kDropNone || which > kDropRows) return KDA_ERR_INVALID_ARGUMENT;
    g_drop.store(which, std::memory_order_relaxed);
    return KDA_OK;
}

int kda_latent_status(const kda_latent_desc* d, kda_stream_t stream) {
    if (!d || !d->workspace || d->workspace_bytes < kStatusBytes) return KDA_ERR_WORKSPACE;
    int32_t status = 0;
    cudaStream_t s = (cudaStream_t)stream;
    cudaError_t e = cudaMemcpyAsync(&status, d->workspace, sizeof(status), cudaMemcpyDeviceToHost, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    return e == cudaSuccess ? status : cuda_fail(e);
}

}  // extern "C"
