// kda_operators_api.cu -- C entries of the operators around the recurrent
// layers: argument checks, choice of path, workspaces.
#include <math.h>

#include <atomic>
#include <numeric>
#include <stdint.h>
#include <string.h>

#include "kda_common.cuh"
#include "kda_latent_cache.cuh"
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
    if (d->flags & ~(KDA_FLAG_CUDA_CORE_PREFILL | KDA_FLAG_NO_CAUSAL | KDA_FLAG_CACHE_8)) return KDA_ERR_INVALID_ARGUMENT;
    if (!(d->scale > 0.f) || !isfinite(d->scale)) return KDA_ERR_INVALID_ARGUMENT;
    if (d->d_k < 1 || d->d_rope < 0 || d->d_v < 1) return KDA_ERR_INVALID_ARGUMENT;
    if (d->num_heads > 65535) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}
static int prefill_desc(const kda_latent_desc* d) {
    if (int rc = latent_common(d)) return rc;
    if (d->flags & KDA_FLAG_CACHE_8) return KDA_ERR_INVALID_ARGUMENT;
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
    if (d->flags & KDA_FLAG_CACHE_8) {
        const int64_t page = kda_latent_cache_page_bytes(d->page_size, d->d_k, d->d_rope);
        if (page == 0) return KDA_ERR_UNSUPPORTED;
        if (d->page_stride < page || d->page_stride % 16 != 0) return KDA_ERR_INVALID_ARGUMENT;
    } else if (d->page_stride < (int64_t)d->page_size * (d->d_k + d->d_rope)) {
        return KDA_ERR_INVALID_ARGUMENT;
    }
    if (d->d_k > 512 || d->d_k + d->d_rope > 640) return KDA_ERR_UNSUPPORTED;
    if ((int64_t)d->max_pages * d->page_size > 0x7fffffffLL) return KDA_ERR_UNSUPPORTED;
    if ((int64_t)d->num_seqs * d->num_queries > 0x7fffffffLL) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}
static bool decode_tc(const kda_latent_desc* d) {
    if (d->flags & KDA_FLAG_CUDA_CORE_PREFILL) return false;
    if (d->flags & KDA_FLAG_CACHE_8)
        return latent_decode8_tc_takes(d->dtype, d->d_k, d->d_rope, d->num_heads, d->num_queries, d->page_size);
    return latent_decode_tc_takes(d->dtype, d->d_k, d->d_rope, d->num_heads, d->num_queries, d->page_size);
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

// Rows of several heads a token, for the rotary positions (bytes).
struct Rows { const void* p; int64_t token, head; size_t row, span, width; };    // row: from a token's first byte behind its last
static Rows rows_of(const void* p, const kda_rotary_part& s, int64_t tokens, size_t e, bool out) {
    const int64_t token = out ? s.out_token_stride : s.token_stride, head = out ? s.out_head_stride : s.head_stride;
    // (one token or one head: no stride)
    Rows r = {p, tokens > 1 ? token * (int64_t)e : 0, s.heads > 1 ? head * (int64_t)e : 0, 0, 0, s.width * e};
    if (!p) return r;
    r.row = (size_t)(s.heads - 1) * (size_t)r.head + r.width;
    r.span = (size_t)(tokens - 1) * (size_t)r.token + r.row;
    return r;
}
// Whether [x, x + a) and [y, y + b) meet, both repeated every s bytes.
static bool meet_modulo(const void* x, size_t a, const void* y, size_t b, size_t s) {
    if (s < a || s < b) return true;
    const uintptr_t u = (uintptr_t)x, v = (uintptr_t)y;
    const size_t d = v >= u ? (v - u) % s : (s - (u - v) % s) % s;     // where b's begins behind a's
    return d < a || d + b > s;
}
static bool rows_meet(const Rows& a, const Rows& b) {
    if (!overlap({a.p, a.span}, {b.p, b.span})) return false;
    // Parts of the same wider rows, a token's all together; or of wider rows that repeat by a divisor of all strides, as
    // where queries and keys lie side by side in each head
    if (a.token == b.token && a.token > 0 && !meet_modulo(a.p, a.row, b.p, b.row, a.token)) return false;
    const int64_t every = std::gcd(std::gcd(a.token, b.token), std::gcd(a.head, b.head));
    return every == 0 || meet_modulo(a.p, a.width, b.p, b.width, every);
}
static int rotary_part(const kda_rotary_part& p, int64_t tokens, int dim) {
    if (p.heads < 1 || p.reserved != 0 || p.offset < 0 || p.width < dim || p.offset > p.width - dim) return KDA_ERR_INVALID_ARGUMENT;
    if (p.token_stride < 0 || p.head_stride < 0 || p.out_token_stride < 0 || p.out_head_stride < 0) return KDA_ERR_INVALID_ARGUMENT;
    if (p.heads > 65535 || p.width > 4096) return KDA_ERR_UNSUPPORTED;
    const int64_t most = 1ll << 46;                    // (no product of a stride with a count passes 64 bits)
    if (p.token_stride > most / (tokens + 1) || p.out_token_stride > most / (tokens + 1) || p.head_stride > most / p.heads ||
        p.out_head_stride > most / p.heads) return KDA_ERR_UNSUPPORTED;
    // The output's rows: heads inside tokens, or tokens inside heads
    const bool h1 = p.heads == 1, t1 = tokens <= 1;
    const bool inside = (h1 || p.out_head_stride >= p.width) && (t1 || p.out_token_stride >= (p.heads - 1) * p.out_head_stride + p.width);
    const bool across = (t1 || p.out_token_stride >= p.width) && (h1 || p.out_head_stride >= (tokens - 1) * p.out_token_stride + p.width);
    return inside || across ? KDA_OK : KDA_ERR_INVALID_ARGUMENT;
}

static int cache_call(const kda_latent_cache_desc* d, bool write, void* latents, void* rope, const int32_t* cu,
                      const int32_t* table, const int32_t* lens, uint8_t* cache, kda_stream_t stream) {
    if (!d || d->num_seqs < 0 || !dtype_ok(d->dtype) || d->total_tokens < 0 || d->flags != 0) return KDA_ERR_INVALID_ARGUMENT;
    if (d->page_size < 1 || d->num_pages < 0 || d->max_pages < 1 || d->rank < 1 || d->d_rope < 0) return KDA_ERR_INVALID_ARGUMENT;
    const int64_t page = kda_latent_cache_page_bytes(d->page_size, d->rank, d->d_rope);
    if (page == 0 || (int64_t)d->max_pages * d->page_size > 0x7fffffffLL || d->total_tokens > 0x7fffffffLL) return KDA_ERR_UNSUPPORTED;
    if (d->page_stride < page || d->page_stride % 16 != 0) return KDA_ERR_INVALID_ARGUMENT;
    if (d->latent_stride < d->rank || d->rope_stride < d->d_rope) return KDA_ERR_INVALID_ARGUMENT;
    const int64_t T = d->total_tokens, N = d->num_seqs;
    if (!cu && T > 0 && (N == 0 || T % N != 0)) return KDA_ERR_INVALID_ARGUMENT;
    if (d->workspace && (d->workspace_bytes < kStatusBytes || misaligned(d->workspace, 256))) return KDA_ERR_WORKSPACE;
    if ((N == 0 || T == 0) && !d->workspace) return KDA_OK;
    if (N > 0 && (!table || !lens || (d->num_pages > 0 && !cache))) return KDA_ERR_INVALID_ARGUMENT;
    if (N > 0 && T > 0 && (!latents || (d->d_rope > 0) != (rope != nullptr))) return KDA_ERR_INVALID_ARGUMENT;
    const size_t e = esize(d->dtype);
    if (misaligned(latents, e) || misaligned(rope, e) || misaligned(cu, 4) || misaligned(table, 4) || misaligned(lens, 4) ||
        misaligned(cache, 16)) return KDA_ERR_INVALID_ARGUMENT;
    const Rows c = {latents, d->latent_stride * (int64_t)e, 0, d->rank * e, span(T, d->latent_stride, d->rank, e), d->rank * e};
    const Rows r = {rope, d->rope_stride * (int64_t)e, 0, d->d_rope * e, span(T, d->rope_stride, d->d_rope, e), d->d_rope * e};
    const Range pages = {cache, span(d->num_pages, d->page_stride, page, 1)}, status = {d->workspace, d->workspace ? kStatusBytes : 0};
    const Range ints[3] = {{cu, cu ? ((size_t)N + 1) * 4 : 0}, {table, (size_t)N * d->max_pages * 4}, {lens, (size_t)N * 4}};
    const Range lat = {latents, c.span}, rop = {rope, r.span};
    if (overlap(pages, lat) || overlap(pages, rop) || overlap(status, lat) || overlap(status, rop) || overlap(status, pages))
        return KDA_ERR_INVALID_ARGUMENT;
    if (write ? any_overlap(&pages, 1, ints, 3) : any_overlap(&lat, 1, ints, 3) || any_overlap(&rop, 1, ints, 3) || rows_meet(c, r))
        return KDA_ERR_INVALID_ARGUMENT;
    if (any_overlap(&status, 1, ints, 3)) return KDA_ERR_INVALID_ARGUMENT;
    LatentCacheArgs a;                                 // (without rows or sequences: the status alone)
    a.dtype = d->dtype; a.N = d->num_seqs; a.rank = d->rank; a.d_rope = d->d_rope; a.page_size = d->page_size;
    a.num_pages = d->num_pages; a.max_pages = d->max_pages; a.T = N > 0 ? T : 0; a.rows_each = cu || N == 0 ? 0 : T / N;
    a.page_stride = d->page_stride; a.latent_stride = d->latent_stride; a.rope_stride = d->rope_stride;
    a.latents = latents; a.rope = rope; a.cu = cu; a.table = table; a.lens = lens; a.cache = cache;
    a.status = (int32_t*)d->workspace;
    const cudaError_t err = latent_cache_launch(a, write, (cudaStream_t)stream);
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
    if (tc && (d->flags & KDA_FLAG_CACHE_8))
        return kStatusBytes + latent_decode8_tc_bytes(d->num_seqs, d->num_queries, d->num_heads, d->page_size, d->max_pages);
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
    const bool codes = (d->flags & KDA_FLAG_CACHE_8) != 0;
    if (misaligned(q, e) || misaligned(cache, codes ? 16 : e) || misaligned(out, e) || misaligned(lse, 4) ||
        misaligned(page_table, 4) || misaligned(lengths, 4)) return KDA_ERR_INVALID_ARGUMENT;
    const int64_t rows = (int64_t)d->num_seqs * d->num_queries, H = d->num_heads, w = d->d_k + d->d_rope;
    const Range outs[3] = {{out, (size_t)rows * H * d->d_k * e}, {lse, (size_t)rows * H * 4},
                           {d->workspace, d->workspace_bytes}};
    const Range ins[4] = {{q, ((size_t)(rows - 1) * d->q_token_stride + (size_t)(H - 1) * d->q_head_stride + w) * e},
                          {cache, codes ? span(d->num_pages, d->page_stride, latent_page_bytes(d->page_size, d->d_k, d->d_rope), 1)
                                        : span(d->num_pages, d->page_stride, (int64_t)d->page_size * w, e)},
                          {page_table, (size_t)d->num_seqs * d->max_pages * 4}, {lengths, (size_t)d->num_seqs * 4}};
    if (any_overlap(outs, 3, ins, 4)) return KDA_ERR_INVALID_ARGUMENT;
    if (workspace_fault(d, kda_latent_decode_workspace_bytes(d))) return KDA_ERR_WORKSPACE;
    LatentDecodeArgs a;
    a.dtype = d->dtype; a.N = d->num_seqs; a.H = d->num_heads; a.Lq = d->num_queries; a.dk = d->d_k; a.dr = d->d_rope;
    a.codes = codes;
    a.drop = g_drop.load(std::memory_order_relaxed);
    a.scale = d->scale; a.q_ts = d->q_token_stride; a.q_hs = d->q_head_stride; a.page_stride = d->page_stride;
    a.page_size = d->page_size; a.num_pages = d->num_pages; a.max_pages = d->max_pages;
    a.q = q; a.cache = cache; a.table = page_table; a.lens = lengths; a.out = out; a.lse = lse;
    a.status = (int32_t*)d->workspace; a.scratch = (char*)d->workspace + kStatusBytes;
    cudaStream_t s = (cudaStream_t)stream;
    cudaError_t err;
    if (decode_tc(d) && codes && latent_decode8_tc_aligned(a)) {
        err = latent_decode8_tc_launch(a, s);
    } else if (decode_tc(d) && !codes && latent_decode_tc_aligned(a)) {
        err = latent_decode_tc_launch(a, s);
    } else {
        err = cudaMemsetAsync(a.status, 0, sizeof(int32_t), s);
        if (err == cudaSuccess) err = latent_decode_simt_launch(a, s);
    }
    return err == cudaSuccess ? KDA_OK : cuda_fail(err);
}

size_t kda_latent_cache_page_bytes(int32_t page_size, int32_t rank, int32_t d_rope) {
    if (page_size < 1 || rank < 16 || rank > 512 || rank % 16 != 0 || d_rope < 0 || d_rope > 128 || d_rope % 8 != 0) return 0;
    return (size_t)latent_page_bytes(page_size, rank, d_rope);
}

int kda_latent_cache_write(const kda_latent_cache_desc* d, const void* latents, const void* rope, const int32_t* cu_seqlens,
                           const int32_t* page_table, const int32_t* lengths, uint8_t* cache, kda_stream_t stream) {
    return cache_call(d, true, (void*)latents, (void*)rope, cu_seqlens, page_table, lengths, cache, stream);
}

int kda_latent_cache_read(const kda_latent_cache_desc* d, const uint8_t* cache, const int32_t* page_table,
                          const int32_t* lengths, const int32_t* cu_seqlens, void* latents, void* rope, kda_stream_t stream) {
    return cache_call(d, false, latents, rope, cu_seqlens, page_table, lengths, (uint8_t*)cache, stream);
}

int kda_rotary_frequencies(int32_t dim, double base, int32_t method, double factor, double original_length, double slow,
                           double fast, double* frequencies) {
    if (dim < 2 || dim % 2 != 0 || !frequencies || !(base > 0.) || !isfinite(base)) return KDA_ERR_INVALID_ARGUMENT;
    if (method < KDA_ROTARY_PLAIN || method > KDA_ROTARY_BY_PARTS) return KDA_ERR_INVALID_ARGUMENT;
    if (dim > 1024) return KDA_ERR_UNSUPPORTED;
    if (method != KDA_ROTARY_PLAIN && (!(factor > 0.) || !isfinite(factor))) return KDA_ERR_INVALID_ARGUMENT;
    if (method == KDA_ROTARY_BASE && dim == 2) return KDA_ERR_INVALID_ARGUMENT;
    if (method == KDA_ROTARY_BY_PARTS && (!(original_length > 0.) || !isfinite(original_length) || !(slow >= 0.) || !(fast > slow) ||
                                          !isfinite(fast))) return KDA_ERR_INVALID_ARGUMENT;
    if (method == KDA_ROTARY_BASE) base *= pow(factor, dim / (dim - 2.));
    for (int i = 0; i < dim / 2; ++i) {
        double f = pow(base, -2. * i / dim);
        if (method == KDA_ROTARY_LINEAR) f /= factor;
        if (method == KDA_ROTARY_BY_PARTS) {
            double w = (original_length * f / 6.283185307179586477 - slow) / (fast - slow);
            w = w < 0. ? 0. : w > 1. ? 1. : w;
            f *= w + (1. - w) / factor;
        }
        frequencies[i] = f;
    }
    return KDA_OK;
}

int kda_rotary(const kda_rotary_desc* d, const void* x, const void* key, const void* positions, const double* frequencies,
               void* out, void* key_out, kda_stream_t stream) {
    if (!d || d->tokens < 0 || d->dim < 2 || d->dim % 2 != 0 || !dtype_ok(d->dtype) || !isfinite(d->scale)) return KDA_ERR_INVALID_ARGUMENT;
    if (d->flags & ~(KDA_FLAG_INTERLEAVED | KDA_FLAG_INVERSE | KDA_FLAG_POSITIONS_64)) return KDA_ERR_INVALID_ARGUMENT;
    if ((key == nullptr) != (key_out == nullptr) && d->tokens > 0) return KDA_ERR_INVALID_ARGUMENT;
    if (d->dim > 1024 || d->tokens > 0x7fffffffLL) return KDA_ERR_UNSUPPORTED;
    const bool two = key != nullptr || key_out != nullptr;
    for (int i = 0; i < (two ? 2 : 1); ++i) {
        if (int rc = rotary_part(i ? d->key : d->x, d->tokens, d->dim)) return rc;
    }
    if (d->tokens == 0) return KDA_OK;
    if (!x || !out || !positions || !frequencies) return KDA_ERR_INVALID_ARGUMENT;
    const size_t e = esize(d->dtype), pos = d->flags & KDA_FLAG_POSITIONS_64 ? 8 : 4;
    if (misaligned(x, e) || misaligned(out, e) || misaligned(key, e) || misaligned(key_out, e) || misaligned(positions, pos) ||
        misaligned(frequencies, 8)) return KDA_ERR_INVALID_ARGUMENT;
    const Rows in[2] = {rows_of(x, d->x, d->tokens, e, false), rows_of(key, d->key, d->tokens, e, false)};
    const Rows to[2] = {rows_of(out, d->x, d->tokens, e, true), rows_of(key_out, d->key, d->tokens, e, true)};
    const Range read[2] = {{positions, (size_t)d->tokens * pos}, {frequencies, (size_t)d->dim / 2 * 8}};
    for (int i = 0; i < 2; ++i) {
        for (int j = 0; j < 2; ++j) {
            const bool own = i == j && to[i].p == in[i].p && to[i].token == in[i].token && to[i].head == in[i].head;
            if (!own && rows_meet(to[i], in[j])) return KDA_ERR_INVALID_ARGUMENT;
            if (overlap({to[i].p, to[i].span}, read[j])) return KDA_ERR_INVALID_ARGUMENT;
        }
    }
    if (rows_meet(to[0], to[1])) return KDA_ERR_INVALID_ARGUMENT;
    const cudaError_t err = rotary_launch(*d, x, key, positions, frequencies, out, key_out, (cudaStream_t)stream);
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
