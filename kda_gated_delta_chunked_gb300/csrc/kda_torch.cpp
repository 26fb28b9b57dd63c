// kda_torch.cpp -- marshalling of torch tensors for the operators around the
// recurrent layers: checks, outputs, descriptors, the C call.  These calls are
// short (a token's norm is 3 us of GPU time), so what Python and ctypes would
// spend on them (12 to 23 us a call on the host) is spent here instead.
//
// The entry points' addresses come from the loaded libkda (bind), so there is
// one library in the process.  Refusals are ValueErrors; an error code of a C
// call is returned as an int, which the Python layer raises.  Work goes to the
// current stream, outputs and workspaces come from torch's allocator on it.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <array>
#include <sstream>
#include <stdexcept>

#include "../../include/kda.h"

namespace {

struct Api {
    decltype(&kda_rms_norm) rms_norm;
    decltype(&kda_matmul_fp8) matmul_fp8;
    decltype(&kda_latent_prefill_workspace_bytes) prefill_bytes;
    decltype(&kda_latent_decode_workspace_bytes) decode_bytes;
    decltype(&kda_latent_prefill) prefill;
    decltype(&kda_latent_decode) decode;
    decltype(&kda_latent_cache_page_bytes) page_bytes;
    decltype(&kda_latent_cache_write) cache_write;
    decltype(&kda_latent_cache_read) cache_read;
    decltype(&kda_rotary) rotary;
} api = {};

template <typename... A>
[[noreturn]] void refuse(const A&... a) {
    std::ostringstream s;
    (s << ... << a);
    throw std::invalid_argument(s.str());
}

const at::Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) refuse(name, " must be a tensor");
    return THPVariable_Unpack(o);
}
// nullptr for None.
const at::Tensor* maybe(PyObject* o, const char* name) { return o == Py_None ? nullptr : &tensor(o, name); }

c10::Device device_of(const at::Tensor& t, const char* name) {
    if (!t.is_cuda() || t.get_device() != c10::cuda::current_device())
        refuse(name, " must be on the current CUDA device: got ", t.device());
    return t.device();
}
// `dim` dimensions, the last dense.
void rows(const at::Tensor& t, const char* name, at::ScalarType type, int64_t dim, c10::Device dev) {
    if (t.scalar_type() != type || t.dim() != dim || t.device() != dev || (t.size(dim - 1) > 1 && t.stride(dim - 1) != 1))
        refuse(name, " must be a ", dim, "-D ", type, " tensor on ", dev, " with a dense last dimension: got ", t.sizes(),
               ", ", t.scalar_type(), ", ", t.device(), ", strides ", t.strides());
}
void dense(const at::Tensor& t, const char* name, at::ScalarType type, at::IntArrayRef shape, c10::Device dev) {
    if (t.scalar_type() != type || t.sizes() != shape || t.device() != dev || !t.is_contiguous())
        refuse(name, " must be a contiguous ", shape, " ", type, " tensor on ", dev, ": got ", t.sizes(), ", ",
               t.scalar_type(), ", ", t.device(), ", strides ", t.strides());
}
int dtype_of(const at::Tensor& t, const char* name) {
    if (t.scalar_type() == at::kBFloat16) return KDA_BF16;
    if (t.scalar_type() == at::kFloat) return KDA_F32;
    refuse(name, " must be float32 or bfloat16: got ", t.scalar_type());
}
// Elements between rows of a 2-D tensor (a single row may carry any stride).
int64_t row_stride(const at::Tensor& t, int64_t width) { return t.size(0) > 1 ? t.stride(0) : width; }

at::Tensor fresh(at::IntArrayRef shape, at::ScalarType type, c10::Device dev) {
    return at::Tensor(at::detail::empty_cuda(shape, type, dev, std::nullopt));
}
template <typename T = void>
T* data(const at::Tensor* t) { return t ? (T*)t->data_ptr() : nullptr; }

kda_stream_t stream_of(c10::Device dev) { return (kda_stream_t)c10::cuda::getCurrentCUDAStream(dev.index()).stream(); }

PyObject* wrap(const at::Tensor& t) {
    if (!t.defined()) Py_RETURN_NONE;
    return THPVariable_Wrap(t);
}
template <size_t N>
PyObject* pack(const std::array<at::Tensor, N>& ts) {
    PyObject* r = PyTuple_New(N);
    if (!r) return nullptr;
    for (size_t i = 0; i < N; ++i) {
        PyObject* o = wrap(ts[i]);
        if (!o) { Py_DECREF(r); return nullptr; }
        PyTuple_SET_ITEM(r, i, o);
    }
    return r;
}

int64_t integer(PyObject* o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) { PyErr_Clear(); refuse("expected an integer"); }
    return v;
}
double number(PyObject* o, const char* name) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) { PyErr_Clear(); refuse(name, " must be a number"); }
    return v;
}

bool truth(PyObject* o, const char* name) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) { PyErr_Clear(); refuse(name, " must be true or false"); }
    return v;
}

// Descriptors hold some sizes in 32 bits.
int32_t narrow(int64_t x, const char* what) {
    if (x > 0x7fffffffLL || x < -0x80000000LL) refuse(what, " is too large: ", x);
    return (int32_t)x;
}

// ------------------------------------------------------------------ operators
// rms_norm(x, weight, residual, eps, normed, quantize, residual_out)
PyObject* rms_norm(PyObject* const* a) {
    const at::Tensor& x = tensor(a[0], "x");
    const at::Tensor *weight = maybe(a[1], "weight"), *residual = maybe(a[2], "residual"), *given = maybe(a[6], "residual_out");
    const bool normed = truth(a[4], "normed"), quantize = truth(a[5], "quantize");
    const c10::Device dev = device_of(x, "x");
    const at::ScalarType type = x.scalar_type();
    kda_norm_desc d = {};
    d.dtype = dtype_of(x, "x");
    if (x.dim() < 1 || x.size(-1) < 1) refuse("x must have rows of at least one element: got ", x.sizes());
    if (!normed && !quantize && !residual) refuse("nothing to compute: normed, quantize or a residual");
    const at::IntArrayRef shape = x.sizes();
    const int64_t dim = shape.back();
    d.rows = x.numel() / dim;
    d.dim = narrow(dim, "x's last dimension");
    d.eps = (float)number(a[3], "eps");
    d.x_stride = d.residual_stride = dim;
    if (x.dim() == 2) {
        rows(x, "x", type, 2, dev);
        d.x_stride = row_stride(x, dim);
    } else if (!x.is_contiguous()) {
        refuse("x must be contiguous unless it is 2-D");
    }
    if (weight) dense(*weight, "weight", type, {dim}, dev);
    if (residual) {
        if (residual->sizes() != shape) refuse("residual must have x's shape ", shape, ": got ", residual->sizes());
        if (x.dim() == 2) {
            rows(*residual, "residual", type, 2, dev);
            d.residual_stride = row_stride(*residual, dim);
        } else {
            dense(*residual, "residual", type, shape, dev);
        }
    } else if (given) {
        refuse("residual_out without a residual");
    }
    at::Tensor y, q, s, h;
    if (given) { dense(*given, "residual_out", type, shape, dev); h = *given; }
    else if (residual) h = fresh(shape, type, dev);
    if (normed) y = fresh(shape, type, dev);
    if (quantize) {
        c10::DimVector blocks(shape.begin(), shape.end());
        blocks.back() = (dim + 127) / 128;
        q = fresh(shape, at::kFloat8_e4m3fn, dev);
        s = fresh(blocks, at::kFloat, dev);
    }
    if (d.rows) {
        const int rc = api.rms_norm(&d, x.data_ptr(), data(weight), data(residual), h.defined() ? h.data_ptr() : nullptr,
                                    normed ? y.data_ptr() : nullptr, quantize ? (uint8_t*)q.data_ptr() : nullptr,
                                    quantize ? (float*)s.data_ptr() : nullptr, stream_of(dev));
        if (rc != KDA_OK) return PyLong_FromLong(rc);
    }
    return pack<4>({y, q, s, h});
}

// matmul_fp8(a, a_scale, b, b_scale, out, out is bf16, flags)
PyObject* matmul_fp8(PyObject* const* p) {
    const at::Tensor &a = tensor(p[0], "a"), &sa = tensor(p[1], "a_scale"), &b = tensor(p[2], "b"), &sb = tensor(p[3], "b_scale");
    const at::Tensor* given = maybe(p[4], "out");
    const c10::Device dev = device_of(a, "a");
    rows(a, "a", at::kFloat8_e4m3fn, 2, dev);
    rows(b, "b", at::kFloat8_e4m3fn, 2, dev);
    kda_matmul_desc d = {};
    const int64_t m = a.size(0), n = b.size(0), k = a.size(1), kb = (k + 127) / 128;
    if (b.size(1) != k || k < 1) refuse("a and b must have rows of the same length: got ", k, " and ", b.size(1));
    dense(sa, "a_scale", at::kFloat, {m, kb}, dev);
    dense(sb, "b_scale", at::kFloat, {(n + 127) / 128, kb}, dev);
    at::Tensor c;
    d.c_stride = n;
    if (given) {
        rows(*given, "out", given->scalar_type(), 2, dev);
        if (given->size(0) != m || given->size(1) != n) refuse("out must be [", m, ", ", n, "]: got ", given->sizes());
        c = *given;
        d.c_stride = row_stride(c, n);
    } else {
        c = fresh({m, n}, truth(p[5], "out_dtype") ? at::kBFloat16 : at::kFloat, dev);
    }
    d.m = m; d.n = narrow(n, "b's rows"); d.k = narrow(k, "the rows' length");
    d.a_stride = row_stride(a, k); d.b_stride = row_stride(b, k);
    d.dtype = dtype_of(c, "out");
    d.flags = narrow(integer(p[6]), "flags");
    if (m && n) {
        const int rc = api.matmul_fp8(&d, (const uint8_t*)a.data_ptr(), (const float*)sa.data_ptr(), (const uint8_t*)b.data_ptr(),
                                      (const float*)sb.data_ptr(), c.data_ptr(), stream_of(dev));
        if (rc != KDA_OK) return PyLong_FromLong(rc);
    }
    return wrap(c);
}

// out, lse and workspace of a latent call: given ones checked, others made.  False: the sizes are not supported.
bool latent_buffers(kda_latent_desc& d, size_t bytes, const at::Tensor* out, const at::Tensor* lse, const at::Tensor* work,
                    at::IntArrayRef shape, at::ScalarType type, c10::Device dev, at::Tensor& o, at::Tensor& l, at::Tensor& w) {
    if (!work && bytes == 0) return false;
    if (out) { dense(*out, "out", type, shape, dev); o = *out; }
    else o = fresh(shape, type, dev);
    const at::IntArrayRef heads = shape.slice(0, shape.size() - 1);
    if (lse) { dense(*lse, "lse", at::kFloat, heads, dev); l = *lse; }
    else l = fresh(heads, at::kFloat, dev);
    if (work) {
        if (!work->is_cuda() || work->device() != dev || !work->is_contiguous()) refuse("workspace must be a contiguous tensor on ", dev);
        w = *work;
    } else {
        w = fresh({(int64_t)bytes}, at::kByte, dev);
    }
    d.workspace = w.data_ptr();
    d.workspace_bytes = w.nbytes();
    return true;
}

// latent_prefill(q, k_nope, k_rope, v, cu_q, cu_k, scale, flags, out, lse, workspace)
PyObject* latent_prefill(PyObject* const* p) {
    const at::Tensor &q = tensor(p[0], "q"), &k = tensor(p[1], "k_nope"), &v = tensor(p[3], "v");
    const at::Tensor *r = maybe(p[2], "k_rope"), *cq = maybe(p[4], "cu_seqlens_q"), *ck = maybe(p[5], "cu_seqlens_k");
    const c10::Device dev = device_of(q, "q");
    const at::ScalarType type = q.scalar_type();
    kda_latent_desc d = {};
    d.dtype = dtype_of(q, "q");
    rows(q, "q", type, 3, dev);
    rows(k, "k_nope", type, 3, dev);
    rows(v, "v", type, 3, dev);
    const int64_t tq = q.size(0), h = q.size(1), tk = k.size(0);
    if (r) {
        rows(*r, "k_rope", type, 2, dev);
        if (r->size(0) != tk) refuse("k_rope must have k_nope's tokens: got ", r->sizes());
        d.d_rope = narrow(r->size(1), "d_rope");
        d.rope_token_stride = r->stride(0);
    }
    if (k.size(1) != h || v.size(0) != tk || v.size(1) != h || k.size(2) + d.d_rope != q.size(2))
        refuse("shapes do not fit: q ", q.sizes(), ", k_nope ", k.sizes(), ", v ", v.sizes(), ", d_rope ", d.d_rope);
    if ((cq == nullptr) != (ck == nullptr)) refuse("both cu_seqlens or neither");
    d.num_seqs = 1;
    if (cq) {
        if (cq->dim() != 1 || cq->size(0) < 1) refuse("cu_seqlens_q must be [N + 1]: got ", cq->sizes());
        dense(*cq, "cu_seqlens_q", at::kInt, cq->sizes(), dev);
        dense(*ck, "cu_seqlens_k", at::kInt, cq->sizes(), dev);
        d.num_seqs = narrow(cq->size(0) - 1, "the number of sequences");
        if (d.num_seqs == 0 && (tq || tk)) refuse("no sequences for ", tq, " queries and ", tk, " keys");
    }
    d.num_heads = narrow(h, "the number of heads");
    d.scale = (float)number(p[6], "scale");
    d.flags = narrow(integer(p[7]), "flags");
    d.d_k = narrow(k.size(2), "d_k");
    d.d_v = narrow(v.size(2), "d_v");
    d.total_q = tq; d.total_k = tk;
    d.q_token_stride = q.stride(0); d.q_head_stride = q.stride(1);
    d.k_token_stride = k.stride(0); d.k_head_stride = k.stride(1);
    d.v_token_stride = v.stride(0); d.v_head_stride = v.stride(1);
    at::Tensor o, l, w;
    if (!latent_buffers(d, api.prefill_bytes(&d), maybe(p[8], "out"), maybe(p[9], "lse"), maybe(p[10], "workspace"),
                        {tq, h, v.size(2)}, type, dev, o, l, w)) return PyLong_FromLong(KDA_ERR_UNSUPPORTED);
    const int rc = api.prefill(&d, q.data_ptr(), k.data_ptr(), data(r), v.data_ptr(), data<const int32_t>(cq),
                               data<const int32_t>(ck), o.data_ptr(), (float*)l.data_ptr(), stream_of(dev));
    if (rc != KDA_OK) return PyLong_FromLong(rc);
    return pack<2>({o, l});
}

// The quantised cache: pages of bytes, dense each; page_size, num_pages and the bytes between pages.
void pages_of(const at::Tensor& c, PyObject* page_size, int64_t rank, int64_t rope, c10::Device dev, int32_t& size, int32_t& pages,
              int64_t& stride) {
    if (page_size == Py_None) refuse("a quantised cache needs page_size");
    size = narrow(integer(page_size), "page_size");
    if (rank < 1 || rope < 0) refuse("rank and d_rope must be 1 and 0 at least: got ", rank, " and ", rope);
    const int64_t bytes = api.page_bytes(size, narrow(rank, "rank"), narrow(rope, "d_rope"));
    if (bytes == 0)
        refuse("a quantised cache has pages of at least one token, ranks that are multiples of 16 up to 512 and d_rope of 8 up to 128: got ",
               size, ", ", rank, ", ", rope);
    if (c.dim() != 2 || c.scalar_type() != at::kByte || c.device() != dev || c.size(1) != bytes || c.stride(1) != 1)
        refuse("cache must be a [pages, ", bytes, "] Byte tensor on ", dev, " with dense pages: got ", c.sizes(), ", ",
               c.scalar_type(), ", ", c.device(), ", strides ", c.strides());
    pages = narrow(c.size(0), "the number of pages");
    stride = c.size(0) > 1 ? c.stride(0) : bytes;
}

// latent_decode(q, cache, page_table, lengths, scale, rank (-1: all but 64), flags, out, lse, workspace, page_size)
PyObject* latent_decode(PyObject* const* p) {
    const at::Tensor &q = tensor(p[0], "q"), &c = tensor(p[1], "cache"), &table = tensor(p[2], "page_table"), &lens = tensor(p[3], "lengths");
    const c10::Device dev = device_of(q, "q");
    const at::ScalarType type = q.scalar_type();
    kda_latent_desc d = {};
    d.dtype = dtype_of(q, "q");
    const bool single = q.dim() == 3;
    rows(q, "q", type, single ? 3 : 4, dev);
    const int64_t n = q.size(0), lq = single ? 1 : q.size(1), h = q.size(-2), width = q.size(-1);
    d.q_head_stride = q.stride(-2);
    d.q_token_stride = lq == 1 ? q.stride(0) : q.stride(1);
    if (lq > 1 && n > 1 && q.stride(0) != lq * d.q_token_stride) refuse("q's sequences and queries must form one strided dimension");
    const bool codes = c.scalar_type() == at::kByte;
    if (!codes && (c.dim() != 3 || c.scalar_type() != type || c.device() != dev || c.size(2) != width ||
                   (width > 1 && c.stride(2) != 1) || (c.size(1) > 1 && c.stride(1) != width)))
        refuse("cache must be a [pages, page_size, ", width, "] ", type, " tensor on ", dev, " with dense pages: got ", c.sizes(),
               ", ", c.scalar_type(), ", ", c.device(), ", strides ", c.strides());
    int64_t rank = integer(p[5]);
    if (rank == -1) rank = width - 64;
    if (rank < 1 || rank > width) refuse("rank must be within 1 .. ", width, ": got ", rank);
    if (table.dim() != 2 || table.size(0) != n) refuse("page_table must be [", n, ", max_pages]: got ", table.sizes());
    dense(table, "page_table", at::kInt, table.sizes(), dev);
    dense(lens, "lengths", at::kInt, {n}, dev);
    d.num_seqs = narrow(n, "the number of sequences"); d.num_heads = narrow(h, "the number of heads");
    d.num_queries = narrow(lq, "the number of queries");
    d.scale = (float)number(p[4], "scale");
    d.flags = narrow(integer(p[6]), "flags");
    d.d_k = d.d_v = narrow(rank, "rank");
    d.d_rope = narrow(width - rank, "d_rope");
    d.max_pages = narrow(table.size(1), "max_pages");
    if (codes) {
        pages_of(c, p[10], rank, width - rank, dev, d.page_size, d.num_pages, d.page_stride);
        d.flags |= KDA_FLAG_CACHE_8;
    } else {
        d.page_size = narrow(c.size(1), "the page size"); d.num_pages = narrow(c.size(0), "the number of pages");
        d.page_stride = c.size(0) > 1 ? c.stride(0) : c.size(1) * width;
        if (d.flags & KDA_FLAG_CACHE_8) refuse("flags say a quantised cache, which is a Byte tensor: got ", c.scalar_type());
        if (p[10] != Py_None && integer(p[10]) != c.size(1)) refuse("page_size is not the cache's: ", c.sizes());
    }
    const int64_t four[4] = {n, lq, h, rank}, three[3] = {n, h, rank};
    at::Tensor o, l, w;
    if (!latent_buffers(d, api.decode_bytes(&d), maybe(p[7], "out"), maybe(p[8], "lse"), maybe(p[9], "workspace"),
                        single ? at::IntArrayRef(three, 3) : at::IntArrayRef(four, 4), type, dev, o, l, w))
        return PyLong_FromLong(KDA_ERR_UNSUPPORTED);
    const int rc = api.decode(&d, q.data_ptr(), c.data_ptr(), (const int32_t*)table.data_ptr(), (const int32_t*)lens.data_ptr(),
                              o.data_ptr(), (float*)l.data_ptr(), stream_of(dev));
    if (rc != KDA_OK) return PyLong_FromLong(rc);
    return pack<2>({o, l});
}

// Sequences, pages and workspace of a call on the quantised cache.
void cache_desc(kda_latent_cache_desc& d, const at::Tensor& c, const at::Tensor& table, const at::Tensor& lens, const at::Tensor* cu,
                PyObject* page_size, const at::Tensor* work, int64_t rank, int64_t rope, c10::Device dev) {
    d.rank = narrow(rank, "rank");
    d.d_rope = narrow(rope, "d_rope");
    pages_of(c, page_size, rank, rope, dev, d.page_size, d.num_pages, d.page_stride);
    if (table.dim() != 2) refuse("page_table must be [sequences, max_pages]: got ", table.sizes());
    const int64_t n = table.size(0);
    dense(table, "page_table", at::kInt, table.sizes(), dev);
    dense(lens, "lengths", at::kInt, {n}, dev);
    d.num_seqs = narrow(n, "the number of sequences");
    d.max_pages = narrow(table.size(1), "max_pages");
    if (cu) dense(*cu, "cu_seqlens", at::kInt, {n + 1}, dev);
    else if (d.total_tokens && (n == 0 || d.total_tokens % n)) refuse(d.total_tokens, " rows are not as many for each of ", n, " sequences: cu_seqlens");
    if (work) {
        if (!work->is_cuda() || work->device() != dev || !work->is_contiguous()) refuse("workspace must be a contiguous tensor on ", dev);
        d.workspace = work->data_ptr();
        d.workspace_bytes = work->nbytes();
    }
}

// latent_cache_write(latents, rope, cache, page_table, lengths, cu_seqlens, page_size, workspace)
PyObject* latent_cache_write(PyObject* const* p) {
    const at::Tensor &x = tensor(p[0], "latents"), &c = tensor(p[2], "cache"), &table = tensor(p[3], "page_table"), &lens = tensor(p[4], "lengths");
    const at::Tensor *r = maybe(p[1], "rope"), *cu = maybe(p[5], "cu_seqlens"), *work = maybe(p[7], "workspace");
    const c10::Device dev = device_of(x, "latents");
    kda_latent_cache_desc d = {};
    d.dtype = dtype_of(x, "latents");
    rows(x, "latents", x.scalar_type(), 2, dev);
    d.total_tokens = x.size(0);
    d.latent_stride = row_stride(x, x.size(1));
    if (r) {
        rows(*r, "rope", x.scalar_type(), 2, dev);
        if (r->size(0) != x.size(0)) refuse("rope must have the latents' rows: got ", r->sizes());
        d.rope_stride = row_stride(*r, r->size(1));
    }
    cache_desc(d, c, table, lens, cu, p[6], work, x.size(1), r ? r->size(1) : 0, dev);
    const int rc = api.cache_write(&d, x.data_ptr(), data<const void>(r), data<const int32_t>(cu), (const int32_t*)table.data_ptr(),
                                   (const int32_t*)lens.data_ptr(), (uint8_t*)c.data_ptr(), stream_of(dev));
    if (rc != KDA_OK) return PyLong_FromLong(rc);
    Py_RETURN_NONE;
}

// latent_cache_read(cache, page_table, lengths, cu_seqlens, total_tokens, page_size, rank, d_rope, out is bf16, latents, rope, workspace)
PyObject* latent_cache_read(PyObject* const* p) {
    const at::Tensor &c = tensor(p[0], "cache"), &table = tensor(p[1], "page_table"), &lens = tensor(p[2], "lengths");
    const at::Tensor *cu = maybe(p[3], "cu_seqlens"), *given = maybe(p[9], "latents"), *given_rope = maybe(p[10], "rope"),
                     *work = maybe(p[11], "workspace");
    const c10::Device dev = device_of(c, "cache");
    const int64_t t = integer(p[4]), rank = integer(p[6]), rope = integer(p[7]);
    if (t < 0) refuse("total_tokens must not be negative: got ", t);
    kda_latent_cache_desc d = {};
    d.total_tokens = t;
    const at::ScalarType type = given ? given->scalar_type() : given_rope ? given_rope->scalar_type() : truth(p[8], "dtype") ? at::kBFloat16 : at::kFloat;
    cache_desc(d, c, table, lens, cu, p[5], work, rank, rope, dev);
    at::Tensor x, r;
    if (given) {
        rows(*given, "latents", type, 2, dev);
        if (given->size(0) != t || given->size(1) != rank) refuse("latents must be [", t, ", ", rank, "]: got ", given->sizes());
        x = *given;
    } else {
        x = fresh({t, rank}, type, dev);
    }
    if (given_rope) {
        rows(*given_rope, "rope", type, 2, dev);
        if (rope == 0 || given_rope->size(0) != t || given_rope->size(1) != rope) refuse("rope must be [", t, ", ", rope, "]: got ", given_rope->sizes());
        r = *given_rope;
    } else if (rope) {
        r = fresh({t, rope}, type, dev);
    }
    d.dtype = dtype_of(x, "latents");
    d.latent_stride = row_stride(x, rank);
    d.rope_stride = rope ? row_stride(r, rope) : 0;
    const int rc = api.cache_read(&d, (const uint8_t*)c.data_ptr(), (const int32_t*)table.data_ptr(), (const int32_t*)lens.data_ptr(),
                                  data<const int32_t>(cu), x.data_ptr(), rope ? r.data_ptr() : nullptr, stream_of(dev));
    if (rc != KDA_OK) return PyLong_FromLong(rc);
    return pack<2>({x, r});
}

// One tensor of a rotary call, [tokens, heads, width] or [tokens, width], and its output.
at::Tensor rotary_one(const at::Tensor& x, const char* name, const at::Tensor* out, const char* out_name, PyObject* offset, int64_t tokens,
                      int64_t dim, at::ScalarType type, c10::Device dev, kda_rotary_part& d) {
    if (x.dim() != 2 && x.dim() != 3) refuse(name, " must be [tokens, heads, channels] or [tokens, channels]: got ", x.sizes());
    rows(x, name, type, x.dim(), dev);
    if (x.size(0) != tokens) refuse(name, " must have a row for each of ", tokens, " positions: got ", x.sizes());
    const int64_t width = x.size(-1), heads = x.dim() == 3 ? x.size(1) : 1;
    const int64_t at = offset == Py_None ? width - dim : integer(offset);
    if (dim > width || at < 0 || at > width - dim) refuse(dim, " channels from ", at, " on are not within ", name, "'s ", width);
    if (heads < 1) refuse(name, " must have heads: got ", x.sizes());
    if (out) {
        rows(*out, out_name, type, x.dim(), dev);
        if (out->sizes() != x.sizes()) refuse(out_name, " must have the shape ", x.sizes(), ": got ", out->sizes());
    }
    const at::Tensor y = out ? *out : fresh(x.sizes(), type, dev);
    d.heads = narrow(heads, "the number of heads");
    d.width = narrow(width, "the channels of a head");
    d.offset = narrow(at, "offset");
    // (sizes of one may carry any stride)
    d.token_stride = tokens > 1 ? x.stride(0) : heads * width;
    d.out_token_stride = tokens > 1 ? y.stride(0) : heads * width;
    d.head_stride = heads > 1 ? x.stride(1) : width;
    d.out_head_stride = heads > 1 ? y.stride(1) : width;
    return y;
}

// rotary(x, positions, frequencies, key, offset, key_offset, scale, flags, out, key_out)
PyObject* rotary(PyObject* const* p) {
    const at::Tensor &x = tensor(p[0], "x"), &pos = tensor(p[1], "positions"), &f = tensor(p[2], "frequencies");
    const at::Tensor *key = maybe(p[3], "key"), *out = maybe(p[8], "out"), *key_out = maybe(p[9], "key_out");
    const c10::Device dev = device_of(x, "x");
    kda_rotary_desc d = {};
    d.dtype = dtype_of(x, "x");
    if (pos.dim() != 1 || (pos.scalar_type() != at::kInt && pos.scalar_type() != at::kLong)) refuse("positions must be [tokens] int32 or int64: got ", pos.sizes(), ", ", pos.scalar_type());
    dense(pos, "positions", pos.scalar_type(), pos.sizes(), dev);
    if (f.dim() != 1 || f.size(0) < 1) refuse("frequencies must be [channels / 2]: got ", f.sizes());
    dense(f, "frequencies", at::kDouble, f.sizes(), dev);
    const int64_t tokens = pos.size(0), dim = 2 * f.size(0);
    d.tokens = tokens;
    d.dim = narrow(dim, "the channels turned");
    d.scale = (float)number(p[6], "scale");
    d.flags = narrow(integer(p[7]), "flags") | (pos.scalar_type() == at::kLong ? KDA_FLAG_POSITIONS_64 : 0);
    if (key_out && !key) refuse("key_out without a key");
    const at::Tensor y = rotary_one(x, "x", out, "out", p[4], tokens, dim, x.scalar_type(), dev, d.x);
    at::Tensor ky;
    if (key) ky = rotary_one(*key, "key", key_out, "key_out", p[5], tokens, dim, x.scalar_type(), dev, d.key);
    if (tokens) {
        const int rc = api.rotary(&d, x.data_ptr(), data<const void>(key), pos.data_ptr(), (const double*)f.data_ptr(), y.data_ptr(),
                                  key ? ky.data_ptr() : nullptr, stream_of(dev));
        if (rc != KDA_OK) return PyLong_FromLong(rc);
    }
    return pack<2>({y, ky});
}

// bind(addresses of the C entry points, in Api's order)
PyObject* bind(PyObject* const* p) {
    void** f = (void**)&api;
    for (size_t i = 0; i < sizeof(Api) / sizeof(void*); ++i) f[i] = (void*)(uintptr_t)integer(p[i]);
    Py_RETURN_NONE;
}

// No C++ exception leaves the module.
template <PyObject* (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
    try {
        if (n != N) refuse("expected ", N, " arguments, got ", n);
        return F(args);
    } catch (const std::invalid_argument& e) {
        PyErr_SetString(PyExc_ValueError, e.what());
    } catch (const c10::OutOfMemoryError& e) {
        PyObject* torch = PyImport_ImportModule("torch");
        PyObject* type = torch ? PyObject_GetAttrString(torch, "OutOfMemoryError") : nullptr;
        PyErr_Clear();
        PyErr_SetString(type ? type : PyExc_MemoryError, e.what_without_backtrace());
        Py_XDECREF(type);
        Py_XDECREF(torch);
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

#define KDA_METHOD(f, n) {#f, (PyCFunction)(void*)(&entry<f, n>), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {KDA_METHOD(bind, 10), KDA_METHOD(rms_norm, 7), KDA_METHOD(matmul_fp8, 7), KDA_METHOD(latent_prefill, 11),
                         KDA_METHOD(latent_decode, 11), KDA_METHOD(latent_cache_write, 8), KDA_METHOD(latent_cache_read, 12),
                         KDA_METHOD(rotary, 10), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_kda_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__kda_torch(void) { return PyModule_Create(&module); }
