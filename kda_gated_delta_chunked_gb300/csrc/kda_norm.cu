// kda_norm.cu -- root-mean-square norm of rows with the residual's addition in
// front and an e4m3 output with one scale per 128 elements behind.
//
//     h = x + r,   y = h rsqrt(mean(h^2) + eps) w,
//     s_b = max(max_{block b} |y|, 1e-12) / 448,   q = e4m3(y / s_b)
//
// Every input is read once and every output written once: bound by HBM bytes.
// The row stays in registers between the sum of squares and the outputs (fp32,
// 8 elements a thread and step).
#include <cuda_fp8.h>

#include "kda_common.cuh"
#include "kda_paths.h"

namespace kda {

struct NormArgs {
    int64_t rows, x_stride, r_stride;
    int dim;
    float eps;
    const void *x, *w, *r;
    void *h, *y;
    uint8_t* q;
    float* s;
};

constexpr int kNormVec = 8;         // elements of a thread's step
constexpr int kNormBlock = 128;     // elements that share a scale

struct Vec8 { float v[kNormVec]; };

// Which elements a thread's step holds.  Aligned rows: 8 consecutive ones, so a
// block of 128 is 16 neighbouring lanes.  Others: every 32nd of the warp's 256
// from its lane on, so that element-wide accesses stay along the row (a row of
// 2051 fp32 elements: 7 us for 777 rows, against 14 with 8 consecutive ones);
// the warp's step is then two whole blocks.
template <bool kAligned>
__device__ __forceinline__ int norm_element(int step, int tpr, int t) {
    return kAligned ? (step * tpr + t) * kNormVec : (step * tpr + (t & ~31)) * kNormVec + (t & 31);
}

// A step's elements as they lie in memory.
template <typename T> struct Raw8;
template <> struct Raw8<__nv_bfloat16> {
    uint32_t w[4];
    __device__ __forceinline__ void vec(const __nv_bfloat16* p) {
        const uint4 u = *(const uint4*)p;
        w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
    }
    __device__ __forceinline__ void set(int i, const __nv_bfloat16* p) {
        const uint32_t b = p ? *(const uint16_t*)p : 0u;
        w[i / 2] = i % 2 ? w[i / 2] | (b << 16) : b;
    }
    __device__ __forceinline__ float get(int i) const {
        return __uint_as_float(i % 2 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
    }
};
template <> struct Raw8<float> {
    float f[8];
    __device__ __forceinline__ void vec(const float* p) {
        const float4 a = ((const float4*)p)[0], b = ((const float4*)p)[1];
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w; f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    }
    __device__ __forceinline__ void set(int i, const float* p) { f[i] = p ? *p : 0.f; }
    __device__ __forceinline__ float get(int i) const { return f[i]; }
};

template <typename T, bool kAligned>
__device__ __forceinline__ Raw8<T> load8(const T* row, int e, int dim) {
    Raw8<T> o;
    if (kAligned && e + kNormVec <= dim) {
        o.vec(row + e);
    } else {
        constexpr int d = kAligned ? 1 : 32;
#pragma unroll
        for (int i = 0; i < kNormVec; ++i) o.set(i, e + i * d < dim ? row + e + i * d : nullptr);
    }
    return o;
}

template <typename T, bool kAligned>
__device__ __forceinline__ void store8(T* row, int e, int dim, const Vec8& x) {
    if (kAligned && e + kNormVec <= dim) {
        if constexpr (sizeof(T) == 2) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const __nv_bfloat162 b = __floats2bfloat162_rn(x.v[2 * i], x.v[2 * i + 1]);
                w[i] = *(const uint32_t*)&b;
            }
            *(uint4*)(row + e) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
            ((float4*)(row + e))[0] = make_float4(x.v[0], x.v[1], x.v[2], x.v[3]);
            ((float4*)(row + e))[1] = make_float4(x.v[4], x.v[5], x.v[6], x.v[7]);
        }
    } else {
        constexpr int d = kAligned ? 1 : 32;
#pragma unroll
        for (int i = 0; i < kNormVec; ++i)
            if (e + i * d < dim) row[e + i * d] = from_f32<T>(x.v[i]);
    }
}

// h of one step: x + r, written out where wanted.
template <typename T, bool kAligned>
__device__ __forceinline__ Vec8 norm_sum8(const NormArgs& a, int64_t row, int e, bool write) {
    const Raw8<T> x = load8<T, kAligned>((const T*)a.x + row * a.x_stride, e, a.dim);
    Vec8 h;
    if (a.r) {
        const Raw8<T> r = load8<T, kAligned>((const T*)a.r + row * a.r_stride, e, a.dim);
#pragma unroll
        for (int i = 0; i < kNormVec; ++i) h.v[i] = x.get(i) + r.get(i);
    } else {
#pragma unroll
        for (int i = 0; i < kNormVec; ++i) h.v[i] = x.get(i);
    }
    if (write && a.h) store8<T, kAligned>((T*)a.h + row * a.dim, e, a.dim, h);
    return h;
}

// The outputs of one step.  All lanes of the warp call it (the block maximum
// crosses lanes); elements behind the row are left out.
template <typename T, bool kAligned>
__device__ __forceinline__ void norm_out8(const NormArgs& a, int64_t row, int e, const Vec8& h, const Raw8<T>& w,
                                          float rstd) {
    Vec8 y;
    if (a.w) {
#pragma unroll
        for (int i = 0; i < kNormVec; ++i) y.v[i] = h.v[i] * rstd * w.get(i);
    } else {
#pragma unroll
        for (int i = 0; i < kNormVec; ++i) y.v[i] = h.v[i] * rstd;
    }
    if (a.y) store8<T, kAligned>((T*)a.y + row * a.dim, e, a.dim, y);
    if (!a.q) return;
    // the step's blocks: one of 16 lanes, or two of the whole warp; behind the row h = 0
    constexpr int kBlocks = kAligned ? 1 : 2, kEach = kNormVec / kBlocks;
    float inv[kBlocks];
    const int blocks = (a.dim + kNormBlock - 1) / kNormBlock;
#pragma unroll
    for (int b = 0; b < kBlocks; ++b) {
        float amax = 0.f;
#pragma unroll
        for (int i = 0; i < kEach; ++i) amax = fmaxf(amax, fabsf(y.v[b * kEach + i]));
#pragma unroll
        for (int o = 1; o < (kAligned ? 16 : 32); o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        amax = fmaxf(amax, 1e-12f);
        const int first = e + b * kNormBlock;          // an element of the block
        const bool writes = kAligned ? e % kNormBlock == 0 : (threadIdx.x & 31) == 0;
        if (writes && first < a.dim) a.s[row * blocks + first / kNormBlock] = amax / 448.f;
        inv[b] = 448.f / amax;
    }
    uint32_t bytes[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float c = inv[kAligned ? 0 : i];
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(y.v[4 * i] * c, y.v[4 * i + 1] * c),
                                                     __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(y.v[4 * i + 2] * c, y.v[4 * i + 3] * c),
                                                     __NV_SATFINITE, __NV_E4M3);
        bytes[i] = lo | (hi << 16);
    }
    uint8_t* q = a.q + row * a.dim + e;
    if (kAligned && e + kNormVec <= a.dim) {
        *(uint2*)q = make_uint2(bytes[0], bytes[1]);
    } else {
        constexpr int d = kAligned ? 1 : 32;
#pragma unroll
        for (int i = 0; i < kNormVec; ++i)
            if (e + i * d < a.dim) q[i * d] = (uint8_t)(bytes[i >> 2] >> (8 * (i & 3)));
    }
}

constexpr int norm_threads(int tpr) { return tpr < 128 ? 128 : tpr; }

// TPR threads share a row; each holds STEPS vectors of it (STEPS = 0: the row
// is too long for registers and is read a second time, out of L2).  Few vectors
// a thread and 1536 threads an SM keep the most bytes on their way: 65536 x 4096
// bf16 to all four outputs 361 us (99% of the measured copy rate), 380 without
// the bound on registers, 406 with the weights read behind the sum.
template <typename T, bool kAligned, int TPR, int STEPS>
__global__ void __launch_bounds__(norm_threads(TPR), sizeof(T) == 2 && (STEPS == 1 || STEPS == 2) ? 1536 / norm_threads(TPR) : 1)
kda_rms_norm_kernel(NormArgs a) {
    constexpr int kThreads = norm_threads(TPR);
    constexpr int kRows = kThreads / TPR;
    constexpr int kWarpsPerRow = TPR / 32;
    const int t = threadIdx.x % TPR;
    const int64_t row_of = (int64_t)blockIdx.x * kRows + threadIdx.x / TPR;
    const bool real = row_of < a.rows;                   // whole warps, since TPR >= 32
    const int64_t row = real ? row_of : a.rows - 1;

    Vec8 h[STEPS > 0 ? STEPS : 1];
    Raw8<T> w[STEPS > 0 ? STEPS : 1];                    // on its way while the row is summed
    float ss = 0.f;
    if constexpr (STEPS > 0) {
#pragma unroll
        for (int k = 0; k < STEPS; ++k)
            h[k] = norm_sum8<T, kAligned>(a, row, norm_element<kAligned>(k, TPR, t), real);
        if (a.w) {
#pragma unroll
            for (int k = 0; k < STEPS; ++k) w[k] = load8<T, kAligned>((const T*)a.w, norm_element<kAligned>(k, TPR, t), a.dim);
        }
#pragma unroll
        for (int k = 0; k < STEPS; ++k)
#pragma unroll
            for (int i = 0; i < kNormVec; ++i) ss += h[k].v[i] * h[k].v[i];
    } else {
        for (int k = 0; k * TPR * kNormVec < a.dim; ++k) {
            const Vec8 x = norm_sum8<T, kAligned>(a, row, norm_element<kAligned>(k, TPR, t), false);
#pragma unroll
            for (int i = 0; i < kNormVec; ++i) ss += x.v[i] * x.v[i];
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if constexpr (kWarpsPerRow > 1) {
        __shared__ float part[kThreads / 32];
        if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = ss;
        __syncthreads();
        const int w0 = threadIdx.x / TPR * kWarpsPerRow;
        ss = 0.f;
#pragma unroll
        for (int w = 0; w < kWarpsPerRow; ++w) ss += part[w0 + w];
    }
    if (!real) return;
    const float rstd = 1.f / sqrtf(ss / (float)a.dim + a.eps);
    if constexpr (STEPS > 0) {
#pragma unroll
        for (int k = 0; k < STEPS; ++k) norm_out8<T, kAligned>(a, row, norm_element<kAligned>(k, TPR, t), h[k], w[k], rstd);
    } else {
        // residual_out may be x or residual: each element is read (again) before it is written, by its thread
        for (int k = 0; k * TPR * kNormVec < a.dim; ++k) {
            const int e = norm_element<kAligned>(k, TPR, t);
            if (a.w) w[0] = load8<T, kAligned>((const T*)a.w, e, a.dim);
            norm_out8<T, kAligned>(a, row, e, norm_sum8<T, kAligned>(a, row, e, true), w[0], rstd);
        }
    }
}

template <typename T, bool kAligned>
static cudaError_t launch_norm(const NormArgs& a, cudaStream_t stream) {
    const int steps = (a.dim + kNormVec - 1) / kNormVec;    // vectors of a row
#define KDA_NORM(tpr, per)                                                                            \
    do {                                                                                              \
        constexpr int th = norm_threads(tpr);                                                     \
        const int64_t blocks = (a.rows + th / tpr - 1) / (th / tpr);                                  \
        kda_rms_norm_kernel<T, kAligned, tpr, per><<<(unsigned)blocks, th, 0, stream>>>(a);           \
        return cudaGetLastError();                                                                    \
    } while (0)
    if (steps <= 32) KDA_NORM(32, 1);
    if (steps <= 64) KDA_NORM(64, 1);
    if (steps <= 128) KDA_NORM(128, 1);
    if (steps <= 256) KDA_NORM(256, 1);
    if (steps <= 512) KDA_NORM(256, 2);
    if (steps <= 1024) KDA_NORM(512, 2);
    if (steps <= 2048) KDA_NORM(512, 4);
    KDA_NORM(512, 0);
#undef KDA_NORM
}

cudaError_t rms_norm_launch(const kda_norm_desc& d, const void* x, const void* weight, const void* residual,
                            void* residual_out, void* normed, uint8_t* quantized, float* scales,
                            cudaStream_t stream) {
    NormArgs a;
    a.rows = d.rows; a.x_stride = d.x_stride; a.r_stride = d.residual_stride; a.dim = d.dim; a.eps = d.eps;
    a.x = x; a.w = weight; a.r = residual; a.h = residual_out; a.y = normed; a.q = quantized; a.s = scales;
    const int64_t esz = d.dtype == KDA_BF16 ? 2 : 4;
    // 16-byte vectors of every row: addresses and row lengths in bytes (the e4m3 rows: 8 bytes)
    uintptr_t bits = (uintptr_t)x | (uintptr_t)weight | (uintptr_t)residual | (uintptr_t)residual_out |
                     (uintptr_t)normed | ((uintptr_t)quantized << 1) | (uintptr_t)(d.x_stride * esz);
    if (residual) bits |= (uintptr_t)(d.residual_stride * esz);
    if (residual_out || normed) bits |= (uintptr_t)(d.dim * esz);
    if (quantized) bits |= (uintptr_t)d.dim << 1;
    const bool aligned = (bits & 15) == 0;
    if (d.dtype == KDA_BF16)
        return aligned ? launch_norm<__nv_bfloat16, true>(a, stream) : launch_norm<__nv_bfloat16, false>(a, stream);
    return aligned ? launch_norm<float, true>(a, stream) : launch_norm<float, false>(a, stream);
}

}  // namespace kda
