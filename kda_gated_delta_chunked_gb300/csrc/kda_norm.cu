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

template <typename T, bool kAligned>
__device__ __forceinline__ Vec8 load8(const T* row, int e, int dim) {
    Vec8 o;
    if (kAligned && e + kNormVec <= dim) {
        if constexpr (sizeof(T) == 2) {
            const uint4 u = *(const uint4*)(row + e);
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                o.v[2 * i] = __uint_as_float(w[i] << 16);
                o.v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            }
        } else {
            const float4 a = ((const float4*)(row + e))[0], b = ((const float4*)(row + e))[1];
            o.v[0] = a.x; o.v[1] = a.y; o.v[2] = a.z; o.v[3] = a.w;
            o.v[4] = b.x; o.v[5] = b.y; o.v[6] = b.z; o.v[7] = b.w;
        }
    } else {
        constexpr int d = kAligned ? 1 : 32;
#pragma unroll
        for (int i = 0; i < kNormVec; ++i) o.v[i] = e + i * d < dim ? to_f32(row[e + i * d]) : 0.f;
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
    Vec8 h = load8<T, kAligned>((const T*)a.x + row * a.x_stride, e, a.dim);
    if (a.r) {
        const Vec8 r = load8<T, kAligned>((const T*)a.r + row * a.r_stride, e, a.dim);
#pragma unroll
        for (int i = 0; i < kNormVec; ++i) h.v[i] += r.v[i];
    }
    if (write && a.h) store8<T, kAligned>((T*)a.h + row * a.dim, e, a.dim, h);
    return h;
}

// The outputs of one step.  All lanes of the warp call it (the block maximum
// crosses lanes); elements behind the row are left out.
template <typename T, bool kAligned>
__device__ __forceinline__ void norm_out8(const NormArgs& a, int64_t row, int e, const Vec8& h, float rstd) {
    Vec8 y;
    if (a.w) {
        const Vec8 w = load8<T, kAligned>((const T*)a.w, e, a.dim);
#pragma unroll
        for (int i = 0; i < kNormVec; ++i) y.v[i] = h.v[i] * rstd * w.v[i];
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
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float c = inv[kAligned ? 0 : i];
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(y.v[4 * i] * c, y.v[4 * i + 1] * c),
                                                     __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(y.v[4 * i + 2] * c, y.v[4 * i + 3] * c),
                                                     __NV_SATFINITE, __NV_E4M3);
        w[i] = lo | (hi << 16);
    }
    uint8_t* q = a.q + row * a.dim + e;
    if (kAligned && e + kNormVec <= a.dim) {
        *(uint2*)q = make_uint2(w[0], w[1]);
    } else {
        constexpr int d = kAligned ? 1 : 32;
#pragma unroll
        for (int i = 0; i < kNormVec; ++i)
            if (e + i * d < a.dim) q[i * d] = (uint8_t)(w[i >> 2] >> (8 * (i & 3)));
    }
}

// TPR threads share a row; each holds STEPS vectors of it (STEPS = 0: the row
// is too long for registers and is read a second time, out of L2).
template <typename T, bool kAligned, int TPR, int STEPS>
__global__ void __launch_bounds__(TPR < 128 ? 128 : TPR)
kda_rms_norm_kernel(NormArgs a) {
    constexpr int kThreads = TPR < 128 ? 128 : TPR;
    constexpr int kRows = kThreads / TPR;
    constexpr int kWarpsPerRow = TPR / 32;
    const int t = threadIdx.x % TPR;
    const int64_t row_of = (int64_t)blockIdx.x * kRows + threadIdx.x / TPR;
    const bool real = row_of < a.rows;                   // whole warps, since TPR >= 32
    const int64_t row = real ? row_of : a.rows - 1;

    Vec8 h[STEPS > 0 ? STEPS : 1];
    float ss = 0.f;
    if constexpr (STEPS > 0) {
#pragma unroll
        for (int k = 0; k < STEPS; ++k) {
            h[k] = norm_sum8<T, kAligned>(a, row, norm_element<kAligned>(k, TPR, t), real);
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
        for (int k = 0; k < STEPS; ++k) norm_out8<T, kAligned>(a, row, norm_element<kAligned>(k, TPR, t), h[k], rstd);
    } else {
        // residual_out may be x or residual: each element is read (again) before it is written, by its thread
        for (int k = 0; k * TPR * kNormVec < a.dim; ++k) {
            const int e = norm_element<kAligned>(k, TPR, t);
            norm_out8<T, kAligned>(a, row, e, norm_sum8<T, kAligned>(a, row, e, true), rstd);
        }
    }
}

template <typename T, bool kAligned>
static cudaError_t launch_norm(const NormArgs& a, cudaStream_t stream) {
    const int steps = (a.dim + kNormVec - 1) / kNormVec;    // vectors of a row
#define KDA_NORM(tpr, per)                                                                            \
    do {                                                                                              \
        constexpr int th = tpr < 128 ? 128 : tpr;                                                     \
        const int64_t blocks = (a.rows + th / tpr - 1) / (th / tpr);                                  \
        kda_rms_norm_kernel<T, kAligned, tpr, per><<<(unsigned)blocks, th, 0, stream>>>(a);           \
        return cudaGetLastError();                                                                    \
    } while (0)
    if (steps <= 32) KDA_NORM(32, 1);
    if (steps <= 64) KDA_NORM(32, 2);
    if (steps <= 128) KDA_NORM(64, 2);
    if (steps <= 256) KDA_NORM(128, 2);
    if (steps <= 512) KDA_NORM(256, 2);
    if (steps <= 1024) KDA_NORM(256, 4);
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
