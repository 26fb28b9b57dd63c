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
#include "kda_per_device.h"

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
__device__ __forceinline__ Vec8 norm_add8(const NormArgs& a, int64_t row, int e, bool write, const Raw8<T>& x, const Raw8<T>& r) {
    Vec8 h;
#pragma unroll
    for (int i = 0; i < kNormVec; ++i) h.v[i] = a.r ? x.get(i) + r.get(i) : x.get(i);
    if (write && a.h) store8<T, kAligned>((T*)a.h + row * a.dim, e, a.dim, h);
    return h;
}
template <typename T, bool kAligned>
__device__ __forceinline__ void norm_load8(const NormArgs& a, int64_t row, int e, Raw8<T>& x, Raw8<T>& r) {
    x = load8<T, kAligned>((const T*)a.x + row * a.x_stride, e, a.dim);
    if (a.r) r = load8<T, kAligned>((const T*)a.r + row * a.r_stride, e, a.dim);
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

// TPR threads share a row (0: the block's, as many warps as the row needs; up to 64
// have other rows beside them); each holds STEPS vectors of it (STEPS = 0: the row
// is too long for registers and is read a second time, out of L2).  Few vectors a
// thread and 1536 threads an SM keep the most bytes on their way: 65536 x 4096 bf16
// to all four outputs 346 us (the copy rate), 380 without the bound on registers,
// 406 with the weights read behind the sum; 16384 x 5120 115 us, 169 with threads
// in powers of two.  Rows of four vectors a thread leave an SM one block, which
// goes on to other rows (LOOP) with their loads on the way while it works on the
// one before: 8192 x 12288 to one output 84 us, 127 a block for each row; with two
// vectors the registers for that cost more than it gives (65536 x 4096: 386).
constexpr int norm_blocks(int esz, int steps) {   // of 512 threads an SM, at least
    return steps == 0 || steps > 2 ? 1 : esz == 2 ? 3 : 2;
}
template <typename T, bool kAligned, int TPR, int STEPS, bool LOOP>
__global__ void __launch_bounds__(512, norm_blocks(sizeof(T), STEPS))
kda_rms_norm_kernel(NormArgs a) {
    constexpr int ROWS = TPR && TPR < 128 ? 128 / TPR : 1;
    constexpr int kWarps = TPR ? TPR / 32 : STEPS == 1 ? 8 : 16;     // of a row at most
    const int tpr = TPR ? TPR : blockDim.x, t = ROWS > 1 ? threadIdx.x % tpr : threadIdx.x, warps = tpr / 32;
    const int64_t step = (int64_t)gridDim.x * ROWS;
    int64_t row_of = (int64_t)blockIdx.x * ROWS + (ROWS > 1 ? threadIdx.x / tpr : 0);
    __shared__ float part[2][16];
    constexpr int kHeld = STEPS > 0 ? STEPS : 1;
    Raw8<T> w[kHeld], x[kHeld], r[kHeld];
    if constexpr (STEPS > 0) {
#pragma unroll
        for (int k = 0; k < STEPS; ++k)
            norm_load8<T, kAligned>(a, row_of < a.rows ? row_of : a.rows - 1, norm_element<kAligned>(k, tpr, t), x[k], r[k]);
        if (a.w) {                                       // on their way while the row is summed
#pragma unroll
            for (int k = 0; k < STEPS; ++k) w[k] = load8<T, kAligned>((const T*)a.w, norm_element<kAligned>(k, tpr, t), a.dim);
        }
    }
    // whole warps have a row or none; all of a block's go round together
    for (int64_t first = (int64_t)blockIdx.x * ROWS, turn = 0; first < a.rows; first += step, row_of += step, turn ^= 1) {
        const bool real = row_of < a.rows;
        const int64_t row = real ? row_of : a.rows - 1;
        Vec8 h[kHeld];
        float ss = 0.f;
        if constexpr (STEPS > 0) {
#pragma unroll
            for (int k = 0; k < STEPS; ++k)
                h[k] = norm_add8<T, kAligned>(a, row, norm_element<kAligned>(k, tpr, t), real, x[k], r[k]);
            if (LOOP && row_of + step < a.rows) {
#pragma unroll
                for (int k = 0; k < STEPS; ++k)
                    norm_load8<T, kAligned>(a, row_of + step, norm_element<kAligned>(k, tpr, t), x[k], r[k]);
            }
#pragma unroll
            for (int k = 0; k < STEPS; ++k)
#pragma unroll
                for (int i = 0; i < kNormVec; ++i) ss += h[k].v[i] * h[k].v[i];
        } else {
            for (int k = 0; k * tpr * kNormVec < a.dim; ++k) {
                const int e = norm_element<kAligned>(k, tpr, t);
                norm_load8<T, kAligned>(a, row, e, x[0], r[0]);
                const Vec8 y = norm_add8<T, kAligned>(a, row, e, false, x[0], r[0]);
#pragma unroll
                for (int i = 0; i < kNormVec; ++i) ss += y.v[i] * y.v[i];
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        if constexpr (kWarps > 1) {                      // (two rounds' sums: nobody is further ahead)
            if ((threadIdx.x & 31) == 0) part[turn][threadIdx.x >> 5] = ss;
            __syncthreads();
            const int w0 = ROWS > 1 ? threadIdx.x / tpr * kWarps : 0;
            ss = 0.f;
#pragma unroll
            for (int i = 0; i < kWarps; ++i) {
                const float p = part[turn][w0 + i];
                ss += TPR || i < warps ? p : 0.f;
            }
        }
        if (real) {
            const float rstd = 1.f / sqrtf(ss / (float)a.dim + a.eps);
            if constexpr (STEPS > 0) {
#pragma unroll
                for (int k = 0; k < STEPS; ++k)
                    norm_out8<T, kAligned>(a, row, norm_element<kAligned>(k, tpr, t), h[k], w[k], rstd);
            } else {
                // residual_out may be x or residual: each element is read (again) before it is written, by its thread
                for (int k = 0; k * tpr * kNormVec < a.dim; ++k) {
                    const int e = norm_element<kAligned>(k, tpr, t);
                    if (a.w) w[0] = load8<T, kAligned>((const T*)a.w, e, a.dim);
                    norm_load8<T, kAligned>(a, row, e, x[0], r[0]);
                    norm_out8<T, kAligned>(a, row, e, norm_add8<T, kAligned>(a, row, e, true, x[0], r[0]), w[0], rstd);
                }
            }
        }
        if (!LOOP) break;
    }
}

template <typename T, bool kAligned, int TPR, int STEPS, bool LOOP>
static cudaError_t launch_rows(const NormArgs& a, int threads, cudaStream_t stream) {
    auto kern = kda_rms_norm_kernel<T, kAligned, TPR, STEPS, LOOP>;
    constexpr int rows = TPR && TPR < 128 ? 128 / TPR : 1;
    int64_t blocks = (a.rows + rows - 1) / rows;
    if (LOOP) {
        static PerDevice resident[17];                   // blocks of so many warps on an SM
        int device = 0, n = 0;
        cudaError_t e = cudaGetDevice(&device);
        if (e == cudaSuccess) e = resident[threads / 32].get(device, n, [&](int& found) {
            return cudaOccupancyMaxActiveBlocksPerMultiprocessor(&found, kern, threads, 0);
        });
        if (e != cudaSuccess) return e;
        blocks = min64(blocks, (int64_t)n * 152);
    }
    kern<<<(unsigned)blocks, threads, 0, stream>>>(a);
    return cudaGetLastError();
}

template <typename T, bool kAligned>
static cudaError_t launch_norm(const NormArgs& a, cudaStream_t stream) {
    const int steps = (a.dim + kNormVec - 1) / kNormVec;    // vectors of a row
    if (steps <= 32) return launch_rows<T, kAligned, 32, 1, false>(a, 128, stream);
    if (steps <= 64) return launch_rows<T, kAligned, 64, 1, false>(a, 128, stream);
    const int warps1 = (steps + 31) / 32, warps2 = (steps + 63) / 64, warps4 = (steps + 127) / 128;
    if (warps1 == 4) return launch_rows<T, kAligned, 128, 1, false>(a, 128, stream);
    if (warps1 == 8) return launch_rows<T, kAligned, 256, 1, false>(a, 256, stream);
    if (warps1 < 8) return launch_rows<T, kAligned, 0, 1, false>(a, 32 * warps1, stream);
    if (warps2 <= 16) return launch_rows<T, kAligned, 0, 2, false>(a, 32 * warps2, stream);
    if (warps4 <= 16) return launch_rows<T, kAligned, 0, 4, true>(a, 32 * warps4, stream);
    return launch_rows<T, kAligned, 0, 0, false>(a, 512, stream);
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
