// kda_latent_cache.cu -- latents quantised into the pages of a cache, and read
// back as rows (layout and rounding: kda.h).
//
//     e = min { e : max |c| <= 448 2^e },   code = e4m3(c / 2^e)
//
// A warp owns a token, a lane every 32nd vector of 16 bytes of its channels: the
// maximum is one reduction, and the warp's accesses lie side by side (with 16
// channels in a row a lane, fp32 rows were read in 42 us instead of 33, for 65536
// tokens).  Division by a power of two is exact, so the code is the latent rounded
// once.  A warp takes one or two neighbouring tokens, whose rows it loads before it
// looks for their places (write), or whose places it finds before it loads any
// (read).
//
// Bound by HBM bytes: 1152 and 641 of them a token in bf16 at rank 512.  65536
// tokens, us in a graph of ten (floor 17 in bf16, 28 in fp32): written 20 and 30,
// read 18 and 32; one token each of 48 sequences 2.0.
//
// Errors in lengths and pages are found by a block of its own, if there is a
// status word: it alone writes it.  The others leave out what is wrong.
#include <cuda_fp8.h>
#include <math.h>
#include <string.h>

#include "kda_common.cuh"
#include "kda_latent_cache.cuh"
#include "kda_launch.cuh"
#include "kda_paths.h"

namespace kda {

constexpr int kLcWarps = 8;

// A lane's channels of a row: kVecs vectors of kVec, 32 kVec channels apart; and its pairs of rotary channels.
template <typename T> struct LcRow {
    static constexpr int kVec = 16 / (int)sizeof(T), kVecs = 512 / (32 * kVec);
    uint4 v[kVecs];
    T rope[2][2];
};
template <typename T>
__device__ __forceinline__ int lc_channel(int i, int lane) { return (i * 32 + lane) * LcRow<T>::kVec; }

template <typename T, bool kWide>
__device__ __forceinline__ void lc_load(const LatentCacheArgs& a, int64_t t, int lane, LcRow<T>& x) {
    const T* p = (const T*)a.latents + t * a.latent_stride;
#pragma unroll
    for (int i = 0; i < LcRow<T>::kVecs; ++i) {
        const int c = lc_channel<T>(i, lane);
        x.v[i] = make_uint4(0, 0, 0, 0);
        if (c >= a.rank) continue;
        if constexpr (kWide) {
            x.v[i] = *(const uint4*)(p + c);
        } else {
            T e[LcRow<T>::kVec];
#pragma unroll
            for (int k = 0; k < LcRow<T>::kVec; ++k) e[k] = p[c + k];
            memcpy(&x.v[i], e, 16);
        }
    }
    const T* r = (const T*)a.rope + t * a.rope_stride;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int c = 64 * i + 2 * lane;
        if (c < a.d_rope) { x.rope[i][0] = r[c]; x.rope[i][1] = r[c + 1]; }
    }
}

// Rows [from, to) of a sequence and the place of its first one.
struct LcSequence { int n; int64_t from, to, place; };

// The sequence of row t, by a whole warp; from == to: there is none, or its bounds or its length are none.
__device__ __forceinline__ LcSequence lc_sequence(const LatentCacheArgs& a, int64_t t) {
    const int lane = threadIdx.x & 31;
    LcSequence s = {0, 0, 0, 0};
    if (!a.cu) {
        s.n = (int)((uint32_t)t / (uint32_t)a.rows_each);              // (rows are below 2^31)
        s.from = s.n * a.rows_each;
        s.to = s.from + a.rows_each;
    } else {
        int lo = 0, hi = a.N;                                      // the last n with cu[n] <= t, 32 of them a look
        while (hi - lo > 1) {
            const int step = (hi - lo + 31) / 32, i = lo + lane * step;
            const uint32_t b = __ballot_sync(0xffffffffu, i < hi && a.cu[i] <= t);
            const int k = b ? 31 - __clz(b) : 0;
            lo += k * step;
            hi = min(lo + step, hi);
        }
        s.n = lo;
        const int from = a.cu[lo], to = a.cu[lo + 1];
        s.from = from;
        s.to = t < from || t >= to || to > (int)a.T || (lo == 0 ? from != 0 : from < 0) ? from : to;
    }
    const int64_t len = a.lens[s.n];
    if (len < 0 || len > (int64_t)a.max_pages * a.page_size) s.to = s.from;
    s.place = len - (s.to - s.from);
    return s;
}

// Page and row of it of tokens t .. t + kTokens - 1 (lane i: token t + i), page -1 where there is none.
template <int kTokens>
__device__ __forceinline__ void lc_places(const LatentCacheArgs& a, int64_t t, int& page, int& row) {
    const int lane = threadIdx.x & 31;
    page = -1;
    row = 0;
    int64_t place = -1;
    int n = 0;
#pragma unroll 1
    for (int i = 0; i < kTokens && t + i < a.T;) {
        const LcSequence s = lc_sequence(a, t + i);
        const int64_t end = s.to > s.from ? s.to : t + i + 1;
        if (lane >= i && lane < kTokens && t + lane < s.to && s.to > s.from) {
            place = s.place + (t + lane - s.from);
            n = s.n;
        }
        i = (int)min64(kTokens, end - t);
    }
    if (lane < kTokens && t + lane < a.T && place >= 0) {
        const uint32_t at = (uint32_t)place, size = (uint32_t)a.page_size;   // (places are below 2^31)
        const int p = a.table[(int64_t)n * a.max_pages + at / size];
        if (p >= 0 && p < a.num_pages) {
            page = p;
            row = (int)(at % size);
        }
    }
}

// The status word, by one block: lengths, and the pages that the call's tokens lie in.
__device__ __forceinline__ void lc_check(const LatentCacheArgs& a) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    bool bad_len = false, bad_page = false;
    for (int n = warp; n < a.N; n += kLcWarps) {
        const int64_t from = a.cu ? a.cu[n] : n * a.rows_each, to = a.cu ? a.cu[n + 1] : from + a.rows_each;
        const int64_t len = a.lens[n];
        const bool off = from < 0 || to < from || to > a.T || (n == 0 && from != 0) || len < 0 ||
                         len > (int64_t)a.max_pages * a.page_size;
        bad_len |= off;
        if (off || to == from) continue;
        const int64_t first = len - (to - from) < 0 ? 0 : len - (to - from);
        for (int64_t p = first / a.page_size + lane; p * a.page_size < len; p += 32) {
            const int x = a.table[(int64_t)n * a.max_pages + p];
            bad_page |= x < 0 || x >= a.num_pages;
        }
    }
    bad_len = __syncthreads_or(bad_len);
    bad_page = __syncthreads_or(bad_page);
    if (threadIdx.x == 0) *a.status = bad_page ? KDA_ERR_BAD_PAGE : bad_len ? KDA_ERR_BAD_SEQLENS : KDA_OK;
}

// The codes of one vector, a byte each, from its first.
template <int kVec> struct LcCodes { uint32_t w[kVec / 4]; };

__device__ __forceinline__ uint32_t lc_code4(float a, float b, float c, float d) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    return lo | hi << 16;
}

// A lane's channels as words: their largest |finite| one (as a float's bits), and their codes under 2^e.  Two of 16 bits
// at once; infinities, which rarely are, are looked for again where the maximum shows one, and become NaN.
__device__ __forceinline__ uint32_t lc_top(uint4 (&v)[2], const __nv_bfloat16*) {
    uint32_t top = 0;
#pragma unroll
    for (int k = 0; k < 2; ++k)
        top = __vmaxu2(__vmaxu2(__vmaxu2(top, v[k].x & 0x7fff7fffu), __vmaxu2(v[k].y & 0x7fff7fffu, v[k].z & 0x7fff7fffu)),
                       v[k].w & 0x7fff7fffu);
    top = max(top & 0xffffu, top >> 16);
    if (top >= 0x7f80u) {
        top = 0;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            uint32_t* u = (uint32_t*)&v[k];
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const uint32_t lo = u[m] & 0x7fffu, hi = u[m] >> 16 & 0x7fffu;
                if (lo >= 0x7f80u) u[m] |= 0x7fffu;
                else top = max(top, lo);
                if (hi >= 0x7f80u) u[m] |= 0x7fff0000u;
                else top = max(top, hi);
            }
        }
    }
    return top << 16;
}
__device__ __forceinline__ uint32_t lc_top(uint4 (&v)[4], const float*) {
    float top = 0.f;
    const float* f = (const float*)v;
#pragma unroll
    for (int k = 0; k < 16; ++k) top = fmaxf(top, fabsf(f[k]));        // (leaves NaN out)
    if (top == INFINITY) {
        top = 0.f;
        float* g = (float*)v;
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            if (fabsf(g[k]) == INFINITY) g[k] = __uint_as_float(0x7fc00000u);
            top = fmaxf(top, fabsf(g[k]));
        }
    }
    return __float_as_uint(top);
}
__device__ __forceinline__ LcCodes<8> lc_codes(const uint4& v, float inv, const __nv_bfloat16*) {
    // (products with powers of two: exact in bf16 where the code is not 0)
    const __nv_bfloat162 by = __nv_bfloat162(__float2bfloat16(inv), __float2bfloat16(inv));
    float2 f[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        __nv_bfloat162 x;
        memcpy(&x, (const uint32_t*)&v + k, 4);
        f[k] = __bfloat1622float2(__hmul2(x, by));
    }
    return {{lc_code4(f[0].x, f[0].y, f[1].x, f[1].y), lc_code4(f[2].x, f[2].y, f[3].x, f[3].y)}};
}
__device__ __forceinline__ LcCodes<4> lc_codes(const uint4& v, float inv, const float*) {
    return {{lc_code4(__uint_as_float(v.x) * inv, __uint_as_float(v.y) * inv, __uint_as_float(v.z) * inv, __uint_as_float(v.w) * inv)}};
}

template <typename T, bool kWide, int kTokens>
__global__ void __launch_bounds__(32 * kLcWarps, sizeof(T) == 2 ? 5 : 4)
kda_latent_cache_write_kernel(const __grid_constant__ LatentCacheArgs a) {
    wait_before();
    follow_me();
    if (a.status && blockIdx.x == gridDim.x - 1) return lc_check(a);
    constexpr int kVec = LcRow<T>::kVec, kVecs = LcRow<T>::kVecs;
    const int lane = threadIdx.x & 31;
    const int64_t t0 = ((int64_t)blockIdx.x * kLcWarps + (threadIdx.x >> 5)) * kTokens;
    if (t0 >= a.T) return;
    LcRow<T> x[kTokens];
#pragma unroll
    for (int i = 0; i < kTokens; ++i)
        if (t0 + i < a.T) lc_load<T, kWide>(a, t0 + i, lane, x[i]);
    int page, row;
    lc_places<kTokens>(a, t0, page, row);
    const int width = latent_row_bytes(a.rank, a.d_rope);
#pragma unroll
    for (int i = 0; i < kTokens; ++i) {
        const int p = __shfl_sync(0xffffffffu, page, i), r = __shfl_sync(0xffffffffu, row, i);
        if (p < 0) continue;
        const uint32_t top = __reduce_max_sync(0xffffffffu, lc_top(x[i].v, (const T*)nullptr));
        const int e = latent_exponent(top);
        const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
        uint8_t* base = a.cache + p * a.page_stride;
        uint8_t* to = base + (int64_t)r * width;
#pragma unroll
        for (int k = 0; k < kVecs; ++k) {
            const LcCodes<kVec> w = lc_codes(x[i].v[k], inv, (const T*)nullptr);
            const int ch = lc_channel<T>(k, lane);
            if (ch >= a.rank) continue;
            if constexpr (kVec == 8) *(uint2*)(to + ch) = make_uint2(w.w[0], w.w[1]);
            else *(uint32_t*)(to + ch) = w.w[0];
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int ch = 64 * k + 2 * lane;
            if (ch >= a.d_rope) continue;
            const __nv_bfloat162 h = __floats2bfloat162_rn(to_f32(x[i].rope[k][0]), to_f32(x[i].rope[k][1]));
            *(uint32_t*)(to + a.rank + 2 * ch) = *(const uint32_t*)&h;
        }
        if (lane == 0) base[(int64_t)a.page_size * width + r] = (uint8_t)(e + kScaleBias);
    }
}

template <typename T, bool kWide, int kTokens>
__global__ void __launch_bounds__(32 * kLcWarps, 8)
kda_latent_cache_read_kernel(const __grid_constant__ LatentCacheArgs a) {
    wait_before();
    follow_me();
    if (a.status && blockIdx.x == gridDim.x - 1) return lc_check(a);
    constexpr int kVec = LcRow<T>::kVec, kVecs = LcRow<T>::kVecs;
    const int lane = threadIdx.x & 31;
    const int64_t t0 = ((int64_t)blockIdx.x * kLcWarps + (threadIdx.x >> 5)) * kTokens;
    if (t0 >= a.T) return;
    int page, row;
    lc_places<kTokens>(a, t0, page, row);
    const int width = latent_row_bytes(a.rank, a.d_rope);
    LcCodes<kVec> w[kTokens][kVecs];
    uint32_t rope[kTokens][2], e[kTokens];
#pragma unroll
    for (int i = 0; i < kTokens; ++i) {
        const int p = __shfl_sync(0xffffffffu, page, i), r = __shfl_sync(0xffffffffu, row, i);
        if (p < 0) continue;
        const uint8_t* base = a.cache + p * a.page_stride;
        const uint8_t* from = base + (int64_t)r * width;
#pragma unroll
        for (int k = 0; k < kVecs; ++k) {
            const int ch = lc_channel<T>(k, lane);
            if (ch >= a.rank) continue;
            if constexpr (kVec == 8) {
                const uint2 u = *(const uint2*)(from + ch);
                w[i][k].w[0] = u.x;
                w[i][k].w[1] = u.y;
            } else {
                w[i][k].w[0] = *(const uint32_t*)(from + ch);
            }
        }
        e[i] = base[(int64_t)a.page_size * width + r];
#pragma unroll
        for (int k = 0; k < 2; ++k)
            if (2 * lane + 64 * k < a.d_rope) rope[i][k] = *(const uint32_t*)(from + a.rank + 4 * lane + 128 * k);
    }
#pragma unroll
    for (int i = 0; i < kTokens; ++i) {
        if (__shfl_sync(0xffffffffu, page, i) < 0) continue;
        const float s = __uint_as_float(e[i] << 23);               // 2^e
        T* out = (T*)a.latents + (t0 + i) * a.latent_stride;
#pragma unroll
        for (int k = 0; k < kVecs; ++k) {
            const int ch = lc_channel<T>(k, lane);
            if (ch >= a.rank) continue;
            T v[kVec];
#pragma unroll
            for (int m = 0; m < kVec / 2; ++m) {
                const __half2 h = __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[i][k].w[m / 2] >> 16 * (m % 2)), __NV_E4M3));
                const float2 f = __half22float2(h);
                v[2 * m] = from_f32<T>(f.x * s);
                v[2 * m + 1] = from_f32<T>(f.y * s);
            }
            if constexpr (kWide) {
                uint4 u;
                memcpy(&u, v, 16);
                *(uint4*)(out + ch) = u;
            } else {
#pragma unroll
                for (int m = 0; m < kVec; ++m) out[ch + m] = v[m];
            }
        }
        T* to = (T*)a.rope + (t0 + i) * a.rope_stride;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int c = 2 * lane + 64 * k;
            if (c >= a.d_rope) continue;
            to[c] = from_f32<T>(__uint_as_float(rope[i][k] << 16));
            to[c + 1] = from_f32<T>(__uint_as_float(rope[i][k] & 0xffff0000u));
        }
    }
}

// ------------------------------------------------------------------- host
template <typename T, bool kWide, int kTokens>
static cudaError_t lc_launch_as(const LatentCacheArgs& a, bool write, cudaStream_t stream) {
    const int64_t blocks = (a.T + kLcWarps * kTokens - 1) / (kLcWarps * kTokens) + (a.status != nullptr);
    return launch_behind(write ? kda_latent_cache_write_kernel<T, kWide, kTokens> : kda_latent_cache_read_kernel<T, kWide, kTokens>,
                         dim3((unsigned)blocks), 32 * kLcWarps, 0, stream, a);
}

template <typename T>
static cudaError_t lc_launch(const LatentCacheArgs& a, bool write, cudaStream_t stream) {
    const bool wide = (((uintptr_t)a.latents | (uintptr_t)(a.latent_stride * (int64_t)sizeof(T))) & 15) == 0;
    // One token a warp while every SM has 32 warps for them, two behind that (65536 tokens, us: one 23, two 20, four 24)
    if (a.T <= 152 * 32) return wide ? lc_launch_as<T, true, 1>(a, write, stream) : lc_launch_as<T, false, 1>(a, write, stream);
    return wide ? lc_launch_as<T, true, 2>(a, write, stream) : lc_launch_as<T, false, 2>(a, write, stream);
}

cudaError_t latent_cache_launch(const LatentCacheArgs& a, bool write, cudaStream_t stream) {
    return a.dtype == KDA_BF16 ? lc_launch<__nv_bfloat16>(a, write, stream) : lc_launch<float>(a, write, stream);
}

}  // namespace kda
