// kda_rotary.cu -- rotary positions of queries and keys.
//
//     theta = position f_i,   (a_i, b_i) -> scale (a_i cos - b_i sin, b_i cos + a_i sin)
//
// Bound by HBM bytes (every channel read once and written once; in place the
// channels beside the turned ones are not touched).  A block takes some rows
// (token and head) and forms their tokens' sines and cosines once, in shared
// memory, while its loads are on their way; a thread takes `kRotSteps` vectors.
//
// The angle: f / (2 pi) turns a position, as a 64-bit fraction of a turn, times
// the position in 64-bit integers that wrap at whole turns.  What is left is off
// by 2^-53 of f / (2 pi), times the position, whatever the position; its first 32
// bits go to sincospi in fp32.
#include "kda_common.cuh"
#include "kda_paths.h"

namespace kda {

constexpr int kRotThreads = 256, kRotSteps = 4;
constexpr int kRotTable = 2048;                     // pairs of a block's tokens
constexpr int kRotDim = 1024;

struct RotPart {
    const char* in;
    char* out;
    int64_t its, ihs, ots, ohs;                     // bytes
    int heads, offset;                              // offset: elements
    int turned, units;                              // vectors (half layout: pairs of them) that are turned; all
};
struct RotArgs {
    RotPart part[2];
    int64_t tokens;
    int dim, rows, units, tokens_block, rows_block; // rows of a token, vectors of a row (of both parts)
    uint32_t by_rows, by_units;                     // 2^32 / rows, 2^32 / units, rounded up
    int flags;
    float scale;
    const void* positions;
    const double* frequencies;
};

// u / d with m = 2^32 / d rounded up: exact while u d < 2^32.
__device__ __forceinline__ int rot_divide(int u, int d, uint32_t m) { return d == 1 ? u : (int)__umulhi((uint32_t)u, m); }

template <int B> struct RotVec;
template <> struct RotVec<16> { uint4 v; };
template <> struct RotVec<8> { uint2 v; };
template <> struct RotVec<4> { uint32_t v; };
template <> struct RotVec<2> { uint16_t v; };

template <typename T, int B>
__device__ __forceinline__ void rot_get(const RotVec<B>& x, float (&f)[B / sizeof(T)]) {
    T e[B / sizeof(T)];
    memcpy(e, &x, B);
#pragma unroll
    for (int i = 0; i < (int)(B / sizeof(T)); ++i) f[i] = to_f32(e[i]);
}
template <typename T, int B>
__device__ __forceinline__ RotVec<B> rot_set(const float (&f)[B / sizeof(T)]) {
    T e[B / sizeof(T)];
#pragma unroll
    for (int i = 0; i < (int)(B / sizeof(T)); ++i) e[i] = from_f32<T>(f[i]);
    RotVec<B> x;
    memcpy(&x, e, B);
    return x;
}

// Which product is rounded by itself is said here, so that every width of access gives the same bits.
__device__ __forceinline__ void rot_turn(float& a, float& b, float2 w) {
    const float p = fmaf(a, w.x, -__fmul_rn(b, w.y)), q = fmaf(b, w.x, __fmul_rn(a, w.y));
    a = p;
    b = q;
}

// B: bytes of a vector.  A unit is what a thread turns or copies at once: with
// neighbouring pairs one vector, else the two vectors of the same pairs (of a
// single element each where B is an element's size, in both layouts).
template <typename T, int B, bool kNear>
__global__ void __launch_bounds__(kRotThreads)
kda_rotary_kernel(const __grid_constant__ RotArgs a) {
    constexpr int V = B / (int)sizeof(T);
    constexpr bool kTwo = !kNear || V == 1;                        // two vectors a unit
    constexpr int kPairs = kTwo ? V : V / 2;
    __shared__ unsigned long long turn[kRotDim / 2];
    __shared__ __align__(16) float2 table[kRotTable];
    const int half = a.dim / 2;
    const int64_t token0 = (int64_t)blockIdx.x * a.tokens_block;
    const int row0 = blockIdx.y * a.rows_block;                    // (more than one y: one token a block)
    const int tokens = (int)min64(a.tokens_block, a.tokens - token0);
    const int rows = a.tokens_block > 1 ? tokens * a.rows : min(a.rows_block, a.rows - row0);
    const int total = rows * a.units;
    for (int base = 0; base < total; base += kRotThreads * kRotSteps) {
        RotVec<B> va[kRotSteps], vb[kRotSteps];
        char* to[kRotSteps];
        int at[kRotSteps];                                         // first pair in the table, -1: a copy
#pragma unroll
        for (int k = 0; k < kRotSteps; ++k) {
            to[k] = nullptr;
            const int u = base + k * kRotThreads + (int)threadIdx.x;
            if (u >= total) continue;
            const int r = rot_divide(u, a.units, a.by_units), unit = u - r * a.units;
            const int token = a.tokens_block > 1 ? rot_divide(r, a.rows, a.by_rows) : 0;
            int head = r - token * a.rows + row0;
            const bool key = head >= a.part[0].heads;
            const RotPart& p = a.part[key];
            if (key) head -= a.part[0].heads;
            if (unit >= p.units) continue;
            const char* from = p.in + (token0 + token) * p.its + head * p.ihs;
            to[k] = p.out + (token0 + token) * p.ots + head * p.ohs;
            int e;
            if (unit < p.turned) {
                at[k] = token * half + unit * kPairs;
                e = p.offset + (kNear ? (V == 1 ? 2 * unit : unit * V) : unit * V);
            } else {
                at[k] = -1;
                e = (unit - p.turned) * V;
                if (e >= p.offset) e += a.dim;
            }
            from += (int64_t)e * (int)sizeof(T);
            to[k] += (int64_t)e * (int)sizeof(T);
            va[k] = *(const RotVec<B>*)from;
            if (kTwo && at[k] >= 0) vb[k] = *(const RotVec<B>*)(from + (kNear ? 1 : half) * (int)sizeof(T));
        }
        if (base == 0) {
            for (int i = threadIdx.x; i < half; i += kRotThreads) {
                double t = a.frequencies[i] * 0.15915494309189533577;      // 1 / (2 pi)
                t -= rint(t);
                turn[i] = (unsigned long long)__double2ll_rn(t * 18446744073709551616.0);
            }
            __syncthreads();
            const float sign = a.flags & KDA_FLAG_INVERSE ? -a.scale : a.scale;
            for (int e = threadIdx.x; e < tokens * half; e += kRotThreads) {
                const int token = e / half;
                const long long pos = a.flags & KDA_FLAG_POSITIONS_64 ? ((const int64_t*)a.positions)[token0 + token]
                                                                     : ((const int32_t*)a.positions)[token0 + token];
                const unsigned long long whole = (unsigned long long)pos * turn[e - token * half];
                float s, c;
                sincospif((float)(int)(whole >> 32) * 0x1p-31f, &s, &c);
                table[e] = make_float2(a.scale * c, sign * s);
            }
            __syncthreads();
        }
        constexpr int64_t kApart = kNear ? sizeof(T) : 0;
#pragma unroll
        for (int k = 0; k < kRotSteps; ++k) {
            if (!to[k]) continue;
            if (at[k] < 0) {
                *(RotVec<B>*)to[k] = va[k];
                continue;
            }
            float2 cs[kPairs];                                     // (at: a multiple of kPairs where that is even)
            if constexpr (kPairs % 2 == 0) {
#pragma unroll
                for (int i = 0; i < kPairs; i += 2) {
                    const float4 w = *(const float4*)(table + at[k] + i);
                    cs[i] = make_float2(w.x, w.y);
                    cs[i + 1] = make_float2(w.z, w.w);
                }
            } else {
                cs[0] = table[at[k]];
            }
            float x[V], y[V];
            rot_get<T, B>(va[k], x);
            if constexpr (kTwo) {
                rot_get<T, B>(vb[k], y);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    rot_turn(x[i], y[i], cs[i]);
                }
                *(RotVec<B>*)to[k] = rot_set<T, B>(x);
                *(RotVec<B>*)(to[k] + (kNear ? kApart : (int64_t)half * (int)sizeof(T))) = rot_set<T, B>(y);
            } else {
#pragma unroll
                for (int i = 0; i < V / 2; ++i) {
                    rot_turn(x[2 * i], x[2 * i + 1], cs[i]);
                }
                *(RotVec<B>*)to[k] = rot_set<T, B>(x);
            }
        }
    }
}

// ------------------------------------------------------------------- host
template <typename T, int B, bool kNear>
static cudaError_t rotary_launch_as(RotArgs a, cudaStream_t stream) {
    constexpr int V = B / (int)sizeof(T);
    a.units = 1;
    a.rows = 0;
    for (RotPart& p : a.part) {
        if (!p.in) { p.heads = 0; continue; }
        p.turned = kNear && V > 1 ? a.dim / V : a.dim / 2 / V;
        p.units = p.turned + p.units / V;                          // (units: channels to copy so far)
        a.units = p.units > a.units ? p.units : a.units;
        a.rows += p.heads;
    }
    // As many rows as give each thread its vectors, of one token or of several (as the table holds)
    const int fit = kRotThreads * kRotSteps / a.units, half = a.dim / 2;
    a.rows_block = fit < 1 ? 1 + a.rows / 65536 : fit;             // (at most 65535 blocks in y)
    a.tokens_block = 1;
    if (a.rows_block >= a.rows) {
        a.tokens_block = a.rows_block / a.rows;
        if (a.tokens_block > kRotTable / half) a.tokens_block = kRotTable / half;
        a.rows_block = a.rows;
    }
    a.by_rows = (uint32_t)((0x100000000ull + a.rows - 1) / a.rows);
    a.by_units = (uint32_t)((0x100000000ull + a.units - 1) / a.units);
    const dim3 grid((unsigned)((a.tokens + a.tokens_block - 1) / a.tokens_block), (unsigned)((a.rows + a.rows_block - 1) / a.rows_block));
    kda_rotary_kernel<T, B, kNear><<<grid, kRotThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

template <typename T, int B>
static cudaError_t rotary_launch_near(const RotArgs& a, cudaStream_t stream) {
    return a.flags & KDA_FLAG_INTERLEAVED ? rotary_launch_as<T, B, true>(a, stream) : rotary_launch_as<T, B, false>(a, stream);
}

cudaError_t rotary_launch(const kda_rotary_desc& d, const void* x, const void* key, const void* positions,
                          const double* frequencies, void* out, void* key_out, cudaStream_t stream) {
    RotArgs a = {};
    a.tokens = d.tokens; a.dim = d.dim; a.flags = d.flags; a.scale = d.scale;
    a.positions = positions; a.frequencies = frequencies;
    const int64_t e = d.dtype == KDA_BF16 ? 2 : 4;
    // 16-byte vectors, or the widest on whose boundaries everything starts that a vector of its own covers
    uint64_t bits = (uint64_t)((d.flags & KDA_FLAG_INTERLEAVED ? d.dim : d.dim / 2) * e);
    for (int i = 0; i < 2; ++i) {
        const kda_rotary_part& s = i ? d.key : d.x;
        RotPart& p = a.part[i];
        p.in = (const char*)(i ? key : x);
        p.out = (char*)(i ? key_out : out);
        if (!p.in) continue;
        p.its = s.token_stride * e; p.ihs = s.head_stride * e; p.ots = s.out_token_stride * e; p.ohs = s.out_head_stride * e;
        p.heads = s.heads; p.offset = s.offset;
        p.units = p.in == p.out ? 0 : s.width - d.dim;
        bits |= (uint64_t)(uintptr_t)p.in | (uint64_t)(uintptr_t)p.out | (uint64_t)(s.offset * e);
        if (d.tokens > 1) bits |= (uint64_t)(p.its | p.ots);
        if (s.heads > 1) bits |= (uint64_t)(p.ihs | p.ohs);
        if (p.units) bits |= (uint64_t)(s.width * e);
    }
    if (d.dtype == KDA_BF16) {
        if ((bits & 15) == 0) return rotary_launch_near<__nv_bfloat16, 16>(a, stream);
        if ((bits & 3) == 0) return rotary_launch_near<__nv_bfloat16, 4>(a, stream);
        return rotary_launch_near<__nv_bfloat16, 2>(a, stream);
    }
    return (bits & 15) == 0 ? rotary_launch_near<float, 16>(a, stream) : rotary_launch_near<float, 4>(a, stream);
}

}  // namespace kda
