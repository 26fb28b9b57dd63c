// kda_rotary.cu -- rotary positions of queries and keys.
//
//     theta = position f_i,   (a_i, b_i) -> scale (a_i cos - b_i sin, b_i cos + a_i sin)
//
// Bound by HBM bytes (every channel read once and written once; in place the
// channels beside the turned ones are not touched).  A block takes some rows
// (token and head) of the queries or of the keys and forms their tokens' sines and
// cosines once, in shared memory, while its first loads are on their way.  A thread
// has a vector or two at a time, the turned ones of all rows before the copied
// ones, so that a warp does one of the two; 32 registers, so that an SM is full of
// them (with four vectors and 64 registers: 32768 tokens of 32 x 192 in 154 us).
// Measured, us in a graph of ten (floor): that 120 (120); 65536 tokens of 8 heads
// of 128 and a key 56 (45); 65536 of one head of 64 9 (2.5: two million sines and
// as many cosines); one token of 32 heads 2.5.
//
// The angle: f / (2 pi) turns a position, as a 64-bit fraction of a turn, times
// the position in 64-bit integers that wrap at whole turns: off by 2^-63 of f / (2 pi)
// and by 2^-64, times the position.  Its first 32 bits go to sincospi in fp32.
#include <math.h>
#include <string.h>

#include "kda_common.cuh"
#include "kda_launch.cuh"
#include "kda_paths.h"

namespace kda {

constexpr int kRotThreads = 256;
constexpr int kRotTable = 2048;                     // pairs of a block's tokens
constexpr int kRotTurns = 4;

struct RotPart {
    const char* in;
    char* out;
    int64_t its, ihs, ots, ohs;                     // bytes
    int heads, offset;                              // offset: elements
    int turned, copied;                             // a row's vectors (half layout: pairs of them) that are turned; the others
    uint32_t by_turned, by_copied, by_heads;        // 2^32 over them, rounded up
    int tokens_block, rows_block;                   // of a block: tokens (then all heads), or rows of one token
    int64_t blocks;
    int across;                                     // blocks of a token
};
struct RotArgs {
    RotPart part[2];
    int64_t tokens;
    int dim, flags;
    float scale;
    const void* positions;
    const double* frequencies;
};

// u / d with m = 2^32 / d rounded up: exact while u d < 2^32.
__device__ __forceinline__ int rot_divide(int u, int d, uint32_t m) { return d == 1 ? u : (int)__umulhi((uint32_t)u, m); }

// f / (2 pi) as a 64-bit fraction of a turn (f finite), from the double's bits: 53 of them times 2^64 / pi, shifted to
// where f's exponent says.  (In fp64, of which the SM has little, this took longer than the sines.)
__device__ __forceinline__ unsigned long long rot_turns(double f) {
    const unsigned long long bits = (unsigned long long)__double_as_longlong(f);
    const int exponent = (int)(bits >> 52 & 0x7ff);
    const unsigned long long m = (bits & 0xfffffffffffffull) | (exponent ? 1ull << 52 : 0ull);
    const unsigned long long k = 5871781006564002453ull;           // 2^64 / pi
    const unsigned long long lo = m * k, hi = __umul64hi(m, k);
    const int down = 1076 - (exponent ? exponent : 1);             // turns 2^64 = (hi, lo) 2^-down
    unsigned long long t;
    if (down >= 128) t = 0;
    else if (down >= 64) t = hi >> (down - 64);
    else if (down > 0) t = hi << (64 - down) | lo >> down;
    else t = down > -64 ? lo << -down : 0;
    return bits >> 63 ? 0 - t : t;
}

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
struct RotShape {
    static constexpr int V = B / (int)sizeof(T);
    static constexpr bool kTwo = !kNear || V == 1;                 // two vectors a unit
    static constexpr int kPairs = kTwo ? V : V / 2;
    static constexpr int kSteps = (B == 16 ? 2 : 4) / (kTwo ? 2 : 1);   // units of a thread at once
};

template <typename T, int B, bool kNear>
__global__ void __launch_bounds__(kRotThreads, 8)
kda_rotary_kernel(const __grid_constant__ RotArgs a) {
    using S = RotShape<T, B, kNear>;
    constexpr int V = S::V, kPairs = S::kPairs, kSteps = S::kSteps;
    __shared__ __align__(16) float2 table[kRotTable];
    wait_before();
    follow_me();
    const int half = a.dim / 2;
    const bool key = blockIdx.x >= a.part[0].blocks;
    const RotPart& p = a.part[key];
    const uint32_t block = blockIdx.x - (key ? (uint32_t)a.part[0].blocks : 0);
    const int64_t token0 = p.across > 1 ? block / (uint32_t)p.across : (int64_t)block * p.tokens_block;
    const int row0 = p.across > 1 ? (int)(block % (uint32_t)p.across) * p.rows_block : 0;
    const int tokens = (int)min64(p.tokens_block, a.tokens - token0);
    const int rows = p.across > 1 ? min(p.rows_block, p.heads - row0) : tokens * p.heads;
    const int turned = rows * p.turned, total = turned + rows * p.copied;
    const char* in = p.in + token0 * p.its + row0 * p.ihs;
    char* out = p.out + token0 * p.ots + row0 * p.ohs;
    const int apart = kNear ? (int)sizeof(T) : half * (int)sizeof(T);
    for (int base = 0; base < total; base += kRotThreads * kSteps) {
        RotVec<B> va[kSteps], vb[kSteps];
        char* to[kSteps];
        int at[kSteps];                                            // first pair in the table, -1: a copy
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
            to[k] = nullptr;
            const int u = base + k * kRotThreads + (int)threadIdx.x;
            if (u >= total) continue;
            int r, e;
            if (u < turned) {
                r = rot_divide(u, p.turned, p.by_turned);
                const int unit = u - r * p.turned;
                e = p.offset + (kNear && V == 1 ? 2 * unit : unit * V);
                at[k] = unit * kPairs;
            } else {
                const int v = u - turned;
                r = rot_divide(v, p.copied, p.by_copied);
                e = (v - r * p.copied) * V;
                if (e >= p.offset) e += a.dim;
                at[k] = -1;
            }
            int token = 0;
            if (p.tokens_block > 1) {
                token = rot_divide(r, p.heads, p.by_heads);
                r -= token * p.heads;
                if (at[k] >= 0) at[k] += token * half;
            }
            const char* from = in + token * p.its + r * p.ihs + e * (int)sizeof(T);
            to[k] = out + token * p.ots + r * p.ohs + e * (int)sizeof(T);
            va[k] = *(const RotVec<B>*)from;
            if (S::kTwo && at[k] >= 0) vb[k] = *(const RotVec<B>*)(from + apart);
        }
        if (base == 0) {
            // A thread's pairs are of one frequency (of one at a time, where there are more frequencies than threads)
            const int each = half < kRotThreads ? kRotThreads / half : 1;      // tokens at once
            const int first = half < kRotThreads ? (int)threadIdx.x / half : 0;
            for (int i = (int)threadIdx.x - first * half; i < half && first < each; i += kRotThreads) {
                const double f = a.frequencies[i];
                const unsigned long long turns = rot_turns(f);
                const bool none = (__double2hiint(f) & 0x7ff00000) == 0x7ff00000;      // infinite or NaN
                const float scale = none ? NAN : a.scale;
                for (int token = first; token < tokens; token += each) {
                    const long long pos = a.flags & KDA_FLAG_POSITIONS_64 ? ((const int64_t*)a.positions)[token0 + token]
                                                                         : ((const int32_t*)a.positions)[token0 + token];
                    const float angle = (float)(int)((unsigned long long)pos * turns >> 32) * 0x1p-31f;    // half turns
                    float s, c;
                    sincospif(angle, &s, &c);
                    table[token * half + i] = make_float2(scale * c, (a.flags & KDA_FLAG_INVERSE ? -scale : scale) * s);
                }
            }
            __syncthreads();
        }
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
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
            if constexpr (S::kTwo) {
                rot_get<T, B>(vb[k], y);
#pragma unroll
                for (int i = 0; i < V; ++i) rot_turn(x[i], y[i], cs[i]);
                *(RotVec<B>*)(to[k] + apart) = rot_set<T, B>(y);
            } else {
#pragma unroll
                for (int i = 0; i < V / 2; ++i) rot_turn(x[2 * i], x[2 * i + 1], cs[i]);
            }
            *(RotVec<B>*)to[k] = rot_set<T, B>(x);
        }
    }
}

// ------------------------------------------------------------------- host
template <typename T, int B, bool kNear>
static cudaError_t rotary_launch_as(RotArgs a, cudaStream_t stream) {
    using S = RotShape<T, B, kNear>;
    const int half = a.dim / 2, block = kRotThreads * S::kSteps;
    auto over = [](int d) { return (uint32_t)((0x100000000ull + d - 1) / (d < 1 ? 1 : d)); };
    for (RotPart& p : a.part) {
        if (!p.in) continue;
        p.turned = half / S::kPairs;
        p.copied /= S::V;                                          // (channels so far)
        p.by_turned = over(p.turned);
        p.by_copied = over(p.copied);
        p.by_heads = over(p.heads);
        // Rows of a block, of one token or of several (as the table holds): up to kRotTurns vectors after one another a
        // thread, while that leaves each SM twice the blocks that it runs at once
        const int units = p.turned + p.copied;
        const int64_t turns = a.tokens * p.heads * units / ((int64_t)block * 152 * 16);
        const int fit = block * (int)(turns < 1 ? 1 : turns > kRotTurns ? kRotTurns : turns) / units;
        p.rows_block = fit < 1 ? 1 : fit;
        p.tokens_block = 1;
        p.across = (p.heads + p.rows_block - 1) / p.rows_block;
        if (p.across == 1) {
            p.tokens_block = p.rows_block / p.heads;
            if (p.tokens_block > kRotTable / half) p.tokens_block = kRotTable / half;
        }
        p.blocks = p.across > 1 ? a.tokens * p.across : (a.tokens + p.tokens_block - 1) / p.tokens_block;
    }
    const int64_t blocks = a.part[0].blocks + a.part[1].blocks;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    return launch_behind(kda_rotary_kernel<T, B, kNear>, dim3((unsigned)blocks), kRotThreads, 0, stream, a);
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
    // 16-byte vectors, or the widest on whose boundaries everything starts that a vector of its own covers (20000 x 4 rows
    // of 100 bf16, 64 turned: 11.7 us with 8 bytes, 15.9 with 4; 98: 15.7; of 100, 50 turned: 27.2 with 2)
    uint64_t bits = (uint64_t)((d.flags & KDA_FLAG_INTERLEAVED ? d.dim : d.dim / 2) * e);
    for (int i = 0; i < 2; ++i) {
        const kda_rotary_part& s = i ? d.key : d.x;
        RotPart& p = a.part[i];
        p.in = (const char*)(i ? key : x);
        p.out = (char*)(i ? key_out : out);
        if (!p.in) continue;
        p.its = s.token_stride * e; p.ihs = s.head_stride * e; p.ots = s.out_token_stride * e; p.ohs = s.out_head_stride * e;
        p.heads = s.heads; p.offset = s.offset;
        p.copied = p.in == p.out ? 0 : s.width - d.dim;
        bits |= (uint64_t)(uintptr_t)p.in | (uint64_t)(uintptr_t)p.out | (uint64_t)(s.offset * e);
        if (d.tokens > 1) bits |= (uint64_t)(p.its | p.ots);
        if (s.heads > 1) bits |= (uint64_t)(p.ihs | p.ohs);
        if (p.copied) bits |= (uint64_t)(s.width * e);
    }
    if (d.dtype == KDA_BF16) {
        if ((bits & 15) == 0) return rotary_launch_near<__nv_bfloat16, 16>(a, stream);
        if ((bits & 7) == 0) return rotary_launch_near<__nv_bfloat16, 8>(a, stream);
        if ((bits & 3) == 0) return rotary_launch_near<__nv_bfloat16, 4>(a, stream);
        return rotary_launch_near<__nv_bfloat16, 2>(a, stream);
    }
    if ((bits & 15) == 0) return rotary_launch_near<float, 16>(a, stream);
    return (bits & 7) == 0 ? rotary_launch_near<float, 8>(a, stream) : rotary_launch_near<float, 4>(a, stream);
}

}  // namespace kda
