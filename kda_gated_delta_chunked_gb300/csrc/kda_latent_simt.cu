// kda_latent_simt.cu -- latent attention on CUDA cores in fp32: every type, head
// size, stride and page size the interface admits.  It is the path of fp32
// inputs and of what the tensor-core kernels do not take, and the second
// opinion on what they do.
//
// One pass over the keys per query row with a running maximum m and sum l:
//
//     m' = max(m, s),  l <- l e^{m - m'} + e^{s - m'},  o <- o e^{m - m'} + e^{s - m'} v
//
// A warp owns a row, its lanes the channels (lane, lane + 32, ...), so a score
// is one warp reduction.  Bound by that reduction's latency, not by memory.
#include <cuda_fp16.h>
#include <string.h>

#include "kda_common.cuh"
#include "kda_latent_cache.cuh"
#include "kda_paths.h"

namespace kda {

constexpr int kSimtWarps = 4;

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// Folds key scores into (m, l, o).  s is the same in every lane.
template <int VC>
__device__ __forceinline__ void online_step(float s, float& m, float& l, float (&o)[VC], const float (&v)[VC]) {
    const float mn = fmaxf(m, s);
    // -infinity hides a key, also before the first finite score, where m is -infinity too (exp(-inf + inf)); a score
    // that is no number, which the maximum leaves out, makes the row one that is none
    const float keep = m == mn ? 1.f : expf(m - mn);
    const float p = s == -INFINITY ? 0.f : expf(s - mn);
    m = mn;
    l = l * keep + p;
#pragma unroll
    for (int c = 0; c < VC; ++c) o[c] = o[c] * keep + p * v[c];
}

// ------------------------------------------------------------- expanded form
template <typename T, int KC, int VC>
__global__ void __launch_bounds__(32 * kSimtWarps)
kda_latent_prefill_simt(LatentPrefillArgs a) {
    const int lane = threadIdx.x & 31;
    const int64_t t = blockIdx.x;
    const int h = blockIdx.y * kSimtWarps + (threadIdx.x >> 5);
    if (blockIdx.x == 0 && blockIdx.y == 0) check_cu_seqlens(a.cu_q, a.cu_k, a.N, a.tq, a.tk, a.status);
    if (h >= a.H || t >= a.tq) return;
    int64_t q0 = 0, q1 = a.tq, k0 = 0, k1 = a.tk;
    if (a.cu_q) {
        const int n = chunk_owner(a.cu_q, a.N, (int)t);
        q0 = a.cu_q[n]; q1 = a.cu_q[n + 1];
        k0 = a.cu_k[n]; k1 = a.cu_k[n + 1];
        k0 = k0 < 0 ? 0 : k0;                          // a malformed array reads nothing outside the tensors
        k1 = k1 > a.tk ? a.tk : k1;
    }
    const int64_t end = a.causal ? min64(k1, k0 + (k1 - k0) - (q1 - q0) + (t - q0) + 1) : k1;

    const int dqk = a.dk + a.dr;
    float q[KC], o[VC], v[VC];
    const T* qp = (const T*)a.q + t * a.q_ts + h * a.q_hs;
#pragma unroll
    for (int c = 0; c < KC; ++c) q[c] = lane + 32 * c < dqk ? to_f32(qp[lane + 32 * c]) : 0.f;
#pragma unroll
    for (int c = 0; c < VC; ++c) o[c] = 0.f;
    float m = -INFINITY, l = 0.f;
    for (int64_t j = k0; j < end; ++j) {
        const T* kp = (const T*)a.k + j * a.k_ts + h * a.k_hs;
        const T* rp = (const T*)a.r + j * a.r_ts;
        const T* vp = (const T*)a.v + j * a.v_ts + h * a.v_hs;
        float s = 0.f;
#pragma unroll
        for (int c = 0; c < KC; ++c) {
            const int e = lane + 32 * c;
            if (e < dqk) s += q[c] * to_f32(e < a.dk ? kp[e] : rp[e - a.dk]);
        }
#pragma unroll
        for (int c = 0; c < VC; ++c) v[c] = lane + 32 * c < a.dv ? to_f32(vp[lane + 32 * c]) : 0.f;
        online_step(warp_sum(s) * a.scale, m, l, o, v);
    }
    T* op = (T*)a.out + (t * a.H + h) * a.dv;
    const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
#pragma unroll
    for (int c = 0; c < VC; ++c)
        if (lane + 32 * c < a.dv) op[lane + 32 * c] = from_f32<T>(o[c] * inv);
    if (a.lse && lane == 0) a.lse[t * a.H + h] = m + logf(l);
}

cudaError_t latent_prefill_simt_launch(const LatentPrefillArgs& a, cudaStream_t stream) {
    const dim3 grid((unsigned)a.tq, (unsigned)((a.H + kSimtWarps - 1) / kSimtWarps));
    if (a.dtype == KDA_BF16)
        kda_latent_prefill_simt<__nv_bfloat16, 8, 8><<<grid, 32 * kSimtWarps, 0, stream>>>(a);
    else
        kda_latent_prefill_simt<float, 8, 8><<<grid, 32 * kSimtWarps, 0, stream>>>(a);
    return cudaGetLastError();
}

// ------------------------------------------------------------- calls without queries or sequences
__global__ void kda_latent_status_of_lengths(const int32_t* cu_q, const int32_t* cu_k, int N, int64_t tq, int64_t tk,
                                             int32_t* status) {
    check_cu_seqlens(cu_q, cu_k, N, tq, tk, status);
}

cudaError_t latent_status_launch(const int32_t* cu_q, const int32_t* cu_k, int N, int64_t tq, int64_t tk, int32_t* status,
                                 cudaStream_t stream) {
    kda_latent_status_of_lengths<<<1, 256, 0, stream>>>(cu_q, cu_k, N, tq, tk, status);
    return cudaGetLastError();
}

// ------------------------------------------------------------- absorbed form
template <typename T, int KC, int VC>
__global__ void __launch_bounds__(32 * kSimtWarps)
kda_latent_decode_simt(LatentDecodeArgs a) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t row = blockIdx.x;                     // (sequence, query)
    const int n = (int)(row / a.Lq), i = (int)(row % a.Lq), h = blockIdx.y;
    const int dqk = a.dk + a.dr;
    int64_t len = a.lens[n];
    if (len < 0 || len > (int64_t)a.max_pages * a.page_size) {
        if (threadIdx.x == 0) record_status(a.status, KDA_ERR_BAD_SEQLENS);
        len = 0;
    }
    const int64_t end = len - a.Lq + i + 1;

    float q[KC], o[VC], v[VC];
    const T* qp = (const T*)a.q + row * a.q_ts + h * a.q_hs;
#pragma unroll
    for (int c = 0; c < KC; ++c) q[c] = lane + 32 * c < dqk ? to_f32(qp[lane + 32 * c]) : 0.f;
#pragma unroll
    for (int c = 0; c < VC; ++c) o[c] = 0.f;
    float m = -INFINITY, l = 0.f;
    for (int64_t j = warp; j < end; j += kSimtWarps) {
        const int page = a.table[(int64_t)n * a.max_pages + j / a.page_size];
        if (page < 0 || page >= a.num_pages) {
            if (lane == 0) record_status(a.status, KDA_ERR_BAD_PAGE);
            continue;
        }
        const T* kp = (const T*)a.cache + page * a.page_stride + (j % a.page_size) * dqk;
        float s = 0.f;
#pragma unroll
        for (int c = 0; c < KC; ++c) {
            const float x = lane + 32 * c < dqk ? to_f32(kp[lane + 32 * c]) : 0.f;
            s += q[c] * x;
            if (c < VC) v[c] = lane + 32 * c < a.dk ? x : 0.f;
        }
        online_step(warp_sum(s) * a.scale, m, l, o, v);
    }
    // The warps' shares of the row meet in shared memory, in warp order.
    __shared__ float sh_o[kSimtWarps][32 * VC], sh_m[kSimtWarps], sh_l[kSimtWarps];
#pragma unroll
    for (int c = 0; c < VC; ++c) sh_o[warp][lane + 32 * c] = o[c];
    if (lane == 0) { sh_m[warp] = m; sh_l[warp] = l; }
    __syncthreads();
    float top = -INFINITY, total = 0.f, w[kSimtWarps];
#pragma unroll
    for (int k = 0; k < kSimtWarps; ++k) top = fmaxf(top, sh_m[k]);
#pragma unroll
    for (int k = 0; k < kSimtWarps; ++k) {
        w[k] = sh_m[k] == top ? (top == -INFINITY ? 0.f : 1.f) : expf(sh_m[k] - top);
        total += w[k] * sh_l[k];
    }
    const float inv = total > 0.f ? 1.f / total : (total == 0.f ? 0.f : total);
    T* op = (T*)a.out + (row * a.H + h) * a.dk;
    for (int e = threadIdx.x; e < a.dk; e += 32 * kSimtWarps) {
        float x = 0.f;
#pragma unroll
        for (int k = 0; k < kSimtWarps; ++k) x += w[k] * sh_o[k][e];
        op[e] = from_f32<T>(x * inv);
    }
    if (a.lse && threadIdx.x == 0) a.lse[row * a.H + h] = top + logf(total);
}

// Four e4m3 codes times 2^-8 as halves, codes 0 and 2, 1 and 3: sign, exponent and mantissa are moved, an exponent of 4
// bits then stands for itself less 8, subnormals too.  (The conversion instruction takes eight cycles of a scheduler.)
__device__ __forceinline__ void four_codes(uint32_t u, uint32_t& even, uint32_t& odd) {
    even = (u << 7 & 0x3f803f80u) | (u << 8 & 0x80008000u);
    odd = (u >> 1 & 0x3f803f80u) | (u & 0x80008000u);
}
// With NaN (all bits but the sign set), which is not itself then.
__device__ __forceinline__ bool nan_codes(uint4 u) {
    auto full = [](uint32_t x) { return (x & 0x7f7f7f7fu) + 0x01010101u; };
    return ((full(u.x) | full(u.y) | full(u.z) | full(u.w)) & 0x80808080u) != 0;
}
__device__ __forceinline__ void nan_halves(uint32_t u, uint32_t& even, uint32_t& odd) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        if ((u >> 16 * k & 0x7fu) == 0x7fu) even |= 0x7fffu << 16 * k;
        if ((u >> 16 * k & 0x7f00u) == 0x7f00u) odd |= 0x7fffu << 16 * k;
    }
}
__device__ __forceinline__ float2 two_halves(uint32_t x) {
    __half2 h;
    memcpy(&h, &x, 4);
    return __half22float2(h);
}

// The same over the quantised cache (kda_latent_cache.cuh).  A lane has 16 channels
// in a row, a token's codes in one access, and up to four rotary ones; four tokens
// at a time, so that their reductions go side by side.  Bound by instructions (about
// 200 a token and row) where there are rows enough, else by latency; sixteen warps a
// row serve both.  fp32, us: one sequence of 700 tokens, 32 heads 35 (four warps a row
// 82); 1 x 30000, 4 heads 1050 (3150); 37 x 3 queries of up to 3001 tokens, 16 heads
// 720; 64 x up to 16384, 32 heads 6170.  (Two heads a warp, eight warps: 720 and 6430;
// the next tokens asked for ahead, which spills: 815 and 7100.)
constexpr int kSimtTokens = 4, kSimt8Warps = 16;

// A lane's share of four tokens.
struct SimtTokens {
    uint4 code[kSimtTokens];
    uint2 rope[kSimtTokens];
    uint32_t byte[kSimtTokens];
    uint32_t there;                                     // a bit a token
};

__device__ __forceinline__ void simt_tokens(const LatentDecodeArgs& a, int n, int64_t j0, int64_t end, int lane, SimtTokens& x) {
    static_assert(kSimtTokens == 4, "the tokens of a page below");
    const int width = latent_row_bytes(a.dk, a.dr);
    const uint32_t size = a.page_size;
    const int32_t* table = a.table + (int64_t)n * a.max_pages;
    x.there = 0;
    uint32_t at = 0;
    int page = -1;
#pragma unroll
    for (int t = 0; t < kSimtTokens; ++t) {
        const uint32_t j = (uint32_t)(j0 + t);                         // (lengths are below 2^31)
        const bool seen = j0 + t < end;
        if (t == 0 || size % 4 != 0) {                                 // (else the four lie in one page)
            const uint32_t p = j / size;
            at = j - p * size;
            page = seen ? table[p] : -1;
        } else {
            ++at;
        }
        const bool there = seen && page >= 0 && page < a.num_pages;
        if (seen && !there && lane == 0) record_status(a.status, KDA_ERR_BAD_PAGE);
        x.code[t] = make_uint4(0, 0, 0, 0);
        x.rope[t] = make_uint2(0, 0);
        x.byte[t] = 0;
        if (!there) continue;
        x.there |= 1u << t;
        const uint8_t* base = (const uint8_t*)a.cache + page * a.page_stride;
        const uint8_t* from = base + (int64_t)at * width;
        if (lane * 16 < a.dk) x.code[t] = *(const uint4*)(from + lane * 16);
        if (lane * 4 < a.dr) x.rope[t] = *(const uint2*)(from + a.dk + lane * 8);
        x.byte[t] = base[(int64_t)size * width + at];
    }
}

template <typename T>
__global__ void __launch_bounds__(32 * kSimt8Warps)
kda_latent_decode8_simt(const __grid_constant__ LatentDecodeArgs a) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t row = blockIdx.x;                     // (sequence, query)
    const int n = (int)(row / a.Lq), i = (int)(row % a.Lq), h = blockIdx.y;
    int64_t len = a.lens[n];
    if (len < 0 || len > (int64_t)a.max_pages * a.page_size) {
        if (threadIdx.x == 0) record_status(a.status, KDA_ERR_BAD_SEQLENS);
        len = 0;
    }
    const int64_t end = len - a.Lq + i + 1;
    const bool mine = lane * 16 < a.dk;

    float q[16], qr[4], o[16], m = -INFINITY, l = 0.f;  // o: times 2^-8
    const T* qp = (const T*)a.q + row * a.q_ts + h * a.q_hs;
#pragma unroll
    for (int c = 0; c < 16; ++c) {
        q[c] = mine ? to_f32(qp[lane * 16 + c]) : 0.f;
        o[c] = 0.f;
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) qr[c] = lane * 4 + c < a.dr ? to_f32(qp[a.dk + lane * 4 + c]) : 0.f;
    for (int64_t j0 = (int64_t)warp * kSimtTokens; j0 < end; j0 += kSimt8Warps * kSimtTokens) {
        SimtTokens x;
        simt_tokens(a, n, j0, end, lane, x);
        uint32_t half[kSimtTokens][8];                                 // channels 0 and 2, 1 and 3, 4 and 6, ...
        float s[kSimtTokens];
#pragma unroll
        for (int t = 0; t < kSimtTokens; ++t) {
            const uint32_t u[4] = {x.code[t].x, x.code[t].y, x.code[t].z, x.code[t].w};
#pragma unroll
            for (int c = 0; c < 4; ++c) four_codes(u[c], half[t][2 * c], half[t][2 * c + 1]);
            if (nan_codes(x.code[t])) {
#pragma unroll
                for (int c = 0; c < 4; ++c) nan_halves(u[c], half[t][2 * c], half[t][2 * c + 1]);
            }
            float dot = 0.f;
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                const float2 f = two_halves(half[t][c]);
                const int at = c / 2 * 4 + c % 2;
                dot = fmaf(q[at + 2], f.y, fmaf(q[at], f.x, dot));
            }
            float y = qr[0] * __uint_as_float(x.rope[t].x << 16);
            y = fmaf(qr[1], __uint_as_float(x.rope[t].x & 0xffff0000u), y);
            y = fmaf(qr[2], __uint_as_float(x.rope[t].y << 16), y);
            y = fmaf(qr[3], __uint_as_float(x.rope[t].y & 0xffff0000u), y);
            s[t] = fmaf(256.f * dot, __uint_as_float(x.byte[t] << 23), y);         // (the byte's bits: 2^e)
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1)
#pragma unroll
            for (int t = 0; t < kSimtTokens; ++t) s[t] += __shfl_xor_sync(0xffffffffu, s[t], d);
        float mn = m;
#pragma unroll
        for (int t = 0; t < kSimtTokens; ++t) {
            s[t] = x.there >> t & 1 ? s[t] * a.scale : -INFINITY;
            mn = fmaxf(mn, s[t]);
        }
        // (as in online_step: -infinity hides a token, also before the first finite score)
        if (m != mn) {                                                 // (the same in every lane)
            const float keep = expf(m - mn);
            m = mn;
            l *= keep;
#pragma unroll
            for (int c = 0; c < 16; ++c) o[c] *= keep;
        }
#pragma unroll
        for (int t = 0; t < kSimtTokens; ++t) {
            const float p = s[t] == -INFINITY ? 0.f : expf(s[t] - mn);
            l += p;
            if (!(x.there >> t & 1)) continue;                         // (in every lane)
            const float w = p * __uint_as_float(x.byte[t] << 23);
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                const float2 f = two_halves(half[t][c]);
                const int at = c / 2 * 4 + c % 2;
                o[at] = fmaf(w, f.x, o[at]);
                o[at + 2] = fmaf(w, f.y, o[at + 2]);
            }
        }
    }
    // The warps' shares of the row meet in shared memory, in warp order.
    __shared__ float sh_o[kSimt8Warps][512], sh_m[kSimt8Warps], sh_l[kSimt8Warps];
#pragma unroll
    for (int c = 0; c < 16; ++c) sh_o[warp][lane * 16 + c] = o[c];
    if (lane == 0) { sh_m[warp] = m; sh_l[warp] = l; }
    __syncthreads();
    float top = -INFINITY, total = 0.f, w[kSimt8Warps];
#pragma unroll
    for (int k = 0; k < kSimt8Warps; ++k) top = fmaxf(top, sh_m[k]);
#pragma unroll
    for (int k = 0; k < kSimt8Warps; ++k) {
        w[k] = sh_m[k] == top ? (top == -INFINITY ? 0.f : 1.f) : expf(sh_m[k] - top);
        total += w[k] * sh_l[k];
    }
    const float inv = total > 0.f ? 256.f / total : (total == 0.f ? 0.f : total);
    T* op = (T*)a.out + (row * a.H + h) * a.dk;
    for (int e = threadIdx.x; e < a.dk; e += 32 * kSimt8Warps) {
        float x = 0.f;
#pragma unroll
        for (int k = 0; k < kSimt8Warps; ++k) x += w[k] * sh_o[k][e];
        op[e] = from_f32<T>(x * inv);
    }
    if (a.lse && threadIdx.x == 0) a.lse[row * a.H + h] = top + logf(total);
}

cudaError_t latent_decode_simt_launch(const LatentDecodeArgs& a, cudaStream_t stream) {
    const dim3 grid((unsigned)((int64_t)a.N * a.Lq), (unsigned)a.H);
    if (a.codes && a.dtype == KDA_BF16)
        kda_latent_decode8_simt<__nv_bfloat16><<<grid, 32 * kSimt8Warps, 0, stream>>>(a);
    else if (a.codes)
        kda_latent_decode8_simt<float><<<grid, 32 * kSimt8Warps, 0, stream>>>(a);
    else if (a.dtype == KDA_BF16)
        kda_latent_decode_simt<__nv_bfloat16, 20, 16><<<grid, 32 * kSimtWarps, 0, stream>>>(a);
    else
        kda_latent_decode_simt<float, 20, 16><<<grid, 32 * kSimtWarps, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace kda
