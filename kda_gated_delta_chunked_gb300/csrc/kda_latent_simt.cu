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
#include "kda_common.cuh"
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

cudaError_t latent_decode_simt_launch(const LatentDecodeArgs& a, cudaStream_t stream) {
    const dim3 grid((unsigned)((int64_t)a.N * a.Lq), (unsigned)a.H);
    if (a.dtype == KDA_BF16)
        kda_latent_decode_simt<__nv_bfloat16, 20, 16><<<grid, 32 * kSimtWarps, 0, stream>>>(a);
    else
        kda_latent_decode_simt<float, 20, 16><<<grid, 32 * kSimtWarps, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace kda
