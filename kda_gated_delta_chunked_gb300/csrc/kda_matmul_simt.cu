// kda_matmul_simt.cu -- the scaled e4m3 product on CUDA cores: rows of any
// alignment, and the second opinion on the tensor-core kernel.
//
//     c = sum over k blocks j of  a_scale[m, j] b_scale[n / 128, j] (sum_{k in j} a b)
//
// 64 x 64 tiles of c, 16 x 16 threads with 4 x 4 elements each, operands
// converted to fp32 in shared memory 32 values of k at a time.  Bound by the
// shared-memory reads of two 4-vectors per 16 multiply-adds.
#include <cuda_fp8.h>

#include "kda_common.cuh"
#include "kda_paths.h"

namespace kda {

constexpr int kMsTile = 64, kMsK = 32;

__device__ __forceinline__ float e4m3_to_f32(uint8_t x) {
    return __half2float(__half(__nv_cvt_fp8_to_halfraw(x, __NV_E4M3)));
}

template <typename T>
__global__ void __launch_bounds__(256)
kda_matmul_fp8_simt(MatmulArgs a) {
    __shared__ float sa[kMsK][kMsTile + 4], sb[kMsK][kMsTile + 4];
    const int64_t m0 = (int64_t)blockIdx.x * kMsTile;
    const int n0 = blockIdx.y * kMsTile;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int kb = (a.k + 127) / 128;
    float c[4][4] = {}, part[4][4] = {};
    for (int k0 = 0; k0 < a.k; k0 += kMsK) {
        __syncthreads();
        for (int i = threadIdx.x; i < kMsTile * kMsK; i += 256) {
            const int r = i / kMsK, k = i % kMsK;
            const bool in_k = k0 + k < a.k;
            sa[k][r] = in_k && m0 + r < a.m ? e4m3_to_f32(a.a[(m0 + r) * a.lda + k0 + k]) : 0.f;
            sb[k][r] = in_k && n0 + r < a.n ? e4m3_to_f32(a.b[(int64_t)(n0 + r) * a.ldb + k0 + k]) : 0.f;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kMsK; ++k) {
            float x[4], y[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) { x[i] = sa[k][ty * 4 + i]; y[i] = sb[k][tx * 4 + i]; }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) part[i][j] += x[i] * y[j];
        }
        if ((k0 + kMsK) % 128 == 0 || k0 + kMsK >= a.k) {         // end of a scale block
            const int j = k0 / 128;
            const float s_b = a.sb[(int64_t)(n0 / 128) * kb + j];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int64_t m = m0 + ty * 4 + i;
                const float s = m < a.m ? a.sa[m * kb + j] * s_b : 0.f;
#pragma unroll
                for (int q = 0; q < 4; ++q) { c[i][q] += s * part[i][q]; part[i][q] = 0.f; }
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int64_t m = m0 + ty * 4 + i;
            const int n = n0 + tx * 4 + q;
            if (m < a.m && n < a.n) ((T*)a.c)[m * a.ldc + n] = from_f32<T>(c[i][q]);
        }
}

cudaError_t matmul_simt_launch(const MatmulArgs& a, cudaStream_t stream) {
    const dim3 grid((unsigned)((a.m + kMsTile - 1) / kMsTile), (unsigned)((a.n + kMsTile - 1) / kMsTile));
    if (a.dtype == KDA_BF16) kda_matmul_fp8_simt<__nv_bfloat16><<<grid, 256, 0, stream>>>(a);
    else kda_matmul_fp8_simt<float><<<grid, 256, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace kda
