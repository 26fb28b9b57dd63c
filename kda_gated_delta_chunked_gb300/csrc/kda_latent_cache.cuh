// kda_latent_cache.cuh -- layout of the quantised cache of latents (kda.h): in a
// page, rows of rank codes and d_rope bf16 channels, then a scale byte a token.
#pragma once

#include <stdint.h>

namespace kda {

constexpr int kScaleBias = 127;                 // a token's byte is e + 127, also the exponent bits of 2^e
constexpr int kScaleLow = -100, kScaleHigh = 120;

__host__ __device__ constexpr int latent_row_bytes(int rank, int d_rope) { return rank + 2 * d_rope; }
__host__ __device__ constexpr int64_t latent_page_bytes(int page_size, int rank, int d_rope) {
    return ((int64_t)page_size * (latent_row_bytes(rank, d_rope) + 1) + 127) / 128 * 128;
}

// The smallest e with x <= 448 2^e, within kScaleLow .. kScaleHigh, of a finite x >= 0 given by its bits:
// x = 1.f 2^(E - 127), 448 = 1.75 2^8.
__device__ __forceinline__ int latent_exponent(uint32_t bits) {
    const int e = (int)(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u);
    return min(max(e, kScaleLow), kScaleHigh);
}

}  // namespace kda
