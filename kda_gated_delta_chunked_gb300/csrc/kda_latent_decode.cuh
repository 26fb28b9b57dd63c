// kda_latent_decode.cuh -- what the tensor-core kernels of latent_decode share: how
// the tiles of all sequences are cut into the CTAs' ranges and walked, and what the
// join of their pieces reads (kda_latent_decode_tc.cu).
#pragma once

#include "kda_common.cuh"
#include "kda_paths.h"
#include "kda_sm100_ops.cuh"

namespace kda {
using namespace sm100;

constexpr int kLdTile = 128;                  // tokens of a tile
constexpr int kLdRank = 512, kLdWidth = 576;
constexpr float kLdUnset = -1e30f;            // reference of a row that has seen no key
constexpr int kLdLate = 1, kLdBadLen = 2, kLdBadPage = 4;   // bits of a CTA's status

struct LdArgs {
    int N, H, Lq, rows, page_size, num_pages, max_pages;
    uint32_t drop;                             // barriers, a bit each, that miss an arrival
    float scale;
    const int32_t *table, *lens;
    __nv_bfloat16* out;
    float* lse;
    int32_t *status, *cta_status;
    float* parts;                              // [groups * G][2][R][kLdPart]
    int64_t* before;                           // [N + 1] tiles ahead of a sequence (where it has tiles); all tiles
    int G;                                     // CTAs of a group
};
constexpr int kLdPart = kLdRank + 4;           // O, ref, sum (rows stay 16-byte aligned)

__device__ __forceinline__ int ld_len(const LdArgs& a, int n) {
    const int len = a.lens[n];
    return len < 0 || (int64_t)len > (int64_t)a.max_pages * a.page_size ? 0 : len;
}
__device__ __forceinline__ int ld_tiles_of(int len) { return (int)(((uint32_t)len + kLdTile - 1) / kLdTile); }   // (up to 2^31 - 1)
__device__ __forceinline__ int ld_tiles(const LdArgs& a, int n) { return ld_tiles_of(ld_len(a, n)); }

// Position in the tiles of a CTA's range; the same in all lanes of a warp, which call it together.
struct LdWalk {
    int n, j, tiles, left;
    bool first;                                // first tile of a segment
    int from;                                  // its tile
    __device__ __forceinline__ bool last() const { return j + 1 == tiles || left == 1; }
    __device__ __forceinline__ int end() const { return j * kLdTile + (kLdTile - 1); }   // its last token (one more may be 2^31)
    __device__ __forceinline__ void settle(const LdArgs& a) {      // on to the next sequence that has tiles
        while (left > 0 && j >= tiles) { ++n; j = 0; tiles = uniform(ld_tiles(a, n)); }
    }
    __device__ __forceinline__ void start(const LdArgs& a, int n0, int j0, int count) {
        n = uniform(n0); j = uniform(j0); left = uniform(count); first = true; from = j;
        tiles = left > 0 ? uniform(ld_tiles(a, n)) : 0;
    }
    __device__ __forceinline__ void next(const LdArgs& a) {
        first = last();
        ++j; --left;
        settle(a);
        if (first) from = j;
    }
};

// Sums (or maxima) over the warp's lanes of R values a lane, to `to`[0 .. R).
template <int R, bool kMax>
__device__ __forceinline__ void ld_columns(const float (&x)[R], float* to, int lane) {
    auto op = [](float a, float b) { return kMax ? fmaxf(a, b) : a + b; };
    constexpr int W = R < 32 ? R : 32;
#pragma unroll
    for (int h = 0; h < R; h += W) {
        float v[W];
#pragma unroll
        for (int i = 0; i < W; ++i) {
            v[i] = x[h + i];
#pragma unroll
            for (int o = 16; o >= W; o >>= 1) v[i] = op(v[i], __shfl_xor_sync(0xffffffffu, v[i], o));
        }
#pragma unroll
        for (int o = W / 2; o > 0; o >>= 1) {
#pragma unroll
            for (int i = 0; i < o; ++i) {
                const bool up = lane & o;
                const float keep = up ? v[i + o] : v[i], send = up ? v[i] : v[i + o];
                v[i] = op(keep, __shfl_xor_sync(0xffffffffu, send, o));
            }
        }
        if (lane < W) to[h + lane] = v[0];                         // lane l has come to hold column l
    }
}

// A CTA's range of the tiles of all sequences, by one warp; `len`: the length of sequence `lane`, which the caller fetches
// ahead.
struct LdCut { int n, j, count; int64_t at, total; bool bad; };     // first sequence, its first tile, tiles; index of the first
__device__ __forceinline__ LdCut ld_cut(const LdArgs& a, int cta, int lane, int len) {
    const int64_t cap = (int64_t)a.max_pages * a.page_size;
    int64_t total = 0;
    bool bad = false;
    int first = 0;                                                 // tiles of sequence `lane`
    for (int b = 0; b < a.N; b += 32) {
        if (b > 0) len = b + lane < a.N ? a.lens[b + lane] : 0;
        bad |= len < 0 || len > cap;
        const int t = len < 0 || len > cap ? 0 : ld_tiles_of(len);
        if (b == 0) first = t;
        total += __reduce_add_sync(0xffffffffu, t);
    }
    bad = __any_sync(0xffffffffu, bad);
    const int64_t parts = min64(a.G, total);       // no empty range between two that hold tiles
    int64_t t0 = 0, t1 = 0;
    if (cta < parts) {
        if (total < (1 << 20)) {
            t0 = (uint32_t)total * cta / (uint32_t)parts;
            t1 = (uint32_t)total * (cta + 1) / (uint32_t)parts;
        } else {
            t0 = total * cta / parts;
            t1 = total * (cta + 1) / parts;
        }
    }
    int64_t before = 0;
    int n0 = 0, j0 = 0;
    if (t1 > t0) {
        for (int b = 0; b < a.N; b += 32) {
            const int n = b + lane;
            const int t = b == 0 ? first : n < a.N ? ld_tiles(a, n) : 0;
            int x = t;                                             // inclusive scan
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, x, o);
                if (lane >= o) x += y;
            }
            const uint32_t hit = __ballot_sync(0xffffffffu, before + x > t0);
            if (hit) {
                const int l = __ffs(hit) - 1;
                n0 = b + l;
                j0 = (int)(t0 - before - (__shfl_sync(0xffffffffu, x, l) - __shfl_sync(0xffffffffu, t, l)));
                break;
            }
            before += __shfl_sync(0xffffffffu, x, 31);
        }
    }
    return {n0, j0, (int)(t1 - t0), t0, total, bad};
}

// Joins the pieces (kda_latent_decode_tc.cu).
cudaError_t latent_decode_join_launch(const LdArgs& a, int R, int groups, cudaStream_t stream);

struct LdPlan { int R, groups, G; size_t before, parts, bytes; };   // offsets behind the CTAs' status

// CTAs and workspace of a call with groups of R rows, from its sizes alone.
inline LdPlan ld_plan(int N, int Lq, int H, int page_size, int max_pages, int R) {
    LdPlan p;
    const int64_t rows = (int64_t)Lq * H;
    p.R = R;
    p.groups = (int)((rows + p.R - 1) / p.R);
    const int64_t tiles = (int64_t)N * (((int64_t)max_pages * page_size + kLdTile - 1) / kLdTile);
    int64_t g = 152 / p.groups;
    g = g < 1 ? 1 : g;
    p.G = (int)(g < tiles ? g : tiles);
    p.before = ((size_t)p.groups * p.G * 4 + 255) / 256 * 256;
    p.parts = p.before + ((size_t)(N + 1) * 8 + 255) / 256 * 256;
    p.bytes = p.parts + (size_t)p.groups * p.G * 2 * p.R * kLdPart * 4;
    return p;
}

}  // namespace kda
