// kda_latent_decode_tc.cu -- absorbed latent attention over a paged cache on the
// tensor cores (bf16, rank 512 + 64 rotary channels).
//
// All Lq * H query rows of a sequence read the same 576-channel latents, so a
// tile of 128 cached tokens is fetched once (1152 bytes a token) and used for
// all of them.  Both products keep the tokens' side at full height and put the
// few query rows along N, where an instruction's time follows them down:
//
//     S^T [128 tokens, R rows]       = C Q^T          36 instructions (576 / 16)
//     P^T                            = exp2(S^T - ref)
//     O^T [4 x 128 channels, R rows] += C^T P^T       4 x 8 instructions (128 / 16)
//
// The second product reads the same shared-memory tile as the first, as an
// MN-major operand: nothing is transposed.  A thread owns a token; the softmax
// reference of a row moves only when some score exceeds it by 2^8, which after
// a sequence's first tile is rare, so the usual tile needs no maximum across
// threads.  Sums stay per thread until a sequence ends.
//
// Work: the tiles of all sequences, in order, are cut into equal ranges, one per
// CTA (152 at most, times the groups of R rows).  A sequence inside one range is
// finished there; pieces of others go to the workspace (unnormalised O, ref,
// sum) and a second kernel joins them in range order.
//
// Bound by HBM: at 6.78 TB/s a tile's 147 KB take an SM 6600 cycles; its
// products and softmax take about 3700.  Shared memory holds the tile, a fifth
// pair of 64-channel pieces on its way, the queries and P.
#include <math.h>

#include "kda_common.cuh"
#include "kda_paths.h"
#include "kda_sm100_ops.cuh"
#include "kda_tensor_map.h"

namespace kda {
using namespace sm100;

constexpr int kLdTile = 128;                  // tokens of a tile
constexpr int kLdRank = 512, kLdWidth = 576;
constexpr int kLdPairs = 5;                   // ring of 128-channel pairs of pieces
constexpr uint32_t kLdPiece = kLdTile * 128;  // 64 channels of a tile
constexpr int kLdThreads = 192;               // 4 softmax warps, producer, matrix instructions
constexpr float kLdUnset = -1e30f;            // reference of a row that has seen no key
constexpr float kLdSlack = 8.f;               // how far (log2) a score may exceed its reference

template <int R>
struct LdShape {
    static constexpr uint32_t kQPiece = R * 128, kQ = 9 * kQPiece;
    static constexpr uint32_t kRow = R * 2, kP = kLdTile * kRow;   // P^T: a token's R values
    static constexpr uint32_t kOffRope = kLdPairs * 2 * kLdPiece, kOffQ = kOffRope + kLdPiece;
    static constexpr uint32_t kOffP = kOffQ + kQ, kOffSmall = kOffP + kP;
    static constexpr uint32_t kSmem = kOffSmall + 1024 + (2 * 4 + 3) * R * 4 + 512;
    static constexpr uint32_t kTmem = R == 16 ? 128 : 256;         // S^T and four blocks of O^T: 5 R columns
    static constexpr uint64_t kSwz = R == 16 ? 6 : 4;
    // 16-byte piece c of token row r of P^T (32- or 64-byte swizzle)
    static __device__ __forceinline__ uint32_t p_at(int r, int c) {
        return R == 16 ? r * 32 + ((c ^ (r >> 2)) & 1) * 16 : r * 64 + ((c ^ (r >> 1)) & 3) * 16;
    }
};

struct LdArgs {
    int N, H, Lq, rows, page_size, num_pages, max_pages;
    float scale;
    const int32_t *table, *lens;
    __nv_bfloat16* out;
    float* lse;
    int32_t *status, *cta_status;
    float* parts;                              // [groups * G][2][R][kLdPart]
    int G;                                     // CTAs of a group
};
constexpr int kLdPart = kLdRank + 4;           // O, ref, sum (rows stay 16-byte aligned)

__device__ __forceinline__ int ld_len(const LdArgs& a, int n) {
    const int len = a.lens[n];
    return len < 0 || (int64_t)len > (int64_t)a.max_pages * a.page_size ? 0 : len;
}
__device__ __forceinline__ int ld_tiles(const LdArgs& a, int n) { return (ld_len(a, n) + kLdTile - 1) / kLdTile; }

// Position in the tiles of a CTA's range; the same in all lanes of a warp, which call it together.
struct LdWalk {
    int n, j, tiles, left;
    bool first;                                // first tile of a segment
    int from;                                  // its tile
    __device__ __forceinline__ bool last() const { return j + 1 == tiles || left == 1; }
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

// Sums (or maxima) over the warp's lanes of R values a lane: lane l gets those of column ld_column(l).
template <int R, bool kMax>
__device__ __forceinline__ float ld_columns(float (&v)[R], int lane) {
    auto op = [](float a, float b) { return kMax ? fmaxf(a, b) : a + b; };
    if constexpr (R == 16) {
#pragma unroll
        for (int i = 0; i < R; ++i) v[i] = op(v[i], __shfl_xor_sync(0xffffffffu, v[i], 16));
    }
#pragma unroll
    for (int o = R == 16 ? 8 : 16; o > 0; o >>= 1) {
#pragma unroll
        for (int i = 0; i < o; ++i) {
            const bool up = lane & o;
            const float keep = up ? v[i + o] : v[i], send = up ? v[i] : v[i + o];
            v[i] = op(keep, __shfl_xor_sync(0xffffffffu, send, o));
        }
    }
    return v[0];
}

template <int R>
__global__ void __launch_bounds__(kLdThreads, 1)
kda_latent_decode_tc(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_c,
                     const LdArgs a) {
    using S = LdShape<R>;
    extern __shared__ uint8_t raw[];
    const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u;
    uint8_t* mem = raw + (base - smem_u32(raw));
    float* ref = (float*)(mem + S::kOffSmall);         // [R] softmax references (log2)
    float* fac = ref + R;                              // [R] factors of a moved reference
    int* query = (int*)(fac + R);                      // [R] query a row belongs to
    float* across = (float*)(query + R);               // [4][R] one value a warp and row
    float* sums = across + 4 * R;                      // [4][R]
    uint64_t* bars = (uint64_t*)(sums + 4 * R);
    uint64_t *full = bars, *empty = full + kLdPairs, *rope_full = empty + kLdPairs, *rope_empty = rope_full + 1,
             *q_full = rope_empty + 1, *q_empty = q_full + 1, *s_full = q_empty + 1, *p_full = s_full + 1,
             *o_full = p_full + 1;
    uint32_t* tmem_at = (uint32_t*)(o_full + 1);
    int* range = (int*)(tmem_at + 1);                  // first sequence, its first tile, tiles
    int* fault = range + 3;

    const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
    const int group = blockIdx.x, cta = blockIdx.y;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (threadIdx.x == 0) {
        for (uint64_t* b = bars; b <= o_full; ++b) mbar_init(b, 1);
        mbar_init(p_full, 4);
        fence_mbar_init();
    }
    if (warp == 0) { tmem_alloc(tmem_at, S::kTmem); tmem_relinquish(); }
    if (warp == 4) {
        // this CTA's range of the tiles of all sequences
        int64_t total = 0;
        bool bad = false;
        for (int b = 0; b < a.N; b += 32) {
            const int n = b + lane;
            if (n < a.N) { const int l = a.lens[n]; bad |= l < 0 || (int64_t)l > (int64_t)a.max_pages * a.page_size; }
            int t = n < a.N ? ld_tiles(a, n) : 0;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
            total += t;
        }
        bad = __any_sync(0xffffffffu, bad);
        const int64_t parts = min64(a.G, total);       // no empty range between two that hold tiles
        const int64_t t0 = cta < parts ? total * cta / parts : 0, t1 = cta < parts ? total * (cta + 1) / parts : 0;
        int64_t before = 0;
        int n0 = 0, j0 = 0;
        if (t1 > t0) {
            for (int b = 0; b < a.N; b += 32) {
                const int n = b + lane;
                const int t = n < a.N ? ld_tiles(a, n) : 0;
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
        if (lane == 0) {
            range[0] = n0; range[1] = j0; range[2] = (int)(t1 - t0);
            *fault = bad ? KDA_ERR_BAD_SEQLENS : KDA_OK;
        }
    }
    if (threadIdx.x < R) {
        ref[threadIdx.x] = kLdUnset;
        query[threadIdx.x] = min((group * R + (int)threadIdx.x) / a.H, a.Lq - 1);
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_at, 0);
    LdWalk w;
    w.start(a, range[0], range[1], range[2]);

    if (warp == 4) {                                                   // ---------------- producer
        const int box = min(a.page_size, kLdTile), boxes = kLdTile / box;
        uint32_t unit = 0, tile = 0, seg = 0;
        bool ok = true, bad_page = false;
        for (; w.left > 0 && ok; w.next(a), ++tile) {
            if (w.first) {
                if (seg > 0) ok = mbar_wait_warp(q_empty, (seg - 1) & 1);
                if (!ok) break;
                if (lane == 0) {
                    mbar_arrive_expect_tx(q_full, S::kQ);
                    for (int c = 0; c < 9; ++c)
                        tma_load_3d_at(base + S::kOffQ + c * S::kQPiece, &map_q, c * 64, group * R, w.n, smem_u32(q_full));
                }
                ++seg;
            }
            // a lane for each box of tokens: its page and row; pages behind the length, and bad ones, read as zeros
            int page = a.num_pages, row = 0;
            if (lane < boxes) {
                const int t = w.j * kLdTile + lane * box;
                if (t < ld_len(a, w.n)) {
                    const int p = a.table[(int64_t)w.n * a.max_pages + t / a.page_size];
                    if (p < 0 || p >= a.num_pages) bad_page = true;
                    else { page = p; row = t % a.page_size; }
                }
            }
            if (tile > 0 && !(ok = mbar_wait_warp(rope_empty, (tile - 1) & 1))) break;
            if (lane == 0) mbar_arrive_expect_tx(rope_full, kLdPiece);
            __syncwarp();
            if (lane < boxes)
                tma_load_3d_at(base + S::kOffRope + lane * box * 128, &map_c, kLdRank, row, page, smem_u32(rope_full));
            for (int p = 0; p < 4; ++p, ++unit) {
                const uint32_t s = unit % kLdPairs, ph = (unit / kLdPairs) & 1;
                if (unit >= kLdPairs && !(ok = mbar_wait_warp(&empty[s], ph ^ 1))) break;
                if (lane == 0) mbar_arrive_expect_tx(&full[s], 2 * kLdPiece);
                __syncwarp();
                if (lane < boxes) {
                    const uint32_t at = base + s * 2 * kLdPiece + lane * box * 128;
                    tma_load_3d_at(at, &map_c, p * 128, row, page, smem_u32(&full[s]));
                    tma_load_3d_at(at + kLdPiece, &map_c, p * 128 + 64, row, page, smem_u32(&full[s]));
                }
            }
        }
        if (bad_page) atomicMax(fault, KDA_ERR_BAD_PAGE);
        if (!ok) { atomicMax(fault, KDA_ERR_TIMEOUT); drain_copies(); }
    } else if (warp == 5) {                                            // ---------------- matrix instructions
        const uint32_t idesc_s = idesc_bf16(128, R), idesc_o = idesc_bf16(128, R, 1, 1);
        uint32_t unit = 0, tile = 0, seg = 0;
        bool ok = true;
        for (; w.left > 0 && ok; w.next(a), ++tile) {
            if (w.first) { ok = mbar_wait_warp(q_full, seg & 1); ++seg; }
            if (ok) ok = mbar_wait_warp(rope_full, tile & 1);
            if (!ok) break;
            tc_fence_after_sync();
            const uint64_t dq = sdesc_k_sw128(base + S::kOffQ);
            if (elect_one()) {
                const uint64_t da = sdesc_k_sw128(base + S::kOffRope);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    mma_bf16_ss(tmem, da + 2 * k, dq + 8 * (S::kQPiece / 16) + 2 * k, idesc_s, k > 0);
            }
            __syncwarp();
            for (int p = 0; p < 4 && ok; ++p) {
                const uint32_t u = unit + p, s = u % kLdPairs, ph = (u / kLdPairs) & 1;
                if (!(ok = mbar_wait_warp(&full[s], ph))) break;
                tc_fence_after_sync();
                const uint64_t da = sdesc_k_sw128(base + s * 2 * kLdPiece);
                const uint64_t db = dq + 2 * p * (S::kQPiece / 16);
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        mma_bf16_ss(tmem, da + (k / 4) * (kLdPiece / 16) + 2 * (k % 4),
                                    db + (k / 4) * (S::kQPiece / 16) + 2 * (k % 4), idesc_s, 1);
                    if (p == 3) {
                        mma_commit(s_full);
                        mma_commit(rope_empty);
                        if (w.last()) mma_commit(q_empty);
                    }
                }
                __syncwarp();
            }
            if (ok) ok = mbar_wait_warp(p_full, tile & 1);
            if (!ok) break;
            tc_fence_after_sync();
            const uint64_t dp = sdesc(base + S::kOffP, 16, 8 * S::kRow, S::kSwz);
            for (int p = 0; p < 4; ++p, ++unit) {
                const uint32_t s = unit % kLdPairs;
                // A: 128 channels = two pieces of 64, MN-major; 16 tokens a step
                const uint64_t da = sdesc(base + s * 2 * kLdPiece, kLdPiece, 1024, 2);
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        mma_bf16_ss(tmem + (1 + p) * R, da + k * (2048 / 16), dp + k * (16 * S::kRow / 16), idesc_o,
                                    !w.first || k > 0);
                    mma_commit(&empty[s]);
                    if (p == 3 && w.last()) mma_commit(o_full);
                }
                __syncwarp();
            }
        }
        if (!ok) atomicMax(fault, KDA_ERR_TIMEOUT);
    } else {                                                           // ---------------- softmax
        const uint32_t lanes = tmem_addr(tmem, 32 * warp, 0);
        const float sc = a.scale * 1.4426950408889634f;
        const int row0 = group * R, live = min(R, a.rows - row0);
        float l[R];
#pragma unroll
        for (int c = 0; c < R; ++c) l[c] = 0.f;
        uint32_t tile = 0, seg = 0;
        bool ok = true;
        for (; w.left > 0; w.next(a), ++tile) {
            ok = bar_and(128, mbar_wait_spin(s_full, tile & 1));
            if (!ok) break;
            tc_fence_after_sync();
            const int len = ld_len(a, w.n);
            const int token = w.j * kLdTile + (int)threadIdx.x;
            float x[R];
            if constexpr (R == 16) tmem_ld16(lanes, x);
            else tmem_ld32(lanes, x);
            tmem_wait_ld();
            tmem_ready(x);
#pragma unroll
            for (int c = 0; c < R; ++c) x[c] *= sc;
            if ((w.j + 1) * kLdTile > len - a.Lq + 1) {                // some row does not see some token
#pragma unroll
                for (int c = 0; c < R; ++c)
                    if (token > len - a.Lq + query[c]) x[c] = -INFINITY;
            }
            bool over = false;
#pragma unroll
            for (int c = 0; c < R; c += 4) {
                const float4 m = *(const float4*)(ref + c);
                over |= x[c] > m.x + kLdSlack || x[c + 1] > m.y + kLdSlack || x[c + 2] > m.z + kLdSlack ||
                        x[c + 3] > m.w + kLdSlack;
            }
            if (!bar_and(128, !over)) {                                // move the references to the maxima
                float v[R];
#pragma unroll
                for (int c = 0; c < R; ++c) v[c] = x[c];
                const float top = ld_columns<R, true>(v, lane);
                if (lane < R) across[warp * R + lane] = top;
                asm volatile("bar.sync 2, 128;" ::: "memory");
                if (threadIdx.x < R) {
                    const int c = threadIdx.x;
                    const float old = ref[c];
                    const float now = fmaxf(old, fmaxf(fmaxf(across[c], across[R + c]),
                                                       fmaxf(across[2 * R + c], across[3 * R + c])));
                    ref[c] = now;
                    fac[c] = ex2(old - now);
                }
                asm volatile("bar.sync 2, 128;" ::: "memory");
#pragma unroll
                for (int c = 0; c < R; ++c) l[c] *= fac[c];
                if (!w.first) {                                        // O^T: the products before S^T are complete
                    for (int p = 1; p <= 4; ++p) {
                        for (int h = 0; h < R; h += 16) {
                            float o[16];
                            tmem_ld16(lanes + p * R + h, o);
                            tmem_wait_ld();
                            tmem_ready(o);
#pragma unroll
                            for (int c = 0; c < 16; ++c) o[c] *= fac[h + c];
                            tmem_st16(lanes + p * R + h, o);
                        }
                    }
                    tmem_wait_st();
                }
            }
#pragma unroll
            for (int c = 0; c < R; c += 8) {
                const float4 m0 = *(const float4*)(ref + c), m1 = *(const float4*)(ref + c + 4);
                const float m[8] = {m0.x, m0.y, m0.z, m0.w, m1.x, m1.y, m1.z, m1.w};
                uint32_t b[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float p0 = ex2(x[c + 2 * i] - m[2 * i]), p1 = ex2(x[c + 2 * i + 1] - m[2 * i + 1]);
                    l[c + 2 * i] += p0;
                    l[c + 2 * i + 1] += p1;
                    const __nv_bfloat162 h = __floats2bfloat162_rn(p0, p1);    // the product's operand: 8 bits
                    b[i] = *(const uint32_t*)&h;
                }
                *(uint4*)(mem + S::kOffP + S::p_at(threadIdx.x, c / 8)) = make_uint4(b[0], b[1], b[2], b[3]);
            }
            if (token >= len) {                                        // weight 0 times what lies behind the length: make it 0
                for (int p = 0; p < 4; ++p) {
                    uint8_t* at = mem + (tile * 4 + p) % kLdPairs * 2 * kLdPiece + threadIdx.x * 128;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        *(uint4*)(at + 16 * i) = make_uint4(0, 0, 0, 0);
                        *(uint4*)(at + kLdPiece + 16 * i) = make_uint4(0, 0, 0, 0);
                    }
                }
            }
            fence_proxy_async_smem();
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(p_full);
            if (!w.last()) continue;

            // end of a segment: sums across the tokens' threads, then O^T out
            const float part = ld_columns<R, false>(l, lane);
            if (lane < R) sums[warp * R + lane] = part;
            ok = bar_and(128, mbar_wait_spin(o_full, seg & 1));
            ++seg;
            if (!ok) break;
            tc_fence_after_sync();
            const bool whole = w.from == 0 && w.j + 1 == w.tiles;
            float* dst = a.parts + ((size_t)(cta * gridDim.x + group) * 2 + (w.from == 0)) * R * kLdPart;
            if (threadIdx.x < R) {
                const int c = threadIdx.x;
                const float total = (sums[c] + sums[R + c]) + (sums[2 * R + c] + sums[3 * R + c]);
                if (whole) {
                    fac[c] = total > 0.f ? 1.f / total : (total == 0.f ? 0.f : total);
                    if (c < live && a.lse) a.lse[(size_t)w.n * a.rows + row0 + c] =
                        total == 0.f ? -INFINITY : (ref[c] + log2f(total)) * 0.6931471805599453f;
                } else {
                    dst[c * kLdPart + kLdRank] = ref[c];
                    dst[c * kLdPart + kLdRank + 1] = total;
                }
            }
            asm volatile("bar.sync 2, 128;" ::: "memory");
            for (int p = 0; p < 4; ++p) {
                const int ch = p * 128 + threadIdx.x;
#pragma unroll
                for (int h = 0; h < R; h += 16) {
                    float o[16];
                    tmem_ld16(lanes + (1 + p) * R + h, o);
                    tmem_wait_ld();
                    tmem_ready(o);
                    if (whole) {
                        __nv_bfloat16* to = a.out + ((size_t)w.n * a.rows + row0 + h) * kLdRank + ch;
#pragma unroll
                        for (int c = 0; c < 16; ++c)
                            if (h + c < live) to[(size_t)c * kLdRank] = __float2bfloat16_rn(o[c] * fac[h + c]);
                    } else {
#pragma unroll
                        for (int c = 0; c < 16; ++c)
                            if (h + c < live) dst[(h + c) * kLdPart + ch] = o[c];
                    }
                }
            }
            asm volatile("bar.sync 2, 128;" ::: "memory");
            if (threadIdx.x < R) ref[threadIdx.x] = kLdUnset;
#pragma unroll
            for (int c = 0; c < R; ++c) l[c] = 0.f;
            asm volatile("bar.sync 2, 128;" ::: "memory");
        }
        if (!ok) atomicMax(fault, KDA_ERR_TIMEOUT);
    }
    tc_fence_before_sync();
    __syncthreads();
    if (warp == 0) tmem_dealloc(tmem, S::kTmem);
    if (threadIdx.x == 0) a.cta_status[cta * gridDim.x + group] = *fault;
}

// Joins the pieces of sequences that several CTAs shared, gives sequences
// without tiles their zeros, and collects the CTAs' status.  A warp a row.
template <int R>
__global__ void __launch_bounds__(256)
kda_latent_decode_join(const LdArgs a, const int groups) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    __shared__ int64_t s_before[8], s_total[8];
    const int n = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (n == 0 && blockIdx.y == 0) {
        int st = KDA_OK;
        for (int i = threadIdx.x; i < a.G * groups; i += 256) st = max(st, a.cta_status[i]);
        st = __syncthreads_or(st == KDA_ERR_BAD_PAGE) ? KDA_ERR_BAD_PAGE
             : __syncthreads_or(st == KDA_ERR_BAD_SEQLENS) ? KDA_ERR_BAD_SEQLENS
             : __syncthreads_or(st == KDA_ERR_TIMEOUT) ? KDA_ERR_TIMEOUT : KDA_OK;
        if (threadIdx.x == 0) *a.status = st;
    }
    int64_t before = 0, total = 0;
    for (int i = threadIdx.x; i < a.N; i += 256) {
        const int t = ld_tiles(a, i);
        total += t;
        if (i < n) before += t;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        before += __shfl_xor_sync(0xffffffffu, before, o);
        total += __shfl_xor_sync(0xffffffffu, total, o);
    }
    if (lane == 0) { s_before[warp] = before; s_total[warp] = total; }
    __syncthreads();
    before = total = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) { before += s_before[i]; total += s_total[i]; }
    const int row = blockIdx.y * 8 + warp;
    if (row >= a.rows) return;
    const int tiles = ld_tiles(a, n);
    __nv_bfloat16* to = a.out + ((size_t)n * a.rows + row) * kLdRank;
    float o[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) o[i] = 0.f;
    float lse = -INFINITY;
    if (tiles > 0) {
        const int64_t parts = min64(a.G, total);
        const int cf = (int)(((before + 1) * parts - 1) / total), cl = (int)(((before + tiles) * parts - 1) / total);
        if (cf == cl) return;                          // finished by its CTA
        const int group = row / R, c = row % R;
        auto piece = [&](int i) {
            return a.parts + (((size_t)(i * groups + group) * 2 + (i == cf)) * R + c) * kLdPart;
        };
        float top = kLdUnset, sum = 0.f;
        for (int i = cf + lane; i <= cl; i += 32) top = fmaxf(top, piece(i)[kLdRank]);
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, s));
        for (int i = cf; i <= cl; ++i) {
            const float* p = piece(i);
            const float wgt = ex2(p[kLdRank] - top);
            sum += wgt * p[kLdRank + 1];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float4 v = *(const float4*)(p + q * 128 + lane * 4);
                o[4 * q] += wgt * v.x; o[4 * q + 1] += wgt * v.y; o[4 * q + 2] += wgt * v.z; o[4 * q + 3] += wgt * v.w;
            }
        }
        const float inv = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);
#pragma unroll
        for (int i = 0; i < 16; ++i) o[i] *= inv;
        if (sum != 0.f) lse = (top + log2f(sum)) * 0.6931471805599453f;
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const __nv_bfloat162 x = __floats2bfloat162_rn(o[4 * q], o[4 * q + 1]), y = __floats2bfloat162_rn(o[4 * q + 2], o[4 * q + 3]);
        *(uint2*)(to + q * 128 + lane * 4) = make_uint2(*(const uint32_t*)&x, *(const uint32_t*)&y);
    }
    if (lane == 0 && a.lse) a.lse[(size_t)n * a.rows + row] = lse;
}

// ------------------------------------------------------------------- host
struct LdPlan { int R, groups, G; size_t bytes; };

// CTAs and workspace of a call, from its sizes alone.
static LdPlan ld_plan(int N, int Lq, int H, int page_size, int max_pages) {
    LdPlan p;
    const int64_t rows = (int64_t)Lq * H;
    p.R = rows <= 16 ? 16 : 32;
    p.groups = (int)((rows + p.R - 1) / p.R);
    const int64_t tiles = (int64_t)N * (((int64_t)max_pages * page_size + kLdTile - 1) / kLdTile);
    int64_t g = 152 / p.groups;
    g = g < 1 ? 1 : g;
    p.G = (int)(g < tiles ? g : tiles);
    const size_t status = ((size_t)p.groups * p.G * 4 + 255) / 256 * 256;
    p.bytes = status + (size_t)p.groups * p.G * 2 * p.R * kLdPart * 4;
    return p;
}

bool latent_decode_tc_takes(int dtype, int dk, int dr, int H, int Lq, int page_size) {
    return dtype == KDA_BF16 && dk == kLdRank && dr == kLdWidth - kLdRank && page_size >= 8 &&
           (page_size & (page_size - 1)) == 0 && (int64_t)Lq * H <= 32 * 1024;
}
size_t latent_decode_tc_bytes(int N, int Lq, int H, int page_size, int max_pages) {
    return N > 0 ? ld_plan(N, Lq, H, page_size, max_pages).bytes : 0;
}
// What the tensor maps need of the call's tensors.
bool latent_decode_tc_aligned(const LatentDecodeArgs& d) {
    const bool flat = d.Lq == 1 || d.H == 1 || d.q_ts == (int64_t)d.H * d.q_hs;   // (query, head) is one strided dimension
    return flat && (((uintptr_t)d.q | (uintptr_t)d.cache | (uintptr_t)d.out) & 15) == 0 && d.q_ts % 8 == 0 &&
           (d.H == 1 || (d.q_hs % 8 == 0 && d.q_hs > 0)) && d.q_ts > 0 && d.page_stride % 8 == 0 && d.num_pages > 0 &&
           d.page_stride < (1ll << 38) && d.q_ts < (1ll << 30);
}

template <int R>
static cudaError_t ld_launch(const LatentDecodeArgs& d, const LdPlan& p, cudaStream_t stream) {
    using S = LdShape<R>;
    static bool ready = false;
    if (!ready) {
        cudaError_t e = cudaFuncSetAttribute(kda_latent_decode_tc<R>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)S::kSmem);
        if (e != cudaSuccess) return e;
        ready = true;
    }
    LdArgs a;
    a.N = d.N; a.H = d.H; a.Lq = d.Lq; a.rows = d.Lq * d.H; a.page_size = d.page_size; a.num_pages = d.num_pages;
    a.max_pages = d.max_pages; a.scale = d.scale; a.table = d.table; a.lens = d.lens; a.out = (__nv_bfloat16*)d.out;
    a.lse = d.lse; a.status = d.status; a.cta_status = (int32_t*)d.scratch; a.G = p.G;
    a.parts = (float*)((char*)d.scratch + ((size_t)p.groups * p.G * 4 + 255) / 256 * 256);
    CUtensorMap mq, mc;
    const uint64_t qd[3] = {kLdWidth, (uint64_t)a.rows, (uint64_t)d.N};
    const uint64_t qs[2] = {(uint64_t)(d.H == 1 ? d.q_ts : d.q_hs) * 2, (uint64_t)d.q_ts * d.Lq * 2};
    const uint32_t qb[3] = {64, R, 1};
    const uint64_t cd[3] = {kLdWidth, (uint64_t)d.page_size, (uint64_t)d.num_pages};
    const uint64_t cs[2] = {kLdWidth * 2, (uint64_t)d.page_stride * 2};
    const uint32_t cb[3] = {64, (uint32_t)(d.page_size < kLdTile ? d.page_size : kLdTile), 1};
    if (!make_map(&mq, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, d.q, qd, qs, qb) ||
        !make_map(&mc, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, d.cache, cd, cs, cb)) return cudaErrorInvalidValue;
    kda_latent_decode_tc<R><<<dim3(p.groups, p.G), kLdThreads, S::kSmem, stream>>>(mq, mc, a);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(d.N, (a.rows + 7) / 8); cfg.blockDim = dim3(256); cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at; cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kda_latent_decode_join<R>, a, p.groups);
}

cudaError_t latent_decode_tc_launch(const LatentDecodeArgs& d, cudaStream_t stream) {
    const LdPlan p = ld_plan(d.N, d.Lq, d.H, d.page_size, d.max_pages);
    return p.R == 16 ? ld_launch<16>(d, p, stream) : ld_launch<32>(d, p, stream);
}

}  // namespace kda
