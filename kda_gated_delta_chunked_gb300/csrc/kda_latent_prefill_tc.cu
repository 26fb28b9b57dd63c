// kda_latent_prefill_tc.cu -- expanded latent attention over packed prompts on
// the tensor cores (bf16; keys 128 + 64 shared rotary channels, values 128).
//
//     S = Q K^T (192 channels),  P = exp2(scale' S - ref),  O += P V
//
// A CTA owns 256 query rows of one head as two tiles of 128 and walks the key
// tiles of 128 that they see.  While the softmax of one tile runs on its own
// warpgroup (a thread a row), the tensor core works on the other:
//
//     PV_j(0)  S_{j+1}(0)  PV_j(1)  S_{j+1}(1)  PV_{j+1}(0) ...
//
// TMEM holds S0 S1 O0 O1 (4 x 128 columns); P overwrites its S as bf16 and is
// read from there, so only V passes through shared memory for the second
// product.  The reference of a row moves only when a score exceeds it by 2^8
// (then the row of O is rescaled), which is rare after the first tiles.
// K (three pieces of 64 channels) and V (two of 64 keys) share one ring of eight
// 16 KB pieces, in the order of their use; with the queries' 96 KB that fills
// shared memory.
//
// Few rows (a chunk of a long prompt, few heads) leave SMs idle and the longest
// row alone decides: then the 2 or 4 CTAs of a cluster share the rows' key tiles,
// and their parts of O are joined, in rank order, in distributed shared memory
// (256 rows of 8192 keys, 16 heads: 123 -> 48 us with 4).
//
// A key tile of both row tiles is 2 x (12 + 8) instructions of 64 cycles, 2560 of
// the tensor pipe; it takes 3400, the turn of product, commit, softmax (about
// 1000 cycles of its warpgroup) and wait.  8192 tokens, 32 heads, causal: 445 us,
// 1.54 PFLOP/s.  Short sequences pay about 9 us for a CTA's start, queries and
// end, one CTA to an SM.
#include <math.h>

#include "kda_common.cuh"
#include "kda_paths.h"
#include "kda_sm100_ops.cuh"
#include "kda_tensor_map.h"

namespace kda {
using namespace sm100;

constexpr int kLpRows = 256;                  // query rows of a CTA
constexpr int kLpKeys = 128;
constexpr uint32_t kLpPiece = 16384;
constexpr int kLpSlots = 8;
constexpr uint32_t kLpOffRing = 6 * kLpPiece, kLpOffSmall = kLpOffRing + kLpSlots * kLpPiece;
constexpr uint32_t kLpRow = 512;              // bytes of an fp32 row of O, where a cluster joins
constexpr int kLpSplits = 4;                  // CTAs that share the keys of a tile of rows at most
constexpr uint32_t kLpOffLse = kLpOffSmall + 256, kLpSmem = kLpOffLse + kLpRows * 4 + 1024;
constexpr int kLpThreads = 384;
constexpr int kLpHeads = 8;                   // heads of a group
constexpr float kLpUnset = -1e30f, kLpSlack = 8.f;

struct LpArgs {
    int N, H, causal, blocks, splits;          // blocks: tiles of rows of a head at most; splits: CTAs that share them
    float scale;
    int64_t tq, tk;
    const int32_t *cu_q, *cu_k;
    __nv_bfloat16* out;
    float* lse;
    int32_t* status;
};

template <bool SHARED>
__global__ void __launch_bounds__(kLpThreads, 1)
kda_latent_prefill_tc(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                      const __grid_constant__ CUtensorMap map_r, const __grid_constant__ CUtensorMap map_v,
                      const LpArgs a) {
    extern __shared__ uint8_t raw[];
    const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u;
    uint8_t* mem = raw + (base - smem_u32(raw));
    uint64_t* q_full = (uint64_t*)(mem + kLpOffSmall);
    uint64_t *kv_full = q_full + 1, *kv_empty = kv_full + 4;   // [2 steps][K, V]
    uint64_t *s_full = kv_empty + 4, *p_full = s_full + 2, *o_full = p_full + 2;
    uint64_t* rows_full = o_full + 2;
    uint32_t* tmem_at = (uint32_t*)(rows_full + 1);
    int* where = (int*)(tmem_at + 1);          // sequence, its tile of rows (-1: none)

    const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
    // Which rows: in groups of heads (whose keys and values then stay in L2), a sequence's last tile, which sees most
    // keys, first, so that what runs last is short (8192 tokens, 32 heads: 488 us a head at a time, 445 in groups).
    const int splits = SHARED ? a.splits : 1, rank = SHARED ? (int)blockIdx.x % splits : 0;   // of the rows' keys
    const int per = a.blocks * kLpHeads, index = (int)blockIdx.x / splits, grp = index / per;
    const int heads = min(kLpHeads, a.H - grp * kLpHeads), in_grp = index - grp * per;
    const int head = grp * kLpHeads + in_grp % heads, block = in_grp / heads;
    if (threadIdx.x == 32) { prefetch_map(&map_q); prefetch_map(&map_k); prefetch_map(&map_r); prefetch_map(&map_v); }
    if (warp == 0) {
        int n = 0, tile = -1;
        if (a.cu_q == nullptr) {
            const int64_t t = (a.tq + kLpRows - 1) / kLpRows - 1 - block;
            tile = t >= 0 ? (int)t : -1;
        } else {
            int before = 0;
            for (int b = 0; b < a.N; b += 32) {
                const int i = b + lane;
                const int len = i < a.N ? a.cu_q[i + 1] - a.cu_q[i] : 0;
                const int t = len > 0 ? (len + kLpRows - 1) / kLpRows : 0;
                int x = t;                                             // inclusive scan
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int y = __shfl_up_sync(0xffffffffu, x, o);
                    if (lane >= o) x += y;
                }
                const uint32_t hit = __ballot_sync(0xffffffffu, before + x > block);
                if (hit) {
                    const int l = __ffs(hit) - 1;
                    n = b + l;
                    tile = before + __shfl_sync(0xffffffffu, x, l) - 1 - block;
                    break;
                }
                before += __shfl_sync(0xffffffffu, x, 31);
            }
        }
        if (lane == 0) { where[0] = n; where[1] = tile; }
        tmem_alloc(tmem_at, 512);
        tmem_relinquish();
    }
    if (threadIdx.x == 0) {
        mbar_init(q_full, 1);
        mbar_init(rows_full, 1);
        for (int i = 0; i < 4; ++i) { mbar_init(&kv_full[i], 1); mbar_init(&kv_empty[i], 1); }
        for (int i = 0; i < 2; ++i) { mbar_init(&s_full[i], 1); mbar_init(&p_full[i], 4); mbar_init(&o_full[i], 1); }
        fence_mbar_init();
    }
    if (blockIdx.x == 0) check_cu_seqlens(a.cu_q, a.cu_k, a.N, a.tq, a.tk, a.status);
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_at, 0);

    const int n = uniform(where[0]), tile = uniform(where[1]);
    int64_t q0 = 0, k0 = 0, lq = a.tq, lk = a.tk;
    if (a.cu_q) {
        q0 = a.cu_q[n]; lq = (int64_t)a.cu_q[n + 1] - q0;
        k0 = a.cu_k[n]; lk = (int64_t)a.cu_k[n + 1] - k0;
        if (k0 < 0 || lk < 0 || k0 + lk > a.tk) lk = 0;                // malformed: reported by block 0
        if (q0 < 0 || q0 + lq > a.tq) lq = 0;
    }
    const int64_t r0 = (int64_t)tile * kLpRows;                        // first row within the sequence
    // keys that the last row of each tile sees, in tiles
    int tiles[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int64_t f = r0 + i * 128;
        const int64_t last = (f + 128 < lq ? f + 128 : lq) - 1;
        int64_t seen = tile < 0 || f >= lq ? 0 : a.causal ? lk - lq + last + 1 : lk;
        seen = seen < 0 ? 0 : seen > lk ? lk : seen;
        tiles[i] = uniform((int)((seen + kLpKeys - 1) / kLpKeys));
    }
    // this CTA's share of the key tiles
    const int steps_all = max(tiles[0], tiles[1]);
    const int start = steps_all * rank / splits, steps = steps_all * (rank + 1) / splits - start;
#pragma unroll
    for (int i = 0; i < 2; ++i) tiles[i] = min(max(tiles[i] - start, 0), steps);

    if (warp < 8) {                                                    // ---------------- softmax
        regs_inc<232>();
        const int i = warp >> 2, quarter = warp & 3, mine = i == 0 ? tiles[0] : tiles[1];
        const int64_t row = r0 + i * 128 + quarter * 32 + lane;        // within the sequence
        const int64_t seen = a.causal ? lk - lq + row : lk - 1;        // last key it sees
        const uint32_t ts = tmem_addr(tmem, 32 * quarter, i * 128), to = ts + 256;
        const float sc = a.scale * 1.4426950408889634f;
        float ref = kLpUnset, l = 0.f;
        bool ok = true;
        for (int j = 0; j < mine; ++j) {
            ok = mbar_wait_warp(&s_full[i], j & 1);
            if (!ok) break;
            tc_fence_after_sync();
            float x[128];
#pragma unroll
            for (int c = 0; c < 128; c += 32) tmem_ld32(ts + c, *(float(*)[32])(x + c));
            tmem_wait_ld();
            tmem_ready(x);
            const int64_t first = (int64_t)(start + j) * kLpKeys;
            if (first + kLpKeys - 1 > (seen < lk - 1 ? seen : lk - 1)) {
                const int64_t end = seen < lk - 1 ? seen : lk - 1;
                const int keep = end < first ? 0 : (int)(end - first + 1);
#pragma unroll
                for (int c = 0; c < 128; ++c) x[c] = c < keep ? x[c] : -INFINITY;
            }
            float m[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
            for (int c = 4; c < 128; c += 4) {
                m[0] = fmaxf(m[0], x[c]); m[1] = fmaxf(m[1], x[c + 1]);
                m[2] = fmaxf(m[2], x[c + 2]); m[3] = fmaxf(m[3], x[c + 3]);
            }
            const float top = fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])) * sc;
            const bool move = top > ref + kLpSlack;
            if (__any_sync(0xffffffffu, move)) {
                const float now = move ? top : ref;
                const float f = ex2(ref - now);
                ref = now;
                l *= f;
                if (j > 0) {                                           // the products before S are complete: O is still
                    for (int c = 0; c < 128; c += 32) {
                        float o[32];
                        tmem_ld32(to + c, o);
                        tmem_wait_ld();
                        tmem_ready(o);
                        uint32_t b[32];
#pragma unroll
                        for (int q = 0; q < 32; ++q) b[q] = __float_as_uint(o[q] * f);
                        tmem_st32(to + c, b);
                    }
                }
            }
            const f32x2 sc2 = pack2(sc, sc), nref = pack2(-ref, -ref);
            float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int c = 0; c < 128; c += 64) {
                uint32_t b[32];
#pragma unroll
                for (int q = 0; q < 32; ++q) {
                    float p0, p1;
                    unpack2(fma2(pack2(x[c + 2 * q], x[c + 2 * q + 1]), sc2, nref), p0, p1);
                    p0 = ex2(p0);
                    p1 = ex2(p1);
                    sum[(q & 1) * 2] += p0;
                    sum[(q & 1) * 2 + 1] += p1;
                    const __nv_bfloat162 h = __floats2bfloat162_rn(p0, p1);    // the product's operand: 8 bits
                    b[q] = *(const uint32_t*)&h;
                }
                tmem_st32(ts + c / 2, b);
            }
            l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
            tmem_wait_st();
            // Weight 0 times what lies behind the last key: make that 0.  Done by the first tile that uses it.
            if (start + j + 1 == steps_all && lk - first < kLpKeys && (i == 0 || j >= tiles[0])) {
                const int r = quarter * 32 + lane;
                const uint32_t u = 5 * j + 3 + r / 64;
                if (r >= lk - first) {
                    if (!mbar_wait_spin(&kv_full[(j & 1) * 2 + 1], (j >> 1) & 1)) record_status(a.status, KDA_ERR_TIMEOUT);
                    uint8_t* at = mem + kLpOffRing + u % kLpSlots * kLpPiece + r % 64 * 128;
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        *(uint4*)(at + 16 * q) = make_uint4(0, 0, 0, 0);
                        *(uint4*)(at + 8192 + 16 * q) = make_uint4(0, 0, 0, 0);
                    }
                    fence_proxy_async_smem();
                }
            }
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_full[i]);
        }
        if (ok && mine > 0) {
            ok = mbar_wait_warp(&o_full[i], 0);
            tc_fence_after_sync();
        }
        if (!ok) record_status(a.status, KDA_ERR_TIMEOUT);
        const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
        if (SHARED) {
            // This CTA's part to shared memory, once neither tile's products read there: [row][128] fp32 in 16-byte
            // pieces turned by the row, and log2 of the rows' sums.
            asm volatile("bar.sync 1, 256;" ::: "memory");
            const int r = i * 128 + quarter * 32 + lane;
            float4* part = (float4*)(mem + r * kLpRow);
#pragma unroll
            for (int c = 0; c < 128; c += 32) {
                float o[32];
                if (mine > 0) {
                    tmem_ld32(to + c, o);
                    tmem_wait_ld();
                    tmem_ready(o);
                }
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    part[(c / 4 + q) ^ lane] = mine > 0 ? make_float4(o[4 * q] * inv, o[4 * q + 1] * inv, o[4 * q + 2] * inv,
                                                                      o[4 * q + 3] * inv)
                                                        : make_float4(0.f, 0.f, 0.f, 0.f);
            }
            ((float*)(mem + kLpOffLse))[r] = l == 0.f ? -INFINITY : ref + log2f(l);
            fence_proxy_async_smem();                                  // read by copies
        } else {
            const bool live = tile >= 0 && row < lq;
            __nv_bfloat16* dst = a.out + ((q0 + (live ? row : 0)) * a.H + head) * 128;
            for (int c = 0; c < 128; c += 32) {
                float o[32];
                if (mine > 0) {
                    tmem_ld32(to + c, o);
                    tmem_wait_ld();
                    tmem_ready(o);
                }
                if (live) {
#pragma unroll
                    for (int q = 0; q < 32; q += 8) {
                        uint32_t b[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            b[e] = mine > 0 ? bf16x2(pack2(o[q + 2 * e] * inv, o[q + 2 * e + 1] * inv)) : 0u;
                        *(uint4*)(dst + c + q) = make_uint4(b[0], b[1], b[2], b[3]);
                    }
                }
            }
            if (live && a.lse)
                a.lse[(q0 + row) * a.H + head] = l == 0.f ? -INFINITY : (ref + log2f(l)) * 0.6931471805599453f;
        }
    } else {
        regs_dec<40>();
        if (warp == 8) {                                               // ---------------- producer
            if (lane == 0 && steps > 0) {
                mbar_arrive_expect_tx(q_full, 6 * kLpPiece);
                for (int p = 0; p < 6; ++p)
                    tma_load_3d_at(base + p * kLpPiece, &map_q, p % 3 * 64, head, (int)(q0 + r0) + p / 3 * 128, smem_u32(q_full));
                bool ok = true;
                uint32_t u = 0;
                for (int j = 0; j < steps && ok; ++j) {
                    const int key = (int)k0 + (start + j) * kLpKeys;
                    for (int p = 0; p < 5; ++p, ++u) {
                        if (u >= kLpSlots) {                           // the piece this one takes the place of
                            const uint32_t o = u - kLpSlots, oj = o / 5, g = (oj & 1) * 2 + (o % 5 >= 3);
                            if (!(ok = mbar_wait_spin(&kv_empty[g], (oj >> 1) & 1))) break;
                        }
                        uint64_t* f = &kv_full[(j & 1) * 2 + (p >= 3)];
                        const uint32_t at = base + kLpOffRing + u % kLpSlots * kLpPiece, bar = smem_u32(f);
                        if (p == 0 || p == 3) mbar_arrive_expect_tx(f, (p == 0 ? 3 : 2) * kLpPiece);
                        if (p < 2) tma_load_3d_at(at, &map_k, p * 64, head, key, bar);
                        else if (p == 2) tma_load_2d(at, &map_r, 0, key, bar);
                        else {
                            tma_load_3d_at(at, &map_v, 0, head, key + (p - 3) * 64, bar);
                            tma_load_3d_at(at + 8192, &map_v, 64, head, key + (p - 3) * 64, bar);
                        }
                    }
                }
                if (!ok) drain_copies();
            }
        } else if (warp == 9 && steps > 0) {
            // Matrix instructions.  One warp for both tiles keeps them in turn; whole products behind one wait
            // each, since a wait costs about 90 cycles and instruction fetches compete with the softmax's.
            const uint32_t idesc_s = idesc_bf16(128, 128), idesc_o = idesc_bf16(128, 128, 0, 1);
            const uint64_t dq = sdesc_k_sw128(base), dk = sdesc_k_sw128(base + kLpOffRing);
            const uint64_t dv = sdesc(base + kLpOffRing, 8192, 1024, 2);
            const int n0 = tiles[0], n1 = tiles[1];
            bool ok = mbar_wait_warp(q_full, 0);
            for (int j = -1; j < steps && ok; ++j) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int mine = i == 0 ? n0 : n1;
                    const uint32_t ts = tmem + i * 128, to = ts + 256;
                    if (j >= 0 && j < mine) {                          // O += P_j V_j
                        ok = mbar_wait_warp(&p_full[i], j & 1);
                        if (ok && (i == 0 || j >= n0)) ok = mbar_wait_warp(&kv_full[(j & 1) * 2 + 1], (j >> 1) & 1);
                        if (!ok) break;
                        tc_fence_after_sync();
                        if (elect_one()) {
                            const uint32_t u = 5 * j + 3;
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const uint64_t db = dv + (u + h) % kLpSlots * (kLpPiece / 16);
#pragma unroll
                                for (int k = 0; k < 4; ++k)
                                    mma_bf16_ts(to, ts + h * 32 + k * 8, db + k * (2048 / 16), idesc_o, j > 0 || h > 0 || k > 0);
                            }
                            if (i == 1 || j >= n1) mma_commit(&kv_empty[(j & 1) * 2 + 1]);   // its last user
                            if (j + 1 == mine) mma_commit(&o_full[i]);
                        }
                        __syncwarp();
                    }
                    const int jn = j + 1;                              // S_{j+1}: behind the product that reads P_j in its place
                    if (jn < mine) {
                        if (i == 0 || jn >= n0) ok = mbar_wait_warp(&kv_full[(jn & 1) * 2], (jn >> 1) & 1);
                        if (!ok) break;
                        tc_fence_after_sync();
                        if (elect_one()) {
                            const uint32_t u = 5 * jn;
#pragma unroll
                            for (int p = 0; p < 3; ++p) {
                                const uint64_t da = dq + (i * 3 + p) * (kLpPiece / 16);
                                const uint64_t db = dk + (u + p) % kLpSlots * (kLpPiece / 16);
#pragma unroll
                                for (int k = 0; k < 4; ++k)
                                    mma_bf16_ss(ts, da + 2 * k, db + 2 * k, idesc_s, p > 0 || k > 0);
                            }
                            mma_commit(&s_full[i]);
                            if (i == 1 || jn >= n1) mma_commit(&kv_empty[(jn & 1) * 2]);
                        }
                        __syncwarp();
                    }
                }
            }
            if (!ok && lane == 0) record_status(a.status, KDA_ERR_TIMEOUT);
        }
    }
    if (SHARED) {
        // Each CTA joins a share of the rows: the others copy their parts of those behind its own, 64 KB in 3300
        // cycles with two CTAs.
        const int share = kLpRows / splits;
        auto rows_of = [&](int c) {
            const int64_t left = lq - r0 - c * share;
            return tile < 0 || left < 0 ? 0 : (int)min64(left, share);
        };
        const int rows = rows_of(rank);
        if (threadIdx.x == 0 && rows) mbar_arrive_expect_tx(rows_full, (splits - 1) * rows * kLpRow);
        __syncwarp();
        cluster_sync();
        if (threadIdx.x < splits && (int)threadIdx.x != rank) {
            const int to = threadIdx.x, slot = rank < to ? rank : rank - 1, count = rows_of(to);
            if (count)
                copy_to_cta(map_cta(base + (kLpRows + slot * share) * kLpRow, to), base + to * share * kLpRow, count * kLpRow,
                            map_cta(smem_u32(rows_full), to));
        }
        __syncwarp();
        if (warp < 8 && rows) {
            // the parts' weights, a lane a row of the warp; then the rows
            const int own = share / 8, first = rank * share + warp * own, count = min(own, rows - warp * own);
            float w[kLpSplits], top = kLpUnset, sum = 0.f;
#pragma unroll
            for (int c = 0; c < kLpSplits; ++c)
                w[c] = c < splits && lane < count ? ld_cluster_f32(map_cta(base + kLpOffLse + (first + lane) * 4, c)) : -INFINITY;
#pragma unroll
            for (int c = 0; c < kLpSplits; ++c) top = fmaxf(top, w[c]);
#pragma unroll
            for (int c = 0; c < kLpSplits; ++c) sum += w[c] = ex2(w[c] - top);
            const float inv = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);
            const int64_t row = (q0 + r0 + first) * a.H + head;
            if (a.lse && lane < count)
                a.lse[row + lane * a.H] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
            const bool ok = mbar_wait_warp(rows_full, 0);
            if (!ok) record_status(a.status, KDA_ERR_TIMEOUT);
#pragma unroll 4
            for (int r = 0; r < count; ++r) {
                float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int c = 0; c < kLpSplits; ++c) {
                    if (c >= splits) break;
                    const int at = c == rank ? first + r : kLpRows + (c < rank ? c : c - 1) * share + warp * own + r;
                    const float4 o = *(const float4*)(mem + at * kLpRow + (lane ^ ((first + r) & 31)) * 16);
                    const float v = __shfl_sync(0xffffffffu, w[c] * inv, r);
                    x.x += v * o.x; x.y += v * o.y; x.z += v * o.z; x.w += v * o.w;
                }
                uint2 b;
                b.x = bf16x2(pack2(x.x, x.y));
                b.y = bf16x2(pack2(x.z, x.w));
                *(uint2*)(a.out + (row + (int64_t)r * a.H) * 128 + lane * 4) = b;
            }
        }
        __syncwarp();
        cluster_sync();                                                // the others may still read this CTA's rows
    }
    tc_fence_before_sync();
    __syncthreads();
    if (warp == 0) tmem_dealloc(tmem, 512);
}

// ------------------------------------------------------------------- host
bool latent_prefill_tc_takes(const LatentPrefillArgs& d) {
    const int64_t st[7] = {d.q_ts, d.q_hs, d.k_ts, d.k_hs, d.v_ts, d.v_hs, d.r_ts};
    for (int i = 0; i < 7; ++i)
        if (st[i] <= 0 || st[i] % 8 || st[i] >= (1ll << 38)) return false;
    return d.dtype == KDA_BF16 && d.dk == 128 && d.dr == 64 && d.dv == 128 && d.tk > 0 &&
           (((uintptr_t)d.q | (uintptr_t)d.k | (uintptr_t)d.r | (uintptr_t)d.v | (uintptr_t)d.out) & 15) == 0;
}

// CTAs that share the keys of a tile of rows.  In units of a key tile's time (1.8
// us) a CTA costs its tiles and 5, or 8 and 10 where 2 and 4 share the keys; the
// longest CTA decides, or all of them on 152 SMs.  The lengths of the sequences
// are on the device: taken as even, the longest half as long again.  Measured, us
// (causal, rows x keys x heads; 1, 2 and 4 CTAs):
//   256 x 8192 x 16   123  72  48      2048 x 2048 x 4     42   31   27
//   256 x 8192 x 32   126  74  60      2048 x 2048 x 16    44   44   74
//   256 x 32768 x 8   459 234 130      8192 x 8192 x 4    126   74  111
//   512 x 512 x 16     21  21  25      8192 x 8192 x 16   234  275  408
//   128 x 128 x 16     13  17  18    32768 x 32768 x 1    455  240  246
static int lp_splits(const LatentPrefillArgs& d) {
    const double n = d.cu_q ? d.N : 1, lq = d.tq / n, lk = d.tk / n;
    const double longest = lk / kLpKeys * (n > 1 ? 1.5 : 1);
    const double mean = (!d.causal ? lk : lk > lq ? lk - lq / 2 : lk / 2) / kLpKeys;
    const double ctas = (d.tq / (double)kLpRows + n / 2) * d.H;
    auto time = [&](int s, double fixed) { return fmax(longest / s + fixed, ctas * s / 152 * (mean / s + fixed)); };
    const double one = 0.9 * time(1, 5), two = time(2, 8), four = time(kLpSplits, 10);
    return one <= fmin(two, four) ? 1 : two <= four ? 2 : kLpSplits;
}

cudaError_t latent_prefill_tc_launch(const LatentPrefillArgs& d, cudaStream_t stream) {
    static bool ready = false;
    if (!ready) {
        const cudaFuncAttribute at = cudaFuncAttributeMaxDynamicSharedMemorySize;
        cudaError_t e = cudaFuncSetAttribute(kda_latent_prefill_tc<false>, at, (int)kLpSmem);
        if (e == cudaSuccess) e = cudaFuncSetAttribute(kda_latent_prefill_tc<true>, at, (int)kLpSmem);
        if (e != cudaSuccess) return e;
        ready = true;
    }
    auto map3 = [&](CUtensorMap* m, const void* p, int width, int64_t tokens, int64_t ts, int64_t hs, int rows) {
        const uint64_t dims[3] = {(uint64_t)width, (uint64_t)d.H, (uint64_t)tokens};
        const uint64_t str[2] = {(uint64_t)hs * 2, (uint64_t)ts * 2};
        const uint32_t box[3] = {64, 1, (uint32_t)rows};
        return make_map(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, p, dims, str, box);
    };
    CUtensorMap mq, mk, mr, mv;
    const uint64_t rd[2] = {64, (uint64_t)d.tk}, rs[1] = {(uint64_t)d.r_ts * 2};
    const uint32_t rb[2] = {64, kLpKeys};
    if (!map3(&mq, d.q, 192, d.tq, d.q_ts, d.q_hs, 128) || !map3(&mk, d.k, 128, d.tk, d.k_ts, d.k_hs, kLpKeys) ||
        !map3(&mv, d.v, 128, d.tk, d.v_ts, d.v_hs, 64) ||
        !make_map(&mr, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, d.r, rd, rs, rb)) return cudaErrorInvalidValue;
    LpArgs a;
    a.N = d.N; a.H = d.H; a.causal = d.causal; a.scale = d.scale; a.tq = d.tq; a.tk = d.tk; a.cu_q = d.cu_q;
    a.cu_k = d.cu_k; a.out = (__nv_bfloat16*)d.out; a.lse = d.lse; a.status = d.status;
    // at most this many tiles of rows, whatever the lengths
    const int64_t blocks = d.cu_q ? d.tq / kLpRows + min64(d.N, d.tq) : (d.tq + kLpRows - 1) / kLpRows;
    a.blocks = (int)blocks;
    a.splits = lp_splits(d);
    if (blocks * d.H * a.splits > 0x7fffffffLL) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(blocks * d.H * a.splits)); cfg.blockDim = dim3(kLpThreads);
    cfg.dynamicSmemBytes = kLpSmem; cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = a.splits; at[0].val.clusterDim.y = 1; at[0].val.clusterDim.z = 1;
    cfg.attrs = at; cfg.numAttrs = a.splits > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, a.splits > 1 ? kda_latent_prefill_tc<true> : kda_latent_prefill_tc<false>, mq, mk, mr, mv, a);
}

}  // namespace kda
