// kda_latent_prefill_tc.cu -- expanded latent attention over packed prompts on
// the tensor cores (bf16; keys 128 + 64 shared rotary channels, values 128).
//
//     S = Q K^T (192 channels),  P = exp2(scale' S - ref),  O += P V
//
// A CTA owns 256 query rows of one head as two tiles of 128 and walks the key
// tiles of 128 that they see.  While the softmax of one tile runs on its own
// eight warps (two threads a row), the tensor core works on the other:
//
//     PV_j(0)  S_{j+1}(0)  PV_j(1)  S_{j+1}(1)  PV_{j+1}(0) ...
//
// TMEM holds S0 S1 O0 O1 (4 x 128 columns); P overwrites its S as bf16 and is
// read from there, so only V passes through shared memory for the second
// product.  The reference of a row moves only when a score exceeds it by 2^8
// (then the row of O is rescaled), which is rare after the first tiles.
// With the queries' 96 KB, rings of five 16 KB pieces for K (64 channels each)
// and three for V (64 keys) fill shared memory.  A piece is freed by the last
// product that reads it, and K and V have a producer each, since V waits for room
// longer than the K behind it.
//
// A CTA that is done takes over the rows of a block that has not started yet, and
// fetches their queries and keys while the last values of its own are weighed.
//
// Few rows (a chunk of a long prompt, few heads) leave SMs idle and the longest
// row alone decides: then the 2 or 4 CTAs of a cluster share the rows' key tiles,
// and their parts of O are joined, in rank order, in distributed shared memory
// (256 rows of 8192 keys, 16 heads: 123 -> 48 us with 4).
//
// A key tile of both row tiles is 2 x (12 + 8) instructions of 64 cycles, 2560 of
// the tensor pipe; it takes 3360.  The pipe starts an instruction about when it is
// issued, and the issuing warp's waits between products are the difference; loads,
// exponentials and maxima are hidden (without them the time is the same).  8192
// tokens, 32 heads, causal: 420 to 425 us by itself, 1.62 PFLOP/s; 438 to 446 in
// a stream of calls, where power bounds the clocks; all keys 812 and 847.  What
// else was measured there (us, by itself): a wait for each of a product's barriers 429, and a thread a row then 461;
// the rings freed a step at a time 470; a warp for each tile's instructions, in
// turns 474; blocks of one tile of rows, one ring, a thread a row 445 (and 100
// prompts of 60 tokens 99 instead of 54).
#include <math.h>

#include "kda_common.cuh"
#include "kda_paths.h"
#include "kda_per_device.h"
#include "kda_sm100_ops.cuh"
#include "kda_tensor_map.h"

namespace kda {
using namespace sm100;

constexpr int kLpRows = 256;                  // query rows of a CTA
constexpr int kLpKeys = 128;
constexpr uint32_t kLpPiece = 16384;
constexpr int kLpSlotsK = 5, kLpSlotsV = 3;
constexpr uint32_t kLpOffK = 6 * kLpPiece, kLpOffV = kLpOffK + kLpSlotsK * kLpPiece, kLpOffSmall = kLpOffV + kLpSlotsV * kLpPiece;
constexpr uint32_t kLpRow = 512;              // bytes of an fp32 row of O, where a cluster joins
constexpr int kLpSplits = 4;                  // CTAs that share the keys of a tile of rows at most
constexpr uint32_t kLpOffLse = kLpOffSmall + 384, kLpSmem = kLpOffLse + kLpRows * 4 + 1024;
constexpr int kLpSoftmax = 16;                // warps: two for 32 rows, half of the keys each
constexpr int kLpThreads = 32 * (kLpSoftmax + 4);
constexpr int kLpHeads = 8;                   // heads of a group
constexpr float kLpUnset = -1e30f, kLpSlack = 8.f;

struct LpArgs {
    int N, H, causal, blocks, splits, drop;    // blocks: tiles of rows of a head at most; splits: CTAs that share them
    float scale;
    int64_t tq, tk;
    const int32_t *cu_q, *cu_k;
    __nv_bfloat16* out;
    float* lse;
    int32_t* status;
};

// 128 + 128 query rows of a head: what every warp needs to know of them.
struct alignas(16) LpItem {
    int q0, lq, k0, lk;                        // their sequence: first row and rows, first key and keys
    int r0, head;                              // first row within the sequence; -1: no more work
    int start, tiles[2];                       // key tiles: first, and how many for each half
};

// A ring of N slots that starts anew with every rows' first piece, so that a piece's slot depends on its place among
// these rows' alone and stays in uniform registers (counted over all rows it does not: 6% of the whole).  A bit for each
// slot keeps the parity of its barriers.
template <int N>
struct LpRing {
    uint32_t bits = 0;
    __device__ __forceinline__ uint32_t parity(int piece) const { return (bits >> piece % N ^ piece / N) & 1; }
    __device__ __forceinline__ void add(int pieces) {
#pragma unroll
        for (int s = 0; s < N; ++s) bits ^= ((pieces - s + N - 1) / N & 1) << s;
    }
};

// Among the 256 threads of a tile's softmax.
__device__ __forceinline__ void tile_sync(int i) { asm volatile("bar.sync %0, 256;" ::"r"(1 + i) : "memory"); }
__device__ __forceinline__ bool barrier_and(int id, int threads, bool v) {
    uint32_t r;
    asm volatile("{\n .reg .pred p, q;\n setp.ne.u32 q, %1, 0;\n barrier.cta.red.and.pred p, %2, %3, q;\n selp.u32 %0, 1, 0, p;\n}"
                 : "=r"(r) : "r"((uint32_t)v), "r"(id), "r"(threads) : "memory");
    return r;
}
__device__ __forceinline__ bool tile_and(int i, bool v) { return barrier_and(1 + i, 256, v); }

template <bool SHARED>
__global__ void __launch_bounds__(kLpThreads, 1)
kda_latent_prefill_tc(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                      const __grid_constant__ CUtensorMap map_r, const __grid_constant__ CUtensorMap map_v,
                      const LpArgs a) {
    extern __shared__ uint8_t raw[];
    const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u;
    uint8_t* mem = raw + (base - smem_u32(raw));
    LpItem* items = (LpItem*)(mem + kLpOffSmall);              // [2]
    uint4* answer = (uint4*)(items + 2);
    uint64_t* q_full = (uint64_t*)(answer + 1);
    uint64_t *q_empty = q_full + 1, *k_full = q_empty + 1, *k_empty = k_full + kLpSlotsK;
    uint64_t *v_full = k_empty + kLpSlotsK, *v_empty = v_full + kLpSlotsV;
    uint64_t *s_full = v_empty + kLpSlotsV, *p_full = s_full + 2, *o_full = p_full + 2;
    uint64_t *item_full = o_full + 2, *item_empty = item_full + 2, *next = item_empty + 2, *answered = next + 1;
    uint64_t* rows_full = answered + 1;
    uint32_t* tmem_at = (uint32_t*)(rows_full + 1);
    int* late = (int*)(tmem_at + 1);                           // a wait gave up

    const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
    const int splits = SHARED ? a.splits : 1, rank = SHARED ? (int)blockIdx.x % splits : 0;   // of the rows' keys
    if (threadIdx.x == 32) { prefetch_map(&map_q); prefetch_map(&map_k); prefetch_map(&map_r); prefetch_map(&map_v); }
    if (warp == 0) {
        tmem_alloc(tmem_at, 512);
        tmem_relinquish();
    }
    if (threadIdx.x == 0) {
        *late = 0;
        const int more = a.drop == kDropCopies;
        mbar_init(q_full, 1 + more);
        mbar_init(rows_full, 1);
        mbar_init(next, 1);
        mbar_init(answered, 1);
        mbar_init(q_empty, 1);
        for (int i = 0; i < kLpSlotsK; ++i) { mbar_init(&k_full[i], 1 + more); mbar_init(&k_empty[i], 1); }
        for (int i = 0; i < kLpSlotsV; ++i) { mbar_init(&v_full[i], 1 + more); mbar_init(&v_empty[i], 1); }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_full[i], 1 + (a.drop == kDropProducts));
            mbar_init(&p_full[i], kLpSoftmax / 2 + (a.drop == kDropWeights));
            mbar_init(&o_full[i], 1 + (a.drop == kDropSecondProducts));
            mbar_init(&item_full[i], 1 + (a.drop == kDropRows)); mbar_init(&item_empty[i], kLpSoftmax + 3);
        }
        fence_mbar_init();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_at, 0);

    if (warp < kLpSoftmax) {                                           // ---------------- softmax
        regs_inc<112>();                                               // 640 x 96 at launch = 512 x 112 + 128 x 32
        // Two threads a row, half of the keys (and of O's channels) each.  They share the row's reference, by way of
        // shared memory when it moves.
        const int i = warp >> 3, half = warp >> 2 & 1, quarter = warp & 3, r = quarter * 32 + lane;
        const uint32_t ts = tmem_addr(tmem, 32 * quarter, i * 128), to = ts + 256 + half * 64;
        float* shared = (float*)(mem + kLpOffLse) + i * 128 + r;
        const float sc = a.scale * 1.4426950408889634f;
        bool ok = true;
        LpRing<kLpSlotsV> v_ring;
        uint32_t tile0 = 0, outs = 0;                                  // this tile's steps and results so far
        for (uint32_t it = 0; ok; ++it) {
            // All who meet at barriers further down leave here together, if one of them gave up: a tile's warps, and where
            // parts are joined both tiles'.
            ok = mbar_wait_warp(&item_full[it & 1], it >> 1 & 1);
            ok = SHARED ? barrier_and(3, 32 * kLpSoftmax, ok) : tile_and(i, ok);
            if (!ok) {
                record_status(a.status, KDA_ERR_TIMEOUT);
                break;
            }
            const LpItem& item = items[it & 1];
            if (item.r0 < 0) break;
            const int mine = uniform(item.tiles[i]);
            const int64_t row = (int64_t)item.r0 + i * 128 + r;        // within the sequence
            int end = item.lk - 1;                                     // last key it sees
            if (a.causal) end = (int)min64(end, (int64_t)item.lk - item.lq + row);
            const int seen = end - item.start * kLpKeys + 1 - half * 64;   // of this thread's
            const int ragged = item.lk % kLpKeys ? item.lk / kLpKeys - item.start : -1;   // step whose tile is not full
            float ref = kLpUnset, l = 0.f;
            for (int j = 0; j < mine; ++j) {
                ok = tile_and(i, ok && mbar_wait_spin(&s_full[i], (tile0 + j) & 1));
                if (!ok) break;
                tc_fence_after_sync();
                float x[64];
                tmem_ld32(ts + half * 64, *(float(*)[32])x);
                tmem_ld32(ts + half * 64 + 32, *(float(*)[32])(x + 32));
                tmem_wait_ld();
                tmem_ready(x);
                const int keep = seen - j * kLpKeys;
                if (keep < 64) {
#pragma unroll
                    for (int c = 0; c < 64; ++c) x[c] = c < keep ? x[c] : -INFINITY;
                }
                float m[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
                for (int c = 4; c < 64; c += 4) {
                    m[0] = fmaxf(m[0], x[c]); m[1] = fmaxf(m[1], x[c + 1]);
                    m[2] = fmaxf(m[2], x[c + 2]); m[3] = fmaxf(m[3], x[c + 3]);
                }
                float top = fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])) * sc;
                // (behind this both halves of S are read, and P may take their place)
                if (!tile_and(i, !(top > ref + kLpSlack))) {
                    if (half) *shared = top;
                    tile_sync(i);
                    float now = ref;
                    if (!half) {
                        top = fmaxf(top, *shared);
                        if (top > ref + kLpSlack) now = top;
                        *shared = now;
                    }
                    tile_sync(i);
                    if (half) now = *shared;
                    const float f = ex2(ref - now);
                    ref = now;
                    l *= f;
                    if (j > 0) {                                       // the products before S are complete: O is still
#pragma unroll 1
                        for (int c = 0; c < 64; c += 16) {
                            float o[16];
                            tmem_ld16(to + c, o);
                            tmem_wait_ld();
                            tmem_ready(o);
#pragma unroll
                            for (int q = 0; q < 16; ++q) o[q] *= f;
                            tmem_st16(to + c, o);
                        }
                    }
                }
                const f32x2 sc2 = pack2(sc, sc), nref = pack2(-ref, -ref);
                float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int c = 0; c < 64; c += 32) {
                    float b[16];
#pragma unroll
                    for (int q = 0; q < 16; ++q) {
                        float p0, p1;
                        unpack2(fma2(pack2(x[c + 2 * q], x[c + 2 * q + 1]), sc2, nref), p0, p1);
                        p0 = ex2(p0);
                        p1 = ex2(p1);
                        sum[(q & 1) * 2] += p0;
                        sum[(q & 1) * 2 + 1] += p1;
                        const __nv_bfloat162 h = __floats2bfloat162_rn(p0, p1);    // the product's operand: 8 bits
                        b[q] = __uint_as_float(*(const uint32_t*)&h);
                    }
                    tmem_st16(ts + half * 32 + c / 2, b);
                }
                l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
                tmem_wait_st();
                // Weight 0 times what lies behind the last key: make that 0.  Done by the first tile that uses it.
                if (j == ragged && (i == 0 || j >= item.tiles[0])) {
                    const int piece = 2 * j + r / 64;
                    if (r >= item.lk % kLpKeys) {
                        if (!mbar_wait_spin(&v_full[piece % kLpSlotsV], v_ring.parity(piece))) {
                            record_status(a.status, KDA_ERR_TIMEOUT);
                            *late = 1;
                        }
                        uint8_t* at = mem + kLpOffV + piece % kLpSlotsV * kLpPiece + half * 8192 + r % 64 * 128;
#pragma unroll
                        for (int q = 0; q < 8; ++q) *(uint4*)(at + 16 * q) = make_uint4(0, 0, 0, 0);
                        fence_proxy_async_smem();
                    }
                }
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[i]);
            }
            // the row's sum, and O once its products are complete
            if (half) *shared = l;
            tile_sync(i);
            if (!half) {
                l += *shared;
                *shared = l;
            }
            ok = tile_and(i, ok && (mine == 0 || mbar_wait_spin(&o_full[i], outs & 1)));
            // (where parts are joined the tiles stay together: neither goes on alone to the vote on the next rows)
            if (SHARED) ok = barrier_and(3, 32 * kLpSoftmax, ok);
            if (half) l = *shared;
            tc_fence_after_sync();
            v_ring.add(2 * max(item.tiles[0], item.tiles[1]));
            tile0 += mine;
            outs += mine > 0;
            if (!ok) record_status(a.status, KDA_ERR_TIMEOUT);
            const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
            if (SHARED) {
                // This CTA's part to shared memory, since neither tile's products read there now: [row][128] fp32 in 16-byte
                // pieces turned by the row, and log2 of the rows' sums.
                float4* part = (float4*)(mem + (i * 128 + r) * kLpRow);
#pragma unroll
                for (int c = 0; c < 64; c += 32) {
                    float o[32];
                    if (mine > 0) {
                        tmem_ld32(to + c, o);
                        tmem_wait_ld();
                        tmem_ready(o);
                    }
#pragma unroll
                    for (int q = 0; q < 8; ++q)
                        part[(half * 16 + c / 4 + q) ^ lane] =
                            mine > 0 ? make_float4(o[4 * q] * inv, o[4 * q + 1] * inv, o[4 * q + 2] * inv, o[4 * q + 3] * inv)
                                     : make_float4(0.f, 0.f, 0.f, 0.f);
                }
                if (half) *shared = l == 0.f ? -INFINITY : ref + log2f(l);
                fence_proxy_async_smem();                              // read by copies
            } else {
                const bool live = row < item.lq;
                const int64_t at = (item.q0 + (live ? row : 0)) * a.H + item.head;
                __nv_bfloat16* dst = a.out + at * 128 + half * 64;
#pragma unroll
                for (int c = 0; c < 64; c += 32) {
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
                if (live && half && a.lse) a.lse[at] = l == 0.f ? -INFINITY : (ref + log2f(l)) * 0.6931471805599453f;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&item_empty[it & 1]);
        }
        if (!ok) *late = 1;
    } else {
        regs_dec<32>();
        if (warp == kLpSoftmax || warp == kLpSoftmax + 3) {                                 // ---------------- producers: queries and keys, values
            // Each its own ring and warp: values wait for room longer than the keys behind them.
            if (lane == 0) {
                bool ok = true;
                LpRing<kLpSlotsK> k_ring;
                LpRing<kLpSlotsV> v_ring;
                uint32_t loaded = 0;
                for (uint32_t it = 0; ok; ++it) {
                    if (!(ok = mbar_wait_spin(&item_full[it & 1], it >> 1 & 1))) break;
                    const LpItem x = items[it & 1];
                    mbar_arrive(&item_empty[it & 1]);
                    if (x.r0 < 0) break;
                    const int steps = max(x.tiles[0], x.tiles[1]), ask = max(steps - 2, 0);
                    int key = x.k0 + x.start * kLpKeys;
                    if (warp == kLpSoftmax) {
                        if (steps == 0) mbar_arrive(next);
                        for (int j = 0; j < steps && ok; ++j, key += kLpKeys) {
                            if (j == ask) mbar_arrive(next);           // the next rows will be wanted soon
#pragma unroll
                            for (int p = 0; p < 3; ++p) {
                                const int piece = 3 * j + p, slot = piece % kLpSlotsK;
                                if (!(ok = mbar_wait_spin(&k_empty[slot], k_ring.parity(piece) ^ 1))) break;
                                const uint32_t at = base + kLpOffK + slot * kLpPiece, bar = smem_u32(&k_full[slot]);
                                mbar_arrive_expect_tx(&k_full[slot], kLpPiece);
                                if (p < 2) tma_load_3d_at(at, &map_k, p * 64, x.head, key, bar);
                                else tma_load_2d(at, &map_r, 0, key, bar);
                            }
                            if (j == 0 && ok) {
                                if (loaded > 0 && !(ok = mbar_wait_spin(q_empty, (loaded - 1) & 1))) break;
                                ++loaded;
                                mbar_arrive_expect_tx(q_full, 6 * kLpPiece);
                                for (int c = 0; c < 6; ++c)
                                    tma_load_3d_at(base + c * kLpPiece, &map_q, c % 3 * 64, x.head,
                                                   x.q0 + x.r0 + c / 3 * 128, smem_u32(q_full));
                            }
                        }
                        k_ring.add(3 * steps);
                    } else {
                        for (int j = 0; j < steps && ok; ++j, key += kLpKeys) {
#pragma unroll
                            for (int p = 0; p < 2; ++p) {
                                const int piece = 2 * j + p, slot = piece % kLpSlotsV;
                                if (!(ok = mbar_wait_spin(&v_empty[slot], v_ring.parity(piece) ^ 1))) break;
                                const uint32_t at = base + kLpOffV + slot * kLpPiece, bar = smem_u32(&v_full[slot]);
                                mbar_arrive_expect_tx(&v_full[slot], kLpPiece);
                                tma_load_3d_at(at, &map_v, 0, x.head, key + p * 64, bar);
                                tma_load_3d_at(at + 8192, &map_v, 64, x.head, key + p * 64, bar);
                            }
                        }
                        v_ring.add(2 * steps);
                    }
                }
                if (!ok) *late = 1;
            }
        } else if (warp == kLpSoftmax + 1) {
            // Matrix instructions.  One warp for both tiles keeps them in turn; whole products behind one wait
            // each, since a wait costs about 90 cycles and instruction fetches compete with the softmax's.
            const uint32_t idesc_s = idesc_bf16(128, 128), idesc_o = idesc_bf16(128, 128, 0, 1);
            const uint64_t dq = sdesc_k_sw128(base), dk = sdesc_k_sw128(base + kLpOffK);
            const uint64_t dv = sdesc(base + kLpOffV, 8192, 1024, 2);
            LpRing<kLpSlotsK> k_ring;
            LpRing<kLpSlotsV> v_ring;
            uint32_t tile0[2] = {0, 0}, loaded = 0;
            bool ok = true;
            for (uint32_t it = 0; ok; ++it) {
                if (!(ok = mbar_wait_warp(&item_full[it & 1], it >> 1 & 1))) break;
                const int n0 = uniform(items[it & 1].tiles[0]), n1 = uniform(items[it & 1].tiles[1]);
                const int r0 = uniform(items[it & 1].r0), steps = max(n0, n1);
                __syncwarp();
                if (lane == 0) mbar_arrive(&item_empty[it & 1]);
                if (r0 < 0) break;
                if (steps == 0) continue;
                ok = mbar_wait_warp(q_full, loaded & 1);
                ++loaded;
                for (int j = -1; j < steps && ok; ++j) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int mine = i == 0 ? n0 : n1;
                        const uint32_t ts = tmem + i * 128, to = ts + 256;
                        const int jn = j + 1;
                        const bool pv = j >= 0 && j < mine, scores = jn < mine;
                        if (pv) {                                      // O += P_j V_j
                            const bool first = i == 0 || j >= n0, last = i == 1 || j >= n1;   // of V's users
                            uint64_t* const p_at = &p_full[i];
                            const uint32_t p_parity = (tile0[i] + j) & 1;
                            if (first)
                                ok = mbar_wait_all<3>({p_at, &v_full[2 * j % kLpSlotsV], &v_full[(2 * j + 1) % kLpSlotsV]},
                                                      {p_parity, v_ring.parity(2 * j), v_ring.parity(2 * j + 1)});
                            else ok = mbar_wait_all<1>({p_at}, {p_parity});
                            if (!ok) break;
                            tc_fence_after_sync();
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const int piece = 2 * j + h, slot = piece % kLpSlotsV;
                                if (elect_one()) {
                                    const uint64_t db = dv + slot * (kLpPiece / 16);
#pragma unroll
                                    for (int k = 0; k < 4; ++k)
                                        mma_bf16_ts(to, ts + h * 32 + k * 8, db + k * (2048 / 16), idesc_o, j > 0 || h > 0 || k > 0);
                                    if (last) mma_commit(&v_empty[slot]);
                                    if (h == 1 && j + 1 == mine) mma_commit(&o_full[i]);
                                }
                                __syncwarp();
                            }
                        }
                        if (ok && scores) {                            // S_{j+1}: behind the product that reads P_j in its place
                            const bool first = i == 0 || jn >= n0, last = i == 1 || jn >= n1;
                            if (first)
                                ok = mbar_wait_all<3>({&k_full[3 * jn % kLpSlotsK], &k_full[(3 * jn + 1) % kLpSlotsK],
                                                       &k_full[(3 * jn + 2) % kLpSlotsK]},
                                                      {k_ring.parity(3 * jn), k_ring.parity(3 * jn + 1), k_ring.parity(3 * jn + 2)});
                            if (!ok) break;
                            tc_fence_after_sync();
#pragma unroll
                            for (int p = 0; p < 3; ++p) {
                                const int piece = 3 * jn + p, slot = piece % kLpSlotsK;
                                if (elect_one()) {
                                    const uint64_t da = dq + (i * 3 + p) * (kLpPiece / 16), db = dk + slot * (kLpPiece / 16);
#pragma unroll
                                    for (int k = 0; k < 4; ++k)
                                        mma_bf16_ss(ts, da + 2 * k, db + 2 * k, idesc_s, p > 0 || k > 0);
                                    if (last) mma_commit(&k_empty[slot]);
                                    if (p == 2) {
                                        mma_commit(&s_full[i]);
                                        if (last && jn + 1 == steps) mma_commit(q_empty);
                                    }
                                }
                                __syncwarp();
                            }
                        }
                        if (!ok) break;
                    }
                }
                k_ring.add(3 * steps);
                v_ring.add(2 * steps);
                tile0[0] += n0;
                tile0[1] += n1;
            }
            if (!ok && lane == 0) record_status(a.status, KDA_ERR_TIMEOUT);
            if (!ok) *late = 1;
        } else if (warp == kLpSoftmax + 2) {                                       // ---------------- which rows
            // In groups of heads (whose keys and values then stay in L2), a sequence's last rows, which see most keys,
            // first, so that what runs last is short (8192 tokens, 32 heads: a tenth less than a head at a time).
            // A CTA that is done with its own takes over those of a block that has not started yet.
            bool ok = true;
            uint32_t it = 0, asked = 0;
            int index = (int)blockIdx.x / splits;
            for (;;) {
                const int per = a.blocks * kLpHeads, grp = index / per;
                const int heads = min(kLpHeads, a.H - grp * kLpHeads), in_grp = index - grp * per;
                const int block = in_grp / heads;
                int n = 0, tile = -1;
                if (a.cu_q == nullptr) {
                    tile = (int)((a.tq + kLpRows - 1) / kLpRows) - 1 - block;
                } else {
                    int before = 0;
                    for (int b = 0; b < a.N; b += 32) {
                        const int s = b + lane;
                        const int len = s < a.N ? a.cu_q[s + 1] - a.cu_q[s] : 0;
                        const int t = len > 0 ? (len + kLpRows - 1) / kLpRows : 0;
                        int x = t;                                     // inclusive scan
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
                if (tile >= 0) {
                    LpItem x;
                    x.head = grp * kLpHeads + in_grp % heads;
                    x.q0 = 0; x.k0 = 0; x.lq = (int)a.tq; x.lk = (int)a.tk; x.r0 = tile * kLpRows;
                    if (a.cu_q) {
                        x.q0 = a.cu_q[n]; x.lq = a.cu_q[n + 1] - x.q0;
                        x.k0 = a.cu_k[n]; x.lk = a.cu_k[n + 1] - x.k0;
                        if (x.k0 < 0 || x.lk < 0 || x.k0 > a.tk - x.lk) x.lk = 0;        // malformed: reported
                        if (x.q0 < 0 || x.q0 > a.tq - x.lq) x.lq = 0;
                    }
                    // keys that the last row of each half sees, in tiles
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int64_t f = (int64_t)x.r0 + i * 128;
                        const int64_t last = min64(f + 128, x.lq) - 1;
                        int64_t seen = f >= x.lq ? 0 : a.causal ? (int64_t)x.lk - x.lq + last + 1 : x.lk;
                        seen = seen < 0 ? 0 : min64(seen, x.lk);
                        x.tiles[i] = (int)((seen + kLpKeys - 1) / kLpKeys);
                    }
                    // this CTA's share of them
                    const int64_t all = max(x.tiles[0], x.tiles[1]);
                    x.start = (int)(all * rank / splits);
                    const int steps = (int)(all * (rank + 1) / splits) - x.start;
#pragma unroll
                    for (int i = 0; i < 2; ++i) x.tiles[i] = min(max(x.tiles[i] - x.start, 0), steps);
                    if (it >= 2 && !(ok = mbar_wait_warp(&item_empty[it & 1], ((it >> 1) - 1) & 1))) break;
                    if (lane == 0) {
                        items[it & 1] = x;
                        mbar_arrive(&item_full[it & 1]);
                    }
                    ++it;
                }
                if (index == 0 && rank == 0) {
                    bool bad = false;
                    for (int s = lane; a.cu_q && s <= a.N; s += 32) {
                        if (s == 0) bad |= a.cu_q[0] != 0 || a.cu_k[0] != 0;
                        else bad |= a.cu_q[s] < a.cu_q[s - 1] || a.cu_k[s] < a.cu_k[s - 1];
                        if (s == a.N) bad |= a.cu_q[s] != a.tq || a.cu_k[s] != a.tk;
                    }
                    bad = __any_sync(0xffffffffu, bad);
                    if (lane == 0) *a.status = bad ? KDA_ERR_BAD_SEQLENS : KDA_OK;
                }
                if (SHARED) break;
                if (tile >= 0) {                                       // as long as the rows take: for all keys that fit
                    if (!(ok = mbar_wait_idle(next, (it - 1) & 1, late))) break;
                }
                __syncwarp();
                if (lane == 0) {
                    fence_proxy_async_smem();                          // the answer before this one is read
                    mbar_arrive_expect_tx(answered, 16);
                    take_block(answer, answered);
                }
                __syncwarp();
                if (!(ok = mbar_wait_warp(answered, asked & 1))) break;
                ++asked;
                if (!taken_block(answer, index)) break;
                index = uniform(index);
            }
            if (ok && it >= 2) ok = mbar_wait_warp(&item_empty[it & 1], ((it >> 1) - 1) & 1);
            if (ok && lane == 0) {
                items[it & 1].r0 = -1;
                mbar_arrive(&item_full[it & 1]);
            }
            if (!ok && lane == 0) record_status(a.status, KDA_ERR_TIMEOUT);
            if (!ok) *late = 1;
        }
    }
    tc_fence_before_sync();
    meet_at_end(late);
    if (SHARED) {
        // Each CTA joins a share of the rows: the others copy their parts of those behind its own, 64 KB in 3300
        // cycles with two CTAs.
        const int share = kLpRows / splits, head = items[0].head;
        const int64_t q0 = items[0].q0, r0 = items[0].r0, lq = items[0].lq;
        auto rows_of = [&](int c) {
            const int64_t left = lq - r0 - c * share;
            return r0 < 0 || left < 0 ? 0 : (int)min64(left, share);
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
        if (warp < kLpSoftmax && rows) {
            // the parts' weights, a lane a row of the warp; then the rows
            const int own = share / kLpSoftmax, first = rank * share + warp * own, count = min(own, rows - warp * own);
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
    static PerDevice memory_set;
    int device = 0, set = 0;
    cudaError_t err = cudaGetDevice(&device);
    if (err == cudaSuccess) err = memory_set.get(device, set, [](int& done) {
        done = 1;
        const cudaFuncAttribute at = cudaFuncAttributeMaxDynamicSharedMemorySize;
        const cudaError_t e = cudaFuncSetAttribute(kda_latent_prefill_tc<false>, at, (int)kLpSmem);
        return e == cudaSuccess ? cudaFuncSetAttribute(kda_latent_prefill_tc<true>, at, (int)kLpSmem) : e;
    });
    if (err != cudaSuccess) return err;
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
    a.drop = d.drop;
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
