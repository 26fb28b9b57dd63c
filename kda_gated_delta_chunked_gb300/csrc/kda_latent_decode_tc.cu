// kda_latent_decode_tc.cu -- absorbed latent attention over a paged cache on the
// tensor cores (bf16, rank 512 + 64 rotary channels).
//
// All Lq * H query rows of a sequence read the same 576-channel latents, so a
// tile of 128 cached tokens is used for R of them at once (16, 32 or 64; more
// rows go in groups of 64 to CTAs of their own).  Each group fetches it twice,
// 1152 bytes a token for the first product and 1024 for the second; memory gives
// it once, L2 the other times (64 x 4096 tokens: 311 MB of DRAM reads with 64
// heads, 319 MB with 128, for 302 MB of cache).  Both products keep the tokens'
// side at full height and put the few query rows along N, where an instruction's
// time follows them down:
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
// products take about 2900 (40 cycles an instruction whatever R up to 32).  A
// tile does not stay in shared memory between its two products: the second
// fetches the 512 channels again, out of L2.  So each product has a stream of
// its own, with a producer warp, a ring and a warp that issues it, and the next
// tiles' scores go ahead while this one's softmax and second product run.
// Measured, us in a graph of ten / one behind a flush of L2 (the join included):
//   64 x 16384 tokens, 16 heads  197 (6.1 TB/s) / 214       64 x 4096, 64 heads   81 / 93
//   64 x 16384, 32 heads         208 / 222                  64 x 4096, 128 heads  122 / 132
//   128 x 1024, 16 heads         39 / 52                    3 x 8192, 128 heads   25 / 37
//   1 x 30000, 32 heads          19 / 30                    1 x 700, 32 heads     12 / 19
//
// A wait on an mbarrier looks at a parity only, so each waiter stays within one
// phase of what it waits for: a ring has one producer and one consumer, both in
// order, and what alternates between tiles has a barrier for odd and even ones.
#include <math.h>

#include "kda_latent_decode.cuh"
#include "kda_launch.cuh"
#include "kda_per_device.h"
#include "kda_tensor_map.h"

namespace kda {

constexpr uint32_t kLdPiece = kLdTile * 128;  // 64 channels of a tile
constexpr int kLdThreads = 256;               // 4 softmax warps, 2 producers, a warp for each product
constexpr float kLdSlack = 8.f;               // how far (log2) a score may exceed its reference

template <int R>
struct LdShape {
    // Slots of three pieces (64 channels; with 64 rows two) for S^T, of two for O^T.  A slot is what one copy a
    // page fills: [8 tokens][piece][token of 8][128 bytes], so that pages of any size make one operand.
    static constexpr int kPieces = R == 64 ? 2 : 3, kUnits = (9 + kPieces - 1) / kPieces;
    static constexpr int kSlotsS = 2, kSlotsV = 2, kSlots = kSlotsS + kSlotsV;
    static constexpr int kBufP = R == 64 ? 1 : 2;
    static constexpr uint32_t kSlotS = kPieces * kLdPiece, kSlotV = 2 * kLdPiece, kOffV = kSlotsS * kSlotS;
    static constexpr uint32_t kQPiece = R * 128, kQ = 9 * kQPiece;
    static constexpr uint32_t kRow = R * 2, kP = kLdTile * kRow;   // P^T: a token's R values
    static constexpr uint32_t kOffQ = kOffV + kSlotsV * kSlotV, kOffP = kOffQ + kQ, kOffSmall = kOffP + kBufP * kP;
    static constexpr uint32_t kSmem = kOffSmall + 1024 + (2 * 4 + 3) * R * 4 + 512;
    static constexpr uint32_t kTmem = R == 16 ? 128 : R == 32 ? 256 : 512;   // two S^T, four blocks of O^T: 6 R columns
    static constexpr uint64_t kSwz = R == 16 ? 6 : R == 32 ? 4 : 2;
    // 16-byte piece c of token row r of P^T (32-, 64- or 128-byte swizzle)
    static __device__ __forceinline__ uint32_t p_at(int r, int c) {
        return R == 16 ? r * 32 + ((c ^ (r >> 2)) & 1) * 16
             : R == 32 ? r * 64 + ((c ^ (r >> 1)) & 3) * 16 : r * 128 + ((c ^ r) & 7) * 16;
    }
};

template <int R>
__global__ void __launch_bounds__(kLdThreads, 1)
kda_latent_decode_tc(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_s,
                     const __grid_constant__ CUtensorMap map_v, const LdArgs a) {
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
    uint64_t *full = bars, *empty = full + S::kSlots,              // first the slots for S^T, then those for O^T
             *full_v = full + S::kSlotsS, *empty_v = empty + S::kSlotsS, *q_full = empty + S::kSlots, *q_empty = q_full + 1,
             *s_full = q_empty + 1, *o_full = s_full + 2,          // [2]: alternate tiles
             *p_full = o_full + 2, *zeroed = p_full + 2,            // zeroed [4]: a pair of pieces each
             *bars_end = zeroed + 4;
    uint32_t* tmem_at = (uint32_t*)bars_end;
    int* range = (int*)(tmem_at + 1);                  // first sequence, its first tile, tiles
    int* fault = range + 3;
    int64_t* range_at = (int64_t*)(((uintptr_t)(fault + 1) + 7) & ~(uintptr_t)7);   // index of the first tile

    const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
    const int group = blockIdx.x, cta = blockIdx.y;
    if (warp == 4) {
        // This CTA's range of the tiles of all sequences.  The producer finds it and starts copying; the other
        // warps wait for it at the barrier.
        const int len = lane < a.N ? a.lens[lane] : 0;                       // on its way while the barriers are made
        if (lane < bars_end - bars) mbar_init(bars + lane, (lane < p_full - bars ? 1 : 4) + (a.drop >> lane & 1));
        if (lane == 0) {
            prefetch_map(&map_s);
            prefetch_map(&map_v);
            prefetch_map(&map_q);
        }
        fence_mbar_init();
        const LdCut cut = ld_cut(a, cta, lane, len);
        if (lane == 0) {
            range[0] = cut.n; range[1] = cut.j; range[2] = cut.count;
            if (cta == 0 && group == 0) a.before[a.N] = cut.total;
            *fault = cut.bad ? kLdBadLen : 0;
            *range_at = cut.at;
        }
        __syncwarp();
        asm volatile("bar.arrive 3, %0;" ::"n"(kLdThreads) : "memory");
    } else {
        if (warp == 0) { tmem_alloc(tmem_at, S::kTmem); tmem_relinquish(); }
        if (threadIdx.x < R) {
            ref[threadIdx.x] = kLdUnset;
            query[threadIdx.x] = min((group * R + (int)threadIdx.x) / a.H, a.Lq - 1);
        }
        tc_fence_before_sync();
        asm volatile("bar.sync 3, %0;" ::"n"(kLdThreads) : "memory");
        tc_fence_after_sync();
    }
    const uint32_t tmem = warp == 4 ? 0 : __shfl_sync(0xffffffffu, *tmem_at, 0);
    const uint32_t base_v = base + S::kOffV;
    if (warp == 4 || warp == 5) {                                      // ---------------- producers: for S^T, for O^T
        const bool scores = warp == 4;
        const int box = min(a.page_size, kLdTile), boxes = kLdTile / box;
        const uint32_t slots = scores ? S::kSlotsS : S::kSlotsV, ring = scores ? base : base_v;
        const uint32_t slot = scores ? S::kSlotS : S::kSlotV;
        const int units = scores ? S::kUnits : 4, pieces = scores ? S::kPieces : 2;
        const CUtensorMap* map = scores ? &map_s : &map_v;
        uint64_t *fulls = scores ? full : full_v, *empties = scores ? empty : empty_v;
        uint32_t seg = 0, s = 0, ph = 1;                               // slot and the parity its emptying has (first round: none)
        // With 32 rows the second fetch, a little later than with 16, may come when L2 has given the lines up, depending
        // on what was in it before: 64 sequences of up to 16384 tokens 107 us by themselves, 132 to 147 between products of
        // 25 to 100 MB of weights.  With the second fetch's lines marked to go first 111 and 113 to 119.  (The first one's
        // marked to stay as well: 109 and 111 to 113, but they stay for whatever follows: four products by the same 64 MB
        // of weights 79 us behind it instead of 72.)  With 16 rows the mark costs 2%, with 64 it changes nothing.
        const uint64_t last_use = l2_drop();
        bool ok = true, bad_page = false;
        LdWalk w;
        w.start(a, range[0], range[1], range[2]);
        for (; w.left > 0 && ok; w.next(a)) {
            if (scores && w.first) {
                if (seg > 0) ok = mbar_wait_warp(q_empty, (seg - 1) & 1);
                if (!ok) break;
                if (lane == 0) {
                    mbar_arrive_expect_tx(q_full, S::kQ);
                    for (int c = 0; c < 9; ++c)
                        tma_load_3d_at(base + S::kOffQ + c * S::kQPiece, &map_q, c * 64, group * R, w.n, smem_u32(q_full));
                }
                __syncwarp();
                ++seg;
            }
            // A lane for each box of tokens: its page and row.  Pages behind the length, and bad ones, read as zeros.
            int row = 0, page = a.num_pages;
            if (lane < boxes) {
                const int t = w.j * kLdTile + lane * box;
                if (t < ld_len(a, w.n)) {
                    const int p = a.table[(int64_t)w.n * a.max_pages + t / a.page_size];
                    if (p < 0 || p >= a.num_pages) bad_page = true;
                    else { page = p; row = t % a.page_size; }
                }
            }
            for (int u = 0; u < units; ++u) {
                if (!(ok = mbar_wait_warp(&empties[s], ph))) break;    // (a fresh barrier counts as emptied)
                if (lane == 0) mbar_arrive_expect_tx(&fulls[s], slot);
                __syncwarp();
                if (lane < boxes) {
                    const uint32_t at = ring + s * slot + lane * (slot / boxes);
                    if (R != 32 || scores) tma_load_5d(at, map, 0, 0, u * pieces, row / 8, page, smem_u32(&fulls[s]));
                    else tma_load_5d(at, map, 0, 0, u * pieces, row / 8, page, smem_u32(&fulls[s]), last_use);
                }
                __syncwarp();
                if (++s == slots) { s = 0; ph ^= 1; }
            }
        }
        if (bad_page) atomicOr(fault, kLdBadPage);
        if (!ok) atomicOr(fault, kLdLate);
    } else if (warp == 6) {                                            // ---------------- S^T
        const uint32_t idesc = idesc_bf16(128, R);
        const uint64_t dq = sdesc_k_sw128(base + S::kOffQ);
        uint32_t s = 0, ph = 0, seg = 0;
        bool ok = true;
        LdWalk w;
        w.start(a, range[0], range[1], range[2]);
        const int count = w.left;
        for (int j = 0; j < count && ok; ++j, w.next(a)) {
            if (w.first) { ok = mbar_wait_warp(q_full, seg & 1); ++seg; }
            if (ok && j >= 2) ok = mbar_wait_warp(&p_full[j & 1], ((j - 2) >> 1) & 1);   // S_{j-2} is read
            const uint32_t d = tmem + (j & 1) * R;
#pragma unroll
            for (int u = 0; u < S::kUnits; ++u) {
                if (ok) ok = mbar_wait_warp(&full[s], ph);
                if (!ok) break;
                tc_fence_after_sync();
                // A: tokens, K-major, 8-token groups a slot's pieces apart
                const uint64_t da = sdesc(base + s * S::kSlotS, 16, S::kPieces * 1024, 2);
                if (elect_one()) {
#pragma unroll
                    for (int p = 0; p < S::kPieces && u * S::kPieces + p < 9; ++p) {
                        const uint64_t db = dq + (u * S::kPieces + p) * (S::kQPiece / 16);
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            mma_bf16_ss(d, da + p * (1024 / 16) + 2 * k, db + 2 * k, idesc, u > 0 || p > 0 || k > 0);
                    }
                    mma_commit(&empty[s]);
                    if (u == S::kUnits - 1) {
                        mma_commit(&s_full[j & 1]);
                        if (w.last()) mma_commit(q_empty);
                    }
                }
                __syncwarp();
                if (++s == S::kSlotsS) { s = 0; ph ^= 1; }
            }
        }
        if (!ok) atomicOr(fault, kLdLate);
    } else if (warp == 7) {                                            // ---------------- O^T += V^T P^T
        const uint32_t idesc = idesc_bf16(128, R, 1, 1);
        uint32_t s = 0, ph = 0, zero = 0;
        bool ok = true;
        LdWalk w;
        w.start(a, range[0], range[1], range[2]);
        const int count = w.left;
        for (int j = 0; j < count && ok; ++j, w.next(a)) {
            if (!(ok = mbar_wait_warp(&p_full[j & 1], (j >> 1) & 1))) break;
            const uint64_t dp = sdesc(base + S::kOffP + j % S::kBufP * S::kP, 16, 8 * S::kRow, S::kSwz);
            const bool ragged = uniform(w.end() >= ld_len(a, w.n));
            for (int p = 0; p < 4; ++p) {
                ok = mbar_wait_warp(&full_v[s], ph);
                if (ok && ragged) ok = mbar_wait_warp(&zeroed[p], zero & 1);
                if (!ok) break;
                tc_fence_after_sync();
                // A: 128 channels = two pieces of 64, MN-major; 16 tokens a step
                const uint64_t da = sdesc(base_v + s * S::kSlotV, 1024, 2048, 2);
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        mma_bf16_ss(tmem + (2 + p) * R, da + k * (4096 / 16), dp + k * (16 * S::kRow / 16), idesc,
                                    !w.first || k > 0);
                    mma_commit(&empty_v[s]);
                    if (p == 3) mma_commit(&o_full[j & 1]);
                }
                __syncwarp();
                if (++s == S::kSlotsV) { s = 0; ph ^= 1; }
            }
            zero += ragged;
        }
        if (!ok) atomicOr(fault, kLdLate);
    } else {                                                           // ---------------- softmax
        const uint32_t lanes = tmem_addr(tmem, 32 * warp, 0);
        const float sc = a.scale * 1.4426950408889634f;
        const int row0 = group * R, live = min(R, a.rows - row0);
        float l[R];
#pragma unroll
        for (int c = 0; c < R; ++c) l[c] = 0.f;
        bool ok = true;
        LdWalk w;
        w.start(a, range[0], range[1], range[2]);
        const int count = w.left;
        for (int j = 0; j < count; ++j, w.next(a)) {
            if (w.first && w.j == 0 && threadIdx.x == 0 && group == 0) a.before[w.n] = *range_at + j;
            ok = bar_and(128, mbar_wait_spin(&s_full[j & 1], (j >> 1) & 1));
            if (!ok) break;
            tc_fence_after_sync();
            const uint32_t at_s = lanes + (j & 1) * R;
            const int len = ld_len(a, w.n);
            const int token = w.j * kLdTile + (int)threadIdx.x;
            float x[R];
            if constexpr (R == 16) {
                tmem_ld16(at_s, x);
            } else {
#pragma unroll
                for (int c = 0; c < R; c += 32) tmem_ld32(at_s + c, *(float(*)[32])(x + c));
            }
            tmem_wait_ld();
            tmem_ready(x);
#pragma unroll
            for (int c = 0; c < R; ++c) x[c] *= sc;
            if (w.end() > len - a.Lq) {                                // some row does not see some token
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
                ld_columns<R, true>(x, across + warp * R, lane);
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
                if (!w.first) {                                        // O^T, once the products into it are complete
                    ok = bar_and(128, mbar_wait_spin(&o_full[(j - 1) & 1], ((j - 1) >> 1) & 1));
                    if (!ok) break;
                    tc_fence_after_sync();
                    for (int p = 2; p <= 5; ++p) {
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
            if (j >= S::kBufP) {                                       // P's buffer: the products that read it are complete
                const int before = j - S::kBufP;
                ok = mbar_wait_warp(&o_full[before & 1], (before >> 1) & 1);
                if (!ok) {                                             // the other warps leave at their next vote, with this one
                    bar_and(128, false);
                    break;
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
                *(uint4*)(mem + S::kOffP + j % S::kBufP * S::kP + S::p_at(threadIdx.x, c / 8)) = make_uint4(b[0], b[1], b[2], b[3]);
            }
            fence_proxy_async_smem();
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_full[j & 1]);
            // Weight 0 times what lies behind the length: make that 0, each pair of pieces as it comes (once the
            // products of the tile before are complete, the ring is at this tile's).
            if (w.end() >= len) {
                if (j > 0) ok = mbar_wait_warp(&o_full[(j - 1) & 1], ((j - 1) >> 1) & 1);
                for (int p = 0; p < 4 && ok; ++p) {
                    const uint32_t u = 4 * j + p, s = u % S::kSlotsV;
                    if (!(ok = mbar_wait_warp(&full_v[s], (u / S::kSlotsV) & 1))) break;
                    uint8_t* at = mem + S::kOffV + s * S::kSlotV + threadIdx.x % 8 * 16;
                    for (int r = len - w.j * kLdTile + (int)threadIdx.x / 8; r < kLdTile; r += 16) {
                        *(uint4*)(at + r / 8 * 2048 + r % 8 * 128) = make_uint4(0, 0, 0, 0);
                        *(uint4*)(at + r / 8 * 2048 + 1024 + r % 8 * 128) = make_uint4(0, 0, 0, 0);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&zeroed[p]);
                }
            }
            if (!w.last()) continue;

            // end of a segment: sums across the tokens' threads, then O^T out
            ld_columns<R, false>(l, sums + warp * R, lane);
            ok = bar_and(128, ok && mbar_wait_spin(&o_full[j & 1], (j >> 1) & 1));
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
            constexpr int W = R < 32 ? R : 32;
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                const int ch = p * 128 + threadIdx.x;
#pragma unroll
                for (int h = 0; h < R; h += W) {
                    float o[W];
                    if constexpr (W == 16) tmem_ld16(lanes + (2 + p) * R + h, o);
                    else tmem_ld32(lanes + (2 + p) * R + h, o);
                    tmem_wait_ld();
                    tmem_ready(o);
                    if (whole) {
                        __nv_bfloat16* to = a.out + ((size_t)w.n * a.rows + row0 + h) * kLdRank + ch;
                        if (h + W <= live) {                           // (256 x 128 rows of 100 tokens: 78 -> 68 us)
#pragma unroll
                            for (int c = 0; c < W; ++c) to[(size_t)c * kLdRank] = __float2bfloat16_rn(o[c] * fac[h + c]);
                        } else {
#pragma unroll
                            for (int c = 0; c < W; ++c)
                                if (h + c < live) to[(size_t)c * kLdRank] = __float2bfloat16_rn(o[c] * fac[h + c]);
                        }
                    } else {                                           // (dead rows too: a condition a store costs more)
#pragma unroll
                        for (int c = 0; c < W; ++c) dst[(h + c) * kLdPart + ch] = o[c];
                    }
                }
            }
            asm volatile("bar.sync 2, 128;" ::: "memory");
            if (threadIdx.x < R) ref[threadIdx.x] = kLdUnset;
#pragma unroll
            for (int c = 0; c < R; ++c) l[c] = 0.f;
            asm volatile("bar.sync 2, 128;" ::: "memory");
        }
        if (!ok) {
            // The join finds the pieces by where the sequences start, those of the tiles that were left among them.
            w.start(a, range[0], range[1], range[2]);
            for (int j = 0; j < count; ++j, w.next(a))
                if (w.j == 0 && threadIdx.x == 0 && group == 0) a.before[w.n] = *range_at + j;
            atomicOr(fault, kLdLate);
        }
    }
    tc_fence_before_sync();
    meet_at_end(fault);
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (warp == 0) tmem_dealloc(tmem, S::kTmem);
    if (threadIdx.x == 0) a.cta_status[cta * gridDim.x + group] = *fault;
}

// Joins the pieces of sequences that several CTAs shared, gives sequences
// without tiles their zeros, and collects the CTAs' status.  A block a row, its
// warps a share of the pieces each: two of them for many rows, sixteen for few,
// and then a block for each 128 of its channels.
template <int R, int Q>                                // Q: 128-channel blocks of a block, 4 or 1
__global__ void __launch_bounds__(512)
kda_latent_decode_join(const LdArgs a, const int groups) {
    extern __shared__ __align__(16) float sh[];        // [warps][128 Q] O
    const int n = blockIdx.x, row = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int warps = blockDim.x >> 5;
    const int ch0 = blockIdx.z * 128 * Q;
    const int tiles = ld_tiles(a, n);
    wait_before();
    follow_me();
    if (n == 0 && row == 0 && blockIdx.z == 0) {
        int st = 0;
        for (int i = threadIdx.x; i < a.G * groups; i += blockDim.x) st |= a.cta_status[i];
        const bool late = __syncthreads_or(st & kLdLate);          // leaves any output unspecified; the others their sequences'
        const bool bad_page = __syncthreads_or(st & kLdBadPage), bad_len = __syncthreads_or(st & kLdBadLen);
        if (threadIdx.x == 0)
            *a.status = late ? KDA_ERR_TIMEOUT : bad_page ? KDA_ERR_BAD_PAGE : bad_len ? KDA_ERR_BAD_SEQLENS : KDA_OK;
    }
    int cf = 0, cl = -1;
    if (tiles > 0) {
        const int64_t total = a.before[a.N], before = a.before[n], parts = min64(a.G, total);
        if (total < (1 << 20)) {
            cf = (int)(((uint32_t)(before + 1) * (uint32_t)parts - 1) / (uint32_t)total);
            cl = (int)(((uint32_t)(before + tiles) * (uint32_t)parts - 1) / (uint32_t)total);
        } else {
            cf = (int)(((before + 1) * parts - 1) / total);
            cl = (int)(((before + tiles) * parts - 1) / total);
        }
        if (cf == cl) return;                          // finished by its CTA
        cf = max(cf, 0);                               // (no piece is looked for outside, also if the lengths changed meanwhile)
        cl = min(cl, a.G - 1);
    }
    const int group = row / R, c = row % R;
    auto piece = [&](int i) {
        return a.parts + (((size_t)(i * groups + group) * 2 + (i == cf)) * R + c) * kLdPart;
    };
    float o[4 * Q];
#pragma unroll
    for (int i = 0; i < 4 * Q; ++i) o[i] = 0.f;
    // With few rows, the warp's first two pieces of each 32 (all, with sixteen warps) on their way beside what weighs them
    // (8-bit cache, 1 x 30000 tokens, 32 heads, with the kernel before: 19.3 us, 17.6 so; with many rows it takes a
    // microsecond more).
    constexpr int kAhead = Q == 1 ? 2 : 0;
    float4 ahead[5][2];
#pragma unroll
    for (int g = 0; g < 5; ++g)
#pragma unroll
        for (int t = 0; t < kAhead; ++t) {
            const int k = warp + t * warps;
            if (k < 32 && cf + 32 * g + k <= cl) ahead[g][t] = *(const float4*)(piece(cf + 32 * g + k) + ch0 + lane * 4);
        }
    // Every warp weighs all pieces (152 at most), a lane each, and adds up its share of them.
    float2 ml[5];
    float top = kLdUnset, sum = 0.f;
#pragma unroll
    for (int g = 0; g < 5; ++g) {
        const int i = cf + 32 * g + lane;
        ml[g] = i <= cl ? *(const float2*)(piece(i) + kLdRank) : make_float2(kLdUnset, 0.f);
    }
#pragma unroll
    for (int g = 0; g < 5; ++g) top = fmaxf(top, ml[g].x);
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, s));
#pragma unroll
    for (int g = 0; g < 5; ++g) {
        const float wgt = ex2(ml[g].x - top);
        sum += wgt * ml[g].y;
        const int here = min(32, cl - cf - 32 * g + 1);
        int k = warp;
#pragma unroll
        for (int t = 0; t < kAhead; ++t) {
            if (k >= here) break;
            const float x = __shfl_sync(0xffffffffu, wgt, k);
            o[0] += x * ahead[g][t].x; o[1] += x * ahead[g][t].y; o[2] += x * ahead[g][t].z; o[3] += x * ahead[g][t].w;
            k += warps;
        }
#pragma unroll 4
        for (; k < here; k += warps) {
            const float x = __shfl_sync(0xffffffffu, wgt, k);
            const float* p = piece(cf + 32 * g + k);
#pragma unroll
            for (int q = 0; q < Q; ++q) {
                const float4 v = *(const float4*)(p + ch0 + q * 128 + lane * 4);
                o[4 * q] += x * v.x; o[4 * q + 1] += x * v.y; o[4 * q + 2] += x * v.z; o[4 * q + 3] += x * v.w;
            }
        }
    }
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, s);
#pragma unroll
    for (int q = 0; q < Q; ++q)
        *(float4*)(sh + warp * 128 * Q + q * 128 + lane * 4) = make_float4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
    __syncthreads();
    const float inv = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);
    for (int e = threadIdx.x * 4; e < 128 * Q; e += blockDim.x * 4) {
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int w = 0; w < warps; ++w) {
            const float4 y = *(const float4*)(sh + w * 128 * Q + e);
            x.x += y.x; x.y += y.y; x.z += y.z; x.w += y.w;
        }
        uint2 b;
        b.x = bf16x2(pack2(x.x * inv, x.y * inv));
        b.y = bf16x2(pack2(x.z * inv, x.w * inv));
        *(uint2*)(a.out + ((size_t)n * a.rows + row) * kLdRank + ch0 + e) = b;
    }
    if (threadIdx.x == 0 && blockIdx.z == 0 && a.lse)
        a.lse[(size_t)n * a.rows + row] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
}

// ------------------------------------------------------------------- host
static int ld_rows(int Lq, int H) {                // rows of a group
    const int64_t rows = (int64_t)Lq * H;
    return rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
}

bool latent_decode_tc_takes(int dtype, int dk, int dr, int H, int Lq, int page_size) {
    return dtype == KDA_BF16 && dk == kLdRank && dr == kLdWidth - kLdRank && page_size >= 8 &&
           (page_size & (page_size - 1)) == 0 && (int64_t)Lq * H <= 32 * 1024;
}
size_t latent_decode_tc_bytes(int N, int Lq, int H, int page_size, int max_pages) {
    return N > 0 ? ld_plan(N, Lq, H, page_size, max_pages, ld_rows(Lq, H)).bytes : 0;
}
// What the tensor maps need of the call's tensors.
bool latent_decode_tc_aligned(const LatentDecodeArgs& d) {
    const bool flat = d.Lq == 1 || d.H == 1 || d.q_ts == (int64_t)d.H * d.q_hs;   // (query, head) is one strided dimension
    return flat && (((uintptr_t)d.q | (uintptr_t)d.cache | (uintptr_t)d.out) & 15) == 0 && d.q_ts % 8 == 0 &&
           (d.H == 1 || (d.q_hs % 8 == 0 && d.q_hs > 0)) && d.q_ts > 0 && d.page_stride % 8 == 0 && d.num_pages > 0 &&
           d.page_stride < (1ll << 38) && d.q_ts < (1ll << 30);
}

template <int R>
static cudaError_t ld_join(const LdArgs& a, int groups, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    // Few rows: more blocks and warps for each (1 x 30000 tokens, 32 heads: 21 us, 43 as for many).  From 256 rows on as
    // for many (16 x 2048, 16 heads: 17 us, 21 as for few).
    const bool many = (int64_t)a.N * a.rows >= 256;
    const int warps = many ? 2 : 16, per = many ? 4 : 1;
    cfg.gridDim = dim3(a.N, a.rows, 4 / per); cfg.blockDim = dim3(32 * warps); cfg.stream = stream;
    cfg.dynamicSmemBytes = warps * 128 * per * 4;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    // It starts as the last CTAs of the kernel before end (128 x 1024 tokens, 16 heads: 56 us behind them, 52 so);
    // started with them, its waiting blocks take from it (4 queries x 30000 tokens, 16 heads: 29 us, 26 so).
    cfg.attrs = at; cfg.numAttrs = 1;
    return many ? cudaLaunchKernelEx(&cfg, kda_latent_decode_join<R, 4>, a, groups)
                : cudaLaunchKernelEx(&cfg, kda_latent_decode_join<R, 1>, a, groups);
}

cudaError_t latent_decode_join_launch(const LdArgs& a, int R, int groups, cudaStream_t stream) {
    return R == 16 ? ld_join<16>(a, groups, stream) : R == 32 ? ld_join<32>(a, groups, stream) : ld_join<64>(a, groups, stream);
}

template <int R>
static cudaError_t ld_launch(const LatentDecodeArgs& d, const LdPlan& p, cudaStream_t stream) {
    using S = LdShape<R>;
    static PerDevice memory_set;
    int device = 0, set = 0;
    cudaError_t err = cudaGetDevice(&device);
    if (err == cudaSuccess) err = memory_set.get(device, set, [](int& done) {
        done = 1;
        return cudaFuncSetAttribute(kda_latent_decode_tc<R>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)S::kSmem);
    });
    if (err != cudaSuccess) return err;
    LdArgs a;
    a.N = d.N; a.H = d.H; a.Lq = d.Lq; a.rows = d.Lq * d.H; a.page_size = d.page_size; a.num_pages = d.num_pages;
    a.max_pages = d.max_pages; a.scale = d.scale; a.table = d.table; a.lens = d.lens; a.out = (__nv_bfloat16*)d.out;
    a.lse = d.lse; a.status = d.status; a.cta_status = (int32_t*)d.scratch; a.G = p.G;
    a.before = (int64_t*)((char*)d.scratch + p.before);
    a.parts = (float*)((char*)d.scratch + p.parts);
    constexpr uint32_t kS = S::kSlots;                 // the barriers' order: full, empty, q_full, q_empty, s, o, p, zeroed
    constexpr uint32_t kDrops[6] = {0, ((1u << kS) - 1) | 1u << 2 * kS, 3u << (2 * kS + 2), 3u << (2 * kS + 4), 3u << (2 * kS + 6),
                                    15u << (2 * kS + 8)};
    a.drop = kDrops[d.drop];
    CUtensorMap mq, ms, mv;
    const uint64_t qd[3] = {kLdWidth, (uint64_t)a.rows, (uint64_t)d.N};
    const uint64_t qs[2] = {(uint64_t)(d.H == 1 ? d.q_ts : d.q_hs) * 2, (uint64_t)d.q_ts * d.Lq * 2};
    const uint32_t qb[3] = {64, R, 1};
    // the cache as [page][8 tokens][piece][token of 8][channel of 64], the last three the innermost
    const uint64_t cd[5] = {64, 8, kLdWidth / 64, (uint64_t)d.page_size / 8, (uint64_t)d.num_pages};
    const uint64_t cs[4] = {kLdWidth * 2, 128, 8 * kLdWidth * 2, (uint64_t)d.page_stride * 2};
    uint32_t cb[5] = {64, 8, (uint32_t)S::kPieces, (uint32_t)(d.page_size < kLdTile ? d.page_size : kLdTile) / 8, 1};
    bool made = make_map(&mq, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, d.q, qd, qs, qb) &&
                make_map(&ms, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, d.cache, cd, cs, cb);
    cb[2] = 2;
    made = made && make_map(&mv, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, d.cache, cd, cs, cb);
    if (!made) return cudaErrorInvalidValue;
    kda_latent_decode_tc<R><<<dim3(p.groups, p.G), kLdThreads, S::kSmem, stream>>>(mq, ms, mv, a);
    err = cudaGetLastError();
    if (err != cudaSuccess) return err;
    return latent_decode_join_launch(a, R, p.groups, stream);
}

cudaError_t latent_decode_tc_launch(const LatentDecodeArgs& d, cudaStream_t stream) {
    const LdPlan p = ld_plan(d.N, d.Lq, d.H, d.page_size, d.max_pages, ld_rows(d.Lq, d.H));
    return p.R == 16 ? ld_launch<16>(d, p, stream) : p.R == 32 ? ld_launch<32>(d, p, stream) : ld_launch<64>(d, p, stream);
}

}  // namespace kda
