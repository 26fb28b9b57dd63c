// kda_matmul_tc.cu -- the scaled e4m3 product on the tensor cores.
//
//     c[m, n] = sum_j  sa[m, j] sb[n / 128, j]  D_j[m, n],   D_j = sum_{k in block j} a b
//
// The scales change with every 128 values of k, so each block's product D_j is
// formed on its own in TMEM (4 instructions of 32 k) and read back, scaled and
// added to fp32 registers while the next blocks' run into other parts of TMEM.  Two shapes of the same loop:
//
//  wide  rows of a along M.  A pair of CTAs (cta_group::2) owns a 256 x BN tile;
//        each loads its 128 rows of a and half of b's rows, so a byte from L2
//        feeds twice the products of a single CTA's tile.  One row of a per
//        lane: its scale and b's block scale make one factor a thread.
//        Persistent: a pair walks tiles in an order that keeps both operands
//        in L2.
//  thin  few rows of a: b's rows along M, a's along N, so b streams through
//        once at full height.  The k blocks are split over the CTAs of a
//        cluster, whose sums meet in distributed shared memory in rank order.
//
// Every wait is bounded; a tile whose wait gave up is filled with NaN.
#include <math.h>

#include "kda_common.cuh"
#include "kda_paths.h"
#include "kda_per_device.h"
#include "kda_sm100_ops.cuh"
#include "kda_tensor_map.h"

namespace kda {
using namespace sm100;

constexpr int kMmEpiWarps = 8;

// ------------------------------------------------------------------- wide
template <int BN>
struct WideShape {
    static constexpr uint32_t kA = 128 * 128, kB = BN / 2 * 128, kStage = kA + kB;
    static constexpr int kStages = BN == 256 ? 4 : 8;              // half for even blocks of k, half for odd ones
    static constexpr int kBufs = 512 / BN;                         // products in TMEM
    static constexpr int kGroups = BN / 128;                       // of 128 columns, each with its own barriers
    static constexpr uint32_t kOut = 128 * BN * 2;                 // output on its way to c, half for each warpgroup
    static constexpr uint32_t kSmem = kStages * kStage + kOut + 1024 + 256;
    static constexpr int kThreads = 32 * (kMmEpiWarps + 4);        // whole warpgroups: registers move between them
};

template <typename T, int BN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(WideShape<BN>::kThreads, 1)
kda_matmul_fp8_wide(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                    const __grid_constant__ CUtensorMap map_c, const int use_map_c, const MatmulArgs g,
                    const int tiles_m, const int tiles_n) {
    using S = WideShape<BN>;
    constexpr int kStages = S::kStages;
    extern __shared__ uint8_t raw[];
    const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u;
    uint8_t* after = raw + (base - smem_u32(raw)) + kStages * S::kStage + S::kOut;
    uint64_t* full = (uint64_t*)after;             // leader: both CTAs' pieces of a stage have landed
    uint64_t* empty = full + kStages;              // the MMAs reading a stage are done
    constexpr int kBufs = S::kBufs;
    constexpr int kGroups = S::kGroups;
    uint64_t* tfull = empty + kStages;             // [kBufs][kGroups] a group of a block's product is in TMEM
    uint64_t* tempty = tfull + kBufs * kGroups;    // [kBufs][kGroups] leader: the pair's epilogue warps have read it
    uint32_t* tmem_at = (uint32_t*)(tempty + kBufs * kGroups);
    int* late = (int*)(tmem_at + 1);               // a wait gave up

    const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    if (threadIdx.x == 0) {
        *late = 0;
        for (int i = 0; i < kStages; ++i) { mbar_init(&full[i], 1 + (g.drop == kDropCopies)); mbar_init(&empty[i], 1); }
        for (int i = 0; i < kBufs * kGroups; ++i) { mbar_init(&tfull[i], 1 + (g.drop == kDropProducts)); mbar_init(&tempty[i], kMmEpiWarps); }
        fence_mbar_init();
    }
    if (warp == 0) { tmem_alloc_pair(tmem_at, 512); tmem_relinquish_pair(); }
    tc_fence_before_sync();
    __syncthreads();
    cluster_sync();
    tc_fence_after_sync();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_at, 0);

    const int kb = (g.k + 127) / 128;
    const int tiles = tiles_m * tiles_n, pairs = gridDim.x / 2, pair = blockIdx.x / 2;
    // 8 tiles of rows beside each other: the tiles in flight form a near square, which reads the least
    auto place = [&](int t, int& tm, int& tn) {
        const int per = 8 * tiles_n, grp = t / per, rows = min(8, tiles_m - grp * 8), r = t - grp * per;
        tm = grp * 8 + r % rows;
        tn = r / rows;
    };

    // Stage of block `it` (counted over the tiles) and the parity of its round: even and odd blocks have a ring
    // each, since a warp each consumes them (in order: a wait on a barrier tells two phases apart, no more).
    auto stage = [&](uint32_t it, uint32_t& ph) {
        constexpr uint32_t kHalf = kStages / 2;
        ph = (it >> 1) / kHalf & 1;
        return (it & 1) * kHalf + (it >> 1) % kHalf;
    };

    // 384 threads x 168 registers at launch = 256 x 232 + 128 x 40
    if (warp < kMmEpiWarps) {                                      // scale, add, store
        regs_inc<232>();
        // A thread sums 128 columns of its row.  Of 256, a warpgroup has a half each; 128 they take in turns, one the even
        // blocks of k and the other the odd ones, and join their sums at the end: a block's wait, reads and sums take a
        // warp about 450 cycles, its products 256 (256 x 6144 x 4096 in a graph: 11.3 us so, 12.0 with both on every block).
        constexpr bool kTurns = BN == 128;
        constexpr int kCols = 128, kOutCols = BN / 2, kStep = kTurns ? 2 : 1;
        const int quarter = warp & 3, half = warp >> 2;
        const int nb_all = (g.n + 127) / 128;
        uint32_t it = 0;
        bool ok = true;
        for (int t = pair; t < tiles; t += pairs) {
            int tm, tn;
            place(t, tm, tn);
            const int64_t row = (int64_t)tm * 256 + rank * 128 + quarter * 32 + lane;
            const int col = tn * BN + half * kOutCols;             // of those it stores
            const float* sa = g.sa + (row < g.m ? row : 0) * kb;
            const float* sb = g.sb + (int64_t)min(kTurns ? tn : col / 128, nb_all - 1) * kb;
            f32x2 acc[kCols / 2];
#pragma unroll
            for (int i = 0; i < kCols / 2; ++i) acc[i] = 0;
            const uint32_t end = it + kb;
            int j = kTurns ? (it + half) & 1 : 0;                  // the turns are counted over the tiles, as the buffers are
            it += j;
            float xa = j < kb ? sa[j] : 0.f, xb = j < kb ? sb[j] : 0.f;   // loaded a block ahead
            for (; j < kb; j += kStep, it += kStep) {
                const float s1 = xa * xb;
                const f32x2 s = pack2(s1, s1);
                const uint32_t d = it % kBufs * kGroups + (kGroups == 2 ? half : 0), dph = it / kBufs & 1;
                if (ok) ok = mbar_wait_spin(&tfull[d], dph);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after_sync();
                const uint32_t at = tmem_addr(tmem, 32 * quarter, it % kBufs * BN + (kTurns ? 0 : half * kCols));
#pragma unroll
                for (int c = 0; c < kCols; c += 64) {              // two loads in flight
                    float f[32], e[32];
                    tmem_ld32(at + c, f);
                    tmem_ld32(at + c + 32, e);
                    if (c == 0) {
                        const int jn = j + kStep < kb ? j + kStep : j;
                        xa = sa[jn];
                        xb = sb[jn];
                    }
                    tmem_wait_ld();
                    tmem_ready(f);
                    tmem_ready(e);
                    if (c + 64 == kCols) {                         // the buffer is read: free it before the last sums
                        tc_fence_before_sync();
                        __syncwarp();
                        if (lane == 0) mbar_arrive_cluster(map_cta(smem_u32(&tempty[d]), 0));
                    }
#pragma unroll
                    for (int i = 0; i < 16; ++i) acc[c / 2 + i] = fma2(pack2(f[2 * i], f[2 * i + 1]), s, acc[c / 2 + i]);
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        acc[c / 2 + 16 + i] = fma2(pack2(e[2 * i], e[2 * i + 1]), s, acc[c / 2 + 16 + i]);
                }
            }
            it = end;
            if (!ok) {
#pragma unroll
                for (int i = 0; i < kCols / 2; ++i) acc[i] = pack2(NAN, NAN);
            }
            if constexpr (kTurns) {
                // The first warpgroup's columns 0 .. 63, then the second's 64 .. 127, each in 32 KB that lie there for
                // the output too: pairs of columns, a row's threads beside each other.
                f32x2* turn = (f32x2*)(raw + (base - smem_u32(raw)) + kStages * S::kStage) + quarter * 32 + lane;
                if (use_map_c && threadIdx.x % 128 == 0) bulk_wait_read_all();
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    asm volatile("bar.sync 3, 256;" ::: "memory");
                    if (half != h) {
#pragma unroll
                        for (int i = 0; i < 32; ++i) turn[i * 128] = acc[h * 32 + i];
                    }
                    asm volatile("bar.sync 3, 256;" ::: "memory");
                    if (half == h) {
#pragma unroll
                        for (int i = 0; i < 32; ++i) acc[i] = h == 0 ? add2(acc[i], turn[i * 128]) : add2(turn[i * 128], acc[32 + i]);
                    }
                }
                asm volatile("bar.sync 3, 256;" ::: "memory");
            }
            if (use_map_c) {
                // Through shared memory and out by TMA: the stores of all SMs' tiles come at once, and the
                // next tile's products need not wait for them.  Boxes of 128 bytes by 128 rows, 128-byte swizzle.
                const uint32_t own = base + kStages * S::kStage + half * (S::kOut / 2);
                const int r = quarter * 32 + lane;
                constexpr int kBox = 128 / sizeof(T), kBoxes = S::kOut / 2 / 16384;   // columns; boxes at a time
#pragma unroll
                for (int c0 = 0; c0 < kOutCols; c0 += kBox) {
                    const uint32_t box = own + c0 / kBox % kBoxes * 16384;
                    if (c0 / kBox % kBoxes == 0) {
                        if (threadIdx.x % 128 == 0) bulk_wait_read_all();
                        asm volatile("bar.sync %0, 128;" ::"r"(1 + half) : "memory");
                    }
#pragma unroll
                    for (int c = 0; c < kBox; c += 16 / sizeof(T)) {
                        const f32x2* v = acc + (c0 + c) / 2;
                        const uint32_t at = box + r * 128 + (c * (int)sizeof(T) / 16 ^ (r & 7)) * 16;
                        uint32_t w[4];
                        if constexpr (sizeof(T) == 2) {
#pragma unroll
                            for (int i = 0; i < 4; ++i) w[i] = bf16x2(v[i]);
                        } else {
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                float lo, hi;
                                unpack2(v[i], lo, hi);
                                w[2 * i] = __float_as_uint(lo);
                                w[2 * i + 1] = __float_as_uint(hi);
                            }
                        }
                        asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                                     "r"(w[3]) : "memory");
                    }
                    fence_proxy_async_smem();
                    asm volatile("bar.sync %0, 128;" ::"r"(1 + half) : "memory");
                    if (threadIdx.x % 128 == 0 && col + c0 < g.n) {
                        tma_store_2d(&map_c, box, col + c0, tm * 256 + rank * 128);
                        bulk_commit();
                    }
                }
            } else {
                // Transposed in the warp's 4 KB of shared memory, so that a store goes along a row: 32 words
                // (fp32, or pairs of bf16) of 32 rows at a time.
                uint32_t* own = (uint32_t*)(raw + (base - smem_u32(raw)) + kStages * S::kStage) + warp * 1024;
                constexpr int kPer = sizeof(T) == 2 ? 2 : 1;       // values of a word
#pragma unroll
                for (int w0 = 0; w0 < kOutCols / kPer; w0 += 32) {
#pragma unroll
                    for (int k = 0; k < 32; ++k) {
                        uint32_t word;
                        if constexpr (kPer == 2) {
                            word = bf16x2(acc[w0 + k]);
                        } else {
                            float lo, hi;
                            unpack2(acc[(w0 + k) / 2], lo, hi);
                            word = __float_as_uint(k & 1 ? hi : lo);
                        }
                        own[lane * 32 + (k ^ lane)] = word;
                    }
                    __syncwarp();
                    const int n = col + (w0 + lane) * kPer;
                    const int rows = (int)min64(32, g.m - (row - lane));
                    T* to = (T*)g.c + (row - lane) * g.ldc + n;
#pragma unroll 4
                    for (int r = 0; r < rows; ++r, to += g.ldc) {
                        const uint32_t word = own[r * 32 + (lane ^ r)];
                        if constexpr (kPer == 1) {
                            if (n < g.n) *(uint32_t*)to = word;
                        } else if (n + 1 < g.n && ((uintptr_t)to & 3) == 0) {
                            *(uint32_t*)to = word;
                        } else {
                            if (n < g.n) *(uint16_t*)to = (uint16_t)word;
                            if (n + 1 < g.n) *((uint16_t*)to + 1) = (uint16_t)(word >> 16);
                        }
                    }
                    __syncwarp();
                }
            }
        }
        if (use_map_c && threadIdx.x % 128 == 0) bulk_wait_all();
        if (!ok) *late = 1;
    } else {
        regs_dec<40>();
        if (warp == kMmEpiWarps || warp == kMmEpiWarps + 3) {      // producers: of even blocks, of odd ones
            const uint32_t own = warp == kMmEpiWarps ? 0 : 1;
            const uint32_t all = (uint32_t)((tiles - pair + pairs - 1) / pairs) * kb;
            int t = pair, j = own, tm, tn;
            place(t, tm, tn);
            bool ok = true;
            for (uint32_t it = own; it < all; it += 2, j += 2) {
                while (j >= kb) { j -= kb; t += pairs; place(t, tm, tn); }
                uint32_t ph;
                const uint32_t s = stage(it, ph);
                if (it >= kStages && !(ok = mbar_wait_warp(&empty[s], ph ^ 1))) break;
                if (elect_one()) {
                    const uint32_t at = base + s * S::kStage, bar = map_cta(smem_u32(&full[s]), 0);
                    if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * S::kStage);
                    tma_load_2d_pair(at, &map_a, j * 128, tm * 256 + (int)rank * 128, bar);
#pragma unroll
                    for (int h = 0; h < kGroups; ++h)              // a group's 128 rows of b: 64 from either CTA
                        tma_load_2d_pair(at + S::kA + h * 8192, &map_b, j * 128, tn * BN + h * 128 + (int)rank * 64, bar);
                }
                __syncwarp();
            }
            if (!ok) *late = 1;
        } else if (warp <= kMmEpiWarps + 2) {
            // Matrix instructions, by the leader: a warp for even blocks and one for odd ones.  One alone needs about
            // 500 cycles for the waits, 4 instructions and the commits, as long as the instructions take.
            if (rank == 0) {
                const uint32_t own = warp - kMmEpiWarps - 1;
                const uint32_t idesc = idesc_e4m3(256, 128);
                const int mine = (tiles - pair + pairs - 1) / pairs;
                const uint32_t all = (uint32_t)mine * kb;
                bool ok = true;
                for (uint32_t it = own; it < all && ok; it += 2) {
                    uint32_t ph;
                    const uint32_t s = stage(it, ph), dph = it / kBufs & 1;
                    const uint64_t da = sdesc_k_sw128(base + s * S::kStage);
                    const uint64_t db = sdesc_k_sw128(base + s * S::kStage + S::kA);
                    ok = mbar_wait_warp(&full[s], ph);
#pragma unroll
                    for (int h = 0; h < kGroups; ++h) {
                        const uint32_t d = it % kBufs * kGroups + h;
                        if (ok && it >= kBufs) ok = mbar_wait_warp(&tempty[d], dph ^ 1);
                        if (!ok) break;
                        tc_fence_after_sync();
                        if (elect_one()) {
#pragma unroll
                            for (int q = 0; q < 4; ++q)
                                mma_f8_ss_pair(tmem + d * 128, da + 2 * q, db + h * (8192 / 16) + 2 * q, idesc, q > 0);
                            mma_commit_pair(&tfull[d], 3);
                            if (h == kGroups - 1) mma_commit_pair(&empty[s], 3);
                        }
                        __syncwarp();
                    }
                }
                if (!ok) *late = 1;
            }
        }
    }
    tc_fence_before_sync();
    meet_at_end(late);
    cluster_sync();                                                // the peer may still read or signal this CTA
    if (warp == 0) tmem_dealloc_pair(tmem, 512);
}

// ------------------------------------------------------------------- thin
// BT rows of a (tokens) a CTA; `splits` CTAs of a cluster share a 128 x BT tile.
constexpr int kThinThreads = 32 * 6;

template <int BT>
struct ThinShape {
    static constexpr uint32_t kA = 128 * 128, kB = BT * 128, kStage = kA + kB;
    static constexpr int kStages = (int)(100 * 1024 / kStage);     // two CTAs on an SM
    static constexpr uint32_t kTmem = 2 * BT < 32 ? 32 : 2 * BT;
    static constexpr uint32_t kScales = kStages * kStage;          // then factors [k blocks of the CTA][BT]
    // sums [BT][128] of the cluster's CTAs: over the stages, which are read by then
    static uint32_t smem(int blocks) { return kScales + (uint32_t)blocks * BT * 4 + 1024 + 256; }
};

template <typename T, int BT>
__global__ void __launch_bounds__(kThinThreads, 2)
kda_matmul_fp8_thin(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                    const MatmulArgs g, const int blocks_per) {
    using S = ThinShape<BT>;
    constexpr int kStages = S::kStages;
    extern __shared__ uint8_t raw[];
    const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u;
    uint8_t* mem = raw + (base - smem_u32(raw));
    float* factors = (float*)(mem + S::kScales);
    uint64_t* full = (uint64_t*)(factors + (size_t)blocks_per * BT);
    uint64_t* empty = full + kStages;
    uint64_t* tfull = empty + kStages;
    uint64_t* tempty = tfull + 2;
    uint32_t* tmem_at = (uint32_t*)(tempty + 2);
    int* late = (int*)(tmem_at + 1);                               // a wait gave up

    const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
    const int splits = gridDim.x;                                  // = the cluster
    const int rank = blockIdx.x, n0 = blockIdx.y * 128;
    const int64_t m0 = (int64_t)blockIdx.z * BT;
    const int kb = (g.k + 127) / 128;
    const int j0 = rank * blocks_per, count = max(0, min(kb, j0 + blocks_per) - j0);
    if (threadIdx.x == 0) {
        *late = 0;
        for (int i = 0; i < kStages; ++i) { mbar_init(&full[i], 1 + (g.drop == kDropCopies)); mbar_init(&empty[i], 1); }
        for (int i = 0; i < 2; ++i) { mbar_init(&tfull[i], 1 + (g.drop == kDropProducts)); mbar_init(&tempty[i], 4); }
        fence_mbar_init();
    }
    if (warp == 0) { tmem_alloc(tmem_at, S::kTmem); tmem_relinquish(); }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_at, 0);

    float acc[BT];
#pragma unroll
    for (int i = 0; i < BT; ++i) acc[i] = 0.f;

    if (warp == 4) {
        if (lane == 0) {
            bool ok = true;
            for (int i = 0; i < count; ++i) {
                const uint32_t s = i % kStages, ph = (i / kStages) & 1;
                if (i >= kStages && !(ok = mbar_wait_spin(&empty[s], ph ^ 1))) break;
                const uint32_t at = base + s * S::kStage, bar = smem_u32(&full[s]);
                mbar_arrive_expect_tx(&full[s], S::kStage);
                tma_load_2d(at, &map_b, (j0 + i) * 128, n0, bar);
                tma_load_2d(at + S::kA, &map_a, (j0 + i) * 128, (int)m0, bar);
            }
            if (!ok) *late = 1;
        }
    } else if (warp == 5) {
        const uint32_t idesc = idesc_e4m3(128, BT);
        bool ok = true;
        for (int i = 0; i < count && ok; ++i) {
            const uint32_t s = i % kStages, ph = (i / kStages) & 1, d = i & 1, dph = (i >> 1) & 1;
            ok = mbar_wait_warp(&full[s], ph);
            if (ok && i >= 2) ok = mbar_wait_warp(&tempty[d], dph ^ 1);
            if (!ok) break;
            tc_fence_after_sync();
            const uint64_t da = sdesc_k_sw128(base + s * S::kStage);
            const uint64_t db = sdesc_k_sw128(base + s * S::kStage + S::kA);
            if (elect_one()) {
#pragma unroll
                for (int q = 0; q < 4; ++q) mma_f8_ss(tmem + d * BT, da + 2 * q, db + 2 * q, idesc, q > 0);
                mma_commit(&empty[s]);
                mma_commit(&tfull[d]);
            }
            __syncwarp();
        }
        if (!ok) *late = 1;
    } else {
        // factors of the CTA's blocks: sa of every token times sb of the 128 rows of b
        const float* sb = g.sb + (int64_t)blockIdx.y * kb + j0;
        for (int i = threadIdx.x; i < count * BT; i += 128) {
            const int j = i % count, t = i / count;                // neighbouring threads: neighbouring blocks of a row
            factors[j * BT + t] = m0 + t < g.m ? g.sa[(m0 + t) * kb + j0 + j] * sb[j] : 0.f;
        }
        asm volatile("bar.sync 1, 128;" ::: "memory");
        bool ok = true;
        for (int i = 0; i < count; ++i) {
            const uint32_t d = i & 1, dph = (i >> 1) & 1;
            ok = __all_sync(0xffffffffu, mbar_wait_spin(&tfull[d], dph));
            if (!ok) break;
            tc_fence_after_sync();
            const uint32_t at = tmem_addr(tmem, 32 * warp, d * BT);
#pragma unroll
            for (int c = 0; c < BT; c += 16) {
                float f[16];
                tmem_ld16(at + c, f);
                tmem_wait_ld();
                tmem_ready(f);
                if (c + 16 == BT) {
                    tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&tempty[d]);
                }
                const float4* w = (const float4*)(factors + i * BT + c);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const float4 x = w[q];
                    acc[c + 4 * q] = fmaf(f[4 * q], x.x, acc[c + 4 * q]);
                    acc[c + 4 * q + 1] = fmaf(f[4 * q + 1], x.y, acc[c + 4 * q + 1]);
                    acc[c + 4 * q + 2] = fmaf(f[4 * q + 2], x.z, acc[c + 4 * q + 2]);
                    acc[c + 4 * q + 3] = fmaf(f[4 * q + 3], x.w, acc[c + 4 * q + 3]);
                }
            }
        }
        if (!ok) {
#pragma unroll
            for (int i = 0; i < BT; ++i) acc[i] = NAN;
        }
        if (!ok) *late = 1;
    }
    // All copies have landed and all MMAs are done (their products were waited for): the stages become sums[t][r].
    tc_fence_before_sync();
    meet_at_end(late);
    if (warp == 0) tmem_dealloc(tmem, S::kTmem);
    const int r = threadIdx.x;                                     // row of b within the tile
    if (splits == 1) {
        if (r < 128 && n0 + r < g.n) {
#pragma unroll
            for (int t = 0; t < BT; ++t)
                if (m0 + t < g.m) ((T*)g.c)[(m0 + t) * g.ldc + n0 + r] = from_f32<T>(acc[t]);
        }
        return;
    }
    float* sums = (float*)mem;
    if (r < 128) {
#pragma unroll
        for (int t = 0; t < BT; ++t) sums[t * 128 + r] = acc[t];
    }
    cluster_sync();
    // each CTA joins and stores its share of the tokens, the splits in rank order; four rows of b a thread
    const int live = (int)min64(BT, g.m - m0);
    for (int i = rank * kThinThreads + threadIdx.x; i < live * 32; i += splits * kThinThreads) {
        float4 part[8];
#pragma unroll
        for (int c = 0; c < 8; ++c)
            if (c < splits) part[c] = ld_cluster_f32x4(map_cta(base + i * 16, c));
        float4 x = part[0];
#pragma unroll
        for (int c = 1; c < 8; ++c)
            if (c < splits) { x.x += part[c].x; x.y += part[c].y; x.z += part[c].z; x.w += part[c].w; }
        const int n = n0 + i % 32 * 4;
        T* to = (T*)g.c + (m0 + i / 32) * g.ldc + n;
        if (n + 4 <= g.n && ((uintptr_t)to & (4 * sizeof(T) - 1)) == 0) {
            if constexpr (sizeof(T) == 2) *(uint2*)to = make_uint2(bf16x2(pack2(x.x, x.y)), bf16x2(pack2(x.z, x.w)));
            else *(float4*)to = x;
        } else {
            const float v[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int q = 0; q < 4; ++q)
                if (n + q < g.n) to[q] = from_f32<T>(v[q]);
        }
    }
    cluster_sync();
}

// ------------------------------------------------------------------- host
static bool make_operand(CUtensorMap* m, const uint8_t* p, int64_t rows, int k, int64_t ld, int box_rows) {
    const uint64_t dims[2] = {(uint64_t)k, (uint64_t)rows}, strides[1] = {(uint64_t)ld};
    const uint32_t box[2] = {128, (uint32_t)box_rows};
    return make_map(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, p, dims, strides, box);
}

template <typename T, int BN>
static cudaError_t launch_wide(const MatmulArgs& a, cudaStream_t stream) {
    using S = WideShape<BN>;
    auto kern = kda_matmul_fp8_wide<T, BN>;
    static PerDevice pairs_at_once;
    int device = 0, resident = 0;
    cudaError_t err = cudaGetDevice(&device);
    if (err == cudaSuccess) err = pairs_at_once.get(device, resident, [&](int& n) {
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)S::kSmem);
        if (e != cudaSuccess) return e;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(2 * 1024); cfg.blockDim = dim3(S::kThreads); cfg.dynamicSmemBytes = S::kSmem;
        e = cudaOccupancyMaxActiveClusters(&n, kern, &cfg);
        n = n > 0 ? n : 1;
        return e;
    });
    if (err != cudaSuccess) return err;
    CUtensorMap ma, mb;
    if (!make_operand(&ma, a.a, a.m, a.k, a.lda, 128) || !make_operand(&mb, a.b, a.n, a.k, a.ldb, 64))
        return cudaErrorInvalidValue;
    // c by TMA where its rows start on 16-byte boundaries
    CUtensorMap mc = ma;
    const bool use_mc = (((uintptr_t)a.c | (uintptr_t)(a.ldc * sizeof(T))) & 15) == 0 && a.ldc < (1ll << 37);
    if (use_mc) {
        const uint64_t dims[2] = {(uint64_t)a.n, (uint64_t)a.m}, strides[1] = {(uint64_t)a.ldc * sizeof(T)};
        const uint32_t box[2] = {128 / sizeof(T), 128};
        if (!make_map(&mc, sizeof(T) == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, a.c, dims,
                      strides, box)) return cudaErrorInvalidValue;
    }
    const int tm = (int)((a.m + 255) / 256), tn = (a.n + BN - 1) / BN;
    const int64_t tiles = (int64_t)tm * tn;
    const int pairs = (int)min64(tiles, resident);
    kern<<<2 * pairs, S::kThreads, S::kSmem, stream>>>(ma, mb, mc, use_mc, a, tm, tn);
    return cudaGetLastError();
}

static void thin_config(cudaLaunchConfig_t& cfg, cudaLaunchAttribute* at, dim3 grid, int cluster, uint32_t smem,
                        cudaStream_t stream) {
    cfg.gridDim = grid; cfg.blockDim = dim3(kThinThreads); cfg.dynamicSmemBytes = smem; cfg.stream = stream;
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = cluster; at[0].val.clusterDim.y = 1; at[0].val.clusterDim.z = 1;
    cfg.attrs = at; cfg.numAttrs = 1;
}

template <typename T, int BT>
static cudaError_t launch_thin(const MatmulArgs& a, cudaStream_t stream, bool& fits) {
    using S = ThinShape<BT>;
    auto kern = kda_matmul_fp8_thin<T, BT>;
    const int kb = (a.k + 127) / 128, tn = (a.n + 127) / 128;
    const int64_t tm = (a.m + BT - 1) / BT, tiles = tn * tm;
    static PerDevice memory_set, clusters_at_once[9];
    int device = 0, set = 0;
    cudaError_t err = cudaGetDevice(&device);
    if (err == cudaSuccess) err = memory_set.get(device, set, [&](int& done) {
        done = 1;
        return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
    });
    // as many splits as run at once, two CTAs on an SM, of four blocks of k at least
    int splits = 1;
    for (int c = 2; c <= 8 && kb >= 4 * c && err == cudaSuccess; ++c) {
        int active = 0;
        err = clusters_at_once[c].get(device, active, [&](int& n) {
            cudaLaunchConfig_t cfg = {};
            cudaLaunchAttribute at[1];
            thin_config(cfg, at, dim3(c, 1024), c, S::smem(24), 0);
            return cudaOccupancyMaxActiveClusters(&n, kern, &cfg);
        });
        if (tiles <= active) splits = c;
    }
    if (err != cudaSuccess) return err;
    const int per = (kb + splits - 1) / splits;
    splits = (kb + per - 1) / per;
    const uint32_t smem = S::smem(per);
    fits = smem <= 227 * 1024;
    if (!fits) return cudaSuccess;
    CUtensorMap ma, mb;
    if (!make_operand(&ma, a.a, a.m, a.k, a.lda, BT) || !make_operand(&mb, a.b, a.n, a.k, a.ldb, 128))
        return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[1];
    thin_config(cfg, at, dim3(splits, tn, (unsigned)tm), splits, smem, stream);
    return cudaLaunchKernelEx(&cfg, kern, ma, mb, a, per);
}

template <typename T>
static cudaError_t launch_matmul(const MatmulArgs& a, cudaStream_t stream) {
    // Measured on a GB300 (us, each of the three the same way, the largest by itself: 430 in a stream of calls; thin with 64
    // rows of a / wide with 128 columns / with 256):
    //   1 x 4096 x 4096  6.4 / 12.5 / 16.8     64 x 8192 x 8192  16.8 / 17.4 / 29.6    128 x 2048 x 4096  7.2 / 11.1 / 17.4
    //   512 x 1024 x 1024  6.2 / 6.8 / 8.2     128 x 6144 x 4096  16.5 / 11.4 / 17.5   1024 x 1024 x 4096  16.9 / 11.5 / 17.5
    //   1024 x 4096 x 4096  42 / 19.6 / 18.3   2048 x 8192 x 4096  140 / 59.7 / 60.0   16384 x 8192 x 4096  1049 / 435 / 386
    // and, with L2 flushed before each, thin against the better of the wide ones
    //   1 x 4096 x 18432  26.8 / 49     64 x 4096 x 18432  31.9 / 42     200 x 1024 x 18432  23.7 / 40     64 x 16384 x 32768  132 / 130
    // thin while its tiles are few (its splits then use SMs that tiles of the others would leave idle); of the wide
    // ones the narrower while all its tiles run at once.
    const int64_t tn = (a.n + 127) / 128;
    if (a.m <= 64 || (a.m + 63) / 64 * tn <= 64) {
        bool fits = true;                                  // the factors of a CTA's blocks of k lie in shared memory
        const cudaError_t e = a.m <= 16 ? launch_thin<T, 16>(a, stream, fits) : a.m <= 32 ? launch_thin<T, 32>(a, stream, fits)
                                        : launch_thin<T, 64>(a, stream, fits);
        if (fits || e != cudaSuccess) return e;
    }
    if ((a.m + 255) / 256 * tn <= 76) return launch_wide<T, 128>(a, stream);
    return launch_wide<T, 256>(a, stream);
}

bool matmul_tc_takes(const MatmulArgs& a) {
    return (((uintptr_t)a.a | (uintptr_t)a.b | (uintptr_t)a.lda | (uintptr_t)a.ldb) & 15) == 0 &&
           a.lda < (1ll << 40) && a.ldb < (1ll << 40);
}

cudaError_t matmul_tc_launch(const MatmulArgs& a, cudaStream_t stream) {
    return a.dtype == KDA_BF16 ? launch_matmul<__nv_bfloat16>(a, stream) : launch_matmul<float>(a, stream);
}

}  // namespace kda
