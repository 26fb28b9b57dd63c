// kda_latent_decode8_tc.cu -- absorbed latent attention over the quantised cache on
// the tensor cores (bf16 queries, rank 512 + 64 rotary channels): the matrix
// instructions take the cache's e4m3 codes as they are.
//
// Token t's latent is 2^e_t c_t with codes c_t, so
//
//     s_tr = 2^e_t (c_t . q_r) + rope_t . q_r,    o_r = sum_t (p_tr 2^e_t) c_t / sum_t p_tr
//
// The other operand has to be of 8 bits too, so it is split into several values
// that add up to it:
//   - a query's channel is 2^x (q1 + q2 / 16) with e4m3 q1, q2 and one x a row: the
//     8 bits of a bf16 exactly, down to 2^-14 of steps where the row's largest is
//     224 to 448 (e4m3's subnormals).  q1 and q2 are columns of one product.
//   - a weight P = p 2^e is p1 + p2 / 8 + p3 / 64 in e5m2, each the rest of the one
//     before: three bits each, off by 2^-8.6 (bf16: 2^-8) for P down to 2^-17 of the
//     row's largest P, below that by 2^-26 of it.  e5m2 for its range: the tokens
//     behind a dominant one are many and small, and would be lost in e4m3's.
//
//     S^T [128 tokens, q1 | q2 | rope: 3 x 32]  = C Q^T        16 + 4 instructions
//     O^T [4 x 128 channels, p1 | p2 | p3: 3 x 32] += C^T P^T  4 x 4 instructions
//
// The rotary channels are bf16 and have columns of their own.  Both products read
// the same tile in shared memory, the second as an MN-major operand: a tile is
// fetched once, 641 bytes a token.  A thread owns a token and half of the rows, so
// the token's scale is a thread's number, and the halves need not wait for one
// another.  The softmax reference of a row bounds P (not p): it moves when some P
// exceeds it by 2^12, and stands at 2^3, so that P stays below 2^15, e5m2's largest
// power of two.
//
// CTAs have groups of 32 query rows; how the tiles are shared out, and the joining
// of the pieces, are kda_latent_decode_tc.cu's.  A warp each copies, issues the one
// product and the other, and fetches the tokens' scales; eight do the softmax, four
// the queries of the sequence that comes next.
//
// One group: bound by HBM.  A tile's 82 KB take an SM 3650 cycles at 6.78 TB/s.
// Several groups, which share a tile in L2: 2500 a tile, and shared memory is busy
// for about as long at its 128 bytes a cycle: 1830 with the operands (an instruction
// of 32, 64, 96 columns takes 40, 48, 56 cycles), 640 with the copies, 100 with the
// weights.  A piece stays for 4200, 900 to arrive (1900 from HBM), 930 the scores,
// 1500 the softmax, 900 the second product, and there is room for two tiles.
// Measured beside it: tiles of 96 tokens, three in shared memory (64 x up to 16384
// tokens, 32 heads 75 us instead of 77; 64 x 4096, 128 heads 121 instead of 108); one
// place for the weights and a ring of nine or ten pieces of codes instead of eight
// (114 and 117 instead of 109).
// The first scores come 3.5 us after the start and their weights 1.2 later, in
// instructions not used before; a sequence's end costs 3, the join 3 to 9.
// Measured, us in a graph of ten / one behind a flush of L2 (the join included):
//   64 x 16384 tokens, 16 heads  110 (6.1 TB/s) / 126       64 x 4096, 64 heads   61 / 68
//   64 x up to 16384, 32 heads   72 / 86                    64 x 4096, 128 heads  103 / 107
//   128 x 1024, 16 heads         23 / 35                    3 x 8192, 128 heads   24 / 29
//   1 x 30000, 32 heads          16 / 25                    1 x 700, 32 heads     11 / 16
//   64 x 8192, 16 heads, pages of 8, of 16 and more: 67, 63 (copies are issued a box of a page at a time)
#include <cuda_fp16.h>
#include <math.h>
#include <string.h>

#include "kda_latent_cache.cuh"
#include "kda_latent_decode.cuh"
#include "kda_launch.cuh"
#include "kda_per_device.h"
#include "kda_tensor_map.h"

namespace kda {

constexpr int kL8Rows = 32;                                  // query rows of a CTA
constexpr int kL8Threads = 512;                              // 8 softmax warps, producer, two products, scales, 4 for the queries
constexpr int kL8Width = latent_row_bytes(kLdRank, kLdWidth - kLdRank);    // bytes of a token's row
constexpr float kL8Slack = 12.f, kL8Stand = 3.f;              // how far (log2) a weight may exceed its reference; the reference's
// Tokens of scales below 2^-30 (latents of 0: 2^-100).  Beside latents of 2^30 and more their P would be lost in fp32, and
// with it their weight in the row's sum: it is held 2^100 times as large until the sum has it (64 x 4096 tokens, 128 heads:
// 102.9 -> 103.9 us).
constexpr int kL8Small = kScaleBias - 30;
constexpr int kL8Lift = 100;                                 // (log2)
constexpr uint32_t kL8Piece = kLdTile * 128;                 // 128 bytes of each token: 128 codes, or the rotary channels
constexpr int kL8Pieces = 5, kL8Tiles = 2;
constexpr uint32_t kL8QPiece = 2 * kL8Rows * 128;            // 128 codes of q1 and q2
constexpr uint32_t kL8P = kLdTile * kL8Rows;                 // one of p1, p2, p3
constexpr uint32_t kL8OffQ = kL8Tiles * kL8Pieces * kL8Piece, kL8OffRope = kL8OffQ + 4 * kL8QPiece,
                   kL8OffP = kL8OffRope + kL8Rows * 128, kL8OffSmall = kL8OffP + 2 * 3 * kL8P;
constexpr int kL8Scales = 4;                                 // segments whose rows' scales are held
constexpr uint32_t kL8Smem = 1024 + kL8OffSmall + (3 + 8 + kL8Scales) * kL8Rows * 4 + 2 * kLdTile + 512;
static_assert(kL8Smem <= 232448, "shared memory of a block");
constexpr uint32_t kL8O = 3 * kL8Rows;                       // first TMEM column of O^T, 96 a block of 128 channels

struct L8Args {
    LdArgs a;
    int64_t q_ts, q_hs, page_stride;
    uint32_t by_heads;                          // 2^31 / H, rounded up
    const __nv_bfloat16* q;
    const uint8_t* cache;
};

// kind::f8f6f4 with fp32 D; A e4m3; B e4m3 or (b_wide) e5m2.
__host__ __device__ constexpr uint32_t idesc_f8(int M, int N, int a_mn, int b_mn, int b_wide) {
    return idesc_e4m3(M, N) | ((uint32_t)b_wide << 10) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16);
}
// 16-byte piece c of token row r of a P^T (32-byte swizzle).
__device__ __forceinline__ uint32_t l8_p_at(int r, int c) { return r * 32 + ((c ^ (r >> 2)) & 1) * 16; }

// 8 or 16 columns of a warp's TMEM lanes.
__device__ __forceinline__ void tmem_ld(uint32_t at, float (&f)[16]) { tmem_ld16(at, f); }
__device__ __forceinline__ void tmem_st(uint32_t at, const float (&f)[16]) { tmem_st16(at, f); }
__device__ __forceinline__ void tmem_ld(uint32_t at, float (&f)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=f"(f[0]), "=f"(f[1]), "=f"(f[2]), "=f"(f[3]), "=f"(f[4]), "=f"(f[5]), "=f"(f[6]), "=f"(f[7])
                 : "r"(at));
}
__device__ __forceinline__ void tmem_st(uint32_t at, const float (&f)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
                 ::"r"(at), "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7])
                 : "memory");
}

// Conversions to eight bits by masks and shifts: the conversion instructions take eight cycles of a scheduler each.

template <typename T> __device__ __forceinline__ uint32_t bits_of(T x) {
    uint32_t b;
    memcpy(&b, &x, 4);
    return b;
}
template <typename T> __device__ __forceinline__ T of_bits(uint32_t b) {
    T x;
    memcpy(&x, &b, 4);
    return x;
}

// Four weights to a word each of e5m2 p1, p2, p3.  An e5m2 is the upper byte of a half: rounded to nine significant bits
// (multiples of 2^-22 below 2^-14), a half is the sum of its upper byte, that of the rest times 8, and what is left of
// that.  (A NaN is lost here; it is in the row's sum.)
__device__ __forceinline__ void l8_split(const float* p, uint32_t& w1, uint32_t& w2, uint32_t& w3) {
    const __half2 eight = __half2(__float2half(8.f), __float2half(8.f));
    uint32_t x[2], y[2], z[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t h = (bits_of(__floats2half2_rn(p[2 * i], p[2 * i + 1])) + 0x00020002u) & 0xfffcfffcu;
        x[i] = h & 0xff00ff00u;
        const __half2 r = __hmul2(__hsub2(of_bits<__half2>(h), of_bits<__half2>(x[i])), eight);
        y[i] = bits_of(r) & 0xff00ff00u;
        z[i] = bits_of(__hmul2(__hsub2(r, of_bits<__half2>(y[i])), eight));
    }
    w1 = __byte_perm(x[0], x[1], 0x7531);
    w2 = __byte_perm(y[0], y[1], 0x7531);
    w3 = __byte_perm(z[0], z[1], 0x7531);
}

// Two bf16 channels, 448 at most, times 2^-120, to e4m3 q1 and 16 times the rest q2 (each code in the lower byte of its
// half).  The factor makes e4m3's exponents bf16's, its subnormals too: a code is sign, exponent and three mantissa bits.
// q1 is rounded to nearest, so that the rest is at most 8 of the 128 steps of a bf16 and its code 256 at most.
__device__ __forceinline__ void l8_codes(__nv_bfloat162 t, uint32_t& q1, uint32_t& q2) {
    const __nv_bfloat162 sixteen = __nv_bfloat162(__float2bfloat16(16.f), __float2bfloat16(16.f));
    auto code = [](uint32_t x) { return (x >> 4 & 0x007f007fu) | (x >> 8 & 0x00800080u); };
    const uint32_t top = (bits_of(t) + 0x00080008u) & 0xfff0fff0u;
    q1 = code(top);
    q2 = code(bits_of(__hmul2(__hsub2(t, of_bits<__nv_bfloat162>(top)), sixteen)));
}

// Sixteen codes with 0 in place of those that are NaN (all bits but the sign set).
__device__ __forceinline__ uint4 l8_no_nan(uint4 x) {
    auto keep = [](uint32_t u) { return u & ~((((u & 0x7f7f7f7fu) + 0x01010101u) >> 7 & 0x01010101u) * 255u); };
    return make_uint4(keep(x.x), keep(x.y), keep(x.z), keep(x.w));
}

// Query row `row` (query, head) of sequence n.
__device__ __forceinline__ const __nv_bfloat16* l8_query(const L8Args& b, int n, int row) {
    const int i = (int)((uint64_t)row * b.by_heads >> 31);             // row / H: exact while row H < 2^31
    return b.q + ((int64_t)n * b.a.Lq + i) * b.q_ts + (row - i * b.a.H) * b.q_hs;
}
__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// The warp's maximum of each column to `to`[column].
template <int N>
__device__ __forceinline__ void l8_maxima(const float (&x)[N], float* to, int lane) {
    float mine = 0.f;
#pragma unroll
    for (int c = 0; c < N; ++c) {
        float top;
        asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(top) : "f"(x[c]));
        if (lane == c) mine = top;
    }
    if (lane < N) to[lane] = mine;
}
__device__ __forceinline__ void prefetch_l2_rows(const void* p, uint32_t bytes) {
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}

__device__ __forceinline__ void l8_store(uint8_t* to, const uint32_t (&w)[4]) { *(uint4*)to = make_uint4(w[0], w[1], w[2], w[3]); }
__device__ __forceinline__ void l8_store(uint8_t* to, const uint32_t (&w)[2]) { *(uint2*)to = make_uint2(w[0], w[1]); }

// A query row in registers (16 channels a lane in two vectors) to q1 and q2 there, by a warp, and what a unit of q1 is
// worth.
__device__ __forceinline__ float l8_convert(uint4& x0, uint4& x1, float sc) {
    uint32_t u[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
    uint32_t top = 0;                                      // largest channel's bits, in each half
#pragma unroll
    for (int k = 0; k < 8; ++k) top = __vmaxu2(top, u[k] & 0x7fff7fffu);
    top = max(top & 0xffffu, top >> 16);
    const bool strange = __any_sync(0xffffffffu, top >= 0x7f80u);
    if (strange) {                                         // infinities and NaN: left out here, the row's unit is NaN
        top = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            if ((u[k] & 0x7fffu) >= 0x7f80u) u[k] &= 0xffff0000u;
            if ((u[k] >> 16 & 0x7fffu) >= 0x7f80u) u[k] &= 0xffffu;
            top = __vmaxu2(top, u[k] & 0x7fff7fffu);
        }
        top = max(top & 0xffffu, top >> 16);
    }
    top = __reduce_max_sync(0xffffffffu, top);
    const int e = latent_exponent(top << 16);
    const __nv_bfloat16 inv = __float2bfloat16(__uint_as_float((uint32_t)(127 - e) << 23));
    const __nv_bfloat162 down = __nv_bfloat162(inv, inv),
                         far = __nv_bfloat162(__float2bfloat16(0x1p-120f), __float2bfloat16(0x1p-120f));
    uint32_t q1[4], q2[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        uint32_t lo[2], hi[2];
#pragma unroll
        for (int h = 0; h < 2; ++h)
            l8_codes(__hmul2(__hmul2(of_bits<__nv_bfloat162>(u[2 * k + h]), down), far), lo[h], hi[h]);
        q1[k] = __byte_perm(lo[0], lo[1], 0x6420);
        q2[k] = __byte_perm(hi[0], hi[1], 0x6420);
    }
    x0 = make_uint4(q1[0], q1[1], q1[2], q1[3]);
    x1 = make_uint4(q2[0], q2[1], q2[2], q2[3]);
    return strange ? NAN : __uint_as_float((uint32_t)(127 + e) << 23) * sc;
}
// To shared memory, with two rotary channels a lane.
__device__ __forceinline__ void l8_put(uint8_t* mem, int r, int lane, uint4 q1, uint4 q2, uint32_t rope) {
    const int swz = r & 7;
    uint8_t* to = mem + kL8OffQ + (lane / 8) * kL8QPiece + r * 128 + ((lane & 7) ^ swz) * 16;
    *(uint4*)to = q1;
    *(uint4*)(to + kL8Rows * 128) = q2;
    *(uint32_t*)(mem + kL8OffRope + r * 128 + ((lane / 4) ^ swz) * 16 + lane % 4 * 4) = rope;
}

// Boxes [from, from + count) of a piece, by a warp: operands in uniform registers, 57 cycles a box (80 with a lane for
// each).  Box b's page is in lane b * step.
template <int B>
__device__ __forceinline__ void l8_issue(uint32_t to, const CUtensorMap* map, int x, int row, int page, int step, int from, int box, uint64_t* bar) {
    int z[B];
#pragma unroll
    for (int i = 0; i < B; ++i) z[i] = __shfl_sync(0xffffffffu, page, (from + i) * step);
    if (elect_one()) {
#pragma unroll
        for (int i = 0; i < B; ++i) tma_load_3d_at(to + (from + i) * box * 128, map, x, row, z[i], smem_u32(bar));
    }
    __syncwarp();
}
__device__ __forceinline__ void l8_boxes(uint32_t to, const CUtensorMap* map, int x, int row, int page, int step, int from, int count, int box,
                                         uint64_t* bar) {
    if (count == 1) l8_issue<1>(to, map, x, row, page, step, from, box, bar);
    else if (count == 2) l8_issue<2>(to, map, x, row, page, step, from, box, bar);
    else if (count == 4) l8_issue<4>(to, map, x, row, page, step, from, box, bar);
    else l8_issue<8>(to, map, x, row, page, step, from, box, bar);
}
// Small pages' boxes are issued by two warps, half of them each (64 x 4096 tokens, 64 heads,
// pages of 8 and 16: 73 and 66 us, 64 and 62 so; 37 x 3 queries, 16 heads, pages of 16: 25.0 and 24.1).
__device__ __forceinline__ bool l8_shared(int boxes) { return boxes >= 8; }

// kHalf: rows of a softmax warp, 16, or 8 where there are no more than 16 rows (16 heads, 256 x 200 tokens: 22.2 us, with
// half of the warps idle 23.8; 64 x 16384: 108 and 110.5).
template <int kHalf>
__global__ void __launch_bounds__(kL8Threads, 1)
kda_latent_decode8_tc(const __grid_constant__ CUtensorMap map, const __grid_constant__ L8Args b) {
    constexpr int R = kL8Rows;
    const LdArgs& a = b.a;
    extern __shared__ uint8_t raw[];
    const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u;
    uint8_t* mem = raw + (base - smem_u32(raw));
    float* ref = (float*)(mem + kL8OffSmall);          // [R] softmax references (log2)
    float* fac = ref + R;                              // [R] factors of a moved reference
    int* query = (int*)(fac + R);                      // [R] query a row belongs to
    float* across = (float*)(query + R);               // [4][R] one value a warp and row
    float* sums = across + 4 * R;                      // [4][R]
    float* worth = sums + 4 * R;                       // [kL8Scales][R] what a unit of a row's q1 is worth (log2 scores)
    uint8_t* scales = (uint8_t*)(worth + kL8Scales * R);           // [2][128] bytes of a tile's tokens
    uint64_t* bars = (uint64_t*)(scales + 2 * kLdTile);
    constexpr int kRing = kL8Tiles * kL8Pieces;
    uint64_t *full = bars, *empty = full + kRing, *q_full = empty + kRing, *q_empty = q_full + 1, *s_full = q_empty + 1,
             *s_empty = s_full + 1, *o_full = s_empty + 1, *p_full = o_full + 2, *c_full = p_full + 2, *q_first = c_full + 2, *bars_end = q_first + 1;
    uint32_t* tmem_at = (uint32_t*)bars_end;
    int* range = (int*)(tmem_at + 1);                  // first sequence, its first tile, tiles
    int* fault = range + 3;
    int* gave = fault + 1;                             // [2] a wait of this half of the softmax's warps gave up
    int64_t* range_at = (int64_t*)(((uintptr_t)(gave + 2) + 7) & ~(uintptr_t)7);   // index of the first tile

    const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
    const int group = blockIdx.x, cta = blockIdx.y;
    wait_before();
    // What the range's start hangs on next, were the sequences equally long: the translations at least are then there.
    if (warp >= 11) {
        const int n = (int)((int64_t)cta * a.N / gridDim.y);
        if (warp == 11) {
            if (lane == 0) prefetch_l2(a.table + (int64_t)n * a.max_pages);
        } else {
            for (int r = warp - 12; r < R && group * R + r < a.rows; r += 4)
                if (lane < 9) prefetch_l2(l8_query(b, n, group * R + r) + lane * 64);
        }
    }
    LdWalk w;
    if (warp == 8) {
        // This CTA's range of the tiles of all sequences.  The producer finds it and starts copying; the other
        // warps wait for it at the barrier.
        const int len = lane < a.N ? a.lens[lane] : 0;                 // on its way while the barriers are made
        if (lane < bars_end - bars) {
            const uint64_t* x = bars + lane;
            const int arrivals = x == s_empty || x == p_full || x == p_full + 1 ? 8 : x == q_full ? 4 : x == q_first ? 12 : 1;
            mbar_init(bars + lane, arrivals + (a.drop >> lane & 1));
        }
        if (lane == 0) prefetch_map(&map);
        fence_mbar_init();
        const LdCut cut = ld_cut(a, cta, lane, len);
        if (lane == 0) {
            range[0] = cut.n; range[1] = cut.j; range[2] = cut.count;
            if (cta == 0 && group == 0) a.before[a.N] = cut.total;
            *fault = cut.bad ? kLdBadLen : 0;
            *range_at = cut.at;
            gave[0] = gave[1] = 0;
        }
        __syncwarp();
        asm volatile("bar.arrive 5, %0;" ::"n"(kL8Threads) : "memory");
        w.start(a, cut.n, cut.j, cut.count);
    } else {
        if (warp == 0) { tmem_alloc(tmem_at, 512); tmem_relinquish(); }
        if (threadIdx.x < R) {
            ref[threadIdx.x] = kLdUnset;
            query[threadIdx.x] = min((group * R + (int)threadIdx.x) / a.H, a.Lq - 1);
        }
        tc_fence_before_sync();
        asm volatile("bar.sync 5, %0;" ::"n"(kL8Threads) : "memory");
        tc_fence_after_sync();
        w.start(a, range[0], range[1], range[2]);
    }
    const uint32_t tmem = warp == 8 ? 0 : __shfl_sync(0xffffffffu, *tmem_at, 0);
    const int count = w.left;
    const int row0 = group * R, live = min(R, a.rows - row0);

    auto load_row = [&](int r, uint4& x0, uint4& x1, uint32_t& rope) {
        x0 = x1 = make_uint4(0, 0, 0, 0);
        rope = 0;
        if (r < live) {
            const __nv_bfloat16* from = l8_query(b, w.n, row0 + r);
            x0 = ((const uint4*)from)[2 * lane];
            x1 = ((const uint4*)from)[2 * lane + 1];
            rope = ((const uint32_t*)(from + kLdRank))[lane];
        }
    };
    if (count > 0 && (warp < 8 || warp >= 12)) {                       // the first queries, by twelve warps (by four: 1.5 us later)
        uint4 x[3][2];
        uint32_t rope[3];
        const int first = warp < 8 ? warp : warp - 4;
#pragma unroll
        for (int i = 0; i < 3; ++i) load_row(first + 12 * i, x[i][0], x[i][1], rope[i]);
#pragma unroll 1
        for (int r = first; r < R; r += 12) {
            float unit = 0.f;                                          // (rows that are none are zeros already)
            if (r < live) unit = l8_convert(x[0][0], x[0][1], a.scale * 1.4426950408889634f);
            l8_put(mem, r, lane, x[0][0], x[0][1], rope[0]);
            if (lane == 0) worth[r] = unit;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                x[i][0] = x[i + 1][0];
                x[i][1] = x[i + 1][1];
                rope[i] = rope[i + 1];
            }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(q_first);
    }

    if (warp == 8) {                                                   // ---------------- producer
        const int box = min(a.page_size, kLdTile), boxes = kLdTile / box, shift = __ffs(a.page_size) - 1;
        bool ok = true, bad_page = false;
        // A lane for each box of tokens: its page, asked for a tile ahead.  Pages behind the length, and bad ones, read
        // as zeros.
        int len = 0, row = 0, page = a.num_pages;
        bool some = false;
        auto ask = [&]() {
            if (w.left <= 0) return;
            if (w.first) len = ld_len(a, w.n);
            const int t = w.j * kLdTile + lane * box;
            some = lane < boxes && t < len;
            row = t & (a.page_size - 1);
            if (some) page = a.table[(int64_t)w.n * a.max_pages + (t >> shift)];
        };
        ask();
        for (int j = 0; j < count && ok; ++j) {
            const int p = page, here = some ? p : a.num_pages, at_row = some ? row : 0;
            const bool asked = some;
            w.next(a);
            ask();
            const bool bad = asked && (here < 0 || here >= a.num_pages);
            bad_page |= bad;
            const int from_page = bad ? a.num_pages : here, in_page = uniform(at_row);     // (not 0: a single box)
            const int at = j % kL8Tiles * kL8Pieces;
            for (int k = 0; k < kL8Pieces; ++k) {
                const int u = k == 0 ? 4 : k - 1;                      // the rotary channels first, they are free first
                if (!(ok = mbar_wait_warp(&empty[at + u], (j / kL8Tiles + 1) & 1))) break;   // (a fresh barrier counts as emptied)
                if (elect_one()) mbar_arrive_expect_tx(&full[at + u], kL8Piece);
                __syncwarp();
                l8_boxes(base + (at + u) * kL8Piece, &map, u * 128, in_page, from_page, 1, 0, l8_shared(boxes) ? boxes / 2 : boxes, box, &full[at + u]);
            }
            // The next tile's rows, dense in a page, to L2: there is no place in shared memory for them yet (64 x up to
            // 16384 tokens, 32 heads 76.5 -> 74.2 us; two or three tiles ahead 77 and 80; 64 x 4096, 64 heads,
            // pages of 16: 62.4 -> 60.5).  Not where issuing many small copies bounds the tiles (pages of 8)
            if (boxes <= 8 && w.left > 0 && some && page >= 0 && page < a.num_pages)
                prefetch_l2_rows(b.cache + page * b.page_stride + (int64_t)row * kL8Width, box * kL8Width);
        }
        if (bad_page) atomicOr(fault, kLdBadPage);
        if (!ok) atomicOr(fault, kLdLate);
    } else if (warp == 9) {                                            // ---------------- S^T
        constexpr uint32_t codes = idesc_f8(128, 2 * R, 0, 0, 0), rope = idesc_bf16(128, R);
        const uint64_t dq = sdesc_k_sw128(base + kL8OffQ), dr = sdesc_k_sw128(base + kL8OffRope);
        uint32_t seg = 0;
        bool ok = true;
        for (int j = 0; j < count && ok; ++j, w.next(a)) {
            if (w.first) {
                ok = seg == 0 ? mbar_wait_warp(q_first, 0) : mbar_wait_warp(q_full, (seg - 1) & 1);
                ++seg;
            }
            const int at = j % kL8Tiles * kL8Pieces;
            const uint32_t here = (j / kL8Tiles) & 1;
            bool ready = true;                                         // the tile is there: no waits behind that for S
#pragma unroll
            for (int k = 0; k < kL8Pieces; ++k) ready &= mbar_test_wait(&full[at + k], here);
            ready = __all_sync(0xffffffffu, ready);
            if (ok && j >= 1) ok = mbar_wait_warp(s_empty, (j - 1) & 1);           // S_{j-1} is read
            // Otherwise the rotary channels and the first codes, two more pieces, the last: a wait each
#pragma unroll
            for (int k = 0; k < 3 && ok; ++k) {
                uint64_t* const two[2] = {&full[at + (k == 0 ? 4 : k == 1 ? 1 : 3)], &full[at + (k == 0 ? 0 : k == 1 ? 2 : 3)]};
                if (!ready && !(ok = mbar_wait_all(two, {here, here}))) break;
                tc_fence_after_sync();
                const uint64_t da = sdesc_k_sw128(base + at * kL8Piece);
                if (elect_one()) {
                    if (k == 0) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) mma_bf16_ss(tmem + 2 * R, da + 4 * (kL8Piece / 16) + 2 * i, dr + 2 * i, rope, i > 0);
                        mma_commit(&empty[at + 4]);
                    }
#pragma unroll
                    for (int u = k == 0 ? 0 : 2 * k - 1; u < (k == 0 ? 1 : k == 1 ? 3 : 4); ++u)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            mma_f8_ss(tmem, da + u * (kL8Piece / 16) + 2 * i, dq + u * (kL8QPiece / 16) + 2 * i, codes, u > 0 || i > 0);
                    if (k == 2) {
                        mma_commit(s_full);
                        if (w.last()) mma_commit(q_empty);
                    }
                }
                __syncwarp();
            }
        }
        if (!ok) atomicOr(fault, kLdLate);
    } else if (warp == 10) {                                           // ---------------- O^T += C^T P^T
        constexpr uint32_t wide = idesc_f8(128, 3 * R, 1, 1, 1);
        bool ok = true;
        for (int j = 0; j < count && ok; ++j, w.next(a)) {
            const int at = j % kL8Tiles * kL8Pieces;
            const uint32_t here = (j / kL8Tiles) & 1;                  // (the first product has awaited them too: no time is lost)
            uint64_t* const pieces[4] = {&full[at], &full[at + 1], &full[at + 2], &full[at + 3]};
            if (!(ok = mbar_wait_all(pieces, {here, here, here, here}) && mbar_wait_warp(&p_full[j & 1], (j >> 1) & 1))) break;
            tc_fence_after_sync();
            // p1, p2 and p3 lie a swizzle atom of 32 rows apart each; 8 tokens 256 bytes
            const uint64_t dp = sdesc(base + kL8OffP + (j & 1) * 3 * kL8P, kL8P, 256, 6);
            if (elect_one()) {
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const uint64_t da = sdesc(base + (at + u) * kL8Piece, kL8Piece, 1024, 2);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        mma_f8_ss(tmem + kL8O + u * 3 * R, da + i * (4096 / 16), dp + i * (1024 / 16), wide, !w.first || i > 0);
                    mma_commit(&empty[at + u]);
                }
                mma_commit(&o_full[j & 1]);
            }
            __syncwarp();
        }
        if (!ok) atomicOr(fault, kLdLate);
    } else if (warp == 11) {                                           // ---------------- scales
        // Four tokens' bytes a lane, 0 (2^-127) where there is nothing, also behind the length in the same four (a byte of
        // 255 there, as memory that nothing has cleared holds, would be 2^128, and 0 times that); and half of small pages'
        // boxes.
        const int shift = __ffs(a.page_size) - 1, box = min(a.page_size, kLdTile), boxes = kLdTile / box;
        // (keep is applied where the word is used: at its load, the boxes would wait for that.  64 x 8192 tokens, 16 heads,
        // pages of 16: 63.5 us, at the load 68.9)
        int len = 0, page = a.num_pages;
        uint32_t keep = 0;
        auto fetch = [&](const LdWalk& x) -> uint32_t {
            const int t = x.j * kLdTile + 4 * lane;
            page = a.num_pages;
            if (x.left <= 0) return 0;
            if (x.first) len = ld_len(a, x.n);
            if (t >= len) return 0;
            const int p = a.table[(int64_t)x.n * a.max_pages + (t >> shift)];
            if (p < 0 || p >= a.num_pages) return 0;
            page = p;
            keep = len - t < 4 ? (1u << 8 * (len - t)) - 1 : ~0u;
            return *(const uint32_t*)(b.cache + p * b.page_stride + (int64_t)a.page_size * kL8Width + (t & (a.page_size - 1)));
        };
        bool ok = true;
        uint32_t now = fetch(w);
        for (int j = 0; j < count && ok; ++j) {
            if (l8_shared(boxes)) {
                const int at = j % kL8Tiles * kL8Pieces;
                for (int k = 0; k < kL8Pieces; ++k) {                  // as the producer
                    const int u = k == 0 ? 4 : k - 1;
                    if (!(ok = mbar_wait_warp(&empty[at + u], (j / kL8Tiles + 1) & 1))) break;
                    l8_boxes(base + (at + u) * kL8Piece, &map, u * 128, 0, page, box / 4, boxes / 2, boxes / 2, box, &full[at + u]);
                }
                if (!ok) break;
            }
            if (j >= 2) ok = mbar_wait_warp(&p_full[j & 1], ((j - 2) >> 1) & 1);    // tile j - 2's bytes are read
            if (!ok) break;
            *(uint32_t*)(scales + (j & 1) * kLdTile + 4 * lane) = now & keep;
            __syncwarp();
            if (lane == 0) mbar_arrive(&c_full[j & 1]);
            w.next(a);
            now = fetch(w);
        }
        if (!ok) atomicOr(fault, kLdLate);
    } else if (warp >= 12) {                                           // ---------------- queries
        const float sc = a.scale * 1.4426950408889634f;
        uint32_t seg = 1;
        bool ok = true;
        for (int j = 0; j < count && ok; ++j, w.next(a)) {
            if (!w.first || j == 0) continue;                          // (the first segment's are done)
            // All rows' loads at once; then one after another by the same instructions (others would be cold), in registers
            // until the last segment's products are done.
            uint4 x[R / 4][2];
            uint32_t rope[R / 4];
#pragma unroll
            for (int i = 0; i < R / 4; ++i) load_row(warp - 12 + 4 * i, x[i][0], x[i][1], rope[i]);
            // (worth: that of the segment four before was read before its last scores were replaced)
#pragma unroll 1
            for (int k = 0; k < R / 4; ++k) {
                float unit = 0.f;
                if (warp - 12 + 4 * k < live) unit = l8_convert(x[0][0], x[0][1], sc);
                if (lane == 0) worth[seg % kL8Scales * R + warp - 12 + 4 * k] = unit;
                const uint4 q1 = x[0][0], q2 = x[0][1];
                const uint32_t same = rope[0];
#pragma unroll
                for (int i = 0; i + 1 < R / 4; ++i) {                  // (round by one: in order again at the end)
                    x[i][0] = x[i + 1][0];
                    x[i][1] = x[i + 1][1];
                    rope[i] = rope[i + 1];
                }
                x[R / 4 - 1][0] = q1;
                x[R / 4 - 1][1] = q2;
                rope[R / 4 - 1] = same;
            }
            // (a whole segment, which may take seconds: up to 40, unless another warp gave up)
            ok = mbar_wait_warp(q_empty, (seg - 1) & 1);
#pragma unroll 1
            for (int k = 1; k < 20 && !ok && !(uniform(*(volatile int*)fault) & kLdLate); ++k) ok = mbar_wait_warp(q_empty, (seg - 1) & 1);
            if (!ok) break;
#pragma unroll
            for (int i = 0; i < R / 4; ++i) l8_put(mem, warp - 12 + 4 * i, lane, x[i][0], x[i][1], rope[i]);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(q_full);
            ++seg;
        }
        if (!ok) atomicOr(fault, kLdLate);
    } else {                                                           // ---------------- softmax
        const int half = warp >> 2, part = warp & 3, r0 = half * kHalf, thread = threadIdx.x & 127;
        const bool idle = r0 >= live;                                  // rows that are none: nothing of theirs is read
        const uint32_t vote = half ? 3 : 1, meet = half ? 4 : 2;
        // A warp whose wait gave up says so at a vote that the others come to next, and all four leave there.
        auto leave = [&]() {
            if (lane == 0) *(volatile int*)(gave + half) = 1;
            __syncwarp();
            bar_and_id(vote, 128, false);
        };
        auto sync = [&]() { asm volatile("bar.sync %0, 128;" ::"r"(meet) : "memory"); };
        const uint32_t lanes = tmem_addr(tmem, 32 * part, 0);
        const float sc = a.scale * 1.4426950408889634f;
        float l[kHalf];
#pragma unroll
        for (int c = 0; c < kHalf; ++c) l[c] = 0.f;
        bool ok = true;
        uint32_t seg = 0;
        int len = 0;
        if (count > 0) len = ld_len(a, w.n);
        for (int j = 0; j < count; ++j) {
            if (w.first) {
                if (w.j == 0 && threadIdx.x == 0 && group == 0) a.before[w.n] = *range_at + j;
                ++seg;
            }
            if (!(ok = mbar_wait_warp(&c_full[j & 1], (j >> 1) & 1))) {
                leave();
                break;
            }
            const int token = w.j * kLdTile + thread;
            // (0 in pages that were cleared, not written: 2^127 for `down` would be too much for the sum)
            const int byte = max((int)scales[(j & 1) * kLdTile + thread], kScaleLow + kScaleBias);
            const float two = __uint_as_float((uint32_t)byte << 23), e = (float)(byte - kScaleBias);
            const bool small = byte < kL8Small;
            const float stand = kL8Stand + (small ? kL8Lift : 0);
            // (also the products of the tile before last are complete then, whose weights this tile's replace: its codes
            // came to where theirs were)
            static_assert(kL8Tiles == 2, "as many buffers for the weights");
            if (!(ok = mbar_wait_warp(s_full, j & 1))) {
                leave();
                break;
            }
            tc_fence_after_sync();
            // y: log2 of the weight times 2^e
            float y[kHalf];
            if (!idle) {
                const float* unit = worth + (seg - 1) % kL8Scales * R + r0;
                float d2[kHalf], dr[kHalf];
                tmem_ld(lanes + r0, y);
                tmem_ld(lanes + R + r0, d2);
                tmem_ld(lanes + 2 * R + r0, dr);
                tmem_wait_ld();
                tmem_ready(y);
                tmem_ready(d2);
                tmem_ready(dr);
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(s_empty);
#pragma unroll
                for (int c = 0; c < kHalf; ++c) y[c] = fmaf(fmaf(d2[c], 0.0625f, y[c]), two * unit[c], fmaf(dr[c], sc, e));
            } else if (lane == 0) {
                mbar_arrive(s_empty);
            }
            if (!idle && w.end() > len - a.Lq) {                          // some row does not see some token
                // Weight 0 times a NaN code of a token that other rows see: make that 0 too.  Those have it in their sums.
                // (A NaN code makes the scores of every row NaN, so that they tell where to look.)
                const bool strange = token > len - a.Lq && token < len && !(y[0] == y[0]);
                if (__any_sync(0xffffffffu, strange)) {
                    const int from = 2 * half, pieces = live <= kHalf ? 4 : 2;     // the other half is idle: all of them
                    const int at = j % kL8Tiles * kL8Pieces + from;
#pragma unroll 1
                    for (int u = 0; u < pieces && ok; ++u) {           // (complete; awaited for the copies to be seen here)
                        ok = mbar_wait_warp(&full[at + u], (j / kL8Tiles) & 1);
#pragma unroll 1
                        for (int i = 0; i < 8 && strange; ++i) {
                            uint4* x = (uint4*)(mem + (at + u) * kL8Piece + thread * 128 + i * 16);
                            *x = l8_no_nan(*x);
                        }
                    }
                    if (!ok) {
                        leave();
                        break;
                    }
                }
#pragma unroll
                for (int c = 0; c < kHalf; ++c)
                    if (token > len - a.Lq + query[r0 + c]) y[c] = -INFINITY;
            }
            // The weights under the references as they are, and under new ones where some weight is too large for that or
            // there are none yet: the same instructions, others would be cold.
            float p[kHalf];
#pragma unroll 1
            for (bool moved = false;; moved = true) {
                bool over = w.first && !moved && !idle;
                if (!idle && !over) {
#pragma unroll
                    for (int c = 0; c < kHalf; c += 4) {
                        const float4 m = *(const float4*)(ref + r0 + c);
                        const float d[4] = {y[c] - m.x, y[c + 1] - m.y, y[c + 2] - m.z, y[c + 3] - m.w};
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            over |= d[k] > kL8Slack;
                            p[c + k] = ex2(d[k] + stand);
                        }
                    }
                } else {                                               // (no register is held for the ones before)
#pragma unroll
                    for (int c = 0; c < kHalf; ++c) p[c] = 0.f;
                }
                if (moved || bar_and_id(vote, 128, !over)) break;
                // Move the references to the maxima
                if (*(volatile int*)(gave + half)) {
                    ok = false;
                    break;
                }
                l8_maxima(y, across + part * R + r0, lane);
                sync();
                if (thread < kHalf) {
                    const int c = r0 + thread;
                    const float old = w.first ? kLdUnset : ref[c];
                    const float now = fmaxf(old, fmaxf(fmaxf(across[c], across[R + c]),
                                                       fmaxf(across[2 * R + c], across[3 * R + c])));
                    ref[c] = now;
                    fac[c] = ex2(old - now);
                }
                sync();
                if (w.first) continue;                                 // (no sums and no O^T yet)
                float f[kHalf];
#pragma unroll
                for (int c = 0; c < kHalf; ++c) {
                    f[c] = fac[r0 + c];
                    l[c] *= f[c];
                }
                // O^T, once the products into it are complete
                ok = bar_and_id(vote, 128, mbar_wait_spin(&o_full[(j - 1) & 1], ((j - 1) >> 1) & 1));
                if (!ok) break;
                tc_fence_after_sync();
#pragma unroll 1
                for (int b = 0; b < 4; ++b) {
                    const uint32_t at = lanes + kL8O + b * 3 * R + r0;
                    float o1[kHalf], o2[kHalf], o3[kHalf];
                    tmem_ld(at, o1);
                    tmem_ld(at + R, o2);
                    tmem_ld(at + 2 * R, o3);
                    tmem_wait_ld();
                    tmem_ready(o1);
                    tmem_ready(o2);
                    tmem_ready(o3);
#pragma unroll
                    for (int c = 0; c < kHalf; ++c) {
                        o1[c] *= f[c];
                        o2[c] *= f[c];
                        o3[c] *= f[c];
                    }
                    tmem_st(at, o1);
                    tmem_st(at + R, o2);
                    tmem_st(at + 2 * R, o3);
                }
                tmem_wait_st();
            }
            if (!ok) break;
            if (!idle) {
                const float down = __uint_as_float((uint32_t)((small ? 254 - kL8Lift : 254) - byte) << 23);   // 2^-e: back from P to p
                const float back = small ? 0x1p-100f : 1.f;
                uint32_t p1[kHalf / 4], p2[kHalf / 4], p3[kHalf / 4];
#pragma unroll
                for (int i = 0; i < kHalf / 4; ++i) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        l[4 * i + k] = fmaf(p[4 * i + k], down, l[4 * i + k]);
                        p[4 * i + k] *= back;
                    }
                    l8_split(p + 4 * i, p1[i], p2[i], p3[i]);
                }
                uint8_t* to = mem + kL8OffP + (j & 1) * 3 * kL8P + l8_p_at(thread, r0 / 16) + r0 % 16;
                l8_store(to, p1);
                l8_store(to + kL8P, p2);
                l8_store(to + 2 * kL8P, p3);
            }
            // Weight 0 times what lies behind the length: make that 0, half of the codes each half of the warps
            if (token >= len) {
                uint8_t* at = mem + ((j % kL8Tiles) * kL8Pieces + 2 * half) * kL8Piece + thread * 128;
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int i = 0; i < 8; ++i) *(uint4*)(at + u * kL8Piece + ((i + thread) & 7) * 16) = make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_smem();
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_full[j & 1]);
            const LdWalk at = w;
            w.next(a);
            if (!at.last()) continue;

            // end of a segment: sums across the tokens' threads, then O^T out
            if (w.left > 0) len = ld_len(a, w.n);
            ld_columns<kHalf, false>(l, sums + part * R + r0, lane);
#pragma unroll
            for (int c = 0; c < kHalf; ++c) l[c] = 0.f;
            ok = bar_and_id(vote, 128, mbar_wait_spin(&o_full[j & 1], (j >> 1) & 1));
            if (!ok) break;
            tc_fence_after_sync();
            const bool whole = at.from == 0 && at.j + 1 == at.tiles;
            float* dst = a.parts + ((size_t)(cta * gridDim.x + group) * 2 + (at.from == 0)) * R * kLdPart;
            if (thread < kHalf) {
                const int c = r0 + thread;
                const float total = (sums[c] + sums[R + c]) + (sums[2 * R + c] + sums[3 * R + c]);
                if (whole) {
                    fac[c] = total > 0.f ? 1.f / total : (total == 0.f ? 0.f : total);
                    if (c < live && a.lse) a.lse[(size_t)at.n * a.rows + row0 + c] =
                        total == 0.f ? -INFINITY : (ref[c] - kL8Stand + log2f(total)) * 0.6931471805599453f;
                } else {
                    dst[c * kLdPart + kLdRank] = ref[c] - kL8Stand;
                    dst[c * kLdPart + kLdRank + 1] = total;
                }
            }
            sync();
#pragma unroll 1
            for (int b = 0; b < 4 && !idle; ++b) {
                const int ch = b * 128 + thread;
                float o[kHalf], o2[kHalf], o3[kHalf];
                const uint32_t from = lanes + kL8O + b * 3 * R + r0;
                tmem_ld(from, o);
                tmem_ld(from + R, o2);
                tmem_ld(from + 2 * R, o3);
                tmem_wait_ld();
                tmem_ready(o);
                tmem_ready(o2);
                tmem_ready(o3);
#pragma unroll
                for (int c = 0; c < kHalf; ++c) o[c] = fmaf(fmaf(o3[c], 0.125f, o2[c]), 0.125f, o[c]);
                if (whole) {
                    __nv_bfloat16* out = a.out + ((size_t)at.n * a.rows + row0 + r0) * kLdRank + ch;
                    if (r0 + kHalf <= live) {
#pragma unroll
                        for (int c = 0; c < kHalf; ++c) out[(size_t)c * kLdRank] = __float2bfloat16_rn(o[c] * fac[r0 + c]);
                    } else {
#pragma unroll
                        for (int c = 0; c < kHalf; ++c)
                            if (r0 + c < live) out[(size_t)c * kLdRank] = __float2bfloat16_rn(o[c] * fac[r0 + c]);
                    }
                } else {                                               // (dead rows too: a condition a store costs more)
#pragma unroll
                    for (int c = 0; c < kHalf; ++c) dst[(r0 + c) * kLdPart + ch] = o[c];
                }
            }
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
    follow_me();
    if (warp == 0) tmem_dealloc(tmem, 512);
    if (threadIdx.x == 0) a.cta_status[cta * gridDim.x + group] = *fault;
}

// ------------------------------------------------------------------- host
bool latent_decode8_tc_takes(int dtype, int dk, int dr, int H, int Lq, int page_size) {
    return dtype == KDA_BF16 && dk == kLdRank && dr == kLdWidth - kLdRank && page_size >= 8 &&
           (page_size & (page_size - 1)) == 0 && (int64_t)Lq * H <= 32 * 1024;
}
size_t latent_decode8_tc_bytes(int N, int Lq, int H, int page_size, int max_pages) {
    return N > 0 ? ld_plan(N, Lq, H, page_size, max_pages, kL8Rows).bytes : 0;
}
// What the tensor map and the vectors need of the call's tensors.
bool latent_decode8_tc_aligned(const LatentDecodeArgs& d) {
    return (((uintptr_t)d.q | (uintptr_t)d.cache | (uintptr_t)d.out) & 15) == 0 &&
           (d.q_ts % 8 == 0 || (int64_t)d.N * d.Lq == 1) && (d.q_hs % 8 == 0 || d.H == 1) && d.num_pages > 0 &&
           d.page_stride < (1ll << 39);
}

template <int kHalf>
static cudaError_t l8_launch(const LdPlan& p, const CUtensorMap& map, const L8Args& b, cudaStream_t stream) {
    static PerDevice memory_set;
    int device = 0, set = 0;
    cudaError_t err = cudaGetDevice(&device);
    if (err == cudaSuccess) err = memory_set.get(device, set, [](int& done) {
        done = 1;
        return cudaFuncSetAttribute(kda_latent_decode8_tc<kHalf>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kL8Smem);
    });
    if (err != cudaSuccess) return err;
    return launch_behind(kda_latent_decode8_tc<kHalf>, dim3(p.groups, p.G), kL8Threads, kL8Smem, stream, map, b);
}

cudaError_t latent_decode8_tc_launch(const LatentDecodeArgs& d, cudaStream_t stream) {
    const LdPlan p = ld_plan(d.N, d.Lq, d.H, d.page_size, d.max_pages, kL8Rows);
    L8Args b;
    LdArgs& a = b.a;
    a.N = d.N; a.H = d.H; a.Lq = d.Lq; a.rows = d.Lq * d.H; a.page_size = d.page_size; a.num_pages = d.num_pages;
    a.max_pages = d.max_pages; a.scale = d.scale; a.table = d.table; a.lens = d.lens; a.out = (__nv_bfloat16*)d.out;
    a.lse = d.lse; a.status = d.status; a.cta_status = (int32_t*)d.scratch; a.G = p.G;
    a.before = (int64_t*)((char*)d.scratch + p.before);
    a.parts = (float*)((char*)d.scratch + p.parts);
    // the barriers' order: full, empty, q_full, q_empty, s_full, s_empty, o_full [2], p_full [2], c_full [2], q_first
    constexpr int kAt = 2 * kL8Tiles * kL8Pieces;
    constexpr uint32_t kDrops[6] = {0, (1u << kAt / 2) - 1, 1u << (kAt + 2), 3u << (kAt + 4), 3u << (kAt + 6), 1u << kAt | 7u << (kAt + 8)};
    a.drop = kDrops[d.drop];
    b.by_heads = (uint32_t)(((1ull << 31) + d.H - 1) / d.H);
    b.q = (const __nv_bfloat16*)d.q; b.q_ts = d.q_ts; b.q_hs = d.q_hs;
    b.cache = (const uint8_t*)d.cache; b.page_stride = d.page_stride;
    CUtensorMap map;
    const uint64_t dims[3] = {(uint64_t)kL8Width, (uint64_t)d.page_size, (uint64_t)d.num_pages};
    const uint64_t strides[2] = {(uint64_t)kL8Width, (uint64_t)d.page_stride};
    const uint32_t box[3] = {128, (uint32_t)(d.page_size < kLdTile ? d.page_size : kLdTile), 1};
    if (!make_map(&map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, d.cache, dims, strides, box)) return cudaErrorInvalidValue;
    const cudaError_t err = a.rows <= 16 ? l8_launch<8>(p, map, b, stream) : l8_launch<16>(p, map, b, stream);
    return err != cudaSuccess ? err : latent_decode_join_launch(a, kL8Rows, p.groups, stream);
}

}  // namespace kda
