// Decode attention in latent space over published rows of packed records
// (hs_packed_attention).
//
// For a request's queries q [heads][576] and its k rows of 416 bytes, each 512
// latent values in 4 bits with 32 scales and 64 others in bf16:
//   out = softmax(scale q K^T) V,  K the 576 values of a row, V its first 512.
// 2176 flops and 26 bytes / heads a row and head: bound by HBM up to about 50
// heads, by the tensor cores beyond.
//
// Work split: a cluster of C CTAs takes one request and up to 64 of its heads,
// each CTA a contiguous range of the rows; the partial results are joined
// through the cluster's shared memory in a fixed order.
//
// The products (tcgen05) have the rows, then the dimensions, as M = 128 and the
// heads as N: S^T = K Q^T and O^T += V^T P^T, so that few heads cost little.  A
// tile of 128 rows lies in shared memory once, in f16, as nine chunks of 64
// dimensions; the second product reads the same chunks the other way round.
//   warps 0-7   load the codes from memory into registers, a tile ahead, and write
//               them as f16 into the chunks that the tile before has left; in a
//               warp the four lanes l, l + 8, l + 16, l + 24 share a row, so that
//               eight consecutive lanes write one column of eight rows (no bank
//               twice) and a load still takes 128 bytes of each;
//   warps 8-15  the queries, then the softmax: a thread per row and half of the heads
//               reads its scores from TMEM and writes P^T as f16;
//   warp 16     one thread issues the products;
//   warp 17     brings the 64 others of the rows straight into their chunk (TMA),
//               up to 32 heads one of two chunks, a tile ahead.  With more than 48
//               heads there is no room for P beside the queries: P then lies over
//               the chunk, and warps 0-7 bring the others;
//   the others  ask for later tiles' rows in L2, as a load from memory takes longer
//               than a tile does.
// Each role has its own part of the start too, so that no register of one is held
// through another's: the rows do not wait for the queries, and with spilled
// registers they would be waited for before the barrier (32 x 2048 rows at 128
// heads 51.4 us, 45.0 without).
//
// Measured: 64 x 2048 rows at 16 heads 28.2 us, at 32 heads 32.2; 32 x 2048 at 128
// heads 42.4.  At 16 heads a tile takes 2.5 us, of which its loads are about half a
// microsecond (all rows from cache: 23.7 us a call, 27.0 at 32 heads); a loop of the
// loads alone takes 2.2 a tile.  What bounds the rest, 147 KB written to shared
// memory as f16 or the 68 products (2.1 to 2.2 if an operand of 128 x 16 keeps each
// at the 64 cycles of a full one, which was not measured), is not known.  At 64 heads
// a tile takes 3.6: scores 0.7 behind the last rows, softmax 0.9, outputs and the next
// rows 2, one after the other: a second tile of 128 rows does not fit.  Start and join
// take 8 us of a call, 11 at 128 heads.
// Other ways, 64 x 2048 at 16 heads and 32 x 2048 at 128: warp-level products on
// the 4-bit rows in registers, whose conversions keep an MMA at 12 cycles instead
// of 8, 28.3 and 88 us; rows and softmax by the same eight warps, whose registers
// do not suffice, 36 and 78; all rows brought by one warp's TMA, 39.7; four warps
// of softmax, 0.3 and 2.5 us more; P as heads of rows, stored value by value, 0.3 and
// 0.9 more; the sums by the softmax instead of by products would save 0.15 and 0.3
// and cost a register for every head.
//
// A value is code * scale, 2 and 4 significant bits: exact in f16.  So are the
// queries' latent parts, scaled by a power of two per head that puts their largest
// near 2^13 (bf16's 8 bits; what falls below 2^-24 then is less than 2^-37 of it).
// The other parts stay in bf16 and get the same factor, less the rows' shift, so
// that one accumulator takes both; where that would put them past 2^81 the factor is
// smaller.
//
// The maximum that exponents are taken from is that of the first tile, and rises
// when a row exceeds it by 2^8, for the eight heads around: only then are maxima
// formed over the rows and O rescaled (32 x 2048 rows at 128 heads 42.4 us, 44.1 for
// all heads at once).  P is rounded to f16 with 2^7 as its unit (so at most 2^15):
// half a step is 2^-11 of a probability down to 2^-21, and 2^-32 below.  Scores,
// maxima, sums and outputs are fp32.
//
// The sums come from the products too, as ones times P^T: that keeps them out of
// the softmax's registers, which hold no score longer than its P takes.
//
// TMEM columns: O^T of dimensions [128 i, 128 i + 128) at i * N, scores at 256, sums
// (the same in every lane) at 384, the ones at 448.
//
// Every wait gives up after a second: the outputs become NaN and
// HS_ATTN_STATUS_TIMEOUT is set (hs_attention_status); products in flight are
// waited for, with the same limit, before the CTA leaves.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <mutex>

#include <cooperative_groups.h>

#include "barriers.cuh"
#include "hs.h"
#include "hs_internal.cuh"
#include "tensor_core.cuh"

namespace hs {
namespace {

namespace cg = cooperative_groups;

constexpr int kTileRows = 128;
constexpr int kAhead = 4;                    // tiles
constexpr int kPackedThreads = 640;
constexpr int kMaxSplits = 16;
constexpr int kMaxN = 64;                    // heads of a CTA
constexpr int kScales = 256, kOthers = 288;  // offsets in a row
constexpr float kUnit = 7.f;                 // log2 of what P is scaled by
constexpr float kRise = 8.f;                 // log2 of how far it may pass that
constexpr float kNoMax = -3.402823466e38f;   // before any row; finite, so that a score of -inf stays below it
constexpr int kUnits = 16;                   // of 32 dimensions, dealt to the CTAs of a cluster for the join

constexpr int kColS = 256, kColL = 384, kColOnes = 448;  // of TMEM

constexpr uint32_t kChunk = kTileRows * 128;              // 64 dimensions of a tile
constexpr uint32_t kOffQ = 9 * kChunk;                    // nine chunks of N rows of 128 bytes
// P over the ninth chunk, which the scores have used by then, or behind the queries
// where they leave room; the ninth chunk's next rows can then be on their way early,
// and with up to 32 heads there is room for two tiles' ninth chunks
__host__ __device__ constexpr bool own_p(int n) { return n <= 48; }
__host__ __device__ constexpr uint32_t off_p(int n) { return own_p(n) ? kOffQ + 9 * n * 128 : 8 * kChunk; }
constexpr uint32_t kPBytes = kTileRows * 128;             // rows of 64 heads, f16
__host__ __device__ constexpr int others_chunks(int n) { return n <= 32 ? 2 : 1; }
__host__ __device__ constexpr uint32_t off_others(int n, int b) { return b == 0 ? 8 * kChunk : off_p(n) + kPBytes; }
constexpr uint32_t kOffBack = kOffQ + 9 * kMaxN * 128;    // [64] from products to scores
constexpr uint32_t kOffBase = kOffBack + kMaxN * 4;       // [64] the maxima, less kUnit
constexpr uint32_t kOffTop = kOffBase + kMaxN * 4;        // [warp][64] of a tile
constexpr uint32_t kOffMl = kOffTop + 4 * kMaxN * 4;      // [kMaxSplits][64] (m, l)
// chunks_full[2], others_full[2], others_free[2], pv_done[2], s_full, p_ready, drained
constexpr uint32_t kOffBar = kOffMl + kMaxSplits * kMaxN * 8;
constexpr int kBars = 11;
constexpr uint32_t kOffWord = kOffBar + 8 * kBars;        // TMEM address, abort flag, tiles begun; [8] from 4 on
constexpr int kWordAbove = 4;                             // eights of heads past the limit, of each softmax warp
constexpr uint32_t kSmem = kOffWord + 48;
static_assert(kSmem <= 232448, "fits an SM");
static_assert(kOffBar % 8 == 0 && kOffWord % 8 == 0 && kOffMl % 8 == 0, "aligned");
static_assert(kPBytes <= kChunk, "P fits a chunk");
static_assert(off_p(48) + kPBytes <= kOffBack && off_p(16) % 1024 == 0 && off_p(48) % 1024 == 0,
              "P fits behind the queries");
static_assert(off_others(32, 1) + kChunk <= kOffBack && off_others(16, 1) % 1024 == 0 && off_others(32, 1) % 1024 == 0,
              "a second ninth chunk fits behind P");
// behind the last tile: parts for the join over the chunks and the queries
constexpr int kMaxParts = 24;                // units of all CTAs' parts in a CTA
constexpr uint32_t kOffWts = kOffBack - kMaxSplits * kMaxN * 4;  // [kMaxSplits][N] their weights
static_assert(kMaxParts * 32 * kMaxN * 4 <= kOffWts && kOffWts % 16 == 0, "parts and weights fit");

__device__ uint32_t g_packed_status;

// From column x on, a box of four rows of the map's tensor, one after the other.
__device__ __forceinline__ void gather4(uint32_t dst, const CUtensorMap *map, int x, const int (&row)[4],
                                        uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cta.global.tile::gather4.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
        "l"(map), "r"(x), "r"(row[0]), "r"(row[1]), "r"(row[2]), "r"(row[3]), "r"(bar)
        : "memory");
}

__device__ __forceinline__ uint32_t scales2(uint32_t two) {
    uint32_t r;
    asm("{\n\t.reg .b16 x, y;\n\tmov.b32 {x, y}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, x;\n\t}" : "=r"(r) : "r"(two));
    return r;
}
// Eight codes to eight f16, times a scale in both halves.
__device__ __forceinline__ void values8(uint32_t codes, uint32_t scale, uint32_t *v) {
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "mov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, d;\n\t"
        "mul.rn.f16x2 %0, %0, %5;\n\t"
        "mul.rn.f16x2 %1, %1, %5;\n\t"
        "mul.rn.f16x2 %2, %2, %5;\n\t"
        "mul.rn.f16x2 %3, %3, %5;\n\t}"
        : "=&r"(v[0]), "=&r"(v[1]), "=&r"(v[2]), "=&r"(v[3])
        : "r"(codes), "r"(scale));
}
__device__ __forceinline__ void load16(uint32_t *v, const void *p) {
    asm volatile("ld.global.nc.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                 : "l"(p));
}
__device__ __forceinline__ void load32(uint32_t *v, const void *p) {
    asm volatile("ld.global.nc.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                 : "l"(p));
}
__device__ __forceinline__ void tmem_ld8(uint32_t addr, uint32_t *v) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                 : "r"(addr));
}
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t *v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
        "%12, %13, %14, %15}, [%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
          "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(addr));
}
__device__ __forceinline__ void tmem_st8(uint32_t addr, const uint32_t *v) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(addr), "r"(v[0]),
                 "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}
__device__ __forceinline__ float power2(int e) {  // e from -126 to 127
    return __int_as_float((e + 127) << 23);
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// Meeting of the softmax warps, and with an OR of `v`.
__device__ __forceinline__ void meet() { asm volatile("bar.sync 1, 256;" ::: "memory"); }
__device__ __forceinline__ bool meet_any(bool v) {
    uint32_t any;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 q, %1, 0;\n\t"
        "barrier.cta.red.or.pred p, 1, 256, q;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(any)
        : "r"((uint32_t)v)
        : "memory");
    return any != 0;
}

// Cluster (request r, heads [N g, N g + N)); CTA `split` of it takes rows
// [split * split_rows, min(k, (split + 1) * split_rows)).
template <int N>
__global__ void __launch_bounds__(kPackedThreads, 1)
    packed_kernel(const __grid_constant__ CUtensorMap map, const PackedArgs a, int split_rows, bool aligned) {
    extern __shared__ __align__(1024) uint8_t smem[];  // the swizzle's period
    constexpr bool kOwnP = own_p(N);
    constexpr uint32_t kOffP = off_p(N);
    constexpr int kOthersChunks = others_chunks(N);  // tile i's others are in i % kOthersChunks
    const uint32_t s0 = smem_addr(smem);
    volatile uint32_t *words = reinterpret_cast<volatile uint32_t *>(smem + kOffWord);
    volatile uint32_t *abort_flag = words + 1;
    volatile uint32_t *tiles_begun = words + 2;  // whose probabilities are there
    // chunks 0 to 3, 4 to 7, the ninth; outputs of the first two dimension tiles, of the others
    auto chunks_full = [&](int i) { return s0 + kOffBar + 8u * i; };
    auto others_full = [&](int b) { return s0 + kOffBar + 8u * (2 + b); };
    auto others_free = [&](int b) { return s0 + kOffBar + 8u * (4 + b); };
    auto pv_done = [&](int i) { return s0 + kOffBar + 8u * (6 + i); };
    const uint32_t s_full = s0 + kOffBar + 8u * 8, p_ready = s0 + kOffBar + 8u * 9,
                   drained = s0 + kOffBar + 8u * 10;
    cg::cluster_group cluster = cg::this_cluster();
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);  // known to be the same in a warp
    const int split = blockIdx.x, nsplit = gridDim.x, r = blockIdx.y, g0 = blockIdx.z * N;
    const int heads = min(N, a.heads - g0);
    const int64_t row0 = (int64_t)split * split_rows;
    const int rows = (int)(row0 < a.k ? min((int64_t)split_rows, a.k - row0) : 0);
    const int tiles = (rows + kTileRows - 1) / kTileRows;
    const int32_t *idx = a.idx + (int64_t)r * a.k + row0;
    float *back = reinterpret_cast<float *>(smem + kOffBack), *base = reinterpret_cast<float *>(smem + kOffBase);

    // ---- the first rows on their way, barriers, TMEM, queries
    // (warps 0-7) of rows 16 warp + lane % 8 and 8 further of a tile, the quarter
    // lane / 8: codes of chunk `quarter` and the fourth after it, 4 and 4 scales, and
    // (without room for P) 32 bytes of the others
    const int quarter = lane >> 3;
    uint32_t codes[2][16], scales[2][2], others[2][8];
    // (checked only when it is used, so that the load stays in flight)
    auto load_index = [&](int j) {
        int32_t row = -1;
        if (j < rows)
            asm volatile("ld.global.nc.b32 %0, [%1];" : "=r"(row) : "l"(idx + j));
        return row;
    };
    auto in_range = [&](int32_t row) { return row >= 0 && (int64_t)row < a.cache_rows; };
    int32_t next[2] = {-1, -1};
    auto load_indices = [&](int tile) {
#pragma unroll
        for (int p = 0; p < 2; ++p) next[p] = load_index(tile * kTileRows + 16 * warp + 8 * p + (lane & 7));
    };
    // 32 bytes of codes and 4 scales of the row next[p] (c = 2: of the others); a
    // masked row is zeros: P of 0 meets no stale bytes
    auto load_piece = [&](int p, int c) {
        uint32_t *v = c < 2 ? codes[p] + 8 * c : others[p];
        const bool use = in_range(next[p]);
        const uint8_t *src = a.cache + (use ? next[p] : 0) * (int64_t)kPackedBytes;
        const uint8_t *from = src + quarter * 32 + (c < 2 ? 128 * c : kOthers);
        if (use) {
            if (aligned) {
                load32(v, from);
            } else {
                load16(v, from);
                load16(v + 4, from + 16);
            }
            if (c < 2)
                asm volatile("ld.global.nc.b32 %0, [%1];"
                             : "=r"(scales[p][c])
                             : "l"(src + kScales + 16 * c + 4 * quarter));
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = 0u;
            if (c < 2) scales[p][c] = 0u;
        }
    };
    // (warp 17) the others of four rows to a lane, straight into their chunk
    int32_t ahead[4];
    auto load_four = [&](int i) {
#pragma unroll
        for (int e = 0; e < 4; ++e) ahead[e] = load_index(i * kTileRows + 4 * lane + e);
    };
    int32_t row4[4];
    uint32_t any_row;
    // a masked row's place gets another row of the tile, whose values its P of 0
    // meets; a tile without any is zeros
    auto fill_masked = [&]() {
        int any = -1;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (in_range(ahead[e])) any = ahead[e];
        any_row = __ballot_sync(0xFFFFFFFFu, any >= 0);
        const int other = __shfl_sync(0xFFFFFFFFu, any, any_row ? __ffs(any_row) - 1 : 0);
#pragma unroll
        for (int e = 0; e < 4; ++e) row4[e] = in_range(ahead[e]) ? ahead[e] : other;
    };
    auto bring_others = [&](int b) {
        const uint32_t at = off_others(N, b);
        if (any_row) {
            if (lane == 0) mbar_expect(others_full(b), kChunk);
            __syncwarp();
            gather4(s0 + at + lane * 512, &map, kOthers / 2, row4, others_full(b));
        } else {
            for (uint32_t c = lane * 16; c < kChunk; c += 512)
                *reinterpret_cast<uint4 *>(smem + at + c) = make_uint4(0u, 0u, 0u, 0u);
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive(others_full(b));
        }
    };
    // (each warp's part in a branch of its own: what one holds takes no registers of
    // the others', who have 96)
    if (warp >= 8 && warp < 16) {
        // the second 32 heads into L2 while the first are on their way
        if (N > 32 && lane < 4) {
            const int n = 32 + 8 * lane + warp - 8;
            if (n < heads)
                asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(
                                 a.q + ((int64_t)r * a.heads + g0 + n) * kLatentRecordBytes),
                             "n"(kLatentRecordBytes)
                             : "memory");
        }
#pragma unroll 1
        for (int n0 = 0; n0 < N; n0 += 32) {
            // (four heads' loads together)
            uint4 x[4][2], z[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int n = n0 + 8 * i + warp - 8;
                x[i][0] = x[i][1] = z[i] = make_uint4(0u, 0u, 0u, 0u);
                const uint8_t *src = a.q + ((int64_t)r * a.heads + g0 + n) * kLatentRecordBytes;
                if (n < heads) {
                    x[i][0] = __ldg(reinterpret_cast<const uint4 *>(src + lane * 16));
                    x[i][1] = __ldg(reinterpret_cast<const uint4 *>(src + 512 + lane * 16));
                    if (lane < 8) z[i] = __ldg(reinterpret_cast<const uint4 *>(src + 1024 + lane * 16));
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int n = n0 + 8 * i + warp - 8;
                if (n >= N) break;
                uint32_t top = 0;
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    top = __vmaxu2(top, __vmaxu2(__vmaxu2(x[i][j].x & 0x7FFF7FFFu, x[i][j].y & 0x7FFF7FFFu),
                                                 __vmaxu2(x[i][j].z & 0x7FFF7FFFu, x[i][j].w & 0x7FFF7FFFu)));
                top = __reduce_max_sync(0xFFFFFFFFu, max(top >> 16, top & 0xFFFFu));
                uint32_t top_o = __vmaxu2(__vmaxu2(z[i].x & 0x7FFF7FFFu, z[i].y & 0x7FFF7FFFu),
                                          __vmaxu2(z[i].z & 0x7FFF7FFFu, z[i].w & 0x7FFF7FFFu));
                top_o = __reduce_max_sync(0xFFFFFFFFu, max(top_o >> 16, top_o & 0xFFFFu));
                const int e = (int)(top >> 7), e_o = (int)(top_o >> 7);
                // the latent part's largest to 2^13 or a little more, the others' below 2^81
                int up = min(140 - e, 126);
                if (e_o < 255) up = min(up, 207 - e_o + a.shift);
                if (e == 255) up = 0;
                const int down = max(-126, min(126, a.shift - up));
                const float factor = power2(up), factor_o = power2(-down);
                const uint32_t at = kOffQ + n * 128;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const uint32_t word[4] = {x[i][j].x, x[i][j].y, x[i][j].z, x[i][j].w};
                    uint32_t h[4];
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        h[c] = pack_f16(__uint_as_float(word[c] << 16) * factor,
                                        __uint_as_float(word[c] & 0xFFFF0000u) * factor);
                    // dimensions [256 j + 8 lane, ... + 8)
                    *reinterpret_cast<uint4 *>(smem + at + (4 * j + (lane >> 3)) * (N * 128) +
                                               (((lane & 7) ^ (n & 7)) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
                }
                if (lane < 8) {
                    const uint32_t word[4] = {z[i].x, z[i].y, z[i].z, z[i].w};
                    uint32_t h[4];
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        h[c] = pack_bf16(__uint_as_float(word[c] << 16) * factor_o,
                                         __uint_as_float(word[c] & 0xFFFF0000u) * factor_o);
                    *reinterpret_cast<uint4 *>(smem + at + 8 * (N * 128) + ((lane ^ (n & 7)) << 4)) =
                        make_uint4(h[0], h[1], h[2], h[3]);
                }
                if (lane == 0) {
                    // (finite, so that a product of 0 stays 0)
                    back[n] = fminf(fmaxf(a.scale_log2 * power2(down), kNoMax), -kNoMax);
                    base[n] = kNoMax;
                }
            }
        }
    } else if (warp >= 16) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        if (warp == 16) {
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                             s0 + kOffWord)
                         : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
        } else if (warp == 17) {
            load_four(0);
            if (lane == 0) {
                *abort_flag = *tiles_begun = 0;
                for (int i = 0; i < 2; ++i) {
                    mbar_init(chunks_full(i), 8);
                    mbar_init(others_full(i), kOwnP ? 1 : 8);
                    mbar_init(others_free(i), 1);
                    mbar_init(pv_done(i), 1);
                }
                mbar_init(s_full, 1);
                mbar_init(p_ready, 8);
                mbar_init(drained, 1);
                mbar_init_done();
            }
            __syncwarp();
            asm volatile("bar.arrive 2, 288;" ::: "memory");
            if (kOwnP && tiles > 0) {
                fill_masked();
                bring_others(0);
            }
        }
    }
    // the queries and TMEM are there; the rows do not wait for them
    uint32_t tmem = 0;
    if (warp >= 8) {
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        fence_before();
        asm volatile("bar.sync 3, 384;" ::: "memory");
        fence_after();
        tmem = words[0];
    }

    bool ok = true;
    // what the join uses: a CTA's units, parts of all CTAs one after the other
    const int share = (kUnits + nsplit - 1) / nsplit;
    float2 *ml_s = reinterpret_cast<float2 *>(smem + kOffMl);
    float4 *parts = reinterpret_cast<float4 *>(smem);
    constexpr uint32_t kUnitVecs = 32 * N / 4;

    if (warp < 8) {
        // ---- rows to f16
        asm volatile("setmaxnreg.inc.sync.aligned.u32 112;");
        load_indices(0);
#pragma unroll
        for (int c = 0; c < (kOwnP ? 2 : 3); ++c)
#pragma unroll
            for (int p = 0; p < 2; ++p) load_piece(p, c);
        load_indices(1);
        asm volatile("bar.sync 2, 288;" ::: "memory");  // the barriers are there
        // of the first row's first 16 bytes in chunk 0; unit j of them is at that ^ 16 j
        uint32_t at = s0 + (16 * warp + (lane & 7)) * 128 + ((lane & 7) << 4);
#pragma unroll 1
        for (int i = 0; i < tiles; ++i) {
            asm volatile("" : "+r"(at));  // addresses formed here, not kept for the loop

            auto signal = [&](uint32_t bar) {
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) mbar_arrive(bar);
            };
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                // the outputs that read these chunks
                if (i > 0) ok = ok && mbar_wait_warp(pv_done(c), (i - 1) & 1, abort_flag);
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    const uint32_t lo = scales2(scales[p][c]), hi = scales2(scales[p][c] >> 16);
                    const uint32_t sc[4] = {__byte_perm(lo, 0u, 0x1010), __byte_perm(lo, 0u, 0x3232),
                                            __byte_perm(hi, 0u, 0x1010), __byte_perm(hi, 0u, 0x3232)};
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        uint32_t v[4];
                        values8(codes[p][8 * c + j], sc[j / 2], v);
                        st_shared16((at + (4 * c + quarter) * kChunk ^ j << 4) + p * 1024, v);
                    }
                }
                signal(chunks_full(c));
            }
            if constexpr (!kOwnP) {
#pragma unroll
                for (int p = 0; p < 2; ++p)
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        st_shared16((at ^ (2 * quarter + j) << 4) + 8 * kChunk + p * 1024, others[p] + 4 * j);
                signal(others_full(0));
            }
            // The next tile's loads.  All at once, they fill the load-store unit for 1.25 us,
            // and the softmax waits behind them: half of them come when it is done, while
            // the outputs' products begin (64 x 2048 rows at 16 heads 28.2 us, all before
            // 29.5, all behind 31.1; 32 x 2048 at 128 heads 45.0, 46.5, 47.8)
            if (i + 1 < tiles) {
                load_piece(0, 0);
                load_piece(1, 0);
                ok = ok && mbar_wait_warp(p_ready, i & 1, abort_flag);
#pragma unroll
                for (int c = 1; c < (kOwnP ? 2 : 3); ++c)
#pragma unroll
                    for (int p = 0; p < 2; ++p) load_piece(p, c);
                load_indices(i + 2);
            }
        }
        __syncthreads_or(!ok);
        if (nsplit > 1) cluster.sync();  // with the softmax warps'
    } else if (warp >= 16) {
        if (warp == 16) {
            // ---- the products: the whole warp waits, one lane issues
            const uint32_t issuer = elect_one();
            constexpr uint32_t kIdescF16 = 1u << 4 | 128u >> 4 << 24 | (uint32_t)N >> 3 << 17;
            constexpr uint32_t kIdescBf16 = kIdescF16 | 1u << 7 | 1u << 10;
            constexpr uint32_t kIdescOnes = kIdescF16 | 1u << 16;  // B is given with its N dimension contiguous
            constexpr uint32_t kIdescPv = kIdescOnes | 1u << 15;   // and A with its M dimension
            const uint64_t k_op = operand(s0, 16), q_op = operand(s0 + kOffQ, 16), p_op = operand(s0 + kOffP, kPBytes),
                           v_op = operand(s0, kChunk);
            // the same answer in every lane, which keeps what follows uniform
            auto wait = [&](uint32_t bar, uint32_t parity) {
                return __all_sync(0xFFFFFFFFu, mbar_try(bar, parity)) ||
                       mbar_wait_warp(bar, parity, abort_flag);
            };
#pragma unroll 1
            for (int i = 0; i < tiles && ok; ++i) {
#pragma unroll 1
                for (int c = 0; c < 8; ++c) {
                    if (c % 4 == 0 && !(ok = wait(chunks_full(c / 4), i & 1))) break;
                    const uint64_t k = k_op + (c * kChunk >> 4), q = q_op + (c * (N * 128) >> 4);
#pragma unroll
                    for (int s = 0; s < 4; ++s)
                        mma_ss(tmem + kColS, k + 2 * s, q + 2 * s, kIdescF16, s > 0 || c > 0, issuer);
                }
                if (!ok) break;
                const int b = i % kOthersChunks;
                if (!(ok = wait(others_full(b), i / kOthersChunks & 1))) break;
                {
                    const uint64_t k = k_op + (off_others(N, b) >> 4), q = q_op + (8 * (N * 128) >> 4);
#pragma unroll
                    for (int s = 0; s < 4; ++s) mma_ss(tmem + kColS, k + 2 * s, q + 2 * s, kIdescBf16, true, issuer);
                }
                mma_commit(s_full, issuer);
                if (kOwnP) mma_commit(others_free(b), issuer);
                if (!(ok = wait(p_ready, i & 1))) break;
                if (lane == 0) *tiles_begun = i + 1;
                fence_after();
                // whole steps of 16 rows up to the tile's last
                const int steps = (min(kTileRows, rows - i * kTileRows) + 15) / 16;
#pragma unroll 1
                for (int m = 0; m < 4; ++m) {
                    const uint64_t v = v_op + (m * 2 * kChunk >> 4);
#pragma unroll
                    for (int s = 0; s < 8; ++s)
                        if (s < steps)
                            mma_ss(tmem + m * N, v + s * (2048 >> 4), p_op + s * (2048 >> 4), kIdescPv, i > 0 || s > 0,
                                   issuer);
                    if (m & 1) mma_commit(pv_done(m >> 1), issuer);
                    // the sums: ones P^T
                    if (m == 1)
#pragma unroll
                        for (int s = 0; s < 8; ++s)
                            if (s < steps)
                                mma_ts(tmem + kColL, tmem + kColOnes, p_op + s * (2048 >> 4), kIdescOnes, i > 0 || s > 0,
                                       issuer);
                }
            }
            // no product may still run when its operands or the TMEM are used otherwise
            mma_commit(drained, issuer);
            mbar_drain(drained, 0);
        } else if (kOwnP && warp == 17) {
            // ---- the others of the tiles behind the first
            int done = min(tiles, 1);
            load_four(1);
#pragma unroll 1
            for (int i = 1; i < tiles; ++i) {
                fill_masked();
                load_four(i + 1);
                const int b = i % kOthersChunks, turn = i / kOthersChunks;
                if (turn > 0) ok = mbar_wait_warp(others_free(b), (turn - 1) & 1, abort_flag);
                if (!ok) break;
                bring_others(b);
                done = i + 1;
            }
            // nothing may land after the CTA has left the chunks (in a normal run the
            // products have waited for all of it)
            for (int i = max(0, done - kOthersChunks); i < done; ++i)
                mbar_drain(others_full(i % kOthersChunks), i / kOthersChunks & 1);
        } else {
            // ---- rows into L2, up to kAhead tiles before their loads
            constexpr int kWarps = kOwnP ? 2 : 3;
            // (by a count and not a barrier's phase, which a warp that falls behind would miss)
            for (int i = 1; i < tiles; ++i) {
                int begun = (int)*tiles_begun;
                for (const uint64_t t0 = globaltimer(); begun + kAhead <= i; begun = (int)*tiles_begun) {
                    if (*abort_flag || globaltimer() - t0 > kWaitLimitNs) break;
                    __nanosleep(100);
                }
                if (begun + kAhead <= i) break;
                if (begun > i) continue;  // too late to help
                for (int j = warp - (20 - kWarps) + kWarps * lane; j < kTileRows; j += kWarps * 32) {
                    const int32_t row = load_index(i * kTileRows + j);
                    if (in_range(row))
                        asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(
                                         a.cache + row * (int64_t)kPackedBytes),
                                     "n"(kPackedBytes)
                                     : "memory");
                }
            }
        }
        __syncthreads_or(!ok);
        if (nsplit > 1) cluster.sync();  // with the softmax warps'
    } else {
        // ---- softmax
        // a half of the heads, [h0, h0 + kHalf), to four warps
        constexpr int kHalf = N / 2;
        const int w = warp & 3, row = 32 * w + lane, half = (warp - 8) >> 2, h0 = half * kHalf;
        const uint32_t lanes = (uint32_t)w * 32 << 16;
        float *top = reinterpret_cast<float *>(smem + kOffTop);
        // heads 0 to 7 of this row in P; unit u of eight heads is at that ^ 16 u
        uint32_t p_at = s0 + kOffP + row * 128 + ((row & 7) << 4);
        if (half == 0) {
            const uint32_t one[16] = {0x3C003C00u, 0x3C003C00u, 0x3C003C00u, 0x3C003C00u, 0x3C003C00u, 0x3C003C00u,
                                      0x3C003C00u, 0x3C003C00u, 0x3C003C00u, 0x3C003C00u, 0x3C003C00u, 0x3C003C00u,
                                      0x3C003C00u, 0x3C003C00u, 0x3C003C00u, 0x3C003C00u};
            tmem_st16(tmem + lanes + kColOnes, one);
            tmem_wait_st();
        }
        int32_t my_row = load_index(row);
#pragma unroll 1
        for (int i = 0; i < tiles; ++i) {
            asm volatile("" : "+r"(p_at));  // addresses formed here, not kept for the loop
            const bool valid = in_range(my_row);
            const int32_t next_row = load_index((i + 1) * kTileRows + row);
            ok = ok && mbar_wait_warp(s_full, i & 1, abort_flag);
            fence_after();
            // eight scores, of products that are there
            auto scores = [&](int c, const uint32_t *x, float *s) {
                float4 f[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) f[e] = reinterpret_cast<const float4 *>(back + h0 + c)[e];
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    s[e] = valid ? __fmul_rn(__uint_as_float(x[e]), (&f[e / 4].x)[e % 4]) : -INFINITY;
            };
            const uint32_t ts = tmem + lanes + kColS + h0;
            // P of eight heads, with the maxima so far; whether a score exceeds them too far
            auto probabilities = [&](int c, const uint32_t *x) {
                float s[8], most = -INFINITY;
                scores(c, x, s);
                float4 m[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) m[e] = reinterpret_cast<const float4 *>(base + h0 + c)[e];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float y = s[e] - (&m[e / 4].x)[e % 4];
                    most = fmaxf(most, y);
                    s[e] = ex2(y);       // (of a masked row 0)
                }
                const uint32_t p[4] = {pack_f16(s[0], s[1]), pack_f16(s[2], s[3]), pack_f16(s[4], s[5]),
                                       pack_f16(s[6], s[7])};
                st_shared16(p_at ^ ((h0 + c) / 8) << 4, p);
                return most > kUnit + kRise;
            };
            // (before the first tile there is no maximum to try)
            constexpr uint32_t kAll = (1u << kHalf / 8) - 1u;
            uint32_t above = i == 0 ? kAll : 0u;  // bit c / 8
            if (i > 0) {
                uint32_t x[2][8];        // the next eight are on their way
                tmem_ld8(ts, x[0]);
#pragma unroll
                for (int c = 0; c < kHalf; c += 8) {
                    const int b = c / 8 & 1;
                    tmem_wait_ld<8>(x[b]);
                    if (c + 8 < kHalf) tmem_ld8(ts + c + 8, x[b ^ 1]);
                    if (probabilities(c, x[b])) above |= 1u << c / 8;
                }
            }
            if (kAll > 1u) {
                above = __reduce_or_sync(0xFFFFFFFFu, above);
                if (lane == 0) words[kWordAbove + warp - 8] = above;
            }
            // (a wait that gave up is seen by all at once, and only here: nobody is left
            // waiting for the others)
            if (meet_any(above != 0 || !ok)) {
                auto above_of = [&](int half) {
                    if (kAll == 1u) return kAll;
                    volatile uint32_t *w4 = words + kWordAbove + 4 * half;
                    return w4[0] | w4[1] | w4[2] | w4[3];
                };
                if (meet_any(!ok)) {
                    ok = false;
                    break;
                }
                // Only the eights of heads with such a score.  Lane l of a warp gets the maximum
                // of the l-th head over the warp's rows: in the last steps half of the heads that
                // a lane still has go to its partner
                const uint32_t mine = above_of(half);
#pragma unroll 1
                for (int c = 0; c < kHalf; c += 8) {
                    if (!(mine >> c / 8 & 1u)) continue;
                    uint32_t x[8];
                    tmem_ld8(ts + c, x);
                    tmem_wait_ld<8>(x);
                    float s[8];
                    scores(c, x, s);
#pragma unroll
                    for (int d = 16; d >= 8; d >>= 1)
#pragma unroll
                        for (int e = 0; e < 8; ++e) s[e] = fmaxf(s[e], __shfl_xor_sync(0xFFFFFFFFu, s[e], d));
#pragma unroll
                    for (int d = 4; d > 0; d >>= 1) {
                        const bool up = lane & d;
#pragma unroll
                        for (int e = 0; e < d; ++e) {
                            const float keep = up ? s[e + d] : s[e], give = up ? s[e] : s[e + d];
                            s[e] = fmaxf(keep, __shfl_xor_sync(0xFFFFFFFFu, give, d));
                        }
                    }
                    if (lane < 8) top[w * kMaxN + h0 + c + lane] = s[0];
                    __syncwarp();            // TMEM is read by whole warps
                }
                meet();
                // the factors of what is there already; the new maxima
                float *f = reinterpret_cast<float *>(smem + kOffMl);
                if (half == 0 && row < N && (above_of(row / kHalf) >> row % kHalf / 8 & 1u)) {
                    const float m = base[row];
                    const float up = fmaxf(m, fmaxf(fmaxf(top[row], top[kMaxN + row]),
                                                    fmaxf(top[2 * kMaxN + row], top[3 * kMaxN + row])) -
                                                  kUnit);
                    f[row] = ex2(m - up);
                    base[row] = up;
                }
                meet();
#pragma unroll 1
                for (int c = 0; c < kHalf; c += 8) {
                    if (!(mine >> c / 8 & 1u)) continue;
                    uint32_t x[8];
                    tmem_ld8(ts + c, x);
                    tmem_wait_ld<8>(x);
                    probabilities(c, x);
                    if (i == 0) continue;
                    // (the products on O so far are done: these scores came behind them)
                    uint32_t o[5][8];
#pragma unroll
                    for (int m = 0; m < 5; ++m) tmem_ld8(tmem + lanes + (m < 4 ? m * N : kColL) + h0 + c, o[m]);
#pragma unroll
                    for (int m = 0; m < 5; ++m) {
                        tmem_wait_ld<8>(o[m]);
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            o[m][e] = __float_as_uint(__uint_as_float(o[m][e]) * f[h0 + c + e]);
                        tmem_st8(tmem + lanes + (m < 4 ? m * N : kColL) + h0 + c, o[m]);
                    }
                }
                tmem_wait_st();
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(p_ready);
            my_row = next_row;
        }
        const int failed = __syncthreads_or(!ok);  // every product is done
        fence_after();
        // ---- this CTA's part: (m, l), then O
        if (warp == 8) {
#pragma unroll
            for (int c = 0; c < N; c += 16) {
                uint32_t x[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) x[e] = 0u;
                if (tiles > 0) {
                    tmem_ld16(tmem + lanes + kColL + c, x);
                    tmem_wait_ld<16>(x);
                }
                if (lane == 0)
#pragma unroll
                    for (int e = 0; e < 16; ++e) top[c + e] = __uint_as_float(x[e]);
                __syncwarp();
            }
        }
        meet();
        if (nsplit == 1) {
            // nothing to join (and k >= 1 rows): a lane has a dimension of the heads (1 x 64
            // rows 6.1 us, 7.9 by way of the join; 100 x 600 18.4, 19.9)
            if (half == 0 && row < N)
                top[row] = failed ? __int_as_float(0x7FC00000) : top[row] == 0.f ? 0.f : power2(a.shift) / top[row];
            meet();
#pragma unroll 1
            for (int m = half; m < 4; m += 2) {
                uint16_t *dst = reinterpret_cast<uint16_t *>(a.out + ((int64_t)r * a.heads + g0) * 1024) + 128 * m +
                                32 * w + lane;
#pragma unroll 1
                for (int c = 0; c < heads; c += 16) {
                    uint32_t x[16];
                    tmem_ld16(tmem + lanes + m * N + c, x);
                    tmem_wait_ld<16>(x);
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        uint16_t y;
                        asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(y) : "f"(__uint_as_float(x[e]) * top[c + e]));
                        if (c + e < heads) dst[(c + e) * 512] = y;
                    }
                }
            }
        } else {
            const float2 mine = row < N ? make_float2(failed ? __int_as_float(0x7FC00000) : base[row], top[row])
                                        : make_float2(0.f, 0.f);
            cluster.sync();                     // all chunks are free
            if (half == 0 && row < N)
                for (int c = 0; c < nsplit; ++c) cluster.map_shared_rank(ml_s, c)[split * N + row] = mine;
            __syncwarp();
#pragma unroll 1
            for (int m = half; m < 4; m += 2) {
                // dimensions [128 m + 32 w, ... + 32): a unit, [split][unit][four heads][dimension]
                const int u = 4 * m + w, to = u / share;
                float4 *dst = cluster.map_shared_rank(parts, to) + (split * share + u - to * share) * kUnitVecs + lane;
#pragma unroll
                for (int c = 0; c < N; c += 16) {
                    uint32_t x[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) x[e] = 0u;
                    if (tiles > 0) {
                        tmem_ld16(tmem + lanes + m * N + c, x);
                        tmem_wait_ld<16>(x);
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        dst[(c / 4 + e) * 32] =
                            make_float4(__uint_as_float(x[4 * e]), __uint_as_float(x[4 * e + 1]),
                                        __uint_as_float(x[4 * e + 2]), __uint_as_float(x[4 * e + 3]));
                }
            }
        }
        fence_before();
    }
    if (!ok && lane == 0) atomicOr(&g_packed_status, HS_ATTN_STATUS_TIMEOUT);
    // the parts are here, and nobody writes to another CTA any more
    if (nsplit > 1)
        cluster.sync();
    else
        __syncthreads();
    if (warp == 16) {
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
    }

    if (nsplit == 1) return;
    // ---- the join: O = sum_c O_c 2^(m_c - M) / L for this CTA's units
    float *wts = reinterpret_cast<float *>(smem + kOffWts);
    if (tid < N) {
        float2 x[kMaxSplits];
        float M = -INFINITY, L = 0.f;
        bool bad = false;
#pragma unroll
        for (int c = 0; c < kMaxSplits; ++c) {
            if (c >= nsplit) break;
            x[c] = ml_s[c * N + tid];
            bad |= x[c].x != x[c].x;
            M = fmaxf(M, x[c].x);
        }
#pragma unroll
        for (int c = 0; c < kMaxSplits; ++c) {
            if (c >= nsplit) break;
            x[c].x = ex2(x[c].x - M);
            L = fmaf(x[c].y, x[c].x, L);
        }
        const float inv = bad ? __int_as_float(0x7FC00000) : L == 0.f ? 0.f : power2(a.shift) / L;
#pragma unroll
        for (int c = 0; c < kMaxSplits; ++c) {
            if (c >= nsplit) break;
            wts[c * N + tid] = x[c].x * inv;
        }
    }
    __syncthreads();
    // a warp takes four heads of a unit, a lane a dimension
    const int units = min(share, kUnits - split * share);
    constexpr int kTogether = 4, kWarps = kPackedThreads / 32;
    for (int i0 = warp; i0 < units * (N / 4); i0 += kTogether * kWarps) {
        float acc[kTogether][4] = {};
        for (int c = 0; c < nsplit; ++c)
#pragma unroll
            for (int b = 0; b < kTogether; ++b) {
                const int i = i0 + b * kWarps, u = i / (N / 4), h = i % (N / 4) * 4;
                if (i >= units * (N / 4)) break;
                const float4 y = parts[(c * share + u) * kUnitVecs + h * 8 + lane];
                const float4 f = *reinterpret_cast<const float4 *>(wts + c * N + h);
                acc[b][0] = fmaf(y.x, f.x, acc[b][0]);
                acc[b][1] = fmaf(y.y, f.y, acc[b][1]);
                acc[b][2] = fmaf(y.z, f.z, acc[b][2]);
                acc[b][3] = fmaf(y.w, f.w, acc[b][3]);
            }
#pragma unroll
        for (int b = 0; b < kTogether; ++b) {
            const int i = i0 + b * kWarps, u = i / (N / 4), h = i % (N / 4) * 4;
            if (i >= units * (N / 4)) break;
            uint16_t *dst = reinterpret_cast<uint16_t *>(a.out + ((int64_t)r * a.heads + g0 + h) * 1024) +
                            (split * share + u) * 32 + lane;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                uint16_t y;
                asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(y) : "f"(acc[b][e]));
                if (h + e < heads) dst[e * 512] = y;
            }
        }
    }
}

using Kernel = void (*)(const CUtensorMap, const PackedArgs, int, bool);
Kernel kernel_for(int n) {
    return n == 16 ? packed_kernel<16> : n == 32 ? packed_kernel<32> : n == 48 ? packed_kernel<48> : packed_kernel<64>;
}

struct DeviceInfo {
    int dev = -1;
    int active[kMaxSplits + 1] = {};  // co-resident clusters by size
};

cudaLaunchConfig_t config(int cluster, int n_req, int groups, cudaLaunchAttribute *attr) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(cluster, n_req, groups);
    cfg.blockDim = dim3(kPackedThreads);
    cfg.dynamicSmemBytes = kSmem;
    attr->id = cudaLaunchAttributeClusterDimension;
    attr->val.clusterDim.x = cluster;
    attr->val.clusterDim.y = 1;
    attr->val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cfg;
}

cudaError_t device_info(DeviceInfo *out) {
    static std::mutex mu;
    static DeviceInfo cached;
    std::lock_guard<std::mutex> lock(mu);
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev != cached.dev) {
        DeviceInfo d;
        d.dev = dev;
        bool big = true;
        for (int n = 16; n <= kMaxN; n += 16) {
            e = cudaFuncSetAttribute(kernel_for(n), cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
            if (e != cudaSuccess) return e;
            big &= cudaFuncSetAttribute(kernel_for(n), cudaFuncAttributeNonPortableClusterSizeAllowed, 1) ==
                   cudaSuccess;
        }
        // (one CTA per SM whatever n is)
        for (int c = 1; c <= (big ? kMaxSplits : 8); ++c) {
            cudaLaunchAttribute attr;
            const cudaLaunchConfig_t cfg = config(c, 1, 1, &attr);
            int n = 0;
            if (cudaOccupancyMaxActiveClusters(&n, kernel_for(kMaxN), &cfg) == cudaSuccess) d.active[c] = n;
        }
        (void)cudaGetLastError();  // a refused query above leaves no sticky error
        cached = d;
    }
    *out = cached;
    return cudaSuccess;
}

}  // namespace

// The cluster size with the least expected time: rounds of co-resident
// clusters, each a start and an end, with the join 2 us more, and the tiles of a CTA's share
// of the rows.
cudaError_t launch_packed_attention(const PackedArgs &a, cudaStream_t st) {
    DeviceInfo di;
    const cudaError_t e = device_info(&di);
    if (e != cudaSuccess) return e;
    const int groups = (a.heads + kMaxN - 1) / kMaxN;
    const int n = ((a.heads + groups - 1) / groups + 15) / 16 * 16;
    const int64_t units = (int64_t)a.n_req * groups;
    const int tiles = (a.k + kTileRows - 1) / kTileRows;
    int best = 1;
    float least = INFINITY;
    for (int c = 1; c <= kMaxSplits && c <= tiles; ++c) {
        if (!di.active[c] || c * ((kUnits + c - 1) / c) > kMaxParts) continue;
        const int64_t rounds = (units + di.active[c] - 1) / di.active[c];
        const float cost = rounds * ((c == 1 ? 5.f : 7.f + 0.1f * c) + 2.4f * ((tiles + c - 1) / c));
        if (cost < least) {
            least = cost;
            best = c;
        }
    }
    const int split_rows = (tiles + best - 1) / best * kTileRows;
    const EncodeTiled encode = encode_tiled();
    if (!encode) return cudaErrorNotSupported;
    // for the others: 64 bf16 of a row; an index is below 2^31
    CUtensorMap map;
    const cuuint64_t dims[2] = {kPackedBytes / 2, (cuuint64_t)std::min<int64_t>(a.cache_rows, 1ll << 31)};
    const cuuint64_t strides[1] = {kPackedBytes};
    const cuuint32_t box[2] = {64, 1}, one[2] = {1, 1};
    if (encode(&map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<uint8_t *>(a.cache), dims, strides, box, one,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return cudaErrorInvalidValue;
    cudaLaunchAttribute attr;
    cudaLaunchConfig_t cfg = config(best, a.n_req, (a.heads + n - 1) / n, &attr);
    cfg.stream = st;
    return cudaLaunchKernelEx(&cfg, kernel_for(n), map, a, split_rows, reinterpret_cast<uintptr_t>(a.cache) % 32 == 0);
}

cudaError_t packed_attention_status(uint32_t *status) {
    uint32_t v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_packed_status, sizeof(v));
    if (e != cudaSuccess) return e;
    *status = v;
    if (v) {
        const uint32_t zero = 0;
        e = cudaMemcpyToSymbol(g_packed_status, &zero, sizeof(zero));
    }
    return e;
}

}  // namespace hs
