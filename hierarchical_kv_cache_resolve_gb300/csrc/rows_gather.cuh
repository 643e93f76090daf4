// The gather of the requests' published rows and attention over them, as
// parts that merge_kernel joins; the code of one CTA, for the kernels of
// group_attention.cu and prefix_attention.cu.
//
// About one multiply-add per byte and query head: bound by HBM at any group
// size, so it is built to keep the gather busy.  The rows of all requests form
// one list of tiles of 16, cut into equal contiguous ranges, one per CTA and
// one CTA per SM: no request count leaves SMs idle.  A warp owns one key-value
// head (with fewer than five heads, several warps take a head's tiles in turn)
// and runs alone: it copies its head's 256-byte key and value blocks of 16
// rows at a time into a ring of its own with 16-byte asynchronous copies,
// zero-filled where a row is masked, so the pipeline needs no barrier between
// warps and no wait that could run out.
//
// The products are warp-level bf16 MMAs (fp32 accumulators): tcgen05's
// smallest tile has 64 rows of queries, of which a request has 1 to 16 per
// key-value head, and a gathered row would have to be spread over its swizzled
// layout.  They are formed transposed, S^T = K Q^T and O^T = V^T P^T, so that
// the 16 keys and the 128 dimensions are the MMA's rows and up to eight query
// heads its columns (two column tiles for 9 to 16): half the MMAs and half the
// accumulators of the other way round, whose 16 rows a group seldom fills.
// P takes the sum of two bf16 terms (error 2^-17).
#pragma once

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "hs_internal.cuh"

namespace hs {
namespace rows {

constexpr int kDim = 128;
constexpr int kTile = 16;                      // rows per tile
constexpr int kRing = 3;                       // tiles in a warp's ring
constexpr int kTileBytes = kTile * 2 * kDim;   // 4096: keys or values of a tile
constexpr int kWarpSmem = kRing * 2 * kTileBytes;
constexpr int kMaxWarps = 8;
static_assert(kMaxWarps * kWarpSmem <= 232448 - 1024, "one CTA's rings fit an SM");

__device__ __forceinline__ uint32_t smem_addr(const void *p) {
    return (uint32_t)__cvta_generic_to_shared(p);
}

// 16 bytes from global to shared memory; n = 0 writes zeros and reads nothing
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, uint32_t n) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n)
                 : "memory");
}

__device__ __forceinline__ void ldsm_x4(uint32_t (&r)[4], uint32_t s) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(s)
                 : "memory");
}

__device__ __forceinline__ void ldsm_x4_t(uint32_t (&r)[4], uint32_t s) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(s)
                 : "memory");
}

__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// An 8x8 matrix of bf16, two of row lane / 4 in each lane, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// (a, b) as two packed bf16 pairs whose sum is a and b to 2^-17
__device__ __forceinline__ void split_bf16(float a, float b, uint32_t &hi, uint32_t &lo) {
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(hi) : "f"(b), "f"(a));
    const float ra = a - __uint_as_float(hi << 16), rb = b - __uint_as_float(hi & 0xFFFF0000u);
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(lo) : "f"(rb), "f"(ra));
}

// Byte of 16-byte chunk c (0..15) of row r in a tile of 256-byte rows: the
// eight rows of a matrix load start on eight different banks.
__device__ __forceinline__ uint32_t swz(int r, int c) {
    return (uint32_t)(r * 256 + ((c ^ (r & 7)) << 4));
}

// CTA `cta` of the p.ctas that share the rows; warps 0 to heads * p.subs - 1
// call it, each on its own; NT column tiles of eight query heads.  `smem`: kWarpSmem bytes for each of them.
template <bool kScores, int NT>
__device__ __forceinline__ void gather_rows_nt(const GroupArgs &a, const RowsPlan &p, int cta,
                                            uint8_t *smem) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int head = warp % a.heads, sub = warp / a.heads;
    const int group = a.q_heads / a.heads;
    const int64_t W = (int64_t)a.heads * 4 * kDim;
    const int64_t t0 = range_start(cta, p.ctas, p.each, p.rest);
    const int64_t t1 = range_start(cta + 1, p.ctas, p.each, p.rest);
    const int r0 = (int)quick_div(t0, p.tiles), r1 = (int)quick_div(t1 - 1, p.tiles);
    const uint32_t ring = smem_addr(smem) + warp * kWarpSmem;
    const int koff = head * 2 * kDim, voff = (a.heads + head) * 2 * kDim;

    // the tiles of this warp in order: request by request, every subs-th of
    // the CTA's tiles of that request
    auto seg_first = [&](int r) { return max(t0, (int64_t)r * p.tiles); };
    auto seg_end = [&](int r) { return min(t1, (int64_t)(r + 1) * p.tiles); };
    int ir = r0;                       // the next tile whose copies are issued
    int64_t it = t0 + sub;
    auto settle = [&]() {
        while (ir <= r1 && it >= seg_end(ir)) {
            ++ir;
            it = seg_first(ir) + sub;  // not used past r1
        }
    };
    settle();
    // row index of lane (< 16) in the next tile, loaded one tile ahead of its
    // use (-1 past the end)
    auto load_row = [&]() {
        int32_t row = -1;
        if (ir <= r1) {
            const int j = (int)(it - (int64_t)ir * p.tiles) * kTile + lane;
            if (lane < kTile && j < a.k) row = __ldg(a.idx + (int64_t)ir * a.k + j);
        }
        return row;
    };
    int32_t raw = load_row();
    // issues the copies of the next tile into ring place b; its valid rows
    auto issue = [&](int b) -> uint32_t {
        const bool use = raw >= 0 && (int64_t)raw < a.cache_rows;
        const uint32_t valid = __ballot_sync(0xFFFFFFFFu, use);
        if (ir <= r1) {
            const uint32_t dst = ring + b * 2 * kTileBytes;
            const int c = lane & 15;
#pragma unroll
            for (int i = 0; i < kTile / 2; ++i) {
                const int r = 2 * i + (lane >> 4);
                const int32_t row = __shfl_sync(0xFFFFFFFFu, raw, r);
                const bool ok = valid >> r & 1u;
                const uint8_t *rec = a.cache + (ok ? row : 0) * W + c * 16;
                copy16(dst + swz(r, c), rec + koff, ok ? 16 : 0);
                copy16(dst + kTileBytes + swz(r, c), rec + voff, ok ? 16 : 0);
            }
            it += p.subs;
            settle();
            raw = load_row();
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        return valid;
    };

    uint32_t valid_q[kRing];           // masks of the tiles in the ring, oldest first
#pragma unroll
    for (int b = 0; b < kRing - 1; ++b) valid_q[b] = issue(b);
    int at = 0;                        // ring place of the oldest tile
    const int g0 = lane >> 2, c2 = (lane & 3) * 2;

    for (int r = r0; r <= r1; ++r) {
        // this head's queries as MMA B fragments, query 8 nt + lane / 4; those
        // past the group are zero
        uint32_t qb[NT][8][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int g = nt * 8 + g0;
            const uint8_t *q =
                a.q + ((int64_t)r * a.q_heads + head * group + g) * (2 * kDim) + c2 * 2;
#pragma unroll
            for (int s = 0; s < 8; ++s)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    qb[nt][s][i] =
                        g < group ? *reinterpret_cast<const uint32_t *>(q + s * 32 + i * 16) : 0u;
        }
        // of queries 8 nt + c2 and 8 nt + c2 + 1
        float m[NT][2], l[NT][2], o[NT][8][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            m[nt][0] = m[nt][1] = -INFINITY;
            l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
            for (int d = 0; d < 8; ++d)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[nt][d][i] = 0.f;
        }

        for (int64_t t = seg_first(r) + sub; t < seg_end(r); t += p.subs) {
            valid_q[kRing - 1] = issue(at >= 1 ? at - 1 : kRing - 1);
            asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 1) : "memory");
            __syncwarp();
            const uint32_t ks = ring + at * 2 * kTileBytes, vs = ks + kTileBytes;
            const uint32_t valid = valid_q[0];
            const bool v0 = valid >> g0 & 1u, v1 = valid >> (g0 + 8) & 1u;  // keys of this lane

            // S^T: rows keys g0 and g0 + 8, columns queries c2 and c2 + 1; even
            // and odd steps of 16 dimensions in two chains
            float s[NT][4], s2[NT][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i) s[nt][i] = s2[nt][i] = 0.f;
            {
                const int key = (lane & 7) + ((lane >> 3) & 1) * 8;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    uint32_t f[4];
                    ldsm_x4(f, ks + swz(key, 2 * i + (lane >> 4)));
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        mma_bf16(i & 1 ? s2[nt] : s[nt], f, qb[nt][i][0], qb[nt][i][1]);
                }
            }
            uint32_t ph[NT][2], pl[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    s[nt][i] = (i < 2 ? v0 : v1) ? (s[nt][i] + s2[nt][i]) * a.scale_log2 : -INFINITY;
                if (kScores) {
                    const int j = (int)(t - (int64_t)r * p.tiles) * kTile + g0;
                    float *sc = a.scores +
                                ((int64_t)r * a.q_heads + head * group + nt * 8 + c2) * a.k + j;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (nt * 8 + c2 + (i & 1) < group && j + (i >> 1) * 8 < a.k)
                            sc[(int64_t)(i & 1) * a.k + (i >> 1) * 8] = s[nt][i];
                }
                float f[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float x = fmaxf(s[nt][i], s[nt][2 + i]);
#pragma unroll
                    for (int d = 4; d <= 16; d <<= 1) x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, d));
                    const float up = fmaxf(m[nt][i], x);
                    // a query with nothing so far: exponents from 0, all its terms 2^-inf
                    const float base = up == -INFINITY ? 0.f : up;
                    f[i] = exp2f(m[nt][i] - base);
                    m[nt][i] = up;
                    s[nt][i] = exp2f(s[nt][i] - base);
                    s[nt][2 + i] = exp2f(s[nt][2 + i] - base);
                    l[nt][i] = l[nt][i] * f[i] + (s[nt][i] + s[nt][2 + i]);
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    split_bf16(s[nt][2 * i], s[nt][2 * i + 1], ph[nt][i], pl[nt][i]);
                    ph[nt][i] = transpose8(ph[nt][i]);
                    pl[nt][i] = transpose8(pl[nt][i]);
                }
#pragma unroll
                for (int d = 0; d < 8; ++d) {
                    o[nt][d][0] *= f[0];
                    o[nt][d][1] *= f[1];
                    o[nt][d][2] *= f[0];
                    o[nt][d][3] *= f[1];
                }
            }
            // O^T: rows dimensions 16 d + g0 and + 8
            {
                const int key = (lane & 7) + (lane >> 4) * 8;
#pragma unroll
                for (int d = 0; d < 8; ++d) {
                    uint32_t f[4];
                    ldsm_x4_t(f, vs + swz(key, 2 * d + ((lane >> 3) & 1)));
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        mma_bf16(o[nt][d], f, ph[nt][0], ph[nt][1]);
                        mma_bf16(o[nt][d], f, pl[nt][0], pl[nt][1]);
                    }
                }
            }
            __syncwarp();  // every lane has read this place before it is refilled
#pragma unroll
            for (int b = 0; b < kRing - 1; ++b) valid_q[b] = valid_q[b + 1];
            at = at + 1 == kRing ? 0 : at + 1;
        }

        // this part: the CTA's rows of request r (of this warp's turn)
        const int64_t part = ((int64_t)cta + r) * p.subs + sub;
        const int64_t row = part * a.q_heads + head * group;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
#pragma unroll
                for (int d = 4; d <= 16; d <<= 1)
                    l[nt][i] += __shfl_xor_sync(0xFFFFFFFFu, l[nt][i], d);
                const int g = nt * 8 + c2 + i;
                if (g >= group) continue;
                float *dst = p.o + (row + g) * kDim + g0;
#pragma unroll
                for (int d = 0; d < 8; ++d) {
                    dst[d * 16] = o[nt][d][i];
                    dst[d * 16 + 8] = o[nt][d][2 + i];
                }
                if (g0 == 0) p.ml[row + g] = make_float2(m[nt][i], l[nt][i]);
            }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
}

template <bool kScores>
__device__ __forceinline__ void gather_rows(const GroupArgs &a, const RowsPlan &p, int cta,
                                            uint8_t *smem) {
    if (a.q_heads / a.heads <= 8)
        gather_rows_nt<kScores, 1>(a, p, cta, smem);
    else
        gather_rows_nt<kScores, 2>(a, p, cta, smem);
}

}  // namespace rows
}  // namespace hs
