// The gather of the requests' published rows and attention over them, as
// parts that merge_kernel joins; the code of one CTA, for the kernels of
// group_attention.cu and prefix_attention.cu.
//
// About one multiply-add per byte and query head: bound by HBM at any group
// size, so it is built to keep the gather busy.  The rows of all requests form
// one list of tiles of 16, cut into equal contiguous ranges, one per CTA and
// one CTA per SM: no request count leaves SMs idle.  Up to four warps bring whole
// records, one asynchronous bulk copy per row, into a ring of tiles in shared
// memory (rows 16 bytes further apart than they are long, so that the eight
// rows of a matrix load start on eight different banks).  A warp for each
// key-value head computes (with fewer than five heads, several warps take a
// head's tiles in turn).  Where a row is masked its place is zeroed.
// Measured at 131072 rows of 4096 bytes: 175 us with 40 CTAs, 79 GB/s each (3
// tiles in the ring, a wait of 500 cycles in 1630 for one), and 86.5 us with
// 152 (6.2 TB/s); 223 and 91.6 us with 16-byte asynchronous copies by the
// computing warps, whose loads waited behind the copies in the SM's load-store
// unit (1400 of 2050 cycles for a tile).  One warp bringing all tiles cost 2 us
// on 5 x 777 rows of 1024 bytes (10.4 us, 8.4 with four).
//
// The products are warp-level bf16 MMAs (fp32 accumulators): tcgen05's
// smallest tile has 64 rows of queries, of which a request has 1 to 16 per
// key-value head, and a gathered row would have to be spread over its swizzled
// layout.  They are formed transposed, S^T = K Q^T and O^T = V^T P^T, so that
// the 16 keys and the 128 dimensions are the MMA's rows and up to eight query
// heads its columns (two column tiles for 9 to 16): half the MMAs and half the
// accumulators of the other way round, whose 16 rows a group seldom fills.
// P takes the sum of two bf16 terms (error 2^-17).
//
// Every wait gives up after a second: the parts become NaN and a status bit is
// set; copies in flight are waited for, with the same limit, before the CTA
// leaves.
#pragma once

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "barriers.cuh"
#include "hs.h"
#include "hs_internal.cuh"

namespace hs {
namespace rows {

constexpr int kDim = 128;
constexpr int kTile = 16;                      // rows per tile
constexpr int kMaxWarps = 8;                   // that compute
constexpr int kMaxSlots = 24;                  // tiles in the ring
constexpr uint32_t kSmem = 231680;
// full[kMaxSlots], empty[kMaxSlots], each slot's valid rows, abort flag; the ring
constexpr uint32_t kOffMask = 16 * kMaxSlots;
constexpr uint32_t kOffAbort = kOffMask + 4 * kMaxSlots;
constexpr uint32_t kOffSlots = 512;
static_assert(kOffAbort + 4 <= kOffSlots && kMaxSlots <= 32, "ring behind the barriers");

// Bytes from a row in the ring to the next.
__host__ __device__ __forceinline__ uint32_t pitch(int heads) { return heads * 4 * kDim + 16; }
// The ring's tiles (3 with 8 heads): tile n of a CTA is in slot n % slots, brought
// by warp slot % bringers of those that bring and taken by turn n % subs, so that
// each side meets a slot's tiles one after the other and knows its barriers'
// phases.
__host__ __device__ __forceinline__ int slots(int heads, int subs) {
    const int n = (int)((kSmem - kOffSlots) / (kTile * pitch(heads)));
    return (n < kMaxSlots ? n : kMaxSlots) / subs * subs;
}
__host__ __device__ __forceinline__ int bringers(int n_slots) { return n_slots < 4 ? n_slots : 4; }

// whole records; both addresses and the size are multiples of 16
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes,
                                          uint32_t bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
            "r"(dst), "l"(src), "r"(bytes), "r"(bar)
        : "memory");
}

__device__ __forceinline__ uint32_t full(uint32_t s0, int slot) { return s0 + 8u * slot; }
__device__ __forceinline__ uint32_t empty(uint32_t s0, int slot) {
    return s0 + 8u * (kMaxSlots + slot);
}

// By one warp, before a barrier of the CTA.
__device__ __forceinline__ void init(const GroupArgs &a, uint8_t *smem) {
    const uint32_t s0 = smem_addr(smem);
    const int lane = threadIdx.x & 31;
    if (lane < kMaxSlots) {
        mbar_init(full(s0, lane), 1);
        mbar_init(empty(s0, lane), a.heads);
    }
    if (lane == 0) *reinterpret_cast<volatile uint32_t *>(smem + kOffAbort) = 0;
    mbar_init_done();
}

// Warp w of those that bring the tiles of CTA `cta` of p.ctas; one that is too
// many returns.
__device__ __forceinline__ void bring(const GroupArgs &a, const RowsPlan &p, int cta,
                                      uint8_t *smem, int w) {
    const int lane = threadIdx.x & 31;
    const uint32_t s0 = smem_addr(smem);
    volatile uint32_t *masks = reinterpret_cast<volatile uint32_t *>(smem + kOffMask);
    volatile uint32_t *abort_flag = reinterpret_cast<volatile uint32_t *>(smem + kOffAbort);
    const uint32_t bytes = a.heads * 4 * kDim, step = pitch(a.heads);
    const int n_slots = slots(a.heads, p.subs), warps = bringers(n_slots);
    if (w >= warps) return;
    const int64_t t0 = range_start(cta, p.ctas, p.each, p.rest);
    const int64_t tiles = range_start(cta + 1, p.ctas, p.each, p.rest) - t0;
    // this warp's slots and tiles: w, w + warps, ...
    auto advance = [&](int &slot) {
        int d = warps;
        slot += warps;
        if (slot >= n_slots) {
            d = n_slots - (slot - warps) + w;
            slot = w;
        }
        return d;
    };
    // row index of lane (< 16) in the warp's next tile, loaded kAhead of them
    // ahead of its use
    int64_t next = w;
    int next_slot = w;
    int r = (int)quick_div(t0, p.tiles), i = (int)(t0 - (int64_t)r * p.tiles) + w;
    auto load_row = [&]() {
        int32_t row = -1;
        if (next < tiles) {
            for (; i >= p.tiles; i -= p.tiles) ++r;
            const int j = i * kTile + lane;  // below 2^31: k is at most 2^30
            if (lane < kTile && j < a.k) row = __ldg(a.idx + (int64_t)r * a.k + j);
            const int d = advance(next_slot);
            next += d;
            i += d;
        }
        return row;
    };
    constexpr int kAhead = 4;
    int32_t ahead[kAhead];
#pragma unroll
    for (int b = 0; b < kAhead; ++b) ahead[b] = load_row();
    uint32_t zeroed = 0;               // slots with rows that this warp has written
    uint32_t round = 0;                // its parity
    int slot = w;
    for (int64_t n = w; n < tiles;) {
        const int32_t row = ahead[0];
#pragma unroll
        for (int b = 0; b + 1 < kAhead; ++b) ahead[b] = ahead[b + 1];
        ahead[kAhead - 1] = load_row();
        const bool use = row >= 0 && (int64_t)row < a.cache_rows;
        const uint32_t valid = __ballot_sync(0xFFFFFFFFu, use);
        if (n >= n_slots) {
            const bool ok = mbar_wait(empty(s0, slot), round ^ 1, abort_flag);
            if (!__all_sync(0xFFFFFFFFu, ok)) break;
            // zeros written here come before the copies
            if (zeroed >> slot & 1u) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            zeroed &= ~(1u << slot);
        }
        const uint32_t dst = kOffSlots + slot * kTile * step;
        if (lane == 0) {
            masks[slot] = valid;
            mbar_expect_more(full(s0, slot), __popc(valid) * bytes);
        }
        __syncwarp();
        if (use)
            bulk_load(s0 + dst + lane * step, a.cache + row * (int64_t)bytes, bytes, full(s0, slot));
        for (uint32_t zero = ~valid & 0xFFFFu; zero; zero &= zero - 1) {
            zeroed |= 1u << slot;
            for (uint32_t c = lane * 16; c < bytes; c += 512)
                *reinterpret_cast<uint4 *>(smem + dst + (__ffs(zero) - 1) * step + c) =
                    make_uint4(0, 0, 0, 0);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(full(s0, slot));
        n += advance(slot);
        if (slot == w) round ^= 1;
    }
    // nothing may land after the CTA has left: the slots' last tiles (one that
    // had none has its wait for the phase before the first, which is over)
    for (int s = w; s < n_slots; s += warps) mbar_drain(full(s0, s), s < slot ? round : round ^ 1);
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

// CTA `cta` of the p.ctas that share the rows; warps 0 to heads * p.subs - 1,
// each on its own; NT column tiles of eight query heads.
template <bool kScores, int NT>
__device__ __forceinline__ void attend_nt(const GroupArgs &a, const RowsPlan &p, int cta,
                                          uint8_t *smem, uint32_t *status) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int head = warp % a.heads, sub = warp / a.heads;
    const int group = a.q_heads / a.heads;
    const int64_t t0 = range_start(cta, p.ctas, p.each, p.rest);
    const int64_t t1 = range_start(cta + 1, p.ctas, p.each, p.rest);
    const int r0 = (int)quick_div(t0, p.tiles), r1 = (int)quick_div(t1 - 1, p.tiles);
    const uint32_t s0 = smem_addr(smem);
    volatile uint32_t *masks = reinterpret_cast<volatile uint32_t *>(smem + kOffMask);
    volatile uint32_t *abort_flag = reinterpret_cast<volatile uint32_t *>(smem + kOffAbort);
    const uint32_t step = pitch(a.heads);
    const int n_slots = slots(a.heads, p.subs);
    // byte of this lane's row and half chunk for the two kinds of matrix loads
    const uint32_t k_at = s0 + kOffSlots + ((lane & 7) + ((lane >> 3) & 1) * 8) * step +
                          head * 2 * kDim + (lane >> 4) * 16;
    const uint32_t v_at = s0 + kOffSlots + ((lane & 7) + (lane >> 4) * 8) * step +
                          (a.heads + head) * 2 * kDim + ((lane >> 3) & 1) * 16;

    // this warp's tiles: every subs-th of the CTA's; the next one
    int64_t t = t0 + sub;
    int slot = sub;
    uint32_t phase = 0;
    bool ok = true;
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

        const int64_t end = min(t1, (int64_t)(r + 1) * p.tiles);
        for (; t < end && ok; t += p.subs) {
            ok = __all_sync(0xFFFFFFFFu, mbar_wait(full(s0, slot), phase, abort_flag));
            if (!ok) break;
            const uint32_t at = slot * kTile * step;
            const uint32_t valid = masks[slot];
            const bool v0 = valid >> g0 & 1u, v1 = valid >> (g0 + 8) & 1u;  // keys of this lane

            // S^T: rows keys g0 and g0 + 8, columns queries c2 and c2 + 1; even
            // and odd steps of 16 dimensions in two chains
            float s[NT][4], s2[NT][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i) s[nt][i] = s2[nt][i] = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                uint32_t f[4];
                ldsm_x4(f, k_at + at + i * 32);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    mma_bf16(i & 1 ? s2[nt] : s[nt], f, qb[nt][i][0], qb[nt][i][1]);
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
#pragma unroll
            for (int d = 0; d < 8; ++d) {
                uint32_t f[4];
                ldsm_x4_t(f, v_at + at + d * 32);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    mma_bf16(o[nt][d], f, ph[nt][0], ph[nt][1]);
                    mma_bf16(o[nt][d], f, pl[nt][0], pl[nt][1]);
                }
            }
            __syncwarp();  // every lane has read this slot before it is refilled
            if (lane == 0) mbar_arrive(empty(s0, slot));
            slot += p.subs;
            if (slot >= n_slots) {
                slot -= n_slots;
                phase ^= 1;
            }
        }
        if (!ok) {  // the merge makes such rows NaN
            if (lane == 0) atomicOr(status, HS_ATTN_STATUS_TIMEOUT);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) m[nt][0] = m[nt][1] = __int_as_float(0x7FC00000);
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
}

template <bool kScores>
__device__ __forceinline__ void attend(const GroupArgs &a, const RowsPlan &p, int cta,
                                       uint8_t *smem, uint32_t *status) {
    if (a.q_heads / a.heads <= 8)
        attend_nt<kScores, 1>(a, p, cta, smem, status);
    else
        attend_nt<kScores, 2>(a, p, cta, smem, status);
}

}  // namespace rows
}  // namespace hs
