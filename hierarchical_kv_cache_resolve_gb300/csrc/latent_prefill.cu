// Causal attention of prompts over expanded keys and values (hs_latent_prefill).
//
// For every head, queries q [192] and keys [K (128), kr (64)] of which kr, the
// part with the position, is the same for all heads, and values V [128]:
//   out_i = softmax_j(scale q_i . [K_j, kr_j]) V_j  over the keys j that query i
// of a sequence may see.  640 flops a pair: bound by the tensor cores.
//
// A CTA takes two tiles of 128 queries of a sequence and head, and blocks of 128
// keys up to the last that its last query sees.  Longest tiles first, for eight
// heads at a time: the reads of a head's keys by tiles side by side meet in L2, and
// few SMs idle at the end (16384 tokens of 32 heads: 1750 us head by head, 1660 by
// eights, 1690 all at once; 4096: 172, 143, 145).  Where the
// pairs are few, or their last round would leave many SMs idle, the blocks of each
// are split among CTAs (latent_prefill_split), whose parts join_kernel joins.  One CTA per SM:
//   warp 8    brings the queries, then keys and values (TMA, 128-byte swizzle)
//             through a ring of eight pieces of 16 KB in the order of use: 64
//             dimensions of 128 keys, or 64 values' 128 dimensions;
//   warp 9    one thread issues S_t = Q_t K^T and O_t += P_t V (tcgen05);
//   warps 0-3 and 4-7  the softmax of tile 0 and 1: a thread per query reads its
//             scores from TMEM, keeps the running maximum and sum in registers
//             and writes P back as bf16 over the scores;
//   warps 10 and 11  look through the values of blocks that some query does not
//             see whole (below), while their scores are on their way.
// While one tile's softmax runs, the tensor core works on the other's products.
//
// P is rounded once to bf16; a query's maximum only rises when a block exceeds it
// by more than 2^8.  O is rescaled by the warp then, by 1 for the queries whose own
// maximum stays: a key has no effect on the queries that do not see it, not even on
// how their probabilities are rounded, and rows that see nothing ask for nothing.
//
// A masked key has P = 0, and 0 V must be 0 whatever V holds: rows behind the
// sequence, which may be anything, are zeroed in shared memory, and so are
// infinities and NaN in a block that some query does not see whole; the first
// key that had one in each dimension is noted, and the queries that do see it
// get it back at the end.
//
// TMEM columns: S_0/P_0 0, S_1/P_1 128, O_0 256, O_1 384.
//
// Every wait gives up after a second: the CTA's rows become NaN and
// HS_ATTN_STATUS_TIMEOUT is set (hs_attention_status); copies and products in
// flight are waited for, with the same limit, before the CTA leaves.
#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>

#include <cuda_bf16.h>

#include "barriers.cuh"
#include "hs.h"
#include "hs_internal.cuh"
#include "tensor_core.cuh"

namespace hs {
namespace {

constexpr int kRows = 128;                   // of a tile of queries
constexpr int kKeys = 128;                   // of a block
constexpr int kQk = 192, kV = 128;
constexpr uint32_t kPiece = 16384;
constexpr int kPieces = 8;                   // of the ring
constexpr uint32_t kAtom = kRows * 128;      // 64 dimensions of 128 rows
constexpr uint32_t kAtomV = 64 * 128;        // 64 dimensions of 64 values
constexpr uint32_t kTileBytes = 3 * kAtom;   // a tile of queries
constexpr int kPrefillThreads = 384;
constexpr int kMaxPrefillSplits = 16;
constexpr int kHeadGroup = 8;
constexpr float kRise = 8.f;                 // log2 of how far P may exceed 1

constexpr uint32_t kOffRing = 2 * kTileBytes;
// full[kPieces], empty[kPieces], s_full[2], p_ready[2][2], q_full, look, looked, drained
constexpr uint32_t kOffBar = kOffRing + kPieces * kPiece;
constexpr int kBars = 2 * kPieces + 10;
constexpr uint32_t kOffWord = kOffBar + 8 * kBars;  // TMEM address, abort flag, odd values seen
constexpr uint32_t kOffOdd = kOffWord + 16;         // first NaN, +inf, -inf of each dimension
constexpr uint32_t kSmem = kOffOdd + 3 * kV * 4;
static_assert(kSmem <= 232448, "fits an SM");
static_assert(kOffBar % 8 == 0 && kOffWord % 16 == 0, "barriers are 8-byte aligned");

__device__ uint32_t g_prefill_status;

constexpr uint32_t kIdescS = kIdesc | (uint32_t)kKeys >> 3 << 17;

// Query tiles of sequence s have the places [starts[s] / 256 + s, ...) of a
// head: room for all of them, as a length of n ends at most n / 256 + 1 tiles
// further on whatever starts[s] is.  The sequence of place `at`.
__device__ __forceinline__ int find_sequence(const int32_t *starts, int n_seq, int n_tok, int at) {
    const int lane = threadIdx.x & 31;
    int lo = 0, hi = n_seq;
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32;
        const int64_t s = lo + (int64_t)lane * step;
        bool below = false;
        if (s < hi) below = min(max(__ldg(starts + s), 0), n_tok) / (2 * kRows) + s <= at;
        const uint32_t b = __ballot_sync(0xFFFFFFFFu, below);
        const int c = __ffs(~b) - 1;         // leading ones; -1: all of them
        const int first = lo + (c < 0 ? 31 : max(c - 1, 0)) * step;
        hi = min(hi, first + step);
        lo = first;
    }
    return lo;
}

__global__ void __launch_bounds__(kPrefillThreads, 1)
    prefill_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap k_map,
                   const __grid_constant__ CUtensorMap kr_map, const __grid_constant__ CUtensorMap v_map,
                   const PrefillArgs a, int places) {
    extern __shared__ __align__(1024) uint8_t smem[];  // the swizzle's period
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);  // known to be the same in a warp
    if (tid == 256) {
        for (const CUtensorMap *map : {&q_map, &k_map, &kr_map, &v_map})
            asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
    }
    // heads in groups: a group's places one after the other, each for all its heads
    // (equal parts of an item side by side, smaller ones behind all others)
    const unsigned items = gridDim.x / (unsigned)a.splits, group_items = (unsigned)(places * a.head_group);
    const int split = a.small_of ? blockIdx.x / items : blockIdx.x % (unsigned)a.splits;
    const unsigned item = a.small_of ? blockIdx.x % items : blockIdx.x / (unsigned)a.splits;
    const int head0 = item / group_items * a.head_group, in_group = min(a.head_group, a.heads - head0);
    const int within = item % group_items, head = head0 + within % in_group, at = within / in_group;

    // the sequence, its queries [q0, q1) and keys [k0, k0 + n_keys)
    const int seq = find_sequence(a.q_starts, a.n_seq, a.n_tok, at);
    const int q0 = min(max(__ldg(a.q_starts + seq), 0), a.n_tok);
    const int q1 = min(max(__ldg(a.q_starts + seq + 1), q0), a.n_tok);
    int k0 = min(max(__ldg(a.k_starts + seq), 0), a.n_keys);
    int n_keys = min(max(__ldg(a.k_starts + seq + 1), k0), a.n_keys) - k0;
    const int tiles = (q1 - q0 + 2 * kRows - 1) / (2 * kRows);
    const int place = at - (q0 / (2 * kRows) + seq);
    if (place < 0 || place >= tiles) return;
    const int first = (tiles - 1 - place) * 2 * kRows;  // query of the sequence
    int ahead = n_keys - (q1 - q0);                     // keys that query 0 sees, less one
    // keys that query i sees
    auto sees = [&](int i) { return min(max(i + 1 + ahead, 0), n_keys); };
    auto blocks_of = [&](int t) {
        const int i0 = first + t * kRows, i1 = min(i0 + kRows, q1 - q0);
        return i0 < i1 ? (sees(i1 - 1) + kKeys - 1) / kKeys : 0;
    };
    if (a.splits > 1) {
        // this CTA's blocks as if they were all
        const int all = max(blocks_of(0), blocks_of(1)), parts = a.small_of ? a.small_of : a.splits;
        const int small = (all + parts - 1) / parts, first_of = a.small_of ? all - small : small;
        const int from = min(split * first_of, all) * kKeys;
        k0 += from;
        ahead -= from;
        n_keys = min(max(n_keys - from, 0), (split == 0 ? first_of : small) * kKeys);
    }
    const int n_of[2] = {blocks_of(0), blocks_of(1)};
    const int n = max(n_of[0], n_of[1]);
    const int partial = sees(first) / kKeys;  // the first block that a query does not see whole

    const uint32_t s0 = smem_addr(smem);
    volatile uint32_t *words = reinterpret_cast<volatile uint32_t *>(smem + kOffWord);
    volatile uint32_t *abort_flag = words + 1;
    int *odd = reinterpret_cast<int *>(smem + kOffOdd);
    const uint32_t bars = s0 + kOffBar;
    auto full = [&](int i) { return bars + 8u * i; };
    auto empty = [&](int i) { return bars + 8u * (kPieces + i); };
    auto s_full = [&](int t) { return bars + 8u * (2 * kPieces + t); };
    auto p_ready = [&](int t, int h) { return bars + 8u * (2 * kPieces + 2 + 2 * t + h); };
    const uint32_t q_full = bars + 8u * (2 * kPieces + 6), look = bars + 8u * (2 * kPieces + 7);
    const uint32_t looked = bars + 8u * (2 * kPieces + 8), drained = bars + 8u * (2 * kPieces + 9);

    // The pieces in the order of use: K of block 0, then V of block j (two pieces)
    // and K of block j + 1 (three); number c is in place c % kPieces.
    const int pieces = 5 * n;
    auto load = [&](int c) {
        const int u = c - 3, j = u < 0 ? 0 : u / 5, w = u < 0 ? -1 : u - j * 5;
        const int slot = c % kPieces;
        const uint32_t dst = s0 + kOffRing + slot * kPiece;
        mbar_expect(full(slot), kPiece);
        if (w == 0 || w == 1) {
            const int x = head * a.kv_head_stride, y = k0 + j * kKeys + w * 64;
            tma_load(dst, &v_map, x, y, full(slot));
            tma_load(dst + kAtomV, &v_map, x + 64, y, full(slot));
        } else {
            const int part = u < 0 ? c : w - 2, y = k0 + (u < 0 ? 0 : j + 1) * kKeys;
            if (part < 2)
                tma_load(dst, &k_map, head * a.kv_head_stride + part * 64, y, full(slot));
            else
                tma_load(dst, &kr_map, 0, y, full(slot));
        }
    };
    if (warp == 9) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                         s0 + kOffWord)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    } else if (warp == 8 && lane == 0) {
        *abort_flag = 0;
        words[2] = 0;
        for (int i = 0; i < kPieces; ++i) {
            mbar_init(full(i), 1);
            mbar_init(empty(i), 1);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(s_full(t), 1);
            mbar_init(p_ready(t, 0), kRows);
            mbar_init(p_ready(t, 1), kRows);
        }
        mbar_init(q_full, 1);
        mbar_init(look, 1);
        mbar_init(looked, 64);
        mbar_init(drained, 1);
        mbar_init_done();
        if (n > 0) {
            mbar_expect(q_full, (n_of[0] > 0 ? kTileBytes : 0) + (n_of[1] > 0 ? kTileBytes : 0));
            for (int t = 0; t < 2; ++t)
                if (n_of[t] > 0)
                    for (int p = 0; p < 3; ++p)
                        tma_load(s0 + t * kTileBytes + p * kAtom, &q_map, head * kQk + p * 64,
                                 q0 + first + t * kRows, q_full);
            for (int c = 0; c < 3; ++c) load(c);
        }
    } else if (warp >= 10) {
        for (int i = tid - 320; i < 3 * kV; i += 64) odd[i] = INT_MAX;
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = words[0];

    if (warp >= 8) asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (warp == 8) {
        // ---- the rest of the pieces
        if (lane == 0 && n > 0) {
            int c = 3;
            for (; c < pieces; ++c) {
                if (c >= kPieces && !mbar_wait(empty(c % kPieces), (c / kPieces - 1) & 1, abort_flag)) break;
                load(c);
            }
            // nothing may land after the CTA has left the ring (in a normal run
            // the products have waited for all of it)
            for (int i = max(0, c - kPieces); i < c; ++i) mbar_drain(full(i % kPieces), (i / kPieces) & 1);
            mbar_drain(q_full, 0);
        }
    } else if (warp == 9) {
        // ---- the products: the whole warp waits, one lane issues
        const uint32_t issuer = elect_one();
        const uint64_t q_op = operand(s0, 16), k_op = operand(s0 + kOffRing, 16),
                       v_op = operand(s0 + kOffRing, kAtomV);
        uint32_t p_phase = 0;               // bit 2 t + h: of p_ready(t, h)
        bool ok = true;
        // the same answer in every lane, which keeps what follows uniform
        auto wait = [&](uint32_t bar, uint32_t parity) {
            return __all_sync(0xFFFFFFFFu, mbar_try(bar, parity)) ||
                   mbar_wait_warp(bar, parity, abort_flag);
        };
        auto wait_piece = [&](int c) { return ok = wait(full(c % kPieces), (c / kPieces) & 1); };
        auto release = [&](int c) { mma_commit(empty(c % kPieces), issuer); };
        // S_t = Q_t K^T of the three pieces from c on; `last`: nobody reads them after
        auto scores = [&](int t, int c, bool last) {
#pragma unroll 1
            for (int p = 0; p < 3; ++p) {
                if (!wait_piece(c + p)) return;
                const uint64_t q = q_op + ((t * kTileBytes + p * kAtom) >> 4);
                const uint64_t k = k_op + (((c + p) % kPieces) * kPiece >> 4);
#pragma unroll
                for (int s = 0; s < 4; ++s)
                    mma_ss(tmem + t * 128, q + 2 * s, k + 2 * s, kIdescS, p + s > 0, issuer);
                if (last) release(c + p);
            }
            mma_commit(s_full(t), issuer);
        };
        // O_t += P_t V of the two pieces from c on, each half of P as it is ready
        auto outputs = [&](int t, int c, bool begin, bool last) {
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {
                const int bar = 2 * t + h;
                if (!wait_piece(c + h) || !(ok = wait(p_ready(t, h), p_phase >> bar & 1u))) return;
                p_phase ^= 1u << bar;
                fence_after();
                const uint64_t v = v_op + (((c + h) % kPieces) * kPiece >> 4);
#pragma unroll
                for (int s = 0; s < 4; ++s)
                    mma_ts(tmem + 256 + t * 128, tmem + t * 128 + h * 32 + s * 8, v + s * (2048 >> 4),
                           kIdescV, !begin || h + s > 0, issuer);
                if (last) release(c + h);
            }
        };
        // the values of block j may be looked through: all before them have been used
        auto may_look = [&](int j) {
            if (j >= partial && j < n && issuer) mbar_arrive(look);
            __syncwarp();
        };
        if (n > 0) {
            ok = wait(q_full, 0);
            for (int t = 0; t < 2 && ok; ++t)
                if (n_of[t] > 0) scores(t, 0, t == 1 || n_of[1] == 0);
            may_look(0);
        }
#pragma unroll 1
        for (int j = 0; j < n && ok; ++j) {
            const int v = 3 + 5 * j;
            if (j >= partial && !(ok = wait(looked, (j - partial) & 1))) break;
#pragma unroll 1
            for (int t = 0; t < 2 && ok; ++t) {
                if (j >= n_of[t]) continue;
                outputs(t, v, j == 0, t == 1 || j >= n_of[1]);
                if (!ok) break;
                if (j + 1 < n_of[t])
                    scores(t, v + 2, t == 1 || j + 1 >= n_of[1]);
                else
                    mma_commit(s_full(t), issuer);
            }
            may_look(j + 1);
        }
        // no product may still run when the TMEM is given back
        mma_commit(drained, issuer);
        mbar_drain(drained, 0);
    } else if (warp >= 10) {
        // ---- values of blocks that some query does not see whole
        const int me = tid - 320;
#pragma unroll 1
        for (int j = partial; j < n; ++j) {
            bool ok = mbar_wait_warp(look, (j - partial) & 1, abort_flag);
            for (int h = 0; h < 2; ++h) {
                const int c = 3 + 5 * j + h;
                ok = ok && mbar_wait_warp(full(c % kPieces), (c / kPieces) & 1, abort_flag);
            }
            if (!ok) break;
            // keys from the first that some query does not see: 16 bytes (dimensions
            // [8 c, 8 c + 8)) of every fourth key to a thread, eight at a time
            const int c = me & 15, start = max(sees(first) - j * kKeys, 0) & ~31;
            const int end = min(kKeys, n_keys - j * kKeys);  // of the sequence
#pragma unroll 1
            for (int k32 = start; k32 < kKeys; k32 += 32) {
                const uint32_t piece = s0 + kOffRing + (3 + 5 * j + (k32 >> 6)) % kPieces * kPiece + (c >> 3) * kAtomV;
                // key k32 + (me >> 4) + 4 e: its eight bytes' column alternates with e
                const int k0 = k32 + (me >> 4);
                const uint32_t at = piece + (k0 & 63) * 128;
                const uint32_t x0 = ((c & 7) ^ (k0 & 7)) << 4, x1 = x0 ^ 64;
                uint32_t w[8][4], any = 0;
#pragma unroll
                for (int e = 0; e < 8; ++e) ld_shared16(at + e * 512 + (e & 1 ? x1 : x0), w[e]);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    if (k0 + 4 * e >= end) {
                        w[e][0] = w[e][1] = w[e][2] = w[e][3] = 0u;
                        st_shared16(at + e * 512 + (e & 1 ? x1 : x0), w[e]);
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) any |= ((w[e][i] & 0x7F807F80u) + 0x00800080u) & 0x80008000u;
                }
                if (!any) continue;
#pragma unroll 1
                for (int e = 0; e < 8; ++e) {
                    const uint32_t from = at + e * 512 + (e & 1 ? x1 : x0);
                    uint16_t *y = reinterpret_cast<uint16_t *>(smem + (from - s0));
#pragma unroll 1
                    for (int i = 0; i < 8; ++i) {
                        const uint32_t v = y[i];
                        if ((v & 0x7F80u) != 0x7F80u) continue;
                        y[i] = 0;
                        atomicMin(odd + (v & 0x7Fu ? 0 : v >> 15 ? 2 : 1) * kV + c * 8 + i, j * kKeys + k0 + 4 * e);
                        words[2] = 1;
                    }
                }
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            mbar_arrive(looked);
        }
    } else {
        // ---- softmax
        asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
        const int t = warp >> 2, row = tid & 127, i = first + t * kRows + row;
        const bool live = i < q1 - q0;
        const int limit = live ? sees(i) : 0;
        const int mine = n_of[t];
        const uint32_t lanes = (uint32_t)(warp & 3) * 32 << 16;
        const uint32_t ts = tmem + lanes + t * 128, to = tmem + lanes + 256 + t * 128;
        const float scale = a.scale_log2;
        uint32_t s_phase = 0;
        bool ok = true;
        float m = -INFINITY, l = 0.f;
#pragma unroll 1
        for (int j = 0; j < mine && ok; ++j) {
            ok = mbar_wait_warp(s_full(t), s_phase, abort_flag);
            if (!ok) break;
            s_phase ^= 1u;
            fence_after();
            const int left = limit - j * kKeys;
            const bool cut = __any_sync(0xFFFFFFFFu, left < kKeys);
            uint32_t s[kKeys];
            float x[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
            tmem_ld32(ts, s);
#pragma unroll
            for (int c = 0; c < kKeys / 32; ++c) {
                tmem_wait_ld<32>(s + c * 32);
                if (c + 1 < kKeys / 32) tmem_ld32(ts + (c + 1) * 32, s + (c + 1) * 32);
                if (cut) {
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (c * 32 + e >= left) s[c * 32 + e] = 0xFF800000u;  // -inf
                }
#pragma unroll
                for (int e = 0; e < 32; e += 8)
#pragma unroll
                    for (int h = 0; h < 4; ++h)
                        x[h] = fmaxf(fmaxf(x[h], __uint_as_float(s[c * 32 + e + 2 * h])),
                                     __uint_as_float(s[c * 32 + e + 2 * h + 1]));
            }
            const float top = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])) * scale;
            // (false as long as a query has seen nothing, true at its first score)
            const bool rise = top > m + kRise;
            if (__any_sync(0xFFFFFFFFu, rise)) {
                // each query by its own scores: what others see must not show in its bits
                const float f = !rise ? 1.f : m == -INFINITY ? 0.f : ex2(m - top);
                if (rise) m = top;
                l *= f;
                if (j > 0) {
                    // the products on O so far are done: these scores came behind them
                    uint32_t o[32];
#pragma unroll 1
                    for (int c = 0; c < 4; ++c) {
                        tmem_ld32(to + c * 32, o);
                        tmem_wait_ld<32>(o);
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                        tmem_st32(to + c * 32, o);
                    }
                }
            }
            const float shift = m == -INFINITY ? 0.f : -m;
            uint64_t scale2 = pair(__float_as_uint(scale), __float_as_uint(scale));
            uint64_t shift2 = pair(__float_as_uint(shift), __float_as_uint(shift));
            // The maximum is rounded, the fused products below are not: what that
            // rounding left, up to 1 here, is a power of two that P and l share, but
            // from 2^31 on it would pass fp32's range.  There the scores are rounded
            // as the maximum was.
            if (fabsf(shift) > 0x1p24f) {
#pragma unroll
                for (int e = 0; e < kKeys; ++e)
                    s[e] = __float_as_uint(__fadd_rn(__fmul_rn(__uint_as_float(s[e]), scale), shift));
                scale2 = 0x3F8000003F800000ull;  // (1, 1)
                shift2 = 0ull;
            }
            __syncwarp();
            uint64_t sum[2] = {0ull, 0ull};
#pragma unroll
            for (int c = 0; c < kKeys / 32; ++c) {
                uint32_t pk[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const uint64_t y = fma2(pair(s[c * 32 + 2 * e], s[c * 32 + 2 * e + 1]), scale2, shift2);
                    const float p0 = ex2(__uint_as_float((uint32_t)y));
                    const float p1 = ex2(__uint_as_float((uint32_t)(y >> 32)));
                    sum[e & 1] = add2(sum[e & 1], pair(__float_as_uint(p0), __float_as_uint(p1)));
                    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(pk[e]) : "f"(p1), "f"(p0));
                }
                tmem_st16(ts + c * 16, pk);
                if (c & 1) {
                    tmem_wait_st();
                    fence_before();
                    mbar_arrive(p_ready(t, c >> 1));
                }
            }
            sum[0] = add2(sum[0], sum[1]);
            l += __uint_as_float((uint32_t)sum[0]) + __uint_as_float((uint32_t)(sum[0] >> 32));
        }
        // every product on O done
        if (mine > 0 && ok) {
            ok = mbar_wait_warp(s_full(t), s_phase, abort_flag);
            fence_after();
        }
        if (!ok && lane == 0) atomicOr(&g_prefill_status, HS_ATTN_STATUS_TIMEOUT);
        // a query that sees nothing gets zeros
        const bool whole = a.splits == 1;
        const float inv = !ok ? __int_as_float(0x7FC00000) : !whole ? 1.f : limit == 0 ? 0.f : 1.f / l;
        const bool odd_values = words[2] != 0;
        const int64_t out_row = (int64_t)(q0 + i) * a.heads + head;
        const int64_t part = (int64_t)split * a.n_tok * a.heads + out_row;
        // whole rows leave through shared memory (the tile's queries are not read any
        // more): a row's 256 bytes stored by its thread take 32 cycles of the
        // load-store unit for every 32 of them
        const uint32_t stage = s0 + t * kTileBytes + row * (2 * kV + 16);
        float *part_o = a.part_o + part * kV;
        // (l < 0: no key of this part is seen)
        if (!whole && live) a.part_ml[part] = make_float2(!ok ? inv : m, ok && limit == 0 ? -1.f : l);
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
            uint32_t o[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = 0u;
            __syncwarp();                    // TMEM is read by whole warps
            if (mine > 0) {
                tmem_ld32(to + c * 32, o);
                tmem_wait_ld<32>(o);
            }
#pragma unroll
            for (int e = 0; e < 32; ++e)
                o[e] = limit == 0 && ok ? 0u : __float_as_uint(__uint_as_float(o[e]) * inv);
            if (live && whole) {
                uint32_t y[16];
#pragma unroll
                for (int h = 0; h < 16; ++h)
                    asm("cvt.rn.bf16x2.f32 %0, %1, %2;"
                        : "=r"(y[h])
                        : "f"(__uint_as_float(o[2 * h + 1])), "f"(__uint_as_float(o[2 * h])));
#pragma unroll
                for (int h = 0; h < 4; ++h) st_shared16(stage + c * 64 + h * 16, y + 4 * h);
            } else if (live) {
#pragma unroll
                for (int e = 0; e < 4; ++e) store32(part_o + c * 32 + e * 8, o + e * 8);
            }
        }
        if (odd_values && live) {
            // what was taken out of the values that this query does see
#pragma unroll 1
            for (int d = 0; d < kV; ++d) {
                const bool up = odd[kV + d] < limit, down = odd[2 * kV + d] < limit, none = odd[d] < limit;
                if (!up && !down && !none) continue;
                __nv_bfloat16 *y = reinterpret_cast<__nv_bfloat16 *>(smem + (stage - s0)) + d;
                float x = whole ? __bfloat162float(*y) : part_o[d];
                if (up) x += INFINITY;
                if (down) x -= INFINITY;
                if (none) x = __int_as_float(0x7FC00000);
                if (whole)
                    *y = __float2bfloat16_rn(x);
                else
                    part_o[d] = x;
            }
        }
        if (live && whole) {
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(a.out + out_row * (2 * kV)),
                         "r"(stage), "n"(2 * kV)
                         : "memory");
            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
            asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
        }
        fence_before();
    }
    __syncthreads();
    if (warp == 9) {
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
    }
}

// O = sum_s O_s 2^(m_s - M) / L over a query and head's parts; a warp each.  Parts
// of a weight that is 0 as a float are added too, for what their values hold: an
// infinity or NaN times 0 is NaN (taking such parts out took 0.5 to 1 us longer;
// keeping infinities as they are, 1.5 to 3).
__global__ void __launch_bounds__(256) join_kernel(const PrefillArgs a) {
    const int lane = threadIdx.x & 31;
    const int64_t row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5), rows = (int64_t)a.n_tok * a.heads;
    if (row >= rows) return;
    // queries of no sequence have no parts
    const int tok = (int)(row / a.heads);
    if (tok < __ldg(a.q_starts) || tok >= __ldg(a.q_starts + a.n_seq)) return;
    const float2 x = lane < a.splits ? a.part_ml[lane * rows + row] : make_float2(-INFINITY, -1.f);
    const bool seen = !(x.y < 0.f);
    float M = x.x;
    const bool bad = __any_sync(0xFFFFFFFFu, M != M);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, d));
    const float base = M == -INFINITY ? 0.f : M, f = seen ? ex2(x.x - base) : 0.f;
    float L = seen ? x.y * f : 0.f;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) L += __shfl_xor_sync(0xFFFFFFFFu, L, d);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int s = 0; s < a.splits; ++s) {     // (parts of which nothing is seen are zeros)
        const float w = __shfl_sync(0xFFFFFFFFu, f, s);
        const float4 y = *reinterpret_cast<const float4 *>(a.part_o + (s * rows + row) * kV + lane * 4);
        acc.x = fmaf(y.x, w, acc.x);
        acc.y = fmaf(y.y, w, acc.y);
        acc.z = fmaf(y.z, w, acc.z);
        acc.w = fmaf(y.w, w, acc.w);
    }
    const float inv = bad ? __int_as_float(0x7FC00000) : __any_sync(0xFFFFFFFFu, seen) ? 1.f / L : 0.f;
    uint2 y;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(y.x) : "f"(acc.y * inv), "f"(acc.x * inv));
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(y.y) : "f"(acc.w * inv), "f"(acc.z * inv));
    *reinterpret_cast<uint2 *>(a.out + row * (2 * kV) + lane * 8) = y;
}

bool encode(CUtensorMap *map, const uint8_t *base, int64_t width, int64_t rows, int64_t stride, int box_rows) {
    const EncodeTiled fn = encode_tiled();
    const cuuint64_t dims[2] = {(cuuint64_t)width, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)stride * 2};
    const cuuint32_t box[2] = {64, (cuuint32_t)box_rows}, one[2] = {1, 1};
    return fn && fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<uint8_t *>(base), dims, strides,
                    box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

namespace {
struct Split {
    int parts, small_of;  // small_of: a second part of all / small_of blocks (0: equal parts)
};
}  // namespace

// Parts of a pair's blocks: as many as let the SMs end together soonest.  The
// lengths are on the device, so half a pair is counted for every further sequence,
// and of queries and keys its share.  Measured: a start and end of 3 us, 7 where a
// part is written, a block of two tiles 1.66 us, parts written and read at 5 TB/s
// behind a launch.  Parts are equal, or two of which the smaller ones fill the SMs
// that the last round of the larger ones leaves idle (2048 tokens behind 30000, 16
// heads: 412 us, 452 whole; 512 behind 9000, 64 heads: 142, 177).
Split latent_prefill_split(int n_tok, int n_keys, int n_seq, int heads) {
    const int64_t pairs = ((int64_t)n_tok + 2 * kRows - 1) / (2 * kRows) + (n_seq - 1) / 2, items = pairs * heads;
    // blocks of a sequence's longest, shortest and average pair
    const double most = std::max(std::ceil((double)n_keys / n_seq / kKeys), 1.);
    const double least = std::max(most - std::max((double)n_tok / n_seq - 2 * kRows, 0.) / kKeys, 1.);
    const double mean = 0.5 * (most + least);
    // `n` equal items in rounds, or, longest first, all SMs busy up to one of the shortest
    auto time = [&](double n, double start, double of) {
        const double rounds = std::ceil(n / kSms) * (start + 1.66 * std::ceil(most / of));
        return std::min(rounds, n / kSms * (start + 1.66 * mean / of) + start + 1.66 * std::ceil(least / of));
    };
    auto parts_time = [&](int s) { return 3. + (double)s * n_tok * heads * (kV * 4 + 8) * 2 / 5e6; };
    Split best = {1, 0};
    double soonest = time((double)items, 3., 1.);
    auto consider = [&](double t, Split split) {
        if (t < soonest) {
            soonest = t;
            best = split;
        }
    };
    for (int s = 2; s <= kMaxPrefillSplits && s <= most; ++s)
        consider(time((double)items * s, 3., s) + parts_time(s), {s, 0});
    // in the last round of the larger parts `idle` SMs take c smaller ones each:
    // 7 + 1.66 (most - small) = c (7 + 1.66 small)
    const int64_t rounds = (items + kSms - 1) / kSms, idle = rounds * kSms - items;
    if (idle > 0) {
        const int64_t c = (items + idle - 1) / idle;
        const double even = (1.66 * most - 7. * (c - 1)) / (1.66 * (c + 1));
        if (even >= 1.) {
            const double of = std::ceil(most / even), small = std::ceil(most / of), large = 7. + 1.66 * (most - small);
            const double t = rounds * large + std::max(c * (7. + 1.66 * small) - large, 0.);
            consider(std::min(t, (double)items / kSms * (14. + 1.66 * mean) + 7. + 1.66 * std::ceil(least / of)) +
                         parts_time(2),
                     {2, (int)of});
        }
    }
    return best;
}

size_t latent_prefill_bytes(int n_tok, int n_keys, int n_seq, int heads) {
    const int s = latent_prefill_split(n_tok, n_keys, n_seq, heads).parts;
    // (16 bytes more, so that the parts can start on 32)
    return s == 1 ? 0 : (size_t)s * n_tok * heads * (kV * 4 + 8) + 16;
}

cudaError_t launch_latent_prefill(PrefillArgs a, void *work, cudaStream_t st) {
    CUtensorMap q, k, kr, v;
    const int64_t width = (int64_t)(a.heads - 1) * a.kv_head_stride + 128;
    // without a key nothing is loaded: the maps only have to be valid
    const int64_t keys = a.n_keys > 0 ? a.n_keys : 1;
    if (!encode(&q, a.q, (int64_t)a.heads * kQk, a.n_tok, (int64_t)a.heads * kQk, kRows) ||
        !encode(&k, a.k, width, keys, a.kv_stride, kKeys) || !encode(&kr, a.kr, 64, keys, a.kr_stride, kKeys) ||
        !encode(&v, a.v, width, keys, a.kv_stride, 64))
        return cudaErrorInvalidValue;
    const cudaError_t e =
        cudaFuncSetAttribute(prefill_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
    if (e != cudaSuccess) return e;
    const int places = a.n_tok / (2 * kRows) + a.n_seq;
    const int64_t rows = (int64_t)a.n_tok * a.heads;
    const Split split = latent_prefill_split(a.n_tok, a.n_keys, a.n_seq, a.heads);
    a.splits = split.parts;
    a.small_of = split.small_of;
    a.head_group = std::min(a.heads, kHeadGroup);
    a.part_o = reinterpret_cast<float *>((reinterpret_cast<uintptr_t>(work) + 31) & ~(uintptr_t)31);
    a.part_ml = reinterpret_cast<float2 *>(a.part_o + a.splits * rows * kV);
    prefill_kernel<<<(unsigned)((int64_t)places * a.heads * a.splits), kPrefillThreads, kSmem, st>>>(q, k, kr, v, a,
                                                                                                 places);
    if (a.splits > 1) join_kernel<<<(unsigned)((rows + 7) / 8), 256, 0, st>>>(a);
    return cudaGetLastError();
}

cudaError_t prefill_status(uint32_t *status) {
    uint32_t v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_prefill_status, sizeof(v));
    if (e != cudaSuccess) return e;
    *status = v;
    if (v) {
        const uint32_t zero = 0;
        e = cudaMemcpyToSymbol(g_prefill_status, &zero, sizeof(zero));
    }
    return e;
}

}  // namespace hs
