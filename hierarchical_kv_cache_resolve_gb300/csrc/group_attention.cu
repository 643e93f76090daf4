// Attention of grouped query heads over per-head token records: over each
// request's published rows, and joined with the partial results of
// prefix_attention.cu over a prefix that all requests share
// (hs_prefix_attention), or with every row's weight added to its position's
// running sum (hs_sparse_attention_weights).
//
// Softmax over a split set of rows: each part keeps m = max s (base 2, scaled),
// l = sum 2^(s - m) and O = sum 2^(s - m) V; parts join as
//   M = max m_p,  O = sum 2^(m_p - M) O_p / sum 2^(m_p - M) l_p.
//
// rows_kernel gathers the published rows.  About one multiply-add per byte
// and query head: bound by HBM at any group size, so it is built to keep the
// gather busy.  The rows of all requests form one list of tiles of 16, cut
// into equal contiguous ranges, one per CTA and one CTA per SM: no request
// count leaves SMs idle.  A warp owns one key-value head (with fewer than
// five heads, several warps take a head's tiles in turn) and runs alone: it
// copies its head's 256-byte key and value blocks of 16 rows at a time into
// a ring of its own with 16-byte asynchronous copies, zero-filled where a row
// is masked, so the pipeline needs no barrier between warps and no wait that
// could run out.  A request's 1 to 16 query heads of the warp's key-value
// head are the 16 rows of a warp-level bf16 MMA (fp32 accumulators);
// tcgen05's smallest tile has 64 rows, and a gathered row would have to be
// spread over its swizzled layout.  P V takes P as the sum of two bf16 terms
// (error 2^-17), which costs MMAs that the gather leaves idle.
//
// merge_kernel joins the parts, rounds once to bf16, and, for the weights,
// turns the scores that rows_kernel left in the workspace into softmax
// weights summed over the query heads, one thread per row: one addition per
// position and call, so equal inputs give equal sums.
#include <cmath>
#include <cstdint>

#include "hs.h"
#include "hs_internal.cuh"

namespace hs {
namespace {

constexpr int kDim = 128;
constexpr int kTile = 16;                      // rows per tile
constexpr int kRing = 3;                       // tiles in a warp's ring
constexpr int kTileBytes = kTile * 2 * kDim;   // 4096: keys or values of a tile
constexpr int kWarpSmem = kRing * 2 * kTileBytes;
constexpr int kMaxWarps = 8;
constexpr int kMergeThreads = 256;
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

template <bool kScores>
__global__ void __launch_bounds__(kMaxWarps * 32, 1)
    rows_kernel(const GroupArgs a, const RowsPlan p) {
    extern __shared__ __align__(128) uint8_t smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int head = warp % a.heads, sub = warp / a.heads;
    const int group = a.q_heads / a.heads;
    const int64_t W = (int64_t)a.heads * 4 * kDim;
    const int64_t t0 = (int64_t)blockIdx.x * p.total / gridDim.x;
    const int64_t t1 = (int64_t)(blockIdx.x + 1) * p.total / gridDim.x;
    const int r0 = (int)(t0 / p.tiles), r1 = (int)((t1 - 1) / p.tiles);
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

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    uint32_t valid_q[kRing];           // masks of the tiles in the ring, oldest first
#pragma unroll
    for (int b = 0; b < kRing - 1; ++b) valid_q[b] = issue(b);
    int at = 0;                        // ring place of the oldest tile
    const int h0 = lane >> 2, c2 = (lane & 3) * 2;

    for (int r = r0; r <= r1; ++r) {
        // this head's queries as MMA A fragments; rows past the group are zero
        uint32_t qa[8][4];
        {
            const uint8_t *q = a.q + ((int64_t)r * a.q_heads + head * group) * (2 * kDim) + c2 * 2;
#pragma unroll
            for (int s = 0; s < 8; ++s)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int row = h0 + (i & 1) * 8;
                    qa[s][i] = row < group ? *reinterpret_cast<const uint32_t *>(
                                                 q + row * 2 * kDim + s * 32 + (i >> 1) * 16)
                                           : 0u;
                }
        }
        float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
        float o[16][4];
#pragma unroll
        for (int n = 0; n < 16; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[n][i] = 0.f;

        for (int64_t t = seg_first(r) + sub; t < seg_end(r); t += p.subs) {
            valid_q[kRing - 1] = issue(at >= 1 ? at - 1 : kRing - 1);
            asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 1) : "memory");
            __syncwarp();
            const uint32_t ks = ring + at * 2 * kTileBytes, vs = ks + kTileBytes;
            const uint32_t valid = valid_q[0];

            float s[2][4];
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) s[n][i] = 0.f;
            {
                const int key = (lane & 7) + (lane >> 4) * 8;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    uint32_t b[4];
                    ldsm_x4(b, ks + swz(key, 2 * i + ((lane >> 3) & 1)));
                    mma_bf16(s[0], qa[i], b[0], b[1]);
                    mma_bf16(s[1], qa[i], b[2], b[3]);
                }
            }
            float x0 = -INFINITY, x1 = -INFINITY;
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const bool v = valid >> (n * 8 + c2 + i) & 1u;
                    s[n][i] = v ? s[n][i] * a.scale_log2 : -INFINITY;
                    s[n][2 + i] = v ? s[n][2 + i] * a.scale_log2 : -INFINITY;
                    x0 = fmaxf(x0, s[n][i]);
                    x1 = fmaxf(x1, s[n][2 + i]);
                }
            if (kScores) {
                const int j0 = (int)(t - (int64_t)r * p.tiles) * kTile + c2;
                float *sc = a.scores + ((int64_t)r * a.q_heads + head * group) * a.k;
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int j = j0 + n * 8 + i;
                        if (j < a.k) {
                            if (h0 < group) sc[(int64_t)h0 * a.k + j] = s[n][i];
                            if (h0 + 8 < group) sc[(int64_t)(h0 + 8) * a.k + j] = s[n][2 + i];
                        }
                    }
            }
#pragma unroll
            for (int d = 1; d <= 2; d <<= 1) {
                x0 = fmaxf(x0, __shfl_xor_sync(0xFFFFFFFFu, x0, d));
                x1 = fmaxf(x1, __shfl_xor_sync(0xFFFFFFFFu, x1, d));
            }
            const float n0 = fmaxf(m0, x0), n1 = fmaxf(m1, x1);
            // a row with nothing so far: exponents from 0, all its terms 2^-inf
            const float b0 = n0 == -INFINITY ? 0.f : n0, b1 = n1 == -INFINITY ? 0.f : n1;
            const float f0 = exp2f(m0 - b0), f1 = exp2f(m1 - b1);
            m0 = n0;
            m1 = n1;
            uint32_t ph[4], pl[4];
            l0 *= f0;
            l1 *= f1;
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                const float p00 = exp2f(s[n][0] - b0), p01 = exp2f(s[n][1] - b0);
                const float p10 = exp2f(s[n][2] - b1), p11 = exp2f(s[n][3] - b1);
                l0 += p00 + p01;
                l1 += p10 + p11;
                split_bf16(p00, p01, ph[n * 2], pl[n * 2]);
                split_bf16(p10, p11, ph[n * 2 + 1], pl[n * 2 + 1]);
            }
#pragma unroll
            for (int n = 0; n < 16; ++n) {
                o[n][0] *= f0;
                o[n][1] *= f0;
                o[n][2] *= f1;
                o[n][3] *= f1;
            }
            {
                const int key = (lane & 7) + ((lane >> 3) & 1) * 8;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    uint32_t b[4];
                    ldsm_x4_t(b, vs + swz(key, 2 * i + (lane >> 4)));
                    mma_bf16(o[2 * i], ph, b[0], b[1]);
                    mma_bf16(o[2 * i + 1], ph, b[2], b[3]);
                    mma_bf16(o[2 * i], pl, b[0], b[1]);
                    mma_bf16(o[2 * i + 1], pl, b[2], b[3]);
                }
            }
            __syncwarp();  // every lane has read this place before it is refilled
#pragma unroll
            for (int b = 0; b < kRing - 1; ++b) valid_q[b] = valid_q[b + 1];
            at = at + 1 == kRing ? 0 : at + 1;
        }

        // this part: the CTA's rows of request r (of this warp's turn)
#pragma unroll
        for (int d = 1; d <= 2; d <<= 1) {
            l0 += __shfl_xor_sync(0xFFFFFFFFu, l0, d);
            l1 += __shfl_xor_sync(0xFFFFFFFFu, l1, d);
        }
        const int64_t part = ((int64_t)blockIdx.x + r) * p.subs + sub;
        const int64_t row = part * a.q_heads + head * group;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int g = h0 + half * 8;
            if (g >= group) continue;
            float *dst = p.o + (row + g) * kDim + c2;
#pragma unroll
            for (int n = 0; n < 16; ++n)
                *reinterpret_cast<float2 *>(dst + n * 8) =
                    make_float2(o[n][half * 2], o[n][half * 2 + 1]);
            if ((lane & 3) == 0)
                p.ml[row + g] = half ? make_float2(m1, l1) : make_float2(m0, l0);
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    // the merge that waits for this grid reads the prefix kernel's parts too
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

// The parts of one request: the prefix kernel's splits, then the CTAs that
// had some of its rows.
struct Parts {
    int n_prefix, n;
    int64_t rows_first;
};

__device__ __forceinline__ Parts parts_of(const RowsPlan &p, int n_prefix, int r) {
    Parts x = {n_prefix, n_prefix, 0};
    if (p.total > 0) {
        // the CTA that has tile t: the last c with c * total / ctas <= t
        const int64_t first = (((int64_t)r * p.tiles + 1) * p.ctas - 1) / p.total;
        const int64_t last = (((int64_t)(r + 1) * p.tiles) * p.ctas - 1) / p.total;
        x.rows_first = (first + r) * p.subs;
        x.n = n_prefix + (int)(last - first + 1) * p.subs;
    }
    return x;
}

// row of part i of (request, query head) in the two part arrays
__device__ __forceinline__ int64_t part_row(const GroupArgs &a, const Parts &x, int i, int r,
                                            int hq) {
    return i < x.n_prefix ? ((int64_t)i * a.n_req + r) * a.q_heads + hq
                          : (x.rows_first + i - x.n_prefix) * a.q_heads + hq;
}

// M = max of the parts' maxima and L = sum 2^(m - M) l of (request, query
// head), by one warp; the same in every lane.
__device__ __forceinline__ float2 join(const GroupArgs &a, const RowsPlan &p, const PrefixPlan &pp,
                                       const Parts &x, int r, int hq, int lane) {
    float M = -INFINITY, L = 0.f;
    bool bad = false;
    for (int i = lane; i < x.n; i += 32) {
        const float2 ml = (i < x.n_prefix ? pp.ml : p.ml)[part_row(a, x, i, r, hq)];
        const float big = fmaxf(M, ml.x), base = big == -INFINITY ? 0.f : big;
        L = L * exp2f(M - base) + ml.y * exp2f(ml.x - base);
        M = big;
        bad |= ml.x != ml.x;               // a part that a wait gave up on
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) {
        const float m2 = __shfl_xor_sync(0xFFFFFFFFu, M, d);
        const float l2 = __shfl_xor_sync(0xFFFFFFFFu, L, d);
        const float big = fmaxf(M, m2), base = big == -INFINITY ? 0.f : big;
        L = L * exp2f(M - base) + l2 * exp2f(m2 - base);
        M = big;
    }
    if (__any_sync(0xFFFFFFFFu, bad)) M = __int_as_float(0x7FC00000);
    return make_float2(M == -INFINITY ? 0.f : M, L);
}

// The first out_blocks CTAs write outputs, `share` warps to a (request, query
// head), four dimensions per lane; the others the weights of 256 rows each.
__global__ void __launch_bounds__(kMergeThreads)
    merge_kernel(const GroupArgs a, const RowsPlan p, const PrefixPlan pp, int out_blocks,
                 int share) {
    __shared__ float4 sum[kMergeThreads];
    __shared__ float2 mi[128];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if ((int)blockIdx.x < out_blocks) {
        const int turn = warp % share;
        const int64_t unit = ((int64_t)blockIdx.x * (kMergeThreads / 32) + warp) / share;
        const bool live = unit < (int64_t)a.n_req * a.q_heads;
        const int r = live ? (int)(unit / a.q_heads) : 0, hq = live ? (int)(unit % a.q_heads) : 0;
        Parts x = parts_of(p, pp.splits, r);
        if (!live) x.n = 0;
        const float2 ML = join(a, p, pp, x, r, hq, lane);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        constexpr int kLoads = 4;
        for (int i0 = turn; i0 < x.n; i0 += kLoads * share) {
            float4 v[kLoads];
            float m[kLoads];
#pragma unroll
            for (int u = 0; u < kLoads; ++u) {
                const int i = i0 + u * share;
                if (i >= x.n) continue;
                const int64_t row = part_row(a, x, i, r, hq);
                v[u] = *reinterpret_cast<const float4 *>((i < x.n_prefix ? pp.o : p.o) +
                                                         row * kDim + lane * 4);
                m[u] = (i < x.n_prefix ? pp.ml : p.ml)[row].x;
            }
#pragma unroll
            for (int u = 0; u < kLoads; ++u) {
                if (i0 + u * share >= x.n) continue;
                const float w = exp2f(m[u] - ML.x);
                acc.x += w * v[u].x;
                acc.y += w * v[u].y;
                acc.z += w * v[u].z;
                acc.w += w * v[u].w;
            }
        }
        sum[threadIdx.x] = acc;
        __syncthreads();
        if (turn != 0 || !live) return;
        for (int s = 1; s < share; ++s) {
            const float4 v = sum[threadIdx.x + s * 32];
            acc.x += v.x;
            acc.y += v.y;
            acc.z += v.z;
            acc.w += v.w;
        }
        const float inv = ML.y == 0.f ? 0.f : 1.f / ML.y;  // no row at all: zeros
        uint2 v;
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(v.x) : "f"(acc.y * inv), "f"(acc.x * inv));
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(v.y) : "f"(acc.w * inv), "f"(acc.z * inv));
        *reinterpret_cast<uint2 *>(a.out + unit * (2 * kDim) + lane * 8) = v;
        return;
    }
    // weights: 256 rows of one request; its maximum and sum per query head first
    const int64_t chunk = (int64_t)blockIdx.x - out_blocks;
    const int per_req = (a.k + kMergeThreads - 1) / kMergeThreads;
    const int r = (int)(chunk / per_req);
    const int j = (int)(chunk % per_req) * kMergeThreads + threadIdx.x;
    const Parts x = parts_of(p, 0, r);
    for (int hq = warp; hq < a.q_heads; hq += kMergeThreads / 32) {
        const float2 ML = join(a, p, pp, x, r, hq, lane);
        if (lane == 0) mi[hq] = make_float2(ML.x, ML.y == 0.f ? 0.f : 1.f / ML.y);
    }
    __syncthreads();
    if (j >= a.k) return;
    const int32_t req = a.req_ids ? a.req_ids[r] : r;
    const int32_t pos = a.sel[(int64_t)r * a.k + j];
    if (req < 0 || req >= a.weight_rows || pos < 0 || pos >= a.n_positions) return;
    const float *sc = a.scores + (int64_t)r * a.q_heads * a.k + j;
    float w = 0.f;
#pragma unroll 8
    for (int hq = 0; hq < a.q_heads; ++hq)
        w += exp2f(sc[(int64_t)hq * a.k] - mi[hq].x) * mi[hq].y;
    // exactly one addition per position and call where positions differ
    if (w != 0.f) atomicAdd(a.weights + (int64_t)req * a.n_positions + pos, w);
}

// Tiles and CTAs for n_req requests of k rows: one CTA per SM, no more than
// one tile for each of a CTA's turns.
RowsPlan rows_plan(int n_req, int heads, int k) {
    RowsPlan p = {};
    p.subs = kMaxWarps / heads;
    p.tiles = (k + kTile - 1) / kTile;
    p.total = (int64_t)n_req * p.tiles;
    const int64_t most = (p.total + p.subs - 1) / p.subs;
    p.ctas = (int)(most < kSms ? most : kSms);
    return p;
}

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

size_t rows_parts(const RowsPlan &p, int n_req) {
    return p.total > 0 ? ((size_t)p.ctas + n_req - 1) * p.subs : 0;
}

// Lays the part arrays out from byte `at` of the workspace (16-byte aligned;
// null to count only); the byte behind them.
template <class Plan>
size_t place(Plan *p, size_t parts, uint8_t *work, size_t at, int q_heads) {
    const size_t rows = parts * q_heads;
    p->o = reinterpret_cast<float *>(work + at);
    at = align256(at + rows * kDim * 4);
    p->ml = reinterpret_cast<float2 *>(work + at);
    return align256(at + rows * sizeof(float2));
}

size_t place_both(PrefixPlan *pp, RowsPlan *p, uint8_t *work, int n_req, int q_heads) {
    const size_t at = place(pp, (size_t)pp->splits * n_req, work, 0, q_heads);
    return place(p, rows_parts(*p, n_req), work, at, q_heads);
}

template <bool kScores>
cudaError_t launch_rows(const GroupArgs &a, const RowsPlan &p, bool overlap, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.ctas);
    cfg.blockDim = dim3(a.heads * p.subs * 32);
    cfg.dynamicSmemBytes = (size_t)a.heads * p.subs * kWarpSmem;
    cfg.stream = st;
    cudaError_t e = cudaFuncSetAttribute(rows_kernel<kScores>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         kMaxWarps * kWarpSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = overlap ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, rows_kernel<kScores>, a, p);
}

cudaError_t launch_merge(const GroupArgs &a, const RowsPlan &p, const PrefixPlan &pp,
                         cudaStream_t st) {
    constexpr int kWarps = kMergeThreads / 32;
    // warps to an output: a round of four loads each, about
    const int64_t rows_parts_each = p.total > 0 ? ((int64_t)p.ctas / a.n_req + 2) * p.subs : 0;
    int share = 1;
    while (share < kWarps && pp.splits + rows_parts_each > 4 * share) share *= 2;
    const int64_t units = (int64_t)a.n_req * a.q_heads;
    const int out_blocks = (int)((units * share + kWarps - 1) / kWarps);
    const int64_t weight_blocks =
        a.weights ? (int64_t)a.n_req * ((a.k + kMergeThreads - 1) / kMergeThreads) : 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(out_blocks + weight_blocks));
    cfg.blockDim = dim3(kMergeThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, merge_kernel, a, p, pp, out_blocks, share);
}

}  // namespace

size_t prefix_attention_bytes(int n_req, int q_heads, int heads, int64_t prefix_len, int k) {
    PrefixPlan pp = prefix_plan(n_req, q_heads, heads, prefix_len);
    RowsPlan p = rows_plan(n_req, heads, k);
    return place_both(&pp, &p, nullptr, n_req, q_heads);
}

size_t attention_weights_bytes(int n_req, int q_heads, int heads, int k) {
    PrefixPlan none = {};
    RowsPlan p = rows_plan(n_req, heads, k);
    return place_both(&none, &p, nullptr, n_req, q_heads) +
           (size_t)n_req * q_heads * k * sizeof(float);
}

cudaError_t launch_prefix_attention(GroupArgs a, void *work, cudaStream_t st) {
    PrefixPlan pp = prefix_plan(a.n_req, a.q_heads, a.heads, a.prefix_len);
    RowsPlan p = rows_plan(a.n_req, a.heads, a.k);
    place_both(&pp, &p, static_cast<uint8_t *>(work), a.n_req, a.q_heads);
    if (pp.splits > 0) {
        const cudaError_t e = launch_prefix(a, pp, st);
        if (e != cudaSuccess) return e;
    }
    if (p.total > 0) {
        const cudaError_t e = launch_rows<false>(a, p, pp.splits > 0, st);
        if (e != cudaSuccess) return e;
    }
    return launch_merge(a, p, pp, st);
}

cudaError_t launch_attention_weights(GroupArgs a, void *work, cudaStream_t st) {
    PrefixPlan none = {};
    RowsPlan p = rows_plan(a.n_req, a.heads, a.k);
    uint8_t *const w = static_cast<uint8_t *>(work);
    a.scores = reinterpret_cast<float *>(w + place_both(&none, &p, w, a.n_req, a.q_heads));
    const cudaError_t e = launch_rows<true>(a, p, false, st);
    return e == cudaSuccess ? launch_merge(a, p, none, st) : e;
}

}  // namespace hs
