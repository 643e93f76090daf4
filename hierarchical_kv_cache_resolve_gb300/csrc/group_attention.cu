// Attention of grouped query heads over per-head token records in parts, and
// what joins them: hs_prefix_attention's parts come from prefix_attention.cu
// (the shared prefix, and the requests' own rows beside it),
// hs_sparse_attention_weights' from the rows kernel here (rows_gather.cuh).
//
// Softmax over a split set of rows: each part keeps m = max s (base 2, scaled),
// l = sum 2^(s - m) and O = sum 2^(s - m) V; parts join as
//   M = max m_p,  O = sum 2^(m_p - M) O_p / sum 2^(m_p - M) l_p.
//
// merge_kernel joins the parts, rounds once to bf16, and, for the weights,
// turns the scores that rows_kernel left in the workspace into softmax
// weights summed over the query heads, one thread per row: one addition per
// position and call, so equal inputs give equal sums.
//
// Measured: hs_sparse_attention_weights 51.6 us for 32 requests of 2048 rows of
// 4096 bytes and 32 query heads (rows 43 us at 6.2 TB/s, merge and weights 8),
// 5.4 us for one request of 64 rows.
#include <cmath>
#include <cstdint>

#include "hs.h"
#include "hs_internal.cuh"
#include "rows_gather.cuh"

namespace hs {
namespace {

constexpr int kDim = 128;
constexpr int kMergeThreads = 256;

__device__ uint32_t g_rows_status;

template <bool kScores>
__global__ void __launch_bounds__(rows::kMaxWarps * 32 + 128, 1)
    rows_kernel(const GroupArgs a, const RowsPlan p) {
    extern __shared__ __align__(128) uint8_t smem[];
    const int w = (int)threadIdx.x / 32 - a.heads * p.subs;  // from 0: those that bring
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (w == 0) rows::init(a, smem);
    __syncthreads();
    if (w >= 0)
        rows::bring(a, p, blockIdx.x, smem, w);
    else
        rows::attend<kScores>(a, p, blockIdx.x, smem, &g_rows_status);
}

// The parts of one request and key-value head: those of the prefix, then the
// CTAs that had some of the request's rows.
struct Parts {
    int n_prefix, n;
    int prefix_first, rows_first;
};

// Of n ranges c * total / n of total = things * each, the one that holds the
// first of thing i's `each` parts, and the one that holds the last:
// ((i * each + 1) * n - 1) / total and ((i + 1) * each * n - 1) / total, less
// the common factor; lead = (n - 1) / each.
__device__ __forceinline__ int first_range(int i, int n, int lead, int things) {
    return (i * n + lead) / things;
}
__device__ __forceinline__ int last_range(int i, int n, int things) {
    return ((i + 1) * n - 1) / things;
}

__device__ __forceinline__ Parts parts_of(const GroupArgs &a, const RowsPlan &p,
                                          const PrefixPlan &pp, int r, int head) {
    Parts x = {0, 0, 0, 0};
    if (pp.groups > 0) {
        const int first = first_range(head, pp.groups, pp.lead, a.heads);
        x.prefix_first = first + head;
        x.n_prefix = x.n = last_range(head, pp.groups, a.heads) - first + 1;
    }
    if (p.ctas > 0) {
        const int first = first_range(r, p.ctas, p.lead, a.n_req);
        x.rows_first = (first + r) * p.subs;
        x.n += (last_range(r, p.ctas, a.n_req) - first + 1) * p.subs;
    }
    return x;
}

// row of part i of (request, query head) in the two part arrays
__device__ __forceinline__ int64_t part_row(const GroupArgs &a, const Parts &x, int i, int r,
                                            int hq) {
    const int group = a.q_heads / a.heads;
    return i < x.n_prefix
               ? (int64_t)((x.prefix_first + i) * a.n_req + r) * group + hq % group
               : (int64_t)(x.rows_first + i - x.n_prefix) * a.q_heads + hq;
}

// The first out_blocks CTAs write outputs, `share` warps to a (request, query
// head), four dimensions per lane; the others the weights of 256 rows each.
// Little work behind long latencies, so each warp loads the (m, l) and the O
// of eight parts at once.
__global__ void __launch_bounds__(kMergeThreads)
    merge_kernel(const GroupArgs a, const RowsPlan p, const PrefixPlan pp, int out_blocks,
                 int share) {
    __shared__ float4 sum[kMergeThreads];
    __shared__ float2 mi[128];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if ((int)blockIdx.x < out_blocks) {
        const int turn = warp % share;
        // (request, query head) pairs: at most 65535 * 128
        const int unit = (int)(blockIdx.x * (kMergeThreads / 32) + warp) / share;
        const bool live = unit < a.n_req * a.q_heads;
        const int r = live ? unit / a.q_heads : 0, hq = live ? unit - r * a.q_heads : 0;
        Parts x = parts_of(a, p, pp, r, hq / (a.q_heads / a.heads));
        if (!live) x.n = 0;
        float M = -INFINITY, L = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        asm volatile("griddepcontrol.wait;" ::: "memory");
        constexpr int kLoads = 8;
        for (int i0 = turn; i0 < x.n; i0 += kLoads * share) {
            float4 v[kLoads];
            float2 ml[kLoads];
#pragma unroll
            for (int u = 0; u < kLoads; ++u) {
                const int i = i0 + u * share;
                ml[u] = make_float2(-INFINITY, 0.f);
                v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (i >= x.n) continue;
                const int64_t row = part_row(a, x, i, r, hq);
                ml[u] = (i < x.n_prefix ? pp.ml : p.ml)[row];
                v[u] = *reinterpret_cast<const float4 *>((i < x.n_prefix ? pp.o : p.o) +
                                                         row * kDim + lane * 4);
            }
            float big = M;
#pragma unroll
            for (int u = 0; u < kLoads; ++u) big = fmaxf(big, ml[u].x);
            const float base = big == -INFINITY ? 0.f : big;
            const float f = exp2f(M - base);
            M = big;
            L *= f;
            acc.x *= f;
            acc.y *= f;
            acc.z *= f;
            acc.w *= f;
#pragma unroll
            for (int u = 0; u < kLoads; ++u) {
                const float w = exp2f(ml[u].x - base);  // NaN: a part that a wait gave up on
                L += w * ml[u].y;
                acc.x += w * v[u].x;
                acc.y += w * v[u].y;
                acc.z += w * v[u].z;
                acc.w += w * v[u].w;
            }
        }
        if (share > 1) {                       // the same for the whole grid
            sum[threadIdx.x] = acc;
            if (lane == 0) mi[warp] = make_float2(M, L);
            __syncthreads();
            if (turn != 0) return;
            float big = M;
            for (int s = 1; s < share; ++s) big = fmaxf(big, mi[warp + s].x);
            const float base = big == -INFINITY ? 0.f : big;
            acc = make_float4(0.f, 0.f, 0.f, 0.f);
            L = 0.f;
            for (int s = 0; s < share; ++s) {
                const float2 ml = mi[warp + s];
                const float4 v = sum[threadIdx.x + s * 32];
                const float w = exp2f(ml.x - base);
                L += w * ml.y;
                acc.x += w * v.x;
                acc.y += w * v.y;
                acc.z += w * v.z;
                acc.w += w * v.w;
            }
        }
        if (!live) return;
        const float inv = L == 0.f ? 0.f : 1.f / L;  // no row at all: zeros
        uint2 v;
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(v.x) : "f"(acc.y * inv), "f"(acc.x * inv));
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(v.y) : "f"(acc.w * inv), "f"(acc.z * inv));
        *reinterpret_cast<uint2 *>(a.out + (int64_t)unit * (2 * kDim) + lane * 8) = v;
        return;
    }
    // weights: 256 rows of one request; its maximum and sum per query head
    // first, by 2 to 32 lanes each
    const int chunk = (int)blockIdx.x - out_blocks;
    const int per_req = (a.k + kMergeThreads - 1) / kMergeThreads;
    const int r = chunk / per_req;
    const int j = (chunk - r * per_req) * kMergeThreads + threadIdx.x;
    const Parts x = parts_of(a, p, pp, r, 0);  // (no prefix)
    int lanes = 2;
    while (lanes < 32 && 2 * lanes * a.q_heads <= kMergeThreads) lanes *= 2;
    const int32_t req = a.req_ids ? a.req_ids[r] : r;
    const int32_t pos = j < a.k ? a.sel[(int64_t)r * a.k + j] : -1;
    // (a masked row's score alone would not do: 2^-inf times a NaN sum is NaN)
    const int32_t row = j < a.k ? __ldg(a.idx + (int64_t)r * a.k + j) : -1;
    const bool live = row >= 0 && (int64_t)row < a.cache_rows && req >= 0 && req < a.weight_rows &&
                      pos >= 0 && pos < a.n_positions;
    const float *sc = a.scores + (int64_t)r * a.q_heads * a.k + j;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // With few blocks the first heads' scores are loaded while the maxima are on
    // their way (1 x 64 rows 6.4 -> 5.5 us, 5 x 777 8.4 -> 7.3); with many the
    // maxima would wait behind them (32 x 2048 50.9 -> 51.9).
    constexpr int kFirst = 16;
    float first[kFirst];
    const int early = gridDim.x > kSms ? 0 : a.q_heads < kFirst ? a.q_heads : kFirst;
    {
        const int hq = threadIdx.x / lanes, turn = threadIdx.x % lanes;
        float M = -INFINITY, L = 0.f;
        float2 next = make_float2(-INFINITY, 0.f);
        const int n = hq < a.q_heads ? x.n : 0;
        if (turn < n) next = p.ml[part_row(a, x, turn, r, hq)];
        asm volatile("" ::: "memory");      // these first
#pragma unroll
        for (int u = 0; u < kFirst; ++u)
            first[u] = live && u < early ? sc[(int64_t)u * a.k] : -INFINITY;
        if (hq < a.q_heads)
            for (int i = turn; i < x.n; i += lanes) {
                const float2 ml = next;
                if (i + lanes < x.n) next = p.ml[part_row(a, x, i + lanes, r, hq)];
                const float big = fmaxf(M, ml.x), base = big == -INFINITY ? 0.f : big;
                L = L * exp2f(M - base) + ml.y * exp2f(ml.x - base);
                M = big;
            }
        for (int d = lanes / 2; d; d >>= 1) {
            const float m2 = __shfl_xor_sync(0xFFFFFFFFu, M, d);
            const float l2 = __shfl_xor_sync(0xFFFFFFFFu, L, d);
            const float big = fmaxf(M, m2), base = big == -INFINITY ? 0.f : big;
            L = L * exp2f(M - base) + l2 * exp2f(m2 - base);
            M = big;
        }
        if (hq < a.q_heads && turn == 0)
            mi[hq] = make_float2(M == -INFINITY ? 0.f : M, L == 0.f ? 0.f : 1.f / L);
    }
    __syncthreads();
    if (!live) return;
    float w = 0.f;
#pragma unroll
    for (int u = 0; u < kFirst; ++u)
        if (u < early) w += exp2f(first[u] - mi[u].x) * mi[u].y;
#pragma unroll 16
    for (int hq = early; hq < a.q_heads; ++hq)
        w += exp2f(sc[(int64_t)hq * a.k] - mi[hq].x) * mi[hq].y;
    // exactly one addition per position and call where positions differ
    if (w != 0.f) atomicAdd(a.weights + (int64_t)req * a.n_positions + pos, w);
}

// Tiles of n_req requests of k rows over at most `ctas` CTAs, no more than one
// tile for each of a CTA's turns.
RowsPlan rows_plan(int n_req, int heads, int k, int ctas) {
    RowsPlan p = {};
    p.subs = rows::kMaxWarps / heads;
    p.tiles = (k + rows::kTile - 1) / rows::kTile;
    p.total = (int64_t)n_req * p.tiles;
    const int64_t most = (p.total + p.subs - 1) / p.subs;
    p.ctas = (int)(most < ctas ? most : ctas);
    if (p.ctas > 0) {
        p.each = p.total / p.ctas;
        p.rest = (int)(p.total % p.ctas);
        p.lead = (p.ctas - 1) / p.tiles;
    }
    return p;
}

// How hs_prefix_attention shares the SMs out between the prefix and the
// requests' own rows: so that both are done at about the same time, by what
// they were measured to cost (in cycles): the prefix as its plan says; a tile
// of 16 rows 1500 for each warp, and 2600 where the prefix is bound by HBM too
// (one pair).
void share_out(int n_req, int q_heads, int heads, int64_t prefix_len, int k, PrefixPlan *pp,
               RowsPlan *p) {
    *pp = prefix_plan(n_req, q_heads, heads, prefix_len, kSms);
    *p = rows_plan(n_req, heads, k, kSms);
    if (pp->groups == 0 || p->total == 0) return;
    const int pairs = (pp->row_tiles + 1) / 2;
    // with `ctas` of the SMs for the rows: the plans; the time, and whether it
    // is the rows'
    auto split = [&](int ctas, bool *rows_last) {
        *pp = prefix_plan(n_req, q_heads, heads, prefix_len, kSms - ctas);
        // what the groups leave over goes to the rows
        const int left = kSms - pp->groups * pairs;
        *p = rows_plan(n_req, heads, k, left > ctas ? left : ctas);
        const int waves = (pp->groups * pairs + p->ctas + kSms - 1) / kSms;
        const double tx = waves * pp->cycles;
        const int turns = p->ctas * p->subs;
        const double ty = (pairs > 1 ? 1500. : 2600.) * (double)((p->total + turns - 1) / turns);
        *rows_last = ty > tx;
        return tx > ty ? tx : ty;
    };
    // more SMs for the rows make them faster and the prefix slower: where the
    // two meet, or one SM fewer
    int lo = 1, hi = kSms - 1;
    bool rows_last;
    while (lo < hi) {
        const int mid = (lo + hi) / 2;
        split(mid, &rows_last);
        if (rows_last)
            lo = mid + 1;
        else
            hi = mid;
    }
    const double at = split(lo, &rows_last);
    if (lo > 1 && split(lo - 1, &rows_last) >= at) split(lo, &rows_last);
}

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

size_t rows_parts(const RowsPlan &p, int n_req) {
    return p.total > 0 ? ((size_t)p.ctas + n_req - 1) * p.subs : 0;
}

// Lays the part arrays out from byte `at` of the workspace (32-byte aligned,
// see aligned_work; null to count only); the byte behind them.
template <class Plan>
size_t place(Plan *p, size_t parts, uint8_t *work, size_t at, int heads_each) {
    const size_t rows = parts * heads_each;
    p->o = reinterpret_cast<float *>(work + at);
    at = align256(at + rows * kDim * 4);
    p->ml = reinterpret_cast<float2 *>(work + at);
    return align256(at + rows * sizeof(float2));
}

// Callers give 16-byte aligned workspaces; parts are written 32 bytes at a time.
uint8_t *aligned_work(void *work) {
    return reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(work) + 31) & ~(uintptr_t)31);
}
constexpr size_t kAlignSlack = 16;

size_t place_both(PrefixPlan *pp, RowsPlan *p, uint8_t *work, int n_req, int q_heads, int heads) {
    const size_t slots = pp->groups > 0 ? (size_t)pp->groups + heads - 1 : 0;
    const size_t at = place(pp, slots * n_req, work, 0, q_heads / heads);
    return place(p, rows_parts(*p, n_req), work, at, q_heads);
}

template <bool kScores>
cudaError_t launch_rows(const GroupArgs &a, const RowsPlan &p, cudaStream_t st) {
    const cudaError_t e = cudaFuncSetAttribute(rows_kernel<kScores>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               rows::kSmem);
    if (e != cudaSuccess) return e;
    const int slots = rows::slots(a.heads, p.subs);
    const int warps = a.heads * p.subs + rows::bringers(slots);
    const size_t ring = (size_t)slots * rows::kTile * rows::pitch(a.heads);
    rows_kernel<kScores><<<p.ctas, warps * 32, rows::kOffSlots + ring, st>>>(a, p);
    return cudaGetLastError();
}

cudaError_t launch_merge(const GroupArgs &a, const RowsPlan &p, const PrefixPlan &pp,
                         cudaStream_t st) {
    constexpr int kWarps = kMergeThreads / 32;
    // warps to an output: about a round of loads each, unless the outputs alone
    // fill the SMs (80 registers: 24 warps each)
    const int64_t parts = (pp.groups > 0 ? pp.groups / a.heads + 2 : 0) +
                          (p.total > 0 ? ((int64_t)p.ctas / a.n_req + 2) * p.subs : 0);
    int share = 1;
    while (share < kWarps && parts > 8 * share && (int64_t)a.n_req * a.q_heads * share < kSms * 12)
        share *= 2;
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

size_t prefix_attention_bytes(int n_req, int q_heads, int heads, int64_t prefix_len, int k,
                              PrefixPlan *pp, RowsPlan *p) {
    share_out(n_req, q_heads, heads, prefix_len, k, pp, p);
    const size_t n = place_both(pp, p, nullptr, n_req, q_heads, heads);
    return n ? n + kAlignSlack : 0;
}

size_t attention_weights_bytes(int n_req, int q_heads, int heads, int k) {
    PrefixPlan none = {};
    RowsPlan p = rows_plan(n_req, heads, k, kSms);
    return place_both(&none, &p, nullptr, n_req, q_heads, heads) +
           (size_t)n_req * q_heads * k * sizeof(float) + kAlignSlack;
}

cudaError_t launch_prefix_attention(const GroupArgs &a, PrefixPlan pp, RowsPlan p, void *work,
                                    cudaStream_t st) {
    place_both(&pp, &p, aligned_work(work), a.n_req, a.q_heads, a.heads);
    cudaError_t e = cudaSuccess;
    if (pp.groups > 0)
        e = launch_prefix(a, pp, p, st);
    else if (p.total > 0)
        e = launch_rows<false>(a, p, st);
    return e == cudaSuccess ? launch_merge(a, p, pp, st) : e;
}

cudaError_t launch_attention_weights(GroupArgs a, void *work, cudaStream_t st) {
    PrefixPlan none = {};
    RowsPlan p = rows_plan(a.n_req, a.heads, a.k, kSms);
    uint8_t *const w = aligned_work(work);
    a.scores = reinterpret_cast<float *>(w + place_both(&none, &p, w, a.n_req, a.q_heads, a.heads));
    const cudaError_t e = launch_rows<true>(a, p, st);
    return e == cudaSuccess ? launch_merge(a, p, none, st) : e;
}

// Reads the rows kernel's status bits on the current device and clears them.
cudaError_t rows_attention_status(uint32_t *status) {
    uint32_t v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_rows_status, sizeof(v));
    if (e != cudaSuccess) return e;
    *status = v;
    if (v) {
        const uint32_t zero = 0;
        e = cudaMemcpyToSymbol(g_rows_status, &zero, sizeof(zero));
    }
    return e;
}

}  // namespace hs
