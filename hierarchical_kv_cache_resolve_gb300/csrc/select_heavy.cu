// The positions a request keeps by accumulated attention weight
// (hs_select_heavy): the `recent` last ones and the heaviest of the others.
//
// The operator reads every weight once and computes little: the floor is the
// read, and what it spends beyond is latency, one step behind the other.
//
// A cluster of up to 16 CTAs takes a request, each a contiguous range of its
// positions, read once and kept in shared memory (what does not fit is read
// again, from L2).  A weight's key is a 32-bit number whose unsigned order is
// the weights' order.  T, the key of the last position kept, is found in three
// steps:
//   a bound B <= T: the maxima of groups of weights, one to four groups to a
//     thread; at least as many groups as positions are wanted have a maximum
//     at or above B, the lower edge of a bin of the maxima's leading 11 bits;
//   the candidates: all keys above B, a little more than are wanted, listed
//     with their positions.  If they are fewer, T = B (many equal weights:
//     zeros, above all);
//   T among the candidates, whose keys every CTA writes into all others' shared
//     memory: counts in 2048 bins over their own range, and again within the bin
//     found until it holds no more keys than a warp can rank.
// So all weights are only compared with B, once, and those of a warp's 128
// neighbours not even that where their maximum is no larger (three in four
// with 2048 of a million wanted); and the CTAs wait for one
// another twice, once for the maxima's counts and once for the lists.  With
// more candidates than the lists hold -- a large k, weights that lie within one
// bin, heavy positions side by side in the range of one CTA -- every CTA counts
// all its keys instead, by 11, 11 and 10 bits.
// Measured, 2048 of independent heavy-tailed weights kept: 11.3 us for 32
// requests of 32768 positions (clusters of 4; about ten steps of 0.5 to 1.3 us),
// 22.8 to 24.3 us for 8 of 2^20 (clusters of 12, 33.5 MB read in 7 us).  Listed
// candidates copied by the CTAs from one another, not written by their finders,
// which leaves memory to be kept until the others are done: 12.0 us; every weight
// compared: 26.4.  With all keys counted, for the 8: 126 us (the first 1000 and
// the last 65536 positions heaviest), 131 (30000 kept), 136 (weights within 10^-4
// of one another), 138 (falling steadily); the last three 31, 26.5 and 25.3 for
// the 32.
// The kept positions -- keys above T, and the first of those equal to it --
// are marked in two bitmaps over the CTA's range, whose prefix sums give each
// its place in ascending order.
#include <cmath>
#include <cstdint>

#include <cooperative_groups.h>

#include "hs.h"
#include "hs_internal.cuh"

namespace hs {
namespace {

namespace cg = cooperative_groups;

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;
constexpr int kSelCluster = 16;
constexpr int kListMax = 8192;        // candidates of a CTA
constexpr int kAllMax = 2 * kListMax; // of the whole cluster, in equal shares
constexpr int kMinChunk = 2048;       // positions per CTA worth splitting for
constexpr int kDynMax = (232448 - 17408) / 4;  // words of shared memory beside the static arrays
constexpr int kWindow = kBins * 32;   // positions the bitmaps hold
constexpr int kWords = 4;             // of a bitmap, to a thread, where memory is left over
static_assert(32 * 32 * kWords < 1 << 16, "two counts in a word");
static_assert(kDynMax > kAllMax + kListMax + kMinChunk, "room for weights");

// Unsigned order of the keys = order of the weights; -0 counts as 0, NaN as
// -infinity.
__device__ __forceinline__ uint32_t order_key(float w) {
    if (w != w) w = -INFINITY;
    const uint32_t u = __float_as_uint(w + 0.f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
constexpr uint32_t kZeroKey = 0x80000000u;

// The largest of a warp's values; NaN counts as nothing.
__device__ __forceinline__ float warp_max(float x) {
    float y;
    asm("redux.sync.max.f32 %0, %1, 0xFFFFFFFF;" : "=f"(y) : "f"(x));
    return y;
}

// Counts this warp's keys by `bin` where `active`.
__device__ __forceinline__ void count(uint32_t *hist, uint32_t key, int shift, uint32_t mask,
                                      bool active, int lane) {
    const uint32_t bin = key >> shift & mask;
    const uint32_t zero = __ballot_sync(0xFFFFFFFFu, active && key == kZeroKey);
    const uint32_t rest = __ballot_sync(0xFFFFFFFFu, active && key != kZeroKey);
    if (zero && lane == 0) atomicAdd(&hist[kZeroKey >> shift & mask], (uint32_t)__popc(zero));
    if (rest) {
        const int first = __ffs(rest) - 1;
        const uint32_t b0 = __shfl_sync(0xFFFFFFFFu, bin, first);
        const bool mine = rest >> lane & 1u;
        const uint32_t same = __ballot_sync(0xFFFFFFFFu, mine && bin == b0);
        if (lane == first) atomicAdd(&hist[b0], (uint32_t)__popc(same));
        if (mine && bin != b0) atomicAdd(&hist[bin], 1u);
    }
}

// The bin, counted from the top, in which the need-th key lies: found[0] the
// bin, found[1] how many of it are wanted, found[2] how many it holds;
// unchanged if there are fewer keys.  One CTA, all threads; empties the counts.
__device__ __forceinline__ void find_bin(uint32_t *counts, uint32_t need, uint32_t *warp_sum,
                                         volatile uint32_t *found) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // thread t has bins 2047 - 2t and 2046 - 2t
    const int b = kBins - 1 - 2 * tid;
    const uint32_t c0 = counts[b], c1 = counts[b - 1];
    counts[b] = counts[b - 1] = 0;
    uint32_t incl = c0 + c1;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, incl, d);
        if (lane >= d) incl += y;
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    uint32_t before = incl - c0 - c1;
    before += __reduce_add_sync(0xFFFFFFFFu, lane < warp ? warp_sum[lane] : 0u);
    if (before < need && need <= before + c0 + c1) {
        const bool second = need > before + c0;
        found[0] = (uint32_t)(second ? b - 1 : b);
        found[1] = need - before - (second ? c0 : 0u);
        found[2] = second ? c1 : c0;
    }
}

__global__ void __launch_bounds__(kSelThreads)
    select_heavy_kernel(const SelectArgs a, int ctas, int held_max, int list_max) {
    // the weights held [held_max]; the candidates' keys of every CTA, and the
    // positions of this one's [list_max each]
    extern __shared__ __align__(16) uint32_t dyn[];
    float *vals = reinterpret_cast<float *>(dyn);
    uint32_t *all = dyn + held_max;
    int32_t *list_pos = reinterpret_cast<int32_t *>(all + ctas * list_max);
    // this CTA's counts and the cluster's, zero between uses; in the end the
    // bitmaps of the keys above T and equal to it
    __shared__ uint32_t hist[kBins], sums[kBins];
    __shared__ uint32_t warp_a[kSelWarps], warp_b[kSelWarps], few[32], ahead_b[kSelWarps];
    __shared__ uint32_t found[3], n_few, n_list, my_top;
    __shared__ uint32_t totals[2][kSelCluster], list_counts[kSelCluster], tops[kSelCluster];
    cg::cluster_group cluster = cg::this_cluster();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int i = blockIdx.x / ctas, rank = blockIdx.x % ctas;
    uint32_t *list = all + rank * list_max;
    int32_t *out = a.sel + (int64_t)i * a.k;
    const int32_t req = a.req_ids ? a.req_ids[i] : i;
    if (req < 0 || req >= a.weight_rows) {  // the whole cluster alike
        for (int j = rank * kSelThreads + tid; j < a.k; j += ctas * kSelThreads) out[j] = -1;
        return;
    }
    const float *w = a.weights + (int64_t)req * a.n_positions;
    int64_t len = a.len ? a.len[i] : a.n_positions;
    len = len < 0 ? 0 : len > a.n_positions ? a.n_positions : len;
    const int recent = (int)(len < a.recent ? len : a.recent);
    const int64_t n = len - recent;         // positions that compete
    const uint32_t want = (uint32_t)(n < a.k - recent ? n : a.k - recent);
    // the ends that need no selection
    for (int j = rank * kSelThreads + tid; j < recent; j += ctas * kSelThreads)
        out[want + j] = (int32_t)(n + j);
    for (int j = want + recent + rank * kSelThreads + tid; j < a.k; j += ctas * kSelThreads)
        out[j] = -1;
    if (want == 0) return;

    const int64_t chunk = (n + ctas - 1) / ctas;
    const int64_t lo = min(n, rank * chunk);
    const int size = (int)(min(n, lo + chunk) - lo);  // this CTA's positions
    const float *wc = w + lo;
    // vector v holds positions 4 v - off .. 4 v - off + 3 of the range, so that
    // whole vectors are aligned in global memory; -infinity outside the range
    const int off = (int)(reinterpret_cast<uintptr_t>(wc) >> 2 & 3);
    const int nv = (off + size + 3) / 4;
    const int held = min(nv, held_max / 4);
    // Vectors v, v + 1024, ..., kEach of them: those below `from` out of shared
    // memory, the others with their global loads issued together; with bit u of
    // `rows` clear, x[u] is left.
    constexpr int kEach = 4;
    auto at = [&](int v, int from, float4 *x, uint32_t rows = 0xFu) {
#pragma unroll
        for (int u = 0; u < kEach; ++u) {
            const int t = v + u * kSelThreads, j = 4 * t - off;
            if (!(rows >> u & 1u)) {
            } else if (t < from) {
                x[u] = reinterpret_cast<const float4 *>(vals)[t];
            } else if (j >= 0 && j + 3 < size) {
                x[u] = __ldg(reinterpret_cast<const float4 *>(wc + j));
            } else {
                x[u] = make_float4(j >= 0 && j < size ? __ldg(wc + j) : -INFINITY,
                                   j + 1 >= 0 && j + 1 < size ? __ldg(wc + j + 1) : -INFINITY,
                                   j + 2 >= 0 && j + 2 < size ? __ldg(wc + j + 2) : -INFINITY,
                                   j + 3 >= 0 && j + 3 < size ? __ldg(wc + j + 3) : -INFINITY);
            }
        }
    };
    // Calls f(key, position, whether it is one) for positions [from, to), kEach
    // single weights' loads at a time: for what seldom runs, in little code.
    auto each = [&](int from, int to, auto f) {
#pragma unroll 1
        for (int j0 = from; j0 < to; j0 += kEach * kSelThreads) {
            float x[kEach];
#pragma unroll
            for (int u = 0; u < kEach; ++u) {
                const int j = j0 + u * kSelThreads + tid;
                x[u] = j >= to ? -INFINITY : j + off < 4 * held ? vals[j + off] : __ldg(wc + j);
            }
#pragma unroll
            for (int u = 0; u < kEach; ++u) {
                const int j = j0 + u * kSelThreads + tid;
                f(order_key(x[u]), j, j < to);
            }
        }
    };

    // ---- read; the maxima's leading bits ------------------------------------
    for (int b = tid; b < kBins; b += kSelThreads) hist[b] = sums[b] = 0;
    if (tid == 0) found[0] = my_top = n_list = 0;
    float4 top = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
    float row_top = -INFINITY;   // of the warp's rows of 32 vectors lane, lane + 32, ...
#pragma unroll 1
    for (int v0 = 0; v0 < nv; v0 += kEach * kSelThreads) {
        float4 x[kEach];
        at(v0 + tid, 0, x);
#pragma unroll
        for (int u = 0; u < kEach; ++u) {
            const int v = v0 + u * kSelThreads + tid;
            if (v < held) reinterpret_cast<float4 *>(vals)[v] = x[u];
            top.x = fmaxf(top.x, x[u].x);   // of a number and NaN, the number
            top.y = fmaxf(top.y, x[u].y);
            top.z = fmaxf(top.z, x[u].z);
            top.w = fmaxf(top.w, x[u].w);
            const float row = warp_max(fmaxf(fmaxf(x[u].x, x[u].y), fmaxf(x[u].z, x[u].w)));
            if (lane == (v0 / kSelThreads + u) % 32) row_top = fmaxf(row_top, row);
        }
    }
    __syncthreads();
    cluster.barrier_arrive();               // this CTA's sums are zero
    const float warp_top = warp_max(row_top);
    if (lane == 0) atomicMax(&my_top, order_key(warp_top));
    // as few groups as are half as many again as the positions wanted
    const uint32_t groups = (uint32_t)ctas * kSelThreads;
    if (2 * groups >= 3 * want) {
        count(hist, order_key(fmaxf(fmaxf(top.x, top.y), fmaxf(top.z, top.w))), 21, 2047u, true,
              lane);
    } else if (4 * groups >= 3 * want) {
        count(hist, order_key(fmaxf(top.x, top.y)), 21, 2047u, true, lane);
        count(hist, order_key(fmaxf(top.z, top.w)), 21, 2047u, true, lane);
    } else {
        count(hist, order_key(top.x), 21, 2047u, true, lane);
        count(hist, order_key(top.y), 21, 2047u, true, lane);
        count(hist, order_key(top.z), 21, 2047u, true, lane);
        count(hist, order_key(top.w), 21, 2047u, true, lane);
    }
    __syncthreads();
    cluster.barrier_wait();
    // adds this CTA's counts to every CTA's sums
    auto add_counts = [&]() {
#pragma unroll 1
        for (int b = tid; b < kBins; b += kSelThreads) {
            const uint32_t c = hist[b];
            if (c)
#pragma unroll 4
                for (int t = 0; t < ctas; ++t) atomicAdd(cluster.map_shared_rank(sums, t) + b, c);
            hist[b] = 0;
        }
    };
    add_counts();
    cluster.sync();
    find_bin(sums, want, warp_a, found);
    __syncthreads();
    const uint32_t B = found[0] << 21;

    // ---- the candidates: keys above B ----------------------------------------
    // (with B in or below -infinity's bin, all; else compared as numbers)
    const bool every = B < 0x00800000u;
    const float fb = __uint_as_float(B & 0x80000000u ? B ^ 0x80000000u : ~B);
    // the warp's rows that have any
    const uint32_t rows = __ballot_sync(0xFFFFFFFFu, every || row_top > fb);
#pragma unroll 1
    for (int v0 = 0; v0 < nv; v0 += kEach * kSelThreads) {
        const uint32_t here = rows >> v0 / kSelThreads % 32;  // kEach divides 32
        if (!(here & ((1u << kEach) - 1u))) continue;
        float4 x[kEach];
        at(v0 + tid, held, x, here);
#pragma unroll
        for (int u = 0; u < kEach; ++u) {
            if (!(here >> u & 1u)) continue;
            const int j = 4 * (v0 + u * kSelThreads + tid) - off;
            const float y[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
            uint32_t hit[4], hits = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                hit[e] = every ? j + e >= 0 && j + e < size : y[e] > fb;
                hits += hit[e];
            }
            if (!__any_sync(0xFFFFFFFFu, hits)) continue;
            uint32_t to = hits;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const uint32_t z = __shfl_up_sync(0xFFFFFFFFu, to, d);
                if (lane >= d) to += z;
            }
            uint32_t base = 0;
            if (lane == 31) base = atomicAdd(&n_list, to);
            to += __shfl_sync(0xFFFFFFFFu, base, 31) - hits;
            // (past the list's end its last place is written over: its contents
            // do not count then)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (hit[e]) {
                    const uint32_t place = min(to++, (uint32_t)list_max - 1);
                    list[place] = order_key(y[e]);
                    list_pos[place] = j + e;
                }
        }
    }
    __syncthreads();
    // warps share the CTAs out: where to write, later whose keys to look at
    const int per = kSelWarps / ctas, other = warp / per, first = (warp - other * per) * 32;
    if (other < ctas && other != rank && n_list <= (uint32_t)list_max) {
        uint32_t *dst = cluster.map_shared_rank(list, other);
#pragma unroll 1
        for (int j = first + lane; j < (int)n_list; j += per * 32) dst[j] = list[j];
    }
    if (tid < ctas) {
        cluster.map_shared_rank(list_counts, tid)[rank] = n_list;
        cluster.map_shared_rank(tops, tid)[rank] = my_top;
    }
    cluster.sync();
    uint64_t candidates = 0;
    uint32_t highest = 0;
    bool listed = true;                     // the lists hold all candidates
#pragma unroll 4
    for (int c = 0; c < ctas; ++c) {
        candidates += list_counts[c];
        highest = max(highest, tops[c]);
        listed &= list_counts[c] <= (uint32_t)list_max;
    }
    const bool from_list = candidates >= want && listed;
    // a longer range's bitmaps where the weights were, in one window
    const bool roomy = from_list && size > kWindow && held_max >= 2 * kWords * kSelThreads;

    uint32_t T = B, need = want - (uint32_t)candidates;
    uint32_t gt0 = 0, eq0 = 0;              // kept and equal ones before this CTA's
    if (from_list) {
        if (roomy)
            for (int b = tid; b < 2 * kWords * kSelThreads; b += kSelThreads) dyn[b] = 0;
        const int total = other < ctas ? (int)list_counts[other] : 0;
        const uint32_t *keys = all + min(other, ctas - 1) * list_max;
        // the need-th largest lies in the first `bins` bins of 1 << shift keys from base
        uint32_t base = B, bins = kBins;
        need = want;
        int shift = max(0, 32 - __clz(highest - B) - 11);
        while (true) {
#pragma unroll 1
            for (int j0 = first; j0 < total; j0 += per * 32) {
                const uint32_t x = j0 + lane < total ? keys[j0 + lane] : 0u;
                const uint32_t bin = (x - base) >> shift;
                const bool in = j0 + lane < total && x >= base && bin < bins;
                const uint32_t some = __ballot_sync(0xFFFFFFFFu, in);
                if (!some) continue;
                // many equal keys: the first lane's bin in one addition
                const int f = __ffs(some) - 1;
                const uint32_t b0 = __shfl_sync(0xFFFFFFFFu, bin, f);
                const uint32_t same = __ballot_sync(0xFFFFFFFFu, in && bin == b0);
                if (lane == f) atomicAdd(&hist[b0], (uint32_t)__popc(same));
                if (in && bin != b0) atomicAdd(&hist[bin], 1u);
            }
            if (tid == 0) n_few = 0;
            __syncthreads();
            find_bin(hist, need, warp_a, found);
            __syncthreads();
            base += found[0] << shift;
            need = found[1];
            if (shift == 0 || found[2] <= 32) break;
            // on within the bin found only: `need` no longer counts the keys above it
            bins = 1u << min(shift, 11);
            shift = max(0, shift - 11);
            __syncthreads();                // every thread has read what was found
        }
        if (shift > 0) {
            // at most 32 keys in the bin, each ranked by a warp
#pragma unroll 1
            for (int j = first + lane; j < total; j += per * 32) {
                const uint32_t x = keys[j];
                if (x >= base && (x - base) >> shift == 0) few[atomicAdd(&n_few, 1u)] = x;
            }
            __syncthreads();
            if (warp < (int)n_few) {
                const uint32_t key = lane < (int)n_few ? few[lane] : 0u, mine = few[warp];
                const uint32_t above = __popc(__ballot_sync(0xFFFFFFFFu, key > mine));
                const uint32_t ahead =
                    __popc(__ballot_sync(0xFFFFFFFFu, key == mine) & ((1u << warp) - 1u));
                if (lane == 0 && above + ahead + 1 == need) {  // one warp
                    found[0] = mine;
                    found[1] = need - above;
                }
            }
            __syncthreads();
            T = found[0];
            need = found[1];
        } else {
            T = base;
        }
        if (other < rank)
#pragma unroll 1
            for (int j = first + lane; j < total; j += per * 32) {
                gt0 += keys[j] > T;
                eq0 += keys[j] == T;
            }
    } else {
        if (candidates >= want) {
            uint32_t prefix = 0;
            need = want;
#pragma unroll 1
            for (int pass = 0; pass < 3; ++pass) {
                const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
                const int bits = pass == 2 ? 10 : 11;
                each(0, size, [&](uint32_t key, int, bool is) {
                    count(hist, key, shift, (1u << bits) - 1u,
                          is && (pass == 0 || key >> (shift + bits) == prefix), lane);
                });
                __syncthreads();
                add_counts();
                cluster.sync();
                find_bin(sums, need, warp_a, found);
                cluster.sync();             // every CTA's sums are zero again
                prefix = prefix << bits | found[0];
                need = found[1];
            }
            T = prefix;
        }
        // kept and equal ones of every CTA
        uint32_t n_gt = 0, n_eq = 0;
        each(0, size, [&](uint32_t key, int, bool is) {
            n_gt += is && key > T;
            n_eq += is && key == T;
        });
        if (tid < 2) totals[tid][rank] = 0;
        __syncthreads();
        n_gt = __reduce_add_sync(0xFFFFFFFFu, n_gt);
        n_eq = __reduce_add_sync(0xFFFFFFFFu, n_eq);
        if (lane == 0) {
            atomicAdd(&totals[0][rank], n_gt);
            atomicAdd(&totals[1][rank], n_eq);
        }
        __syncthreads();
        if (tid < ctas && tid != rank) {
            cluster.map_shared_rank(totals[0], tid)[rank] = totals[0][rank];
            cluster.map_shared_rank(totals[1], tid)[rank] = totals[1][rank];
        }
        cluster.sync();
        cluster.barrier_arrive();           // no other CTA's memory is needed
        if (tid < rank) {
            gt0 = totals[0][tid];
            eq0 = totals[1][tid];
        }
    }
    // (the sums over the threads are taken with the first window's)

    // ---- marked and written in order -----------------------------------------
    uint32_t *gt_bits = roomy ? dyn : hist;
    uint32_t *eq_bits = roomy ? gt_bits + kWords * kSelThreads : sums;
    const int window = roomy ? kWords * kSelThreads * 32 : kWindow;
    const int n_mine = from_list ? (int)list_counts[rank] : 0;
    for (int w0 = 0; w0 < size || w0 == 0; w0 += window) {
        const int w1 = min(size - w0, window);  // positions w0 + [0, w1)
        auto mark = [&](uint32_t key, int j) {
            if (key < T || j < 0 || j >= w1) return;
            atomicOr((key > T ? gt_bits : eq_bits) + (j >> 5), 1u << (j & 31));
        };
        if (from_list) {
#pragma unroll 1
            for (int j = tid; j < n_mine; j += kSelThreads)
                mark(list[j], list_pos[j] - w0);
        } else {
            each(w0, w0 + w1, [&](uint32_t key, int j, bool is) {
                if (is) mark(key, j - w0);
            });
        }
        const uint32_t g0 = __reduce_add_sync(0xFFFFFFFFu, gt0);
        const uint32_t q0 = __reduce_add_sync(0xFFFFFFFFu, eq0);
        __syncthreads();
        // a thread writes a few consecutive words
        const int words = (w1 + 31) / 32;
        const int each_words = words <= kSelThreads / 4 ? 1 : words <= kSelThreads / 2 ? 2 : kWords;
        const bool busy = warp * 32 * each_words < words, last = w0 + window >= size;
        uint32_t g[kWords] = {}, q[kWords] = {};
        uint32_t ng = 0, nq = 0, incl = 0;  // this thread's; up to it (equal ones << 16)
        if (busy) {
#pragma unroll
            for (int e = 0; e < kWords; ++e) {
                const int b = each_words * tid + e;
                if (e < each_words && b < words) {
                    g[e] = gt_bits[b];
                    q[e] = eq_bits[b];
                    if (!last) gt_bits[b] = eq_bits[b] = 0;
                }
                ng += __popc(g[e]);
                nq += __popc(q[e]);
            }
            incl = ng | nq << 16;           // a warp has at most 32 * 32 * kWords
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, incl, d);
                if (lane >= d) incl += y;
            }
        }
        // a warp's words, and what its threads had before the window
        if (lane == 31) {
            warp_a[warp] = incl & 0xFFFFu;
            warp_b[warp] = incl >> 16;
        }
        if (lane == 0) {
            few[warp] = g0;
            ahead_b[warp] = q0;
        }
        __syncthreads();
        if (busy || !last) {
            const uint32_t wg = warp_a[lane], wq = warp_b[lane];
            gt0 = __reduce_add_sync(0xFFFFFFFFu, few[lane]);
            eq0 = __reduce_add_sync(0xFFFFFFFFu, ahead_b[lane]);
            uint32_t pg = gt0 + (incl & 0xFFFFu) - ng +
                          __reduce_add_sync(0xFFFFFFFFu, lane < warp ? wg : 0u);
            uint32_t pq = eq0 + (incl >> 16) - nq +
                          __reduce_add_sync(0xFFFFFFFFu, lane < warp ? wq : 0u);
#pragma unroll
            for (int e = 0; e < kWords; ++e) {
                uint32_t any = g[e] | q[e];
                while (any) {
                    const int b = __ffs(any) - 1;
                    any &= any - 1;
                    const bool above = g[e] >> b & 1u;
                    if (above || pq < need)
                        out[pg + min(pq, need)] =
                            (int32_t)(lo + w0 + (each_words * tid + e) * 32 + b);
                    pg += above;
                    pq += !above;
                }
            }
            // carried on by one thread
            const uint32_t next_g = gt0 + __reduce_add_sync(0xFFFFFFFFu, wg);
            const uint32_t next_q = eq0 + __reduce_add_sync(0xFFFFFFFFu, wq);
            gt0 = tid == 0 ? next_g : 0u;
            eq0 = tid == 0 ? next_q : 0u;
        }
        if (!last) __syncthreads();         // the window's words and sums are read
    }
    if (!from_list) cluster.barrier_wait();
}

}  // namespace

// The cluster of a request: as many CTAs as have kMinChunk positions or more
// each and as keep every request's cluster on the GPU at once with a CTA to an
// SM -- a cluster lies within one GPC, whose SMs its size has to divide well
// (cudaOccupancyMaxActiveClusters on GB300: 7 clusters of 16, 8 of 12, 15 of
// 8, 36 of 4, 76 of 2; eight requests of 2^20 positions as clusters of 16 ran
// in two waves, 47 us against 20 for one).
cudaError_t launch_select_heavy(const SelectArgs &a, int n_req, cudaStream_t st) {
    static const struct {
        int ctas, clusters;
    } sizes[] = {{16, 7}, {12, 8}, {8, 15}, {4, 36}, {2, 76}};
    int ctas = 1;
    for (const auto &s : sizes)
        if (n_req <= s.clusters && a.n_positions >= (int64_t)s.ctas * kMinChunk) {
            ctas = s.ctas;
            break;
        }
    // a range's positions fit 31 bits with room for a step of the loops
    while (a.n_positions > (int64_t)ctas << 30) ctas *= 2;
    // a range's weights start at any of the four words of a vector
    const int list_max = kAllMax / ctas < kListMax ? kAllMax / ctas : kListMax;
    const int most = (kDynMax - (ctas + 1) * list_max) / 4 * 4;
    const int64_t chunk = (a.n_positions + ctas - 1) / ctas + 3;
    const int held_max = (int)(chunk < most ? (chunk + 3) / 4 * 4 : most);
    const size_t smem = ((size_t)held_max + (ctas + 1) * list_max) * 4;
    cudaError_t e = cudaFuncSetAttribute(select_heavy_kernel,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         kDynMax * 4);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(select_heavy_kernel,
                                 cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)n_req * ctas);
    cfg.blockDim = dim3(kSelThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ctas;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, select_heavy_kernel, a, ctas, held_max, list_max);
}

}  // namespace hs
