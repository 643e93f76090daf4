// The positions a request keeps by accumulated attention weight
// (hs_select_heavy): the `recent` last ones and the heaviest of the others.
//
// A radix selection: a weight becomes a 32-bit key whose unsigned order is
// the weights' order; three passes of 11, 11 and 10 bits count the keys that
// share the prefix found so far and narrow down the key T of the last
// position kept, then the positions with keys above T, and the first of
// those equal to it, are written in ascending order.  The operator reads
// every weight once and has few operations: the floor is the read, what it
// spends is latency, one pass behind the other.
//
// A cluster of up to 16 CTAs takes a request, each a contiguous range of its
// positions, read from global memory once and kept in shared memory as keys
// (what does not fit is read again, from L2).  The counts of a pass are added
// into CTA 0's through distributed shared memory, where one scan finds the
// bin.  A weight of exactly 0 -- a position that was never selected -- is
// often the most frequent, so its count is taken by ballot, as is that of the
// first lane's bin: what is left for shared-memory atomics seldom collides.
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
constexpr int kKeysMax = 51200;       // keys a CTA keeps in shared memory
constexpr int kMinChunk = 2048;       // positions per CTA worth splitting for
constexpr int kUnroll = 8;            // loads in flight per thread

// Unsigned order of the keys = order of the weights; -0 counts as 0, NaN as
// -infinity.
__device__ __forceinline__ uint32_t order_key(float w) {
    if (w != w) w = -INFINITY;
    const uint32_t u = __float_as_uint(w + 0.f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
constexpr uint32_t kZeroKey = 0x80000000u;

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

__global__ void __launch_bounds__(kSelThreads)
    select_heavy_kernel(const SelectArgs a, int ctas) {
    extern __shared__ uint32_t keys[];
    __shared__ uint32_t hist[kBins];   // this CTA's counts
    __shared__ uint32_t sums[kBins];   // CTA 0: the cluster's
    __shared__ uint32_t warp_a[kSelWarps], warp_b[kSelWarps];
    __shared__ uint32_t found[2];      // CTA 0: the bin, and how many of it are wanted
    __shared__ uint32_t totals[2][kSelCluster];
    cg::cluster_group cluster = cg::this_cluster();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int i = blockIdx.x / ctas, rank = blockIdx.x % ctas;
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
    const int want = (int)(n < a.k - recent ? n : a.k - recent);
    // the ends that need no selection
    for (int j = rank * kSelThreads + tid; j < recent; j += ctas * kSelThreads)
        out[want + j] = (int32_t)(n + j);
    for (int j = want + recent + rank * kSelThreads + tid; j < a.k; j += ctas * kSelThreads)
        out[j] = -1;
    if (want == 0) return;

    const int64_t chunk = (n + ctas - 1) / ctas;
    const int64_t lo = min(n, rank * chunk);
    const int size = (int)(min(n, lo + chunk) - lo);  // this CTA's positions
    const int held = min(size, kKeysMax);
    const float *wc = w + lo;
    for (int b = tid; b < kBins; b += kSelThreads) hist[b] = sums[b] = 0;
    __syncthreads();
    cluster.barrier_arrive();               // CTA 0's sums are zero

    uint32_t prefix = 0, need = (uint32_t)want;
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
        const uint32_t mask = pass == 2 ? 1023u : 2047u;
        const int above = shift + (pass == 2 ? 10 : 11);
        if (pass == 0) {
            for (int j0 = 0; j0 < size; j0 += kUnroll * kSelThreads) {
                float x[kUnroll];
#pragma unroll
                for (int u = 0; u < kUnroll; ++u) {
                    const int j = j0 + u * kSelThreads + tid;
                    x[u] = j < size ? __ldg(wc + j) : 0.f;
                }
#pragma unroll
                for (int u = 0; u < kUnroll; ++u) {
                    const int j = j0 + u * kSelThreads + tid;
                    if (j0 + u * kSelThreads >= size) break;
                    const uint32_t key = order_key(x[u]);
                    if (j < held) keys[j] = key;
                    count(hist, key, shift, mask, j < size, lane);
                }
            }
        } else {
            for (int j0 = 0; j0 < size; j0 += kSelThreads) {
                const int j = j0 + tid;
                const uint32_t key = j < held ? keys[j] : j < size ? order_key(__ldg(wc + j)) : 0u;
                count(hist, key, shift, mask, j < size && key >> above == prefix, lane);
            }
        }
        __syncthreads();
        if (pass == 0) cluster.barrier_wait();
        uint32_t *lead = cluster.map_shared_rank(sums, 0);
        for (int b = tid; b < kBins; b += kSelThreads) {
            if (hist[b]) atomicAdd(&lead[b], hist[b]);
            hist[b] = 0;
        }
        cluster.sync();
        if (rank == 0) {
            // thread t has bins 2047 - 2t and 2046 - 2t; how many keys lie above
            const int b = kBins - 1 - 2 * tid;
            const uint32_t c0 = sums[b], c1 = sums[b - 1];
            sums[b] = sums[b - 1] = 0;
            uint32_t incl = c0 + c1;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, incl, d);
                if (lane >= d) incl += y;
            }
            if (lane == 31) warp_a[warp] = incl;
            __syncthreads();
            uint32_t before = incl - c0 - c1;
            for (int v = 0; v < warp; ++v) before += warp_a[v];
            if (before < need && need <= before + c0 + c1) {
                const bool second = need > before + c0;
                found[0] = (uint32_t)(second ? b - 1 : b);
                found[1] = need - before - (second ? c0 : 0u);
            }
        }
        cluster.sync();
        const uint32_t *f = cluster.map_shared_rank(found, 0);
        prefix = prefix << (pass == 2 ? 10 : 11) | f[0];
        need = f[1];
    }

    // keys above T are kept, and the first `need` positions of those equal to
    // it.  Each warp walks a contiguous part, twice: to count, and to write.
    const uint32_t T = prefix;
    const int part = (int)((chunk + kSelThreads - 1) / kSelThreads) * 32;
    const int p0 = min(size, warp * part), p1 = min(size, p0 + part);
    auto key_at = [&](int j) {
        return j < held ? keys[j] : order_key(__ldg(wc + j));
    };
    uint32_t n_gt = 0, n_eq = 0;
    for (int j = p0 + lane; j < p1; j += 32) {
        const uint32_t key = key_at(j);
        n_gt += key > T;
        n_eq += key == T;
    }
    n_gt = __reduce_add_sync(0xFFFFFFFFu, n_gt);
    n_eq = __reduce_add_sync(0xFFFFFFFFu, n_eq);
    if (lane == 0) {
        warp_a[warp] = n_gt;
        warp_b[warp] = n_eq;
    }
    __syncthreads();
    uint32_t gt0 = 0, eq0 = 0, gt_all = 0, eq_all = 0;
    {
        const uint32_t ga = warp_a[lane], eb = warp_b[lane];
        gt0 = __reduce_add_sync(0xFFFFFFFFu, lane < warp ? ga : 0u);
        eq0 = __reduce_add_sync(0xFFFFFFFFu, lane < warp ? eb : 0u);
        gt_all = __reduce_add_sync(0xFFFFFFFFu, ga);
        eq_all = __reduce_add_sync(0xFFFFFFFFu, eb);
    }
    if (tid < ctas) {
        cluster.map_shared_rank(totals[0], tid)[rank] = gt_all;
        cluster.map_shared_rank(totals[1], tid)[rank] = eq_all;
    }
    cluster.sync();  // also the last access to another CTA's shared memory
    for (int c = 0; c < rank; ++c) {
        gt0 += totals[0][c];
        eq0 += totals[1][c];
    }
    const uint32_t below = (1u << lane) - 1u;
    for (int j0 = p0; j0 < p1; j0 += 32) {
        const int j = j0 + lane;
        const uint32_t key = j < p1 ? key_at(j) : 0u;
        const uint32_t gt = __ballot_sync(0xFFFFFFFFu, j < p1 && key > T);
        const uint32_t eq = __ballot_sync(0xFFFFFFFFu, j < p1 && key == T);
        if (gt | eq) {
            const uint32_t e = eq0 + __popc(eq & below);
            if ((gt >> lane & 1u) || ((eq >> lane & 1u) && e < need))
                out[gt0 + __popc(gt & below) + min(e, need)] = (int32_t)(lo + j);
            gt0 += __popc(gt);
            eq0 += __popc(eq);
        }
    }
}

}  // namespace

// The cluster of a request: as many CTAs, a power of two up to 16, as keep
// the grid on the SMs at once and each at kMinChunk positions or more.
cudaError_t launch_select_heavy(const SelectArgs &a, int n_req, cudaStream_t st) {
    int ctas = 1;
    while (ctas < kSelCluster && (int64_t)n_req * 2 * ctas <= kSms &&
           a.n_positions >= (int64_t)2 * ctas * kMinChunk)
        ctas *= 2;
    const int64_t chunk = (a.n_positions + ctas - 1) / ctas;
    const size_t smem = (size_t)(chunk < kKeysMax ? chunk : kKeysMax) * 4;
    cudaError_t e = cudaFuncSetAttribute(select_heavy_kernel,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, kKeysMax * 4);
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
    return cudaLaunchKernelEx(&cfg, select_heavy_kernel, a, ctas);
}

}  // namespace hs
