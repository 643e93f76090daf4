// The positions a request keeps by accumulated attention weight
// (hs_select_heavy): the `recent` last ones and the heaviest of the others.
//
// A radix selection: a weight becomes a 32-bit key whose unsigned order is
// the weights' order; four passes of 8 bits narrow down the key of the last
// position kept, then one pass writes the kept positions in ascending order.
#include <cstdint>

#include "hs.h"
#include "hs_internal.cuh"

namespace hs {
namespace {

constexpr int kSelThreads = 1024;

// Unsigned order of the keys = order of the weights; -0 counts as 0, NaN as
// -infinity.
__device__ __forceinline__ uint32_t order_key(float w) {
    if (w != w) w = -INFINITY;
    const uint32_t u = __float_as_uint(w + 0.f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__global__ void __launch_bounds__(kSelThreads) select_heavy_kernel(const SelectArgs a) {
    __shared__ uint32_t hist[256];
    __shared__ uint32_t warp_gt[32], warp_eq[32];
    __shared__ uint32_t s_prefix, s_need;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int i = blockIdx.x;
    int32_t *out = a.sel + (int64_t)i * a.k;
    const int32_t req = a.req_ids ? a.req_ids[i] : i;
    if (req < 0 || req >= a.weight_rows) {
        for (int j = tid; j < a.k; j += kSelThreads) out[j] = -1;
        return;
    }
    const float *w = a.weights + (int64_t)req * a.n_positions;
    int64_t len = a.len ? a.len[i] : a.n_positions;
    len = len < 0 ? 0 : len > a.n_positions ? a.n_positions : len;
    const int recent = (int)(len < a.recent ? len : a.recent);
    const int64_t n = len - recent;                       // positions that compete
    const int want = (int)(n < a.k - recent ? n : a.k - recent);
    if (tid == 0) {
        s_prefix = 0;
        s_need = want;
    }
    for (int shift = 24; shift >= 0; shift -= 8) {
        for (int b = tid; b < 256; b += kSelThreads) hist[b] = 0;
        __syncthreads();
        const uint32_t prefix = s_prefix;
        for (int64_t j = tid; j < n; j += kSelThreads) {
            const uint32_t key = order_key(w[j]);
            if (shift == 24 || (key >> (shift + 8)) == prefix) atomicAdd(&hist[(key >> shift) & 255], 1u);
        }
        __syncthreads();
        if (tid == 0) {
            uint32_t need = s_need;
            int b = 255;
            while (b > 0 && hist[b] < need) need -= hist[b--];
            s_prefix = prefix << 8 | (uint32_t)b;
            s_need = need;
        }
        __syncthreads();
    }
    // keys above T are kept, and the first `need` positions of those equal to it
    const uint32_t T = s_prefix, need = s_need;
    uint32_t done_gt = 0, done_eq = 0;
    for (int64_t j0 = 0; j0 < n; j0 += kSelThreads) {
        const int64_t j = j0 + tid;
        const uint32_t key = j < n ? order_key(w[j]) : 0u;
        const uint32_t gt = __ballot_sync(0xFFFFFFFFu, j < n && key > T);
        const uint32_t eq = __ballot_sync(0xFFFFFFFFu, j < n && key == T);
        if (lane == 0) {
            warp_gt[warp] = __popc(gt);
            warp_eq[warp] = __popc(eq);
        }
        __syncthreads();
        uint32_t gt0 = done_gt, eq0 = done_eq;
        for (int v = 0; v < 32; ++v) {
            if (v < warp) {
                gt0 += warp_gt[v];
                eq0 += warp_eq[v];
            }
            done_gt += warp_gt[v];
            done_eq += warp_eq[v];
        }
        const uint32_t below = (1u << lane) - 1u;
        gt0 += __popc(gt & below);
        eq0 += __popc(eq & below);
        const bool is_gt = gt >> lane & 1u, is_eq = (eq >> lane & 1u) && eq0 < need;
        if (want > 0 && (is_gt || is_eq)) out[gt0 + (eq0 < need ? eq0 : need)] = (int32_t)j;
        __syncthreads();
    }
    for (int j = tid; j < recent; j += kSelThreads) out[want + j] = (int32_t)(n + j);
    for (int j = want + recent + tid; j < a.k; j += kSelThreads) out[j] = -1;
}

}  // namespace

cudaError_t launch_select_heavy(const SelectArgs &a, int n_req, cudaStream_t st) {
    select_heavy_kernel<<<n_req, kSelThreads, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace hs
