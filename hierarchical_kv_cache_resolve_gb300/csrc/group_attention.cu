// Attention of grouped query heads over per-head token records: over a prefix
// that all requests share and over each request's published rows
// (hs_prefix_attention), or over the published rows alone with every row's
// weight added to its position's running sum (hs_sparse_attention_weights).
//
// One warp per (request, query head), four dimensions per lane, online
// softmax (base 2).  The weights need the final maximum and sum, so the
// scores go to the workspace and a second kernel turns them into weights.
#include <cmath>
#include <cstdint>

#include "hs.h"
#include "hs_internal.cuh"

namespace hs {
namespace {

constexpr int kDim = 128;

__device__ __forceinline__ void load4(const uint8_t *p, float *f) {
    const uint2 x = *reinterpret_cast<const uint2 *>(p);
    f[0] = __uint_as_float(x.x << 16);
    f[1] = __uint_as_float(x.x & 0xFFFF0000u);
    f[2] = __uint_as_float(x.y << 16);
    f[3] = __uint_as_float(x.y & 0xFFFF0000u);
}

__global__ void __launch_bounds__(128) group_attention_kernel(const GroupArgs a) {
    const int lane = threadIdx.x & 31;
    const int64_t unit = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    if (unit >= (int64_t)a.n_req * a.q_heads) return;
    const int r = (int)(unit / a.q_heads), hq = (int)(unit % a.q_heads);
    const int h = hq / (a.q_heads / a.heads);
    const int64_t W = (int64_t)a.heads * 4 * kDim;
    float q[4], o[4] = {0.f, 0.f, 0.f, 0.f};
    load4(a.q + unit * kDim * 2 + lane * 8, q);
    float m = -INFINITY, l = 0.f;
    for (int64_t j = 0; j < a.prefix_len + a.k; ++j) {
        const uint8_t *rec;
        bool use = true;
        if (j < a.prefix_len) {
            rec = a.prefix + j * W;
        } else {
            const int32_t row = a.idx[(int64_t)r * a.k + (j - a.prefix_len)];
            use = row >= 0 && row < a.cache_rows;
            rec = a.cache + (use ? row : 0) * W;
        }
        float kf[4], vf[4];
        load4(rec + h * 2 * kDim + lane * 8, kf);
        load4(rec + (a.heads + h) * 2 * kDim + lane * 8, vf);
        float s = q[0] * kf[0] + q[1] * kf[1] + q[2] * kf[2] + q[3] * kf[3];
#pragma unroll
        for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
        s = use ? s * a.scale_log2 : -INFINITY;
        if (a.weights && lane == 0) a.scores[unit * a.k + j] = s;
        if (s == -INFINITY) continue;
        const float mx = fmaxf(m, s), c = exp2f(m - mx), p = exp2f(s - mx);
        l = l * c + p;
#pragma unroll
        for (int d = 0; d < 4; ++d) o[d] = o[d] * c + p * vf[d];
        m = mx;
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
    uint2 v;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(v.x) : "f"(o[1] * inv), "f"(o[0] * inv));
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(v.y) : "f"(o[3] * inv), "f"(o[2] * inv));
    *reinterpret_cast<uint2 *>(a.out + unit * kDim * 2 + lane * 8) = v;
    if (a.weights && lane == 0) a.ml[unit] = make_float2(m, inv);
}

__global__ void __launch_bounds__(256) add_weights_kernel(const GroupArgs a) {
    const int r = blockIdx.y;
    const int j = blockIdx.x * 256 + threadIdx.x;
    if (j >= a.k) return;
    const int32_t req = a.req_ids ? a.req_ids[r] : r;
    const int32_t pos = a.sel[(int64_t)r * a.k + j];
    if (req < 0 || req >= a.weight_rows || pos < 0 || pos >= a.n_positions) return;
    float w = 0.f;
    for (int hq = 0; hq < a.q_heads; ++hq) {
        const float2 ml = a.ml[(int64_t)r * a.q_heads + hq];
        const float s = a.scores[((int64_t)r * a.q_heads + hq) * a.k + j];
        if (s != -INFINITY) w += exp2f(s - ml.x) * ml.y;
    }
    if (w != 0.f) atomicAdd(a.weights + (int64_t)req * a.n_positions + pos, w);
}

}  // namespace

size_t prefix_attention_bytes(int, int, int, int64_t, int) { return 0; }

size_t attention_weights_bytes(int n_req, int q_heads, int, int k) {
    return (size_t)n_req * q_heads * (sizeof(float2) + sizeof(float) * (size_t)k);
}

cudaError_t launch_prefix_attention(GroupArgs a, void *, cudaStream_t st) {
    const int64_t units = (int64_t)a.n_req * a.q_heads;
    group_attention_kernel<<<(unsigned)((units + 3) / 4), 128, 0, st>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_attention_weights(GroupArgs a, void *work, cudaStream_t st) {
    const int64_t units = (int64_t)a.n_req * a.q_heads;
    a.ml = static_cast<float2 *>(work);
    a.scores = reinterpret_cast<float *>(a.ml + units);
    group_attention_kernel<<<(unsigned)((units + 3) / 4), 128, 0, st>>>(a);
    add_weights_kernel<<<dim3((a.k + 255) / 256, a.n_req), 256, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace hs
