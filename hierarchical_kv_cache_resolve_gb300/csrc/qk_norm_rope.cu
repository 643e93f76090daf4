// RMS norm of each query and key head with the position rotation in the same
// pass (hs_qk_norm_rope): the producer of the queries and token records that
// the per-head attention consumers read.
//
// For a head x of 128 elements:  y = x * rsqrt(mean(x^2) + eps) * w, then each
// pair (a, b) of the first rot_dim dimensions turns by t = pos * inv_freq[i]:
// (a cos t - b sin t, a sin t + b cos t).  Everything is fp32 up to one
// rounding to bf16 at the end.
//
// The angle.  pos * inv_freq in fp32 is off by a tenth of a radian at a
// million positions.  The launch gives the frequency in turns as a 64-bit
// fraction, inv_freq / 2 pi * 2^64, so the product with the position modulo
// 2^64 -- one integer multiply -- is the angle's exact fraction of a turn;
// its top 32 bits, as a signed fraction of half a turn, go to sincospif.
//
// Work split: eight lanes share a head, each with 16 bytes of either half of
// it, so that a pair (i, i + 64) of a fully rotated head is in one lane and
// the sum of squares takes three shuffles.  A warp reads four heads at a time.
#include <cstdint>

#include "hs.h"
#include "hs_internal.cuh"

namespace hs {
namespace {

constexpr int kDim = 128;
constexpr int kQkThreads = 256;

__device__ __forceinline__ float lo(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float hi(uint32_t x) { return __uint_as_float(x & 0xFFFF0000u); }

__device__ __forceinline__ uint32_t pack2(float a, float b) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}

__device__ __forceinline__ void unpack8(const uint4 &x, float *f) {
    f[0] = lo(x.x); f[1] = hi(x.x); f[2] = lo(x.y); f[3] = hi(x.y);
    f[4] = lo(x.z); f[5] = hi(x.z); f[6] = lo(x.w); f[7] = hi(x.w);
}

__device__ __forceinline__ uint4 pack8(const float *f) {
    return make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
}

// One octet of lanes per (token, head); heads in the order queries, keys,
// values.  Element e of the lane: dimension 8 ol + e (e < 8) or
// 64 + 8 ol + e - 8.
__global__ void __launch_bounds__(kQkThreads) qk_norm_rope_kernel(const QkArgs a) {
    const int ol = threadIdx.x & 7;
    const int per_tok = a.q_heads + 2 * a.heads;
    const int64_t total = (int64_t)a.n_tok * per_tok;
    const int64_t step = (int64_t)gridDim.x * (kQkThreads / 8);
    const int64_t first = (int64_t)blockIdx.x * (kQkThreads / 8) + threadIdx.x / 8;
    // every octet of a warp goes round the loop the same number of times
    // (shuffles below); those past the end work on nothing
    const int64_t rounds = (total + step - 1) / step;
    for (int64_t it = 0; it < rounds; ++it) {
        const int64_t unit = first + it * step;
        const bool live = unit < total;
        const int64_t tok = live ? unit / per_tok : 0;
        const int head = live ? (int)(unit - tok * per_tok) : 0;
        int64_t row = 0;
        if (head >= a.q_heads) row = a.rows ? a.rows[tok] : tok;
        const bool store = live && (head < a.q_heads || (row >= 0 && row < a.record_rows));
        const uint8_t *src;
        uint8_t *dst;
        if (head < a.q_heads) {
            src = a.q + (tok * a.q_stride + (int64_t)head * kDim) * 2;
            dst = a.q_out + (tok * a.q_heads + head) * (int64_t)(kDim * 2);
        } else if (head < a.q_heads + a.heads) {
            src = a.k + (tok * a.k_stride + (int64_t)(head - a.q_heads) * kDim) * 2;
            dst = a.records + (row * 2 * a.heads + (head - a.q_heads)) * (int64_t)(kDim * 2);
        } else {
            src = a.v + (tok * a.v_stride + (int64_t)(head - a.q_heads - a.heads) * kDim) * 2;
            dst = a.records + (row * 2 * a.heads + (head - a.q_heads)) * (int64_t)(kDim * 2);
        }
        uint4 x0 = make_uint4(0, 0, 0, 0), x1 = x0;
        if (store) {
            x0 = *reinterpret_cast<const uint4 *>(src + ol * 16);
            x1 = *reinterpret_cast<const uint4 *>(src + 128 + ol * 16);
        }
        const bool value = head >= a.q_heads + a.heads;
        float f[16];
        unpack8(x0, f);
        unpack8(x1, f + 8);
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 16; ++e) ss += f[e] * f[e];
#pragma unroll
        for (int d = 1; d < 8; d <<= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, d);
        const float rs = rsqrtf(ss * (1.f / kDim) + a.eps);
        const uint8_t *w = head < a.q_heads ? a.wq : a.wk;
        if (w) {
            float g[16];
            unpack8(*reinterpret_cast<const uint4 *>(w + ol * 16), g);
            unpack8(*reinterpret_cast<const uint4 *>(w + 128 + ol * 16), g + 8);
#pragma unroll
            for (int e = 0; e < 16; ++e) f[e] = f[e] * rs * g[e];
        } else {
#pragma unroll
            for (int e = 0; e < 16; ++e) f[e] *= rs;
        }
        const uint32_t pos = a.rot_dim && live ? (uint32_t)a.pos[tok] : 0u;
        float y[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            const int dim = (e < 8 ? 0 : 64) + 8 * ol + (e & 7);
            // the dimension this one is paired with, its place, and the pair's number
            int pd = dim, i = 0;
            bool second = false;
            if (dim < a.rot_dim) {
                if (a.interleaved) {
                    pd = dim ^ 1;
                    i = dim >> 1;
                    second = dim & 1;
                } else {
                    const int half = a.rot_dim / 2;
                    second = dim >= half;
                    pd = second ? dim - half : dim + half;
                    i = second ? dim - half : dim;
                }
            }
            // its value: element pe of lane (pd % 64) / 8 of the octet
            const int pl = (pd & 63) >> 3, pe = (pd & 7) + (pd >= 64 ? 8 : 0);
            float other = 0.f;
            for (int c = 0; c < 16; ++c) {
                const float v = __shfl_sync(0xFFFFFFFFu, f[c], pl, 8);
                if (c == pe) other = v;
            }
            y[e] = f[e];
            if (dim < a.rot_dim) {
                const uint64_t turn = (uint64_t)(int64_t)(int32_t)pos * a.freq[i];
                float sn, cs;
                sincospif((float)(int32_t)(turn >> 32) * 0x1p-31f, &sn, &cs);
                y[e] = second ? other * sn + f[e] * cs : f[e] * cs - other * sn;
            }
        }
        if (store) {
            *reinterpret_cast<uint4 *>(dst + ol * 16) = value ? x0 : pack8(y);
            *reinterpret_cast<uint4 *>(dst + 128 + ol * 16) = value ? x1 : pack8(y + 8);
        }
    }
}

}  // namespace

cudaError_t launch_qk_norm_rope(const QkArgs &a, cudaStream_t st) {
    const int64_t units = (int64_t)a.n_tok * (a.q_heads + 2 * a.heads);
    const int64_t blocks = (units + kQkThreads / 8 - 1) / (kQkThreads / 8);
    qk_norm_rope_kernel<<<(unsigned)(blocks < 152 * 8 ? blocks : 152 * 8), kQkThreads, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace hs
