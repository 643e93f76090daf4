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
// Bound by HBM: every head is read once and written once.  Eight lanes share
// a head, two 16-byte chunks of it each, chosen so that both ends of every
// rotated pair are in one lane: the chunks of dimensions 8 l and
// rot_dim / 2 + 8 l (the two halves of the rotated part), then what does not
// rotate; or, interleaved, the lane's 16 consecutive dimensions.  The lane's
// pairs are numbers 8 l to 8 l + 7 either way.  The sum of squares takes
// three shuffles.  A warp takes one token and a run of its heads, four at a
// time with the loads of sixteen in flight, and computes the token's angles
// once, while the first of them arrive.
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

constexpr int kBatch = 4;  // loads in flight: kBatch heads per octet

__device__ __forceinline__ uint4 load16(const void *p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// Unit = (token, run of `run` heads, a multiple of four, in the order queries,
// keys, values); one warp each.
template <bool kInterleaved>
__global__ void __launch_bounds__(kQkThreads) qk_norm_rope_kernel(const QkArgs a, int run,
                                                                  int runs) {
    const int lane = threadIdx.x & 31, ol = lane & 7, oct = lane >> 3;
    const int64_t unit = (int64_t)blockIdx.x * (kQkThreads / 32) + (threadIdx.x >> 5);
    const int64_t tok = unit / runs;
    if (tok >= a.n_tok) return;
    const int h0 = (int)(unit - tok * runs) * run;
    const int all = a.q_heads + 2 * a.heads;
    const int h1 = min(all, h0 + run);
    const bool turns = ol < a.rot_dim / 16;  // this lane's pairs rotate
    // byte offsets of the lane's two chunks
    int c0, c1;
    if (kInterleaved) {
        c0 = ol * 32;
        c1 = c0 + 16;
    } else if (turns) {
        c0 = ol * 16;
        c1 = c0 + a.rot_dim;                 // rot_dim / 2 elements further
    } else {
        c0 = a.rot_dim * 2 + (ol - a.rot_dim / 16) * 32;
        c1 = c0 + 16;
    }
    // where head hd of the token is read and written (null: not written)
    int64_t row = tok;
    if (a.rows && h1 > a.q_heads) row = __ldg(a.rows + tok);
    const bool keep = row >= 0 && row < a.record_rows;
    auto source = [&](int hd) -> const uint8_t * {
        if (hd < a.q_heads) return a.q + (tok * a.q_stride + (int64_t)hd * kDim) * 2;
        hd -= a.q_heads;
        if (hd < a.heads) return a.k + (tok * a.k_stride + (int64_t)hd * kDim) * 2;
        return a.v + (tok * a.v_stride + (int64_t)(hd - a.heads) * kDim) * 2;
    };
    auto target = [&](int hd) -> uint8_t * {
        if (hd < a.q_heads) return a.q_out + (tok * a.q_heads + hd) * (int64_t)(kDim * 2);
        return keep ? a.records + (row * 2 * a.heads + (hd - a.q_heads)) * (int64_t)(kDim * 2)
                    : nullptr;
    };

    uint4 x0[kBatch], x1[kBatch];
    auto load = [&](int b0) {
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int hd = b0 + b * 4 + oct;
            x0[b] = x1[b] = make_uint4(0u, 0u, 0u, 0u);
            if (hd < h1) {
                const uint8_t *src = source(hd);
                x0[b] = load16(src + c0);
                x1[b] = load16(src + c1);
            }
        }
    };
    load(h0);
    float cs[8], sn[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        cs[e] = 1.f;
        sn[e] = 0.f;
    }
    if (turns && h0 < a.q_heads + a.heads) {
        const uint64_t pos = (uint64_t)(int64_t)__ldg(a.pos + tok);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint64_t turn = pos * a.freq[8 * ol + e];
            sincospif((float)(int32_t)(turn >> 32) * 0x1p-31f, &sn[e], &cs[e]);
        }
    }
    const uint4 one = make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u);
    uint4 wq0 = one, wq1 = one, wk0 = one, wk1 = one;
    if (a.wq) {
        wq0 = load16(a.wq + c0);
        wq1 = load16(a.wq + c1);
    }
    if (a.wk) {
        wk0 = load16(a.wk + c0);
        wk1 = load16(a.wk + c1);
    }

    for (int b0 = h0; b0 < h1; b0 += kBatch * 4) {
        if (b0 > h0) load(b0);
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int hd = b0 + b * 4 + oct;
            if (b0 + b * 4 >= h1) break;     // the whole warp
            uint4 y0 = x0[b], y1 = x1[b];
            if (b0 + b * 4 < a.q_heads + a.heads) {  // some octet has a query or key
                float f[16], g[16];
                unpack8(y0, f);
                unpack8(y1, f + 8);
                float ss = 0.f;
#pragma unroll
                for (int e = 0; e < 16; ++e) ss += f[e] * f[e];
#pragma unroll
                for (int d = 1; d < 8; d <<= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, d);
                const float rs = rsqrtf(ss * (1.f / kDim) + a.eps);
                const bool query = hd < a.q_heads;
                unpack8(query ? wq0 : wk0, g);
                unpack8(query ? wq1 : wk1, g + 8);
#pragma unroll
                for (int e = 0; e < 16; ++e) f[e] = f[e] * rs * g[e];
                if (turns) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        // pair e of the lane
                        const int i = kInterleaved ? 2 * e : e, j = kInterleaved ? 2 * e + 1 : e + 8;
                        const float u = f[i] * cs[e] - f[j] * sn[e];
                        f[j] = f[i] * sn[e] + f[j] * cs[e];
                        f[i] = u;
                    }
                }
                if (hd < a.q_heads + a.heads) {
                    y0 = pack8(f);
                    y1 = pack8(f + 8);
                }
            }
            if (hd < h1) {
                uint8_t *dst = target(hd);
                if (dst) {
                    *reinterpret_cast<uint4 *>(dst + c0) = y0;
                    *reinterpret_cast<uint4 *>(dst + c1) = y1;
                }
            }
        }
    }
    // The records may be host memory that a resolve behind this launch starts
    // reading before the grid's own flush: they are there before the CTA ends.
    if (h1 > a.q_heads) __threadfence_system();
}

}  // namespace

// Heads per warp: all of a token's where there are tokens enough for the SMs,
// fewer (down to four) where there are not, so that a decode step's few
// tokens still spread.
cudaError_t launch_qk_norm_rope(const QkArgs &a, cudaStream_t st) {
    const int all = a.q_heads + 2 * a.heads;
    const int quads = (all + 3) / 4;
    int runs = 1;
    while (runs < quads && (int64_t)a.n_tok * runs < kSms * 16) runs *= 2;
    if (runs > quads) runs = quads;
    const int run = (quads + runs - 1) / runs * 4;
    runs = (all + run - 1) / run;
    const int64_t units = (int64_t)a.n_tok * runs;
    const unsigned blocks = (unsigned)((units + kQkThreads / 32 - 1) / (kQkThreads / 32));
    if (a.interleaved)
        qk_norm_rope_kernel<true><<<blocks, kQkThreads, 0, st>>>(a, run, runs);
    else
        qk_norm_rope_kernel<false><<<blocks, kQkThreads, 0, st>>>(a, run, runs);
    return cudaGetLastError();
}

}  // namespace hs
