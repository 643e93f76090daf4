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
// fraction, inv_freq / 2 pi * 2^64 to one unit, so the product with the position
// modulo 2^64 -- one integer multiply -- is the angle's fraction of a turn, to
// 2^-33 of one at any position.  Its top 32 bits, as a signed fraction of half a
// turn, are rounded to fp32 (2^-25 of half a turn, which is what remains) and go
// to sincospif.
//
// Bound by HBM: every head is read once and written once.  Eight lanes share
// a head, two 16-byte chunks of it each, chosen so that both ends of every
// rotated pair are in one lane: the chunks of dimensions 8 l and
// rot_dim / 2 + 8 l (the two halves of the rotated part), then what does not
// rotate; or, interleaved, the lane's 16 consecutive dimensions.  The lane's
// pairs are numbers 8 l to 8 l + 7 either way.  The sum of squares takes
// three shuffles.  A warp takes a token, computes its angles once, and goes
// through its query, key and value heads four at a time, four such groups
// loaded together; arithmetic is on packed pairs of fp32, since the issue
// slots are what comes next after the memory.
// Measured: 132 us for 32768 tokens of 32 query and 8 key-value heads, 806 MB
// read and written at 6.1 TB/s; 3.8 us for 8 such tokens.
#include <cstdint>

#include "hs.h"
#include "hs_internal.cuh"

namespace hs {
namespace {

constexpr int kDim = 128;
constexpr int kQkThreads = 256;

constexpr int kQkCtas = 2;   // resident CTAs per SM
constexpr int kBatch = 4;    // groups of four heads whose loads are issued together

// two fp32 in one register pair
__device__ __forceinline__ uint64_t pair(float a, float b) {
    return (uint64_t)__float_as_uint(a) | (uint64_t)__float_as_uint(b) << 32;
}
__device__ __forceinline__ float first(uint64_t x) { return __uint_as_float((uint32_t)x); }
__device__ __forceinline__ float second(uint64_t x) { return __uint_as_float((uint32_t)(x >> 32)); }
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t neg2(uint64_t a) { return a ^ 0x8000000080000000ull; }

// two packed bf16 as fp32, and back
__device__ __forceinline__ uint64_t widen(uint32_t x) {
    return (uint64_t)(x << 16) | (uint64_t)(x & 0xFFFF0000u) << 32;
}
__device__ __forceinline__ uint32_t narrow(uint64_t x) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(second(x)), "f"(first(x)));
    return r;
}

__device__ __forceinline__ uint4 load16(const void *p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// Unit = (token, run of `run` heads, in the order queries, keys, values); the
// warps of the grid take the units in turn.
template <bool kInterleaved>
__global__ void __launch_bounds__(kQkThreads, kQkCtas)
    qk_norm_rope_kernel(const QkArgs a, int run, int runs) {
    const int lane = threadIdx.x & 31, ol = lane & 7, oct = lane >> 3;
    const int64_t units = (int64_t)a.n_tok * runs;
    const int64_t step = (int64_t)gridDim.x * (kQkThreads / 32);
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
    c0 += oct * 2 * kDim;
    c1 += oct * 2 * kDim;

    // cosines and sines of the lane's pairs, two pairs to a word: of the token
    // of this unit, computed behind the unit's first loads
    uint64_t cs[4], sn[4];
    int32_t pos = 0;
    bool stale = false;
    auto angles = [&]() {
        stale = false;
        const uint64_t at = (uint64_t)(int64_t)pos;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float s0, q0, s1, q1;
            const uint64_t t0 = at * a.freq[8 * ol + 2 * e], t1 = at * a.freq[8 * ol + 2 * e + 1];
            sincospif((float)(int32_t)(t0 >> 32) * 0x1p-31f, &s0, &q0);
            sincospif((float)(int32_t)(t1 >> 32) * 0x1p-31f, &s1, &q1);
            cs[e] = pair(q0, q1);
            sn[e] = pair(s0, s1);
        }
    };

    // heads [0, n) that lie at src and go to dst, normed and turned
    auto heads = [&](const uint8_t *src, uint8_t *dst, int n, const uint8_t *w, bool keep) {
        uint64_t g[8];
        {
            const uint4 one = make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u);
            const uint4 g0 = w ? load16(w + c0 - oct * 2 * kDim) : one;
            const uint4 g1 = w ? load16(w + c1 - oct * 2 * kDim) : one;
            g[0] = widen(g0.x); g[1] = widen(g0.y); g[2] = widen(g0.z); g[3] = widen(g0.w);
            g[4] = widen(g1.x); g[5] = widen(g1.y); g[6] = widen(g1.z); g[7] = widen(g1.w);
        }
        for (int h = 0; h < n; h += 4 * kBatch) {
            uint4 x0[kBatch], x1[kBatch];
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                x0[b] = x1[b] = make_uint4(0u, 0u, 0u, 0u);
                if (h + 4 * b + oct < n) {
                    const uint8_t *p = src + (h + 4 * b) * (2 * kDim);
                    x0[b] = load16(p + c0);
                    x1[b] = load16(p + c1);
                }
            }
            if (stale) angles();
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                if (h + 4 * b >= n) break;   // the whole warp
                uint64_t f[8];
                f[0] = widen(x0[b].x); f[1] = widen(x0[b].y);
                f[2] = widen(x0[b].z); f[3] = widen(x0[b].w);
                f[4] = widen(x1[b].x); f[5] = widen(x1[b].y);
                f[6] = widen(x1[b].z); f[7] = widen(x1[b].w);
                uint64_t s2 = mul2(f[0], f[0]);
#pragma unroll
                for (int e = 1; e < 8; ++e) s2 = fma2(f[e], f[e], s2);
                float ss = first(s2) + second(s2);
#pragma unroll
                for (int d = 1; d < 8; d <<= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, d);
                const float r = rsqrtf(ss * (1.f / kDim) + a.eps);
                const uint64_t rr = pair(r, r);
#pragma unroll
                for (int e = 0; e < 8; ++e) f[e] = mul2(mul2(f[e], rr), g[e]);
                if (turns) {
                    if (kInterleaved) {
                        // word e holds pair e: (a, b) -> (a c - b s, a s + b c)
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const float c = e & 1 ? second(cs[e >> 1]) : first(cs[e >> 1]);
                            const float s = e & 1 ? second(sn[e >> 1]) : first(sn[e >> 1]);
                            const float u = first(f[e]), v = second(f[e]);
                            f[e] = pair(u * c - v * s, u * s + v * c);
                        }
                    } else {
                        // words e and e + 4 hold the first and second ends of
                        // pairs 2e and 2e + 1
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const uint64_t u = f[e], v = f[e + 4];
                            f[e] = fma2(u, cs[e], neg2(mul2(v, sn[e])));
                            f[e + 4] = fma2(u, sn[e], mul2(v, cs[e]));
                        }
                    }
                }
                if (keep && h + 4 * b + oct < n) {
                    uint8_t *p = dst + (h + 4 * b) * (2 * kDim);
                    *reinterpret_cast<uint4 *>(p + c0) =
                        make_uint4(narrow(f[0]), narrow(f[1]), narrow(f[2]), narrow(f[3]));
                    *reinterpret_cast<uint4 *>(p + c1) =
                        make_uint4(narrow(f[4]), narrow(f[5]), narrow(f[6]), narrow(f[7]));
                }
            }
        }
    };

    for (int64_t unit = (int64_t)blockIdx.x * (kQkThreads / 32) + (threadIdx.x >> 5); unit < units;
         unit += step) {
        const int64_t tok = unit / runs;
        const int h0 = (int)(unit - tok * runs) * run, h1 = h0 + run;
        // the unit's queries, keys and values
        const int kv0 = a.q_heads, v0 = kv0 + a.heads, all = v0 + a.heads;
        const int q1 = min(h1, kv0), ka = max(h0, kv0), kb = min(h1, v0), va = max(h0, v0),
                  vb = min(h1, all);
        int64_t row = tok;
        if (a.rows && h1 > kv0) row = __ldg(a.rows + tok);
        const bool keep = row >= 0 && row < a.record_rows;
        uint8_t *rec = a.records + (keep ? row : 0) * (int64_t)(a.heads * 4 * kDim);
        stale = turns && h0 < v0;
        if (stale) pos = __ldg(a.pos + tok);
        if (h0 < kv0)
            heads(a.q + (tok * a.q_stride + (int64_t)h0 * kDim) * 2,
                  a.q_out + (tok * a.q_heads + h0) * (int64_t)(2 * kDim), q1 - h0, a.wq, true);
        if (ka < kb)
            heads(a.k + (tok * a.k_stride + (int64_t)(ka - kv0) * kDim) * 2,
                  rec + (ka - kv0) * 2 * kDim, kb - ka, a.wk, keep);
        if (va < vb && keep) {
            // values go over as they are
            const uint8_t *src = a.v + (tok * a.v_stride + (int64_t)(va - v0) * kDim) * 2;
            uint8_t *dst = rec + (va - kv0) * 2 * kDim;
            const int bytes = (vb - va) * 2 * kDim;
            for (int o = lane * 16; o < bytes; o += 4 * 512) {
                uint4 x[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (o + e * 512 < bytes) x[e] = load16(src + o + e * 512);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (o + e * 512 < bytes) *reinterpret_cast<uint4 *>(dst + o + e * 512) = x[e];
            }
        }
    }
    // The records may be host memory that a resolve behind this launch starts
    // reading before the grid's own flush: they are there before the CTA ends.
    __threadfence_system();
}

}  // namespace

// Heads per unit: all of a token's where there are tokens enough for every
// warp, fewer (down to four) where there are not, so that a decode step's few
// tokens still spread over the SMs, but no more units than warps.
cudaError_t launch_qk_norm_rope(const QkArgs &a, cudaStream_t st) {
    constexpr int kWarps = kQkThreads / 32;
    const int all = a.q_heads + 2 * a.heads;
    const int quads = (all + 3) / 4;
    const int64_t warps = kSms * kQkCtas * kWarps;
    int runs = (int)(warps / a.n_tok < quads ? warps / a.n_tok : quads);
    if (runs < 1) runs = 1;
    const int run = (quads + runs - 1) / runs * 4;
    runs = (all + run - 1) / run;
    const int64_t blocks = ((int64_t)a.n_tok * runs + kWarps - 1) / kWarps;
    const unsigned grid = (unsigned)(blocks < kSms * kQkCtas ? blocks : kSms * kQkCtas);
    if (a.interleaved)
        qk_norm_rope_kernel<true><<<grid, kQkThreads, 0, st>>>(a, run, runs);
    else
        qk_norm_rope_kernel<false><<<grid, kQkThreads, 0, st>>>(a, run, runs);
    return cudaGetLastError();
}

}  // namespace hs
