// Attention of a batch over a prefix that all its requests share
// (the prefix half of hs_prefix_attention).
//
// The queries of all requests that use one key-value head are rows of one
// matrix, so scores and outputs are matrix products on the tensor cores
// (tcgen05, accumulators in TMEM) and the prefix is read once for the whole
// batch.  For R requests of g query heads per key-value head the products do
// 4 * 128 * R g flops for 512 bytes: bound by HBM below about R g = 70, by
// the tensor cores above a few hundred.
//
// Work split: a CTA takes one key-value head, up to two tiles of 128 rows and
// a contiguous range of 128-key blocks; the ranges are cut so that the grid
// covers the 152 SMs once, and merge_kernel joins their parts.  One CTA per
// SM:
//   warp 8    brings key and value blocks (32 KB each, TMA, 128-byte swizzle)
//             into a ring of five, in the order the products use them;
//   warp 9    one thread issues S_t = Q_t K^T and O_t += P_t V;
//   warps 0-3 and 4-7  the softmax of tile 0 and 1: a thread per row reads
//             its 128 scores from TMEM, keeps the running maximum and sum in
//             registers and writes P back as bf16 over the scores, where the
//             second product takes it from (its only rounding).
// While one tile's softmax runs, the tensor core works on the other's
// products.  With a single tile of rows (few queries, bound by HBM) the two
// softmax groups take every other key block of the same rows, and the two
// results are joined in shared memory at the end.
//
// The maximum only rises when a block exceeds it by more than 2^8: until then
// P is at most 2^8 too large, which bf16 and the fp32 sums hold as exactly,
// and O needs no rescaling pass through the registers.  The scores' scale is
// applied as |scale| with the queries' sign turned, so that the row maximum
// can be taken before scaling.
//
// TMEM columns: S_0/P_0 0, S_1/P_1 128, O_0 256, O_1 384.
//
// Every wait gives up after a second: the CTA's rows become NaN and
// HS_ATTN_STATUS_TIMEOUT is set (hs_attention_status); copies and products in
// flight are waited for, with the same limit, before the CTA leaves.
#include <cmath>
#include <cstdint>

#include <cuda.h>

#include "hs.h"
#include "hs_internal.cuh"

namespace hs {
namespace {

constexpr int kDim = 128;
constexpr int kBlock = 128;                     // keys per block, rows per tile
constexpr uint32_t kTileBytes = kBlock * kDim * 2;  // 32 KB
constexpr uint32_t kAtom = kBlock * 128;        // 64 of the 128 dimensions: 16 KB
constexpr int kSlots = 5;
constexpr int kPrefixThreads = 384;             // three warpgroups; the last two warps idle
constexpr uint64_t kWaitLimitNs = 1000000000ull;
constexpr float kRise = 8.f;                    // log2 of how far P may exceed 1

constexpr uint32_t kOffQ = 0;                       // two tiles
constexpr uint32_t kOffRing = 2 * kTileBytes;
constexpr uint32_t kOffBar = kOffRing + kSlots * kTileBytes;
// full[kSlots], empty[kSlots], s_full[2], p_half[2], p_ready[2], drained
constexpr int kBars = 2 * kSlots + 7;
constexpr uint32_t kOffWord = kOffBar + 8 * kBars;  // TMEM address, abort flag
constexpr uint32_t kSmem = kOffWord + 16 + 1024;    // and room to align to 1 KB
static_assert(kSmem <= 232448, "fits an SM");
// after the main loop the ring holds the second group's O [32 chunks][128
// rows] of float4 and (m, l) [128]
static_assert(kTileBytes * 2 + kBlock * 8 <= kSlots * kTileBytes, "the exchange fits the ring");

__device__ uint32_t g_prefix_status;

__device__ __forceinline__ uint32_t smem_addr(const void *p) {
    return (uint32_t)__cvta_generic_to_shared(p);
}

__device__ __forceinline__ uint64_t globaltimer() {
    uint64_t t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}

__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void mbar_expect(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
                 : "memory");
}

__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

// Waits for the phase of `bar` with this parity; false after the limit, or
// once another wait of the CTA has given up.
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity,
                                          volatile uint32_t *abort_flag) {
    if (mbar_try(bar, parity)) return true;
    const uint64_t t0 = globaltimer();
    while (!mbar_try(bar, parity)) {
        if (*abort_flag || globaltimer() - t0 > kWaitLimitNs) {
            *abort_flag = 1;
            return false;
        }
    }
    return true;
}

// The same without regard to the flag: what must have ended before the CTA
// may reuse or leave its memory.
__device__ __forceinline__ void mbar_drain(uint32_t bar, uint32_t parity) {
    const uint64_t t0 = globaltimer();
    while (!mbar_try(bar, parity) && globaltimer() - t0 <= kWaitLimitNs) {
    }
}

__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap *map, int x, int y,
                                         uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

// Shared-memory matrix descriptor, 128-byte swizzle: address, the strides
// between 64-element chunks of a row-contiguous operand (lead) and between
// groups of eight 128-byte rows (1 KB), all in 16-byte units.  The address is
// below 2^18, so bytes / 16 may be added to a descriptor.
__device__ __forceinline__ uint64_t operand(uint32_t addr, uint32_t lead) {
    return (uint64_t)(addr >> 4) | (uint64_t)(lead >> 4) << 16 | (uint64_t)(1024 >> 4) << 32 |
           1ull << 46 | 2ull << 61;
}

// fp32 accumulators, bf16 operands, N = 128, M = 128; bit 16: B is given with
// its N dimension contiguous
constexpr uint32_t kIdesc = 1u << 4 | 1u << 7 | 1u << 10 | (128u >> 3) << 17 | (128u >> 4) << 24;
constexpr uint32_t kIdescV = kIdesc | 1u << 16;

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
        : "memory");
}

__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                       bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
        : "memory");
}

// One lane of a converged warp, the same one every time.
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xFFFFFFFF;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r));
    return r != 0;
}

// `bar` gets an arrival once every product issued so far by this thread is done
__device__ __forceinline__ void mma_commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                     bar)
                 : "memory");
}


// 32 columns of this thread's TMEM lane; complete after tmem_wait_ld
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t *v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
        "%12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, "
        "%30, %31}, [%32];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
          "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]),
          "=r"(v[14]), "=r"(v[15]), "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]),
          "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]), "=r"(v[25]),
          "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
        : "r"(addr));
}

__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t *v) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, "
        "%10, %11, %12, %13, %14, %15};" ::"r"(v[0]),
        "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
        "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(addr)
        : "memory");
}

__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t *v) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, "
        "%10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, "
        "%28, %29, %30, %31};" ::"r"(v[0]),
        "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
        "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]),
        "r"(v[16]), "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]),
        "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]), "r"(v[29]),
        "r"(v[30]), "r"(v[31]), "r"(addr)
        : "memory");
}

// Waits for this warp's TMEM loads; v[0..n) may be used only from here on
// (the empty statements keep the compiler from using them earlier).
template <int n>
__device__ __forceinline__ void tmem_wait_ld(uint32_t *v) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < n; ++i) asm volatile("" : "+r"(v[i]));
}
__device__ __forceinline__ void tmem_wait_st() {
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void fence_before() {
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void fence_after() {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

// two fp32 at once
__device__ __forceinline__ uint64_t pair(uint32_t a, uint32_t b) { return (uint64_t)b << 32 | a; }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__global__ void __launch_bounds__(kPrefixThreads, 1)
    prefix_kernel(const __grid_constant__ CUtensorMap map, const GroupArgs a, const PrefixPlan p) {
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    uint8_t *smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
    const uint32_t s0 = smem_addr(smem);
    volatile uint32_t *words = reinterpret_cast<volatile uint32_t *>(smem + kOffWord);
    volatile uint32_t *abort_flag = words + 1;
    const uint32_t bars = s0 + kOffBar;
    auto full = [&](int i) { return bars + 8u * i; };
    auto empty = [&](int i) { return bars + 8u * (kSlots + i); };
    auto s_full = [&](int t) { return bars + 8u * (2 * kSlots + t); };
    auto p_half = [&](int t) { return bars + 8u * (2 * kSlots + 2 + t); };
    auto p_ready = [&](int t) { return bars + 8u * (2 * kSlots + 4 + t); };
    const uint32_t drained = bars + 8u * (2 * kSlots + 6);

    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);  // known to be the same in a warp
    // the CTAs that read the same keys are neighbours
    const int pairs = (p.row_tiles + 1) / 2;
    const int pair_id = blockIdx.x % pairs, head = (blockIdx.x / pairs) % a.heads;
    const int split = blockIdx.x / pairs / a.heads;
    const int group = a.q_heads / a.heads;
    const int64_t n_rows = (int64_t)a.n_req * group;
    // one tile: its two halves of the blocks go to the two groups
    const bool alone = 2 * pair_id + 1 == p.row_tiles;
    const int b0 = (int)((int64_t)split * p.blocks / p.splits);
    const int b1 = (int)((int64_t)(split + 1) * p.blocks / p.splits);
    const int n = b1 - b0;  // >= 1
    const int ahead = min(alone ? 2 : 1, n);

    // The ring's items in the order the products use them: K of the first
    // blocks, then V of block j and K of block j + ahead.
    auto load = [&](int i) {
        const int u = i - ahead, both = 2 * (n - ahead);  // both: V, K, V, K, ...; then V only
        const bool is_k = u < 0 || (u < both && (u & 1));
        const int block = u < 0 ? i : u < both ? u / 2 + (u & 1 ? ahead : 0) : u - (n - ahead);
        const int x = (is_k ? head : a.heads + head) * kDim, slot = i % kSlots;
        const uint32_t dst = s0 + kOffRing + slot * kTileBytes;
        mbar_expect(full(slot), kTileBytes);
        tma_load(dst, &map, x, (b0 + block) * kBlock, full(slot));
        tma_load(dst + kAtom, &map, x + 64, (b0 + block) * kBlock, full(slot));
    };
    if (warp == 9) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                         s0 + kOffWord)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    } else if (warp == 8 && lane == 0) {
        *abort_flag = 0;
        for (int i = 0; i < kSlots; ++i) {
            mbar_init(full(i), 1);
            mbar_init(empty(i), 1);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(s_full(t), 1);
            mbar_init(p_half(t), kBlock);
            mbar_init(p_ready(t), kBlock);
        }
        mbar_init(drained, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        for (int i = 0; i < kSlots && i < 2 * n; ++i) load(i);
    }
    // softmax groups: thread = row (TMEM lane) of tile t
    const int t = (warp >> 2) & 1, row = tid & 127;
    const int64_t m_row = (int64_t)(2 * pair_id + (alone ? 0 : t)) * kBlock + row;
    const bool live = m_row < n_rows;
    const int64_t q_row = live ? m_row / group * a.q_heads + head * group + m_row % group : 0;
    // the queries' sign bits are turned for a negative scale; for scale 0 the
    // queries become 0, so that a masked score stays -inf
    const bool flat = a.scale_log2 == 0.f;
    const float scale = flat ? 1.f : fabsf(a.scale_log2);
    if (warp < 8 && (!alone || t == 0)) {
        const uint32_t flip = a.scale_log2 < 0.f ? 0x80008000u : 0u;
        const uint4 *src = reinterpret_cast<const uint4 *>(a.q + q_row * (2 * kDim));
        uint8_t *dst = smem + kOffQ + t * kTileBytes + row * 128;
#pragma unroll
        for (int c = 0; c < 16; ++c) {
            uint4 x = live && !flat ? __ldg(src + c) : make_uint4(0u, 0u, 0u, 0u);
            x.x ^= flip;
            x.y ^= flip;
            x.z ^= flip;
            x.w ^= flip;
            *reinterpret_cast<uint4 *>(dst + (c >> 3) * kAtom + (((c & 7) ^ (row & 7)) << 4)) = x;
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = words[0];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    if (warp >= 8) asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (warp == 8) {
        // ---- the rest of the ring's items
        if (lane == 0) {
            int i = kSlots;
            for (; i < 2 * n; ++i) {
                if (!mbar_wait(empty(i % kSlots), (i / kSlots - 1) & 1, abort_flag)) break;
                load(i);
            }
            // nothing may land after the CTA has left the ring (in a normal run
            // the products have waited for all of it)
            const int issued = min(i, 2 * n);
            for (int j = max(0, issued - kSlots); j < issued; ++j)
                mbar_drain(full(j % kSlots), (j / kSlots) & 1);
        }
    } else if (warp == 9) {
        // ---- the products: the whole warp waits, one lane issues
        const bool issuer = elect_one();
        bool ok = true;
        const uint64_t q_op = operand(s0 + kOffQ, 16);
        const uint64_t k_op = operand(s0 + kOffRing, 16), v_op = operand(s0 + kOffRing, kAtom);
        int slot = 0;                       // of the next item, and its phase
        uint32_t phase = 0;
        auto next = [&]() {
            if (++slot == kSlots) {
                slot = 0;
                phase ^= 1;
            }
        };
        auto arrived = [&](int at, uint32_t ph) {
            const bool r = mbar_wait(full(at), ph, abort_flag);
            fence_after();
            return r;
        };
        auto commit = [&](uint32_t bar) {
            if (issuer) mma_commit(bar);
        };
        // S_t = Q_t K^T, 16 dimensions at a time
        auto scores = [&](int tile, int at) {
            const uint64_t q = q_op + (alone ? 0 : tile) * (kTileBytes >> 4);
            const uint64_t k = k_op + at * (kTileBytes >> 4);
            const uint32_t d = tmem + tile * 128;
            if (issuer) {
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    const uint64_t off = ((c >> 2) * kAtom + (c & 3) * 32) >> 4;
                    mma_ss(d, q + off, k + off, kIdesc, c > 0);
                }
            }
        };
        // O_t += P_t V, 16 keys at a time, each half of P as it is ready
        auto values = [&](int tile, int at, int turn, bool add) {
            const uint64_t v = v_op + at * (kTileBytes >> 4);
            const uint32_t pt = tmem + tile * 128, d = tmem + 256 + tile * 128;
            if (!mbar_wait(p_half(tile), turn & 1, abort_flag)) return false;
            fence_after();
            if (issuer) {
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    mma_ts(d, pt + c * 8, v + c * (2048 >> 4), kIdescV, add || c > 0);
            }
            if (!mbar_wait(p_ready(tile), turn & 1, abort_flag)) return false;
            fence_after();
            if (issuer) {
#pragma unroll
                for (int c = 4; c < 8; ++c)
                    mma_ts(d, pt + c * 8, v + c * (2048 >> 4), kIdescV, true);
            }
            return true;
        };
        if (alone) {
            for (int j = 0; j < ahead && ok; ++j) {
                if (!(ok = arrived(slot, phase))) break;
                scores(j, slot);
                commit(s_full(j));
                commit(empty(slot));
                next();
            }
            for (int j = 0; j < n && ok; ++j) {
                const int tile = j & 1;
                if (!(ok = arrived(slot, phase))) break;
                if (!(ok = values(tile, slot, j >> 1, j >= 2))) break;
                commit(empty(slot));
                next();
                if (j + 2 < n) {
                    if (!(ok = arrived(slot, phase))) break;
                    scores(tile, slot);
                    commit(empty(slot));
                    next();
                }
                commit(s_full(tile));
            }
        } else {
            if ((ok = arrived(slot, phase))) {
                for (int tile = 0; tile < 2; ++tile) {
                    scores(tile, slot);
                    commit(s_full(tile));
                }
                commit(empty(slot));
                next();
            }
            for (int j = 0; j < n && ok; ++j) {
                const bool more = j + 1 < n;
                const int v_slot = slot;
                const uint32_t v_phase = phase;
                next();
                for (int tile = 0; tile < 2; ++tile) {
                    if (tile == 0 && !(ok = arrived(v_slot, v_phase))) break;
                    if (!(ok = values(tile, v_slot, j, j > 0))) break;
                    if (tile == 1) commit(empty(v_slot));
                    if (more) {
                        if (tile == 0 && !(ok = arrived(slot, phase))) break;
                        scores(tile, slot);
                        if (tile == 1) commit(empty(slot));
                    }
                    commit(s_full(tile));
                }
                if (more) next();
            }
        }
        // no product may still run when the TMEM is given back
        commit(drained);
        mbar_drain(drained, 0);
    } else if (warp < 8) {
        // ---- softmax
        asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
        const uint32_t lanes = (uint32_t)(warp & 3) * 32 << 16;
        const uint32_t ts = tmem + lanes + t * 128, to = tmem + lanes + 256 + t * 128;
        // blocks b0 + first, + step, ...
        const int first = alone ? t : 0, step = alone ? 2 : 1;
        const int mine = n > first ? (n - first + step - 1) / step : 0;
        float m = -INFINITY, l = 0.f;
        bool ok = true;
        for (int j = 0; j < mine; ++j) {
            ok = mbar_wait(s_full(t), j & 1, abort_flag);
            if (!__all_sync(0xFFFFFFFFu, ok)) {
                ok = false;
                break;
            }
            fence_after();
            const int64_t left = a.prefix_len - (int64_t)(b0 + first + j * step) * kBlock;
            uint32_t s[128];
            float x[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
            tmem_ld32(ts, s);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                tmem_wait_ld<32>(s + c * 32);
                if (c < 3) tmem_ld32(ts + (c + 1) * 32, s + (c + 1) * 32);
                if (left < kBlock) {
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (c * 32 + e >= (int)left) s[c * 32 + e] = 0xFF800000u;  // -inf
                }
#pragma unroll
                for (int e = 0; e < 32; e += 8)
#pragma unroll
                    for (int h = 0; h < 4; ++h)
                        x[h] = fmaxf(fmaxf(x[h], __uint_as_float(s[c * 32 + e + 2 * h])),
                                     __uint_as_float(s[c * 32 + e + 2 * h + 1]));
            }
            const float top = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])) * scale;
            if (__any_sync(0xFFFFFFFFu, top > m + kRise || m == -INFINITY)) {
                const float up = fmaxf(m, top);
                const float f = m == -INFINITY ? 0.f : ex2(m - up);
                m = up;
                l *= f;
                if (j > 0) {  // s_full came after the products on O
                    uint32_t o[32];
#pragma unroll 1
                    for (int c = 0; c < 4; ++c) {
                        tmem_ld32(to + c * 32, o);
                        tmem_wait_ld<32>(o);
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                        tmem_st32(to + c * 32, o);
                    }
                }
            }
            const float shift = m == -INFINITY ? 0.f : -m;
            const uint64_t scale2 = pair(__float_as_uint(scale), __float_as_uint(scale));
            const uint64_t shift2 = pair(__float_as_uint(shift), __float_as_uint(shift));
            uint64_t sum[2] = {0ull, 0ull};
#pragma unroll
            for (int c = 0; c < 4; ++c) {
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
                    mbar_arrive(c == 1 ? p_half(t) : p_ready(t));
                }
            }
            sum[0] = add2(sum[0], sum[1]);
            l += __uint_as_float((uint32_t)sum[0]) + __uint_as_float((uint32_t)(sum[0] >> 32));
        }
        // every product on O done
        if (ok && mine > 0) {
            ok = mbar_wait(s_full(t), mine & 1, abort_flag);
            fence_after();
        }
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok && lane == 0) atomicOr(&g_prefix_status, HS_ATTN_STATUS_TIMEOUT);
        if (!ok) m = __int_as_float(0x7FC00000);  // the merge makes such rows NaN

        float4 *xo = reinterpret_cast<float4 *>(smem + kOffRing);
        float2 *xml = reinterpret_cast<float2 *>(smem + kOffRing + 2 * kTileBytes);
        const bool sender = alone && t == 1;
        float f1 = 1.f, f2 = 0.f;
        if (alone) {
            // both groups' products are done: nothing reads the ring any more
            asm volatile("bar.sync 1, 256;" ::: "memory");
            if (sender) {
                xml[row] = make_float2(m, mine > 0 ? l : 0.f);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t o[32];
                    if (mine > 0) {
                        tmem_ld32(to + c * 32, o);
                        tmem_wait_ld<32>(o);
                    }
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        xo[(c * 8 + e) * kBlock + row] =
                            mine > 0 ? make_float4(__uint_as_float(o[4 * e]),
                                                   __uint_as_float(o[4 * e + 1]),
                                                   __uint_as_float(o[4 * e + 2]),
                                                   __uint_as_float(o[4 * e + 3]))
                                     : make_float4(0.f, 0.f, 0.f, 0.f);
                }
            }
            asm volatile("bar.sync 1, 256;" ::: "memory");
            if (!sender) {
                const float2 ml = xml[row];
                if (ml.x != ml.x) m = ml.x;
                const float M = m != m ? m : fmaxf(m, ml.x);
                const float base = M == -INFINITY ? 0.f : M;
                f1 = ex2(m - base);
                f2 = ex2(ml.x - base);
                l = l * f1 + ml.y * f2;
                m = M;
            }
        }
        if (!sender) {
            const int64_t part = ((int64_t)split * a.n_req) * a.q_heads + q_row;
            float4 *dst = reinterpret_cast<float4 *>(p.o + part * kDim);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                uint32_t o[32];
                tmem_ld32(to + c * 32, o);
                tmem_wait_ld<32>(o);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    float4 v = make_float4(__uint_as_float(o[4 * e]), __uint_as_float(o[4 * e + 1]),
                                           __uint_as_float(o[4 * e + 2]),
                                           __uint_as_float(o[4 * e + 3]));
                    if (alone) {
                        const float4 u = xo[(c * 8 + e) * kBlock + row];
                        v.x = v.x * f1 + u.x * f2;
                        v.y = v.y * f1 + u.y * f2;
                        v.z = v.z * f1 + u.z * f2;
                        v.w = v.w * f1 + u.w * f2;
                    }
                    if (live) dst[c * 8 + e] = v;
                }
            }
            if (live) p.ml[part] = make_float2(m, l);
        }
        fence_before();
    }
    __syncthreads();
    if (warp == 9) {
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
    }
}

using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                 const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                 const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's tensor-map encoder, looked up once (nullptr: not available).
EncodeTiled encode_tiled() {
    static const EncodeTiled fn = [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                             &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<EncodeTiled>(f);
    }();
    return fn;
}

}  // namespace

// Splits of the prefix's key blocks: as many as fill the SMs once with a CTA
// for every key-value head and pair of row tiles, and at least two blocks
// each (one for each softmax group).
PrefixPlan prefix_plan(int n_req, int q_heads, int heads, int64_t prefix_len) {
    PrefixPlan p = {};
    if (prefix_len < 1) return p;
    const int64_t rows = (int64_t)n_req * (q_heads / heads);
    p.blocks = (int)((prefix_len + kBlock - 1) / kBlock);
    p.row_tiles = (int)((rows + kBlock - 1) / kBlock);
    const int units = heads * ((p.row_tiles + 1) / 2);
    int s = kSms / units;
    if (s > (p.blocks + 1) / 2) s = (p.blocks + 1) / 2;
    p.splits = s < 1 ? 1 : s;
    return p;
}

cudaError_t launch_prefix(const GroupArgs &a, const PrefixPlan &p, cudaStream_t st) {
    const EncodeTiled encode = encode_tiled();
    if (!encode) return cudaErrorNotSupported;
    CUtensorMap map;
    const cuuint64_t dims[2] = {(cuuint64_t)a.heads * 2 * kDim, (cuuint64_t)a.prefix_len};
    const cuuint64_t strides[1] = {(cuuint64_t)a.heads * 4 * kDim};
    const cuuint32_t box[2] = {64, kBlock}, one[2] = {1, 1};
    if (encode(&map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<uint8_t *>(a.prefix), dims,
               strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return cudaErrorInvalidValue;
    cudaError_t e = cudaFuncSetAttribute(prefix_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)kSmem);
    if (e != cudaSuccess) return e;
    const int units = a.heads * ((p.row_tiles + 1) / 2);
    prefix_kernel<<<(unsigned)units * p.splits, kPrefixThreads, kSmem, st>>>(map, a, p);
    return cudaGetLastError();
}

cudaError_t prefix_attention_status(uint32_t *status) {
    uint32_t v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_prefix_status, sizeof(v));
    if (e != cudaSuccess) return e;
    *status = v;
    if (v) {
        const uint32_t zero = 0;
        e = cudaMemcpyToSymbol(g_prefix_status, &zero, sizeof(zero));
    }
    return e;
}

}  // namespace hs
