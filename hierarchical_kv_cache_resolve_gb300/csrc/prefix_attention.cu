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
// Work split: the key blocks of all key-value heads, head after head, are cut
// into equal contiguous ranges, one for each group of CTAs; the CTAs of a group
// take the same range (their reads meet in L2) for a pair of row tiles of 128
// each.  The first CTAs of the grid take the requests' own rows instead
// (rows_gather.cuh): the two share the GPU at once, so the rows' reads use the
// bandwidth that the products leave and neither waits for the other's last CTA.
// merge_kernel joins all parts.  One CTA per SM:
//   warp 8    brings key and value blocks (TMA, 128-byte swizzle) into a ring
//             of 160 KB, in the order the products use them;
//   warps 9 and 10  one thread issues S_t = Q_t K^T and O_t += P_t V;
//   warps 0-3 and 4-7  the softmax of tile 0 and 1: a thread per row reads
//             its scores from TMEM, keeps the running maximum and sum in
//             registers and writes P back as bf16 over the scores, where the
//             second product takes it from.
// Pairs of tiles take blocks of 128 keys, and one warp issues the products of
// both in turn: while one tile's softmax runs, the tensor core works on the
// other's products.  (Measured at 512 queries to a head on 131072 keys beside
// 2048 rows, the products then still issued under a branch: 237 us; blocks of
// 64 keys with their scores in two buffers 280, as a product of N = 64 runs at
// two thirds of the rate; a warp for each tile 310; sixteen softmax warps, two
// threads to a row, 250.)
// With a single tile of rows (few queries, bound by HBM and latency) the two
// softmax groups take every other block of the same rows, each with a ring and
// a product warp of its own, and the two results are joined in shared memory
// behind the last block of a head.  Here blocks of 64 keys in two buffers are
// the faster ones, as softmax and products of a short range overlap earlier:
// 8.4 us against 9.7 at 517 keys, 16.8 against 18.8 at 57 queries on 20011.
// The whole call measures 7.5 us at 2 requests of 8 heads on 517 keys and 33
// rows, 16.4 at 57 queries to each of 4 heads on 20011 keys, 40 at 128 queries
// to each of 8 heads on 32768 keys and 512 rows (5.0 TB/s, 6.4 between the start
// and the end) and 210 to 219 at 512 queries on 131072 keys and 2048 rows (1.3
// PFLOP/s beside 2.5 TB/s).  Without the rows the products take 2470 cycles for
// 128 keys of a pair, of which the tensor pipe needs 2056, at the 1.57 to 1.75
// GHz that power leaves: 1.58 PFLOP/s for the call.
//
// P is rounded once to bf16 (2^-8 of each probability, which averages out over
// the keys to about the output's own rounding).  A second bf16 term for what
// the rounding left was measured: it lengthens the chain from one block's
// scores to the next, 18.7 -> 20.3 us at 57 queries to a head on 20011 keys
// and 237 -> 284 us at 512 queries on 131072.
//
// The maximum only rises when a block exceeds it by more than 2^8: until then
// P is at most 2^8 too large, which bf16 and the fp32 sums hold as exactly,
// and O needs no rescaling pass through the registers.  The scores' scale is
// applied as |scale| with the queries' sign turned, so that the row maximum
// can be taken before scaling.
//
// TMEM columns: S_0/P_0 0, S_1/P_1 128 (or two buffers of 64 each), O_0 256,
// O_1 384.
//
// Every wait gives up after a second: the CTA's rows become NaN and
// HS_ATTN_STATUS_TIMEOUT is set (hs_attention_status); copies and products in
// flight are waited for, with the same limit, before the CTA leaves.
#include <cmath>
#include <cstdint>

#include <cuda.h>

#include "barriers.cuh"
#include "hs.h"
#include "hs_internal.cuh"
#include "rows_gather.cuh"

namespace hs {
namespace {

constexpr int kDim = 128;
constexpr int kRows = 128;                      // of a tile of queries
constexpr uint32_t kTileBytes = kRows * kDim * 2;   // 32 KB of queries
constexpr uint32_t kAtom = kRows * 128;         // 64 of their 128 dimensions: 16 KB
constexpr uint32_t kRingBytes = 160 << 10;
// keys of a block
__host__ __device__ constexpr int block_keys(bool alone) { return alone ? 64 : 128; }
constexpr int kPrefixThreads = 384;             // three warpgroups; the last warp idles
constexpr float kRise = 8.f;                    // log2 of how far P may exceed 1

constexpr uint32_t kOffQ = 0;                       // two tiles
constexpr uint32_t kOffRing = 2 * kTileBytes;
constexpr uint32_t kOffBar = kOffRing + kRingBytes;
constexpr int kMaxSlots = 10;
// full[kMaxSlots], empty[kMaxSlots], s_full[2][2], p_ready[2][2], q_full, drained
constexpr int kBars = 2 * kMaxSlots + 10;
constexpr uint32_t kOffWord = kOffBar + 8 * kBars;  // TMEM address, abort flag
// with one tile of rows: both groups' (m, l) [2][128]; half of each group's O
// goes to the other through the query tiles' places
constexpr uint32_t kOffXml = kOffWord + 16;
constexpr uint32_t kSmem = kOffXml + 2 * kRows * 8;
static_assert(kSmem <= 232448, "fits an SM");
static_assert(kOffBar % 8 == 0 && kOffXml % 8 == 0, "barriers and (m, l) are 8-byte aligned");
static_assert(64 * kRows * 4 <= kTileBytes, "half of O fits a query tile's place");
static_assert(rows::kSmem <= kSmem, "the row CTAs' rings fit");

__device__ uint32_t g_prefix_status;

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

// fp32 accumulators, bf16 operands, M = 128; bit 16: B is given with
// its N dimension contiguous
constexpr uint32_t kIdesc = 1u << 4 | 1u << 7 | 1u << 10 | 128u >> 4 << 24;
constexpr uint32_t kIdescV = kIdesc | 128u >> 3 << 17 | 1u << 16;  // N = 128

// Products and arrivals are issued by the lane where `on` is not 0, by
// predicate: a branch around them would leave the warp's uniform registers out
// of use, and moving the operands there one by one took about as long as the
// products (60 cycles each; 182 us for 174 at 512 queries to a head on 131072
// keys).
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       bool add, uint32_t on) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %4, 0;\n\t"
        "setp.ne.u32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add), "r"(on)
        : "memory");
}

__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                       bool add, uint32_t on) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %4, 0;\n\t"
        "setp.ne.u32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)add), "r"(on)
        : "memory");
}

// 1 in one lane of a converged warp, the same one every time.
__device__ __forceinline__ uint32_t elect_one() {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xFFFFFFFF;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r));
    return r;
}

// `bar` gets an arrival once every product issued so far by this thread is done
__device__ __forceinline__ void mma_commit(uint32_t bar, uint32_t on) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.u32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(
            bar),
        "r"(on)
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

// 32 bytes to a 32-byte boundary
__device__ __forceinline__ void store32(float *p, const uint32_t *v) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]),
                 "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

__device__ __forceinline__ void st_shared16(uint32_t addr, const uint32_t *v) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v[0]), "r"(v[1]),
                 "r"(v[2]), "r"(v[3])
                 : "memory");
}
__device__ __forceinline__ void ld_shared16(uint32_t addr, uint32_t *v) {
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                 : "r"(addr)
                 : "memory");
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

// kAlone: one tile of rows, whose blocks (of 64 keys, their scores in two
// buffers) go to the two groups in turn; else pairs of tiles (the last one's
// second may be empty) and blocks of 128 keys.
template <bool kAlone>
__global__ void __launch_bounds__(kPrefixThreads, 1)
    prefix_kernel(const __grid_constant__ CUtensorMap map, const GroupArgs a, const PrefixPlan p,
                  const RowsPlan rp) {
    extern __shared__ __align__(1024) uint8_t smem[];  // the swizzle's period
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);  // known to be the same in a warp
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if ((int)blockIdx.x < rp.ctas) {  // (0 without own rows)
        if (warp == 8) rows::init(a, smem);
        __syncthreads();
        if (warp >= 8) {
            asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
            rows::bring(a, rp, blockIdx.x, smem, warp - 8);
        } else {
            asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
            if (warp < a.heads * rp.subs)
                rows::attend<false>(a, rp, blockIdx.x, smem, &g_prefix_status);
        }
        return;
    }
    constexpr int kKeys = block_keys(kAlone);
    constexpr uint32_t kItemBytes = kKeys * kDim * 2;  // keys or values of a block
    constexpr uint32_t kItemAtom = kKeys * 128;        // 64 of their dimensions
    constexpr int kSlots = kRingBytes / kItemBytes;
    constexpr uint32_t kIdescS = kIdesc | (uint32_t)kKeys >> 3 << 17;
    // buffers of scores of a tile, and parts of P whose products are released
    // one by one: a block of 64 keys each, or the halves of one of 128
    constexpr int kBufs = kAlone ? 2 : 1, kParts = kAlone ? 1 : 2;
    static_assert(kSlots <= kMaxSlots && kBufs * kKeys == 128, "ring and TMEM");
    const uint32_t s0 = smem_addr(smem);
    volatile uint32_t *words = reinterpret_cast<volatile uint32_t *>(smem + kOffWord);
    volatile uint32_t *abort_flag = words + 1;
    const uint32_t bars = s0 + kOffBar;
    auto full = [&](int i) { return bars + 8u * i; };
    auto empty = [&](int i) { return bars + 8u * (kMaxSlots + i); };
    // of tile t and scores buffer b; of tile t and buffer or half b
    auto s_full = [&](int t, int b) { return bars + 8u * (2 * kMaxSlots + 2 * t + b); };
    auto p_ready = [&](int t, int b) { return bars + 8u * (2 * kMaxSlots + 4 + 2 * t + b); };
    const uint32_t q_full = bars + 8u * (2 * kMaxSlots + 8), drained = bars + 8u * (2 * kMaxSlots + 9);

    // the CTAs that read the same keys are neighbours
    const int pairs = (p.row_tiles + 1) / 2;
    const int cta = (int)blockIdx.x - rp.ctas;
    const int pair_id = cta % pairs, g = cta / pairs;
    const int group = a.q_heads / a.heads;
    const int n_rows = a.n_req * group;  // at most 65535 * 16
    const int each = p.total / p.groups, rest = p.total % p.groups;
    const int t0 = range_start(g, p.groups, each, rest), t1 = range_start(g + 1, p.groups, each, rest);
    const int head0 = t0 / p.blocks, head1 = (t1 - 1) / p.blocks;
    // blocks [first, first + n) of a head are this group's; n >= 1
    auto first_block = [&](int head) { return max(0, t0 - head * p.blocks); };
    auto count = [&](int head) { return min(p.blocks, t1 - head * p.blocks) - first_block(head); };
    // how many blocks' keys come before the first block's values
    auto ahead_of = [&](int n) { return min(kAlone ? 4 : 1, n); };

    // The ring.  Items come in the order the products use them: for a head, K of
    // the first blocks, then V of block j and K of block j + ahead.  Pairs of
    // tiles both use every item; with one tile each group has a ring of its own
    // for its every other block, so that each ring is waited on in its order.
    constexpr int kRing = kAlone ? kSlots / 2 : kSlots;
    int put[2] = {0, 0};                    // items put into each ring (loading thread)
    auto load = [&](int head, int i) {
        const int n = count(head), ahead = ahead_of(n);
        const int u = i - ahead, both = 2 * (n - ahead);  // both: V, K, V, K, ...; then V only
        const bool is_k = u < 0 || (u < both && (u & 1));
        const int block = u < 0 ? i : u < both ? u / 2 + (u & 1 ? ahead : 0) : u - (n - ahead);
        const int ring = kAlone ? block & 1 : 0, c = ring ? put[1]++ : put[0]++;
        const int slot = ring * kRing + c % kRing;
        if (c >= kRing && !mbar_wait(empty(slot), (c / kRing - 1) & 1, abort_flag)) {
            ring ? --put[1] : --put[0];
            return false;
        }
        const int x = (is_k ? head : a.heads + head) * kDim;
        const int y = (first_block(head) + block) * kKeys;
        const uint32_t dst = s0 + kOffRing + slot * kItemBytes;
        mbar_expect(full(slot), kItemBytes);
        tma_load(dst, &map, x, y, full(slot));
        tma_load(dst + kItemAtom, &map, x + 64, y, full(slot));
        return true;
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
        for (int t = 0; t < 2; ++t)
            for (int b = 0; b < 2; ++b) {
                mbar_init(s_full(t, b), 1);
                mbar_init(p_ready(t, b), kRows);
            }
        mbar_init(q_full, 2 * kRows);
        mbar_init(drained, kAlone ? 2 : 1);
        mbar_init_done();
        // two items before the queries' loads, which the rest would delay
        load(head0, 0);
        load(head0, 1);
    }
    // softmax groups: thread = row (TMEM lane) of tile t
    const int t = (warp >> 2) & 1, row = tid & 127;
    const int m_row = (2 * pair_id + (kAlone ? 0 : t)) * kRows + row;
    const bool live = m_row < n_rows;
    // the queries' sign bits are turned for a negative scale; for scale 0 the
    // queries become 0, so that a masked score stays -inf
    const bool flat = a.scale_log2 == 0.f;
    const float scale = flat ? 1.f : fabsf(a.scale_log2);
    auto load_q = [&](int head) {
        if (kAlone && t == 1) return;
        const uint32_t flip = a.scale_log2 < 0.f ? 0x80008000u : 0u;
        // a warp's 32 rows, two at a time: 16 lanes to a row of 256 bytes
        const int c = lane & 15, at0 = (warp & 3) * 32 + (lane >> 4);
        const int m0 = m_row - row + at0;
        int r = m0 / group, h = m0 - r * group;  // request and head of the group
        uint8_t *dst = smem + kOffQ + t * kTileBytes + (c >> 3) * kAtom;
        const uint8_t *src = a.q + (int64_t)head * group * (2 * kDim) + c * 16;
        uint4 x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            x[i] = make_uint4(0u, 0u, 0u, 0u);
            if (r < a.n_req && !flat)
                x[i] = __ldg(reinterpret_cast<const uint4 *>(src + (int64_t)(r * a.q_heads + h) * (2 * kDim)));
            h += 2;
#pragma unroll
            for (int w = 0; w < 2; ++w)
                if (h >= group) {
                    h -= group;
                    ++r;
                }
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int at = at0 + 2 * i;
            x[i].x ^= flip;
            x[i].y ^= flip;
            x[i].z ^= flip;
            x[i].w ^= flip;
            *reinterpret_cast<uint4 *>(dst + at * 128 + (((c & 7) ^ (at & 7)) << 4)) = x[i];
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    };
    if (warp < 8) load_q(head0);
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = words[0];

    if (warp >= 8) asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (warp == 8) {
        // ---- the rest of the ring's items
        if (lane == 0) {
            bool ok = true;
#pragma unroll 1
            for (int head = head0; head <= head1 && ok; ++head)
#pragma unroll 1
                for (int i = head == head0 ? 2 : 0, n = 2 * count(head); i < n && ok; ++i)
                    ok = load(head, i);
            // nothing may land after the CTA has left the ring (in a normal run
            // the products have waited for all of it)
#pragma unroll 1
            for (int ring = 0; ring < kSlots / kRing; ++ring)
#pragma unroll 1
                for (int c = max(0, put[ring] - kRing); c < put[ring]; ++c)
                    mbar_drain(full(ring * kRing + c % kRing), (c / kRing) & 1);
        }
    } else if (warp == 9 || (kAlone && warp == 10)) {
        // ---- the products: the whole warp waits, one lane issues.  One warp
        // for a pair of tiles; with one tile, one for each group's blocks.
        const int ring = kAlone ? warp - 9 : 0;
        const uint32_t issuer = elect_one();
        const uint64_t q_op = operand(s0 + kOffQ, 16);
        const uint64_t k_op = operand(s0 + kOffRing, 16), v_op = operand(s0 + kOffRing, kItemAtom);
        uint32_t p_phase = 0;               // bit 2 t + b: of p_ready(t, b)
        bool ok = true;
        // the same answer in every lane, which keeps what follows uniform
        auto wait = [&](uint32_t bar, uint32_t parity) {
            return __all_sync(0xFFFFFFFFu, mbar_try(bar, parity)) ||
                   __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity, abort_flag));
        };
        // the ring's items one after the other
        int at = kRing - 1;
        uint32_t round = 1;                 // its parity
        auto next_item = [&]() {
            if (++at == kRing) {
                at = 0;
                round ^= 1;
            }
            const int slot = ring * kRing + at;
            ok = wait(full(slot), round);
            return slot;
        };
        auto release = [&](int slot) {
            mma_commit(empty(slot), issuer);
        };
        // S_t = Q_t K^T into buffer b, 16 dimensions at a time
        auto scores = [&](int tile, int b, int slot) {
            const uint64_t q = q_op + (kAlone ? 0 : tile * (kTileBytes >> 4));
            const uint64_t k = k_op + slot * (kItemBytes >> 4);
#pragma unroll
            for (int c = 0; c < 8; ++c)
                mma_ss(tmem + tile * 128 + b * kKeys, q + (((c >> 2) * kAtom + (c & 3) * 32) >> 4),
                       k + (((c >> 2) * kItemAtom + (c & 3) * 32) >> 4), kIdescS, c > 0, issuer);
        };
        auto signal = [&](int tile, int b) {
            mma_commit(s_full(tile, b), issuer);
        };
        // O_t += P_t V, 16 keys at a time, each part of P as it is ready
        auto outputs = [&](int tile, int b, int slot, bool first) {
            const uint64_t v = v_op + slot * (kItemBytes >> 4);
            const uint32_t pt = tmem + tile * 128 + b * kKeys, d = tmem + 256 + tile * 128;
#pragma unroll
            for (int part = 0; part < kParts; ++part) {
                const int bar = 2 * tile + b + part;
                if (!(ok = wait(p_ready(tile, b + part), p_phase >> bar & 1u))) return false;
                p_phase ^= 1u << bar;
                fence_after();
#pragma unroll
                for (int c = 4 * part; c < 4 * part + 4; ++c)
                    mma_ts(d, pt + c * 8, v + c * (2048 >> 4), kIdescV, c > 0 || !first, issuer);
            }
            return true;
        };
#pragma unroll 1
        for (int head = head0; head <= head1 && ok; ++head) {
            const int n = count(head);
            ok = wait(q_full, (head - head0) & 1);
            fence_after();
            if constexpr (kAlone) {
                // this group's blocks: every other.  The first scores into both
                // buffers
                int b = 0;
#pragma unroll 1
                for (int j = ring; j < min(n, 4); j += 2, ++b) {
                    const int k = next_item();
                    if (!ok) break;
                    scores(ring, b, k);
                    signal(ring, b);
                    release(k);
                }
                // (no block: the softmax group waits for one arrival all the same, so
                // that it cannot get two heads ahead of this warp)
                if (ring >= n) signal(ring, 0);
                // then O += P V of a block, and into the buffer that held its scores
                // those of the group's block after next
                b = 0;
#pragma unroll 1
                for (int j = ring; j < n && ok; j += 2, b ^= 1) {
                    const int v = next_item();
                    if (!ok || !outputs(ring, b, v, j < 2)) break;
                    release(v);
                    if (j + 4 < n) {
                        const int k = next_item();
                        if (!ok) break;
                        scores(ring, b, k);
                        signal(ring, b);
                        release(k);
                    } else {
                        signal(ring, b);
                    }
                }
            } else {
                // the first scores of both tiles; then the tiles in turn: O_t += P_t V
                // of a block and S_t of the next
                int k = next_item();
#pragma unroll 1
                for (int tile = 0; tile < 2 && ok; ++tile) {
                    scores(tile, 0, k);
                    signal(tile, 0);
                    if (tile == 1) release(k);
                }
#pragma unroll 1
                for (int j = 0; j < n && ok; ++j) {
                    const int v = next_item();
#pragma unroll 1
                    for (int tile = 0; tile < 2 && ok; ++tile) {
                        if (!outputs(tile, 0, v, j == 0)) break;
                        if (tile == 1) release(v);
                        if (j + 1 < n) {
                            if (tile == 0) k = next_item();
                            if (!ok) break;
                            scores(tile, 0, k);
                            if (tile == 1) release(k);
                        }
                        signal(tile, 0);
                    }
                }
            }
        }
        // no product may still run when the TMEM is given back
        mma_commit(drained, issuer);
        mbar_drain(drained, 0);
    } else if (warp < 8) {
        // ---- softmax
        asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
        const uint32_t lanes = (uint32_t)(warp & 3) * 32 << 16;
        const uint32_t ts = tmem + lanes + t * 128, to = tmem + lanes + 256 + t * 128;
        const int first = kAlone ? t : 0, step = kAlone ? 2 : 1;  // of the head's blocks
        uint32_t s_phase = 0;
        bool ok = true;
        for (int head = head0; head <= head1; ++head) {
            if (head > head0) load_q(head);
            mbar_arrive(q_full);
            const int n = count(head), b0 = first_block(head);
            const int mine = n > first ? (n - first + step - 1) / step : 0;
            float m = -INFINITY, l = 0.f;
            bool far = false;               // a maximum of the warp is past 2^24
#pragma unroll 1
            for (int j = 0; j < mine && ok; ++j) {
                const int buf = j & (kBufs - 1);
                ok = mbar_wait(s_full(t, buf), s_phase >> buf & 1u, abort_flag);
                if (!__all_sync(0xFFFFFFFFu, ok)) {
                    ok = false;
                    break;
                }
                s_phase ^= 1u << buf;
                fence_after();
                const uint32_t tb = ts + buf * kKeys;
                const int64_t left = a.prefix_len - (int64_t)(b0 + first + j * step) * kKeys;
                uint32_t s[kKeys];
                float x[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                tmem_ld32(tb, s);
#pragma unroll
                for (int c = 0; c < kKeys / 32; ++c) {
                    tmem_wait_ld<32>(s + c * 32);
                    if (c + 1 < kKeys / 32) tmem_ld32(tb + (c + 1) * 32, s + (c + 1) * 32);
                    if (left < kKeys) {
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
                    far = __any_sync(0xFFFFFFFFu, m > -INFINITY && fabsf(m) > 0x1p24f);
                    l *= f;
                    if (j > 0) {
                        // the products on O so far are done: these scores came
                        // behind them, or with two buffers those are that the
                        // other one gets next (waited for again in their turn)
                        if (kBufs == 2) {
                            ok = mbar_wait(s_full(t, 1 - buf), s_phase >> (1 - buf) & 1u, abort_flag);
                            if (!__all_sync(0xFFFFFFFFu, ok)) {
                                ok = false;
                                break;
                            }
                            fence_after();
                        }
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
                uint64_t scale2 = pair(__float_as_uint(scale), __float_as_uint(scale));
                uint64_t shift2 = pair(__float_as_uint(shift), __float_as_uint(shift));
                // The maximum is rounded, the fused products below are not: what that
                // rounding left, up to 1 here, is a power of two that P and l share, but
                // from 2^31 on it would pass fp32's range.  There the scores are rounded
                // as the maximum was.
                if (far) {
#pragma unroll
                    for (int e = 0; e < kKeys; ++e)
                        s[e] = __float_as_uint(
                            __fadd_rn(__fmul_rn(__uint_as_float(s[e]), scale), shift));
                    scale2 = 0x3F8000003F800000ull;  // (1, 1)
                    shift2 = 0ull;
                }
                uint64_t sum[2] = {0ull, 0ull};
#pragma unroll
                for (int c = 0; c < kKeys / 32; ++c) {
                    uint32_t pk[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const uint64_t y =
                            fma2(pair(s[c * 32 + 2 * e], s[c * 32 + 2 * e + 1]), scale2, shift2);
                        const float p0 = ex2(__uint_as_float((uint32_t)y));
                        const float p1 = ex2(__uint_as_float((uint32_t)(y >> 32)));
                        sum[e & 1] = add2(sum[e & 1], pair(__float_as_uint(p0), __float_as_uint(p1)));
                        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(pk[e]) : "f"(p1), "f"(p0));
                    }
                    tmem_st16(tb + c * 16, pk);
                    if (c & 1) {
                        tmem_wait_st();
                        fence_before();
                        mbar_arrive(p_ready(t, kAlone ? buf : c >> 1));
                    }
                }
                sum[0] = add2(sum[0], sum[1]);
                l += __uint_as_float((uint32_t)sum[0]) + __uint_as_float((uint32_t)(sum[0] >> 32));
            }
            // every product on O done: the last arrival of each buffer that was used
#pragma unroll 1
            for (int buf = 0; buf < max(1, min(mine, kBufs)) && ok; ++buf) {
                ok = mbar_wait(s_full(t, buf), s_phase >> buf & 1u, abort_flag);
                s_phase ^= 1u << buf;
                fence_after();
            }
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok && lane == 0) atomicOr(&g_prefix_status, HS_ATTN_STATUS_TIMEOUT);
            if (!ok) m = __int_as_float(0x7FC00000);  // the merge makes such rows NaN

            // the part of (group, head): rows of 512 bytes, one to a thread
            const int64_t part = (int64_t)(g + head) * n_rows + m_row;
            float *dst = p.o + part * kDim;
            asm volatile("" : "+l"(dst));  // computed here, not ahead of the loop over heads
            if (!kAlone || n == 1) {  // (one block: group 0's)
#pragma unroll 1
                for (int c = 0; c < 4 && mine > 0; ++c) {
                    uint32_t o[32];
                    tmem_ld32(to + c * 32, o);
                    tmem_wait_ld<32>(o);
                    if (live)
#pragma unroll
                        for (int e = 0; e < 4; ++e) store32(dst + c * 32 + e * 8, o + e * 8);
                }
            } else {
                // one tile: group t joins both groups' columns [64 t, 64 t + 64)
                // and hands the others over
                uint32_t give = s0 + kOffQ + (1 - t) * kTileBytes + row * 16;
                uint32_t take = s0 + kOffQ + t * kTileBytes + row * 16;
                asm volatile("" : "+r"(give), "+r"(take));  // as dst
                float2 *xml = reinterpret_cast<float2 *>(smem + kOffXml);
                xml[t * kRows + row] = make_float2(m, l);
                // both groups' products are done: the queries are not read any more
                asm volatile("bar.sync 1, 256;" ::: "memory");
#pragma unroll 1
                for (int c = 0; c < 2; ++c) {
                    uint32_t o[32];
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = 0u;
                    if (mine > 0) {
                        tmem_ld32(to + (1 - t) * 64 + c * 32, o);
                        tmem_wait_ld<32>(o);
                    }
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        st_shared16(give, o + 4 * e);
                        give += kRows * 16;
                    }
                }
                asm volatile("bar.sync 1, 256;" ::: "memory");
                const float2 ml = xml[(1 - t) * kRows + row];
                const float M = m != m ? m : ml.x != ml.x ? ml.x : fmaxf(m, ml.x);
                const float base = M == -INFINITY ? 0.f : M;
                const float f1 = ex2(m - base), f2 = ex2(ml.x - base);
                l = l * f1 + ml.y * f2;
                m = M;
#pragma unroll 1
                for (int c = 0; c < 2; ++c) {
                    uint32_t o[32];
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = 0u;
                    if (mine > 0) {
                        tmem_ld32(to + t * 64 + c * 32, o);
                        tmem_wait_ld<32>(o);
                    }
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        uint32_t v[4];
                        ld_shared16(take, v);
                        take += kRows * 16;
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            o[4 * e + i] = __float_as_uint(__uint_as_float(o[4 * e + i]) * f1 +
                                                           __uint_as_float(v[i]) * f2);
                    }
                    if (live)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            store32(dst + t * 64 + c * 32 + e * 8, o + e * 8);
                }
                // the next head's queries go where this one's columns were taken from
                if (head < head1) asm volatile("bar.sync 1, 256;" ::: "memory");
            }
            if ((!kAlone || t == 0) && live) p.ml[part] = make_float2(m, l);
            fence_before();  // the next head's products write over S and O
        }
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

// The prefix over at most `ctas` CTAs: as many groups of a CTA for every pair
// of row tiles as fit (more CTAs than SMs run one behind the other), each at
// two blocks or more unless the prefix is short.  A multiple of the heads
// where the longer ranges cost less than another start and end: no range then
// reaches into a second head.
PrefixPlan prefix_plan(int n_req, int q_heads, int heads, int64_t prefix_len, int ctas) {
    PrefixPlan p = {};
    if (prefix_len < 1) return p;
    const int64_t rows = (int64_t)n_req * (q_heads / heads);
    p.row_tiles = (int)((rows + kRows - 1) / kRows);
    const int keys = block_keys(p.row_tiles == 1);
    p.blocks = (int)((prefix_len + keys - 1) / keys);
    p.total = heads * p.blocks;  // at most 2^28
    const int pairs = (p.row_tiles + 1) / 2;
    // A range of two blocks has one for each softmax group.  Ranges of one need
    // no join of the groups, but are twice as many parts to merge: as long as
    // those are what a few warps load at once (517 keys: 8.2 -> 7.5 us, 600 of
    // pairs 13.8 -> 13.2; but 4000 keys 9.9 -> 10.4, 1100 of pairs 14.6 -> 15.2).
    const int one_each = heads * p.blocks;
    const bool single = one_each <= ctas / pairs && p.blocks <= (p.row_tiles == 1 ? 16 : 8);
    const int most = single ? one_each : heads * ((p.blocks + 1) / 2);
    // measured: a CTA's start and end at a head, and 128 keys of a pair of tiles,
    // or of one (bound by HBM).  With the whole multiple where it pays: 48.1 ->
    // 43.5 us at 128 queries to each of 8 heads on 32768 keys, 104 groups instead
    // of 109.
    const float block = (p.row_tiles == 1 ? 3000.f : 2500.f) / 128 * keys;
    auto cycles = [&](int groups) {
        const int longest = (p.total + groups - 1) / groups;
        const int heads_more = groups % heads == 0 ? 0 : (longest - 1) / p.blocks + 1;
        return 13000.f * (1 + heads_more) + block * longest;
    };
    p.groups = ctas / pairs;
    if (p.groups > most) p.groups = most;
    if (p.groups < 1) p.groups = 1;
    p.cycles = cycles(p.groups);
    const int whole = p.groups / heads * heads;
    if (whole > 0 && cycles(whole) <= p.cycles) {
        p.groups = whole;
        p.cycles = cycles(whole);
    }
    p.lead = (p.groups - 1) / p.blocks;
    return p;
}

cudaError_t launch_prefix(const GroupArgs &a, const PrefixPlan &p, const RowsPlan &rows,
                          cudaStream_t st) {
    const EncodeTiled encode = encode_tiled();
    if (!encode) return cudaErrorNotSupported;
    CUtensorMap map;
    const cuuint64_t dims[2] = {(cuuint64_t)a.heads * 2 * kDim, (cuuint64_t)a.prefix_len};
    const cuuint64_t strides[1] = {(cuuint64_t)a.heads * 4 * kDim};
    const cuuint32_t box[2] = {64, (cuuint32_t)block_keys(p.row_tiles == 1)}, one[2] = {1, 1};
    if (encode(&map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<uint8_t *>(a.prefix), dims,
               strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return cudaErrorInvalidValue;
    const auto kernel = p.row_tiles == 1 ? prefix_kernel<true> : prefix_kernel<false>;
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
    if (e != cudaSuccess) return e;
    const int pairs = (p.row_tiles + 1) / 2;
    kernel<<<(unsigned)(rows.ctas + p.groups * pairs), kPrefixThreads, kSmem, st>>>(map, a, p, rows);
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
