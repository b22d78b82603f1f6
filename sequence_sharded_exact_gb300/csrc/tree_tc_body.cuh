// tree_tc_body.cuh -- tensor-core path of the attention over a cache (tree.cuh) for bf16 queries and a bf16
// or e4m3 cache, head dim RA_TREE_HD (128 or 64).  Compiled once per head dim (tree_tc.cu: 128,
// tree_tc_d64.cu: 64), and again through a window (RA_TREE_WINDOW 1: tree_window_tc.cu, tree_window_tc_d64.cu); the
// including file names the host entry point through RA_TREE_LAUNCH.
//
// One CTA per SM walks its items (tree.cuh): one kv head's tile of query rows against its cached rows, 128
// at a time.  For query rows X and cached rows K, V of a tile:
//   S = X K^T (TMEM), P = 2^(S c - m) (bf16, over S's columns), O += P V (TMEM), the running m, l per row.
// A weight goes into P V as two bf16 values (kExact), off by 2^-15 of itself, where the memory bounds the kernel, which
// hardly feels it (a bf16 cache, up to 128 query rows: 1.49 us per tile in place of 1.44), and where the output is
// float32: the output before rounding, or a part that others are to be folded into.  Otherwise as one, off by up to 2^-8 of
// itself: the output's relative error is then 0.0023, where its own rounding to bf16 makes 0.0017.  Two would take ragged e4m3
// caches from 131 to 140 us and 256 query rows from 72 to 80.
// A query row is a TMEM lane and a thread, so its maximum and sum need no exchange between threads.
//   * Up to 128 query rows (kNq = 1): the two softmax warpgroups take turns at the tiles, each with its own
//     m, l and O, so that one tile's exponentials run beside the other's products; they join the two at the
//     item's end (both read both O's: a warp of either group reaches the same TMEM lanes), half the
//     columns each.
//   * More (kNq = 2): 256 query rows as two 128-row tiles that share every K/V tile, a warpgroup each.
//   * m follows the row maximum only when that grows by more than 2^8: O / l does not depend on the
//     reference, O in TMEM is then seldom rescaled, and S is read once.
//   * Warps: 0-3 and 4-7 softmax; 8 loads the queries and K, 10 V (TMA, one thread each); 9 issues the MMAs; 11
//     fetches the rows' scales (e4m3); 12-15 prepare V.
// Rows that must not count: scores of unseen rows are set to -infinity before the maximum, but 0 * NaN in
// P V would still be NaN, so warps 12-15 clear the rows of V behind the sequence, and non-finite elements
// of drafted tokens' rows, in shared memory before the product; those elements are added afterwards to
// the rows that do see them (rare, from global memory).
// e4m3: K goes into the products as it is cached.  The queries are split into two 8-bit parts, x 2^-e = hi + lo with
// a power-of-two scale per row that brings its largest element to 224 or more: hi in e4m3 takes four significant bits, lo
// in e5m2 the other four of a bf16, exactly (they are at most 8 units of its last place), down to elements of 2^-6, 2^-13 of
// the row's largest; what is smaller is off by at most 2^-14, 2^-21 of the largest (lo in e4m3, whose steps end at 2^-9,
// was exact down to 2^-2 and off by up to 2^-10).  So S is two 8-bit products at twice the rate, with float32
// sums.  The row and column scales are applied to
// S.  P keeps bf16 (an e4m3 P would lose weights below 2^-9 of the largest, which add up over a long
// cache), so warps 12-15 turn V into bf16, exactly, scale included.
//
// What bounds it, per tile of 128 cached rows on each of 152 SMs, d = 128 (launches apart):
//   * bf16, up to 128 query rows: 1.43 to 1.47 us for 64 KB, 6.8 to 7.0 TB/s: the memory.  (Up to 8 rows take
//     tree_mma_bf16.cu.)
//   * bf16, 256 rows: 1.80 us.  The products take 1.06 of them; S, the softmax and P V of a warpgroup's query rows follow
//     one another on one S, whose columns P takes (at d = 128 TMEM is full: two S, two O; at d = 64 half of O's is free,
//     and kept so).
//   * e4m3, up to 128 rows: 1.57 to 1.63 us for 32 KB.  Shared memory serves 1600 of some 2800 cycles at 128 bytes each:
//     copies 256, S 512 (hi and lo), V to bf16 450, P V 256, scales 130; the rest is the same chain.  Up to 16 rows
//     take tree_mma.cu (0.95 us up to 8).  256 rows: 2.7 us.
// The sum of the weights as they are rounded, for one bf16 value each, takes 0.12 us of a tile's (an uncorrected sum shifts
// a row whose keys share a weight by up to 2^-8).
// What did not help: S in halves of 64 columns, two per warpgroup (256 rows: 2.29 us: twice the issue and waits);
// warpgroups that take half of each tile's keys (e4m3 1.58); V's e4m3 to bf16 by moving bits (its instructions are not
// what takes the time); loading a whole row of V ahead; the e4m3 queries split by warps 12-15 (later at the start, no
// earlier at an item's end); one thread of a diverged warp issuing (256 rows 1.90 in place of 1.67 us: descriptors then
// are not uniform registers).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cudaTypedefs.h>
#include <math.h>

#include <mutex>

#include "ra_internal.h"
#include "ra_ptx.cuh"
#include "tree.cuh"

namespace ra {
namespace {

constexpr int kHd = RA_TREE_HD;
static_assert(kHd == 128 || kHd == 64, "head dim");
constexpr bool kWin = RA_TREE_WINDOW;
using Walk = TreeWalkOf<kWin>;
using Seq = TreeSeqOf<kWin>::type;
constexpr int kThreads = 512;
constexpr uint32_t kTmemCols = 512, kColS = 0, kColO = 256;  // S_w at 128 w, O_w at 256 + 128 w
constexpr long long kWaitLimit = 10000000000ll;

template <bool kE4, int kNq>
struct Cfg {
    static constexpr int kSlotsK = kE4 ? (kNq == 1 ? 4 : 3) : (kNq == 1 ? 3 : 2);
    static constexpr int kSlotsL = kE4 ? (kNq == 1 ? 3 : 2) : 2;  // V as loaded
    static constexpr int kSlotsP = 2;                             // V as prepared (e4m3; bf16 is prepared in place)
    static_assert(kE4 || kSlotsP == kSlotsL, "bf16: a barrier per slot in place");
    static constexpr int kSlotsX = kE4 ? 8 : 1;                   // rows' scales
    static constexpr uint32_t kBytesK = 128 * kHd * (kE4 ? 1 : 2);
    static constexpr uint32_t kBytesV = 128 * kHd * 2;
    static constexpr uint32_t kBytesQ = 128 * kHd * 2;  // of one 128-row tile: bf16, or the hi and lo halves

    static constexpr uint32_t kQ = 0;
    static constexpr uint32_t kK = kQ + kNq * kBytesQ;
    static constexpr uint32_t kL = kK + kSlotsK * kBytesK;  // slots of kBytesK: V is loaded in the cache's type
    static constexpr uint32_t kP = kL + kSlotsL * kBytesK;
    static constexpr uint32_t kX = kP + (kE4 ? kSlotsP * kBytesV : 0);  // [slots][2][128] float
    static constexpr uint32_t kMl = kX + (kE4 ? kSlotsX * 1024 : 0);    // [2][128] float4 (kNq == 1)
    static constexpr uint32_t kQs = kMl + (kNq == 1 ? 4096 : 0);        // [2][kNq * 128] float (e4m3)
    static constexpr uint32_t kPoison = kQs + (kE4 ? 2 * kNq * 512 : 0);  // [8] int
    static constexpr uint32_t kBar = kPoison + 32;

    static constexpr int bQFull = 0, bQEmpty = 1, bS = 2, bP = 4, bO = 6, bEpi = 8, bDrain = 10;
    static constexpr int bKFull = 11, bKEmpty = bKFull + kSlotsK;
    static constexpr int bLFull = bKEmpty + kSlotsK, bLEmpty = bLFull + kSlotsL;
    static constexpr int bPFull = bLEmpty + kSlotsL, bPEmpty = bPFull + kSlotsP;
    static constexpr int bXFull = bPEmpty + kSlotsP, bXEmpty = bXFull + kSlotsX;
    static constexpr int kBars = bXEmpty + kSlotsX;

    static constexpr uint32_t kSlot = kBar + kBars * 8;
    static constexpr uint32_t kAbort = kSlot + 8;
    static constexpr uint32_t kSmem = kAbort + 8 + 1024;  // slack for the 1024-byte alignment of the base
    static_assert(kSmem <= 232448, "shared memory");
};

struct Maps {
    CUtensorMap q, k, v;
};

// A bounded wait, short enough to be inlined at every use: the loops of the roles run side by side and have to
// stay in the instruction cache together.  Gives up after kWaitLimit cycles (over 4 s at the highest clock), or
// when another warp has.
__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, const WaitCtl& ctl)
{
    if (mbar_try_wait(bar, parity)) return true;
    const long long t0 = clock64();
    while (!mbar_try_wait(bar, parity)) {
        if (*ctl.abort) return false;
        if (clock64() - t0 > kWaitLimit) {
            *ctl.abort = 1;
            atomicOr(ctl.status, kStatusTimeout);
            return false;
        }
    }
    return true;
}
// The whole warp's: every lane learns whether all of them saw the phase.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, const WaitCtl& ctl)
{
    return __all_sync(0xffffffffu, wait(bar, parity, ctl));
}

__device__ __forceinline__ void drain_wait(uint32_t bar, uint32_t parity)
{
    const uint64_t t0 = global_timer_ns();
    while (!mbar_try_wait(bar, parity)) {
        if (global_timer_ns() - t0 > 1000000000ull) return;
    }
}

// A place in a ring of kSlots slots and the parity of its use: full barriers are waited for with `par`, empty ones
// (which the first round finds free) with `par ^ 1`.
template <int kSlots>
struct Ring {
    int slot = 0;
    uint32_t par = 0, round = 0;
    __device__ __forceinline__ void next()
    {
        if (++slot == kSlots) {
            slot = 0;
            par ^= 1;
            round = 1;
        }
    }
};

// Shared-memory descriptors.  K-major operands of bf16 and of 128-column e4m3 have 128-byte rows and that
// swizzle; 64-column e4m3 rows are 64 bytes with the 64-byte swizzle (layout 4, 8-row groups of 512 bytes).
template <bool kE4>
constexpr bool kNarrow = kE4 && kHd == 64;
template <bool kE4>
__host__ __device__ constexpr uint32_t kmajor_hi()
{
    return kNarrow<kE4> ? (((512u >> 4) & 0x3FFFu) | (1u << 14) | (4u << 29)) : sdesc_sw128_hi(1024);
}

// The issuing warp runs as a whole, so that descriptors and addresses are the same in every lane and stay in uniform
// registers; one elected lane (`lead`) issues.
__device__ __forceinline__ uint32_t elect()
{
    uint32_t e;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
    return e;
}
__device__ __forceinline__ void lead_mma_ss(uint32_t lead, uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p, l;\n\t"
        "setp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 l, %5, 0;\n\t"
        "@l tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(lead)
        : "memory");
}
__device__ __forceinline__ void lead_mma_ts(uint32_t lead, uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p, l;\n\t"
        "setp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 l, %5, 0;\n\t"
        "@l tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(lead)
        : "memory");
}
__device__ __forceinline__ void lead_commit(uint32_t lead, uint32_t bar)
{
    asm volatile(
        "{\n\t.reg .pred l;\n\tsetp.ne.b32 l, %1, 0;\n\t"
        "@l tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar), "r"(lead)
        : "memory");
}

// kind::f8f6f4 (f32 accumulate): B in e4m3 (format 0), A in e4m3 or e5m2 (format 1); the other fields as kind::f16's.
__host__ __device__ constexpr uint32_t idesc_8bit_f32(int M, int N, bool a_e5m2)
{
    return (1u << 4) | (a_e5m2 ? 1u << 7 : 0u) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
__device__ __forceinline__ void lead_mma_ss_8bit(uint32_t lead, uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                                 uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p, l;\n\t"
        "setp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 l, %5, 0;\n\t"
        "@l tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(lead)
        : "memory");
}

// S_w = X K^T.
template <bool kE4, int kNq>
__device__ __forceinline__ void issue_s(uint32_t lead, uint32_t sbase, uint32_t tmem, int w, int slot)
{
    using C = Cfg<kE4, kNq>;
    const uint32_t q = sdesc_sw128_lo(sbase + C::kQ + (kNq == 2 ? (uint32_t)w * C::kBytesQ : 0u), 16);
    const uint32_t k = sdesc_sw128_lo(sbase + C::kK + (uint32_t)slot * C::kBytesK, 16);
    const uint32_t d = tmem + kColS + (uint32_t)w * 128;
    constexpr uint32_t hi = kmajor_hi<kE4>();
    if constexpr (kE4) {
#pragma unroll
        for (int part = 0; part < 2; ++part)
#pragma unroll
            for (int kk = 0; kk < kHd / 32; ++kk)
                lead_mma_ss_8bit(lead, d, sdesc_at(q, (uint32_t)part * 128 * kHd + (uint32_t)kk * 32, hi), sdesc_at(k, (uint32_t)kk * 32, hi),
                            idesc_8bit_f32(128, 128, part == 1), part + kk > 0 ? 1u : 0u);
    } else {
#pragma unroll
        for (int kk = 0; kk < kHd / 16; ++kk) {
            const uint32_t off = (uint32_t)(kk >> 2) * 16384u + (uint32_t)(kk & 3) * 32u;
            lead_mma_ss(lead, d, sdesc_at(q, off, hi), sdesc_at(k, off, hi), idesc_bf16_f32(128, 128, false, false), kk > 0 ? 1u : 0u);
        }
    }
}

// O_w (+)= P_w V.  (kExact: of each 32 keys' columns of S the first 16 hold P's upper parts, the others what is left.)
template <bool kExact>
__device__ __forceinline__ void issue_pv(uint32_t lead, uint32_t v_addr, uint32_t tmem, int w, bool accumulate)
{
    const uint32_t v = sdesc_sw128_lo(v_addr, 16384);
    constexpr uint32_t hi = sdesc_sw128_hi(1024);
#pragma unroll
    for (int kk = 0; kk < 8; ++kk)
#pragma unroll
        for (int part = 0; part < (kExact ? 2 : 1); ++part)
            lead_mma_ts(lead, tmem + kColO + (uint32_t)w * 128,
                        tmem + kColS + (uint32_t)w * 128 + (uint32_t)(kExact ? (kk >> 1) * 32 + part * 16 + (kk & 1) * 8 : kk * 8),
                        sdesc_at(v, (uint32_t)kk * 2048u, hi), idesc_bf16_f32(128, kHd, false, true), part + kk > 0 || accumulate ? 1u : 0u);
}

// ------------------------------------------------------------------------------------------------
// loads
// ------------------------------------------------------------------------------------------------
template <bool kE4, int kNq>
__device__ __forceinline__ void load_qk_role(const TreeArgs& a, uint32_t sbase, const Maps& maps, Walk w, const WaitCtl& ctl)
{
    using C = Cfg<kE4, kNq>;
    auto bar = [&](int i) { return sbase + C::kBar + 8u * (uint32_t)i; };
    uint32_t kc = 0, item = 0;
    bool ok = true;
    do {
        if (w.goes_on()) a.border[blockIdx.x] = w.border(a, blockIdx.x);
        const int z = w.b * a.Hkv + w.g;
        if constexpr (!kE4) {
            if (item > 0 && !wait(bar(C::bQEmpty), (item - 1) & 1, ctl)) break;
            mbar_arrive_expect_tx(bar(C::bQFull), kNq * C::kBytesQ);
            for (int t = 0; t < kNq; ++t)
                for (int h = 0; h < kHd / 64; ++h)
                    tma_load_3d(sbase + C::kQ + (uint32_t)t * C::kBytesQ + (uint32_t)h * 16384u, &maps.q, bar(C::bQFull), h * 64,
                                w.r * a.rt + t * 128, z);
            ++item;
        }
        for (int t = w.t0; t < w.t1; ++t, ++kc) {
            const int slot = (int)(kc % C::kSlotsK);
            const uint32_t use = kc / C::kSlotsK;
            if (use > 0 && !wait(bar(C::bKEmpty + slot), (use - 1) & 1, ctl)) { ok = false; break; }
            mbar_arrive_expect_tx(bar(C::bKFull + slot), C::kBytesK);
            const uint32_t dst = sbase + C::kK + (uint32_t)slot * C::kBytesK;
            if constexpr (kE4) {
                tma_load_3d(dst, &maps.k, bar(C::bKFull + slot), 0, tree_row(w.s, t * kTreeTile, kTreeTile), z);
            } else {
                for (int h = 0; h < kHd / 64; ++h)
                    tma_load_3d(dst + (uint32_t)h * 16384u, &maps.k, bar(C::bKFull + slot), h * 64, tree_row(w.s, t * kTreeTile, kTreeTile), z);
            }
        }
    } while (ok && w.next(a));
    if (item > 0) drain_wait(bar(C::bQFull), (item - 1) & 1);
    for (uint32_t s = 0; s < (uint32_t)C::kSlotsK && s < kc; ++s)
        drain_wait(bar(C::bKFull + (int)((kc - 1 - s) % C::kSlotsK)), ((kc - 1 - s) / C::kSlotsK) & 1);
}

template <bool kE4, int kNq>
__device__ __forceinline__ void load_v_role(const TreeArgs& a, uint32_t sbase, const Maps& maps, Walk w, const WaitCtl& ctl)
{
    using C = Cfg<kE4, kNq>;
    auto bar = [&](int i) { return sbase + C::kBar + 8u * (uint32_t)i; };
    uint32_t vc = 0;
    bool ok = true;
    do {
        const int z = w.b * a.Hkv + w.g;
        for (int t = w.t0; t < w.t1; ++t, ++vc) {
            const int slot = (int)(vc % C::kSlotsL);
            const uint32_t use = vc / C::kSlotsL;
            if (use > 0 && !wait(bar(C::bLEmpty + slot), (use - 1) & 1, ctl)) { ok = false; break; }
            const uint32_t dst = sbase + C::kL + (uint32_t)slot * C::kBytesK;
            if constexpr (kE4) {
                // rows are contiguous and V is not a product's operand here: one untiled copy, no row past the cache
                const int row0 = tree_row(w.s, t * kTreeTile, kTreeTile), rows = a.cap - row0 < kTreeTile ? a.cap - row0 : kTreeTile;
                mbar_arrive_expect_tx(bar(C::bLFull + slot), (uint32_t)rows * kHd);
                bulk_load_1d(dst, static_cast<const uint8_t*>(a.v) + ((long long)z * a.cap + row0) * kHd,
                             (uint32_t)rows * kHd, bar(C::bLFull + slot));
            } else {
                mbar_arrive_expect_tx(bar(C::bLFull + slot), C::kBytesK);
                for (int h = 0; h < kHd / 64; ++h)
                    tma_load_3d(dst + (uint32_t)h * 16384u, &maps.v, bar(C::bLFull + slot), h * 64, tree_row(w.s, t * kTreeTile, kTreeTile), z);
            }
        }
    } while (ok && w.next(a));
    for (uint32_t s = 0; s < (uint32_t)C::kSlotsL && s < vc; ++s)
        drain_wait(bar(C::bLFull + (int)((vc - 1 - s) % C::kSlotsL)), ((vc - 1 - s) / C::kSlotsL) & 1);
}

// The scales of a tile's rows, 2^e as float32, k's then v's; four tiles' bytes are in flight at a time.
template <int kNq>
__device__ __forceinline__ void scale_role(const TreeArgs& a, uint32_t sbase, uint8_t* smem, Walk w, const WaitCtl& ctl)
{
    using C = Cfg<true, kNq>;
    auto bar = [&](int i) { return sbase + C::kBar + 8u * (uint32_t)i; };
    const int lane = threadIdx.x & 31;
    uint32_t xc = 0;
    do {
        const long long row0 = ((long long)w.b * a.Hkv + w.g) * a.cap;
        for (int t = w.t0; t < w.t1;) {
            const int n = w.t1 - t < 4 ? w.t1 - t : 4;
            uint32_t raw[4][4];  // k's byte in bits 0-7, v's in 8-15
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int row = tree_row(w.s, (t + u) * kTreeTile, kTreeTile) + i * 32 + lane;
                    raw[u][i] = 0;
                    if (u < n && row < w.s.end)
                        raw[u][i] = (uint32_t)a.k_exp[row0 + row] | (uint32_t)a.v_exp[row0 + row] << 8;
                }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                if (u >= n) break;
                const int slot = (int)(xc % C::kSlotsX);
                const uint32_t use = xc / C::kSlotsX;
                if (use > 0 && !warp_wait(bar(C::bXEmpty + slot), (use - 1) & 1, ctl)) return;
                float* x = reinterpret_cast<float*>(smem + C::kX + slot * 1024);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[i * 32 + lane] = __uint_as_float((raw[u][i] & 0xffu) << 23);
                    x[128 + i * 32 + lane] = __uint_as_float((raw[u][i] >> 8) << 23);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(C::bXFull + slot));
                ++xc;
            }
            t += n;
        }
    } while (w.next(a));
}

// ------------------------------------------------------------------------------------------------
// V (and, for e4m3, the queries) as the products take them
// ------------------------------------------------------------------------------------------------
// Clears the non-finite halves of a packed bf16 pair; true if there was one.
__device__ __forceinline__ bool clear_nonfinite(uint32_t& w)
{
    bool hit = false;
    if ((w & 0x7f80u) == 0x7f80u) {
        w &= 0xffff0000u;
        hit = true;
    }
    if ((w & 0x7f800000u) == 0x7f800000u) {
        w &= 0x0000ffffu;
        hit = true;
    }
    return hit;
}

// bf16: only the tiles that reach past the prefix are touched, in place; the others are passed on (a warp that
// skipped a tile's phase could take the slot's previous phase for the one it waits for).
template <int kNq>
__device__ __forceinline__ void prep_bf16_role(const TreeArgs& a, uint32_t sbase, uint8_t* smem, Walk w, const WaitCtl& ctl)
{
    using C = Cfg<false, kNq>;
    auto bar = [&](int i) { return sbase + C::kBar + 8u * (uint32_t)i; };
    const int row = threadIdx.x & 127;
    uint32_t vc = 0, item = 0;
    do {
        for (int t = w.t0; t < w.t1; ++t, ++vc) {
            const int slot = (int)(vc % C::kSlotsL);
            if (!warp_wait(bar(C::bLFull + slot), (vc / C::kSlotsL) & 1, ctl)) return;
            const int k0 = tree_row(w.s, t * kTreeTile, kTreeTile);
            if (tree_masked(w.s, k0, kTreeTile)) {
                uint8_t* v = smem + C::kL + (uint32_t)slot * C::kBytesK;
                const int key = k0 + row;
                if (tree_partly(w.s, key)) {
                    bool hit = false;
                    for (int c = 0; c < kHd / 8; ++c) {
                        uint4* p = reinterpret_cast<uint4*>(v + (c >> 3) * 16384 + row * 128 + (((c & 7) ^ (row & 7)) << 4));
                        if (tree_dead(w.s, key)) {
                            *p = make_uint4(0, 0, 0, 0);
                            continue;
                        }
                        uint4 x = *p;
                        const bool bad = clear_nonfinite(x.x) | clear_nonfinite(x.y) | clear_nonfinite(x.z) | clear_nonfinite(x.w);
                        if (bad) *p = x;
                        hit |= bad;
                    }
                    if (hit) *reinterpret_cast<volatile int*>(smem + C::kPoison + (item & 7) * 4) = (int)item + 1;
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            }
            __syncwarp();
            if ((threadIdx.x & 31) == 0) mbar_arrive(bar(C::bPFull + slot));
        }
        ++item;
    } while (w.next(a));
}

__device__ __forceinline__ uint32_t qk_offset(int row, int c16)  // 16-byte chunk of a K-major e4m3 row
{
    return kHd == 128 ? (uint32_t)(row * 128 + ((c16 ^ (row & 7)) << 4)) : (uint32_t)(row * 64 + ((c16 ^ ((row >> 1) & 3)) << 4));
}

// An item's queries as hi (e4m3) and lo (e5m2) with the row's scale, by the softmax warps; kHd / 8 lanes share a row.  Rows
// past the kv head's keep what they hold: it reaches no row of S that is read.
template <int kNq>
__device__ __forceinline__ void split_queries(const TreeArgs& a, uint8_t* smem, int b, int g, int r, uint32_t item)
{
    using C = Cfg<true, kNq>;
    constexpr int kLanes = kHd / 8, kStep = 256 / kLanes, kU = 8;
    const int tid = threadIdx.x, c = tid % kLanes;
    const int rows = a.R - r * a.rt < kNq * 128 ? a.R - r * a.rt : kNq * 128;
    const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) +
                                                      (((long long)b * a.Hkv + g) * a.R + (long long)r * a.rt) * kHd) + c;
    const int rows_up = (rows + kStep - 1) / kStep * kStep;  // the same for a whole warp
    float* scale = reinterpret_cast<float*>(smem + C::kQs) + (item & 1) * kNq * 128;
#pragma unroll 1
    for (int x0 = tid / kLanes; x0 < rows_up; x0 += kStep * kU) {
        uint4 v[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int x = x0 + u * kStep;
            v[u] = x < rows ? src[(long long)x * (kHd / 8)] : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int x = x0 + u * kStep;
            if (x >= rows_up) break;
            const uint32_t p[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
            uint32_t big = 0;  // bits of the largest magnitude: bf16 in the upper half, ordered as integers
#pragma unroll
            for (int i = 0; i < 4; ++i) big = max(big, max(p[i] << 16 & 0x7fff0000u, p[i] & 0x7fff0000u));
#pragma unroll
            for (int o = kLanes / 2; o > 0; o >>= 1) big = max(big, __shfl_xor_sync(0xffffffffu, big, o));
            const bool finite = big < 0x7f800000u;
            int e = (int)(big >> 23) - 135 + ((big & 0x7fffffu) > 0x600000u ? 1 : 0);
            e = !finite || e < -126 ? -126 : e;
            const float down = finite ? __uint_as_float((uint32_t)(127 - e) << 23) : 0.f;
            // a row that is not finite: its elements that are not become NaN below (times 0), and with them its scores, of which
            // the mask still hides what it hides
            if (c == 0 && x < rows) scale[x] = __uint_as_float((uint32_t)(127 + e) << 23);
            uint2 hi, lo;
            uint32_t* ph = &hi.x;
            uint32_t* pl = &lo.x;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float f0 = __uint_as_float(p[2 * i] << 16) * down, f1 = __uint_as_float(p[2 * i] & 0xffff0000u) * down;
                const float f2 = __uint_as_float(p[2 * i + 1] << 16) * down, f3 = __uint_as_float(p[2 * i + 1] & 0xffff0000u) * down;
                ph[i] = (uint32_t)e4m3x2(f0, f1) | (uint32_t)e4m3x2(f2, f3) << 16;
                float h0, h1, h2, h3;
                e4m3x4_to_float(ph[i], h0, h1, h2, h3);
                pl[i] = (uint32_t)e5m2x2(f0 - h0, f1 - h1) | (uint32_t)e5m2x2(f2 - h2, f3 - h3) << 16;
            }
            uint8_t* q = smem + C::kQ + (uint32_t)(x >> 7) * C::kBytesQ + qk_offset(x & 127, c >> 1) + (c & 1) * 8;
            if (x < rows) {
                *reinterpret_cast<uint2*>(q) = hi;
                *reinterpret_cast<uint2*>(q + 128 * kHd) = lo;
            }
        }
    }
}

template <int kNq>
__device__ __forceinline__ void prep_e4m3_role(const TreeArgs& a, uint32_t sbase, uint8_t* smem, Walk w, const WaitCtl& ctl)
{
    using C = Cfg<true, kNq>;
    auto bar = [&](int i) { return sbase + C::kBar + 8u * (uint32_t)i; };
    const int row = threadIdx.x & 127, lane = threadIdx.x & 31;
    Ring<C::kSlotsL> rl;
    Ring<C::kSlotsP> rp;
    Ring<C::kSlotsX> rx;
    uint32_t item = 0;
    do {
        for (int t = w.t0; t < w.t1; ++t, rl.next(), rp.next(), rx.next()) {
            const int sl = rl.slot, sp = rp.slot, sx = rx.slot;
            if (!warp_wait(bar(C::bXFull + sx), rx.par, ctl)) return;
            if (!warp_wait(bar(C::bLFull + sl), rl.par, ctl)) return;
            if (rp.round && !warp_wait(bar(C::bPEmpty + sp), rp.par ^ 1, ctl)) return;
            const uint8_t* src = smem + C::kL + (uint32_t)sl * C::kBytesK;
            uint8_t* dst = smem + C::kP + (uint32_t)sp * C::kBytesV;
            const __nv_bfloat162 up = __float2bfloat162_rn(reinterpret_cast<const float*>(smem + C::kX + sx * 1024)[128 + row]);
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(C::bXEmpty + sx));
            const int k0 = tree_row(w.s, t * kTreeTile, kTreeTile), key = k0 + row;
            const bool past = tree_dead(w.s, key), drafted = tree_partly(w.s, key);
            bool hit = false;
            // a thread has a row; starting each at another chunk keeps a warp's accesses in different banks
            auto at = [&](int i) { return (i + row) & (kHd / 16 - 1); };
            auto convert = [&](const uint4& x, uint32_t (&o)[8]) {
                const uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float f0, f1, f2, f3;
                    e4m3x4_to_float(u[j], f0, f1, f2, f3);
                    __nv_bfloat162 p0 = __hmul2(__floats2bfloat162_rn(f0, f1), up), p1 = __hmul2(__floats2bfloat162_rn(f2, f3), up);
                    o[2 * j] = *reinterpret_cast<const uint32_t*>(&p0);
                    o[2 * j + 1] = *reinterpret_cast<const uint32_t*>(&p1);
                }
            };
            auto store = [&](int c, const uint32_t (&o)[8]) {
                uint8_t* p = dst + (c >> 2) * 16384 + row * 128;
                *reinterpret_cast<uint4*>(p + ((((2 * c) & 7) ^ (row & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
                *reinterpret_cast<uint4*>(p + ((((2 * c + 1) & 7) ^ (row & 7)) << 4)) = make_uint4(o[4], o[5], o[6], o[7]);
            };
            if (!tree_masked(w.s, k0, kTreeTile)) {  // no branch inside: the chunks' conversions overlap
                uint4 x0 = *reinterpret_cast<const uint4*>(src + row * kHd + at(0) * 16);
                uint4 x1 = *reinterpret_cast<const uint4*>(src + row * kHd + at(1) * 16);
#pragma unroll 1
                for (int i = 0; i < kHd / 16; i += 2) {
                    const uint4 n0 = *reinterpret_cast<const uint4*>(src + row * kHd + at(i + 2) * 16);
                    const uint4 n1 = *reinterpret_cast<const uint4*>(src + row * kHd + at(i + 3) * 16);
                    uint32_t o[8], p[8];
                    convert(x0, o);
                    convert(x1, p);
                    store(at(i), o);
                    store(at(i + 1), p);
                    x0 = n0;
                    x1 = n1;
                }
            } else {
#pragma unroll 1
                for (int i = 0; i < kHd / 16; ++i) {
                    const int c = at(i);
                    uint32_t o[8];
                    convert(*reinterpret_cast<const uint4*>(src + row * kHd + c * 16), o);
                    if (drafted) {
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            if (past)
                                o[j] = 0;
                            else
                                hit |= clear_nonfinite(o[j]);
                        }
                    }
                    store(c, o);
                }
            }
            if (hit) *reinterpret_cast<volatile int*>(smem + C::kPoison + (item & 7) * 4) = (int)item + 1;
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(bar(C::bPFull + sp));
                mbar_arrive(bar(C::bLEmpty + sl));
            }
        }
        ++item;
    } while (w.next(a));
}

// ------------------------------------------------------------------------------------------------
// MMA issue (one warp, one lane of it)
// ------------------------------------------------------------------------------------------------
// An item's jobs, one S and one P V each: tile by tile, and (kNq == 2) warpgroup 0's query rows, then 1's.  Job j
// belongs to warpgroup j & 1; its S is issued once P V of job j - 2, which reads the same TMEM columns, is.  A
// commit costs the issuing warp 50 to 180 cycles, so there are two per job: S is ready (which also says that P V
// of job j - 2 is done, and that K has been read), and V has been read.
template <bool kE4, int kNq, bool kExact>
__device__ __forceinline__ void mma_role(const TreeArgs& a, uint32_t sbase, uint32_t tmem, Walk w, const WaitCtl& ctl)
{
    using C = Cfg<kE4, kNq>;
    auto bar = [&](int i) { return sbase + C::kBar + 8u * (uint32_t)i; };
    Ring<C::kSlotsK> rk;
    Ring<C::kSlotsP> rv;
    uint32_t item = 0, pc = 0;  // pc: a parity bit per warpgroup
    const uint32_t lead = elect();
    tmem = __shfl_sync(0xffffffffu, tmem, 0);
    bool ok = true;
    do {
        if (!warp_wait(bar(C::bQFull), item++ & 1, ctl)) break;
        tc_fence_after_sync();
        const int n = __shfl_sync(0xffffffffu, w.t1 - w.t0, 0) * kNq;
#pragma unroll 1
        for (int j = 0; j < n + 2; ++j) {
            const int wg = j & 1;
            if (j >= 2) {
                ok = warp_wait(bar(C::bPFull + rv.slot), rv.par, ctl) && warp_wait(bar(C::bP + wg), pc >> wg & 1, ctl);
                if (!ok) break;
                pc ^= 1u << wg;
                tc_fence_after_sync();
                issue_pv<kExact>(lead, sbase + (kE4 ? C::kP + (uint32_t)rv.slot * C::kBytesV : C::kL + (uint32_t)rv.slot * C::kBytesK), tmem, wg, j >= 4);
                if (j >= n) lead_commit(lead, bar(C::bO + wg));  // the warpgroup's last job of the item
                if (kNq == 1 || wg == 1) {
                    lead_commit(lead, bar((kE4 ? C::bPEmpty : C::bLEmpty) + rv.slot));
                    rv.next();
                }
            }
            if (j < n) {
                if (kNq == 1 || wg == 0) {
                    ok = warp_wait(bar(C::bKFull + rk.slot), rk.par, ctl);
                    if (!ok) break;
                    tc_fence_after_sync();
                }
                issue_s<kE4, kNq>(lead, sbase, tmem, wg, rk.slot);
                lead_commit(lead, bar(C::bS + wg));  // the softmax warps release K
                if (kNq == 1 || wg == 1) rk.next();
                if (j == n - 1) lead_commit(lead, bar(C::bQEmpty));
            }
        }
    } while (ok && w.next(a));
    lead_commit(lead, bar(C::bDrain));
    drain_wait(bar(C::bDrain), 0);
}

// ------------------------------------------------------------------------------------------------
// softmax warpgroups
// ------------------------------------------------------------------------------------------------
// Which of the 64 rows from k0 query token t sees, one bit each; for tiles that reach past the prefix.
// reach: the first row of the prefix in the token's window.
__device__ __forceinline__ unsigned long long low_bits(int n) { return n >= 64 ? ~0ull : (n > 0 ? (1ull << n) - 1 : 0ull); }
__device__ __forceinline__ unsigned long long seen_bits(const TreeArgs& a, const Seq& s, int b, int t, int k0, int reach)
{
    const int p = s.len - k0;  // rows of the prefix among them
    unsigned long long bits = low_bits(p);
    if constexpr (kWin) bits &= ~low_bits(reach - k0) | low_bits(tree_sinks(s) - k0);
    if (t >= s.cnt) return bits;
    const int j0 = p < 0 ? -p : 0, j1 = 64 - p < s.cnt ? 64 - p : s.cnt;
    if (!a.mask) {
        const int to = j1 < t + 1 ? j1 : t + 1;  // one past the last drafted token up to t
        if constexpr (kWin) {
            const int from = t - a.window + 1 > j0 ? t - a.window + 1 : j0, first = a.sinks - s.len < to ? a.sinks - s.len : to;
            return bits | (low_bits(p + to) & ~low_bits(p + from)) | (low_bits(p + first) & ~low_bits(p + j0));
        } else {
            const int n = to - j0;
            return n > 0 ? bits | (n >= 64 ? ~0ull : (1ull << n) - 1) << (p + j0) : bits;
        }
    }
    const uint8_t* m = a.mask + ((a.mask_batched ? (long long)b * a.T : 0) + t) * a.T;
    const bool wide = (reinterpret_cast<uintptr_t>(a.mask) & 15) == 0 && a.T % 16 == 0;  // rows of whole 16-byte words
#pragma unroll 1
    for (int j = j0 & ~15; j < j1; j += 16) {
        uint32_t w = 0;  // drafted tokens j .. j + 15, one bit each
        if (wide) {
            const uint4 v = *reinterpret_cast<const uint4*>(m + j);
            const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {  // a byte's bit 7 says that it is not 0; the product gathers the four
                const uint32_t y = ((u[i] & 0x7f7f7f7fu) + 0x7f7f7f7fu | u[i]) >> 7 & 0x01010101u;
                w |= (y * 0x01020408u >> 24 & 15u) << 4 * i;
            }
        } else {
            uint8_t v[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = j + i < j1 ? m[j + i] : (uint8_t)0;
#pragma unroll
            for (int i = 0; i < 16; ++i) w |= v[i] ? 1u << i : 0u;
        }
        if (j < j0) w &= ~0u << (j0 - j);
        if (j + 16 > j1) w &= (1u << (j1 - j)) - 1;
        const int to = p + j;  // the first of them among the 64 rows; below 0 only bits that j0 has cleared
        bits |= to < 0 ? (unsigned long long)(w >> -to) : (unsigned long long)w << to;
    }
    return bits;
}

template <bool kE4, int kNq, bool kExact>
__device__ __forceinline__ void softmax_role(const TreeArgs& a, uint32_t sbase, uint8_t* smem, uint32_t tmem, Walk w,
                                             const WaitCtl& ctl)
{
    using C = Cfg<kE4, kNq>;
    auto bar = [&](int i) { return sbase + C::kBar + 8u * (uint32_t)i; };
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int wg = warp >> 2;
    const int rw = (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lanes + kColS + (uint32_t)wg * 128;
    const uint32_t tO = tmem + lanes + kColO + (uint32_t)wg * 128;
    uint32_t jobs = 0, tiles = 0, item = 0;  // this warpgroup's jobs, all tiles, items so far
    uint32_t pairs = 0;                      // items that both warpgroups had jobs of (kNq == 1)

    auto split = [&](int b, int g, int r, uint32_t it) {
        split_queries<kNq>(a, smem, b, g, r, it);
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(C::bQFull));
    };
    if constexpr (kE4) split(w.b, w.g, w.r, 0);
    do {
        const int x = w.r * a.rt + (kNq == 2 ? wg * 128 : 0) + rw;  // query row of the kv head
        const int tq = x % a.T;
        const bool live = x < a.R && tq < w.s.cnt;
        const bool any_live = __any_sync(0xffffffffu, live);
        const int n = w.t1 - w.t0;
        float m_run = -INFINITY, l_run = 0.f, den_run = 0.f, sl2 = a.scale_log2;
        bool first = true;
        int reach = 0;
        if constexpr (kWin) reach = live ? tree_reach(a, w.s, w.b, tq) : 0;
        for (int i = kNq == 1 ? wg : 0; i < n; i += kNq == 1 ? 2 : 1) {
            const int k0 = tree_row(w.s, (w.t0 + i) * kTreeTile, kTreeTile);
            const bool masked = tree_masked(w.s, k0, kTreeTile);
            unsigned long long seen[2] = {~0ull, ~0ull};
            if (masked && any_live) {
#pragma unroll 1
                for (int h = 0; h < 2; ++h) {
                    const unsigned long long v = seen_bits(a, w.s, w.b, tq, k0 + 64 * h, reach);
                    seen[0] = h ? seen[0] : v;
                    seen[1] = v;
                }
            }
            const uint32_t job = jobs++;
            if (!warp_wait(bar(C::bS + wg), job & 1, ctl)) return;
            const uint32_t tile = tiles + (uint32_t)i;  // of all this CTA's
            if (lane == 0 && (warp & 3) == 0 && (kNq == 1 || wg == 1))  // S of both warpgroups is in job order
                mbar_arrive(bar(C::bKEmpty + (int)(tile % C::kSlotsK)));
            const int sx = (int)(tile % C::kSlotsX);
            if (!any_live) {  // no query row in these lanes: what P holds there reaches no row that is read
                if (lane == 0) {
                    if constexpr (kE4) mbar_arrive(bar(C::bXEmpty + sx));
                    mbar_arrive(bar(C::bP + wg));
                }
                continue;
            }
            tc_fence_after_sync();
            const float4* xs = nullptr;
            if constexpr (kE4) {
                if (!warp_wait(bar(C::bXFull + sx), (tile / C::kSlotsX) & 1, ctl)) return;
                xs = reinterpret_cast<const float4*>(smem + C::kX + sx * 1024);
                if (first)
                    sl2 = a.scale_log2 * reinterpret_cast<const float*>(smem + C::kQs)[(item & 1) * kNq * 128 + (kNq == 2 ? wg * 128 : 0) + rw];
            }
            // 32 columns of S at a time, their weights written over S as it is read.  The loop is not unrolled:
            // the roles' loops run side by side and wait for the instruction cache when they do not fit it.
            float2 s2 = make_float2(0.f, 0.f), d2 = make_float2(0.f, 0.f);  // of the weights, and of the weights as rounded
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
                uint32_t r[32];
                float4 sc[kE4 ? 8 : 1];
                if constexpr (kE4) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) sc[e] = xs[8 * c + e];
                }
                tmem_ld_32x32b_x32(tS + 32 * c, r);
                tmem_ld_wait(r);
                if constexpr (kE4) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float2 u0 = mul2(make_float2(__uint_as_float(r[4 * e]), __uint_as_float(r[4 * e + 1])), make_float2(sc[e].x, sc[e].y));
                        const float2 u1 = mul2(make_float2(__uint_as_float(r[4 * e + 2]), __uint_as_float(r[4 * e + 3])), make_float2(sc[e].z, sc[e].w));
                        r[4 * e] = __float_as_uint(u0.x);
                        r[4 * e + 1] = __float_as_uint(u0.y);
                        r[4 * e + 2] = __float_as_uint(u1.x);
                        r[4 * e + 3] = __float_as_uint(u1.y);
                    }
                }
                if (masked) {
                    const uint32_t bits = (uint32_t)((c < 2 ? seen[0] : seen[1]) >> (32 * (c & 1)));
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (!(bits & 1u << e)) r[e] = __float_as_uint(-INFINITY);
                }
                float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int e = 0; e < 32; e += 2) m4[(e >> 1) & 3] = max3f(m4[(e >> 1) & 3], __uint_as_float(r[e]), __uint_as_float(r[e + 1]));
                const float m_new = max3f(max3f(m4[0], m4[1], m4[2]), m4[3], -INFINITY) * sl2;
                const bool raise = live && m_new > m_run + 8.0f;
                if (__any_sync(0xffffffffu, raise)) {
                    // The reference goes up, by a whole number of binades once there is one, and with it go the
                    // sums, O (the previous job's P V is done: S of this one was committed after it), and the
                    // weights of this tile's columns so far, which a power of two leaves as they are rounded.
                    const float to = raise ? (m_run == -INFINITY ? m_new : m_run + ceilf(m_new - m_run)) : m_run;
                    const float alpha = to == m_run ? 1.0f : ex2_approx(m_run - to);
                    l_run *= alpha;
                    den_run *= alpha;
                    s2 = mul2(s2, make_float2(alpha, alpha));
                    d2 = mul2(d2, make_float2(alpha, alpha));
                    m_run = to;
#pragma unroll 1
                    for (int k = first ? 0 : kHd / 16; k > 0; --k) {
                        uint32_t o[16];
                        tmem_ld_32x32b_x16(tO + 16 * (k - 1), o);
                        tmem_ld_wait(o);
#pragma unroll
                        for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                        tmem_st_32x32b_x16(tO + 16 * (k - 1), o);
                    }
                    const __nv_bfloat162 a2 = __float2bfloat162_rn(alpha);
#pragma unroll 1
                    for (int k = 0; k < (kExact ? 2 * c : c); ++k) {
                        uint32_t o[16];
                        tmem_st_wait();
                        tmem_ld_32x32b_x16(tS + 16 * k, o);
                        tmem_ld_wait(o);
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            __nv_bfloat162 v = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&o[e]), a2);
                            o[e] = *reinterpret_cast<const uint32_t*>(&v);
                        }
                        tmem_st_32x32b_x16(tS + 16 * k, o);
                    }
                }
                const float ref = m_run == -INFINITY ? 0.f : m_run;
                const float2 scale2 = make_float2(sl2, sl2), nref2 = make_float2(-ref, -ref);
                float2 s4[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)}, d4[2] = {s4[0], s4[0]};
                uint32_t pk[kExact ? 32 : 16];
#pragma unroll
                for (int e = 0; e < 32; e += 2) {
                    const float2 x2 = fma2(make_float2(__uint_as_float(r[e]), __uint_as_float(r[e + 1])), scale2, nref2);
                    const float2 p2 = make_float2(ex2_approx(x2.x), ex2_approx(x2.y));
                    s4[(e >> 1) & 1] = add2(s4[(e >> 1) & 1], p2);
                    if constexpr (kExact) {
                        split_weights(p2, pk[e / 2], pk[16 + e / 2]);
                    } else {
                        pk[e / 2] = pack_bf16x2(p2.x, p2.y);
                        d4[(e >> 1) & 1] = add_bf16x2(d4[(e >> 1) & 1], pk[e / 2]);
                    }
                }
                if constexpr (kExact)
                    tmem_st_32x32b_x32(tS + 32 * c, pk);
                else
                    tmem_st_32x32b_x16(tS + 16 * c, pk);
                s2 = add2(s2, add2(s4[0], s4[1]));
                d2 = add2(d2, add2(d4[0], d4[1]));
            }
            if constexpr (kE4) {
                if (lane == 0) mbar_arrive(bar(C::bXEmpty + sx));
            }
            // The normaliser is the sum of the weights as the product gets them: where many keys share a weight their
            // roundings go the same way, and a row that one key dominates is divided by that key's.  lse takes the
            // unrounded sum.
            l_run += s2.x + s2.y;
            den_run += d2.x + d2.y;
            tmem_st_wait();
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(C::bP + wg));
            first = false;
        }

        if constexpr (kE4) {  // the next item's queries, while the last products run
            Walk next = w;
            if (next.next(a)) {
                if (!warp_wait(bar(C::bQEmpty), item & 1, ctl)) return;
                split(next.b, next.g, next.r, item + 1);
            }
        }

        // the item's rows: O of both warpgroups (kNq == 1), or of this one
        float m = m_run, l = l_run, den = kExact ? l_run * kWeightUp : den_run, w0 = 1.f, w1 = 0.f;
        const int n1 = kNq == 1 ? n >> 1 : 0;
        if constexpr (kNq == 1) {
            float4* ml = reinterpret_cast<float4*>(smem + C::kMl);
            ml[wg * 128 + rw] = make_float4(m, l, den, 0.f);
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(C::bEpi));
            if (!warp_wait(bar(C::bEpi), item & 1, ctl)) return;
            const float4 a0 = ml[rw], a1 = ml[128 + rw];
            m = fmaxf(a0.x, a1.x);
            const float ref = m == -INFINITY ? 0.f : m;
            w0 = ex2_approx(a0.x - ref);
            w1 = ex2_approx(a1.x - ref);
            l = a0.y * w0 + a1.y * w1;
            den = a0.z * w0 + a1.z * w1;
            if (a0.x == -INFINITY && a0.y != 0.f) l = den = a0.y;  // NaN scores alone leave no maximum
            if (a1.x == -INFINITY && a1.y != 0.f) l = den = a1.y;
            if (!warp_wait(bar(C::bO + 0), item & 1, ctl)) return;
            if (n1 > 0 && !warp_wait(bar(C::bO + 1), pairs++ & 1, ctl)) return;
        } else {
            if (!warp_wait(bar(C::bO + wg), item & 1, ctl)) return;
        }
        tc_fence_after_sync();
        const bool row = x < a.R;  // a query row of the kv head, if not of a token that the sequence has
        if (__any_sync(0xffffffffu, row)) {
            const bool whole = w.whole(), none = !live || (m == -INFINITY && l == 0.f);
            const bool poison = *reinterpret_cast<volatile int*>(smem + C::kPoison + (item & 7) * 4) == (int)item + 1;
            const float inv = whole ? (none ? 0.f : 1.0f / den) : 1.0f;
            const long long grow = ((long long)w.b * a.Hkv + w.g) * a.R + x;
            const long long pslot = (long long)blockIdx.x * 2 + (w.first ? 0 : 1);
            const int prow = (kNq == 2 ? wg * 128 : 0) + rw;
            constexpr int kCols = kNq == 1 ? kHd / 2 : kHd;
            const int col0 = kNq == 1 ? wg * kCols : 0;
#pragma unroll 1
            for (int c = col0; c < col0 + kCols; c += 32) {
                uint32_t o[32];
                __syncwarp();  // the lanes without a row have gone ahead
                tmem_ld_32x32b_x32(tmem + lanes + kColO + (kNq == 2 ? (uint32_t)wg * 128u : 0u) + c, o);
                tmem_ld_wait(o);
                if constexpr (kNq == 1) {
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * w0);
                    if (n1 > 0) {
                        uint32_t o1[32];
                        tmem_ld_32x32b_x32(tmem + lanes + kColO + 128 + c, o1);
                        tmem_ld_wait(o1);
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(fmaf(__uint_as_float(o1[e]), w1, __uint_as_float(o[e])));
                    }
                }
                if (poison && live) {
                    // (through a window the prefix's rows that some tokens do not see come first)
                    for (int j = tree_first_partly(w.s) - w.s.len; j < w.s.cnt; ++j) {
                        const int key = w.s.len + j;
                        if (j < 0 && !tree_partly(w.s, key)) {
                            j = -1;  // on to the drafted tokens
                            continue;
                        }
                        const int x = tree_list_row(w.s, key, kTreeTile);
                        if (x < w.t0 * kTreeTile || x >= w.t1 * kTreeTile || !(j < 0 ? key >= reach : tree_sees<kWin>(a, w.s, w.b, tq, j))) continue;
                        const long long src = ((long long)w.b * a.Hkv + w.g) * a.cap + key;
#pragma unroll
                        for (int e = 0; e < 32; ++e) {
                            float v;
                            if constexpr (kE4) {
                                float z0, z1, z2;
                                e4m3x4_to_float(static_cast<const uint8_t*>(a.v)[src * kHd + c + e], v, z0, z1, z2);
                                v *= __uint_as_float((uint32_t)a.v_exp[src] << 23);
                            } else {
                                v = __bfloat162float(static_cast<const __nv_bfloat16*>(a.v)[src * kHd + c + e]);
                            }
                            if (!(fabsf(v) <= 3.3895314e38f)) o[e] = __float_as_uint(__uint_as_float(o[e]) + v);  // past bf16's largest
                        }
                    }
                }
                if (!row) continue;
                if (whole && a.bf16_out) {
                    uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + grow * kHd + c);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        uint32_t pk[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            pk[i] = none ? 0u
                                         : pack_bf16x2(__uint_as_float(o[8 * e + 2 * i]) * inv, __uint_as_float(o[8 * e + 2 * i + 1]) * inv);
                        dst[e] = make_uint4(pk[0], pk[1], pk[2], pk[3]);
                    }
                } else if (whole) {
                    float4* dst = reinterpret_cast<float4*>(static_cast<float*>(a.out) + grow * kHd + c);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        dst[e] = none ? make_float4(0.f, 0.f, 0.f, 0.f)
                                      : make_float4(__uint_as_float(o[4 * e]) * inv, __uint_as_float(o[4 * e + 1]) * inv,
                                                    __uint_as_float(o[4 * e + 2]) * inv, __uint_as_float(o[4 * e + 3]) * inv);
                } else {  // column by column: a warp's rows lie side by side
                    float* dst = a.part_o + (pslot * kHd + c) * a.rt + prow;
#pragma unroll
                    for (int e = 0; e < 32; ++e) dst[(long long)e * a.rt] = __uint_as_float(o[e]);
                }
            }
            if (row && (kNq == 2 || wg == 0)) {
                if (whole)
                    a.lse[grow] = none ? -INFINITY : (m + log2f(l)) * kLn2;
                else
                    *reinterpret_cast<float4*>(a.part_ml + (pslot * a.rt + prow) * 4) = make_float4(m, l, den, 0.f);
            }
        }
        if constexpr (kNq == 1) {  // the next item's products overwrite both O's
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(C::bEpi + 1));
            if (!warp_wait(bar(C::bEpi + 1), item & 1, ctl)) return;
            tc_fence_after_sync();
        }
        tiles += (uint32_t)n;
        ++item;
    } while (w.next(a));
}

template <bool kE4, int kNq, bool kExact>
__global__ void __launch_bounds__(kThreads, 1) tree_tc_kernel(const __grid_constant__ Maps maps, const TreeArgs a)
{
    using C = Cfg<kE4, kNq>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kAbort);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kSlot);

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kBars; ++i) {
            uint32_t cnt = 1;
            if (i == C::bP || i == C::bP + 1) cnt = 4;                              // softmax warps of one group
            if (i == C::bEpi || i == C::bEpi + 1) cnt = 8;                          // of both
            if (i >= C::bPFull && i < C::bPEmpty) cnt = 4;                          // warps 12-15
            if (kE4 && i == C::bQFull) cnt = 8;                                     // softmax warps
            if (kE4 && i >= C::bLEmpty && i < C::bPFull) cnt = 4;
            if (kE4 && i >= C::bXEmpty) cnt = 4 * kNq + 4;                          // the warps that read a tile's scales
            mbar_init(sbase + C::kBar + 8u * (uint32_t)i, cnt);
        }
        for (int i = 0; i < 8; ++i) reinterpret_cast<int*>(smem + C::kPoison)[i] = 0;
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 9) {
        tmem_alloc(smem_u32(tmem_slot), kTmemCols);
        tmem_relinquish();
    }
    Walk w;
    const bool work = w.begin(a, blockIdx.x);  // the same for every warp
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    const WaitCtl ctl{abort_flag, a.status, 0};

    if (work) {
        if (warp < 8) {
            softmax_role<kE4, kNq, kExact>(a, sbase, smem, tmem, w, ctl);
        } else if (warp == 8) {
            if (lane == 0) a.border[blockIdx.x].x = -1;  // (the walk's last item may say otherwise)
            if (lane == 0) load_qk_role<kE4, kNq>(a, sbase, maps, w, ctl);
        } else if (warp == 9) {
            mma_role<kE4, kNq, kExact>(a, sbase, tmem, w, ctl);
        } else if (warp == 10) {
            if (lane == 0) load_v_role<kE4, kNq>(a, sbase, maps, w, ctl);
        } else if (warp == 11) {
            if constexpr (kE4) scale_role<kNq>(a, sbase, smem, w, ctl);
        } else {
            if constexpr (kE4)
                prep_e4m3_role<kNq>(a, sbase, smem, w, ctl);
            else
                prep_bf16_role<kNq>(a, sbase, smem, w, ctl);
        }
    }
    if (!work && threadIdx.x == 0) a.border[blockIdx.x] = make_int4(-1, 0, 0, 0);
    if constexpr (kWin) {
        if (!work && a.whole) tree_clear_item<kHd>(a, blockIdx.x);
    }
    tc_fence_before_sync();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// ------------------------------------------------------------------------------------------------
// host side
// ------------------------------------------------------------------------------------------------
PFN_cuTensorMapEncodeTiled_v12000 encode_fn()
{
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    });
    return fn;
}

// [heads][rows][kHd] of 1- or 2-byte elements, boxes of 128 rows and the swizzled row's columns (64 bf16, all e4m3).
bool make_map(CUtensorMap* map, const void* base, long long rows, long long heads, bool bytes)
{
    auto fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t es = bytes ? 1 : 2;
    cuuint64_t dims[3] = {(cuuint64_t)kHd, (cuuint64_t)rows, (cuuint64_t)heads};
    cuuint64_t strides[2] = {(cuuint64_t)kHd * es, (cuuint64_t)rows * kHd * es};
    cuuint32_t box[3] = {bytes ? (cuuint32_t)kHd : 64u, 128u, 1u};
    cuuint32_t estr[3] = {1, 1, 1};
    return fn(map, bytes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides,
              box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              bytes && kHd == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool kE4, int kNq, bool kExact>
cudaError_t launch(const TreeArgs& a, const Maps& maps, cudaStream_t s)
{
    using C = Cfg<kE4, kNq>;
    static std::mutex mu;
    static bool done[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    {
        std::lock_guard<std::mutex> lk(mu);
        if (!done[dev]) {
            e = cudaFuncSetAttribute(tree_tc_kernel<kE4, kNq, kExact>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmem);
            if (e != cudaSuccess) return e;
            done[dev] = true;
        }
    }
    tree_tc_kernel<kE4, kNq, kExact><<<a.ctas, kThreads, C::kSmem, s>>>(maps, a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t RA_TREE_LAUNCH(const TreeArgs& a, bool e4m3, cudaStream_t s)
{
    Maps maps;
    const long long heads = (long long)a.B * a.Hkv;
    if (!make_map(&maps.q, a.q, a.R, heads, false) || !make_map(&maps.k, a.k, a.cap, heads, e4m3) ||
        !make_map(&maps.v, a.v, a.cap, heads, e4m3))
        return cudaErrorInvalidValue;
    if (a.rt == 128) return !e4m3 ? launch<false, 1, true>(a, maps, s) : a.bf16_out ? launch<true, 1, false>(a, maps, s) : launch<true, 1, true>(a, maps, s);
    if (a.bf16_out) return e4m3 ? launch<true, 2, false>(a, maps, s) : launch<false, 2, false>(a, maps, s);
    return e4m3 ? launch<true, 2, true>(a, maps, s) : launch<false, 2, true>(a, maps, s);
}

}  // namespace ra
