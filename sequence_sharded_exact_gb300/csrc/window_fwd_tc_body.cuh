// window_fwd_tc_body.cuh -- tensor-core forward of the attention through a window (window.cuh) for sm_103a: bf16, head
// dim RA_WIN_HD (128 or 64), any length.  Compiled once per head dim (window_fwd_tc.cu: 128, window_fwd_tc_d64.cu: 64); the
// including file names the host entry point through RA_WIN_FWD_LAUNCH.
//
// One CTA per SM, persistent.  A work unit is two tiles of 128 queries that share every K/V tile: two heads of one kv
// head's group at the same positions where the group is even, else 256 consecutive positions of one head.  Two heads meet
// W / 128 + 1 key tiles, 256 positions W / 128 + 2, of which each query tile sees all but one.  Units that share keys are
// neighbours, so that they run at the same time and K and V come from L2.
//   * warp 8 loads (TMA, one thread): Q tiles, and K and V tiles through rings.
//   * warp 9 issues tcgen05.mma (one thread): S_w = Q_w K^T into TMEM, O_w += P_w V with P_w from TMEM; the next tile's S
//     between the two P V, so that the tensor cores work while the softmax warps do.
//   * warps 0-3 and 4-7: softmax of query tile 0 and 1, thread = row = TMEM lane: the row's maximum and sum need no exchange.
//     m follows the maximum only when that grows by more than 2^8 (O / l does not depend on the reference).  Hidden scores are
//     set to -infinity by a bit each, in the tiles that are not wholly visible: one at each end of the window, and the sinks'.
//   * warps 10-11 look through V in those tiles: a weight of 0 would not hide what is not finite, so such elements are
//     cleared in shared memory, and added to the rows that do see them at the unit's end (rare, from global memory).
//   * TMEM: S0 columns [0,128), S1 [128,256), O0 from 256, O1 from 384.
// The weights go into P V as one bf16 value each; the row is divided by the sum of the unrounded weights, but for the
// tile's largest, which counts as rounded: a row that one key dominates gets that key's value exactly.
#include <cuda_bf16.h>
#include <math.h>

#include "window_tc.cuh"

namespace ra {
namespace {

constexpr int kTile = kWinTile;
constexpr int kHd = RA_WIN_HD;
static_assert(kHd == 128 || kHd == 64, "head dim");
constexpr int kHalves = kHd / 64;              // 128-byte-swizzle boxes (64 columns) per row
constexpr int kStages = kHd == 64 ? 4 : 2;     // K/V ring
static_assert(kStages < 8, "units that warps 10-11 may be ahead have poison slots of their own");
constexpr int kThreads = 384;
constexpr uint32_t kHalfBytes = kTile * 64 * 2;
constexpr uint32_t kTileBytes = kHalves * kHalfBytes;

constexpr uint32_t kSmemQ = 0;
constexpr uint32_t kSmemK = kSmemQ + 2 * kTileBytes;
constexpr uint32_t kSmemV = kSmemK + kStages * kTileBytes;
constexpr uint32_t kSmemBar = kSmemV + kStages * kTileBytes;

enum : int {
    BAR_Q_FULL = 0,
    BAR_Q_EMPTY = 1,
    BAR_K_FULL = 2,
    BAR_V_FULL = BAR_K_FULL + kStages,
    BAR_K_EMPTY = BAR_V_FULL + kStages,   // both S MMAs have read K
    BAR_V_EMPTY = BAR_K_EMPTY + kStages,  // both P V MMAs have read V, and warps 10-11 have passed the tile
    BAR_V_READY = BAR_V_EMPTY + kStages,  // warps 10-11 have looked through V (tiles that are not wholly visible)
    BAR_S_FULL = BAR_V_READY + kStages,
    BAR_P_FULL = BAR_S_FULL + 2,
    BAR_O_DONE = BAR_P_FULL + 2,
    BAR_DRAIN = BAR_O_DONE + 2,
    BAR_COUNT = BAR_DRAIN + 1
};

constexpr uint32_t kSmemTmemSlot = kSmemBar + BAR_COUNT * 8;
constexpr uint32_t kSmemAbort = kSmemTmemSlot + 8;
constexpr uint32_t kSmemPoison = kSmemAbort + 8;                    // [8] int: unit + 1 that holds cleared elements
constexpr uint32_t kSmemBytes = kSmemPoison + 32 + 1024;            // slack for the 1024-byte alignment of the base
static_assert(kSmemBytes <= 232448, "shared memory");

constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColS0 = 0, kColO0 = 256;
constexpr uint64_t kWaitLimitNs = 4000000000ull;

struct FwdArgs {
    Geometry geo, store_geo;  // of the loads; of out and lse
    Band band;
    int H, Hkv, G;
    int pair;         // 1: a unit is two heads at 128 positions; 0: 256 positions of one head
    int blocks;       // blocks of 128 or 256 positions
    int rows;         // heads, or pairs of them, of a kv head
    long long units;  // B * Hkv * blocks * rows
    const __nv_bfloat16* v;
    void* out;
    float* lse;
    int out_f32;
    unsigned int* status;
    float scale_log2;
};

struct Unit {
    int zk;        // b * Hkv + kv head
    int zq, zq1;   // b * H + head of the two query tiles
    int p, p1;     // their first positions
    TileRun run;   // key tiles
};

__device__ __forceinline__ Unit unit_of(const FwdArgs& a, long long item)
{
    Unit u;
    const int row = (int)(item % a.rows);
    long long rest = item / a.rows;
    const int blk = (int)(rest % a.blocks);
    u.zk = (int)(rest / a.blocks);
    u.zq = u.zk * a.G + row * (a.pair ? 2 : 1);
    u.zq1 = a.pair ? u.zq + 1 : u.zq;
    u.p = blk * (a.pair ? kTile : 2 * kTile);
    u.p1 = a.pair ? u.p : u.p + kTile;
    u.run = key_tiles(a.band, u.p, a.pair ? kTile : 2 * kTile, kTile);
    return u;
}

// Do all rows of both query tiles see all of the keys?
__device__ __forceinline__ bool whole_tile(const FwdArgs& a, const Unit& u, int k0)
{
    return band_tile_whole(a.band, u.p, a.pair ? kTile : 2 * kTile, k0, kTile);
}

// ------------------------------------------------------------------------------------------------
// softmax warpgroups
// ------------------------------------------------------------------------------------------------
__device__ __forceinline__ void softmax_role(const FwdArgs& a, uint32_t sbase, uint8_t* smem, uint32_t tmem, const WaitCtl& ctl)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int w = warp >> 2;                // query tile of this warpgroup
    const int rw = (warp & 3) * 32 + lane;  // row within the tile = TMEM lane
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lane_off + kColS0 + (uint32_t)w * 128;
    const uint32_t tO = tmem + lane_off + kColO0 + (uint32_t)w * 128;
    const uint32_t bar_s = sbase + kSmemBar + 8 * (BAR_S_FULL + w);
    const uint32_t bar_p = sbase + kSmemBar + 8 * (BAR_P_FULL + w);
    const uint32_t bar_o = sbase + kSmemBar + 8 * (BAR_O_DONE + w);
    const float sl2 = a.scale_log2;
    uint32_t tcount = 0, ucount = 0;

    for (long long item = blockIdx.x; item < a.units; item += gridDim.x, ++ucount) {
        const Unit u = unit_of(a, item);
        const int q0 = w ? u.p1 : u.p, p = q0 + rw, ntiles = u.run.count();
        float m_run = -INFINITY, l_run = 0.f, c_run = 0.f;
        for (int jj = 0; jj < ntiles; ++jj, ++tcount) {
            const int k0 = u.run.at(jj) * kTile;
            const bool whole = band_tile_whole(a.band, q0, kTile, k0, kTile);
            uint32_t seen[4] = {~0u, ~0u, ~0u, ~0u};
            if (!whole) {
                const Seen s = seen_keys(a.band, p, k0);
#pragma unroll
                for (int c = 0; c < 4; ++c) seen[c] = s.word(32 * c);
            }
            if (!mbar_wait(bar_s, tcount & 1, ctl)) return;
            tc_fence_after_sync();
            __syncwarp();
            uint32_t r[4][32];
            tmem_ld_32x32b_x32(tS + 0, r[0]);
            tmem_ld_32x32b_x32(tS + 32, r[1]);
            tmem_ld_wait(r[0]);
            tmem_ld_wait(r[1]);
            tmem_ld_32x32b_x32(tS + 64, r[2]);
            tmem_ld_32x32b_x32(tS + 96, r[3]);
            float m8[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) m8[i] = -INFINITY;
            auto hide_and_max = [&](int c4) {
                if (!whole) {
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (!(seen[c4] & (1u << e))) r[c4][e] = __float_as_uint(-INFINITY);
                }
#pragma unroll
                for (int e = 0; e < 32; e += 2)
                    m8[(e >> 1) & 7] = max3f(m8[(e >> 1) & 7], __uint_as_float(r[c4][e]), __uint_as_float(r[c4][e + 1]));
            };
            hide_and_max(0);
            hide_and_max(1);
            tmem_ld_wait(r[2]);
            tmem_ld_wait(r[3]);
            hide_and_max(2);
            hide_and_max(3);
            const float mx = max3f(max3f(m8[0], m8[1], m8[2]), max3f(m8[3], m8[4], m8[5]), fmaxf(m8[6], m8[7]));
            const float m_tile = mx * sl2;
            float m_new = m_run;
            if (m_tile > m_run + 8.0f) m_new = m_tile;
            const float alpha = (m_new == m_run) ? 1.0f : ex2_approx(m_run - m_new);
            const float ref = m_new == -INFINITY ? 0.f : m_new;
            const float2 scale2 = make_float2(sl2, sl2), nref2 = make_float2(-ref, -ref);
            float2 s4[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) s4[i] = make_float2(0.f, 0.f);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                uint32_t pk[32];
#pragma unroll
                for (int cc = 0; cc < 2; ++cc) {
                    const int c4 = half * 2 + cc;
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        const float2 x2 = fma2(make_float2(__uint_as_float(r[c4][e]), __uint_as_float(r[c4][e + 1])), scale2, nref2);
                        const float2 p2 = make_float2(ex2_approx(x2.x), ex2_approx(x2.y));
                        s4[(e >> 1) & 3] = add2(s4[(e >> 1) & 3], p2);
                        pk[cc * 16 + e / 2] = pack_bf16x2(p2.x, p2.y);
                    }
                }
                tmem_st_32x32b_x32(tS + half * 32, pk);
            }
            const float2 s2 = add2(add2(s4[0], s4[1]), add2(s4[2], s4[3]));
            const float p_max = ex2_approx(fmaf(mx, sl2, -ref));
            const float p_max_bf16 = __uint_as_float(pack_bf16x2(p_max, 0.f) << 16);
            l_run = l_run * alpha + (s2.x + s2.y);
            c_run = c_run * alpha + (p_max_bf16 - p_max);
            tmem_st_wait();
            if (__any_sync(0xffffffffu, jj > 0 && alpha != 1.0f)) {
                if (!mbar_wait(bar_o, (tcount - 1) & 1, ctl)) return;  // O of the previous tile is complete
                tc_fence_after_sync();
#pragma unroll 1
                for (int c4 = 0; c4 < kHd / 32; ++c4) {
                    uint32_t o[32];
                    tmem_ld_32x32b_x32(tO + c4 * 32, o);
                    tmem_ld_wait(o);
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        const float2 v = mul2(make_float2(__uint_as_float(o[e]), __uint_as_float(o[e + 1])), make_float2(alpha, alpha));
                        o[e] = __float_as_uint(v.x);
                        o[e + 1] = __float_as_uint(v.y);
                    }
                    tmem_st_32x32b_x32(tO + c4 * 32, o);
                }
                tmem_st_wait();
            }
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_p);
            m_run = m_new;
        }
        // the unit's rows
        if (!mbar_wait(bar_o, (tcount - 1) & 1, ctl)) return;
        tc_fence_after_sync();
        __syncwarp();
        const float inv = 1.0f / (l_run + c_run);
        const bool row = p < a.band.L;
        const long long row_g = (long long)(w ? u.zq1 : u.zq) * a.band.L + (row ? buffer_row(a.store_geo, p) : 0);
        const bool poison = *reinterpret_cast<volatile int*>(smem + kSmemPoison + (ucount & 7) * 4) == (int)ucount + 1;
#pragma unroll 1
        for (int c = 0; c < kHd; c += 32) {
            uint32_t o[32];
            tmem_ld_32x32b_x32(tO + c, o);
            tmem_ld_wait(o);
            if (poison && row) {
                for (int jj = 0; jj < ntiles; ++jj) {
                    const int k0 = u.run.at(jj) * kTile;
                    if (whole_tile(a, u, k0)) continue;
                    for (int j = k0; j < k0 + kTile && j < a.band.L; ++j) {
                        if (!band_sees(a.band, p, j)) continue;
                        const __nv_bfloat16* v = a.v + ((long long)u.zk * a.band.L + buffer_row(a.geo, j)) * kHd + c;
#pragma unroll
                        for (int e = 0; e < 32; ++e) {
                            const float x = __bfloat162float(v[e]);
                            if (!(fabsf(x) <= 3.3895314e38f)) o[e] = __float_as_uint(__uint_as_float(o[e]) + x);  // past bf16's largest
                        }
                    }
                }
            }
            if (!row) continue;
            if (a.out_f32) {
                float4* dst = reinterpret_cast<float4*>(static_cast<float*>(a.out) + row_g * kHd + c);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    dst[e] = make_float4(__uint_as_float(o[4 * e]) * inv, __uint_as_float(o[4 * e + 1]) * inv,
                                         __uint_as_float(o[4 * e + 2]) * inv, __uint_as_float(o[4 * e + 3]) * inv);
            } else {
                uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + row_g * kHd + c);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    uint32_t pk[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        pk[i] = pack_bf16x2(__uint_as_float(o[8 * e + 2 * i]) * inv, __uint_as_float(o[8 * e + 2 * i + 1]) * inv);
                    dst[e] = make_uint4(pk[0], pk[1], pk[2], pk[3]);
                }
            }
        }
        if (row) a.lse[row_g] = (m_run + log2f(l_run)) * kLn2;
    }
}

// ------------------------------------------------------------------------------------------------
// loads (one thread)
// ------------------------------------------------------------------------------------------------
__device__ __forceinline__ void load_role(const FwdArgs& a, uint32_t sbase, const CUtensorMap* tmQ, const CUtensorMap* tmK,
                                          const CUtensorMap* tmV, const WaitCtl& ctl)
{
    auto bar = [&](int i) { return sbase + kSmemBar + 8u * (uint32_t)i; };
    tma_prefetch_desc(tmQ);
    tma_prefetch_desc(tmK);
    tma_prefetch_desc(tmV);
    uint32_t kc = 0, qc = 0, nk = 0, nv = 0;  // tiles; loads sent of Q, K and V
    bool ok = true;
    for (long long item = blockIdx.x; ok && item < a.units; item += gridDim.x) {
        const Unit u = unit_of(a, item);
        if (qc > 0 && !mbar_wait(bar(BAR_Q_EMPTY), (qc - 1) & 1, ctl)) break;
        mbar_arrive_expect_tx(bar(BAR_Q_FULL), 2 * kTileBytes);
        for (int w = 0; w < 2; ++w) {
            // (a second tile that lies behind the sequence is read from its end: zeros)
            const int row = (w ? u.p1 : u.p) < a.band.L ? window_tma_row(a.geo, w ? u.p1 : u.p) : a.geo.L;
            for (int half = 0; half < kHalves; ++half)
                tma_load_4d(sbase + kSmemQ + (uint32_t)(w * kHalves + half) * kHalfBytes, tmQ, bar(BAR_Q_FULL), half * 64, row, w ? u.zq1 : u.zq);
        }
        ++qc;
        const int ntiles = u.run.count();
        for (int jj = 0; jj < ntiles; ++jj, ++kc) {
            const int row = window_tma_row(a.geo, u.run.at(jj) * kTile);
            const int stage = (int)(kc % kStages);
            const uint32_t use = kc / kStages;
            if (use > 0 && !mbar_wait(bar(BAR_K_EMPTY + stage), (use - 1) & 1, ctl)) { ok = false; break; }
            mbar_arrive_expect_tx(bar(BAR_K_FULL + stage), kTileBytes);
            for (int half = 0; half < kHalves; ++half)
                tma_load_4d(sbase + kSmemK + (uint32_t)stage * kTileBytes + (uint32_t)half * kHalfBytes, tmK, bar(BAR_K_FULL + stage), half * 64,
                            row, u.zk);
            ++nk;
            if (use > 0 && !mbar_wait(bar(BAR_V_EMPTY + stage), (use - 1) & 1, ctl)) { ok = false; break; }
            mbar_arrive_expect_tx(bar(BAR_V_FULL + stage), kTileBytes);
            for (int half = 0; half < kHalves; ++half)
                tma_load_4d(sbase + kSmemV + (uint32_t)stage * kTileBytes + (uint32_t)half * kHalfBytes, tmV, bar(BAR_V_FULL + stage), half * 64,
                            row, u.zk);
            ++nv;
        }
    }
    // Copies still in flight land before the CTA's shared memory goes away.
    if (qc > 0) drain_wait(bar(BAR_Q_FULL), (qc - 1) & 1);
    for (uint32_t s = 1; s <= (uint32_t)kStages; ++s) {
        if (s <= nk) drain_wait(bar(BAR_K_FULL + (int)((nk - s) % kStages)), ((nk - s) / kStages) & 1);
        if (s <= nv) drain_wait(bar(BAR_V_FULL + (int)((nv - s) % kStages)), ((nv - s) / kStages) & 1);
    }
}

// ------------------------------------------------------------------------------------------------
// V of the tiles that are not wholly visible (warps 10-11)
// ------------------------------------------------------------------------------------------------
__device__ __forceinline__ void check_role(const FwdArgs& a, uint32_t sbase, uint8_t* smem, const WaitCtl& ctl)
{
    auto bar = [&](int i) { return sbase + kSmemBar + 8u * (uint32_t)i; };
    const int tid = threadIdx.x & 63, lane = threadIdx.x & 31;
    uint32_t kc = 0, ucount = 0;
    for (long long item = blockIdx.x; item < a.units; item += gridDim.x, ++ucount) {
        const Unit u = unit_of(a, item);
        const int ntiles = u.run.count();
        for (int jj = 0; jj < ntiles; ++jj, ++kc) {
            const int stage = (int)(kc % kStages);
            // (every tile is waited for: a phase left out would be taken for the one before it)
            const bool ok = mbar_wait(bar(BAR_V_FULL + stage), (kc / kStages) & 1, ctl);
            if (!__all_sync(0xffffffffu, ok)) return;
            if (!whole_tile(a, u, u.run.at(jj) * kTile)) {
                uint4* v = reinterpret_cast<uint4*>(smem + kSmemV + (uint32_t)stage * kTileBytes);
                bool hit = false;
#pragma unroll 4
                for (int i = tid; i < (int)(kTileBytes / 16); i += 64) {
                    uint4 x = v[i];
                    uint32_t* px = &x.x;
                    bool bad = false;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        if ((px[e] & 0x7f80u) == 0x7f80u) px[e] &= 0xffff0000u, bad = true;
                        if ((px[e] & 0x7f800000u) == 0x7f800000u) px[e] &= 0x0000ffffu, bad = true;
                    }
                    if (bad) v[i] = x;
                    hit |= bad;
                }
                if (hit) *reinterpret_cast<volatile int*>(smem + kSmemPoison + (ucount & 7) * 4) = (int)ucount + 1;
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(BAR_V_READY + stage));
            }
            if (lane == 0) mbar_arrive(bar(BAR_V_EMPTY + stage));
        }
    }
}

// ------------------------------------------------------------------------------------------------
// MMA issue (one thread)
// ------------------------------------------------------------------------------------------------
struct FwdDesc {
    uint32_t q, k, v;  // low words of the tiles' descriptors (K and V at stage 0)
};
constexpr uint32_t kDescHi = sdesc_sw128_hi(1024);

__device__ __forceinline__ void issue_qk(const FwdDesc& dsc, uint32_t tmem, int w, int stage)
{
    constexpr uint32_t idesc = idesc_bf16_f32(128, 128, false, false);
    const uint32_t kb = dsc.k + (uint32_t)stage * (kTileBytes >> 4);
#pragma unroll
    for (int kk = 0; kk < kHd / 16; ++kk) {
        const uint32_t off = (uint32_t)(kk >> 2) * kHalfBytes + (uint32_t)(kk & 3) * 32u;
        mma_ss(tmem + kColS0 + (uint32_t)w * 128, sdesc_at(dsc.q, (uint32_t)w * kTileBytes + off, kDescHi), sdesc_at(kb, off, kDescHi), idesc,
               kk > 0 ? 1u : 0u);
    }
}

__device__ __forceinline__ void issue_pv(const FwdDesc& dsc, uint32_t tmem, int w, int stage, bool accumulate)
{
    constexpr uint32_t idesc = idesc_bf16_f32(128, kHd, false, true);
    const uint32_t vb = dsc.v + (uint32_t)stage * (kTileBytes >> 4);
    const uint32_t acc0 = accumulate ? 1u : 0u;
#pragma unroll
    for (int kk = 0; kk < 8; ++kk)
        mma_ts(tmem + kColO0 + (uint32_t)w * 128, tmem + kColS0 + (uint32_t)w * 128 + (uint32_t)kk * 8, sdesc_at(vb, (uint32_t)kk * 2048u, kDescHi),
               idesc, kk > 0 ? 1u : acc0);
}

__device__ __forceinline__ void mma_role(const FwdArgs& a, uint32_t sbase, uint32_t tmem, const WaitCtl& ctl)
{
    auto bar = [&](int i) { return sbase + kSmemBar + 8u * (uint32_t)i; };
    FwdDesc dsc;
    dsc.q = sdesc_sw128_lo(sbase + kSmemQ, 16);
    dsc.k = sdesc_sw128_lo(sbase + kSmemK, 16);
    dsc.v = sdesc_sw128_lo(sbase + kSmemV, kHalfBytes);
    long long item = blockIdx.x;
    Unit u = unit_of(a, item);
    uint32_t kc = 0, qc = 0, checked = 0;  // checked: a parity bit per stage, of the tiles that warps 10-11 look through
    int jj = 0, ntiles = u.run.count();
    if (!mbar_wait(bar(BAR_Q_FULL), 0, ctl)) goto drain;
    if (!mbar_wait(bar(BAR_K_FULL + 0), 0, ctl)) goto drain;
    tc_fence_after_sync();
    issue_qk(dsc, tmem, 0, 0);
    tc_commit(bar(BAR_S_FULL + 0));
    issue_qk(dsc, tmem, 1, 0);
    tc_commit(bar(BAR_S_FULL + 1));
    tc_commit(bar(BAR_K_EMPTY + 0));
    if (ntiles == 1) tc_commit(bar(BAR_Q_EMPTY));
    while (true) {
        const int stage = (int)(kc % kStages), nstage = (int)((kc + 1) % kStages);
        const bool whole = whole_tile(a, u, u.run.at(jj) * kTile);
        int jn = jj + 1, nn = ntiles;
        bool has_next = true;
        Unit un = u;
        if (jn == ntiles) {
            jn = 0;
            item += gridDim.x;
            has_next = item < a.units;
            if (has_next) {
                un = unit_of(a, item);
                nn = un.run.count();
            }
        }
        if (whole) {
            if (!mbar_wait(bar(BAR_V_FULL + stage), (kc / kStages) & 1, ctl)) goto drain;
        } else {
            if (!mbar_wait(bar(BAR_V_READY + stage), (checked >> stage) & 1, ctl)) goto drain;
            checked ^= 1u << stage;
        }
        if (!mbar_wait(bar(BAR_P_FULL + 0), kc & 1, ctl)) goto drain;
        tc_fence_after_sync();
        issue_pv(dsc, tmem, 0, stage, jj > 0);
        tc_commit(bar(BAR_O_DONE + 0));
        if (has_next) {
            if (jn == 0) {
                ++qc;
                if (!mbar_wait(bar(BAR_Q_FULL), qc & 1, ctl)) goto drain;
            }
            if (!mbar_wait(bar(BAR_K_FULL + nstage), ((kc + 1) / kStages) & 1, ctl)) goto drain;
            tc_fence_after_sync();
            issue_qk(dsc, tmem, 0, nstage);
            tc_commit(bar(BAR_S_FULL + 0));
        }
        if (!mbar_wait(bar(BAR_P_FULL + 1), kc & 1, ctl)) goto drain;
        tc_fence_after_sync();
        issue_pv(dsc, tmem, 1, stage, jj > 0);
        tc_commit(bar(BAR_O_DONE + 1));
        tc_commit(bar(BAR_V_EMPTY + stage));
        if (!has_next) break;
        issue_qk(dsc, tmem, 1, nstage);
        tc_commit(bar(BAR_S_FULL + 1));
        tc_commit(bar(BAR_K_EMPTY + nstage));
        if (jn == nn - 1) tc_commit(bar(BAR_Q_EMPTY));
        u = un;
        ntiles = nn;
        jj = jn;
        ++kc;
    }
drain:
    tc_commit(bar(BAR_DRAIN));  // flips once every MMA issued by this thread has completed
    drain_wait(bar(BAR_DRAIN), 0);
}

__global__ void __launch_bounds__(kThreads, 1)
window_fwd_tc_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                     const FwdArgs a)
{
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    const int warp = threadIdx.x >> 5;
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kSmemAbort);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kSmemTmemSlot);

    if (threadIdx.x == 0) {
        for (int i = 0; i < BAR_COUNT; ++i) {
            uint32_t cnt = 1;
            if (i == BAR_P_FULL || i == BAR_P_FULL + 1) cnt = 4;
            if (i >= BAR_V_EMPTY && i < BAR_V_READY) cnt = 3;                 // the MMAs' commit, warps 10 and 11
            if (i >= BAR_V_READY && i < BAR_S_FULL) cnt = 2;
            mbar_init(sbase + kSmemBar + 8u * (uint32_t)i, cnt);
        }
        for (int i = 0; i < 8; ++i) reinterpret_cast<int*>(smem + kSmemPoison)[i] = 0;
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 9) {
        tmem_alloc(smem_u32(tmem_slot), kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    const WaitCtl ctl{abort_flag, a.status, kWaitLimitNs};

    // Registers: launched with 384 x 168 = 64512; softmax warpgroups 2 x 128 x 192, the others 128 x 120 = 64512.
    if (warp < 8)
        asm volatile("setmaxnreg.inc.sync.aligned.u32 192;" ::: "memory");
    else
        asm volatile("setmaxnreg.dec.sync.aligned.u32 120;" ::: "memory");

    if (warp < 8) {
        softmax_role(a, sbase, smem, tmem, ctl);
    } else if (warp == 8) {
        if ((threadIdx.x & 31) == 0) load_role(a, sbase, &tmQ, &tmK, &tmV, ctl);
    } else if (warp == 9) {
        if ((threadIdx.x & 31) == 0) mma_role(a, sbase, tmem, ctl);
    } else {
        check_role(a, sbase, smem, ctl);
    }

    tc_fence_before_sync();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, kTmemCols);
    }
}

}  // namespace

cudaError_t RA_WIN_FWD_LAUNCH(const WindowArgs& w, unsigned int* status, cudaStream_t s)
{
    CUtensorMap tq, tk, tv;
    if (!make_map(&tq, w.q, w.geo, (long long)w.B * w.H, kHd) || !make_map(&tk, w.k, w.geo, (long long)w.B * w.Hkv, kHd) ||
        !make_map(&tv, w.v, w.geo, (long long)w.B * w.Hkv, kHd))
        return cudaErrorInvalidValue;
    FwdArgs a;
    a.geo = w.geo;
    a.store_geo = w.store_geo;
    a.band = w.band;
    a.H = w.H;
    a.Hkv = w.Hkv;
    a.G = w.G;
    a.pair = w.G % 2 == 0;
    const int block = a.pair ? kTile : 2 * kTile;
    a.blocks = (w.band.L + block - 1) / block;
    a.rows = a.pair ? w.G / 2 : w.G;
    a.units = (long long)w.B * w.Hkv * a.blocks * a.rows;
    a.v = static_cast<const __nv_bfloat16*>(w.v);
    a.out = w.o;
    a.lse = w.lse;
    a.out_f32 = w.out_dtype == 0;
    a.status = status;
    a.scale_log2 = w.scale_log2;
    static std::mutex mu;
    static bool done[64];
    const cudaError_t e = allow_smem(window_fwd_tc_kernel, (int)kSmemBytes, mu, done);
    if (e != cudaSuccess) return e;
    const long long sms = device_sm_count();
    window_fwd_tc_kernel<<<(unsigned)(a.units < sms ? a.units : sms), kThreads, kSmemBytes, s>>>(tq, tk, tv, a);
    return cudaGetLastError();
}

}  // namespace ra
