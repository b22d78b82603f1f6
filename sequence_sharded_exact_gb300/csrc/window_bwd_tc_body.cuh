// window_bwd_tc_body.cuh -- tensor-core backward of the attention through a window (window.cuh) for sm_103a: bf16, head
// dim RA_WIN_HD (128 or 64), any length.  Compiled once per head dim (window_bwd_tc.cu: 128, window_bwd_tc_d64.cu: 64); the
// including file names the host entry point through RA_WIN_BWD_LAUNCH.
//
//   P = exp(s - lse),  dS = P (dO . v - D) / sqrt(d),  dV = P^T dO,  dK = dS^T Q,  dQ = dS K.
//
// One CTA per SM, persistent.  A work unit is one tile of 128 keys of one kv head and the query tiles that see it, head by
// head: W / 128 + 1 of them, so that units are alike in every layout (the tiles are runs of natural positions).  A tile with
// sinks is seen by all (later) queries: it is cut into segments about as long as the other units, each of which
// leaves its dK and dV in the workspace; a last kernel adds them in order.  Without that one CTA would walk the whole
// sequence for them.  The tiles of a last round that would leave half of the SMs idle are cut likewise.
//   * warp 12: TMA loads of the unit's K and V and, through 2 stages, of each query tile's Q (with its lse) and dO (with its
//     D); the vectors, in natural order and padded to whole tiles (lse with +infinity: those rows' P is 0), by bulk copy.
//   * warp 13: tcgen05.mma issue, per query tile t: dV += P^T_t dO_t (P^T from TMEM), S^T_{t+1} = K Q_{t+1}^T, dQ^T_t = K^T
//     dS^T_t, dK += dS^T_t Q_t (dS^T from shared memory for both), dP^T_{t+1} = V dO_{t+1}^T: the next tile's S^T runs while
//     the math warps compute dS^T of this one.
//   * warps 0-7 (two warpgroups of 64 query columns each, thread = key row): P^T = 2^(S^T c - lse2), to TMEM as bf16, then
//     dS^T, to shared memory; at a unit's end dK and dV.
//   * warps 8-11 (thread = head-dim index): dQ^T out of TMEM, added into the float32 accumulator (natural order, in the
//     workspace) with coalesced reductions, paced so that they leave room in the memory-instruction queue.
//   * TMEM columns (head dim 128): X = [0,128) S^T then P^T; Y = [128,256) dP^T, then dQ^T once phase B has read dP^T; dK
//     [256,384), dV [384,512).  Head dim 64: dQ^T has columns of its own (X 0, Y 128, dQ^T 256, dK 384, dV 448), and K is
//     loaded twice, so that dQ^T's rows 64-127 repeat rows 0-63 and all four dQ warps have 64 columns each to add.
//   * every wait is bounded; a wait that runs out sets the device status word and the CTA stops.
// dP^T waits for dQ^T's read-out where they share Y; the order in which dQ's sums arrive varies.
// P and dS go into the products as one bf16 value each (off by at most 2^-8, of either sign, so that it averages over a sum's
// terms); scores, P, D and all sums are float32.  What the rounding leaves as a second value would be three more products beside five.
//
// Measured with what comes before and after it (window_aux.cu), 32 : 8 heads of 128: 32K tokens, window 4096 4.8 ms (1.06 PFLOP/s;
// this kernel 4.3), 64K tokens 8.8 ms, window 1024 2.92 ms without sinks and 3.25 with 4 (whose tile is seen by all 512 query
// tiles of a head: 11 % more pairs, of which few count).  dQ's reductions bound it.
#include <cuda_bf16.h>
#include <math.h>

#include "window_tc.cuh"

namespace ra {
namespace {

constexpr int kKT = kWinTile;   // keys of a tile
constexpr int kQT = kWinTile;   // queries of a tile
constexpr int kHd = RA_WIN_HD;
static_assert(kHd == 128 || kHd == 64, "head dim");
constexpr int kHalves = kHd / 64;  // 128-byte-swizzle boxes (64 bf16 head-dim columns) per row
constexpr int kStages = 2;     // query-tile stages (Q + lse, dO + D)
constexpr int kThreads = 512;  // 16 warps: 0-7 math, 8-11 dQ, 12 TMA loads, 13 MMA, 14-15 idle
constexpr uint32_t kHalf = 128 * 128;            // 16 KB: 128 rows x 64 bf16 columns
constexpr uint32_t kTileBytes = kHalves * kHalf; // a 128-row K, V, Q or dO tile (32 KB at d = 128)
constexpr uint32_t kDsBytes = 2 * kHalf;         // dS^T: 128 keys x 128 queries (bf16)
constexpr uint32_t kVecBytes = kQT * 4;          // lse or D of one query tile (float32)

// Head dim 64 has TMEM and shared memory to spare: dQ^T gets columns of its own (so the next dP^T
// need not wait for the dQ read-out), and K is loaded twice, back to back, so that the M = 128
// product dQ^T = K^T dS^T computes its rows 0-63 twice and all four dQ warps can reduce (rows
// 0-63 give the query columns 0-63, rows 64-127 the columns 64-127).
constexpr bool kD64 = kHd == 64;
constexpr uint32_t kSmemK = 0;                                   // d = 64: K, then K again
constexpr uint32_t kSmemV = kSmemK + (kD64 ? 2 : 1) * kTileBytes;
constexpr uint32_t kSmemQ = kSmemV + kTileBytes;                 // kStages x 32 KB
constexpr uint32_t kSmemDO = kSmemQ + kStages * kTileBytes;      // kStages x 32 KB
constexpr uint32_t kSmemDS = kSmemDO + kStages * kTileBytes;     // dS^T: 2 query blocks x 128 keys x 128 B
constexpr uint32_t kSmemLse = kSmemDS + kDsBytes;                // kStages x 512 B
constexpr uint32_t kSmemD = kSmemLse + kStages * kVecBytes;      // kStages x 512 B
constexpr uint32_t kSmemBar = kSmemD + kStages * kVecBytes;

enum : int {
    BAR_KV_FULL = 0,
    BAR_KV_EMPTY,
    BAR_Q_FULL,                           // kStages: Q tile and its lse landed
    BAR_DO_FULL = BAR_Q_FULL + kStages,   // kStages: dO tile and its D landed
    BAR_Q_EMPTY = BAR_DO_FULL + kStages,  // kStages: S^T and dK have read the Q tile
    BAR_DO_EMPTY = BAR_Q_EMPTY + kStages, // kStages: dP^T and dV have read the dO tile
    BAR_ST_FULL = BAR_DO_EMPTY + kStages,
    BAR_DPT_FULL,
    BAR_P_READY,   // 8 math warps
    BAR_DS_READY,  // 8 math warps
    BAR_DQ_FULL,
    BAR_DQ_FREE,   // 4 dQ warps
    BAR_ACC_FULL,
    BAR_ACC_FREE,  // 8 math warps
    BAR_DRAIN,
    BAR_COUNT
};

constexpr uint32_t kSmemTmemSlot = kSmemBar + BAR_COUNT * 8;
constexpr uint32_t kSmemAbort = kSmemTmemSlot + 8;
constexpr uint32_t kSmemBytes = kSmemAbort + 8;
// The base of dynamic shared memory sits right after the 1 KB the system reserves, so it is
// 1024-byte aligned (the 128-byte swizzle atoms need that); the kernel checks it and stops with
// RA_DEVICE_LAYOUT if not, instead of reserving 1 KB of slack that this layout does not have.
static_assert(kSmemBytes <= 232448, "shared memory budget");

constexpr uint32_t kColX = 0, kColY = 128;
constexpr uint32_t kColDQ = kD64 ? 256 : kColY;  // d = 128: dQ^T reuses Y once phase B has read dP^T
constexpr uint32_t kColDK = kD64 ? 384 : 256, kColDV = kD64 ? 448 : 384;
constexpr uint64_t kWaitLimitNs = 4000000000ull;

struct BwdArgs {
    Geometry geo, store_geo;  // of the loads; of the gradients' rows
    Band band;
    int G, T;          // query heads of a kv head; tiles of the sequence
    int sink_tiles, segs;  // tiles that hold sinks; segments of each of them (1: none is cut)
    unsigned sink_items, items;
    unsigned per;      // items of a kv head, and the sinks' segments of all items, 2^-32 (not kTail)
    unsigned long long share;
    unsigned whole;    // of the other tiles, those with a unit of their own; the rest have tail_segs
    int tail_segs;
    const float* lse2;  // -lse log2(e), [B H][T 128]
    const float* Dv;    // [B H][T 128]
    float* dq_acc;      // [B H][T 128][d]
    void* dk;
    void* dv;
    float* part;        // [segments][2][128][d]: their dK, dV
    int grad_bf16;
    unsigned int* status;
    float scale, scale_log2;
};

struct KvUnit {
    int zk;         // b * Hkv + kv head
    int k0;         // first key's position
    int t0, nt;     // query tiles [t0, t0 + nt) of every head
    int from;       // kTail: the unit's first of these G * nt, head by head
    int ntiles;     // and how many it has (otherwise all)
    long long slot; // segment's place in `part`, or -1
};

// Items, kTail: the segments of the sinks' tiles, then the other tiles, and the segments of those of the last round.  (A kernel
// without these is compiled apart: their code in it costs a unit 0.5 to 1 us.)  Otherwise, kv head by kv head, the tiles in
// order, with the segments of the sinks' spread evenly among them: segment s meets the query tiles that its neighbours do, which
// are then in L2 (64K tokens of 32 : 8 heads of 128, 4 sinks: all segments first, Q, dO and dQ came from memory once more:
// window 1024 3.50 ms in place of 3.25, window 128 1.85 in place of 1.75).
template <bool kTail>
__device__ __forceinline__ KvUnit unit_of(const BwdArgs& a, unsigned item)
{
    KvUnit u;
    bool sink;
    int tile, seg = 0, cut = 0;
    if constexpr (!kTail) {
        u.zk = (int)(item / a.per);
        const unsigned x = item - (unsigned)u.zk * a.per;
        const unsigned before = (unsigned)(x * a.share >> 32);  // segments before it
        sink = (unsigned)((x + 1) * a.share >> 32) > before;
        if (sink) {
            seg = (int)(before / (unsigned)a.sink_tiles);
            tile = (int)(before - (unsigned)(seg * a.sink_tiles));
        } else {
            tile = a.sink_tiles + (int)(x - before);
        }
    } else if (sink = item < a.sink_items; sink) {
        const unsigned per = (unsigned)(a.sink_tiles * a.segs), x = item % per;
        u.zk = (int)(item / per);
        tile = (int)(x / (unsigned)a.segs);
        seg = (int)(x % (unsigned)a.segs);
    } else {
        const unsigned per = (unsigned)(a.T - a.sink_tiles);
        unsigned x = item - a.sink_items;
        if (x >= a.whole) {
            cut = 1 + (int)((x - a.whole) % (unsigned)a.tail_segs);
            x = a.whole + (x - a.whole) / (unsigned)a.tail_segs;
        }
        u.zk = (int)(x / per);
        tile = a.sink_tiles + (int)(x % per);
    }
    u.k0 = tile * kKT;
    const QueryRun r = query_tiles(a.band, u.k0, kKT, kQT);
    const int n = r.last - r.first, segs = sink ? a.segs : 1;
    const int from = (int)((long long)n * seg / segs), to = (int)((long long)n * (seg + 1) / segs);
    u.t0 = r.first + from;
    u.nt = to - from;
    u.from = 0;
    u.ntiles = u.nt * a.G;
    u.slot = sink && a.segs > 1 ? ((long long)u.zk * a.sink_tiles + tile) * a.segs + seg : -1LL;
    if (kTail && cut) {
        const long long all = u.ntiles;
        u.from = (int)(all * (cut - 1) / a.tail_segs);
        u.ntiles = (int)(all * cut / a.tail_segs) - u.from;
        u.slot = (a.segs > 1 ? (long long)a.sink_items : 0) + (item - a.sink_items - a.whole);
    }
    return u;
}

// The t-th query tile of a unit: head within the group, and first position.
template <bool kTail>
struct QWalk {
    int hh = 0, t = 0;
    __device__ __forceinline__ explicit QWalk(const KvUnit& u)
    {
        if (kTail && u.from > 0) {
            hh = u.from / u.nt;
            t = u.from % u.nt;
        }
    }
    __device__ __forceinline__ void next(const KvUnit& u, int& head, int& q0)
    {
        head = hh;
        q0 = (u.t0 + t) * kQT;
        if (++t == u.nt) {
            t = 0;
            ++hh;
        }
    }
};

// 128-byte-swizzled address of 16-byte chunk `ch` of row `r` in a region of 128-byte rows.
__device__ __forceinline__ uint32_t sw128(uint32_t region, int r, int ch)
{
    return region + (uint32_t)r * 128u + ((uint32_t)(ch ^ (r & 7)) << 4);
}

// 16 bytes of shared memory (every lane of a warp reads the same words: one broadcast)
__device__ __forceinline__ float4 lds_f4(uint32_t addr)
{
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr)
                 : "memory");
    return v;
}

__device__ __forceinline__ uint32_t stage_of(uint32_t x) { return x % kStages; }
__device__ __forceinline__ uint32_t phase_of(uint32_t x) { return (x / kStages) & 1u; }

// ------------------------------------------------------------------------------------------------
// math warpgroups
// ------------------------------------------------------------------------------------------------
// Phase A: P^T = 2^(S^T c - lse2) for the warpgroup's query columns [64w, 64w+64), kept in p[] for
// phase B and written to TMEM as bf16 pairs (columns [64w, 64w+32) of X) for dV += P^T dO.
// seen: a bit per column; hidden ones have P = 0.
template <bool kWhole>
__device__ __forceinline__ void phase_a(const BwdArgs& a, uint32_t tmem, uint32_t lane_off, int w, const uint32_t (&seen)[2],
                                        uint32_t s_lse, float (&p)[64])
{
    const uint32_t tx = tmem + lane_off + kColX + (uint32_t)w * 64;
    uint32_t sv[64];
    tmem_ld_32x32b_x64(tx, sv);
    tmem_ld_wait(sv);
    uint32_t pk[32];
    const float2 sc2 = make_float2(a.scale_log2, a.scale_log2);
#pragma unroll
    for (int e4 = 0; e4 < 16; ++e4) {
        const float4 l4 = lds_f4(s_lse + (uint32_t)(w * 64 + e4 * 4) * 4u);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int col = e4 * 4 + h * 2;
            const uint32_t x0 = sv[col];
            const uint32_t x1 = sv[col + 1];
            const float2 lq = h == 0 ? make_float2(l4.x, l4.y) : make_float2(l4.z, l4.w);
            const float2 xv = fma2(make_float2(__uint_as_float(x0), __uint_as_float(x1)), sc2, lq);
            float p0 = ex2_approx(xv.x), p1 = ex2_approx(xv.y);
            if (!kWhole && !(seen[col >> 5] & (1u << (col & 31)))) p0 = 0.f;
            if (!kWhole && !(seen[col >> 5] & (2u << (col & 31)))) p1 = 0.f;
            p[col] = p0;
            p[col + 1] = p1;
            pk[e4 * 2 + h] = pack_bf16x2(p0, p1);
        }
    }
    tmem_st_32x32b_x32(tx, pk);
    tmem_st_wait();
}

// Phase B: dS^T = P^T (dP^T - D) / sqrt(d) for the warpgroup's query columns, in two halves of 32,
// -> 128-byte-swizzled shared memory (query block w: key row r, its 128-byte row), where it is
// both the A operand of dK (K-major: key rows, query columns contiguous) and the B operand of
// dQ^T (N-major).
__device__ __forceinline__ void phase_b(const BwdArgs& a, uint32_t sbase, uint32_t tmem, uint32_t lane_off, int w,
                                        int r, uint32_t s_d, const float (&p)[64])
{
    const uint32_t ty = tmem + lane_off + kColY + (uint32_t)w * 64;
    const float2 sc = make_float2(a.scale, a.scale), neg1 = make_float2(-1.f, -1.f);
    const uint32_t region = sbase + kSmemDS + (uint32_t)w * kHalf;
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
        uint32_t dp[32];
        tmem_ld_32x32b_x32(ty + (uint32_t)hf * 32, dp);
        tmem_ld_wait(dp);
        uint32_t dsp[16];
#pragma unroll
        for (int e4 = 0; e4 < 8; ++e4) {
            const float4 dq = lds_f4(s_d + (uint32_t)(w * 64 + hf * 32 + e4 * 4) * 4u);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int col = e4 * 4 + h * 2;
                const int pc = hf * 32 + col;
                const float2 d2 = h == 0 ? make_float2(dq.x, dq.y) : make_float2(dq.z, dq.w);
                // dS = (dP - D) * P * scale
                const float2 t = fma2(d2, neg1, make_float2(__uint_as_float(dp[col]), __uint_as_float(dp[col + 1])));
                const float2 ds = mul2(t, mul2(make_float2(p[pc], p[pc + 1]), sc));
                dsp[e4 * 2 + h] = pack_bf16x2(ds.x, ds.y);
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(sw128(region, r, hf * 4 + j)),
                         "r"(dsp[4 * j]), "r"(dsp[4 * j + 1]), "r"(dsp[4 * j + 2]), "r"(dsp[4 * j + 3])
                         : "memory");
    }
}

// Per query tile t the warpgroups run phase A then phase B; dQ^T is the dQ warps' business.
template <bool kTail>
__device__ __forceinline__ void math_role(const BwdArgs& a, uint32_t sbase, uint32_t tmem, const WaitCtl& ctl)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int w = warp >> 2;                    // query-column half owned by this warpgroup
    const int r = (warp & 3) * 32 + lane;       // TMEM lane = key row
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    auto bar = [&](int i) { return sbase + kSmemBar + 8u * (uint32_t)i; };
    uint32_t gt = 0, uc = 0;
    for (unsigned item = blockIdx.x; item < a.items; item += gridDim.x) {
        {
            const KvUnit u = unit_of<kTail>(a, item);
            if (u.ntiles == 0) continue;
            QWalk<kTail> walk(u);
            for (int t = 0; t < u.ntiles; ++t, ++gt) {
                int hh, q0;
                walk.next(u, hh, q0);
                const bool whole = band_tile_whole(a.band, q0, kQT, u.k0, kKT);
                uint32_t seen[2] = {~0u, ~0u};
                if (!whole) {
                    const Seen v = seen_queries(a.band, u.k0 + r, q0);
                    seen[0] = v.word(64 * w);
                    seen[1] = v.word(64 * w + 32);
                }
                const uint32_t st = stage_of(gt), sp = phase_of(gt);
                float p[64];
                if (!mbar_wait(bar(BAR_ST_FULL), gt & 1, ctl)) goto done;
                if (!mbar_wait(bar(BAR_Q_FULL + (int)st), sp, ctl)) goto done;
                tc_fence_after_sync();
                __syncwarp();
                if (whole)
                    phase_a<true>(a, tmem, lane_off, w, seen, sbase + kSmemLse + st * kVecBytes, p);
                else
                    phase_a<false>(a, tmem, lane_off, w, seen, sbase + kSmemLse + st * kVecBytes, p);
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(BAR_P_READY));
                if (!mbar_wait(bar(BAR_DPT_FULL), gt & 1, ctl)) goto done;
                if (!mbar_wait(bar(BAR_DO_FULL + (int)st), sp, ctl)) goto done;
                tc_fence_after_sync();
                __syncwarp();
                phase_b(a, sbase, tmem, lane_off, w, r, sbase + kSmemD + st * kVecBytes, p);
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(BAR_DS_READY));
            }
            // epilogue: dK, dV of key row r, columns [w d/2, (w+1) d/2)
            if (!mbar_wait(bar(BAR_ACC_FULL), uc & 1, ctl)) goto done;
            tc_fence_after_sync();
            __syncwarp();
            const bool row = u.k0 + r < a.band.L;
            const long long krow = (long long)u.zk * a.band.L + (row ? buffer_row(a.store_geo, u.k0 + r) : 0);
#pragma unroll 1
            for (int which = 0; which < 2; ++which) {
                const uint32_t col = (which == 0 ? kColDK : kColDV) + (uint32_t)w * (kHd / 2);
                void* base = which == 0 ? a.dk : a.dv;
#pragma unroll 1
                for (int c = 0; c < kHd / 64; ++c) {
                    uint32_t x[32];
                    __syncwarp();  // the lanes of keys behind the sequence have gone ahead
                    tmem_ld_32x32b_x32(tmem + lane_off + col + c * 32, x);
                    tmem_ld_wait(x);
                    const int at = w * (kHd / 2) + c * 32;
                    if (u.slot < 0 && a.grad_bf16) {
                        uint4* d = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(base) + krow * kHd + at);
                        if (!row) continue;
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            d[e] = make_uint4(pack_bf16x2(__uint_as_float(x[8 * e]), __uint_as_float(x[8 * e + 1])),
                                              pack_bf16x2(__uint_as_float(x[8 * e + 2]), __uint_as_float(x[8 * e + 3])),
                                              pack_bf16x2(__uint_as_float(x[8 * e + 4]), __uint_as_float(x[8 * e + 5])),
                                              pack_bf16x2(__uint_as_float(x[8 * e + 6]), __uint_as_float(x[8 * e + 7])));
                    } else {
                        float4* d = reinterpret_cast<float4*>(u.slot < 0 ? static_cast<float*>(base) + krow * kHd + at
                                                                         : a.part + ((u.slot * 2 + which) * kKT + r) * kHd + at);
                        if (!row) continue;
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            d[e] = make_float4(__uint_as_float(x[4 * e]), __uint_as_float(x[4 * e + 1]),
                                               __uint_as_float(x[4 * e + 2]), __uint_as_float(x[4 * e + 3]));
                    }
                }
            }
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(BAR_ACC_FREE));
            ++uc;
        }
    }
done:
    return;
}

// ------------------------------------------------------------------------------------------------
// dQ warpgroup (warps 8-11, thread = head-dim index): dQ^T of each query tile out of TMEM, then
// added into the float32 accumulator, [B H][T 128][d] in natural order.  All four warps reduce: at d = 64, where rows 64-127
// repeat rows 0-63 (K lies twice), warps 8-9 the query columns 0-63 and warps 10-11 the columns 64-127.  Its columns are freed
// as soon as they are in registers, so the next dP^T does not wait for the reductions.
// ------------------------------------------------------------------------------------------------
__device__ __forceinline__ void red_add_f32(float* addr, float v)
{
    asm volatile("red.global.add.f32 [%0], %1;" ::"l"(addr), "f"(v) : "memory");
}

// The reductions go out in 16 groups of 8 per thread with a pause between groups: issued at once they fill the SM's
// memory-instruction queue, and every other warp's shared-memory and barrier traffic waits behind them (64K tokens, window
// 4096: 9.44 ms without pauses, 9.16 with 60 ns, 8.93 with 80, 8.84 with 100 and 40 where the next tile is already
// waiting; at d = 64 80 and none then are better: 16K tokens, 512 on both sides 530 us in place of 540).
// They are what bounds the kernel: without them it takes 6.95.  Bulk reductions out of shared memory (16 KB at a time) took
// 8.54 there, but need dO's second stage for their room (8.14 without the reductions themselves) and made head dim 64 a
// fifth slower (530 -> 652 us), since the products' operands take most of what shared memory serves.
__device__ __forceinline__ void red_group(float* dst, const uint32_t (&x)[64], int c0, uint32_t gap_ns)
{
#pragma unroll
    for (int g = 0; g < 8; ++g) {
        if (gap_ns) __nanosleep(gap_ns);
#pragma unroll
        for (int c = 0; c < 8; ++c) red_add_f32(dst + (long long)(c0 + 8 * g + c) * kHd, __uint_as_float(x[8 * g + c]));
    }
}

template <bool kTail>
__device__ __forceinline__ void dq_role(const BwdArgs& a, uint32_t sbase, uint32_t tmem, const WaitCtl& ctl)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int dcol = (warp & 3) * 32 + lane;  // TMEM lane = head-dim index
    const uint32_t ty = tmem + ((uint32_t)((warp & 3) * 32) << 16) + kColDQ;
    const uint32_t dq_c0 = kD64 && (warp & 3) >= 2 ? 64u : 0u;  // d = 64: this warp's query columns
    auto bar = [&](int i) { return sbase + kSmemBar + 8u * (uint32_t)i; };
    uint32_t gt = 0;
    for (unsigned item = blockIdx.x; item < a.items; item += gridDim.x) {
        {
            const KvUnit u = unit_of<kTail>(a, item);
            if (u.ntiles == 0) continue;
            QWalk<kTail> walk(u);
            for (int t = 0; t < u.ntiles; ++t, ++gt) {
                int hh, q0;
                walk.next(u, hh, q0);
                const bool behind = __shfl_sync(0xffffffffu, mbar_test_wait(bar(BAR_DQ_FULL), gt & 1), 0) != 0;
                const uint32_t gap_ns = kD64 ? (behind ? 0u : 80u) : (behind ? 40u : 100u);
                if (!mbar_wait(bar(BAR_DQ_FULL), gt & 1, ctl)) return;
                tc_fence_after_sync();
                __syncwarp();
                if constexpr (kD64) {
                    // rows 0-63 (warps 8-9): query columns 0-63; rows 64-127 (warps 10-11, the same
                    // values from the second copy of K): query columns 64-127
                    uint32_t xa[64], xb[64];
                    tmem_ld_32x32b_x64(ty, xa);
                    tmem_ld_32x32b_x64(ty + 64, xb);
                    tmem_ld_wait(xa);
                    tmem_ld_wait(xb);
                    tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(BAR_DQ_FREE));
                    const long long zq = (long long)u.zk * a.G + hh;
                    float* dst = a.dq_acc + (zq * a.T * kQT + q0) * kHd + (dcol & 63);
                    if (dq_c0 == 0)
                        red_group(dst, xa, 0, gap_ns);
                    else
                        red_group(dst, xb, 64, gap_ns);
                } else {
                    uint32_t xa[64], xb[64];
                    tmem_ld_32x32b_x64(ty, xa);
                    tmem_ld_32x32b_x64(ty + 64, xb);
                    tmem_ld_wait(xa);
                    tmem_ld_wait(xb);
                    tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(BAR_DQ_FREE));
                    const long long zq = (long long)u.zk * a.G + hh;
                    float* dst = a.dq_acc + (zq * a.T * kQT + q0) * kHd + dcol;
                    red_group(dst, xa, 0, gap_ns);
                    red_group(dst, xb, 64, gap_ns);
                }
            }
        }
    }
}

// ------------------------------------------------------------------------------------------------
// TMA producer (one thread)
// ------------------------------------------------------------------------------------------------
template <bool kTail>
__device__ __forceinline__ void producer_role(const BwdArgs& a, uint32_t sbase, const CUtensorMap* tmQ,
                                              const CUtensorMap* tmK, const CUtensorMap* tmV,
                                              const CUtensorMap* tmDO, const WaitCtl& ctl)
{
    auto bar = [&](int i) { return sbase + kSmemBar + 8u * (uint32_t)i; };
    tma_prefetch_desc(tmQ);
    tma_prefetch_desc(tmK);
    tma_prefetch_desc(tmV);
    tma_prefetch_desc(tmDO);
    uint32_t uc = 0, qc = 0, nq = 0, nd = 0;  // units, query tiles; loads sent of Q and dO
    bool ok = true;
    for (unsigned item = blockIdx.x; ok && item < a.items; item += gridDim.x) {
        const KvUnit u = unit_of<kTail>(a, item);
        if (u.ntiles == 0) continue;
        if (uc > 0 && !mbar_wait(bar(BAR_KV_EMPTY), (uc - 1) & 1, ctl)) break;
        const int krow = window_tma_row(a.geo, u.k0);
        mbar_arrive_expect_tx(bar(BAR_KV_FULL), (kD64 ? 3 : 2) * kTileBytes);
#pragma unroll
        for (int half = 0; half < kHalves; ++half) {
            tma_load_4d(sbase + kSmemK + (uint32_t)half * kHalf, tmK, bar(BAR_KV_FULL), half * 64, krow, u.zk);
            tma_load_4d(sbase + kSmemV + (uint32_t)half * kHalf, tmV, bar(BAR_KV_FULL), half * 64, krow, u.zk);
        }
        if constexpr (kD64) tma_load_4d(sbase + kSmemK + kTileBytes, tmK, bar(BAR_KV_FULL), 0, krow, u.zk);
        ++uc;
        QWalk<kTail> walk(u);
        for (int t = 0; t < u.ntiles; ++t, ++qc) {
            int hh, q0;
            walk.next(u, hh, q0);
            const uint32_t st = stage_of(qc), use = qc / kStages;
            const int zq = u.zk * a.G + hh, qrow = window_tma_row(a.geo, q0);
            const long long qbase = (long long)zq * a.T * kQT + q0;
            // Q with its lse first: S^T and phase A need them; dO and D follow
            if (use > 0 && !mbar_wait(bar(BAR_Q_EMPTY + (int)st), (use - 1) & 1, ctl)) { ok = false; break; }
            mbar_arrive_expect_tx(bar(BAR_Q_FULL + (int)st), kTileBytes + kVecBytes);
#pragma unroll
            for (int half = 0; half < kHalves; ++half)
                tma_load_4d(sbase + kSmemQ + st * kTileBytes + (uint32_t)half * kHalf, tmQ, bar(BAR_Q_FULL + (int)st), half * 64, qrow, zq);
            bulk_load_1d(sbase + kSmemLse + st * kVecBytes, a.lse2 + qbase, kVecBytes, bar(BAR_Q_FULL + (int)st));
            ++nq;
            if (use > 0 && !mbar_wait(bar(BAR_DO_EMPTY + (int)st), (use - 1) & 1, ctl)) { ok = false; break; }
            mbar_arrive_expect_tx(bar(BAR_DO_FULL + (int)st), kTileBytes + kVecBytes);
#pragma unroll
            for (int half = 0; half < kHalves; ++half)
                tma_load_4d(sbase + kSmemDO + st * kTileBytes + (uint32_t)half * kHalf, tmDO, bar(BAR_DO_FULL + (int)st), half * 64, qrow, zq);
            bulk_load_1d(sbase + kSmemD + st * kVecBytes, a.Dv + qbase, kVecBytes, bar(BAR_DO_FULL + (int)st));
            ++nd;
        }
    }
    // Copies still in flight must land before the CTA's shared memory goes away.
    if (uc > 0) drain_wait(bar(BAR_KV_FULL), (uc - 1) & 1);
    for (uint32_t s = 1; s <= (uint32_t)kStages; ++s) {
        if (s <= nq) drain_wait(bar(BAR_Q_FULL + (int)stage_of(nq - s)), phase_of(nq - s));
        if (s <= nd) drain_wait(bar(BAR_DO_FULL + (int)stage_of(nd - s)), phase_of(nd - s));
    }
}

// ------------------------------------------------------------------------------------------------
// MMA issue (one warp, one lane of it)
// ------------------------------------------------------------------------------------------------
// Operand descriptors, as the low words of their shared-memory descriptors (query-tile operands
// at stage 0): K-major views have LBO 16, N- or M-major views LBO = the distance between their
// 64-element column blocks (16 KB everywhere here).  A stage or a k-step is a constant added.
// At d = 64 the M-major K view's second block (rows 64-127 of dQ^T) is K's second copy, which follows the first in shared
// memory: rows 64-127 are rows 0-63 again, and warps 10-11 read them for the query columns 64-127.
struct BwdDesc {
    uint32_t k_k, v_k;    // K and V tiles, K-major (A of S^T and dP^T)
    uint32_t k_m;         // K tile, M-major (A of dQ^T = K^T dS^T)
    uint32_t q_k, do_k;   // Q and dO tiles, K-major (B of S^T and dP^T)
    uint32_t q_n, do_n;   // Q and dO tiles, N-major (B of dK and dV)
    uint32_t ds_n;        // dS^T, N-major (B of dQ^T)
    uint32_t ds_k;        // dS^T, K-major (A of dK)
};
constexpr uint32_t kDescHi = sdesc_sw128_hi(1024);
constexpr uint32_t kId = idesc_bf16_f32(128, 128, false, false);     // S^T, dP^T: both K-major
constexpr uint32_t kIdTs = idesc_bf16_f32(128, kHd, false, true);    // dV (A TMEM), dK (A K-major): B N-major
constexpr uint32_t kIdDQ = idesc_bf16_f32(128, 128, true, true);     // dQ^T: A M-major, B N-major

__device__ __forceinline__ BwdDesc make_desc(uint32_t sbase)
{
    BwdDesc d;
    d.k_k = sdesc_sw128_lo(sbase + kSmemK, 16);
    d.v_k = sdesc_sw128_lo(sbase + kSmemV, 16);
    d.k_m = sdesc_sw128_lo(sbase + kSmemK, kHalf);
    d.q_k = sdesc_sw128_lo(sbase + kSmemQ, 16);
    d.do_k = sdesc_sw128_lo(sbase + kSmemDO, 16);
    d.q_n = sdesc_sw128_lo(sbase + kSmemQ, kHalf);
    d.do_n = sdesc_sw128_lo(sbase + kSmemDO, kHalf);
    d.ds_n = sdesc_sw128_lo(sbase + kSmemDS, kHalf);
    d.ds_k = sdesc_sw128_lo(sbase + kSmemDS, 16);
    return d;
}

// TMEM column of the A operand for k-step kk of a product over the 128 query columns: the bf16
// pairs of warpgroup w's columns [64w, 64w+64) sit at [64w, 64w+32) of the region.
__device__ __forceinline__ uint32_t a_col(int kk) { return (uint32_t)(kk >> 2) * 64u + (uint32_t)(kk & 3) * 8u; }

// D (tmem) = A B over the head dimension, both K-major in shared memory (S^T = K Q^T, dP^T = V dO^T)
__device__ __forceinline__ void issue_kmajor(uint32_t lead, uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo)
{
#pragma unroll
    for (int kk = 0; kk < kHd / 16; ++kk) {
        const uint32_t off = (uint32_t)(kk >> 2) * kHalf + (uint32_t)(kk & 3) * 32u;
        lead_mma_ss(lead, d_tmem, sdesc_at(a_lo, off, kDescHi), sdesc_at(b_lo, off, kDescHi), kId, kk > 0);
    }
}

// acc (tmem) += A (tmem, bf16 pairs) B over the 128 query rows, B N-major in shared memory
// (dV += P^T dO)
__device__ __forceinline__ void issue_ts(uint32_t lead, uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo, bool accumulate)
{
    const uint32_t acc0 = accumulate ? 1u : 0u;
#pragma unroll
    for (int kk = 0; kk < 8; ++kk)
        lead_mma_ts(lead, d_tmem, a_tmem + a_col(kk), sdesc_at(b_lo, (uint32_t)kk * 2048u, kDescHi), kIdTs, kk > 0 ? 1u : acc0);
}

// dK += dS^T Q over the 128 query rows: A = dS^T K-major (query block kk / 4, 16 queries = 32 bytes
// of each 128-byte key row), B = Q N-major
__device__ __forceinline__ void issue_dk(uint32_t lead, uint32_t tmem, const BwdDesc& dsc, uint32_t q_lo, bool accumulate)
{
    const uint32_t a_lo = dsc.ds_k, b_lo = q_lo;
    const uint32_t acc0 = accumulate ? 1u : 0u;
#pragma unroll
    for (int kk = 0; kk < 8; ++kk)
        lead_mma_ss(lead, tmem + kColDK, sdesc_at(a_lo, (uint32_t)(kk >> 2) * kHalf + (uint32_t)(kk & 3) * 32u, kDescHi),
               sdesc_at(b_lo, (uint32_t)kk * 2048u, kDescHi), kIdTs, kk > 0 ? 1u : acc0);
}

// dQ^T = K^T dS^T over the 128 key rows
__device__ __forceinline__ void issue_dq(uint32_t lead, uint32_t tmem, const BwdDesc& dsc)
{
    const uint32_t a_lo = dsc.k_m, b_lo = dsc.ds_n;
#pragma unroll
    for (int kk = 0; kk < 8; ++kk)
        lead_mma_ss(lead, tmem + kColDQ, sdesc_at(a_lo, (uint32_t)kk * 2048u, kDescHi), sdesc_at(b_lo, (uint32_t)kk * 2048u, kDescHi),
               kIdDQ, kk > 0);
}

template <bool kTail>
__device__ __forceinline__ void mma_role(const BwdArgs& a, uint32_t sbase, uint32_t tmem, const WaitCtl& ctl)
{
    auto bar = [&](int i) { return sbase + kSmemBar + 8u * (uint32_t)i; };
    constexpr uint32_t kStageLo = kTileBytes >> 4;  // one query-tile stage, in descriptor units
    uint32_t gt = 0, uc = 0;
    bool issued = false;
    const uint32_t lead = elect();
    tmem = __shfl_sync(0xffffffffu, tmem, 0);
    const BwdDesc dsc = make_desc(sbase);
    for (unsigned item = blockIdx.x; item < a.items; item += gridDim.x) {
        {
            const KvUnit u = unit_of<kTail>(a, item);
            if (u.ntiles == 0) continue;
            if (!warp_wait(bar(BAR_KV_FULL), uc & 1, ctl)) goto drain;
            issued = true;
            tc_fence_after_sync();
            // the unit's first S^T and dP^T; later ones are issued one tile ahead (below)
            {
                const uint32_t st = stage_of(gt), sp = phase_of(gt);
                if (!warp_wait(bar(BAR_Q_FULL + (int)st), sp, ctl)) goto drain;
                tc_fence_after_sync();
                issue_kmajor(lead, tmem + kColX, dsc.k_k, dsc.q_k + st * kStageLo);
                lead_commit(lead, bar(BAR_ST_FULL));
                // Y: the previous tile's dQ^T must have been read out (d = 128, where it shares Y)
                if (!kD64 && gt > 0 && !warp_wait(bar(BAR_DQ_FREE), (gt - 1) & 1, ctl)) goto drain;
                if (!warp_wait(bar(BAR_DO_FULL + (int)st), sp, ctl)) goto drain;
                tc_fence_after_sync();
                issue_kmajor(lead, tmem + kColY, dsc.v_k, dsc.do_k + st * kStageLo);
                lead_commit(lead, bar(BAR_DPT_FULL));
            }
            for (int t = 0; t < u.ntiles; ++t, ++gt) {
                const uint32_t st = stage_of(gt);
                // dV += P^T dO (P^T in X); the accumulators must have been written out at a unit's start
                if (!warp_wait(bar(BAR_P_READY), gt & 1, ctl)) goto drain;
                if (t == 0 && uc > 0 && !warp_wait(bar(BAR_ACC_FREE), (uc - 1) & 1, ctl)) goto drain;
                tc_fence_after_sync();
                issue_ts(lead, tmem + kColDV, tmem + kColX, dsc.do_n + st * kStageLo, t > 0);
                lead_commit(lead, bar(BAR_DO_EMPTY + (int)st));
                const bool more = t + 1 < u.ntiles;
                const uint32_t nst = stage_of(gt + 1), nsp = phase_of(gt + 1);
                // next S^T into X, which dV above has read; it runs while phase B computes dS^T
                if (more) {
                    if (!warp_wait(bar(BAR_Q_FULL + (int)nst), nsp, ctl)) goto drain;
                    tc_fence_after_sync();
                    issue_kmajor(lead, tmem + kColX, dsc.k_k, dsc.q_k + nst * kStageLo);
                    lead_commit(lead, bar(BAR_ST_FULL));
                }
                // dQ^T = K^T dS^T (d = 128: into Y, whose dP^T phase B has read; d = 64: into its own
                // columns, once the previous tile's dQ^T is out), then dK += dS^T Q
                if (!warp_wait(bar(BAR_DS_READY), gt & 1, ctl)) goto drain;
                if (kD64 && gt > 0 && !warp_wait(bar(BAR_DQ_FREE), (gt - 1) & 1, ctl)) goto drain;
                tc_fence_after_sync();
                issue_dq(lead, tmem, dsc);
                lead_commit(lead, bar(BAR_DQ_FULL));
                issue_dk(lead, tmem, dsc, dsc.q_n + st * kStageLo, t > 0);
                lead_commit(lead, bar(BAR_Q_EMPTY + (int)st));
                // next dP^T into Y (d = 128: once dQ^T has been read out of it)
                if (more) {
                    if (!kD64 && !warp_wait(bar(BAR_DQ_FREE), gt & 1, ctl)) goto drain;
                    if (!warp_wait(bar(BAR_DO_FULL + (int)nst), nsp, ctl)) goto drain;
                    tc_fence_after_sync();
                    issue_kmajor(lead, tmem + kColY, dsc.v_k, dsc.do_k + nst * kStageLo);
                    lead_commit(lead, bar(BAR_DPT_FULL));
                }
            }
            lead_commit(lead, bar(BAR_KV_EMPTY));
            lead_commit(lead, bar(BAR_ACC_FULL));
            ++uc;
        }
    }
drain:
    if (issued) {
        lead_commit(lead, bar(BAR_DRAIN));
        drain_wait(bar(BAR_DRAIN), 0);
    }
}

// ------------------------------------------------------------------------------------------------
// kernel
// ------------------------------------------------------------------------------------------------
template <bool kTail>
__global__ void __launch_bounds__(kThreads, 1)
window_bwd_tc_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
              const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmDO, const __grid_constant__ BwdArgs a)
{
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t sbase = smem_u32(smem);
    const int warp = threadIdx.x >> 5;
    if (sbase & 1023u) {  // see kSmemBytes; uniform across the CTA, before any barrier or TMEM use
        if (threadIdx.x == 0) atomicOr(a.status, kStatusLayout);
        return;
    }
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kSmemAbort);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kSmemTmemSlot);
    if (threadIdx.x == 0) {
        for (int i = 0; i < BAR_COUNT; ++i) {
            const bool by_math = i == BAR_P_READY || i == BAR_DS_READY || i == BAR_ACC_FREE;
            mbar_init(sbase + kSmemBar + 8u * (uint32_t)i, by_math ? 8u : (i == BAR_DQ_FREE ? 4u : 1u));
        }
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 13) {
        tmem_alloc(smem_u32(tmem_slot), 512);
        tmem_relinquish();
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    asm volatile("griddepcontrol.wait;" ::: "memory");  // for D, lse, the cleared dQ and the copies
    const uint32_t tmem = *tmem_slot;
    const WaitCtl ctl{abort_flag, a.status, kWaitLimitNs};
    // Register split: launched with 512 x 128 = 65536 registers; math warpgroups 2 x 128 x 144, the
    // dQ warpgroup 128 x 152 and the TMA/MMA warpgroup 128 x 72 = 65536 (per SM sub-partition
    // 144 + 144 + 152 + 72 = 512).
    if (warp < 8)
        asm volatile("setmaxnreg.inc.sync.aligned.u32 144;" ::: "memory");
    else if (warp < 12)
        asm volatile("setmaxnreg.inc.sync.aligned.u32 152;" ::: "memory");
    else
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;" ::: "memory");
    if (warp < 8) {
        math_role<kTail>(a, sbase, tmem, ctl);
    } else if (warp < 12) {
        dq_role<kTail>(a, sbase, tmem, ctl);
    } else if (warp == 12) {
        if ((threadIdx.x & 31) == 0) producer_role<kTail>(a, sbase, &tmQ, &tmK, &tmV, &tmDO, ctl);
    } else if (warp == 13) {
        mma_role<kTail>(a, sbase, tmem, ctl);
    }
    tc_fence_before_sync();
    __syncthreads();
    if (warp == 13) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, 512);
    }
}

template <bool kTail>
cudaError_t launch(const WindowBwdPlan& p, const BwdArgs& a, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                   const CUtensorMap& tdo, cudaStream_t s)
{
    static std::mutex mu;
    static bool done[64];
    const cudaError_t e = allow_smem(window_bwd_tc_kernel<kTail>, (int)kSmemBytes, mu, done);
    if (e != cudaSuccess) return e;
    const long long sms = device_sm_count();
    return launch_next(p.early, window_bwd_tc_kernel<kTail>, (unsigned)(a.items < sms ? a.items : sms), kThreads, kSmemBytes, s, tq, tk, tv, tdo, a);
}

}  // namespace

cudaError_t RA_WIN_BWD_LAUNCH(const WindowArgs& w, const WindowBwdPlan& p, unsigned int* status, cudaStream_t s)
{
    CUtensorMap tq, tk, tv, tdo;
    if (!make_map(&tq, w.q, w.geo, (long long)w.B * w.H, kHd) || !make_map(&tk, w.k, w.geo, (long long)w.B * w.Hkv, kHd) ||
        !make_map(&tv, w.v, w.geo, (long long)w.B * w.Hkv, kHd) || !make_map(&tdo, w.dout, w.geo, (long long)w.B * w.H, kHd))
        return cudaErrorInvalidValue;
    BwdArgs a;
    a.geo = w.geo;
    a.store_geo = w.store_geo;
    a.band = w.band;
    a.G = w.G;
    a.T = p.tiles;
    a.sink_tiles = p.sink_tiles;
    a.segs = p.segs;
    a.sink_items = (unsigned)p.sink_items;  // (below 2^31: the call's check)
    const unsigned segments = (unsigned)(p.sink_tiles * p.segs);  // of a kv head
    a.per = segments + (unsigned)(p.tiles - p.sink_tiles);
    a.share = (((unsigned long long)segments << 32) + a.per - 1) / a.per;  // rounded up: the last one comes too
    a.whole = (unsigned)p.whole;
    a.tail_segs = p.tail_segs;
    a.items = (unsigned)(p.sink_items + p.whole + p.tail * p.tail_segs);
    a.lse2 = p.lse2;
    a.Dv = p.D;
    a.dq_acc = p.dq;
    a.part = p.part;
    a.dk = w.dk;
    a.dv = w.dv;
    a.grad_bf16 = w.grad_dtype == 1;
    a.status = status;
    a.scale = w.scale;
    a.scale_log2 = w.scale_log2;
    return a.tail_segs > 1 ? launch<true>(p, a, tq, tk, tv, tdo, s) : launch<false>(p, a, tq, tk, tv, tdo, s);
}

}  // namespace ra
