// window_fwd_tc_body.cuh -- tensor-core forward of the attention through a window (window.cuh) for sm_103a: bf16, head
// dim RA_WIN_HD (128 or 64), any length.  Compiled once per head dim (window_fwd_tc.cu: 128, window_fwd_tc_d64.cu: 64); the
// including file names the host entry point through RA_WIN_FWD_LAUNCH.
//
// One CTA per SM, persistent.  A work unit is two tiles of 128 queries that share every K/V tile: two heads of one kv
// head's group at the same positions where the group is even, else 256 consecutive positions of one head.  Two heads meet
// W / 128 + 1 key tiles, 256 positions W / 128 + 2, of which each query tile sees all but one.  Units that share keys are
// neighbours, so that they run at the same time and K and V come from L2.
//   * warp 8 loads (TMA, one thread): Q tiles, and K and V tiles through rings.
//   * warp 9 issues tcgen05.mma: S_w = Q_w K^T into TMEM, O_w += P_w V with P_w from TMEM; the next tile's S
//     between the two P V, so that the tensor cores work while the softmax warps do.
//   * warps 0-3 and 4-7: softmax of query tile 0 and 1, thread = row = TMEM lane: the row's maximum and sum need no exchange.
//     m follows the maximum only when that grows by more than 2^8 (O / l does not depend on the reference).  Hidden scores are
//     set to -infinity by a bit each, in the tiles that are not wholly visible: one at each end of the window, and the
//     sinks'.  The other tiles' code knows nothing of masks (with both in one, 64K tokens without sinks took 2.83 ms in place of 2.64).
//   * A weight of 0 does not hide a value that is not finite: the rows whose O comes out so are looked at again (rare), once
//     the CTA's units are done: no wait of the pipeline, all of which have limits, then depends on how long that takes.
//   * TMEM: S0 columns [0,128), S1 [128,256), O0 from 256, O1 from 384.
// The weights go into P V as one bf16 value each (off by at most 2^-8, of either sign, so that it averages over a row's keys; what
// the rounding leaves as a second value would be a third product beside two, of a kernel that the products bound); the row is
// divided by the sum of the unrounded weights, but for the tile's largest, which counts as rounded: a row that one key dominates gets
// that key's value exactly.
//
// Measured, 64K tokens of 32 : 8 heads of 128: window 4096 2.55 to 2.69 ms (1590 to 1670 TFLOP/s over the visible pairs: the power
// cap), window 1024 870 us (1250), window 128 345 us (two masked tiles a unit: the chain from a unit's first S to its output, 3.5 us
// beside its tiles, bounds it).  A tile of sinks costs what any tile does: window 1024 with 4 sinks 960 us.  Head dim 64, 16K
// tokens of 2 x 16 heads, 512 on both sides: 223 us; dense 1010 TFLOP/s: issue slots, exponentials and products of 64
// columns are each near half of the time (half of the exponentials left out: 5 % faster).
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
constexpr int kThreads = 384;  // (warps 10-11 only complete the third warpgroup)
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
    BAR_V_EMPTY = BAR_K_EMPTY + kStages,  // both P V MMAs have read V
    BAR_S_FULL = BAR_V_EMPTY + kStages,
    BAR_P_FULL = BAR_S_FULL + 2,
    BAR_O_DONE = BAR_P_FULL + 2,
    BAR_DRAIN = BAR_O_DONE + 2,
    BAR_COUNT = BAR_DRAIN + 1
};

constexpr uint32_t kSmemTmemSlot = kSmemBar + BAR_COUNT * 8;
constexpr uint32_t kSmemAbort = kSmemTmemSlot + 8;
constexpr uint32_t kSmemOdd = kSmemAbort + 8;  // are there rows to mend; and behind it mend_rows' words
constexpr uint32_t kSmemBytes = kSmemOdd + 8 + (kTile + 2) * (kHd / 16) * 4 + 1024;  // slack for the 1024-byte alignment of the base
static_assert(kSmemBytes <= 232448, "shared memory");
static_assert(kSmemK - kSmemQ >= 256 * kHd * 2 && kStages * kTileBytes >= kTile * kHd * 2, "mend_rows' rows");

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
    unsigned units;   // B * Hkv * blocks * rows
    const __nv_bfloat16 *q, *k, *v;
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

__device__ __forceinline__ Unit unit_of(const FwdArgs& a, unsigned item)
{
    Unit u;
    const unsigned rest = item / (unsigned)a.rows, row = item - rest * (unsigned)a.rows;
    u.zk = (int)(rest / (unsigned)a.blocks);
    const int blk = (int)(rest - (unsigned)u.zk * (unsigned)a.blocks);
    u.zq = u.zk * a.G + (int)row * (a.pair ? 2 : 1);
    u.zq1 = a.pair ? u.zq + 1 : u.zq;
    u.p = blk * (a.pair ? kTile : 2 * kTile);
    u.p1 = a.pair ? u.p : u.p + kTile;
    u.run = key_tiles(a.band, u.p, a.pair ? kTile : 2 * kTile, kTile);
    return u;
}

// 32 bytes of a row at a time where it lies on such a boundary: half the requests of 16 bytes (64K tokens: window 4096
// 2.90 -> 2.86 ms, window 128 423 -> 390 us).
__device__ __forceinline__ void store32(void* p, bool wide, const uint32_t* v)
{
    if (wide) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]),
                     "r"(v[5]), "r"(v[6]), "r"(v[7])
                     : "memory");
    } else {
        static_cast<uint4*>(p)[0] = make_uint4(v[0], v[1], v[2], v[3]);
        static_cast<uint4*>(p)[1] = make_uint4(v[4], v[5], v[6], v[7]);
    }
}

// ------------------------------------------------------------------------------------------------
// softmax warpgroups
// ------------------------------------------------------------------------------------------------
// x of any of the 256 softmax threads; all of them call it.
__device__ __forceinline__ bool any_softmax_thread(bool x)
{
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, 1, 256, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)x)
        : "memory");
    return r != 0;
}

constexpr float kMaxF32 = 3.4028234e38f;
constexpr int kWords = kHd / 32;   // a bit per column
constexpr int kSigns = 2 * kWords; // columns with +infinity (or NaN), then those with -infinity (or NaN)

// Which of 64 columns (32 at head dim 64) of a row of V are not finite.
__device__ __forceinline__ void signs_of(const uint4* v, uint32_t (&plus)[kWords / 2], uint32_t (&minus)[kWords / 2])
{
#pragma unroll
    for (int w = 0; w < kWords / 2; ++w) plus[w] = minus[w] = 0;
#pragma unroll
    for (int g = 0; g < kHd / 16; ++g) {
        const uint4 x = v[g];
        const uint32_t y[4] = {x.x, x.y, x.z, x.w};
        uint32_t any = 0;  // an exponent of ones
#pragma unroll
        for (int i = 0; i < 4; ++i) any |= (y[i] & 0x7f807f80u) + 0x00800080u;
        if (!(any & 0x80008000u)) continue;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint32_t f = y[e >> 1] >> 16 * (e & 1) & 0xffffu;
            if ((f & 0x7f80u) != 0x7f80u) continue;
            const bool nan = (f & 0x7fu) != 0;
            if (nan || !(f & 0x8000u)) plus[g >> 2] |= 1u << ((8 * g + e) & 31);
            if (nan || (f & 0x8000u)) minus[g >> 2] |= 1u << ((8 * g + e) & 31);
        }
    }
}

// Which of the 8 elements of the output from number `at` on are not finite.
__device__ __forceinline__ uint32_t odd_columns(const FwdArgs& a, long long at)
{
    uint32_t bits = 0;
    if (a.out_f32) {
        const uint4* x = reinterpret_cast<const uint4*>(static_cast<float*>(a.out) + at);
        const uint4 y = x[0], z = x[1];
        const uint32_t f[8] = {y.x, y.y, y.z, y.w, z.x, z.y, z.z, z.w};
#pragma unroll
        for (int e = 0; e < 8; ++e) bits |= (uint32_t)((f[e] & 0x7f800000u) == 0x7f800000u) << e;
    } else {
        const uint4 x = *reinterpret_cast<const uint4*>(static_cast<__nv_bfloat16*>(a.out) + at);
        const uint32_t f[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int e = 0; e < 8; ++e) bits |= (uint32_t)((f[e >> 1] >> 16 * (e & 1) & 0x7f80u) == 0x7f80u) << e;
    }
    return bits;
}

// A row's columns `lost`, from the keys [k0, e) that it sees, which lie in shared memory: q by 16 bytes from every thread in turns.
__device__ __forceinline__ void sum_tile(const FwdArgs& a, const uint4* q, const uint4* k, const uint4* v, int p, int k0, int e, float lse2,
                                         const uint32_t (&lost)[kWords], float (&sum)[kHd])
{
    for (int j = k0; j < e; ++j, k += kHd / 8, v += kHd / 8) {
        if (!band_sees(a.band, p, j)) continue;
        float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
        for (int g = 0; g < kHd / 8; ++g) {
            const uint4 x = q[g * 256], y = k[g];
            const uint32_t w[4] = {x.x, x.y, x.z, x.w}, z[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                s[i] = fmaf(__uint_as_float(w[i] << 16), __uint_as_float(z[i] << 16), s[i]);
                s[i] = fmaf(__uint_as_float(w[i] & 0xffff0000u), __uint_as_float(z[i] & 0xffff0000u), s[i]);
            }
        }
        const float weight = ex2_approx(fmaf((s[0] + s[1]) + (s[2] + s[3]), a.scale_log2, lse2));
#pragma unroll
        for (int w = 0; w < kWords; ++w) {
            if (!lost[w]) continue;
#pragma unroll 1
            for (int g = 0; g < 4; ++g) {
                const uint32_t cols = lost[w] >> 8 * g & 0xffu;
                if (!cols) continue;
                const uint4 x = v[4 * w + g];
                const uint32_t y[4] = {x.x, x.y, x.z, x.w};
                float* to = sum + 32 * w + 8 * g;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (cols >> i & 1) to[i] = fmaf(weight, __uint_as_float(i & 1 ? y[i >> 1] & 0xffff0000u : y[i >> 1] << 16), to[i]);
            }
        }
    }
}

// After the CTA's last unit, where no wait depends on how long this takes: the rows whose output came out with elements that are
// not finite.  Such an element becomes the sum of what is not finite among the values that its row sees in its column (a bit per
// sign is all of that sum), whatever their weights; one that sees none there, and so has it from a hidden value or from a sum past
// float32, is summed once more from the visible keys alone.  The softmax warps read V by tiles, each thread half a row, and a
// row takes a tile that it sees whole at once; for such sums K and V go through the room of the rings and Q's tiles, which
// nothing else uses by then.  16K tokens of 8 : 2 heads of 128, window 8192 (0.31 ms without such values): a value that every row
// sees 1.1 ms, none of V finite 1.8, one NaN, beside which 127 rows of each head are summed once more, 10 (key by key for each row,
// inside the pipeline: 18, 708 and 73).  It costs calls without such values up to 1.5 % (64K tokens, window 128: 338 -> 343 us).
__device__ __noinline__ void mend_rows(const FwdArgs& a, uint8_t* smem)
{
    uint32_t *all = reinterpret_cast<uint32_t*>(smem + kSmemOdd + 8), *keys = all + 2 * kSigns;  // of a tile, two in turns; of each of its keys
    const int t = threadIdx.x, w = t >> 7, rw = t & 127;
    if (t < 2 * kSigns) all[t] = 0;
    for (unsigned item = blockIdx.x; item < a.units; item += gridDim.x) {
        const Unit u = unit_of(a, item);
        const int q0 = w ? u.p1 : u.p, p = q0 + rw;
        const bool in = p < a.band.L;
        const long long zq = w ? u.zq1 : u.zq, row = zq * a.band.L + (in ? buffer_row(a.store_geo, p) : 0);
        const float lse = in ? a.lse[row] : 0.f;
        uint32_t odd[kWords], seen[kSigns];
        bool any = false;
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
            odd[i] = seen[i] = seen[kWords + i] = 0;
            if (in && fabsf(lse) <= kMaxF32)  // (else so are the row's scores)
#pragma unroll
                for (int g = 0; g < 4; ++g) odd[i] |= odd_columns(a, row * kHd + 32 * i + 8 * g) << 8 * g;
            any |= odd[i] != 0;
        }
        if (!any_softmax_thread(any)) continue;
        for (int jj = 0; jj < u.run.count(); ++jj) {
            const int k0 = u.run.at(jj) * kTile, key = t >> 1, half = t & 1;
            uint32_t plus[kWords / 2] = {}, minus[kWords / 2] = {}, *now = all + (jj & 1) * kSigns;
            if (k0 + key < a.band.L)
                signs_of(reinterpret_cast<const uint4*>(a.v + ((long long)u.zk * a.band.L + buffer_row(a.geo, k0 + key)) * kHd + half * (kHd / 2)), plus, minus);
            bool found = false;
#pragma unroll
            for (int i = 0; i < kWords / 2; ++i) {
                const int at = half * (kWords / 2) + i;
                keys[key * kSigns + at] = plus[i];
                keys[key * kSigns + kWords + at] = minus[i];
                if (plus[i]) atomicOr(now + at, plus[i]);
                if (minus[i]) atomicOr(now + kWords + at, minus[i]);
                found |= (plus[i] | minus[i]) != 0;
            }
            if (any_softmax_thread(found)) {
                if (any && band_tile_whole(a.band, q0, kTile, k0, kTile)) {
#pragma unroll
                    for (int i = 0; i < kSigns; ++i) seen[i] |= now[i];
                } else if (any) {
                    const Seen s = seen_keys(a.band, p, k0);
#pragma unroll 1
                    for (int c = 0; c < kTile; ++c)
                        if (s.word(c & ~31) >> (c & 31) & 1) {
#pragma unroll
                            for (int i = 0; i < kSigns; ++i) seen[i] |= keys[c * kSigns + i];
                        }
                }
            }
            if (t < kSigns) all[((jj + 1) & 1) * kSigns + t] = 0;  // the next tile's, last read before the barrier above
            any_softmax_thread(false);                             // the tile has been read
        }
        if (t < 2 * kSigns) all[t] = 0;
        uint32_t lost[kWords], none = 0;
#pragma unroll
        for (int i = 0; i < kWords; ++i) none |= lost[i] = odd[i] & ~(seen[i] | seen[kWords + i]);
        float sum[kHd];
        if (any_softmax_thread(none != 0)) {
            uint4 *q = reinterpret_cast<uint4*>(smem + kSmemQ) + t, *k = reinterpret_cast<uint4*>(smem + kSmemK), *v = reinterpret_cast<uint4*>(smem + kSmemV);
            if (none) {
                const uint4* x = reinterpret_cast<const uint4*>(a.q + (zq * a.band.L + buffer_row(a.geo, p)) * kHd);
                for (int g = 0; g < kHd / 8; ++g) q[g * 256] = x[g];
                for (int c = 0; c < kHd; ++c) sum[c] = 0.f;
            }
            for (int jj = 0; jj < u.run.count(); ++jj) {
                const int k0 = u.run.at(jj) * kTile, e = k0 + kTile < a.band.L ? k0 + kTile : a.band.L;
                any_softmax_thread(false);  // the tile before this has been read
#pragma unroll 4
                for (int x = t; x < (e - k0) * (kHd / 8); x += 256) {
                    const long long at = ((long long)u.zk * a.band.L + buffer_row(a.geo, k0 + x / (kHd / 8))) * (kHd / 8) + x % (kHd / 8);
                    k[x] = reinterpret_cast<const uint4*>(a.k)[at];
                    v[x] = reinterpret_cast<const uint4*>(a.v)[at];
                }
                any_softmax_thread(false);
                if (none) sum_tile(a, q, k, v, p, k0, e, -lse * kLog2e, lost, sum);
            }
        }
#pragma unroll
        for (int i = 0; i < kWords; ++i)
#pragma unroll 1
            for (uint32_t left = odd[i]; left; left &= left - 1) {
                const uint32_t bit = left & (0u - left);
                const int c = 32 * i + __ffs(left) - 1;
                const float x = lost[i] & bit ? sum[c] : seen[i] & bit ? (seen[kWords + i] & bit ? __uint_as_float(0x7fffffffu) : INFINITY) : -INFINITY;
                if (a.out_f32)
                    static_cast<float*>(a.out)[row * kHd + c] = x;
                else
                    static_cast<__nv_bfloat16*>(a.out)[row * kHd + c] = __float2bfloat16_rn(x);
            }
    }
}

// What a softmax thread keeps of its row: the reference, the sum of the weights, and the sum of what rounding added to the
// tiles' largest.
struct Sums {
    float m = -INFINITY, l = 0.f, c = 0.f;
};
// Where it works: its lane's S and O, the barriers, the scores' factor.
struct Place {
    uint32_t tS, tO, bar_s, bar_p, bar_o;
    float sl2;
    int lane;
};

// One tile: S to weights.  rescales: O holds something.
template <bool kMasked>
__device__ __forceinline__ bool softmax_tile(const Seen& seen, const Place& x, bool rescales, uint32_t tcount, Sums& row, const WaitCtl& ctl)
{
    if (!mbar_wait(x.bar_s, tcount & 1, ctl)) return false;
    tc_fence_after_sync();
    __syncwarp();
    uint32_t r[4][32];
    tmem_ld_32x32b_x32(x.tS + 0, r[0]);
    tmem_ld_32x32b_x32(x.tS + 32, r[1]);
    tmem_ld_wait(r[0]);
    tmem_ld_wait(r[1]);
    tmem_ld_32x32b_x32(x.tS + 64, r[2]);
    tmem_ld_32x32b_x32(x.tS + 96, r[3]);
    float m8[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) m8[i] = -INFINITY;
    auto hide_and_max = [&](int c4) {
        if constexpr (kMasked) {
            const uint32_t word = seen.word(32 * c4);
#pragma unroll
            for (int e = 0; e < 32; ++e)
                if (!(word & (1u << e))) r[c4][e] = __float_as_uint(-INFINITY);
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
    const float m_tile = mx * x.sl2;
    float m_new = row.m;
    if (m_tile > row.m + 8.0f) m_new = m_tile;
    const float alpha = (m_new == row.m) ? 1.0f : ex2_approx(row.m - m_new);
    const float ref = m_new == -INFINITY ? 0.f : m_new;
    const float2 scale2 = make_float2(x.sl2, x.sl2), nref2 = make_float2(-ref, -ref);
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
        tmem_st_32x32b_x32(x.tS + half * 32, pk);
    }
    const float2 s2 = add2(add2(s4[0], s4[1]), add2(s4[2], s4[3]));
    const float p_max = ex2_approx(fmaf(mx, x.sl2, -ref));
    const float p_max_bf16 = __uint_as_float(pack_bf16x2(p_max, 0.f) << 16);
    row.l = row.l * alpha + (s2.x + s2.y);
    row.c = row.c * alpha + (p_max_bf16 - p_max);
    tmem_st_wait();
    if (__any_sync(0xffffffffu, rescales && alpha != 1.0f)) {
        if (!mbar_wait(x.bar_o, (tcount - 1) & 1, ctl)) return false;  // O of the previous tile is complete
        tc_fence_after_sync();
        __syncwarp();
#pragma unroll 1
        for (int c4 = 0; c4 < kHd / 32; ++c4) {
            uint32_t o[32];
            tmem_ld_32x32b_x32(x.tO + c4 * 32, o);
            tmem_ld_wait(o);
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
                const float2 v = mul2(make_float2(__uint_as_float(o[e]), __uint_as_float(o[e + 1])), make_float2(alpha, alpha));
                o[e] = __float_as_uint(v.x);
                o[e + 1] = __float_as_uint(v.y);
            }
            tmem_st_32x32b_x32(x.tO + c4 * 32, o);
        }
        tmem_st_wait();
    }
    tc_fence_before_sync();
    __syncwarp();
    if (x.lane == 0) mbar_arrive(x.bar_p);
    row.m = m_new;
    return true;
}

// False if a wait ran out.
__device__ __forceinline__ bool softmax_role(const FwdArgs& a, uint32_t sbase, uint32_t tmem, const WaitCtl& ctl)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int w = warp >> 2;                // query tile of this warpgroup
    const int rw = (warp & 3) * 32 + lane;  // row within the tile = TMEM lane
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tO = tmem + lane_off + kColO0 + (uint32_t)w * 128, bar_o = sbase + kSmemBar + 8 * (BAR_O_DONE + w);
    const Place x{tmem + lane_off + kColS0 + (uint32_t)w * 128, tO, sbase + kSmemBar + 8 * (BAR_S_FULL + w), sbase + kSmemBar + 8 * (BAR_P_FULL + w),
                  bar_o, a.scale_log2, lane};
    const bool wide = (reinterpret_cast<uintptr_t>(a.out) & 31u) == 0;
    uint32_t tcount = 0, ucount = 0;

    for (unsigned item = blockIdx.x; item < a.units; item += gridDim.x, ++ucount) {
        const Unit u = unit_of(a, item);
        const int q0 = w ? u.p1 : u.p, p = q0 + rw, ntiles = u.run.count();
        Sums row;
        for (int jj = 0; jj < ntiles; ++jj, ++tcount) {
            const int k0 = u.run.at(jj) * kTile;
            if (band_tile_whole(a.band, q0, kTile, k0, kTile)) {
                if (!softmax_tile<false>(Seen{}, x, jj > 0, tcount, row, ctl)) return false;
            } else {
                if (!softmax_tile<true>(seen_keys(a.band, p, k0), x, jj > 0, tcount, row, ctl)) return false;
            }
        }
        // the unit's rows
        if (!mbar_wait(bar_o, (tcount - 1) & 1, ctl)) return false;
        tc_fence_after_sync();
        __syncwarp();
        const float inv = 1.0f / (row.l + row.c), lse = (row.m + log2f(row.l)) * kLn2;
        const bool in = p < a.band.L;
        const long long zq = w ? u.zq1 : u.zq, row_g = zq * a.band.L + (in ? buffer_row(a.store_geo, p) : 0);
        float2 odd = make_float2(0.f, 0.f);  // NaN if an element is not finite
#pragma unroll 1
        for (int c = 0; c < kHd; c += 32) {
            uint32_t o[32];
            __syncwarp();  // the lanes of rows behind the sequence have gone ahead
            tmem_ld_32x32b_x32(tO + c, o);
            tmem_ld_wait(o);
            if (!in) continue;
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
                const float2 v = mul2(make_float2(__uint_as_float(o[e]), __uint_as_float(o[e + 1])), make_float2(inv, inv));
                odd = fma2(v, make_float2(0.f, 0.f), odd);
                o[e] = __float_as_uint(v.x);
                o[e + 1] = __float_as_uint(v.y);
            }
            if (a.out_f32) {
                float* dst = static_cast<float*>(a.out) + row_g * kHd + c;
#pragma unroll
                for (int e = 0; e < 4; ++e) store32(dst + 8 * e, wide, o + 8 * e);
            } else {
                __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.out) + row_g * kHd + c;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    uint32_t pk[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) pk[i] = pack_bf16x2(__uint_as_float(o[16 * e + 2 * i]), __uint_as_float(o[16 * e + 2 * i + 1]));
                    store32(dst + 16 * e, wide, pk);
                }
            }
        }
        if (in) a.lse[row_g] = lse;
        if (odd.x + odd.y != 0.f) asm volatile("st.shared.u32 [%0], 1;" ::"r"(sbase + kSmemOdd) : "memory");
    }
    return true;
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
    for (unsigned item = blockIdx.x; ok && item < a.units; item += gridDim.x) {
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
// MMA issue (one warp, one lane of it)
// ------------------------------------------------------------------------------------------------
struct FwdDesc {
    uint32_t q, k, v;  // low words of the tiles' descriptors (K and V at stage 0)
};
constexpr uint32_t kDescHi = sdesc_sw128_hi(1024);

__device__ __forceinline__ void issue_qk(uint32_t lead, const FwdDesc& dsc, uint32_t tmem, int w, int stage)
{
    constexpr uint32_t idesc = idesc_bf16_f32(128, 128, false, false);
    const uint32_t kb = dsc.k + (uint32_t)stage * (kTileBytes >> 4);
#pragma unroll
    for (int kk = 0; kk < kHd / 16; ++kk) {
        const uint32_t off = (uint32_t)(kk >> 2) * kHalfBytes + (uint32_t)(kk & 3) * 32u;
        lead_mma_ss(lead, tmem + kColS0 + (uint32_t)w * 128, sdesc_at(dsc.q, (uint32_t)w * kTileBytes + off, kDescHi), sdesc_at(kb, off, kDescHi), idesc,
               kk > 0 ? 1u : 0u);
    }
}

__device__ __forceinline__ void issue_pv(uint32_t lead, const FwdDesc& dsc, uint32_t tmem, int w, int stage, bool accumulate)
{
    constexpr uint32_t idesc = idesc_bf16_f32(128, kHd, false, true);
    const uint32_t vb = dsc.v + (uint32_t)stage * (kTileBytes >> 4);
    const uint32_t acc0 = accumulate ? 1u : 0u;
#pragma unroll
    for (int kk = 0; kk < 8; ++kk)
        lead_mma_ts(lead, tmem + kColO0 + (uint32_t)w * 128, tmem + kColS0 + (uint32_t)w * 128 + (uint32_t)kk * 8, sdesc_at(vb, (uint32_t)kk * 2048u, kDescHi),
               idesc, kk > 0 ? 1u : acc0);
}

__device__ __forceinline__ void mma_role(const FwdArgs& a, uint32_t sbase, uint32_t tmem, const WaitCtl& ctl)
{
    auto bar = [&](int i) { return sbase + kSmemBar + 8u * (uint32_t)i; };
    const uint32_t lead = elect();
    tmem = __shfl_sync(0xffffffffu, tmem, 0);
    FwdDesc dsc;
    dsc.q = sdesc_sw128_lo(sbase + kSmemQ, 16);
    dsc.k = sdesc_sw128_lo(sbase + kSmemK, 16);
    dsc.v = sdesc_sw128_lo(sbase + kSmemV, kHalfBytes);
    unsigned item = blockIdx.x;
    uint32_t kc = 0, qc = 0;
    int jj = 0, ntiles = unit_of(a, item).run.count();
    if (!warp_wait(bar(BAR_Q_FULL), 0, ctl)) goto drain;
    if (!warp_wait(bar(BAR_K_FULL + 0), 0, ctl)) goto drain;
    tc_fence_after_sync();
    issue_qk(lead, dsc, tmem, 0, 0);
    lead_commit(lead, bar(BAR_S_FULL + 0));
    issue_qk(lead, dsc, tmem, 1, 0);
    lead_commit(lead, bar(BAR_S_FULL + 1));
    lead_commit(lead, bar(BAR_K_EMPTY + 0));
    if (ntiles == 1) lead_commit(lead, bar(BAR_Q_EMPTY));
    while (true) {
        const int stage = (int)(kc % kStages), nstage = (int)((kc + 1) % kStages);
        const int jn = jj + 1 == ntiles ? 0 : jj + 1;
        if (jn == 0) item += gridDim.x;
        const bool has_next = item < a.units;
        if (!warp_wait(bar(BAR_V_FULL + stage), (kc / kStages) & 1, ctl)) goto drain;
        if (!warp_wait(bar(BAR_P_FULL + 0), kc & 1, ctl)) goto drain;
        tc_fence_after_sync();
        issue_pv(lead, dsc, tmem, 0, stage, jj > 0);
        lead_commit(lead, bar(BAR_O_DONE + 0));
        if (has_next) {
            if (jn == 0) {
                ++qc;
                if (!warp_wait(bar(BAR_Q_FULL), qc & 1, ctl)) goto drain;
            }
            if (!warp_wait(bar(BAR_K_FULL + nstage), ((kc + 1) / kStages) & 1, ctl)) goto drain;
            tc_fence_after_sync();
            issue_qk(lead, dsc, tmem, 0, nstage);
            lead_commit(lead, bar(BAR_S_FULL + 0));
        }
        if (!warp_wait(bar(BAR_P_FULL + 1), kc & 1, ctl)) goto drain;
        tc_fence_after_sync();
        issue_pv(lead, dsc, tmem, 1, stage, jj > 0);
        lead_commit(lead, bar(BAR_O_DONE + 1));
        lead_commit(lead, bar(BAR_V_EMPTY + stage));
        if (!has_next) break;
        issue_qk(lead, dsc, tmem, 1, nstage);
        lead_commit(lead, bar(BAR_S_FULL + 1));
        lead_commit(lead, bar(BAR_K_EMPTY + nstage));
        if (jn == 0) ntiles = unit_of(a, item).run.count();
        if (jn == ntiles - 1) lead_commit(lead, bar(BAR_Q_EMPTY));
        jj = jn;
        ++kc;
    }
drain:
    lead_commit(lead, bar(BAR_DRAIN));  // flips once every MMA issued by this thread has completed
    drain_wait(bar(BAR_DRAIN), 0);
}

__global__ void __launch_bounds__(kThreads, 1)
window_fwd_tc_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                     const __grid_constant__ FwdArgs a)
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
            mbar_init(sbase + kSmemBar + 8u * (uint32_t)i, cnt);
        }
        *abort_flag = 0;
        *reinterpret_cast<uint32_t*>(smem + kSmemOdd) = 0;
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

    // Registers: launched with 384 x 168 = 64512; softmax warpgroups 2 x 128 x 200, the others 128 x 104 = 64512.
    if (warp < 8)
        asm volatile("setmaxnreg.inc.sync.aligned.u32 200;" ::: "memory");
    else
        asm volatile("setmaxnreg.dec.sync.aligned.u32 104;" ::: "memory");

    if (warp < 8) {
        const bool done = softmax_role(a, sbase, tmem, ctl);
        __syncwarp();
        if (!any_softmax_thread(!done) && *reinterpret_cast<volatile uint32_t*>(smem + kSmemOdd))
            mend_rows(a, smem);
    } else if (warp == 8) {
        if ((threadIdx.x & 31) == 0) load_role(a, sbase, &tmQ, &tmK, &tmV, ctl);
    } else if (warp == 9) {
        mma_role(a, sbase, tmem, ctl);
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
    a.units = (unsigned)((long long)w.B * w.Hkv * a.blocks * a.rows);  // below 2^30: the call's check
    a.q = static_cast<const __nv_bfloat16*>(w.q);
    a.k = static_cast<const __nv_bfloat16*>(w.k);
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
