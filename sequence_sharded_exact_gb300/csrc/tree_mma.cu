// tree_mma.cu -- attention over an e4m3 cache (tree.cuh) for bf16 queries, up to 16 query rows per kv head.
//
// So few rows leave the 128-row products of tree_tc_body.cuh nearly empty, and what bounds that path over an e4m3
// cache is V's way through shared memory as bf16.  Here a warp works on 16 cached rows by itself, in products whose
// 16 rows are cached rows or columns of V and whose 8 columns are queries (mma.m16n8k16, f16, float32 sums):
//   S^T = K Q^T,  O^T += V^T P^T  (twice, with one set of operands, for 9 to 16 rows),
// with operands that a thread puts together in registers: every e4m3 value is an f16, by one conversion per two of
// them, and nothing goes back to shared memory.  The order of a product's contraction and of its rows is free: thread
// (t, g) of a warp (t = lane % 4, g = lane / 4) takes d / 4 neighbouring elements of K's rows g and g + 8, and of V's rows
// 2t, 2t + 1, 2t + 8, 2t + 9 the d / 8 from d / 8 g on, whose bytes it pairs up.  S^T's weights become P^T's operand by
// a transposition of 8 x 8 within the warp.
//   * Queries: x 2^-e in f16, e such that the row's largest lies in [2^14, 2^15): a bf16's eight bits are exact down
//     to 2^-28 of it.  The scales of rows and keys are applied to S.
//   * Weights: p 2^ev_j in f16, ev_j the exponent of key j's V row, 2^7 at a reference M of their own: eleven bits down to
//     2^-21 of the largest, weight and scale together; where scales far apart put a weight that counts below that, what f16
//     does not hold of it is added in float32 (one row at a time: slow, and seldom).  The sum l takes p itself, at its
//     reference m.  Both follow the query's maximum only when that grows by more than 2^8: a vote per 16 rows, and
//     reductions only where it says so.
//   * A CTA's warps take 16 rows in turn, with rings of their own that the TMA fills; m, l, M and O are
//     a warp's own until the item's end, where they meet in shared memory, in warp order.  The next item's first rows
//     and its queries are on their way meanwhile.
//
// What bounds it: the memory, nearly.  A tile of 128 rows of 8 kv heads' e4m3 cache (d = 128) costs each of 152 SMs
// 0.95 us, 5.2 TB/s (tree_tc_body.cuh: 1.57), one token over 131072 rows 53 us with both launches (it: 91).  A group of 16
// rows is some 400 instructions, issued in about half of the cycles: latency, which 16 warps per SM hide; 24 do not fit the
// registers (80 each: spills, 60 us at 32 tiles per SM in place of 38), a third stage per ring changes nothing.  With query
// rows as the products' 16 rows there are twice as many products and registers (65 us).  9 to 16 query rows: 131072 rows in
// 87 us (88 there, before it summed its weights as they are rounded), 64 sequences of 1000 rows in 62 in place of 83
// (d = 64: 54 for 73, 38 for 64).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>

#include "tree_mma.cuh"

namespace ra {
namespace {

constexpr int kStages = 2;
constexpr int kBelow = 8;        // binades by which a row's scale may lie below the largest contribution's unlooked at
constexpr float kCounts = 40.f;  // and a score below the largest, and count

template <int D, int kWarps, int N>  // N: query rows in eights
struct Cfg {
    static constexpr int kPerSm = N == 1 ? kTreeMmaWarps / kWarps : tree_mma16_ctas_per_sm(D);
    static constexpr uint32_t kHalf = kKeys * D;                          // bytes of 16 rows
    static constexpr uint32_t kRings = kWarps * kStages * 2 * kHalf;      // [warps][stages][k, v]
    static constexpr uint32_t kX = kRings;                                // exchange: [warps][N D / 16][lanes] float4
    static constexpr uint32_t kMl = kX + kWarps * N * 32 * D;             // [2 items][warps][8 N] m, l, M, 0
    static constexpr uint32_t kBar = kMl + 2 * kWarps * 8 * N * 16;
    static constexpr uint32_t kAbort = kBar + kWarps * kStages * 8;
    static constexpr uint32_t kSmem = kAbort + 8 + 1024;  // slack for the 1024-byte alignment of the base
    static_assert((kSmem + 1024) * kPerSm <= 233472, "shared memory");
};

__device__ __forceinline__ void e4m3x4_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi)
{
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}

__device__ __forceinline__ void mma16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_f16x2(float a, float b)
{
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// A V byte that stands for no finite float32 at its row's scale: NaN, and from kHuge on the values that pass 2^128.
constexpr int kHuge = 247;
__device__ __forceinline__ bool not_finite(uint32_t x, int scale)
{
    const uint32_t mag = x & 127u;
    return mag == 127u || (scale >= kHuge && (scale == 255 || mag >= (uint32_t)(262 - scale) << 3));
}

// 2^n, 0 below the smallest normal number; n <= 127.
__device__ __forceinline__ float pow2(int n) { return __uint_as_float((uint32_t)max(127 + n, 0) << 23); }

// Byte offset of 16-byte chunk c of row r in the TMA's 128- (d = 128) or 64-byte swizzle.
template <int D>
__device__ __forceinline__ uint32_t at16(int r, int c)
{
    return D == 128 ? (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4)) : (uint32_t)(r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
}

// Query row x of a kv head, elements (D / 4) t .. of thread t of its quad.
template <int D>
__device__ __forceinline__ void load_query(const TreeArgs& a, long long head, int x, uint32_t (&f)[D / 8])
{
    const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) + (head * a.R + x) * D) + (threadIdx.x & 3) * (D / 32);
#pragma unroll
    for (int c = 0; c < D / 32; ++c) {
        const uint4 v = x < a.R ? src[c] : make_uint4(0, 0, 0, 0);
        f[4 * c] = v.x, f[4 * c + 1] = v.y, f[4 * c + 2] = v.z, f[4 * c + 3] = v.w;
    }
}

// It as the operand of S^T's k steps, two registers each: elements (D / 4) t + 4 s .. + 3 of step s.  Returns the row's
// scale times the scores'.
template <int D>
__device__ __forceinline__ float convert_query(const TreeArgs& a, uint32_t (&f)[D / 8])
{
    uint32_t big = 0;  // bits of the largest magnitude: bf16 in the upper half, ordered as integers
#pragma unroll
    for (int i = 0; i < D / 8; ++i) big = max(big, max(f[i] << 16 & 0x7fff0000u, f[i] & 0x7fff0000u));
    big = max(big, __shfl_xor_sync(0xffffffffu, big, 1));
    big = max(big, __shfl_xor_sync(0xffffffffu, big, 2));
    const bool finite = big < 0x7f800000u;
    int e = (int)(big >> 23) - 127 - 14;
    e = e < -126 ? -126 : e;
    const float down = pow2(-e);
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
        f[i] = finite ? pack_f16x2(__uint_as_float(f[i] << 16) * down, __uint_as_float(f[i] & 0xffff0000u) * down) : 0u;
    return finite ? pow2(e) * a.scale_log2 : __uint_as_float(0x7fc00000u);
}

template <int D, int kWarps, int N, bool kWin>
__global__ void __launch_bounds__(32 * kWarps, Cfg<D, kWarps, N>::kPerSm) tree_mma_kernel(const __grid_constant__ Maps maps, const TreeArgs a)
{
    using C = Cfg<D, kWarps, N>;
    constexpr int kTiles = D / 16;  // 16-row tiles of O^T
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, t4 = lane & 3, g8 = lane >> 2;
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kAbort);
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (threadIdx.x == 0) {
        for (int i = 0; i < kWarps * kStages; ++i) mbar_init(sbase + C::kBar + 8u * (uint32_t)i, 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    __syncthreads();
    using Walk = TreeWalkOf<kWin>;
    Walk w;
    if (!w.begin(a, blockIdx.x)) {  // the same for every warp
        if (threadIdx.x == 0) a.border[blockIdx.x] = make_int4(-1, 0, 0, 0);
        if constexpr (kWin) {
            if (a.whole) tree_clear_item<D>(a, blockIdx.x);
        }
        return;
    }
    const WaitCtl ctl{abort_flag, a.status, 0};
    const uint32_t ring_at = (uint32_t)warp * kStages * 2 * C::kHalf, bars = sbase + C::kBar + 8u * (uint32_t)(warp * kStages);
    int4 border = make_int4(-1, 0, 0, 0);
    uint32_t used = 0, sent = 0;  // of the ring (sent: lane 0's)

    uint32_t bytes = 0, coming[4], qr[N][D / 8], item = 0;
    // An item's first rows, scales and queries set out.
    constexpr int kStep = kWarps * kKeys;  // the warp's 16-row groups of an item: from group_row on, every kWarps-th
    auto group_row = [&](const Walk& w) { return w.t0 * kTreeTile + warp * kKeys; };
    auto groups = [&](const Walk& w) {
        const int last = tree_list_end(w.s, kTreeTile), end = w.t1 * kTreeTile < last ? w.t1 * kTreeTile : last, all = (end - w.t0 * kTreeTile + kKeys - 1) / kKeys;
        return all > warp ? (all - warp + kWarps - 1) / kWarps : 0;
    };
    auto send = [&](const Walk& w, int i) {  // rows of the warp's i-th group
        if (lane == 0 && !*abort_flag) {
            const uint32_t slot = sent % kStages, bar = bars + 8u * slot, dst = sbase + ring_at + slot * 2 * C::kHalf;
            mbar_arrive_expect_tx(bar, 2 * C::kHalf);
            const int row = tree_row(w.s, group_row(w) + i * kStep, kTreeTile);
            tma_load_3d(dst, &maps.k, bar, 0, row, w.b * a.Hkv + w.g);
            tma_load_3d(dst + C::kHalf, &maps.v, bar, 0, row, w.b * a.Hkv + w.g);
            ++sent;
        }
    };
    // lane's key's scale byte of group i: K's of key lane, V's of key lane - 16; four groups' in use, four on their
    // way (a register that is moved on is waited for)
    auto scale_byte = [&](const Walk& w, int i) {
        const int row = tree_row(w.s, group_row(w) + i * kStep, kTreeTile) + (lane & 15);
        const uint8_t* exps = (lane < kKeys ? a.k_exp : a.v_exp) + ((long long)w.b * a.Hkv + w.g) * a.cap;
        return i < groups(w) && !tree_dead(w.s, row) ? (uint32_t)exps[row] : (uint32_t)kHuge - 1;  // (of no row: never far below)
    };
    auto set_out = [&](const Walk& w) {
        for (int i = 0; i < kStages && i < groups(w); ++i) send(w, i);
#pragma unroll
        for (int e = 0; e < 4; ++e) coming[e] = scale_byte(w, e);
#pragma unroll
        for (int c = 0; c < N; ++c) load_query<D>(a, (long long)w.b * a.Hkv + w.g, 8 * c + g8, qr[c]);
    };
    set_out(w);

    bool more;
    do {
        if (w.goes_on()) border = w.border(a, blockIdx.x);
        const int row0 = group_row(w), n = groups(w);
        float o[N][kTiles][4], m[N][2], l[N][2], sl[N][2];  // queries 8 c + 2t + u
        float top[N][2];                                    // M
        int low = 0;                                        // V's scale bytes below this are far from M's
        uint32_t live = 0;                                  // bit 2 c + u
        int reach[N][2];
#pragma unroll
        for (int c = 0; c < N; ++c) {
            const float scale = convert_query<D>(a, qr[c]);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int x = 8 * c + 2 * t4 + u;
                sl[c][u] = __shfl_sync(0xffffffffu, scale, (2 * t4 + u) * 4);
                m[c][u] = -INFINITY;
                l[c][u] = 0.f;
                top[c][u] = -INFINITY;
                if (x < a.R && x % a.T < w.s.cnt) live |= 1u << (2 * c + u);
                // (a column without a query sees no row that is dead: those have no scale of their own)
                if constexpr (kWin) reach[c][u] = x < a.R && x % a.T < w.s.cnt ? tree_reach(a, w.s, w.b, x % a.T) : w.s.len;
            }
#pragma unroll
            for (int j = 0; j < kTiles; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[c][j][e] = 0.f;
        }
        auto sees = [&](int c, int u, int key) {
            if constexpr (kWin)
                if (key < w.s.len) return key >= reach[c][u] || key < w.s.sinks;
            return key < w.s.len ||
                   (key < w.s.end && (live >> (2 * c + u) & 1) && tree_sees<kWin>(a, w.s, w.b, (8 * c + 2 * t4 + u) % a.T, key - w.s.len));
        };

#pragma unroll 1
        for (int i = 0; i < n; ++i) {
            const uint32_t slot = used % kStages;
            const uint8_t* kp = smem + ring_at + slot * 2 * C::kHalf;
            if ((i & 3) == 0) {
                bytes = coming[0] | coming[1] << 8 | coming[2] << 16 | coming[3] << 24;
#pragma unroll
                for (int e = 0; e < 4; ++e) coming[e] = scale_byte(w, i + 4 + e);
            }
            const uint32_t byte = bytes & 255u;
            bytes >>= 8;
            // keys g and g + 8: scales of K, exponents of V
            const float ks[2] = {__uint_as_float(__shfl_sync(0xffffffffu, byte, g8) << 23), __uint_as_float(__shfl_sync(0xffffffffu, byte, g8 + 8) << 23)};
            const float ve[2] = {(float)(int)__shfl_sync(0xffffffffu, byte, g8 + 16) - 127.f, (float)(int)__shfl_sync(0xffffffffu, byte, g8 + 24) - 127.f};
            // a row of V whose scale is huge, or far below that of what contributes most
            bool strange = __any_sync(0xffffffffu, lane >= kKeys && (byte >= (uint32_t)kHuge || (int)byte < low));
            warp_wait(bars + 8u * slot, (used / kStages) & 1, ctl);
            ++used;

            float s[N][4];
#pragma unroll
            for (int c = 0; c < N; ++c)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[c][e] = 0.f;
#pragma unroll
            for (int h = 0; h < D / 64; ++h) {  // 16 bytes of each key at a time: four k steps
                const uint4 x0 = *reinterpret_cast<const uint4*>(kp + at16<D>(g8, D == 128 ? 2 * t4 + h : t4));
                const uint4 x1 = *reinterpret_cast<const uint4*>(kp + at16<D>(g8 + 8, D == 128 ? 2 * t4 + h : t4));
                const uint32_t w0[4] = {x0.x, x0.y, x0.z, x0.w}, w1[4] = {x1.x, x1.y, x1.z, x1.w};
#pragma unroll
                for (int st = 0; st < 4; ++st) {
                    uint32_t a0, a1, a2, a3;
                    e4m3x4_to_f16(w0[st], a0, a2);
                    e4m3x4_to_f16(w1[st], a1, a3);
#pragma unroll
                    for (int c = 0; c < N; ++c) mma16(s[c], a0, a1, a2, a3, qr[c][2 * (4 * h + st)], qr[c][2 * (4 * h + st) + 1]);
                }
            }

            const int k0 = tree_row(w.s, row0 + i * kStep, kTreeTile);
            const bool masked = tree_masked(w.s, k0, kKeys);
            bool raise = false;
            float y[N][2][2];  // scores: [query][key]
#pragma unroll
            for (int c = 0; c < N; ++c)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        y[c][u][e] = s[c][2 * e + u] * ks[e] * sl[c][u];
                        if (masked && !sees(c, u, k0 + g8 + 8 * e)) y[c][u][e] = -INFINITY;
                        raise |= y[c][u][e] > m[c][u] + 8.f || y[c][u][e] + ve[e] > top[c][u] + 8.f;
                    }
                }
            if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
                for (int c = 0; c < N; ++c)
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        float my = fmaxf(y[c][u][0], y[c][u][1]), mz = fmaxf(y[c][u][0] + ve[0], y[c][u][1] + ve[1]);
#pragma unroll
                        for (int d = 4; d < 32; d <<= 1) {
                            my = fmaxf(my, __shfl_xor_sync(0xffffffffu, my, d));
                            mz = fmaxf(mz, __shfl_xor_sync(0xffffffffu, mz, d));
                        }
                        if (my > m[c][u] + 8.f) {
                            l[c][u] *= ex2_approx(m[c][u] - my);
                            m[c][u] = my;
                        }
                        float alpha = 1.f;
                        if (mz > top[c][u] + 8.f) {
                            alpha = ex2_approx(top[c][u] - mz);
                            top[c][u] = mz;
                        }
#pragma unroll
                        for (int j = 0; j < kTiles; ++j) {
                            o[c][j][u] *= alpha;
                            o[c][j][2 + u] *= alpha;
                        }
                    }
                low = 0;
#pragma unroll
                for (int c = 0; c < N; ++c)
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const float at = top[c][u] - m[c][u];  // the scale of what contributes most
                        if (at > -200.f && at < 300.f) low = max(low, (int)at + 127 - kBelow);
                    }
                low = __reduce_max_sync(0xffffffffu, low);
                strange = strange || __any_sync(0xffffffffu, lane >= kKeys && (int)byte < low);
            }
            const uint8_t* vp = kp + C::kHalf;
            // What float16 does not hold of the weights that count among the scores is added in float32, row by row: one element
            // far above the others takes its row's scale up, and M with it, while the other columns are the other rows'.  (Rows of the
            // smallest scale are zeros, mostly, and all below 2^-117.)
            if (strange) {
#pragma unroll
                for (int c = 0; c < N; ++c) {
                    float left[2][2];
                    uint32_t rows = 0;
#pragma unroll
                    for (int u = 0; u < 2; ++u)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float p = ex2_approx(y[c][u][e] + (ve[e] - (top[c][u] == -INFINITY ? 0.f : top[c][u] - 7.f)));
                            left[u][e] = p < pow2(-14) && y[c][u][e] > m[c][u] - kCounts && ve[e] > -126.f ? p - __half2float(__float2half_rn(p)) : 0.f;
                            if (left[u][e] != 0.f) rows |= 1u << (g8 + 8 * e);
                        }
                    rows = __reduce_or_sync(0xffffffffu, rows);
#pragma unroll 1
                    for (; rows; rows &= rows - 1) {
                        const int r = __ffs(rows) - 1, er = (int)__shfl_sync(0xffffffffu, byte, r + 16);
                        float lw[2];
#pragma unroll
                        for (int u = 0; u < 2; ++u) lw[u] = __shfl_sync(0xffffffffu, r < 8 ? left[u][0] : left[u][1], (r & 7) * 4 + t4);
#pragma unroll
                        for (int j = 0; j < D / 8; ++j) {
                            const int d = g8 * (D / 8) + j;
                            const uint32_t x = vp[at16<D>(r, d >> 4) + (d & 15)];
                            float v, y0, y1, y2;
                            e4m3x4_to_float(x, v, y0, y1, y2);
                            if (not_finite(x, er)) v = 0.f;  // (added below)
#pragma unroll
                            for (int u = 0; u < 2; ++u) o[c][j / 2][2 * (j & 1) + u] = fmaf(lw[u], v, o[c][j / 2][2 * (j & 1) + u]);
                        }
                    }
                }
            }
            uint32_t pb[N][2];
#pragma unroll
            for (int c = 0; c < N; ++c) {
                float p[2][2];  // [key][query]
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const float ref = m[c][u] == -INFINITY ? 0.f : m[c][u], at = top[c][u] == -INFINITY ? 0.f : top[c][u] - 7.f;
                    l[c][u] += ex2_approx(y[c][u][0] - ref) + ex2_approx(y[c][u][1] - ref);
#pragma unroll
                    for (int e = 0; e < 2; ++e) p[e][u] = ex2_approx(y[c][u][e] + (ve[e] - at));
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) pb[c][e] = transpose8(pack_f16x2(p[e][0], p[e][1]));
            }

            // V: rows 2t, 2t + 1, 2t + 8, 2t + 9, eight of the thread's d / 8 columns at a time
#pragma unroll
            for (int part = 0; part < D / 64; ++part) {
                uint32_t vw[4][2];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int r = 2 * t4 + (e & 1) + 8 * (e >> 1);
                    const uint2 v = *reinterpret_cast<const uint2*>(vp + (D == 128 ? at16<D>(r, g8) + part * 8 : at16<D>(r, g8 >> 1) + (g8 & 1) * 8));
                    vw[e][0] = v.x, vw[e][1] = v.y;
                }
                // Rows behind the sequence count as zeros.  NaN, and values whose scale takes them past float32, are
                // cleared and added to the queries that see them: a weight of 0 would not hide them from the others.
                if (masked || strange) {
                    bool odd = lane >= kKeys && byte >= (uint32_t)kHuge;
#pragma unroll
                    for (int e = 0; e < 4; ++e)
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            if (tree_dead(w.s, k0 + 2 * t4 + (e & 1) + 8 * (e >> 1))) vw[e][q] = 0;
                            odd |= (((vw[e][q] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) != 0;  // a byte of NaN
                        }
                    if (__any_sync(0xffffffffu, odd)) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int er = (int)__shfl_sync(0xffffffffu, byte, 2 * t4 + (e & 1) + 8 * (e >> 1) + 16);
#pragma unroll
                            for (int q = 0; q < 2; ++q)
#pragma unroll 1
                                for (int sh = 0; sh < 32; sh += 8)
                                    if (not_finite(vw[e][q] >> sh & 255u, er)) vw[e][q] &= ~(255u << sh);
                        }
#pragma unroll 1
                        for (int r = 0; r < kKeys; ++r) {
                            const int er = (int)__shfl_sync(0xffffffffu, byte, r + 16);
                            if (tree_dead(w.s, k0 + r)) continue;
#pragma unroll
                            for (int c = 0; c < N; ++c) {
                                const bool s0 = sees(c, 0, k0 + r), s1 = sees(c, 1, k0 + r);
#pragma unroll
                                for (int j = 0; j < 8; ++j) {
                                    const int d = g8 * (D / 8) + part * 8 + j;
                                    const uint32_t x = vp[at16<D>(r, d >> 4) + (d & 15)];
                                    if (!not_finite(x, er)) continue;
                                    float v, y0, y1, y2;
                                    e4m3x4_to_float(x, v, y0, y1, y2);
                                    v *= __uint_as_float((uint32_t)er << 23);
                                    if (s0) o[c][part * 4 + j / 2][2 * (j & 1)] += v;
                                    if (s1) o[c][part * 4 + j / 2][2 * (j & 1) + 1] += v;
                                }
                            }
                        }
                    }
                }
#pragma unroll
                for (int q = 0; q < 2; ++q)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {  // columns 4q + 2h, + 1 of the eight
                        uint32_t a0, a1, a2, a3;
                        e4m3x4_to_f16(__byte_perm(vw[0][q], vw[1][q], h ? 0x7362 : 0x5140), a0, a1);
                        e4m3x4_to_f16(__byte_perm(vw[2][q], vw[3][q], h ? 0x7362 : 0x5140), a2, a3);
#pragma unroll
                        for (int c = 0; c < N; ++c) mma16(o[c][part * 4 + 2 * q + h], a0, a1, a2, a3, pb[c][0], pb[c][1]);
                    }
            }
            __syncwarp();  // all lanes have read the slot
            if (i + kStages < n) send(w, i + kStages);
        }

        const bool whole = w.whole();
        const int z = w.b * a.Hkv + w.g, cnt = w.s.cnt;
        const long long pslot = (long long)blockIdx.x * 2 + (w.first ? 0 : 1);
        more = w.next(a);
        if (more) set_out(w);

        // the item's rows: the eight warps' m, l, E and O, in warp order (the next item's m, l come elsewhere: some warps
        // may still read these; its O are written behind the next barrier)
        float4* ml = reinterpret_cast<float4*>(smem + C::kMl) + (item++ & 1) * kWarps * 8 * N;
#pragma unroll
        for (int c = 0; c < N; ++c)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) l[c][u] += __shfl_xor_sync(0xffffffffu, l[c][u], d);
                if (g8 == 0) ml[(warp * N + c) * 8 + 2 * t4 + u] = make_float4(m[c][u], l[c][u], top[c][u], 0.f);
            }
        __syncthreads();
        float4* xs = reinterpret_cast<float4*>(smem + C::kX);
        constexpr int kFours = D / 32, kVecs = 2 * N * kFours;  // float4 per thread: [c][u][fours of its d / 8 columns]
        auto join = [&](int x, float& mr, float& lr, float& tr) {  // m, l and M of all
            mr = tr = -INFINITY;
            for (int k = 0; k < kWarps; ++k) {
                const float4 v = ml[k * 8 * N + x];
                mr = fmaxf(mr, v.x);
                tr = fmaxf(tr, v.z);
            }
            const float ref = mr == -INFINITY ? 0.f : mr;
            lr = 0.f;
            for (int k = 0; k < kWarps; ++k) {
                const float4 v = ml[k * 8 * N + x];
                // NaN scores alone leave no maximum
                lr = v.x == -INFINITY && v.y != 0.f ? v.y : fmaf(v.y, ex2_approx(v.x - ref), lr);
            }
        };
#pragma unroll
        for (int c = 0; c < N; ++c)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                float mr, lr, tr;
                join(8 * c + 2 * t4 + u, mr, lr, tr);
                const float f = ex2_approx(top[c][u] - (tr == -INFINITY ? 0.f : tr));
#pragma unroll
                for (int k = 0; k < kFours; ++k)
                    xs[(warp * kVecs + (2 * c + u) * kFours + k) * 32 + lane] =
                        make_float4(o[c][2 * k][u] * f, o[c][2 * k][2 + u] * f, o[c][2 * k + 1][u] * f, o[c][2 * k + 1][2 + u] * f);
            }
        __syncthreads();
#pragma unroll 1
        for (int v = warp; v < kVecs; v += kWarps) {  // vector v of every warp
            const int row = v / (2 * kFours) * 8 + 2 * t4 + v / kFours % 2, d = g8 * (D / 8) + v % kFours * 4;
            if (row >= a.R) continue;
            float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int k = 0; k < kWarps; ++k) {
                const float4 y = xs[(k * kVecs + v) * 32 + lane];
                sum.x += y.x, sum.y += y.y, sum.z += y.z, sum.w += y.w;
            }
            float mr, lr, tr;
            join(row, mr, lr, tr);
            const bool none = row % a.T >= cnt || (mr == -INFINITY && lr == 0.f);
            const long long grow = (long long)z * a.R + row;
            // from M's reference to m's, in two steps: one could pass float32's range where the result does not
            const float inv = whole ? 1.0f / lr : 1.0f, up = ex2_approx(0.5f * (tr - 7.f - (mr == -INFINITY ? 0.f : mr)));
            float* ps = &sum.x;
#pragma unroll
            for (int e = 0; e < 4; ++e) ps[e] = none ? 0.f : ps[e] * up * inv * up;
            if (whole) {
                if (a.bf16_out)
                    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + grow * D + d) =
                        make_uint2(pack_bf16x2(sum.x, sum.y), pack_bf16x2(sum.z, sum.w));
                else
                    *reinterpret_cast<float4*>(static_cast<float*>(a.out) + grow * D + d) = sum;
                if (d == 0) a.lse[grow] = none ? -INFINITY : (mr + log2f(lr)) * kLn2;
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) a.part_o[(pslot * D + d + e) * a.rt + row] = ps[e];
                if (d == 0) *reinterpret_cast<float4*>(a.part_ml + (pslot * a.rt + row) * 4) = make_float4(mr, lr, lr, 0.f);
            }
        }
    } while (more);
    if (threadIdx.x == 0) a.border[blockIdx.x] = border;
    if (lane == 0) {  // after a wait that gave up, copies may still be on their way
        for (uint32_t k = 1; k <= (uint32_t)kStages && k <= sent; ++k)
            drain_wait(bars + 8u * ((sent - k) % kStages), ((sent - k) / kStages) & 1);
    }
}

// [heads][cap][D] bytes, boxes of 16 rows, in the swizzle of a whole row.
template <int D>
bool make_map(CUtensorMap* map, const void* base, long long rows, long long heads)
{
    auto fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)rows, (cuuint64_t)heads};
    cuuint64_t strides[2] = {(cuuint64_t)D, (cuuint64_t)rows * D};
    cuuint32_t box[3] = {(cuuint32_t)D, (cuuint32_t)kKeys, 1u};
    cuuint32_t estr[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              D == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int kWarps, int N, bool kWin>
cudaError_t launch_as(const TreeArgs& a, cudaStream_t s)
{
    using C = Cfg<D, kWarps, N>;
    Maps maps;
    const long long heads = (long long)a.B * a.Hkv;
    if (!make_map<D>(&maps.k, a.k, a.cap, heads) || !make_map<D>(&maps.v, a.v, a.cap, heads)) return cudaErrorInvalidValue;
    static std::mutex mu;
    static bool done[64];
    const cudaError_t e = allow_smem(tree_mma_kernel<D, kWarps, N, kWin>, (int)C::kSmem, mu, done);
    if (e != cudaSuccess) return e;
    tree_mma_kernel<D, kWarps, N, kWin><<<a.ctas, 32 * kWarps, C::kSmem, s>>>(maps, a);
    return cudaGetLastError();
}

template <int D, int kWarps, int N>
cudaError_t launch(const TreeArgs& a, cudaStream_t s)
{
    return a.window ? launch_as<D, kWarps, N, true>(a, s) : launch_as<D, kWarps, N, false>(a, s);
}

}  // namespace

cudaError_t launch_tree_mma(const TreeArgs& a, int d, int warps, cudaStream_t s)
{
    if (a.rt == kTreeMmaE4m3Rows) return d == 128 ? launch<128, 4, 2>(a, s) : launch<64, 4, 2>(a, s);
    if (warps == 8) return d == 128 ? launch<128, 8, 1>(a, s) : launch<64, 8, 1>(a, s);
    return d == 128 ? launch<128, 4, 1>(a, s) : launch<64, 4, 1>(a, s);
}

}  // namespace ra
