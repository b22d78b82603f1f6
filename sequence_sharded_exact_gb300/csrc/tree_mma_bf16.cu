// tree_mma_bf16.cu -- attention over a bf16 cache (tree.cuh) for bf16 queries, up to 8 query rows per kv head.
//
// The products of tree_mma.cu, S^T = K Q^T and O^T += V^T P^T with 16 cached rows, or columns of V, against 8 queries
// (mma.m16n8k16, bf16, float32 sums), a warp by itself with 16 cached rows at a time; K and V are operands as they
// are cached, V by transposing loads (ldmatrix).  P is two bf16 parts, two products in place of one at no cost here; its
// reference follows the maximum only when that grows by more than 2^8: a vote per 16 rows, and reductions only where it
// says so.  A CTA has four warps, two or three CTAs run on an SM: while one joins its
// warps' results at an item's end the others stream.
//
// What bounds it: the memory.  A tile of 128 rows of 8 kv heads (d = 128, 64 KB) costs each of 152 SMs 1.32 us, 7.5
// TB/s; one token over 131072 rows takes 85 us with both launches (tree_tc_body.cuh: 88), one over 19 tiles, a tile
// an SM, 11.5 (12.7), 512 sequences of 129 rows 72 (120): no 128 query rows to fill, and no pipeline of
// warps with different parts to drain at every item's end.
#include <cuda_bf16.h>
#include <math.h>

#include "tree_mma.cuh"

namespace ra {
namespace {

constexpr int kWarps = 4, kThreads = 32 * kWarps, kStages = 2;

template <int D>
struct Cfg {
    static constexpr uint32_t kHalf = kKeys * D * 2;                      // bytes of 16 rows
    static constexpr uint32_t kRings = kWarps * kStages * 2 * kHalf;      // [warps][stages][k, v], 64 columns after 64
    static constexpr int kXRow = 64 + 4;                                  // floats: queries' rows fall into different banks
    static constexpr uint32_t kX = kRings;                                // exchange: [warps][8][kXRow] float
    static constexpr uint32_t kMl = kX + kWarps * 8 * kXRow * 4;          // [2 items][warps][8] m, l, normaliser, 0
    static constexpr uint32_t kBar = kMl + 2 * kWarps * 8 * 16;
    static constexpr uint32_t kAbort = kBar + kWarps * kStages * 8;
    static constexpr uint32_t kSmem = kAbort + 8 + 1024;  // slack for the 1024-byte alignment of the base
    static_assert(kThreads == 8 * 16, "a thread per row and four of 64 columns");
    static_assert((kSmem + 1024) * 3 <= 233472, "shared memory");
};

__device__ __forceinline__ void mma16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Four 8 x 8 matrices of 16-bit values whose rows the lanes name, eight lanes a matrix.
__device__ __forceinline__ void load_matrices(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void load_matrices_transposed(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

// Byte offset of 16-byte chunk c of row r: 64 columns after 64, in the TMA's 128-byte swizzle.
__device__ __forceinline__ uint32_t at16(int r, int c) { return (uint32_t)((c >> 3) * 2048 + r * 128 + (((c & 7) ^ (r & 7)) << 4)); }

__device__ __forceinline__ bool not_finite(uint32_t half) { return (half & 0x7f80u) == 0x7f80u; }

template <int D, bool kWin>
__global__ void __launch_bounds__(kThreads, 3) tree_mma_bf16_kernel(const __grid_constant__ Maps maps, const TreeArgs a)
{
    using C = Cfg<D>;
    constexpr int kTiles = D / 16;  // k steps of S^T, 16-row tiles of O^T
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
    uint32_t qr[2 * kTiles], item = 0;
    // the warp's 16-row groups of an item: from group_row on, every kWarps-th
    auto group_row = [&](const Walk& w) { return w.t0 * kTreeTile + warp * kKeys; };
    auto groups = [&](const Walk& w) {
        const int last = tree_list_end(w.s, kTreeTile), end = w.t1 * kTreeTile < last ? w.t1 * kTreeTile : last, all = (end - w.t0 * kTreeTile + kKeys - 1) / kKeys;
        return all > warp ? (all - warp + kWarps - 1) / kWarps : 0;
    };
    auto send = [&](const Walk& w, int i) {
        if (lane == 0 && !*abort_flag) {
            const uint32_t slot = sent % kStages, bar = bars + 8u * slot, dst = sbase + ring_at + slot * 2 * C::kHalf;
            const int row = tree_row(w.s, group_row(w) + i * kWarps * kKeys, kTreeTile), z = w.b * a.Hkv + w.g;
            mbar_arrive_expect_tx(bar, 2 * C::kHalf);
            for (int h = 0; h < D / 64; ++h) {
                tma_load_3d(dst + (uint32_t)h * 2048u, &maps.k, bar, h * 64, row, z);
                tma_load_3d(dst + C::kHalf + (uint32_t)h * 2048u, &maps.v, bar, h * 64, row, z);
            }
            ++sent;
        }
    };
    // An item's first rows, and its queries as the operand of S^T's k steps (columns 16 s + 2t, + 1, + 8, + 9 of row g).
    auto set_out = [&](const Walk& w) {
        for (int i = 0; i < kStages && i < groups(w); ++i) send(w, i);
        const uint32_t* q = reinterpret_cast<const uint32_t*>(static_cast<const __nv_bfloat16*>(a.q) +
                                                             (((long long)w.b * a.Hkv + w.g) * a.R + g8) * D) + t4;
#pragma unroll
        for (int s = 0; s < kTiles; ++s) {
            qr[2 * s] = g8 < a.R ? q[8 * s] : 0u;
            qr[2 * s + 1] = g8 < a.R ? q[8 * s + 4] : 0u;
        }
    };
    set_out(w);
    // the lane's row and chunk of the four matrices of a 16 x 16 block: of K as it lies, of V transposed
    const int kr = (lane & 7) + (lane & 8), kc = lane >> 4, vr = (lane & 7) + (lane >> 4) * 8, vc = lane >> 3 & 1;

    bool more;
    do {
        if (w.goes_on()) border = w.border(a, blockIdx.x);
        const int row0 = group_row(w), n = groups(w);
        float o[kTiles][4], m[2], l[2];  // queries 2t + u
        bool live[2];
        int reach[2] = {0, 0};
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int x = 2 * t4 + u;
            m[u] = -INFINITY;
            l[u] = 0.f;
            live[u] = x < a.R && x % a.T < w.s.cnt;
            if constexpr (kWin) reach[u] = live[u] ? tree_reach(a, w.s, w.b, x % a.T) : w.s.len;
        }
#pragma unroll
        for (int j = 0; j < kTiles; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[j][e] = 0.f;
        auto sees = [&](int u, int key) {
            if constexpr (kWin)
                if (key < w.s.len) return key >= reach[u] || key < w.s.sinks;
            return key < w.s.len || (key < w.s.end && live[u] && tree_sees<kWin>(a, w.s, w.b, (2 * t4 + u) % a.T, key - w.s.len));
        };

#pragma unroll 1
        for (int i = 0; i < n; ++i) {
            const uint32_t slot = used % kStages, k_at = sbase + ring_at + slot * 2 * C::kHalf, v_at = k_at + C::kHalf;
            warp_wait(bars + 8u * slot, (used / kStages) & 1, ctl);
            ++used;
            float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int st = 0; st < kTiles; ++st) {
                uint32_t k[4];
                load_matrices(k, k_at + at16(kr, 2 * st + kc));
                mma16(s, k, qr[2 * st], qr[2 * st + 1]);
            }
            const int k0 = tree_row(w.s, row0 + i * kWarps * kKeys, kTreeTile);
            const bool masked = tree_masked(w.s, k0, kKeys);
            bool raise = false;
            float y[2][2];  // scores: [query][key]
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    y[u][e] = s[2 * e + u] * a.scale_log2;
                    if (masked && !sees(u, k0 + g8 + 8 * e)) y[u][e] = -INFINITY;
                    raise |= y[u][e] > m[u] + 8.f;
                }
            if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    float my = fmaxf(y[u][0], y[u][1]), alpha = 1.f;
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) my = fmaxf(my, __shfl_xor_sync(0xffffffffu, my, d));
                    if (my > m[u] + 8.f) {
                        alpha = ex2_approx(m[u] - my);
                        m[u] = my;
                    }
                    l[u] *= alpha;
#pragma unroll
                    for (int j = 0; j < kTiles; ++j) {
                        o[j][u] *= alpha;
                        o[j][2 + u] *= alpha;
                    }
                }
            }
            uint32_t pb[2], pl[2];
            {
                float p[2][2];  // [key][query]
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const float ref = m[u] == -INFINITY ? 0.f : m[u];
                    p[0][u] = ex2_approx(y[u][0] - ref);
                    p[1][u] = ex2_approx(y[u][1] - ref);
                    l[u] += p[0][u] + p[1][u];
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    uint32_t hi, lo;
                    split_weights(make_float2(p[e][0], p[e][1]), hi, lo);
                    pb[e] = transpose8(hi);
                    pl[e] = transpose8(lo);
                }
            }
            // Rows of V behind the sequence count as zeros, and what is not finite in drafted tokens' rows is cleared and
            // added to the queries that see it: a weight of 0 would not hide it from the others.
            if (masked) {
                uint8_t* v = smem + ring_at + slot * 2 * C::kHalf + C::kHalf;
                const int r = lane >> 1, key = k0 + r;
                bool odd = false;
                if (tree_partly(w.s, key)) {
#pragma unroll 1
                    for (int c = lane & 1; c < D / 8; c += 2) {
                        uint4* at = reinterpret_cast<uint4*>(v + at16(r, c));
                        uint4 x = *at;
                        uint32_t* px = &x.x;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            if (tree_dead(w.s, key)) {
                                px[e] = 0;
                                continue;
                            }
                            if (not_finite(px[e])) px[e] &= 0xffff0000u, odd = true;
                            if (not_finite(px[e] >> 16)) px[e] &= 0x0000ffffu, odd = true;
                        }
                        *at = x;
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the slot is filled again
                }
                if (__any_sync(0xffffffffu, odd)) {
                    const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(a.v) + (((long long)w.b * a.Hkv + w.g) * a.cap + k0) * D + g8;
#pragma unroll 1
                    for (int r = 0; r < kKeys; ++r) {
                        if (!tree_partly(w.s, k0 + r) || tree_dead(w.s, k0 + r)) continue;
                        const bool s0 = sees(0, k0 + r), s1 = sees(1, k0 + r);
#pragma unroll
                        for (int j = 0; j < 2 * kTiles; ++j) {
                            const float x = __bfloat162float(src[(long long)r * D + 8 * j]);
                            if (fabsf(x) <= 3.3895314e38f) continue;  // bf16's largest
                            if (s0) o[j >> 1][2 * (j & 1)] += x;
                            if (s1) o[j >> 1][2 * (j & 1) + 1] += x;
                        }
                    }
                }
                __syncwarp();
            }
#pragma unroll
            for (int j = 0; j < kTiles; ++j) {
                uint32_t v[4];
                load_matrices_transposed(v, v_at + at16(vr, 2 * j + vc));
                mma16(o[j], v, pb[0], pb[1]);
                mma16(o[j], v, pl[0], pl[1]);
            }
            __syncwarp();  // all lanes have read the slot
            if (i + kStages < n) send(w, i + kStages);
        }

        const bool whole = w.whole();
        const int z = w.b * a.Hkv + w.g, cnt = w.s.cnt;
        const long long pslot = (long long)blockIdx.x * 2 + (w.first ? 0 : 1);
        more = w.next(a);
        if (more) set_out(w);

        // the item's rows: the warps' m, l and O, in warp order (the next item's m, l come elsewhere: some warps may still
        // read these; its O are written behind the next barrier)
        float4* ml = reinterpret_cast<float4*>(smem + C::kMl) + (item++ & 1) * kWarps * 8;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) {
                l[u] += __shfl_xor_sync(0xffffffffu, l[u], d);
            }
            if (g8 == 0) ml[warp * 8 + 2 * t4 + u] = make_float4(m[u], l[u], l[u] * kWeightUp, 0.f);
        }
        __syncthreads();
        float* xs = reinterpret_cast<float*>(smem + C::kX);
        float f[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            float top = -INFINITY;
            for (int k = 0; k < kWarps; ++k) top = fmaxf(top, ml[k * 8 + 2 * t4 + u].x);
            f[u] = ex2_approx(m[u] - (top == -INFINITY ? 0.f : top));
        }
        // a thread sums four columns of one row, 64 columns of all rows at a time
        const int row = threadIdx.x >> 4;
        float top = -INFINITY, lr = 0.f, dr = 0.f;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) top = fmaxf(top, ml[k * 8 + row].x);
        const float ref = top == -INFINITY ? 0.f : top;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) {
            const float4 y = ml[k * 8 + row];
            const float g = ex2_approx(y.x - ref);
            const bool nan = y.x == -INFINITY && y.y != 0.f;  // NaN scores alone leave no maximum
            lr = nan ? y.y : fmaf(y.y, g, lr);
            dr = nan ? y.y : fmaf(y.z, g, dr);
        }
        const bool none = row % a.T >= cnt || (top == -INFINITY && lr == 0.f);
        const long long grow = (long long)z * a.R + row;
        const float inv = whole ? 1.0f / dr : 1.0f;
#pragma unroll
        for (int part = 0; part < D / 64; ++part) {
            if (part) __syncthreads();
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    xs[(warp * 8 + 2 * t4 + u) * C::kXRow + 8 * j + g8] = o[part * 4 + (j >> 1)][2 * (j & 1) + u] * f[u];
            __syncthreads();
            if (row >= a.R) continue;
            const int at = (threadIdx.x & 15) * 4, d = part * 64 + at;
            float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int k = 0; k < kWarps; ++k) {
                const float4 y = *reinterpret_cast<const float4*>(xs + (k * 8 + row) * C::kXRow + at);
                sum.x += y.x, sum.y += y.y, sum.z += y.z, sum.w += y.w;
            }
            float* ps = &sum.x;
#pragma unroll
            for (int e = 0; e < 4; ++e) ps[e] = none ? 0.f : ps[e] * inv;
            if (whole) {
                if (a.bf16_out)
                    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + grow * D + d) =
                        make_uint2(pack_bf16x2(sum.x, sum.y), pack_bf16x2(sum.z, sum.w));
                else
                    *reinterpret_cast<float4*>(static_cast<float*>(a.out) + grow * D + d) = sum;
                if (d == 0) a.lse[grow] = none ? -INFINITY : (top + log2f(lr)) * kLn2;
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) a.part_o[(pslot * D + d + e) * a.rt + row] = ps[e];
                if (d == 0) *reinterpret_cast<float4*>(a.part_ml + (pslot * a.rt + row) * 4) = make_float4(top, lr, dr, 0.f);
            }
        }
    } while (more);
    if (threadIdx.x == 0) a.border[blockIdx.x] = border;
    if (lane == 0) {  // after a wait that gave up, copies may still be on their way
        for (uint32_t k = 1; k <= (uint32_t)kStages && k <= sent; ++k)
            drain_wait(bars + 8u * ((sent - k) % kStages), ((sent - k) / kStages) & 1);
    }
}

// [heads][cap][D] bf16, boxes of 16 rows of 64 columns.
template <int D>
bool make_map(CUtensorMap* map, const void* base, long long rows, long long heads)
{
    auto fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)rows, (cuuint64_t)heads};
    cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)rows * D * 2};
    cuuint32_t box[3] = {64u, (cuuint32_t)kKeys, 1u};
    cuuint32_t estr[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool kWin>
cudaError_t launch(const TreeArgs& a, cudaStream_t s)
{
    using C = Cfg<D>;
    Maps maps;
    const long long heads = (long long)a.B * a.Hkv;
    if (!make_map<D>(&maps.k, a.k, a.cap, heads) || !make_map<D>(&maps.v, a.v, a.cap, heads)) return cudaErrorInvalidValue;
    static std::mutex mu;
    static bool done[64];
    const cudaError_t e = allow_smem(tree_mma_bf16_kernel<D, kWin>, (int)C::kSmem, mu, done);
    if (e != cudaSuccess) return e;
    tree_mma_bf16_kernel<D, kWin><<<a.ctas, kThreads, C::kSmem, s>>>(maps, a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_tree_mma_bf16(const TreeArgs& a, int d, cudaStream_t s)
{
    if (a.window) return d == 128 ? launch<128, true>(a, s) : launch<64, true>(a, s);
    return d == 128 ? launch<128, false>(a, s) : launch<64, false>(a, s);
}

}  // namespace ra
