// window_aux.cu -- what the tensor-core kernels of the attention through a window need before and after them (HBM-bound).
//
// Before the backward: D = dout . out per row, lse in log2 units and the float32 accumulator of dQ cleared, all in natural
// order and padded to whole tiles of 128 positions (rows behind the sequence: -lse2 = -infinity, which makes their P 0).
// After it: dQ from the accumulator to the layout's rows, and dK and dV of the tiles that were cut, added over their segments in
// order.
// Layouts that TMA cannot read in natural order with one box (window_tc.cuh) are copied into it first, in the same launch.
// A group of d / 8 lanes has a row, 8 elements (16 bytes of bf16) each.
#include <cuda_bf16.h>
#include <math.h>

#include "ra_internal.h"
#include "ra_ptx.cuh"
#include "window.cuh"

namespace ra {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ void spread8(const uint4& v, float (&f)[8])
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        f[2 * e] = __uint_as_float(w[e] << 16);
        f[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
    }
}
__device__ __forceinline__ void load8(const void* p, long long i, bool bf16, float (&f)[8])
{
    if (bf16) {
        spread8(*reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p) + i), f);
    } else {
        const float4* v = reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
        const float4 a = v[0], b = v[1];
        f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
    }
}
__device__ __forceinline__ void store8(void* p, long long i, bool bf16, const float (&f)[8])
{
    if (bf16) {
        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p) + i) =
            make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
    } else {
        float4* v = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
        v[0] = make_float4(f[0], f[1], f[2], f[3]);
        v[1] = make_float4(f[4], f[5], f[6], f[7]);
    }
}

// Row `x` of a padded natural-order array -> its head, position and (if in the sequence) row in the layout's buffers.
struct Row {
    int z, p;
    bool in;
    long long at;
};
__device__ __forceinline__ Row row_of(const Geometry& g, int padded, long long x)
{
    Row r;
    r.z = (int)(x / padded);
    r.p = (int)(x - (long long)r.z * padded);
    r.in = r.p < g.L;
    r.at = r.in ? (long long)r.z * g.L + buffer_row(g, r.p) : 0;
    return r;
}

// q, k and v, whose rows are copied into natural order.
struct Copies {
    const uint4* src[3];
    uint4* dst[3];
    long long rows[3];
};
template <int D>
__device__ __forceinline__ void copy_rows(const Geometry& g, const uint4* src, uint4* dst, long long rows, long long x0, long long step)
{
    constexpr int kLanes = D / 8, U = 4;  // four loads on their way
    const int c = threadIdx.x % kLanes;
    for (long long x = x0; x < rows; x += U * step) {
        uint4 v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const long long y = x + u * step;
            if (y >= rows) break;
            const long long z = y / g.L;
            v[u] = src[(z * g.L + buffer_row(g, (int)(y - z * g.L))) * kLanes + c];
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (x + u * step < rows) dst[(x + u * step) * kLanes + c] = v[u];
    }
}

template <int D>
__global__ void __launch_bounds__(kThreads) copy_kernel(const Geometry g, const Copies copies)
{
    constexpr int kLanes = D / 8;
    const long long x0 = (long long)blockIdx.x * (kThreads / kLanes) + threadIdx.x / kLanes, step = (long long)gridDim.x * (kThreads / kLanes);
#pragma unroll
    for (int i = 0; i < 3; ++i) copy_rows<D>(g, copies.src[i], copies.dst[i], copies.rows[i], x0, step);
}

// kCopies: dout's rows in natural order too (dout_copy), and the others.
template <int D, bool kCopies>
__global__ void __launch_bounds__(kThreads) before_kernel(const Geometry g, const void* out, bool out_bf16, const void* dout, uint4* dout_copy,
                                                          const float* lse, float* lse2, float* Dv, float* dq, int padded, long long rows,
                                                          const Copies copies)
{
    constexpr int kLanes = D / 8;
    const int c = threadIdx.x % kLanes * 8;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const long long x0 = (long long)blockIdx.x * (kThreads / kLanes) + threadIdx.x / kLanes, step = (long long)gridDim.x * (kThreads / kLanes);
    const long long up = (rows + 31) / 32 * 32;
    for (long long x = x0; x < up; x += step) {
        const bool has = x < rows;
        const Row r = row_of(g, padded, has ? x : 0);
        float sum = 0.f;
        if (has && r.in) {
            float a[8], b[8];
            const uint4 raw = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(dout) + r.at * D + c);
            load8(out, r.at * D + c, out_bf16, a);
            spread8(raw, b);
            if constexpr (kCopies) dout_copy[((long long)r.z * g.L + r.p) * kLanes + c / 8] = raw;
#pragma unroll
            for (int e = 0; e < 8; ++e) sum = fmaf(a[e], b[e], sum);
        }
#pragma unroll
        for (int s = kLanes / 2; s > 0; s >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, s);
        if (!has) continue;
        const float zero[8] = {};
        store8(dq, x * D + c, false, zero);
        if (c == 0) {
            Dv[x] = sum;
            lse2[x] = r.in ? -kLog2e * lse[r.at] : -INFINITY;
        }
    }
    if constexpr (kCopies) {
#pragma unroll
        for (int i = 0; i < 3; ++i) copy_rows<D>(g, copies.src[i], copies.dst[i], copies.rows[i], x0, step);
    }
}

// dQ's rows, in the buffers' order, and behind them dK and dV of the tiles that were cut: segments [2][128][D] added in order.
struct After {
    Geometry g;
    Band band;
    const float *acc, *part;
    void *dq, *dk, *dv;
    int bf16, padded, sink_tiles, segs, tiles, G, tail_segs;
    long long rows, cut_rows;        // of dQ; of dK and dV, 2 * 128 for each tile that was cut
    long long sink_cut, whole;       // the sinks' tiles of all heads, if they were; then those behind the first `whole` others
};
template <int D, bool kCut>
__global__ void __launch_bounds__(kThreads) after_kernel(const After a)
{
    constexpr int kLanes = D / 8;
    const int c = threadIdx.x % kLanes * 8;
    const long long x0 = (long long)blockIdx.x * (kThreads / kLanes) + threadIdx.x / kLanes, step = (long long)gridDim.x * (kThreads / kLanes);
    asm volatile("griddepcontrol.wait;" ::: "memory");  // for the backward's sums
    for (long long x = x0; x < a.rows; x += step) {
        const int z = (int)(x / a.g.L), r = (int)(x - (long long)z * a.g.L);
        float f[8];
        load8(a.acc, ((long long)z * a.padded + natural_position(a.g, r)) * D + c, false, f);
        store8(a.dq, x * D + c, a.bf16, f);
    }
    if constexpr (kCut) {
        for (long long x = x0; x < a.cut_rows; x += step) {
            const int r = (int)(x % kWindowTile), which = (int)(x / kWindowTile % 2);
            const long long at = x / (2 * kWindowTile), item = at < a.sink_cut ? at : at - a.sink_cut;
            long long slot;
            int z, tile, segs;
            if (at < a.sink_cut) {
                z = (int)(item / a.sink_tiles);
                tile = (int)(item % a.sink_tiles);
                segs = a.segs;
                slot = item * segs;
            } else {
                const int per = a.tiles - a.sink_tiles;
                z = (int)((a.whole + item) / per);
                tile = a.sink_tiles + (int)((a.whole + item) % per);
                segs = a.tail_segs;
                slot = a.sink_cut * a.segs + item * segs;
            }
            const int p = tile * kWindowTile + r;
            if (p >= a.g.L) continue;
            const QueryRun q = query_tiles(a.band, tile * kWindowTile, kWindowTile, kWindowTile);
            const long long n = (long long)(q.last - q.first) * (at < a.sink_cut ? 1 : a.G);
            float sum[8] = {};
            for (int s = 0; s < segs; ++s) {
                if (n * s / segs == n * (s + 1) / segs) continue;  // an empty segment leaves nothing
                float f[8];
                load8(a.part, (((slot + s) * 2 + which) * kWindowTile + r) * D + c, false, f);
#pragma unroll
                for (int e = 0; e < 8; ++e) sum[e] += f[e];
            }
            store8(which ? a.dv : a.dk, ((long long)z * a.g.L + buffer_row(a.g, p)) * D + c, a.bf16, sum);
        }
    }
}

unsigned blocks(long long rows, int d)
{
    const long long per = kThreads / (d / 8), want = (rows + per - 1) / per, most = (long long)device_sm_count() * 16;
    return (unsigned)(want < most ? want : most);
}

size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

// Units of a tile of the last round, and pairs of tiles that each has at least.  (Two sequences of 1000 tokens, units of 8 pairs:
// 25.2 us uncut, 26.2 cut in two, 27.4 in four.)  Of all units the kernel with them costs up to 1 us, a pair takes 1.35: no cut
// where the rounds are more than half the pairs of a unit.
constexpr int kTailSegs = 4, kTailRun = 5;

}  // namespace

WindowBwdPlan window_bwd_plan(const Band& b, int B, int H, int Hkv, int d)
{
    WindowBwdPlan p = {};
    p.tiles = (b.L + kWindowTile - 1) / kWindowTile;
    p.sink_tiles = (b.S + kWindowTile - 1) / kWindowTile;
    p.segs = p.tail_segs = 1;
    const long long near = ((long long)b.W + kWindowTile - 1) / kWindowTile + 1, unit = b.causal ? near : 2 * near - 1;  // query tiles
    if (p.sink_tiles > 0) {
        // segments about as long as the other units, but no more than a few for every SM of any GPU in all
        const long long most = 640 / ((long long)B * Hkv * p.sink_tiles);
        long long segs = (p.tiles + unit - 1) / unit;
        if (segs > most) segs = most;
        p.segs = segs < 1 ? 1 : (int)segs;
        p.sink_items = (long long)B * Hkv * p.sink_tiles * p.segs;
    }
    p.whole = (long long)B * Hkv * (p.tiles - p.sink_tiles);
    const long long last = (p.sink_items + p.whole) % kWindowCtas, cut = last < p.whole ? last : p.whole;
    const long long run = (unit < p.tiles ? unit : p.tiles) * (H / Hkv);  // pairs of tiles of a unit
    if (cut > 0 && 2 * ((p.sink_items + p.whole) / kWindowCtas) <= run) {
        const long long room = (kWindowCtas - (last - cut)) / cut, most = run / kTailRun;
        const long long segs = room < most ? room : most;
        p.tail_segs = segs < 1 ? 1 : segs > kTailSegs ? kTailSegs : (int)segs;
    }
    p.tail = p.tail_segs > 1 ? cut : 0;
    p.whole -= p.tail;
    const size_t rows = (size_t)B * H * p.tiles * kWindowTile;
    p.early = rows * d * sizeof(float) <= (size_t)128 << 20;
    p.lse_at = 0;
    p.D_at = p.lse_at + up256(rows * sizeof(float));
    p.dq_at = p.D_at + up256(rows * sizeof(float));
    p.part_at = p.dq_at + up256(rows * d * sizeof(float));
    p.bytes = p.part_at + up256((size_t)p.parts() * 2 * kWindowTile * d * sizeof(float));
    return p;
}

namespace {

Copies copies_of(const WindowArgs& a, const WindowCopies& w)
{
    Copies c;
    const long long L = a.band.L, q = (long long)a.B * a.H * L, kv = (long long)a.B * a.Hkv * L;
    const void* src[3] = {a.q, a.k, a.v};
    void* dst[3] = {w.q, w.k, w.v};
    for (int i = 0; i < 3; ++i) {
        c.src[i] = static_cast<const uint4*>(src[i]);
        c.dst[i] = static_cast<uint4*>(dst[i]);
        c.rows[i] = i ? kv : q;
    }
    return c;
}

}  // namespace

cudaError_t launch_window_copies(const WindowArgs& a, const WindowCopies& w, int d, cudaStream_t s)
{
    const Copies c = copies_of(a, w);
    if (d == 128)
        copy_kernel<128><<<blocks(c.rows[0], d), kThreads, 0, s>>>(a.store_geo, c);
    else
        copy_kernel<64><<<blocks(c.rows[0], d), kThreads, 0, s>>>(a.store_geo, c);
    return cudaGetLastError();
}

cudaError_t launch_window_bwd_before(const WindowArgs& a, const WindowBwdPlan& p, const WindowCopies& w, int d, cudaStream_t s)
{
    const int padded = p.tiles * kWindowTile;
    const long long rows = (long long)a.B * a.H * padded;
    const Copies c = copies_of(a, w);
    const auto kernel = d == 128 ? (w.dout ? before_kernel<128, true> : before_kernel<128, false>)
                                 : (w.dout ? before_kernel<64, true> : before_kernel<64, false>);
    kernel<<<blocks(rows, d), kThreads, 0, s>>>(a.store_geo, a.out, a.saved_dtype == 1, a.dout, static_cast<uint4*>(w.dout), a.lse, p.lse2, p.D,
                                                p.dq, padded, rows, c);
    return cudaGetLastError();
}

cudaError_t launch_window_bwd_after(const WindowArgs& w, const WindowBwdPlan& p, int d, cudaStream_t s)
{
    After a;
    a.g = w.store_geo;
    a.band = w.band;
    a.acc = p.dq;
    a.part = p.part;
    a.dq = w.dq;
    a.dk = w.dk;
    a.dv = w.dv;
    a.bf16 = w.grad_dtype == 1;
    a.padded = p.tiles * kWindowTile;
    a.sink_tiles = p.sink_tiles;
    a.segs = p.segs;
    a.tiles = p.tiles;
    a.G = w.G;
    a.tail_segs = p.tail_segs;
    a.rows = (long long)w.B * w.H * w.band.L;
    a.sink_cut = p.segs > 1 ? (long long)w.B * w.Hkv * p.sink_tiles : 0;
    a.whole = p.whole;
    a.cut_rows = (a.sink_cut + p.tail) * 2 * kWindowTile;
    const auto kernel = d == 128 ? (a.cut_rows ? after_kernel<128, true> : after_kernel<128, false>)
                                 : (a.cut_rows ? after_kernel<64, true> : after_kernel<64, false>);
    return launch_next(p.early, kernel, blocks(a.rows + a.cut_rows, d), kThreads, 0, s, a);
}

}  // namespace ra
