// window_simt.cu -- attention through a window (window.cuh) on the CUDA cores: float32, any layout and length.
//
// A block of 256 threads takes 64 consecutive positions of one head (queries, or keys in the dK/dV kernel) and walks the
// tiles of 64 that they meet.  Every operand lies transposed in shared memory, [d][64], as float32: the products over the
// head dimension (scores, dout . v) read four values of both operands with two 16-byte loads for 16 multiply-adds, and
// the products over positions (P V, dS K, P^T dO, dS^T Q) read four consecutive positions of a column likewise.
// Backward: blocks over query tiles for dQ, and over key tiles and query heads for dK and dV, both recompute P =
// exp(s - lse): seven products in place of five, and no sum whose order varies.  The heads' parts of dK and dV, and the
// segments' of the sinks' tiles, which all later queries see, are added in order by a last launch.
//
// What bounds it: the 16-byte loads from shared memory, two for 16 multiply-adds, and what the few warps of a block leave of
// their latency.  4096 tokens of 8 : 2 heads of 128, window 1024: forward 661 us (23 TFLOP/s), backward 1.81 ms; 1235
// tokens of 6 : 2 heads of 64, window 200: 43 and 94 us.  Eight rows a thread in place of four: head dim 64 as fast, 128 a tenth
// slower (too few warps).
#include <cuda_bf16.h>
#include <math.h>

#include <mutex>

#include "window.cuh"

namespace ra {
namespace {

constexpr int kT = 64, kStride = kT + 4, kThreads = 256;

__device__ __forceinline__ void load4(const float* p, float (&f)[4])
{
    const float4 v = *reinterpret_cast<const float4*>(p);
    f[0] = v.x, f[1] = v.y, f[2] = v.z, f[3] = v.w;
}
__device__ __forceinline__ void store1(void* p, long long i, float v, int dtype)
{
    if (dtype == 1)
        static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
    else
        static_cast<float*>(p)[i] = v;
}

// 64 positions from p0 of one head's rows: fetched into registers, and put into shared memory, transposed to [D][kStride];
// positions past the sequence are zeros.  Both tiles of a step are fetched before the barrier that frees their room: all
// loads are then on their way at once, beside the other warps' last products (1235 tokens of 6 heads of 64, forward 43 us in
// place of 48).  Fetched a whole tile ahead: no faster with one block on an SM, head dim 128, and a block fewer at head dim 64
// (4096 tokens of 32 heads 848 us in place of 716).
template <int D>
struct Tile {
    float f[D / 16][4];
    __device__ __forceinline__ void fetch(const Geometry& g, const float* head, int p0)
    {
        const int p = p0 + threadIdx.x % kT;
        const float* src = p < g.L ? head + (long long)buffer_row(g, p) * D + threadIdx.x / kT * 4 : nullptr;
#pragma unroll
        for (int u = 0; u < D / 16; ++u) {
#pragma unroll
            for (int i = 0; i < 4; ++i) f[u][i] = 0.f;
            if (src) load4(src + 16 * u, f[u]);
        }
    }
    // Is a value that this thread has not finite?
    __device__ __forceinline__ bool put(float* dst, float scale = 1.f) const
    {
        dst += threadIdx.x / kT * 4 * kStride + threadIdx.x % kT;
        float odd = 0.f;  // NaN if one is
#pragma unroll
        for (int u = 0; u < D / 16; ++u)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                dst[(16 * u + i) * kStride] = f[u][i] * scale;
                odd = fmaf(f[u][i], 0.f, odd);
            }
        return odd != 0.f;
    }
};
static_assert(kThreads / kT * 4 == 16, "a thread's columns");

template <int D>
__device__ __forceinline__ void load_tile(const Geometry& g, const float* head, int p0, float* dst, float scale = 1.f)
{
    Tile<D> t;
    t.fetch(g, head, p0);
    t.put(dst, scale);
}

// acc[i][j] += sum_c a[c][4 ty + i] b[c][4 tx + j].
template <int D>
__device__ __forceinline__ void dot_tile(const float* a, const float* b, float (&acc)[4][4])
{
    const float* pa = a + threadIdx.x / 16 * 4;
    const float* pb = b + threadIdx.x % 16 * 4;
#pragma unroll 8
    for (int c = 0; c < D; ++c) {
        float x[4], y[4];
        load4(pa + c * kStride, x);
        load4(pb + c * kStride, y);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(x[i], y[j], acc[i][j]);
    }
}

constexpr float kMaxF32 = 3.4028234e38f;

// acc[i][k] += sum_j w[4 ty + i][j] b[tx + 16 k][j].  Hidden terms have a weight of 0.  Where b holds what is not finite they
// are left out, so that it stays out of the sums: they are then marked by a weight below 0 (kNegative: P) or by the 0 (kZero: dS).
// kValues: as kNegative, and what is not finite and seen counts whole, also with a weight that is 0 in float32 only.
enum Hidden { kNone, kNegative, kZero, kValues };
template <int D, Hidden kHow>
__device__ __forceinline__ void apply_rows(const float* w, const float* b, float (&acc)[4][D / 16])
{
    const float* pw = w + threadIdx.x / 16 * 4 * kStride;
    const float* pb = b + threadIdx.x % 16 * kStride;
#pragma unroll 2
    for (int j = 0; j < kT; j += 4) {
        float x[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) load4(pw + i * kStride + j, x[i]);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
            float y[4];
            load4(pb + 16 * k * kStride + j, y);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (kHow == kValues && x[i][e] == 0.f && !(fabsf(y[e]) <= kMaxF32))
                        acc[i][k] += y[e];
                    else if (kHow == kNone || (kHow == kZero ? x[i][e] != 0.f : !(x[i][e] < 0.f)))
                        acc[i][k] = fmaf(x[i][e], y[e], acc[i][k]);
                }
        }
    }
}
template <int D, Hidden kHow>
__device__ __forceinline__ void apply_tile(bool plain, const float* w, const float* b, float (&acc)[4][D / 16])
{
    if (plain)
        apply_rows<D, kNone>(w, b, acc);
    else
        apply_rows<D, kHow>(w, b, acc);
}

__device__ __forceinline__ void put4(float* w, const float (&x)[4][4])
{
#pragma unroll
    for (int i = 0; i < 4; ++i)
        *reinterpret_cast<float4*>(w + (threadIdx.x / 16 * 4 + i) * kStride + threadIdx.x % 16 * 4) =
            make_float4(x[i][0], x[i][1], x[i][2], x[i][3]);
}

__device__ __forceinline__ float max16(float v)
{
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
__device__ __forceinline__ float sum16(float v)
{
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

template <int D>
__global__ void __launch_bounds__(kThreads) window_fwd_simt_kernel(const WindowArgs a)
{
    extern __shared__ __align__(16) float sm[];
    float *sq = sm, *sk = sq + D * kStride, *sv = sk + D * kStride, *sp = sv + D * kStride;
    const int tiles = (a.band.L + kT - 1) / kT;
    const int q0 = (int)(blockIdx.x % tiles) * kT, zq = (int)(blockIdx.x / tiles), zk = zq / a.G;  // (b H + h) / G = b Hkv + g
    const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
    const long long per = (long long)a.band.L * D;
    load_tile<D>(a.geo, static_cast<const float*>(a.q) + zq * per, q0, sq, a.scale_log2);
    float m[4], l[4], o[4][D / 16];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.f;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) o[i][k] = 0.f;
    }
    const TileRun run = key_tiles(a.band, q0, kT, kT);
    for (int t = 0; t < run.count(); ++t) {
        const int k0 = run.at(t) * kT;
        Tile<D> tk, tv;
        tk.fetch(a.geo, static_cast<const float*>(a.k) + zk * per, k0);
        tv.fetch(a.geo, static_cast<const float*>(a.v) + zk * per, k0);
        __syncthreads();
        tk.put(sk);
        const bool odd = __syncthreads_or(tv.put(sv));
        float s[4][4] = {};
        dot_tile<D>(sq, sk, s);
        const bool whole = band_tile_whole(a.band, q0, kT, k0, kT);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int p = q0 + 4 * ty + i;
            float mx = -INFINITY, sum = 0.f;
            unsigned hidden = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int key = k0 + 4 * tx + j;
                if (!whole && (key >= a.band.L || !band_sees(a.band, p, key))) hidden |= 1u << j;
                if (!(hidden >> j & 1u)) mx = fmaxf(mx, s[i][j]);
            }
            const float mn = fmaxf(m[i], max16(mx)), ref = mn == -INFINITY ? 0.f : mn, alpha = exp2f(m[i] - ref);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const bool hides = hidden >> j & 1u;
                s[i][j] = hides ? 0.f : exp2f(s[i][j] - ref);
                sum += s[i][j];
                if (odd && hides) s[i][j] = -1.f;
            }
            l[i] = l[i] * alpha + sum16(sum);
            m[i] = mn;
            if (alpha != 0.f) {
#pragma unroll
                for (int k = 0; k < D / 16; ++k) o[i][k] *= alpha;
            } else {
#pragma unroll
                for (int k = 0; k < D / 16; ++k)
                    if (fabsf(o[i][k]) <= kMaxF32) o[i][k] = 0.f;  // (what is not finite stays)
            }
        }
        put4(sp, s);
        __syncthreads();
        apply_tile<D, kValues>(!odd, sp, sv, o);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int p = q0 + 4 * ty + i;
        if (p >= a.band.L) continue;
        const long long row = (long long)zq * a.band.L + buffer_row(a.geo, p);
        const float inv = 1.f / l[i];
#pragma unroll
        for (int k = 0; k < D / 16; ++k) static_cast<float*>(a.o)[row * D + tx + 16 * k] = o[i][k] * inv;
        if (tx == 0) a.lse[row] = (m[i] + log2f(l[i])) * kLn2;
    }
}

// P (`hides` where hidden) and dS (0) of a tile whose rows are queries, or keys, from the scores and dout . v.
template <bool kKeyRows>
__device__ __forceinline__ void weights(const WindowArgs& a, int r0, int c0, float hides, const float (&lse2)[4], const float (&Dv)[4], float (&s)[4][4],
                                        float (&dp)[4][4])
{
    const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int r = r0 + 4 * ty + i, c = c0 + 4 * tx + j, p = kKeyRows ? c : r, key = kKeyRows ? r : c;
            const bool sees = p < a.band.L && key < a.band.L && band_sees(a.band, p, key);
            s[i][j] = sees ? exp2f(s[i][j] - lse2[kKeyRows ? j : i]) : hides;
            dp[i][j] = sees ? s[i][j] * (dp[i][j] - Dv[kKeyRows ? j : i]) * a.scale : 0.f;
        }
}

// dQ of 64 queries.
template <int D>
__device__ __forceinline__ void bwd_queries(const WindowArgs& a, float* sm, int zq, int q0)
{
    float *sq = sm, *sd = sq + D * kStride, *sk = sd + D * kStride, *sv = sk + D * kStride, *sp = sv + D * kStride;
    const int zk = zq / a.G, ty = threadIdx.x / 16, tx = threadIdx.x % 16;
    const long long per = (long long)a.band.L * D;
    load_tile<D>(a.geo, static_cast<const float*>(a.q) + zq * per, q0, sq, a.scale_log2);
    load_tile<D>(a.geo, static_cast<const float*>(a.dout) + zq * per, q0, sd);
    float lse2[4], Dv[4], acc[4][D / 16] = {};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int p = q0 + 4 * ty + i;
        const bool has = p < a.band.L;
        lse2[i] = has ? a.lse[(long long)zq * a.band.L + buffer_row(a.geo, p)] * kLog2e : 0.f;
        Dv[i] = has ? a.D[(long long)zq * a.band.L + p] : 0.f;
    }
    const TileRun run = key_tiles(a.band, q0, kT, kT);
    for (int t = 0; t < run.count(); ++t) {
        const int k0 = run.at(t) * kT;
        Tile<D> tk, tv;
        tk.fetch(a.geo, static_cast<const float*>(a.k) + zk * per, k0);
        tv.fetch(a.geo, static_cast<const float*>(a.v) + zk * per, k0);
        __syncthreads();
        tv.put(sv);
        const bool odd = __syncthreads_or(tk.put(sk));
        float s[4][4] = {}, dp[4][4] = {};
        dot_tile<D>(sq, sk, s);
        dot_tile<D>(sd, sv, dp);
        weights<false>(a, q0, k0, 0.f, lse2, Dv, s, dp);
        put4(sp, dp);
        __syncthreads();
        apply_tile<D, kZero>(!odd || band_tile_whole(a.band, q0, kT, k0, kT), sp, sk, acc);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int p = q0 + 4 * ty + i;
        if (p >= a.band.L) continue;
        const long long row = (long long)zq * a.band.L + buffer_row(a.geo, p);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) store1(a.dq, row * D + tx + 16 * k, acc[i][k], a.grad_dtype);
    }
}

// dK and dV of 64 keys from one query head and the query tiles [t0, t1): to the gradients, or to `part` [2][64][D].
template <int D>
__device__ __forceinline__ void bwd_keys(const WindowArgs& a, float* sm, int zq, int k0, int t0, int t1, float* part)
{
    float *sk = sm, *sv = sk + D * kStride, *sq = sv + D * kStride, *sd = sq + D * kStride, *sp = sd + D * kStride, *ss = sp + kT * kStride;
    const int zk = zq / a.G, ty = threadIdx.x / 16, tx = threadIdx.x % 16;
    const long long per = (long long)a.band.L * D;
    load_tile<D>(a.geo, static_cast<const float*>(a.k) + zk * per, k0, sk, a.scale_log2);
    load_tile<D>(a.geo, static_cast<const float*>(a.v) + zk * per, k0, sv);
    float dk[4][D / 16] = {}, dv[4][D / 16] = {};
    for (int t = t0; t < t1; ++t) {
        const int q0 = t * kT;
        Tile<D> tq, td;
        tq.fetch(a.geo, static_cast<const float*>(a.q) + zq * per, q0);
        td.fetch(a.geo, static_cast<const float*>(a.dout) + zq * per, q0);
        __syncthreads();
        bool odd = tq.put(sq);
        odd |= td.put(sd);
        float lse2[4], Dv[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int p = q0 + 4 * tx + j;
            const bool has = p < a.band.L;
            lse2[j] = has ? a.lse[(long long)zq * a.band.L + buffer_row(a.geo, p)] * kLog2e : 0.f;
            Dv[j] = has ? a.D[(long long)zq * a.band.L + p] : 0.f;
        }
        odd = __syncthreads_or(odd);
        float s[4][4] = {}, dp[4][4] = {};
        dot_tile<D>(sk, sq, s);
        dot_tile<D>(sv, sd, dp);
        weights<true>(a, k0, q0, odd ? -1.f : 0.f, lse2, Dv, s, dp);
        put4(sp, s);
        put4(ss, dp);
        __syncthreads();
        const bool plain = !odd || band_tile_whole(a.band, q0, kT, k0, kT);
        apply_tile<D, kNegative>(plain, sp, sd, dv);
        apply_tile<D, kZero>(plain, ss, sq, dk);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = 4 * ty + i;
        if (k0 + r >= a.band.L) continue;
        const long long row = (long long)zk * a.band.L + buffer_row(a.geo, k0 + r);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
            const int c = tx + 16 * k;
            if (part) {
                part[r * D + c] = dk[i][k];
                part[(kT + r) * D + c] = dv[i][k];
            } else {
                store1(a.dk, row * D + c, dk[i][k], a.grad_dtype);
                store1(a.dv, row * D + c, dv[i][k], a.grad_dtype);
            }
        }
    }
}

// One launch for both, so that the blocks of each fill the SMs beside the other's.  The sinks' tiles come first, in
// segments: they are the longest.
template <int D>
__global__ void __launch_bounds__(kThreads) window_bwd_simt_kernel(const WindowArgs a, const WindowSimtPlan p, float* parts)
{
    extern __shared__ __align__(16) float sm[];
    long long x = blockIdx.x;
    if (x < p.key_blocks) {
        const int zq = (int)(x % ((long long)a.B * a.H));
        int tile = (int)(x / ((long long)a.B * a.H)), seg = 0, segs = 1;
        if (tile < p.sink_tiles * p.segs) {
            seg = tile % p.segs;
            tile /= p.segs;
            segs = p.segs;
        } else {
            tile -= p.sink_tiles * (p.segs - 1);
        }
        const QueryRun run = query_tiles(a.band, tile * kT, kT, kT);
        const int n = run.last - run.first;
        bwd_keys<D>(a, sm, zq, tile * kT, run.first + (int)((long long)n * seg / segs), run.first + (int)((long long)n * (seg + 1) / segs),
                    p.parts ? parts + x * 2 * kT * D : nullptr);
    } else {
        x -= p.key_blocks;
        bwd_queries<D>(a, sm, (int)(x / p.tiles), (int)(x % p.tiles) * kT);
    }
}

// dK and dV: the parts of a tile's query heads and segments, added in order.
template <int D>
__global__ void __launch_bounds__(kThreads) window_join_simt_kernel(const WindowArgs a, const WindowSimtPlan p, const float* parts)
{
    const long long total = (long long)a.B * a.Hkv * a.band.L * D, heads = (long long)a.B * a.H;
    for (long long e = (long long)blockIdx.x * kThreads + threadIdx.x; e < total; e += (long long)gridDim.x * kThreads) {
        const int c = (int)(e % D), zk = (int)(e / D / a.band.L), pos = (int)(e / D - (long long)zk * a.band.L);
        const int tile = pos / kT, r = pos % kT;
        const bool sink = tile < p.sink_tiles;
        const int segs = sink ? p.segs : 1;
        const long long slot = sink ? (long long)tile * p.segs : tile + (long long)p.sink_tiles * (p.segs - 1);
        float dk = 0.f, dv = 0.f;
        for (int h = 0; h < a.G; ++h)
            for (int s = 0; s < segs; ++s) {
                const float* x = parts + ((slot + s) * heads + (long long)zk * a.G + h) * 2 * kT * D + r * D + c;
                dk += x[0];
                dv += x[kT * D];
            }
        const long long row = (long long)zk * a.band.L + buffer_row(a.geo, pos);
        store1(a.dk, row * D + c, dk, a.grad_dtype);
        store1(a.dv, row * D + c, dv, a.grad_dtype);
    }
}

// D = dout . out per row, in natural order: a warp per row.
template <int D>
__global__ void __launch_bounds__(kThreads) window_rowdot_kernel(const WindowArgs a, float* Dv)
{
    const long long rows = (long long)a.B * a.H * a.band.L;
    const int lane = threadIdx.x & 31;
    for (long long x = (long long)blockIdx.x * (kThreads / 32) + threadIdx.x / 32; x < rows; x += (long long)gridDim.x * (kThreads / 32)) {
        const long long z = x / a.band.L, row = z * a.band.L + buffer_row(a.geo, (int)(x - z * a.band.L));
        float sum = 0.f;
        for (int c = lane; c < D; c += 32) {
            sum = fmaf(static_cast<const float*>(a.out)[row * D + c], static_cast<const float*>(a.dout)[row * D + c], sum);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane == 0) Dv[x] = sum;
    }
}

constexpr size_t tile_bytes(int d) { return (size_t)d * kStride * sizeof(float); }
constexpr size_t kWeightBytes = (size_t)kT * kStride * sizeof(float);

template <typename K>
cudaError_t allow(K kernel, size_t smem, std::mutex& mu, bool (&done)[64])
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lk(mu);
    if (!done[dev]) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
        done[dev] = true;
    }
    return cudaSuccess;
}

template <int D>
cudaError_t fwd(const WindowArgs& a, cudaStream_t s)
{
    static std::mutex mu;
    static bool done[64];
    constexpr size_t smem = 3 * tile_bytes(D) + kWeightBytes;
    cudaError_t e = allow(window_fwd_simt_kernel<D>, smem, mu, done);
    if (e != cudaSuccess) return e;
    const long long blocks = (long long)a.B * a.H * ((a.band.L + kT - 1) / kT);
    window_fwd_simt_kernel<D><<<(unsigned)blocks, kThreads, smem, s>>>(a);
    return cudaGetLastError();
}

template <int D>
cudaError_t bwd(const WindowArgs& a, const WindowSimtPlan& p, float* Dv, float* parts, cudaStream_t s)
{
    static std::mutex mu;
    static bool done[64];
    constexpr size_t smem = 4 * tile_bytes(D) + 2 * kWeightBytes;
    cudaError_t e = allow(window_bwd_simt_kernel<D>, smem, mu, done);
    if (e != cudaSuccess) return e;
    const long long rows = (long long)a.B * a.H * a.band.L, need = (rows + kThreads / 32 - 1) / (kThreads / 32);
    const long long most = (long long)device_sm_count() * 8;
    window_rowdot_kernel<D><<<(unsigned)(need < most ? need : most), kThreads, 0, s>>>(a, Dv);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    window_bwd_simt_kernel<D><<<(unsigned)(p.key_blocks + a.B * (long long)a.H * p.tiles), kThreads, smem, s>>>(a, p, parts);
    if ((e = cudaGetLastError()) != cudaSuccess || !p.parts) return e;
    const long long blocks = ((long long)a.B * a.Hkv * a.band.L * D + kThreads - 1) / kThreads;
    window_join_simt_kernel<D><<<(unsigned)(blocks < most ? blocks : most), kThreads, 0, s>>>(a, p, parts);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_window_fwd_simt(const WindowArgs& a, int d, cudaStream_t s)
{
    return d == 128 ? fwd<128>(a, s) : fwd<64>(a, s);
}

WindowSimtPlan window_simt_plan(const Band& b, int B, int H, int Hkv, int d)
{
    WindowSimtPlan p = {};
    p.tiles = (b.L + kT - 1) / kT;
    p.sink_tiles = (b.S + kT - 1) / kT;
    p.segs = 1;
    if (p.sink_tiles > 0) {  // segments about as long as the other tiles' runs, but no more than a few for every SM in all
        const long long near = ((long long)b.W + kT - 1) / kT + 1, unit = b.causal ? near : 2 * near - 1;
        const long long most = 1024 / ((long long)B * H * p.sink_tiles);
        long long segs = (p.tiles + unit - 1) / unit;
        if (segs > most) segs = most;
        p.segs = segs < 1 ? 1 : (int)segs;
    }
    p.key_blocks = (long long)B * H * (p.tiles + (long long)p.sink_tiles * (p.segs - 1));
    p.parts = H != Hkv || p.segs > 1;
    p.D_bytes = ((size_t)B * H * b.L * sizeof(float) + 255) & ~size_t(255);
    p.bytes = p.D_bytes + (p.parts ? (size_t)p.key_blocks * 2 * kT * d * sizeof(float) : 0);
    return p;
}

cudaError_t launch_window_bwd_simt(const WindowArgs& args, const WindowSimtPlan& p, void* workspace, int d, cudaStream_t s)
{
    WindowArgs a = args;
    float *D = static_cast<float*>(workspace), *parts = reinterpret_cast<float*>(static_cast<char*>(workspace) + p.D_bytes);
    a.D = D;
    return d == 128 ? bwd<128>(a, p, D, parts, s) : bwd<64>(a, p, D, parts, s);
}

}  // namespace ra
