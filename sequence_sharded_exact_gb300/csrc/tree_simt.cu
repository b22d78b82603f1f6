// tree_simt.cu -- attention over a cache (tree.cuh) on the CUDA cores: float32 queries, any cache.
//
// Four warps work through the CTA's tiles in chunks of 32 cached rows, staged in shared memory as
// float32.  Scores: lane = cached row, each warp takes kRows / 4 query rows, so a row's maximum and sum
// are shuffles in its warp, which alone keeps that row's running (m, l).  Output: thread = column (two
// threads share a column's query rows when d = 64), the weights come from shared memory.  Masked
// weights are stored as -1 and left out by a comparison, so that a masked row's values never meet the sums.
//
// What bounds it: shared memory, which every product is fed from (the most frequent stall; an instruction is issued in 0.39
// of the cycles).  A chunk of 16 query rows is 512 fused multiply-adds and about 200 loads from shared memory per
// thread; each of the next chunk's loads from memory is under way meanwhile.  Four CTAs on an SM leave 128 registers a
// thread: 12 rows spill 28 bytes of them at d = 64 and 88 at d = 128.  128 rows of d = 64 against 20 query rows (two
// tiles of 12) cost an SM 6.9 us; with two tiles of 16 and loads that are waited for at once 11.5.  Tiles are 32 rows, a
// chunk, so that short caches spread over all SMs: one sequence of 9000 rows and 20 query rows 19 + 9 us (both
// launches) in place of 25 + 12.
#include "ra_internal.h"
#include "ra_ptx.cuh"
#include "tree.cuh"

namespace ra {
namespace {

constexpr int kThreads = 128;
constexpr int kChunk = 32;
static_assert(kTreeSimtTile % kChunk == 0, "a tile is whole chunks");

// 16 bytes of a cached row as float32.
template <typename T>
__device__ __forceinline__ void spread16(const uint4& v, float up, float* f);
template <>
__device__ __forceinline__ void spread16<float>(const uint4& v, float, float* f)
{
    f[0] = __uint_as_float(v.x);
    f[1] = __uint_as_float(v.y);
    f[2] = __uint_as_float(v.z);
    f[3] = __uint_as_float(v.w);
}
template <>
__device__ __forceinline__ void spread16<uint8_t>(const uint4& v, float up, float* f)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        e4m3x4_to_float(w[i], f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
#pragma unroll
        for (int j = 0; j < 4; ++j) f[4 * i + j] *= up;
    }
}

// A thread's part of a chunk's keys and values as they are cached, on their way from memory while the chunk before
// is worked on; rows from `end` on are zeros.
template <typename TC, int D>
struct Chunk {
    static constexpr int kPer = 16 / sizeof(TC), kN = kChunk * D / kPer / kThreads;
    uint4 k[kN], v[kN];
    float uk[kN], uv[kN];
    __device__ __forceinline__ void load(const TreeArgs& a, long long row0, int k0, int end)
    {
#pragma unroll
        for (int n = 0; n < kN; ++n) {
            const int e = threadIdx.x + n * kThreads, j = e / (D / kPer), c = e % (D / kPer) * kPer;
            k[n] = v[n] = make_uint4(0, 0, 0, 0);
            uk[n] = uv[n] = 1.f;
            if (k0 + j >= end) continue;
            const long long src = row0 + k0 + j;
            if (sizeof(TC) == 1) {
                uk[n] = __uint_as_float((uint32_t)a.k_exp[src] << 23);
                uv[n] = __uint_as_float((uint32_t)a.v_exp[src] << 23);
            }
            k[n] = *reinterpret_cast<const uint4*>(static_cast<const TC*>(a.k) + src * D + c);
            v[n] = *reinterpret_cast<const uint4*>(static_cast<const TC*>(a.v) + src * D + c);
        }
    }
    template <int kStride>
    __device__ __forceinline__ void store(float (*ks)[kStride], float (*vs)[D]) const
    {
#pragma unroll
        for (int n = 0; n < kN; ++n) {
            const int e = threadIdx.x + n * kThreads, j = e / (D / kPer), c = e % (D / kPer) * kPer;
            float fk[kPer], fv[kPer];
            spread16<TC>(k[n], uk[n], fk);
            spread16<TC>(v[n], uv[n], fv);
#pragma unroll
            for (int i = 0; i < kPer; i += 4) {
                *reinterpret_cast<float4*>(&ks[j][c + i]) = make_float4(fk[i], fk[i + 1], fk[i + 2], fk[i + 3]);
                *reinterpret_cast<float4*>(&vs[j][c + i]) = make_float4(fv[i], fv[i + 1], fv[i + 2], fv[i + 3]);
            }
        }
    }
};

template <typename TC, int D, int ROWS>
__global__ void __launch_bounds__(kThreads, kTreeSimtCtasPerSm) tree_simt_kernel(const TreeArgs a)
{
    constexpr int RW = ROWS / 4;            // query rows per warp in the scores
    constexpr int SPLIT = kThreads / D;     // threads per output column
    constexpr int RC = ROWS / SPLIT;        // query rows per thread in the output
    constexpr int kStride = D + 4;          // keys: consecutive rows fall into different banks
    __shared__ __align__(16) float qs[ROWS][D];
    __shared__ __align__(16) float ks[kChunk][kStride];
    __shared__ __align__(16) float vs[kChunk][D];
    __shared__ __align__(16) float ps[ROWS][kChunk];
    __shared__ float al[ROWS];
    __shared__ float ml[ROWS][2];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int col = tid % D, part = tid / D;
    TreeWalk w;
    int4 border = make_int4(-1, 0, 0, 0);
    if (!w.begin(a, blockIdx.x)) {
        if (tid == 0) a.border[blockIdx.x] = border;
        return;
    }
    do {
        if (w.goes_on()) border = w.border(a, blockIdx.x);
        const long long head = (long long)w.b * a.Hkv + w.g;
        const float* q = static_cast<const float*>(a.q) + (head * a.R + (long long)w.r * a.rt) * D;
        const int rows = a.R - w.r * a.rt < a.rt ? a.R - w.r * a.rt : a.rt;
        __syncthreads();
        for (int e = tid; e < ROWS * D; e += kThreads) {
            const int x = e / D;
            qs[x][e % D] = x < rows ? q[e] * a.scale_log2 : 0.f;
        }
        float m[RW], l[RW], acc[RC];
#pragma unroll
        for (int i = 0; i < RW; ++i) {
            m[i] = -INFINITY;
            l[i] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < RC; ++i) acc[i] = 0.f;
        const int end = w.t1 * kTreeSimtTile < w.s.end ? w.t1 * kTreeSimtTile : w.s.end;
        Chunk<TC, D> next;
        next.load(a, head * a.cap, w.t0 * kTreeSimtTile, end);
        for (int k0 = w.t0 * kTreeSimtTile; k0 < end; k0 += kChunk) {
            __syncthreads();
            next.store(ks, vs);
            if (k0 + kChunk < end) next.load(a, head * a.cap, k0 + kChunk, end);
            __syncthreads();
            float sc[RW];
#pragma unroll
            for (int i = 0; i < RW; ++i) sc[i] = 0.f;
#pragma unroll 4
            for (int c = 0; c < D; c += 4) {
                const float4 kv = *reinterpret_cast<const float4*>(&ks[lane][c]);
#pragma unroll
                for (int i = 0; i < RW; ++i) {
                    const float4 qv = *reinterpret_cast<const float4*>(&qs[warp * RW + i][c]);
                    sc[i] = fmaf(qv.x, kv.x, sc[i]);
                    sc[i] = fmaf(qv.y, kv.y, sc[i]);
                    sc[i] = fmaf(qv.z, kv.z, sc[i]);
                    sc[i] = fmaf(qv.w, kv.w, sc[i]);
                }
            }
            const int key = k0 + lane;
            const bool drafted = k0 + kChunk > w.s.len;  // the chunk holds drafted tokens, or rows past the end
#pragma unroll
            for (int i = 0; i < RW; ++i) {
                const int x = w.r * a.rt + warp * RW + i, t = x % a.T;
                bool sees = key < end;
                if (drafted && key >= w.s.len && sees) sees = t < w.s.cnt && x < a.R && tree_sees(a, w.b, t, key - w.s.len);
                float mx = sees ? sc[i] : -INFINITY;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                const float mn = fmaxf(m[i], mx), ref = mn == -INFINITY ? 0.f : mn;
                const float p = sees ? ex2_approx(sc[i] - ref) : 0.f;
                const float alpha = ex2_approx(m[i] - ref);
                float sum = p;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                l[i] = l[i] * alpha + sum;
                m[i] = mn;
                ps[warp * RW + i][lane] = sees ? p : -1.f;
                if (lane == 0) al[warp * RW + i] = alpha;
            }
            __syncthreads();
#pragma unroll
            for (int i = 0; i < RC; ++i) acc[i] *= al[part * RC + i];
            if (!drafted) {
#pragma unroll 2
                for (int j = 0; j < kChunk; j += 4) {
                    const float v0 = vs[j][col], v1 = vs[j + 1][col], v2 = vs[j + 2][col], v3 = vs[j + 3][col];
#pragma unroll
                    for (int i = 0; i < RC; ++i) {
                        const float4 pv = *reinterpret_cast<const float4*>(&ps[part * RC + i][j]);
                        acc[i] = fmaf(pv.x, v0, acc[i]);
                        acc[i] = fmaf(pv.y, v1, acc[i]);
                        acc[i] = fmaf(pv.z, v2, acc[i]);
                        acc[i] = fmaf(pv.w, v3, acc[i]);
                    }
                }
            } else {
                for (int j = 0; j < kChunk; ++j) {
                    const float v0 = vs[j][col];
#pragma unroll
                    for (int i = 0; i < RC; ++i) {
                        const float p = ps[part * RC + i][j];
                        if (!(p < 0.f)) acc[i] = fmaf(p, v0, acc[i]);  // NaN weights stay
                    }
                }
            }
        }
#pragma unroll
        for (int i = 0; i < RW; ++i)
            if (lane == 0) {
                ml[warp * RW + i][0] = m[i];
                ml[warp * RW + i][1] = l[i];
            }
        __syncthreads();
        const bool whole = w.whole();
        const long long slot = (long long)blockIdx.x * 2 + (w.first ? 0 : 1);
#pragma unroll
        for (int i = 0; i < RC; ++i) {
            const int x = part * RC + i;
            if (x >= rows) continue;
            const float mm = ml[x][0], ll = ml[x][1];
            if (whole) {
                const bool none = (mm == -INFINITY && ll == 0.f) || (w.r * a.rt + x) % a.T >= w.s.cnt;
                const float o = none ? 0.f : acc[i] / ll;
                const long long dst = head * a.R + w.r * a.rt + x;
                static_cast<float*>(a.out)[dst * D + col] = o;
                if (col == 0) a.lse[dst] = none ? -INFINITY : (mm + log2f(ll)) * kLn2;
            } else {
                a.part_o[(slot * D + col) * a.rt + x] = acc[i];
                if (col == 0) *reinterpret_cast<float4*>(a.part_ml + (slot * a.rt + x) * 4) = make_float4(mm, ll, ll, 0.f);
            }
        }
    } while (w.next(a));
    if (tid == 0) a.border[blockIdx.x] = border;
}

template <typename TC, int D>
cudaError_t launch_rows(const TreeArgs& a, cudaStream_t s)
{
    switch (a.rt) {
        case 4: tree_simt_kernel<TC, D, 4><<<a.ctas, kThreads, 0, s>>>(a); break;
        case 8: tree_simt_kernel<TC, D, 8><<<a.ctas, kThreads, 0, s>>>(a); break;
        case 12: tree_simt_kernel<TC, D, 12><<<a.ctas, kThreads, 0, s>>>(a); break;
        default: tree_simt_kernel<TC, D, 16><<<a.ctas, kThreads, 0, s>>>(a);
    }
    return cudaGetLastError();
}

template <typename TC>
cudaError_t launch_d(const TreeArgs& a, int d, cudaStream_t s)
{
    return d == 128 ? launch_rows<TC, 128>(a, s) : launch_rows<TC, 64>(a, s);
}

}  // namespace

// Query rows per tile, a multiple of 4 (the warps): as few tiles as 16 rows each allow, and as even.
int tree_simt_rows(int R)
{
    const int tiles = (R + 15) / 16, rows = (R + tiles - 1) / tiles;
    return (rows + 3) / 4 * 4;
}

cudaError_t launch_tree_simt(const TreeArgs& a, int d, int cache_dtype, cudaStream_t s)
{
    return cache_dtype == kCacheE4m3 ? launch_d<uint8_t>(a, d, s) : launch_d<float>(a, d, s);
}

}  // namespace ra
