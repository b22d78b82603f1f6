// norm_rope.cu -- the norm of every query and key head with the rotation by natural position in the
// same pass, and its backward (HBM-bound).
//
// Forward, for one row x of d elements (one head of one token at natural position p), w the weights
// of its kind (queries or keys), R(p) the rotation of rope.cu (pair (2i, 2i+1) by p base^(-2i/d)):
//   r = 1 / sqrt(mean(x^2) + eps),   y = R(p) (x r w).
// Backward, with g = R(-p) dy:
//   dw = sum over rows of g x r,   u = g w,   dx = r (u - x r^2 mean(u x)).
// Nothing of the forward is kept but x: r costs one reduction that the backward needs the row for
// anyway, so storing it would add traffic and save nothing.
//
// What bounds it: the forward reads and writes each element once, the backward reads two and
// writes one; the arithmetic is below 20 operations an element.  16 bytes per lane, d * size / 16
// lanes per row, so a row's sums are shuffles inside the group that holds it.  A group owns one
// (batch, position) and walks heads: the angles (64-bit fixed-point turns, as in rope.cu) are
// computed once for all the heads it walks, which counts: with 8 heads per group in place of 40 the
// forward of 64K positions took 258 us in place of 214 (as it was then).  Loads of four heads are issued before the
// first is used (two or eight: 240, 232 us).  All sums are float32; the output is rounded once.
//
// Positions with several axes (time, height, width of images and video): each pair of a head takes the position along
// its axis, read once per group; everything else is as above.  Without weights the rotation alone, whose gradient is
// the rotation back.  Measured, 48K tokens of 32 + 8 heads of 128 in bf16 with three axes and the norm: forward 166 us (6.05 TB/s,
// 0.89 of the copy rate; one position 163), backward 249 us (0.90).  The rows fetched into L2 ahead of the positions: 162 us,
// but 61 in place of 58 at 16K tokens.
//
// With few tokens one group per position would leave most SMs idle, so the heads of a position are
// then split over several groups, which repeat the angles.
//
// Measured, 64K positions of 32 + 8 heads of 128 in bf16: forward 208 us (6.45 TB/s, 0.95 of the copy
// rate), backward 320 us (6.30 TB/s, 0.93).  What is left are the shuffles and the products between
// loads: more heads in flight cost registers and so the other blocks that hide them (the bf16 forward spills 40 bytes as
// it is, to keep four blocks on an SM).  32 bytes a lane in place of 16 took the forward 6 us further and the backward 14 back, and would need rows on 32-byte
// boundaries.
#include <cuda_bf16.h>
#include <math.h>
#include <string.h>

#include "ra_internal.h"

namespace ra {
namespace {

constexpr int kThreads = 256;

struct NormRopeArgs {
    Geometry geo;
    int B, H, Hkv, rows, row_off;  // rows per head in the buffers; whole-sequence row of local row 0
    int splits;                    // groups that share a position's heads
    const int* pos;                // [B][rows] natural positions, or null: from the layout
    const void *q, *k;             // inputs, element strides below
    long long qs[3], ks[3];        // batch, head, row
    const float *wq, *wk;
    const void *dyq, *dyk;         // backward: contiguous gradients of the outputs
    void *oq, *ok;                 // forward: outputs; backward: dq, dk (contiguous)
    float* partial;                // backward: [gridDim.x][2][d] sums of dw
    float eps;
    unsigned long long turn[64];   // theta_i / (2 pi) in units of 2^-64 turn
    long long axis_step;           // with axes: positions of one axis, B * rows
    float sign;                    // rotation alone: -1 turns back
    uint8_t axis[64];              // each pair's axis
};

// What a kernel is compiled for: the norm with the rotation by one position, by a position along each pair's axis, or
// that rotation alone.
enum class Kind { kNatural, kAxes, kAxesAlone };

template <typename T>
struct Pack;
template <>
struct Pack<__nv_bfloat16> {
    static constexpr int kElems = 8;
    static __device__ __forceinline__ void unpack(const uint4& v, float (&f)[8])
    {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ uint4 pack(const float (&f)[8])
    {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 p = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&p);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};
template <>
struct Pack<float> {
    static constexpr int kElems = 4;
    static __device__ __forceinline__ void unpack(const uint4& v, float (&f)[4])
    {
        f[0] = __uint_as_float(v.x);
        f[1] = __uint_as_float(v.y);
        f[2] = __uint_as_float(v.z);
        f[3] = __uint_as_float(v.w);
    }
    static __device__ __forceinline__ uint4 pack(const float (&f)[4])
    {
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    }
};

template <int LPR>
__device__ __forceinline__ unsigned group_mask()
{
    if (LPR == 32) return 0xffffffffu;
    return ((1u << (LPR & 31)) - 1u) << (threadIdx.x & 31 & ~(LPR - 1));
}

template <int LPR>
__device__ __forceinline__ float group_sum(float v, unsigned mask)
{
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(mask, v, o);
    return v;
}

// cos and sin of this lane's pairs at natural position p.
template <int PAIRS, Kind kKind>
__device__ __forceinline__ void angles(const NormRopeArgs& a, int ch, long long p, float (&c)[PAIRS], float (&s)[PAIRS])
{
    long long along[PAIRS];  // with axes p is the token's place in an axis's positions
#pragma unroll
    for (int j = 0; j < PAIRS; ++j) along[j] = kKind == Kind::kNatural ? p : a.pos[a.axis[ch * PAIRS + j] * a.axis_step + p];
#pragma unroll
    for (int j = 0; j < PAIRS; ++j) {
        const unsigned long long u = (unsigned long long)along[j] * a.turn[ch * PAIRS + j];
        // as a signed fraction, [-1/2, 1/2) turn: a small angle of either sign keeps a float32's precision
        sincospif(2.0f * ((float)(int)(unsigned)(u >> 32) * 2.3283064365386963e-10f), &s[j], &c[j]);  // 2^-32
        if (kKind == Kind::kAxesAlone) s[j] *= a.sign;
    }
}

// One group's position and heads.
struct Item {
    int b, r, h0, h1;
    long long p;
};

// kFew: the heads of a position are shared out, and all counts fit 32 bits (a 64-bit division is a hundred instructions:
// of 5.4 us that 128 tokens took 0.6).
template <bool kFew, Kind kKind>
__device__ __forceinline__ Item item_of(const NormRopeArgs& a, long long idx)
{
    Item it;
    if constexpr (kFew) {
        const unsigned i = (unsigned)idx, rows = (unsigned)a.rows, n = (unsigned)a.splits, heads = (unsigned)(a.H + a.Hkv);
        const unsigned rest = i / rows, b = rest / n, c = rest - b * n;
        it.r = (int)(i - rest * rows);
        it.b = (int)b;
        it.h0 = (int)(c * heads / n);
        it.h1 = (int)((c + 1) * heads / n);
    } else {
        it.r = (int)(idx % a.rows);
        it.b = (int)(idx / a.rows);
        it.h0 = 0;
        it.h1 = a.H + a.Hkv;
    }
    if constexpr (kKind != Kind::kNatural)
        it.p = (long long)it.b * a.rows + it.r;
    else
        it.p = a.pos ? a.pos[(long long)it.b * a.rows + it.r] : natural_position(a.geo, it.r + a.row_off);
    return it;
}

template <typename T, int D, int U, bool kNorm>
__device__ __forceinline__ void fwd_heads(const T* x, long long xs, T* y, long long ys, int count, const float* w,
                                          const float* c, const float* s, float eps, unsigned mask)
{
    constexpr int V = Pack<T>::kElems, LPR = D / V;
    for (int h = 0; h < count; h += U) {
        uint4 raw[U];
#pragma unroll
        for (int u = 0; u < U; ++u) raw[u] = *reinterpret_cast<const uint4*>(x + (h + u < count ? h + u : h) * xs);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (h + u >= count) break;
            float f[V];
            Pack<T>::unpack(raw[u], f);
            float r = 1.f;
            if constexpr (kNorm) {
                float ss = 0.f;
#pragma unroll
                for (int e = 0; e < V; ++e) ss = fmaf(f[e], f[e], ss);
                ss = group_sum<LPR>(ss, mask);
                r = rsqrtf(ss * (1.0f / D) + eps);
            }
#pragma unroll
            for (int j = 0; j < V / 2; ++j) {
                const float a0 = kNorm ? f[2 * j] * r * w[2 * j] : f[2 * j], a1 = kNorm ? f[2 * j + 1] * r * w[2 * j + 1] : f[2 * j + 1];
                f[2 * j] = a0 * c[j] - a1 * s[j];
                f[2 * j + 1] = a0 * s[j] + a1 * c[j];
            }
            *reinterpret_cast<uint4*>(y + (h + u) * ys) = Pack<T>::pack(f);
        }
    }
}

template <typename T, int D, bool kFew, Kind kKind>
__global__ void __launch_bounds__(kThreads, 4) norm_rope_kernel(const NormRopeArgs a)
{
    constexpr int V = Pack<T>::kElems, LPR = D / V, U = 4;
    constexpr bool kNorm = kKind != Kind::kAxesAlone;
    const int ch = threadIdx.x % LPR;
    const unsigned mask = group_mask<LPR>();
    const long long total = (long long)a.B * a.rows * a.splits;
    const long long step = (long long)gridDim.x * (kThreads / LPR);
    float wq[V], wk[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
        wq[e] = kNorm ? a.wq[ch * V + e] : 1.f;
        wk[e] = kNorm ? a.wk[ch * V + e] : 1.f;
    }
    for (long long idx = (long long)blockIdx.x * (kThreads / LPR) + threadIdx.x / LPR; idx < total; idx += step) {
        const Item it = item_of<kFew, kKind>(a, idx);
        float c[V / 2], s[V / 2];
        angles<V / 2, kKind>(a, ch, it.p, c, s);
        const long long ys = (long long)a.rows * D;
        const int q1 = it.h1 < a.H ? it.h1 : a.H, k0 = it.h0 > a.H ? it.h0 : a.H;
        if (it.h0 < q1)
            fwd_heads<T, D, U, kNorm>(static_cast<const T*>(a.q) + it.b * a.qs[0] + it.h0 * a.qs[1] + it.r * a.qs[2] + ch * V, a.qs[1],
                               static_cast<T*>(a.oq) + ((long long)it.b * a.H + it.h0) * ys + (long long)it.r * D + ch * V, ys,
                               q1 - it.h0, wq, c, s, a.eps, mask);
        if (k0 < it.h1)
            fwd_heads<T, D, U, kNorm>(static_cast<const T*>(a.k) + it.b * a.ks[0] + (k0 - a.H) * a.ks[1] + it.r * a.ks[2] + ch * V, a.ks[1],
                               static_cast<T*>(a.ok) + ((long long)it.b * a.Hkv + k0 - a.H) * ys + (long long)it.r * D + ch * V, ys,
                               it.h1 - k0, wk, c, s, a.eps, mask);
    }
}

template <typename T, int D, int U>
__device__ __forceinline__ void bwd_heads(const T* x, long long xs, const T* dy, T* dx, long long ys, int count, const float* w,
                                          float* dw, const float* c, const float* s, float eps, unsigned mask)
{
    constexpr int V = Pack<T>::kElems, LPR = D / V;
    for (int h = 0; h < count; h += U) {
        uint4 rx[U], rg[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int hh = h + u < count ? h + u : h;
            rx[u] = *reinterpret_cast<const uint4*>(x + hh * xs);
            rg[u] = *reinterpret_cast<const uint4*>(dy + hh * ys);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (h + u >= count) break;
            float f[V], g[V];
            Pack<T>::unpack(rx[u], f);
            Pack<T>::unpack(rg[u], g);
            float ss = 0.f, dot = 0.f, p[V];  // p = g w
#pragma unroll
            for (int j = 0; j < V / 2; ++j) {
                const float g0 = g[2 * j] * c[j] + g[2 * j + 1] * s[j], g1 = g[2 * j + 1] * c[j] - g[2 * j] * s[j];
                g[2 * j] = g0;
                g[2 * j + 1] = g1;
                p[2 * j] = g0 * w[2 * j];
                p[2 * j + 1] = g1 * w[2 * j + 1];
                ss = fmaf(f[2 * j], f[2 * j], ss);
                ss = fmaf(f[2 * j + 1], f[2 * j + 1], ss);
                dot = fmaf(p[2 * j], f[2 * j], dot);
                dot = fmaf(p[2 * j + 1], f[2 * j + 1], dot);
            }
#pragma unroll
            for (int o = LPR / 2; o > 0; o >>= 1) {
                ss += __shfl_xor_sync(mask, ss, o);
                dot += __shfl_xor_sync(mask, dot, o);
            }
            const float r = rsqrtf(ss * (1.0f / D) + eps);
            const float m = dot * r * (1.0f / D);  // mean(g w x r)
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float xh = f[e] * r;
                dw[e] = fmaf(g[e], xh, dw[e]);
                f[e] = r * fmaf(-xh, m, p[e]);
            }
            *reinterpret_cast<uint4*>(dx + (h + u) * ys) = Pack<T>::pack(f);
        }
    }
}

// dw is summed per lane over the rows it meets, then over the block's groups, in a fixed order;
// norm_rope_dw_kernel adds the blocks' sums in block order, so the result does not vary from run to run.
template <typename T, int D, bool kFew, Kind kKind>
__global__ void __launch_bounds__(kThreads, kNormRopeBwdPerSm) norm_rope_bwd_kernel(const NormRopeArgs a)
{
    constexpr int V = Pack<T>::kElems, LPR = D / V, U = 4, kGroups = kThreads / LPR;
    __shared__ float sums[kGroups][2 * D];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int ch = threadIdx.x % LPR, grp = threadIdx.x / LPR;
    const unsigned mask = group_mask<LPR>();
    const long long total = (long long)a.B * a.rows * a.splits;
    const long long step = (long long)gridDim.x * kGroups;
    float wq[V], wk[V], dq[V], dk[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
        wq[e] = a.wq[ch * V + e];
        wk[e] = a.wk[ch * V + e];
        dq[e] = dk[e] = 0.f;
    }
    for (long long idx = (long long)blockIdx.x * kGroups + grp; idx < total; idx += step) {
        const Item it = item_of<kFew, kKind>(a, idx);
        float c[V / 2], s[V / 2];
        angles<V / 2, kKind>(a, ch, it.p, c, s);
        const long long ys = (long long)a.rows * D;
        const int q1 = it.h1 < a.H ? it.h1 : a.H, k0 = it.h0 > a.H ? it.h0 : a.H;
        if (it.h0 < q1) {
            const long long o = ((long long)it.b * a.H + it.h0) * ys + (long long)it.r * D + ch * V;
            bwd_heads<T, D, U>(static_cast<const T*>(a.q) + it.b * a.qs[0] + it.h0 * a.qs[1] + it.r * a.qs[2] + ch * V, a.qs[1],
                               static_cast<const T*>(a.dyq) + o, static_cast<T*>(a.oq) + o, ys, q1 - it.h0, wq, dq, c, s,
                               a.eps, mask);
        }
        if (k0 < it.h1) {
            const long long o = ((long long)it.b * a.Hkv + k0 - a.H) * ys + (long long)it.r * D + ch * V;
            bwd_heads<T, D, U>(static_cast<const T*>(a.k) + it.b * a.ks[0] + (k0 - a.H) * a.ks[1] + it.r * a.ks[2] + ch * V, a.ks[1],
                               static_cast<const T*>(a.dyk) + o, static_cast<T*>(a.ok) + o, ys, it.h1 - k0, wk, dk, c, s,
                               a.eps, mask);
        }
    }
#pragma unroll
    for (int e = 0; e < V; ++e) {
        sums[grp][ch * V + e] = dq[e];
        sums[grp][D + ch * V + e] = dk[e];
    }
    __syncthreads();
    for (int col = threadIdx.x; col < 2 * D; col += kThreads) {
        float t = 0.f;
#pragma unroll
        for (int g = 0; g < kGroups; ++g) t += sums[g][col];
        a.partial[(long long)blockIdx.x * 2 * D + col] = t;
    }
}

__global__ void __launch_bounds__(1024) norm_rope_dw_kernel(const float* partial, int blocks, int d, float* dwq, float* dwk)
{
    __shared__ float part[32][33];
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const int col = blockIdx.x * 32 + tx;  // d is 64 or 128: 2 d columns in whole warps
    float t = 0.f;
    asm volatile("griddepcontrol.wait;" ::: "memory");  // for the partial sums
#pragma unroll 4
    for (int b = ty; b < blocks; b += 32) t += partial[(long long)b * 2 * d + col];
    part[ty][tx] = t;
    __syncthreads();
    if (ty == 0) {
        t = 0.f;
#pragma unroll
        for (int i = 0; i < 32; ++i) t += part[i][tx];
        if (col < d)
            dwq[col] = t;
        else
            dwk[col - d] = t;
    }
}

template <typename T, int D, Kind kKind>
cudaError_t launch_kind(NormRopeArgs& a, bool backward, float* dwq, float* dwk, cudaStream_t s)
{
    constexpr int LPR = D / Pack<T>::kElems, kGroups = kThreads / LPR;
    // Groups enough for 1024 threads on every SM, as long as a position has heads to share out.
    const long long tokens = (long long)a.B * a.rows;
    const long long want = (long long)device_sm_count() * 1024 / LPR;
    long long splits = (want + tokens - 1) / tokens;
    if (splits > a.H + a.Hkv) splits = a.H + a.Hkv;
    const long long heads = (long long)a.H + a.Hkv;
    const bool few = splits > 1 && heads * heads <= 0x7fffffffLL && tokens * splits <= 0x7fffffffLL;
    a.splits = few ? (int)splits : 1;
    long long grid = (tokens * a.splits + kGroups - 1) / kGroups;
    if (!backward) {  // a block per group of positions: the last ones fill the SMs evenly
        if (grid > 0x7fffffffLL) grid = 0x7fffffffLL;
        if (few)
            norm_rope_kernel<T, D, true, kKind><<<(unsigned)grid, kThreads, 0, s>>>(a);
        else
            norm_rope_kernel<T, D, false, kKind><<<(unsigned)grid, kThreads, 0, s>>>(a);
        return cudaGetLastError();
    }
    if constexpr (kKind == Kind::kAxesAlone) {
        return cudaErrorInvalidValue;  // (a rotation's gradient is a rotation)
    } else {
        // as many blocks as are resident, which take the positions in turns: their dw leave a partial sum each
        const long long most = (long long)device_sm_count() * kNormRopeBwdPerSm;
        if (grid > most) grid = most;
        if (grid > kNormRopeBwdBlocks) grid = kNormRopeBwdBlocks;
        if (few)
            norm_rope_bwd_kernel<T, D, true, kKind><<<(unsigned)grid, kThreads, 0, s>>>(a);
        else
            norm_rope_bwd_kernel<T, D, false, kKind><<<(unsigned)grid, kThreads, 0, s>>>(a);
        cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
        // starts while the first launch runs and waits for its results in the kernel
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(2 * D / 32);
        cfg.blockDim = dim3(1024);
        cfg.stream = s;
        cudaLaunchAttribute early;
        early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
        early.val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = &early;
        cfg.numAttrs = 1;
        return cudaLaunchKernelEx(&cfg, norm_rope_dw_kernel, static_cast<const float*>(a.partial), (int)grid, D, dwq, dwk);
    }
}

template <typename T, int D>
cudaError_t launch(NormRopeArgs& a, Kind kind, bool backward, float* dwq, float* dwk, cudaStream_t s)
{
    switch (kind) {
        case Kind::kAxes: return launch_kind<T, D, Kind::kAxes>(a, backward, dwq, dwk, s);
        case Kind::kAxesAlone: return launch_kind<T, D, Kind::kAxesAlone>(a, backward, dwq, dwk, s);
        default: return launch_kind<T, D, Kind::kNatural>(a, backward, dwq, dwk, s);
    }
}

}  // namespace

cudaError_t launch_norm_rope(const Problem& p, const NormRope& n, cudaStream_t s)
{
    NormRopeArgs a;
    a.geo = p.geo();
    a.B = p.B;
    a.H = p.H;
    a.Hkv = p.Hkv;
    a.rows = n.shard < 0 ? p.L : p.L / p.n;
    a.row_off = n.shard < 0 ? 0 : n.shard * (p.L / p.n);
    a.pos = n.positions;
    a.q = n.q;
    a.k = n.k;
    for (int i = 0; i < 3; ++i) {
        a.qs[i] = n.q_strides[i];
        a.ks[i] = n.k_strides[i];
    }
    a.wq = n.wq;
    a.wk = n.wk;
    a.dyq = n.dyq;
    a.dyk = n.dyk;
    a.oq = n.out_q;
    a.ok = n.out_k;
    a.partial = n.partial;
    a.eps = (float)n.eps;
    bool backward = n.dyq != nullptr;
    Kind kind = Kind::kNatural;
    a.axis_step = 0;
    a.sign = 1.f;
    memset(a.axis, 0, sizeof(a.axis));
    if (n.axes.count == 0) {
        rope_turns(n.base, p.d, a.turn);
    } else {
        rope_axes_turns(n.base, p.d, n.axes, a.turn);
        a.axis_step = (long long)p.B * a.rows;
        for (int x = 0, i = 0; x < n.axes.count; ++x)
            for (int u = 0; u < n.axes.sections[x]; ++u, ++i) a.axis[i] = (uint8_t)x;
        kind = n.wq ? Kind::kAxes : Kind::kAxesAlone;
    }
    if (kind == Kind::kAxesAlone && backward) {  // the gradients, turned back
        a.q = n.dyq;
        a.k = n.dyk;
        a.sign = -1.f;
        const long long row = p.d, head = (long long)a.rows * p.d;
        a.qs[0] = p.H * head, a.qs[1] = head, a.qs[2] = row;
        a.ks[0] = p.Hkv * head, a.ks[1] = head, a.ks[2] = row;
        backward = false;
    }
    if (p.dtype == 1)
        return p.d == 128 ? launch<__nv_bfloat16, 128>(a, kind, backward, n.dwq, n.dwk, s)
                          : launch<__nv_bfloat16, 64>(a, kind, backward, n.dwq, n.dwk, s);
    return p.d == 128 ? launch<float, 128>(a, kind, backward, n.dwq, n.dwk, s) : launch<float, 64>(a, kind, backward, n.dwq, n.dwk, s);
}

}  // namespace ra
