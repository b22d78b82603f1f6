// tree_join.cu -- second launch of the attention over a cache (tree.cuh): joins the partials of the
// items that several CTAs share, and writes zeros and -infinity to the rows that see nothing.
//
// For the partials (m_c, l_c, den_c, o_c) of a row, c in CTA order, M = max m_c and w_c = 2^(m_c - M):
//   out = sum w_c o_c / sum w_c den_c,  lse = (M + log2 sum w_c l_c) ln 2.
// What bounds it is latency: a row has up to kTreeMaxCtas partials of d floats, all still in L2, and few rows
// leave few blocks.  A block has one row, its four warps every fourth partial, a lane d / 32 columns, and
// each warp loads eight partials before it needs the first; the warps' sums meet in a fixed order.
// (One warp per row, walking its partials one by one: decoding over 19 partials took 15 us of 100.)
#include <cuda_bf16.h>

#include "ra_internal.h"
#include "ra_ptx.cuh"
#include "tree.cuh"

namespace ra {
namespace {

constexpr int kWarps = 4;

template <int V>
struct Cols {
    float f[V];
};
__device__ __forceinline__ Cols<4> load_cols(const float* p, Cols<4>)
{
    const float4 v = *reinterpret_cast<const float4*>(p);
    return {{v.x, v.y, v.z, v.w}};
}
__device__ __forceinline__ Cols<2> load_cols(const float* p, Cols<2>)
{
    const float2 v = *reinterpret_cast<const float2*>(p);
    return {{v.x, v.y}};
}

template <int D>
__global__ void __launch_bounds__(kWarps * 32) tree_join_kernel(const TreeArgs a)
{
    constexpr int V = D / 32;
    __shared__ float sums[kWarps][D + 2];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long x = blockIdx.x;  // query row: sequence, kv head, row of the head's group
    const int row = (int)(x % a.R);
    const int g = (int)(x / a.R % a.Hkv), b = (int)(x / a.R / a.Hkv);
    const int r = row / a.rt, i = row % a.rt;
    const TreeSeq s = tree_seq(a, b);
    const int nt = tree_tiles(s);
    int c0 = 0, c1 = -1, head = 0;
    if (nt && row % a.T < s.cnt) {
        long long total, before;
        tree_totals(a, b, total, before);
        const long long first = before + ((long long)g * a.nrt + r) * nt;
        c0 = tree_owner(a, total, first);
        c1 = tree_owner(a, total, first + nt - 1);
        head = tree_first(a, total, c0) < first ? 1 : 0;  // c0 comes to this item after another one
    }
    // the partials are the first launch's; everything above needed the lengths alone
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (s.bad && g == 0 && row == 0 && threadIdx.x == 0) atomicOr(a.status, kStatusRange);
    if (c0 == c1 && nt) return;  // written whole by that CTA
    auto at = [&](int c) { return ((long long)c * 2 + (c == c0 ? head : 0)) * a.rt + i; };
    float m = -INFINITY;
    for (int c = c0 + lane; c <= c1; c += 32) m = fmaxf(m, a.part_ml[at(c) * 4]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float ref = m == -INFINITY ? 0.f : m;
    float l = 0.f, den = 0.f, o[V];
#pragma unroll
    for (int e = 0; e < V; ++e) o[e] = 0.f;
    constexpr int U = 8;
    for (int c = c0 + warp; c <= c1; c += kWarps * U) {
        float4 ml[U];
        Cols<V> p[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const long long k = at(c + u * kWarps <= c1 ? c + u * kWarps : c);
            ml[u] = *reinterpret_cast<const float4*>(a.part_ml + k * 4);
            p[u] = load_cols(a.part_o + k * D + lane * V, Cols<V>());
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (c + u * kWarps > c1) break;
            const float w = ex2_approx(ml[u].x - ref);
            l = fmaf(ml[u].y, w, l);
            den = fmaf(ml[u].z, w, den);
#pragma unroll
            for (int e = 0; e < V; ++e) o[e] = fmaf(p[u].f[e], w, o[e]);
        }
    }
#pragma unroll
    for (int e = 0; e < V; ++e) sums[warp][lane * V + e] = o[e];
    if (lane == 0) {
        sums[warp][D] = l;
        sums[warp][D + 1] = den;
    }
    __syncthreads();
    l = den = 0.f;
#pragma unroll
    for (int k = 0; k < kWarps; ++k) {
        l += sums[k][D];
        den += sums[k][D + 1];
    }
    const bool none = m == -INFINITY && l == 0.f;
    const float inv = none ? 0.f : 1.0f / den;
    if (threadIdx.x < D / 2) {  // two columns each
        float2 t = make_float2(0.f, 0.f);
#pragma unroll
        for (int k = 0; k < kWarps; ++k) {
            t.x += sums[k][threadIdx.x * 2];
            t.y += sums[k][threadIdx.x * 2 + 1];
        }
        if (a.bf16_out)
            static_cast<uint32_t*>(a.out)[(x * D >> 1) + threadIdx.x] = none ? 0u : pack_bf16x2(t.x * inv, t.y * inv);
        else
            static_cast<float2*>(a.out)[(x * D >> 1) + threadIdx.x] = none ? make_float2(0.f, 0.f) : make_float2(t.x * inv, t.y * inv);
    }
    if (threadIdx.x == 0) a.lse[x] = none ? -INFINITY : (m + log2f(l)) * kLn2;
}

}  // namespace

// How a problem is cut: its path, query rows per row tile, and the most CTAs of the first launch, known without a
// device (the workspace is sized by it).
struct Cut {
    bool tc;
    int rt, nrt, ctas;
};

static Cut cut_of(const Cache& c, int H, int T, int dtype)
{
    Cut u;
    const int R = H / c.Hkv * T;
    u.tc = dtype == 1;
    u.rt = u.tc ? (R <= 128 ? 128 : 256) : tree_simt_rows(R);
    u.nrt = (R + u.rt - 1) / u.rt;
    const long long most = (long long)c.B * c.Hkv * u.nrt * ((c.cap + kTreeTile - 1) / kTreeTile);
    const int cap = u.tc ? kTreeMaxTcCtas : kTreeMaxCtas;
    u.ctas = (int)(most < cap ? most : cap);
    return u;
}

static size_t ml_bytes(const Cut& u) { return tree_align((size_t)u.ctas * 2 * u.rt * 4 * sizeof(float)); }

size_t tree_workspace_size(const Cache& c, int H, int T, int dtype)
{
    const Cut u = cut_of(c, H, T, dtype);
    return ml_bytes(u) + tree_align((size_t)u.ctas * 2 * u.rt * c.d * sizeof(float));
}

cudaError_t launch_tree(const Cache& c, const Tree& t, cudaStream_t s)
{
    const Cut u = cut_of(c, t.H, t.T, t.dtype);
    TreeArgs a;
    a.B = c.B;
    a.H = t.H;
    a.Hkv = c.Hkv;
    a.G = t.H / c.Hkv;
    a.T = t.T;
    a.R = a.G * t.T;
    a.cap = c.cap;
    a.rt = u.rt;
    a.nrt = u.nrt;
    const int resident = device_sm_count() * (u.tc ? 1 : kTreeSimtCtasPerSm);
    a.ctas = u.ctas < resident ? u.ctas : resident;
    a.mask_batched = t.mask_batched;
    a.bf16_out = t.out_dtype == 1;
    a.lens = t.lens;
    a.ntok = t.ntok;
    a.mask = t.mask;
    a.q = t.q;
    a.k = c.k;
    a.v = c.v;
    a.k_exp = c.k_exp;
    a.v_exp = c.v_exp;
    a.out = t.out;
    a.lse = t.lse;
    a.status = t.status;
    a.scale_log2 = kLog2e / sqrtf((float)c.d);
    a.part_ml = static_cast<float*>(t.workspace);
    a.part_o = reinterpret_cast<float*>(static_cast<char*>(t.workspace) + ml_bytes(u));
    cudaError_t e;
    if (u.tc)
        e = c.d == 128 ? launch_tree_tc_d128(a, c.dtype == kCacheE4m3, s) : launch_tree_tc_d64(a, c.dtype == kCacheE4m3, s);
    else
        e = launch_tree_simt(a, c.d, c.dtype, s);
    return e != cudaSuccess ? e : launch_tree_join(a, c.d, s);
}

cudaError_t launch_tree_join(const TreeArgs& a, int d, cudaStream_t s)
{
    const long long rows = (long long)a.B * a.Hkv * a.R;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)rows);
    cfg.blockDim = dim3(kWarps * 32);
    cfg.stream = s;
    // starts while the first launch runs; it waits for that one's results in the kernel
    cudaLaunchAttribute early;
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &early;
    cfg.numAttrs = 1;
    return d == 128 ? cudaLaunchKernelEx(&cfg, tree_join_kernel<128>, a) : cudaLaunchKernelEx(&cfg, tree_join_kernel<64>, a);
}

}  // namespace ra
