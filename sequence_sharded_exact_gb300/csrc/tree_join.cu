// tree_join.cu -- second launch of the attention over a cache (tree.cuh): joins the partials of the
// items that several CTAs share, and writes zeros and -infinity to the rows that see nothing.
//
// For the partials (m_c, l_c, o_c) of a row, M = max m_c:  out = sum 2^(m_c - M) o_c / sum 2^(m_c - M) l_c,
// lse = (M + log2 sum) ln 2, in CTA order.  One warp per query row; the lanes hold d / 32 elements.
// Bound by latency: the partials are a few hundred KB and still in L2.
#include <cuda_bf16.h>

#include "ra_internal.h"
#include "ra_ptx.cuh"
#include "tree.cuh"

namespace ra {
namespace {

constexpr int kRowsPerBlock = 4;  // one warp each

template <int D>
__global__ void __launch_bounds__(kRowsPerBlock * 32) tree_join_kernel(const TreeArgs a)
{
    constexpr int V = D / 32;
    const int lane = threadIdx.x & 31;
    const long long rows = (long long)a.B * a.Hkv * a.R;
    const long long x = (long long)blockIdx.x * kRowsPerBlock + (threadIdx.x >> 5);
    if (x >= rows) {
        asm volatile("griddepcontrol.wait;" ::: "memory");
        return;
    }
    const int row = (int)(x % a.R);
    const int g = (int)(x / a.R % a.Hkv), b = (int)(x / a.R / a.Hkv);
    const int r = row / a.rt, i = row % a.rt;
    const TreeSeq s = tree_seq(a, b);
    if (s.bad && g == 0 && row == 0 && lane == 0) atomicOr(a.status, kStatusRange);
    const int nt = tree_tiles(s);
    int c0 = 0, c1 = -1;
    long long total = 0, first = 0;
    if (nt && row % a.T < s.cnt) {
        long long before;
        tree_totals(a, b, total, before);
        first = before + ((long long)g * a.nrt + r) * nt;
        c0 = tree_owner(a, total, first);
        c1 = tree_owner(a, total, first + nt - 1);
    }
    // the partials are the first launch's; everything above needed the lengths alone
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (c0 == c1 && nt) return;  // written whole by that CTA
    float m = -INFINITY;
    for (int c = c0; c <= c1; ++c) {
        const int slot = c == c0 && tree_first(a, total, c) < first ? 1 : 0;
        m = fmaxf(m, a.part_ml[(((long long)c * 2 + slot) * a.rt + i) * 4]);
    }
    const float ref = m == -INFINITY ? 0.f : m;
    float l = 0.f, den = 0.f, o[V];
#pragma unroll
    for (int e = 0; e < V; ++e) o[e] = 0.f;
    for (int c = c0; c <= c1; ++c) {
        const int slot = c == c0 && tree_first(a, total, c) < first ? 1 : 0;
        const long long at = ((long long)c * 2 + slot) * a.rt + i;
        const float4 ml = *reinterpret_cast<const float4*>(a.part_ml + at * 4);
        const float w = ex2_approx(ml.x - ref);
        l = fmaf(ml.y, w, l);
        den = fmaf(ml.z, w, den);
#pragma unroll
        for (int e = 0; e < V; ++e) o[e] = fmaf(a.part_o[at * D + lane * V + e], w, o[e]);
    }
    const bool none = m == -INFINITY && l == 0.f;
    const float inv = none ? 0.f : 1.0f / den;
    const long long dst = (((long long)b * a.Hkv + g) * a.R + row) * D + lane * V;
    if (a.bf16_out) {
        __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + dst;
#pragma unroll
        for (int e = 0; e < V; e += 2) *reinterpret_cast<uint32_t*>(out + e) = pack_bf16x2(o[e] * inv, o[e + 1] * inv);
    } else {
        float* out = static_cast<float*>(a.out) + dst;
#pragma unroll
        for (int e = 0; e < V; ++e) out[e] = o[e] * inv;
    }
    if (lane == 0) a.lse[((long long)b * a.Hkv + g) * a.R + row] = none ? -INFINITY : (m + log2f(l)) * kLn2;
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
    cfg.gridDim = dim3((unsigned)((rows + kRowsPerBlock - 1) / kRowsPerBlock));
    cfg.blockDim = dim3(kRowsPerBlock * 32);
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
