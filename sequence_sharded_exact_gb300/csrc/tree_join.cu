// tree_join.cu -- second launch of the attention over a cache (tree.cuh): joins the partials of the
// items that several CTAs share, and writes zeros and -infinity to the rows of sequences without tokens.
//
// For the partials (m_c, l_c, den_c, o_c) of a row, c in CTA order, M = max m_c and w_c = 2^(m_c - M):
//   out = sum w_c o_c / sum w_c den_c,  lse = (M + log2 sum w_c l_c) ln 2.
// What bounds it is latency: a row has up to kTreeMaxCtas partials of d floats, all still in L2.  A unit is 32
// rows (a lane each: the partials are stored column by column) and 4 or 16 columns.  With few units a block's
// eight warps share one of 4 columns and take its partials in turn, eight each, 32 loads, at a time; each keeps a
// running maximum of its own, and they meet in shared memory in a fixed order.  With more units than blocks a
// unit has 16 columns and three partials are loaded at a time, by as few warps as keep all of them busy: four,
// two or one.  (One warp per row, walking its partials one by one: decoding over 19 partials took 15 us of 100;
// eight warps per unit whatever the number: 18.5 us in place of 13 for 64 items of 128 rows over 152 CTAs,
// 15.5 in place of 11.5 for 16 items of 256.)
#include <cuda_bf16.h>

#include "ra_internal.h"
#include "ra_ptx.cuh"
#include "tree.cuh"

namespace ra {
namespace {

constexpr int kWarps = 8, kMaxCols = 16;

// 32 rows from i0 and kCols columns from col0 of one item, U partials at a time, by `group` warps of which this is number `part`; every warp of
// the block calls this at the same time, those without a unit with has = false.
template <int D, int kCols, int U>
__device__ __forceinline__ void join_unit(const TreeArgs& a, bool has, int c0, const int4& item, int i0, int col0, int group, int part,
                                          float (&so)[kWarps][kMaxCols][33], float (&sm)[kWarps][3][32])
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, i = i0 + lane;
    const int b = item.x, g = item.y / a.nrt, r = item.y % a.nrt, c1 = item.z, head = item.w & 1, cnt = has ? item.w >> 1 : 0;
    auto lives = [&](int k) { return k < a.rt && r * a.rt + k < a.R && (r * a.rt + k) % a.T < cnt; };
    const bool live = lives(i);
    float m = -INFINITY, l = 0.f, den = 0.f, o[kCols];
#pragma unroll
    for (int e = 0; e < kCols; ++e) o[e] = 0.f;
    if (live) {
#pragma unroll 1
        for (int c = c0 + part; c <= c1; c += group * U) {
            float4 ml[U];
            float p[U][kCols];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int cc = c + u * group;
                if (cc > c1) break;
                const long long slot = (long long)cc * 2 + (cc == c0 ? head : 0);
                ml[u] = *reinterpret_cast<const float4*>(a.part_ml + (slot * a.rt + i) * 4);
#pragma unroll
                for (int e = 0; e < kCols; ++e) p[u][e] = a.part_o[(slot * D + col0 + e) * a.rt + i];
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (c + u * group > c1) break;
                const float mn = fmaxf(m, ml[u].x), ref = mn == -INFINITY ? 0.f : mn;
                const float keep = ex2_approx(m - ref), w = ex2_approx(ml[u].x - ref);
                m = mn;
                l = fmaf(ml[u].y, w, l * keep);
                den = fmaf(ml[u].z, w, den * keep);
                if (ml[u].x == -INFINITY && ml[u].y != 0.f) l = den = ml[u].y;  // NaN scores leave no maximum
#pragma unroll
                for (int e = 0; e < kCols; ++e) o[e] = fmaf(p[u][e], w, o[e] * keep);
            }
        }
    }
    sm[warp][0][lane] = m;
    sm[warp][1][lane] = l;
    sm[warp][2][lane] = den;
#pragma unroll
    for (int e = 0; e < kCols; ++e) so[warp][e][lane] = o[e];
    __syncthreads();
    // 32 rows of column pairs
    constexpr int kPairs = kCols / 2;
    const int w0 = warp - part;
#pragma unroll 1
    for (int t0 = part * 32 + lane; has && t0 < 32 * kPairs; t0 += group * 32) {
        const int k = t0 / kPairs, pair = t0 % kPairs;
        if (i0 + k >= a.rt || r * a.rt + i0 + k >= a.R) break;
        const bool dead = !lives(i0 + k);
        float2 t = make_float2(0.f, 0.f);
        m = -INFINITY;
        l = den = 0.f;
        if (!dead) {
            for (int w = w0; w < w0 + group; ++w) m = fmaxf(m, sm[w][0][k]);
            const float ref = m == -INFINITY ? 0.f : m;
            for (int w = w0; w < w0 + group; ++w) {
                const float f = ex2_approx(sm[w][0][k] - ref);
                l = fmaf(sm[w][1][k], f, l);
                den = fmaf(sm[w][2][k], f, den);
                t.x = fmaf(so[w][2 * pair][k], f, t.x);
                t.y = fmaf(so[w][2 * pair + 1][k], f, t.y);
            }
        }
        const bool none = m == -INFINITY && l == 0.f;
        const float inv = 1.0f / den;
        t = none ? make_float2(0.f, 0.f) : make_float2(t.x * inv, t.y * inv);
        const long long x = ((long long)b * a.Hkv + g) * a.R + (long long)r * a.rt + i0 + k;
        const long long dst = (x * D + col0) / 2 + pair;
        if (a.bf16_out)
            static_cast<uint32_t*>(a.out)[dst] = pack_bf16x2(t.x, t.y);
        else
            static_cast<float2*>(a.out)[dst] = t;
        if (pair == 0 && col0 == 0) a.lse[x] = none ? -INFINITY : (m + log2f(l)) * kLn2;
    }
}

template <int D, int kCols, int U>
__device__ __forceinline__ void join_units(const TreeArgs& a, int n, int chunks, const int4* items, const short* list, float (&so)[kWarps][kMaxCols][33],
                                           float (&sm)[kWarps][3][32])
{
    const int warp = threadIdx.x >> 5, units = n * chunks * (D / kCols);
    int group = kWarps;
    while (group > 1 && units > (int)gridDim.x * (kWarps / group)) group >>= 1;
    for (int u0 = blockIdx.x; u0 < units; u0 += gridDim.x * (kWarps / group)) {
        const int u = u0 + warp / group * (int)gridDim.x;
        const bool has = u < units;
        const int c0 = has ? list[u / (chunks * (D / kCols))] : 0;
        const int4 item = has ? items[u / (chunks * (D / kCols))] : make_int4(0, 0, 0, 0);
        join_unit<D, kCols, U>(a, has, c0, item, u / (D / kCols) % chunks * 32, u % (D / kCols) * kCols, group, warp % group, so, sm);
        __syncthreads();
    }
}

template <int D>
__global__ void __launch_bounds__(kWarps * 32, 2) tree_join_kernel(const TreeArgs a)
{
    __shared__ float so[kWarps][kMaxCols][33];
    __shared__ float sm[kWarps][3][32];
    __shared__ int4 items[kTreeMaxCtas];
    __shared__ short list[kTreeMaxCtas];
    __shared__ int count[kWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int chunks = (tree_item_rows(a) + 31) / 32;
    // sequences without tokens, and lengths outside their ranges: a turn for every block (nothing here depends on the
    // first launch, which leaves their rows alone)
    for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
        const TreeSeq s = tree_seq(a, b);
        if (s.bad && threadIdx.x == 0) atomicOr(a.status, kStatusRange);
        if (s.end) continue;
        const long long rows = (long long)a.Hkv * a.R, row0 = b * rows;
        for (long long e = threadIdx.x; e < rows * D / 2; e += blockDim.x) {
            if (a.bf16_out)
                static_cast<uint32_t*>(a.out)[row0 * D / 2 + e] = 0u;
            else
                static_cast<float2*>(a.out)[row0 * D / 2 + e] = make_float2(0.f, 0.f);
        }
        for (long long e = threadIdx.x; e < rows; e += blockDim.x) a.lse[row0 + e] = -INFINITY;
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");  // for the first launch's results
    // the borders that an item goes over, in order
    constexpr int kRounds = (kTreeMaxCtas + kWarps * 32 - 1) / (kWarps * 32);
    int4 mine[kRounds];
#pragma unroll
    for (int k = 0; k < kRounds; ++k) {
        const int c = k * kWarps * 32 + (int)threadIdx.x;
        mine[k] = c < a.ctas ? a.border[c] : make_int4(-1, 0, 0, 0);
    }
    int n = 0;
#pragma unroll
    for (int k = 0; k < kRounds; ++k) {
        if (k * kWarps * 32 >= a.ctas) break;
        const unsigned votes = __ballot_sync(0xffffffffu, mine[k].x >= 0);
        if (lane == 0) count[warp] = __popc(votes);
        __syncthreads();
        int before = n;
        for (int j = 0; j < kWarps; ++j) {
            if (j < warp) before += count[j];
            n += count[j];
        }
        if (mine[k].x >= 0) {
            const int at = before + __popc(votes & ((1u << lane) - 1u));
            items[at] = mine[k];
            list[at] = (short)(k * kWarps * 32 + (int)threadIdx.x);
        }
        __syncthreads();
    }
    if (n * chunks * (D / 4) <= (int)gridDim.x)
        join_units<D, 4, 8>(a, n, chunks, items, list, so, sm);
    else
        join_units<D, 16, 3>(a, n, chunks, items, list, so, sm);
}

}  // namespace

// How a problem is cut: its path, query rows per row tile, and the most CTAs of the first launch, known without a
// device (the workspace is sized by it).
enum class Path { kSimt, kMma, kTc };

struct Cut {
    Path path;
    int tile, rt, nrt, ctas;
};

static Cut cut_of(const Cache& c, int H, int T, int dtype)
{
    Cut u;
    const int R = H / c.Hkv * T;
    u.path = dtype != 1 ? Path::kSimt : R <= (c.dtype == kCacheE4m3 ? kTreeMmaE4m3Rows : kTreeMmaRows) ? Path::kMma : Path::kTc;
    u.tile = u.path == Path::kSimt ? kTreeSimtTile : kTreeTile;
    u.rt = u.path == Path::kSimt ? tree_simt_rows(R) : u.path == Path::kMma ? (R <= kTreeMmaRows ? kTreeMmaRows : kTreeMmaE4m3Rows) : R <= 128 ? 128 : 256;
    u.nrt = (R + u.rt - 1) / u.rt;
    const long long most = (long long)c.B * c.Hkv * u.nrt * ((c.cap + u.tile - 1) / u.tile);
    const int cap = u.path == Path::kSimt ? kTreeMaxCtas : u.path == Path::kMma ? kTreeMaxMmaCtas : kTreeMaxTcCtas;
    u.ctas = (int)(most < cap ? most : cap);
    return u;
}

static size_t border_bytes(const Cut& u) { return tree_align((size_t)u.ctas * sizeof(int4)); }
static size_t ml_bytes(const Cut& u) { return tree_align((size_t)u.ctas * 2 * u.rt * 4 * sizeof(float)); }

size_t tree_workspace_size(const Cache& c, int H, int T, int dtype)
{
    const Cut u = cut_of(c, H, T, dtype);
    return border_bytes(u) + ml_bytes(u) + tree_align((size_t)u.ctas * 2 * u.rt * c.d * sizeof(float));
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
    a.tile = u.tile;
    a.rt = u.rt;
    a.nrt = u.nrt;
    const int sms = device_sm_count();
    const bool e4m3 = c.dtype == kCacheE4m3, many = (long long)c.B * c.Hkv >= (long long)kTreeMmaManyItems * sms;
    const int resident = sms * (u.path == Path::kSimt ? kTreeSimtCtasPerSm : u.path == Path::kTc ? 1 : u.rt == kTreeMmaE4m3Rows ? tree_mma16_ctas_per_sm(c.d) : e4m3 ? (many ? 4 : 2) : many ? 3 : 2);
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
    char* ws = static_cast<char*>(t.workspace);
    a.border = reinterpret_cast<int4*>(ws);
    a.part_ml = reinterpret_cast<float*>(ws + border_bytes(u));
    a.part_o = reinterpret_cast<float*>(ws + border_bytes(u) + ml_bytes(u));
    cudaError_t e;
    if (u.path == Path::kMma)
        e = e4m3 ? launch_tree_mma(a, c.d, many ? 4 : 8, s) : launch_tree_mma_bf16(a, c.d, s);
    else if (u.path == Path::kTc)
        e = c.d == 128 ? launch_tree_tc_d128(a, e4m3, s) : launch_tree_tc_d64(a, e4m3, s);
    else
        e = launch_tree_simt(a, c.d, c.dtype, s);
    return e != cudaSuccess ? e : launch_tree_join(a, c.d, s);
}

cudaError_t launch_tree_join(const TreeArgs& a, int d, cudaStream_t s)
{
    const long long most = (long long)(a.ctas > 1 ? a.ctas - 1 : 1) * ((tree_item_rows(a) + 31) / 32) * (d / 4);
    const long long resident = (long long)device_sm_count() * 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(most < resident ? most : resident));
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
