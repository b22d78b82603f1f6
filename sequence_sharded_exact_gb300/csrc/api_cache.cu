// api_cache.cu -- the C ABI of the operators around a key/value cache (declared in include/ringattn.h):
// norms and rotation of queries and keys, the cache's writes and reads, and the attention over it.
#include <math.h>

#include "../../include/ringattn.h"
#include "ra_internal.h"

static_assert(ra::kStatusRange == RA_DEVICE_RANGE && ra::kCacheE4m3 == RA_E4M3, "codes agree with the ABI");

namespace ra {
namespace {

int elem_bytes(int dtype) { return dtype == RA_F32 ? 4 : (dtype == RA_BF16 ? 2 : 1); }

// Element strides (batch, head, row) of an input: the caller's, or a contiguous [B][heads][rows][d]'s.
// A stride that moves the pointer has to keep rows on 16-byte boundaries; one of an axis of length 1 is
// never used.
ra_status take_strides(const char* name, const long long* given, int B, int heads, long long rows, int d, int dtype, long long out[3])
{
    const long long own[3] = {heads * rows * d, rows * d, d};
    const long long len[3] = {B, heads, rows};
    const int per = 16 / elem_bytes(dtype);
    for (int i = 0; i < 3; ++i) {
        out[i] = given ? given[i] : own[i];
        if (len[i] == 1) {
            out[i] = 0;
            continue;
        }
        if (out[i] < 0 || out[i] % per != 0)
            return fail(RA_ERR_INVALID_ARG, "%s stride %lld is negative or not a multiple of 16 bytes", name, out[i]);
        if (out[i] >= (1LL << 40)) return fail(RA_ERR_UNSUPPORTED, "%s stride %lld is too large", name, out[i]);
    }
    return RA_OK;
}

// int32 arrays of the caller: slices of larger ones are common, so 4-byte alignment is enough.
ra_status check_ints(const char* name, const int* p, bool optional)
{
    if (!p) return optional ? RA_OK : fail(RA_ERR_INVALID_ARG, "%s is NULL", name);
    if (reinterpret_cast<uintptr_t>(p) & 3u) return fail(RA_ERR_INVALID_ARG, "%s is not 4-byte aligned", name);
    return RA_OK;
}

ra_status check_workspace(const void* ws, size_t have, size_t need)
{
    ra_status st = check_ptrs({ws});
    if (st != RA_OK) return st;
    if (reinterpret_cast<uintptr_t>(ws) & 255u) return fail(RA_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
    if (have < need) return fail(RA_ERR_INVALID_ARG, "workspace too small: %zu < %zu bytes", have, need);
    return RA_OK;
}

ra_status norm_rope_impl(Problem p, NormRope n, const long long* qs, const long long* ks, bool backward, size_t workspace_bytes,
                         void* workspace, void* stream)
{
    ra_status st = check_problem(p);
    if (st != RA_OK) return st;
    if ((long long)p.H + p.Hkv >= (1LL << 30)) return fail(RA_ERR_UNSUPPORTED, "too many heads");
    if (n.shard < -1 || n.shard >= p.n) return fail(RA_ERR_INVALID_ARG, "shard %d outside [-1, n_shards)", n.shard);
    if (!(n.base > 0.0) || !isfinite(n.base)) return fail(RA_ERR_INVALID_ARG, "base must be positive and finite");
    if (!(n.eps >= 0.0) || !isfinite(n.eps)) return fail(RA_ERR_INVALID_ARG, "eps must be >= 0 and finite");
    const bool axes = n.axes.count > 0, alone = axes && !n.wq && !n.wk;  // the rotation alone
    if ((st = check_ptrs({n.out_q, n.out_k})) != RA_OK) return st;
    if (!alone && (st = check_ptrs({n.wq, n.wk})) != RA_OK) return st;
    if (!(alone && backward) && (st = check_ptrs({n.q, n.k})) != RA_OK) return st;
    if ((st = check_ints("positions", n.positions, !axes)) != RA_OK) return st;
    const long long rows = n.shard < 0 ? p.L : p.L / p.n;
    if ((st = take_strides("q", qs, p.B, p.H, rows, p.d, p.dtype, n.q_strides)) != RA_OK) return st;
    if ((st = take_strides("k", ks, p.B, p.Hkv, rows, p.d, p.dtype, n.k_strides)) != RA_OK) return st;
    if (backward && (st = check_ptrs({n.dyq, n.dyk})) != RA_OK) return st;
    if (backward && !alone) {
        if ((st = check_ptrs({n.dwq, n.dwk})) != RA_OK) return st;
        if ((st = check_workspace(workspace, workspace_bytes, ring_attn_qk_norm_rope_bwd_workspace_size(p.d))) != RA_OK) return st;
        n.partial = static_cast<float*>(workspace);
    }
    if ((st = check_device()) != RA_OK) return st;
    cudaError_t e = launch_norm_rope(p, n, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, axes ? (backward ? "ring_attn_qk_rope_axes_bwd launch" : "ring_attn_qk_rope_axes launch")
                                               : backward ? "ring_attn_qk_norm_rope_bwd launch" : "ring_attn_qk_norm_rope launch");
    return RA_OK;
}

ra_status take_axes(int d, int axes, const int* sections, int spectrum, RopeAxes& out)
{
    if (axes < 1 || axes > kMaxAxes) return fail(RA_ERR_INVALID_ARG, "axes must lie in [1, %d] (got %d)", kMaxAxes, axes);
    if (!sections) return fail(RA_ERR_INVALID_ARG, "sections is NULL");
    if (spectrum != RA_SPECTRUM_WHOLE && spectrum != RA_SPECTRUM_AXIS) return fail(RA_ERR_INVALID_ARG, "unknown spectrum %d", spectrum);
    out = RopeAxes{};
    out.count = axes;
    out.own_spectrum = spectrum == RA_SPECTRUM_AXIS;
    long long sum = 0;
    for (int i = 0; i < axes; ++i) {
        if (sections[i] < 0) return fail(RA_ERR_INVALID_ARG, "section %d is negative", i);
        out.sections[i] = sections[i];
        sum += sections[i];
    }
    if (sum != d / 2) return fail(RA_ERR_INVALID_ARG, "the sections must have d / 2 = %d pairs in all (got %lld)", d / 2, sum);
    return RA_OK;
}

ra_status check_cache(const Cache& c, int dtype)
{
    if (c.B < 1 || c.Hkv < 1 || c.cap < 1)
        return fail(RA_ERR_INVALID_ARG, "B, Hkv, cap must be >= 1 (got %d %d %d)", c.B, c.Hkv, c.cap);
    if (dtype != RA_F32 && dtype != RA_BF16) return fail(RA_ERR_INVALID_ARG, "unknown dtype %d", dtype);
    if (c.dtype != dtype && c.dtype != RA_E4M3)
        return fail(RA_ERR_INVALID_ARG, "cache dtype %d is neither the tensors' dtype %d nor RA_E4M3", c.dtype, dtype);
    if (c.d != 64 && c.d != 128) return fail(RA_ERR_UNSUPPORTED, "head dim %d not supported (64 or 128)", c.d);
    if ((long long)c.B * c.Hkv >= (1LL << 30) || c.cap >= (1 << 30) || (long long)c.B * c.Hkv * c.cap >= (1LL << 40) / c.d)
        return fail(RA_ERR_UNSUPPORTED, "cache too large");
    ra_status st = check_ptrs({c.k, c.v});
    if (st != RA_OK) return st;
    if (c.dtype == RA_E4M3 && (!c.k_exp || !c.v_exp)) return fail(RA_ERR_INVALID_ARG, "an e4m3 cache needs k_exp and v_exp");
    return RA_OK;
}

Cache cache_of(const void* k, const void* v, const void* ke, const void* ve, int B, int Hkv, int cap, int d, int dtype)
{
    return Cache{B, Hkv, cap, d, dtype, const_cast<void*>(k), const_cast<void*>(v),
                 static_cast<uint8_t*>(const_cast<void*>(ke)), static_cast<uint8_t*>(const_cast<void*>(ve))};
}

ra_status check_tree(const Cache& c, int H, int T)
{
    if (H < 1 || T < 1) return fail(RA_ERR_INVALID_ARG, "H, T must be >= 1 (got %d %d)", H, T);
    if (H % c.Hkv != 0) return fail(RA_ERR_INVALID_ARG, "H (%d) must be a multiple of Hkv (%d)", H, c.Hkv);
    if ((long long)H * T >= (1LL << 30) || (long long)c.B * H * T >= (1LL << 31))
        return fail(RA_ERR_UNSUPPORTED, "too many query rows");
    return RA_OK;
}

ra_status tree_impl(const Cache& c, Tree t, size_t workspace_bytes, void* stream, const char* what)
{
    ra_status st = check_cache(c, t.dtype);
    if (st != RA_OK) return st;
    if ((st = check_tree(c, t.H, t.T)) != RA_OK) return st;
    if (t.out_dtype != t.dtype && t.out_dtype != RA_F32) return fail(RA_ERR_INVALID_ARG, "out_dtype must be the dtype of q or RA_F32");
    if ((st = check_ptrs({t.q, t.out, t.lse})) != RA_OK) return st;
    if ((st = check_ints("lens", t.lens, false)) != RA_OK || (st = check_ints("ntok", t.ntok, true)) != RA_OK) return st;
    if ((st = check_workspace(t.workspace, workspace_bytes,
                              ring_attn_tree_fwd_workspace_size(c.B, t.H, c.Hkv, t.T, c.d, c.cap, t.dtype, c.dtype))) != RA_OK)
        return st;
    if ((st = check_device()) != RA_OK) return st;
    cudaError_t e;
    t.status = status_word(&e);
    if (!t.status) return cuda_fail(e, "status word");
    e = launch_tree(c, t, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, what);
    return RA_OK;
}

}  // namespace
}  // namespace ra

using namespace ra;

extern "C" {

ra_status ring_attn_qk_norm_rope(const void* q, const long long* q_strides, const void* k, const long long* k_strides,
                                 const float* wq, const float* wk, void* q_out, void* k_out, int B, int H, int Hkv, int L, int d,
                                 int n_shards, int shard, int layout, int dtype, double base, double eps, const int* positions,
                                 void* stream)
{
    NormRope n = {};
    n.q = q;
    n.k = k;
    n.wq = wq;
    n.wk = wk;
    n.out_q = q_out;
    n.out_k = k_out;
    n.positions = positions;
    n.shard = shard;
    n.base = base;
    n.eps = eps;
    return norm_rope_impl(Problem{B, H, Hkv, L, d, n_shards, 1, layout, dtype}, n, q_strides, k_strides, false, 0, nullptr, stream);
}

size_t ring_attn_qk_norm_rope_bwd_workspace_size(int d)
{
    return d < 1 ? 0 : ((size_t)kNormRopeBwdBlocks * 2 * d * sizeof(float) + 255) & ~size_t(255);
}

ra_status ring_attn_qk_norm_rope_bwd(const void* q, const long long* q_strides, const void* k, const long long* k_strides,
                                     const float* wq, const float* wk, const void* dq_out, const void* dk_out, void* dq, void* dk,
                                     float* dwq, float* dwk, void* workspace, size_t workspace_bytes, int B, int H, int Hkv, int L,
                                     int d, int n_shards, int shard, int layout, int dtype, double base, double eps,
                                     const int* positions, void* stream)
{
    NormRope n = {};
    n.q = q;
    n.k = k;
    n.wq = wq;
    n.wk = wk;
    n.dyq = dq_out;
    n.dyk = dk_out;
    n.out_q = dq;
    n.out_k = dk;
    n.dwq = dwq;
    n.dwk = dwk;
    n.positions = positions;
    n.shard = shard;
    n.base = base;
    n.eps = eps;
    return norm_rope_impl(Problem{B, H, Hkv, L, d, n_shards, 1, layout, dtype}, n, q_strides, k_strides, true, workspace_bytes,
                          workspace, stream);
}

ra_status ring_attn_qk_rope_axes(const void* q, const long long* q_strides, const void* k, const long long* k_strides,
                                 const float* wq, const float* wk, void* q_out, void* k_out, int B, int H, int Hkv, int rows, int d,
                                 int axes, const int* sections, int spectrum, int dtype, double base, double eps,
                                 const int* positions, void* stream)
{
    NormRope n = {};
    n.q = q;
    n.k = k;
    n.wq = wq;
    n.wk = wk;
    n.out_q = q_out;
    n.out_k = k_out;
    n.positions = positions;
    n.shard = -1;
    n.base = base;
    n.eps = eps;
    const ra_status st = take_axes(d, axes, sections, spectrum, n.axes);
    if (st != RA_OK) return st;
    return norm_rope_impl(Problem{B, H, Hkv, rows, d, 1, 1, RA_LAYOUT_CONTIGUOUS, dtype}, n, q_strides, k_strides, false, 0, nullptr, stream);
}

ra_status ring_attn_qk_rope_axes_bwd(const void* q, const long long* q_strides, const void* k, const long long* k_strides,
                                     const float* wq, const float* wk, const void* dq_out, const void* dk_out, void* dq, void* dk,
                                     float* dwq, float* dwk, void* workspace, size_t workspace_bytes, int B, int H, int Hkv, int rows,
                                     int d, int axes, const int* sections, int spectrum, int dtype, double base, double eps,
                                     const int* positions, void* stream)
{
    NormRope n = {};
    n.q = q;
    n.k = k;
    n.wq = wq;
    n.wk = wk;
    n.dyq = dq_out;
    n.dyk = dk_out;
    n.out_q = dq;
    n.out_k = dk;
    n.dwq = dwq;
    n.dwk = dwk;
    n.positions = positions;
    n.shard = -1;
    n.base = base;
    n.eps = eps;
    ra_status st = take_axes(d, axes, sections, spectrum, n.axes);
    if (st != RA_OK) return st;
    if (!dq_out) return fail(RA_ERR_INVALID_ARG, "dq_out is NULL");  // (what tells the backward from the forward)
    return norm_rope_impl(Problem{B, H, Hkv, rows, d, 1, 1, RA_LAYOUT_CONTIGUOUS, dtype}, n, q_strides, k_strides, true, workspace_bytes,
                          workspace, stream);
}

ra_status ring_attn_cache_write(const void* k, const long long* k_strides, const void* v, const long long* v_strides,
                                void* k_cache, void* v_cache, void* k_exp, void* v_exp, const int* lens, const int* ntok, int B,
                                int Hkv, int T, int d, int cap, int dtype, int cache_dtype, void* stream)
{
    const Cache c = cache_of(k_cache, v_cache, k_exp, v_exp, B, Hkv, cap, d, cache_dtype);
    ra_status st = check_cache(c, dtype);
    if (st != RA_OK) return st;
    if (T < 1) return fail(RA_ERR_INVALID_ARG, "T must be >= 1 (got %d)", T);
    if (T >= (1 << 30) || (long long)B * Hkv * T >= (1LL << 40) / d) return fail(RA_ERR_UNSUPPORTED, "too many rows");
    if (!lens && T > cap) return fail(RA_ERR_INVALID_ARG, "T (%d) rows from row 0 do not fit the cache (%d rows)", T, cap);
    if ((st = check_ptrs({k, v})) != RA_OK) return st;
    if ((st = check_ints("lens", lens, true)) != RA_OK || (st = check_ints("ntok", ntok, true)) != RA_OK) return st;
    long long ks[3], vs[3];
    if ((st = take_strides("k", k_strides, B, Hkv, T, d, dtype, ks)) != RA_OK) return st;
    if ((st = take_strides("v", v_strides, B, Hkv, T, d, dtype, vs)) != RA_OK) return st;
    if ((st = check_device()) != RA_OK) return st;
    cudaError_t e;
    unsigned int* sw = status_word(&e);
    if (!sw) return cuda_fail(e, "status word");
    e = launch_cache_write(c, T, k, ks, v, vs, lens, ntok, dtype, sw, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "ring_attn_cache_write launch");
    return RA_OK;
}

ra_status ring_attn_cache_read(const void* k_cache, const void* v_cache, const void* k_exp, const void* v_exp, void* k, void* v,
                               int B, int Hkv, int row0, int rows, int d, int cap, int dtype, int cache_dtype, void* stream)
{
    const Cache c = cache_of(k_cache, v_cache, k_exp, v_exp, B, Hkv, cap, d, cache_dtype);
    ra_status st = check_cache(c, dtype);
    if (st != RA_OK) return st;
    if (row0 < 0 || rows < 0 || row0 > cap || rows > cap - row0)
        return fail(RA_ERR_INVALID_ARG, "rows [%d, %d + %d) outside the cache (%d rows)", row0, row0, rows, cap);
    if (rows == 0) return RA_OK;
    if ((st = check_ptrs({k, v})) != RA_OK) return st;
    if ((st = check_device()) != RA_OK) return st;
    cudaError_t e = launch_cache_read(c, row0, rows, k, v, dtype, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "ring_attn_cache_read launch");
    return RA_OK;
}

size_t ring_attn_tree_fwd_workspace_size(int B, int H, int Hkv, int T, int d, int cap, int dtype, int cache_dtype)
{
    if (B < 1 || H < 1 || Hkv < 1 || T < 1 || d < 1 || cap < 1 || H % Hkv != 0 || (long long)H * T >= (1LL << 30)) return 0;
    return tree_workspace_size(cache_of(nullptr, nullptr, nullptr, nullptr, B, Hkv, cap, d, cache_dtype), H, T, dtype);
}

ra_status ring_attn_tree_fwd(const void* q, const void* k_cache, const void* v_cache, const void* k_exp, const void* v_exp,
                             const int* lens, const int* ntok, const unsigned char* mask, int mask_batched, void* out, float* lse,
                             void* workspace, size_t workspace_bytes, int B, int H, int Hkv, int T, int d, int cap, int dtype,
                             int cache_dtype, int out_dtype, void* stream)
{
    const Cache c = cache_of(k_cache, v_cache, k_exp, v_exp, B, Hkv, cap, d, cache_dtype);
    return tree_impl(c, Tree{H, T, dtype, out_dtype, q, lens, ntok, mask, mask_batched ? 1 : 0, out, lse, workspace, nullptr, 0, 0, nullptr},
                     workspace_bytes, stream, "ring_attn_tree_fwd launch");
}

ra_status ring_attn_tree_window_fwd(const void* q, const void* k_cache, const void* v_cache, const void* k_exp, const void* v_exp,
                                    const int* lens, const int* ntok, const unsigned char* mask, int mask_batched,
                                    const int* positions, void* out, float* lse, void* workspace, size_t workspace_bytes, int B, int H,
                                    int Hkv, int T, int d, int cap, int window, int sinks, int dtype, int cache_dtype, int out_dtype,
                                    void* stream)
{
    const Cache c = cache_of(k_cache, v_cache, k_exp, v_exp, B, Hkv, cap, d, cache_dtype);
    if (window < 1) return fail(RA_ERR_INVALID_ARG, "window must be >= 1 (got %d)", window);
    if (sinks < 0) return fail(RA_ERR_INVALID_ARG, "sinks must be >= 0 (got %d)", sinks);
    if (positions && !mask) return fail(RA_ERR_INVALID_ARG, "positions need a mask: without one token t is at lens + t");
    ra_status st = check_ints("positions", positions, true);
    if (st != RA_OK) return st;
    return tree_impl(c, Tree{H, T, dtype, out_dtype, q, lens, ntok, mask, mask_batched ? 1 : 0, out, lse, workspace, nullptr, window, sinks, positions},
                     workspace_bytes, stream, "ring_attn_tree_window_fwd launch");
}

}  // extern "C"
