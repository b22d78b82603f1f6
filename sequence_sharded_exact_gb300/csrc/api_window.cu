// api_window.cu -- the C ABI of the attention through a window over whole sequences (declared in include/ringattn.h).
#include <math.h>

#include "../../include/ringattn.h"
#include "ra_internal.h"
#include "window_tc.cuh"

namespace ra {
namespace {

size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

ra_status check_window(const Problem& p, int window, int sinks)
{
    ra_status st = check_problem(p);
    if (st != RA_OK) return st;
    if (window < 1) return fail(RA_ERR_INVALID_ARG, "window must be >= 1 (got %d)", window);
    if (sinks < 0) return fail(RA_ERR_INVALID_ARG, "sinks must be >= 0 (got %d)", sinks);
    if (p.L >= (1 << 30) || (long long)p.B * p.H * ((p.L + 63) / 64) >= (1LL << 30))
        return fail(RA_ERR_UNSUPPORTED, "problem too large");
    return RA_OK;
}

ra_status check_space(const void* ws, size_t have, size_t need)
{
    if (need == 0) return RA_OK;
    ra_status st = check_ptrs({ws});
    if (st != RA_OK) return st;
    if (reinterpret_cast<uintptr_t>(ws) & 255u) return fail(RA_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
    if (have < need) return fail(RA_ERR_INVALID_ARG, "workspace too small: %zu < %zu bytes", have, need);
    return RA_OK;
}

WindowArgs args_of(const Problem& p, int window, int sinks)
{
    WindowArgs a = {};
    a.geo = a.store_geo = p.geo();
    a.band = Band{p.L, window < p.L ? window : p.L, sinks < p.L ? sinks : p.L, p.causal};
    a.B = p.B;
    a.H = p.H;
    a.Hkv = p.Hkv;
    a.G = p.H / p.Hkv;
    a.scale = 1.0f / sqrtf((float)p.d);
    a.scale_log2 = kLog2e / sqrtf((float)p.d);
    return a;
}

// bf16 inputs that TMA cannot read in natural order are copied into it, one after another in the workspace.
bool copies(const Problem& p) { return p.dtype == RA_BF16 && !window_tma_reads(p.geo()); }
size_t copy_bytes(const Problem& p, int heads) { return up256((size_t)p.B * heads * p.L * p.d * 2); }

WindowCopies copies_at(const Problem& p, void* at, bool backward)
{
    char* x = static_cast<char*>(at);
    WindowCopies w;
    w.q = x;
    w.k = x + copy_bytes(p, p.H);
    w.v = x + copy_bytes(p, p.H) + copy_bytes(p, p.Hkv);
    w.dout = backward ? x + copy_bytes(p, p.H) + 2 * copy_bytes(p, p.Hkv) : nullptr;
    return w;
}

// The products read the copies.
void read_copies(WindowArgs& a, const WindowCopies& w)
{
    a.q = w.q;
    a.k = w.k;
    a.v = w.v;
    if (w.dout) a.dout = w.dout;
    a.geo = make_geometry(a.band.L, 1, RA_LAYOUT_CONTIGUOUS, a.band.causal);
}

}  // namespace
}  // namespace ra

using namespace ra;

extern "C" {

size_t ring_attn_window_fwd_workspace_size(int B, int H, int Hkv, int L, int d, int n_shards, int layout, int dtype)
{
    const Problem p{B, H, Hkv, L, d, n_shards, 1, layout, dtype};
    if (check_window(p, 1, 0) != RA_OK || !copies(p)) return 0;
    return copy_bytes(p, H) + 2 * copy_bytes(p, Hkv);
}

ra_status ring_attn_window_fwd(const void* q, const void* k, const void* v, void* out, float* lse, void* workspace,
                               size_t workspace_bytes, int B, int H, int Hkv, int L, int d, int n_shards, int window, int sinks,
                               int causal, int layout, int dtype, int out_dtype, void* stream)
{
    const Problem p{B, H, Hkv, L, d, n_shards, causal, layout, dtype};
    ra_status st = check_window(p, window, sinks);
    if (st != RA_OK) return st;
    if (out_dtype != dtype && out_dtype != RA_F32) return fail(RA_ERR_INVALID_ARG, "out_dtype must be the dtype of q or RA_F32");
    if ((st = check_ptrs({q, k, v, out, lse})) != RA_OK) return st;
    if ((st = check_space(workspace, workspace_bytes, ring_attn_window_fwd_workspace_size(B, H, Hkv, L, d, n_shards, layout, dtype))) != RA_OK)
        return st;
    if ((st = check_device()) != RA_OK) return st;
    WindowArgs a = args_of(p, window, sinks);
    a.q = q;
    a.k = k;
    a.v = v;
    a.o = out;
    a.lse = lse;
    a.out_dtype = out_dtype;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (dtype == RA_BF16) {
        unsigned int* sw = status_word(&e);
        if (!sw) return cuda_fail(e, "status word");
        if (copies(p)) {
            const WindowCopies w = copies_at(p, workspace, false);
            if ((e = launch_window_copies(a, w, d, s)) != cudaSuccess) return cuda_fail(e, "ring_attn_window_fwd copies");
            read_copies(a, w);
        }
        e = d == 128 ? launch_window_fwd_tc_d128(a, sw, s) : launch_window_fwd_tc_d64(a, sw, s);
    } else {
        e = launch_window_fwd_simt(a, d, s);
    }
    if (e != cudaSuccess) return cuda_fail(e, "ring_attn_window_fwd launch");
    return RA_OK;
}

size_t ring_attn_window_bwd_workspace_size(int B, int H, int Hkv, int L, int d, int n_shards, int window, int sinks, int causal,
                                           int layout, int dtype)
{
    const Problem p{B, H, Hkv, L, d, n_shards, causal, layout, dtype};
    if (check_window(p, window, sinks) != RA_OK) return 0;
    if (dtype == RA_F32) return window_simt_plan(args_of(p, window, sinks).band, B, H, Hkv, d).bytes;
    return window_bwd_plan(args_of(p, window, sinks).band, B, H, Hkv, d).bytes +
           (copies(p) ? 2 * copy_bytes(p, H) + 2 * copy_bytes(p, Hkv) : 0);
}

ra_status ring_attn_window_bwd(const void* q, const void* k, const void* v, const void* out, const float* lse, const void* dout,
                               void* dq, void* dk, void* dv, void* workspace, size_t workspace_bytes, int B, int H, int Hkv, int L,
                               int d, int n_shards, int window, int sinks, int causal, int layout, int dtype, int out_dtype,
                               int grad_dtype, void* stream)
{
    const Problem p{B, H, Hkv, L, d, n_shards, causal, layout, dtype};
    ra_status st = check_window(p, window, sinks);
    if (st != RA_OK) return st;
    if (out_dtype != dtype && out_dtype != RA_F32) return fail(RA_ERR_INVALID_ARG, "out_dtype must be the dtype of q or RA_F32");
    if (grad_dtype != RA_F32 && grad_dtype != RA_BF16) return fail(RA_ERR_INVALID_ARG, "unknown grad dtype %d", grad_dtype);
    if ((st = check_ptrs({q, k, v, out, lse, dout, dq, dk, dv})) != RA_OK) return st;
    const size_t need = ring_attn_window_bwd_workspace_size(B, H, Hkv, L, d, n_shards, window, sinks, causal, layout, dtype);
    if ((st = check_space(workspace, workspace_bytes, need)) != RA_OK) return st;
    if ((st = check_device()) != RA_OK) return st;
    WindowArgs a = args_of(p, window, sinks);
    a.q = q;
    a.k = k;
    a.v = v;
    a.out = out;
    a.dout = dout;
    a.lse = const_cast<float*>(lse);
    a.dq = dq;
    a.dk = dk;
    a.dv = dv;
    a.saved_dtype = out_dtype;
    a.grad_dtype = grad_dtype;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (dtype == RA_BF16) {
        unsigned int* sw = status_word(&e);
        if (!sw) return cuda_fail(e, "status word");
        char* ws = static_cast<char*>(workspace);
        WindowBwdPlan plan = window_bwd_plan(a.band, B, H, Hkv, d);
        plan.lse2 = reinterpret_cast<float*>(ws + plan.lse_at);
        plan.D = reinterpret_cast<float*>(ws + plan.D_at);
        plan.dq = reinterpret_cast<float*>(ws + plan.dq_at);
        plan.part = reinterpret_cast<float*>(ws + plan.part_at);
        const WindowCopies w = copies(p) ? copies_at(p, ws + plan.bytes, true) : WindowCopies{};
        e = launch_window_bwd_before(a, plan, w, d, s);
        if (w.dout) read_copies(a, w);
        if (e == cudaSuccess) e = d == 128 ? launch_window_bwd_tc_d128(a, plan, sw, s) : launch_window_bwd_tc_d64(a, plan, sw, s);
        if (e == cudaSuccess) e = launch_window_bwd_after(a, plan, d, s);
    } else {
        e = launch_window_bwd_simt(a, window_simt_plan(a.band, B, H, Hkv, d), workspace, d, s);
    }
    if (e != cudaSuccess) return cuda_fail(e, "ring_attn_window_bwd launch");
    return RA_OK;
}

}  // extern "C"
