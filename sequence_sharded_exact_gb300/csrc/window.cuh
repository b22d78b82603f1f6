// window.cuh -- attention of a whole sequence through a sliding window, with a few first tokens that stay visible
// (sinks): what its kernels share.
//
// Natural positions p (query) and j (key) of a sequence of L tokens, window W >= 1, S sinks:
//   causal:  p sees j  iff  j <= p and (p - j < W or j < S);      otherwise:  iff  |p - j| < W or j < S.
//   s = q k / sqrt(d),  out = sum_j exp(s_j - lse) v_j,  lse = ln sum_j exp(s_j);
//   D = dout . out,  P = exp(s - lse),  dS = P (dout . v - D) / sqrt(d),  dq = dS k,  dk = dS^T q,  dv = P^T dout,
// dk and dv summed over the query heads that share a kv head.  Every row sees itself.
//
// The kernels work in natural order whatever the layout: a tile is a run of consecutive positions, so that a query tile
// meets W / tile + 1 key tiles and the sinks' in every layout (in the striped one's buffer order a tile of 128 rows spans
// 128 n positions, and most of what it meets would lie outside the window).  Only loads and stores know the layout.
#pragma once

#include "ra_internal.h"

namespace ra {

// Clamped to the sequence: 1 <= W <= L, 0 <= S <= L.
struct Band {
    int L, W, S, causal;
};

RA_HD bool band_sees(const Band& b, int p, int j)
{
    if (b.causal) return j <= p && (p - j < b.W || j < b.S);
    return (p - j < b.W && j - p < b.W) || j < b.S;
}

// Do all of the queries [q0, q0 + nq) see all of the keys [k0, k0 + nk), every one of them in the sequence?
RA_HD bool band_tile_whole(const Band& b, int q0, int nq, int k0, int nk)
{
    const int q1 = q0 + nq - 1, k1 = k0 + nk - 1;
    if (q1 >= b.L || k1 >= b.L || (b.causal && k1 > q0)) return false;
    return k1 < b.S || (q1 - k0 < b.W && (b.causal || k1 - q0 < b.W));
}

// The key tiles (of `tile` positions) that queries [q0, q0 + rows) meet: [first, last) and [0, sinks), those inside the window
// before the sinks' and its two ends: a maximum over a whole tile seldom has to be raised afterwards, one over the few keys
// that a row sees of the others often.
struct TileRun {
    int sinks, first, last;
    RA_HD int count() const { return sinks + last - first; }
    RA_HD int at(int i) const
    {
        const int inside = last - first > 2 ? last - first - 2 : 0;
        if (i < inside) return first + 1 + i;
        i -= inside;
        return i < sinks ? i : i == sinks ? first : last - 1;
    }
};

RA_HD TileRun key_tiles(const Band& b, int q0, int rows, int tile)
{
    const int q1 = q0 + rows < b.L ? q0 + rows : b.L;  // one past the last query
    const int lo = q0 - b.W + 1 > 0 ? q0 - b.W + 1 : 0;
    const int hi = b.causal || b.W > b.L - q1 ? (b.causal ? q1 : b.L) : q1 + b.W - 1;  // one past the last key of a window
    TileRun r;
    r.first = lo / tile;
    r.last = (hi + tile - 1) / tile;
    const int limit = b.causal && b.S > q1 ? q1 : b.S;  // one past the last sink that a query sees
    const int st = (limit + tile - 1) / tile;
    if (st >= r.first) {  // the sinks' tiles run into the window's: one run
        r.first = 0;
        r.sinks = 0;
        if (st > r.last) r.last = st;
    } else {
        r.sinks = st;
    }
    return r;
}

// The query tiles [first, last) that keys [k0, k0 + rows) meet, through the window or as sinks.
struct QueryRun {
    int first, last;
};

RA_HD QueryRun query_tiles(const Band& b, int k0, int rows, int tile)
{
    const int k1 = k0 + rows < b.L ? k0 + rows : b.L;
    QueryRun r;
    if (k0 < b.S) {  // sinks: every query, or (causal) every later one
        r.first = b.causal ? k0 / tile : 0;
        r.last = (b.L + tile - 1) / tile;
        return r;
    }
    const int lo = b.causal ? k0 : (k0 - b.W + 1 > 0 ? k0 - b.W + 1 : 0);
    const int hi = b.W > b.L - k1 ? b.L : k1 + b.W - 1;
    r.first = lo / tile;
    r.last = (hi + tile - 1) / tile;
    return r;
}

struct WindowArgs {
    Geometry geo;        // of the inputs (out and lse apart)
    Geometry store_geo;  // of all others
    Band band;
    int B, H, Hkv, G;
    const void *q, *k, *v;
    const void *out, *dout;  // backward
    void* o;                 // forward
    const float* D;          // backward: [B][H][L], natural order
    float* lse;
    void *dq, *dk, *dv;
    float scale, scale_log2;
    int out_dtype, grad_dtype, saved_dtype;
};

// CUDA-core path: float32 (window_simt.cu).
cudaError_t launch_window_fwd_simt(const WindowArgs& a, int d, cudaStream_t s);
struct WindowSimtPlan {
    int tiles, sink_tiles, segs;  // of 64 positions
    bool parts;                   // dK and dV are joined from parts
    long long key_blocks;
    size_t D_bytes, bytes;        // workspace: D, then the parts
};
WindowSimtPlan window_simt_plan(const Band& b, int B, int H, int Hkv, int d);
cudaError_t launch_window_bwd_simt(const WindowArgs& a, const WindowSimtPlan& p, void* workspace, int d, cudaStream_t s);


// Tensor-core path, bf16, layouts that window_tma_reads (window_tc.cuh).
cudaError_t launch_window_fwd_tc_d128(const WindowArgs& a, unsigned int* status, cudaStream_t s);
cudaError_t launch_window_fwd_tc_d64(const WindowArgs& a, unsigned int* status, cudaStream_t s);

// The backward's cut and its workspace.
constexpr int kWindowTile = 128;
constexpr int kWindowCtas = 152;  // a round of units: the SMs of the whole GPU (with fewer the results are the same)
struct WindowBwdPlan {
    int tiles, sink_tiles, segs;  // tiles of the sequence and with sinks; segments of each of the latter
    // The launches start while the one before them runs, where dQ's accumulator is at most 128 MB: two sequences of 1000 tokens
    // of 8 heads of 64 take 25.4 us in place of 28.2, but 64K tokens of 32 heads of 128 (1 GB) 8.92 ms in place of 8.80.
    bool early;
    long long sink_items;         // segments in all (0: no sinks)
    // The other tiles: `whole` of them have a unit each, the `tail` behind these, which would fill a last round of CTAs in part,
    // are cut into tail_segs units each (1: none is): 5005 tokens in 7 stripes, 368 units in 3 rounds of 152, 216 -> 203 us;
    // 2048 tokens of 8 : 2 heads of 128, window 512, 32 units, 57 -> 32 us.
    long long whole, tail;
    int tail_segs;
    long long parts() const { return (segs > 1 ? sink_items : 0) + (tail_segs > 1 ? tail * tail_segs : 0); }
    size_t lse_at, D_at, dq_at, part_at, bytes;
    float *lse2, *D, *dq, *part;
};
WindowBwdPlan window_bwd_plan(const Band& b, int B, int H, int Hkv, int d);  // (no CUDA call)
cudaError_t launch_window_bwd_tc_d128(const WindowArgs& a, const WindowBwdPlan& p, unsigned int* status, cudaStream_t s);
cudaError_t launch_window_bwd_tc_d64(const WindowArgs& a, const WindowBwdPlan& p, unsigned int* status, cudaStream_t s);
// Copies in natural order, where TMA cannot read the inputs so (dout null: none, but for the forward's).
struct WindowCopies {
    void *q, *k, *v, *dout;
};
cudaError_t launch_window_copies(const WindowArgs& a, const WindowCopies& w, int d, cudaStream_t s);
// What comes before and after the backward (window_aux.cu): D, lse2, a cleared dq and the copies; dq and the sinks' dk, dv.
cudaError_t launch_window_bwd_before(const WindowArgs& a, const WindowBwdPlan& p, const WindowCopies& w, int d, cudaStream_t s);
cudaError_t launch_window_bwd_after(const WindowArgs& a, const WindowBwdPlan& p, int d, cudaStream_t s);

// Launches a kernel that may start while the one before it in the stream runs (early) and waits for its results itself.
template <typename K, typename... A>
cudaError_t launch_next(bool early, K kernel, unsigned grid, unsigned threads, size_t smem, cudaStream_t s, const A&... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = early ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace ra
