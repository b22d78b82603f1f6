// ra_internal.h -- declarations shared by the translation units of libringattn (not installed).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <initializer_list>

#include "ra_geometry.h"

namespace ra {

// Arguments of one attention problem, validated by the entry points.
struct Problem {
    int B, H, Hkv, L, d, n, causal, layout, dtype;
    Geometry geo() const { return make_geometry(L, n, layout, causal); }
    long long q_rows() const { return (long long)B * H * L; }
    long long kv_rows() const { return (long long)B * Hkv * L; }
};

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// bits of the device status word (the ABI's RA_DEVICE_* values; api.cu checks they agree)
constexpr unsigned kStatusTimeout = 1u;
constexpr unsigned kStatusLayout = 2u;
constexpr unsigned kStatusRange = 4u;

// One device's block call (the per-device data path of the multi-device ring): the query rows are
// those of shard q_shard alone and the keys those of shard kv_shard alone, each in a local buffer
// of S = L / n rows per head holding rows [shard * S, (shard + 1) * S) of the whole-sequence
// layout.  Positions, masks and the ring step (q_shard - kv_shard) mod n come from the whole
// sequence's geometry; only the addressing of the buffers changes.
struct BlockView {
    int q_shard = 0, kv_shard = 0;
    int acc_kv = 0;  // backward: add dK, dV into the float32 outputs (1) or store them (0)
};

// Output mode of a forward kernel.
enum FwdMode {
    kFwdFused = 0,     // all ring steps, write out (dtype) + lse
    kFwdRingStep = 1,  // one ring step, write float32 partial + lse (-inf when nothing visible)
    kFwdRingStepAcc = 2,  // one ring step folded into a running float32 output + lse, in place
    kFwdFusedF32 = 3,  // all ring steps, write out as float32 (before any rounding to dtype) + lse
};

// Does the mode walk every ring step (the whole K/V sequence) rather than one?
__host__ __device__ inline bool fwd_all_steps(int mode) { return mode == kFwdFused || mode == kFwdFusedF32; }

// SIMT (CUDA-core) kernels: any shape, f32 or bf16 inputs.
// blk (optional): one device's block call; the forward then runs ring step
// (q_shard - kv_shard) mod n for shard q_shard only (mode kFwdRingStep or kFwdRingStepAcc), the
// backward adds dQ into a float32 dq and stores or adds dK, dV (float32) as blk->acc_kv says.
cudaError_t launch_fwd_simt(const Problem& p, const void* q, const void* k, const void* v,
                            void* out, float* lse, int mode, int step, cudaStream_t s,
                            const BlockView* blk = nullptr);
cudaError_t launch_bwd_simt(const Problem& p, const void* q, const void* k, const void* v,
                            const void* dout, const float* D, const float* lse, void* dq,
                            void* dk, void* dv, int grad_dtype, cudaStream_t s,
                            const BlockView* blk = nullptr);

// Tensor-core kernels (TMA + tcgen05 + TMEM), bf16, d = 128 or 64: forward with chunk length %
// 256 == 0, backward with chunk length % 128 == 0.
bool tc_fwd_supported(const Problem& p);
// visits (optional, n x n): +1 at [query shard][key shard] for every tile pair computed.
cudaError_t launch_fwd_tc(const Problem& p, const void* q, const void* k, const void* v,
                          void* out, float* lse, int mode, int step, unsigned int* status,
                          cudaStream_t s, unsigned long long* visits = nullptr,
                          const BlockView* blk = nullptr);
bool tc_bwd_supported(const Problem& p);
cudaError_t launch_bwd_tc(const Problem& p, const void* q, const void* k, const void* v,
                          const void* dout, const float* D, const float* lse, float* dq_acc,
                          void* dk, void* dv, int grad_dtype, unsigned int* status,
                          cudaStream_t s, unsigned long long* visits = nullptr,
                          const BlockView* blk = nullptr);

// HBM-bound helper kernels.
// Rotary position embedding by natural position, in place, of a [B][H][L][d] buffer (p.H heads),
// or (shard >= 0) of one device's [B][H][L/n][d] buffer holding shard `shard`'s rows.
cudaError_t launch_rope(const Problem& p, void* x, double base, int inverse, cudaStream_t s, int shard = -1);
// theta_i / (2 pi) for theta_i = base^(-2i/d), i < d / 2, in units of 2^-64 turn (0 behind them).
void rope_turns(double base, int d, unsigned long long (&turn)[64]);

// Norm of every query and key head, then the rotation (dyq null), or the gradients of that.
struct NormRope {
    const void *q, *k;          // [B][heads][rows][d] by element strides (batch, head, row), d contiguous
    long long q_strides[3], k_strides[3];
    const float *wq, *wk;       // [d]
    const void *dyq, *dyk;      // backward: gradients of the outputs, contiguous
    void *out_q, *out_k;        // outputs, or dq and dk, contiguous
    float *dwq, *dwk, *partial; // backward: [d] each; kNormRopeBwdBlocks * 2 * d floats of scratch
    const int* positions;       // [B][rows], or null: natural positions of the layout
    int shard;                  // -1: whole-sequence buffers; else one device's shard
    double base, eps;
};
constexpr int kNormRopeBwdPerSm = 2;  // blocks of the backward on an SM
constexpr int kNormRopeBwdBlocks = 160 * kNormRopeBwdPerSm;  // and the most it launches (152 SMs here), which sizes the workspace
cudaError_t launch_norm_rope(const Problem& p, const NormRope& n, cudaStream_t s);

// A key/value cache: k, v [B][Hkv][cap][d] of `dtype` (a tensor dtype, or kCacheE4m3 with the rows'
// exponents + 127 in k_exp, v_exp [B][Hkv][cap]).
constexpr int kCacheE4m3 = 2;
struct Cache {
    int B, Hkv, cap, d, dtype;
    void *k, *v;
    uint8_t *k_exp, *v_exp;
};
// Tokens t < ntok[b] of k, v (element strides batch, head, row; d contiguous) to rows lens[b] + t.
cudaError_t launch_cache_write(const Cache& c, int T, const void* k, const long long* ks, const void* v, const long long* vs,
                               const int* lens, const int* ntok, int dtype, unsigned int* status, cudaStream_t s);
// Rows [row0, row0 + rows) of every head to k, v [B][Hkv][rows][d] of `dtype`.
cudaError_t launch_cache_read(const Cache& c, int row0, int rows, void* k, void* v, int dtype, cudaStream_t s);

// Attention of T drafted tokens per sequence over the cache (tree.cuh).
struct Tree {
    int H, T, dtype, out_dtype;
    const void* q;              // [B][H][T][d]
    const int *lens, *ntok;     // [B]; ntok may be null
    const uint8_t* mask;        // [B][T][T] or [T][T] truth values, or null: token t sees tokens <= t
    int mask_batched;
    void* out;                  // [B][H][T][d] out_dtype
    float* lse;                 // [B][H][T]
    void* workspace;
    unsigned int* status;
};
size_t tree_workspace_size(const Cache& c, int H, int T, int dtype);
cudaError_t launch_tree(const Cache& c, const Tree& t, cudaStream_t s);

// Ulysses all-to-all re-layout between the token split [n][B][S][H][row] and the head split
// [n][B][H/n][L][row] (direction 0 token -> head, 1 back); row_bytes a multiple of 4.
cudaError_t launch_ulysses_a2a(const Geometry& geo, int B, int H, int row_bytes, const void* src, void* dst,
                               int direction, cudaStream_t s);
cudaError_t launch_lse_merge(float* o_acc, float* lse_acc, const float* o_part,
                             const float* lse_part, long long rows, int d, cudaStream_t s);
cudaError_t launch_convert(const float* src, void* dst, int dst_dtype, long long count,
                           float scale, cudaStream_t s);
cudaError_t launch_bwd_preprocess(const void* out, const void* dout, int dtype, long long rows,
                                  int d, float* D, cudaStream_t s,
                                  int out_dtype = -1);
cudaError_t launch_zero(float* dst, long long count, cudaStream_t s);
// acc[i] += part[i] for count float32 values.
cudaError_t launch_add(float* acc, const float* part, long long count, cudaStream_t s);

// One thread waits on an mbarrier nothing completes (bounded wait of limit_ns); *returned = 1 when
// the wait gave up (and the timeout bit is set in *status), 2 if it completed.
cudaError_t launch_bounded_wait_selftest(unsigned int* status, unsigned long long limit_ns, unsigned int* returned,
                                         cudaStream_t s);

// Number of SMs of the current device (cached per device).
int device_sm_count();

// Shared by the entry points (api.cu).  fail / cuda_fail record the message and return the status;
// the checks return RA_OK or have failed.
int fail(int status, const char* fmt, ...);
int cuda_fail(cudaError_t e, const char* what);
int check_device();
int check_problem(const Problem& p);
int check_ptrs(std::initializer_list<const void*> ptrs);
// Device address of the status word of the current device, or null with *err set.
unsigned int* status_word(cudaError_t* err);

// Records `msg` as the calling thread's last error (ring_attn_last_error) and returns `status`.
int set_last_error(int status, const char* msg);

}  // namespace ra
