// window_tc.cuh -- what the tensor-core kernels of the attention through a window share: tiles of 128 consecutive
// positions out of buffers in any layout.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include <mutex>

#include "ra_internal.h"
#include "ra_ptx.cuh"
#include "window.cuh"

namespace ra {

constexpr int kWinTile = kWindowTile;  // positions of a tile

// Can TMA read 128 consecutive positions of this layout with one box?  Contiguous: always; zigzag: chunks of whole tiles;
// striped: a box of n shards by 128 / n rows, whose shard index runs fastest, is a run of positions.
RA_HD bool window_tma_reads(const Geometry& g)
{
    if (g.layout == 1) return g.Lc % kWinTile == 0;
    return g.layout != 2 || kWinTile % g.n == 0;
}

// Row coordinate of the tile that starts at position p (a multiple of 128) in the maps below.
RA_HD int window_tma_row(const Geometry& g, int p)
{
    return g.layout == 2 ? p / g.n : buffer_row(g, p);
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z)
{
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %6, %4, %5}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(0)
        : "memory");
}

// Columns c in [0, n) of a word of 32 from column `at`, one bit each.
__device__ __forceinline__ uint32_t bits_below(int n, int at)
{
    const int k = n - at;
    return k <= 0 ? 0u : k >= 32 ? ~0u : (1u << k) - 1u;
}

// A row's view of a tile of columns: [lo, hi) and [0, first).
struct Seen {
    int lo, hi, first;
    __device__ __forceinline__ uint32_t word(int at) const
    {
        return (bits_below(hi, at) & ~bits_below(lo, at)) | bits_below(first, at);
    }
};

// Keys k0 + c that the query at position p sees.
__device__ __forceinline__ Seen seen_keys(const Band& b, int p, int k0)
{
    const int end = (b.causal && p < b.L ? p + 1 : b.L) - k0;  // one past the last key that may count
    Seen s;
    s.lo = p - b.W + 1 - k0;
    s.hi = b.causal ? end : (p + b.W - k0 < end ? p + b.W - k0 : end);
    s.first = b.S - k0 < end ? b.S - k0 : end;
    return s;
}

// Queries q0 + c that see the key at position j.
__device__ __forceinline__ Seen seen_queries(const Band& b, int j, int q0)
{
    const int end = b.L - q0;
    Seen s;
    s.lo = (b.causal ? j : j - b.W + 1) - q0;
    s.hi = j >= b.L ? s.lo : j < b.S || j + b.W > b.L ? end : j + b.W - q0;  // (sinks: to the end)
    s.first = j < b.S && !b.causal ? end : 0;
    return s;
}

namespace {

PFN_cuTensorMapEncodeTiled_v12000 encode_fn()
{
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    });
    return fn;
}

// [heads][shards][rows][d] bf16 as (d, shards, rows, heads), boxes of 64 columns by 128 positions in natural order, 128-byte
// swizzle.  One "shard" of all rows unless striped.  Positions past the sequence read as zeros.
bool make_map(CUtensorMap* map, const void* base, const Geometry& g, long long heads, int d)
{
    auto fn = encode_fn();
    if (!fn) return false;
    const int n = g.layout == 2 ? g.n : 1;
    const cuuint64_t rows = (cuuint64_t)(g.layout == 2 ? g.S : g.L);
    cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)n, rows, (cuuint64_t)heads};
    cuuint64_t strides[3] = {rows * (cuuint64_t)d * 2, (cuuint64_t)d * 2, (cuuint64_t)g.L * d * 2};
    cuuint32_t box[4] = {64, (cuuint32_t)n, (cuuint32_t)(kWinTile / n), 1};
    cuuint32_t estr[4] = {1, 1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Wait without the abort shortcut, for draining copies and MMAs already in flight.
__device__ __forceinline__ void drain_wait(uint32_t bar, uint32_t parity)
{
    const uint64_t t0 = global_timer_ns();
    while (!mbar_try_wait(bar, parity)) {
        if (global_timer_ns() - t0 > 1000000000ull) return;
    }
}

// The issuing warp runs as a whole, so that descriptors and addresses are the same in every lane and stay in uniform
// registers; one elected lane (`lead`) issues.  (One thread of a diverged warp issues more slowly than the softmax warps
// work: the forward of 64K tokens, window 128, took 485 us with 64 registers that way, 422 with 120.)
__device__ __forceinline__ uint32_t elect()
{
    uint32_t e;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
    return e;
}
__device__ __forceinline__ void lead_mma_ss(uint32_t lead, uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p, l;\n\t"
        "setp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 l, %5, 0;\n\t"
        "@l tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(lead)
        : "memory");
}
__device__ __forceinline__ void lead_mma_ts(uint32_t lead, uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p, l;\n\t"
        "setp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 l, %5, 0;\n\t"
        "@l tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(lead)
        : "memory");
}
__device__ __forceinline__ void lead_commit(uint32_t lead, uint32_t bar)
{
    asm volatile(
        "{\n\t.reg .pred l;\n\tsetp.ne.b32 l, %1, 0;\n\t"
        "@l tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar), "r"(lead)
        : "memory");
}
// A wait of the whole warp: every lane learns whether all of them saw the phase.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, const WaitCtl& ctl)
{
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, ctl));
}

// Allows a kernel `smem` bytes of shared memory, once per device.
template <typename K>
cudaError_t allow_smem(K kernel, int smem, std::mutex& mu, bool (&done)[64])
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lk(mu);
    if (!done[dev]) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        done[dev] = true;
    }
    return cudaSuccess;
}

}  // namespace
}  // namespace ra
