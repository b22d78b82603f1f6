// tree_mma.cuh -- what the kernels for few query rows per kv head (tree_mma.cu, tree_mma_bf16.cu) share.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include <mutex>

#include "ra_internal.h"
#include "ra_ptx.cuh"
#include "tree.cuh"

namespace ra {
namespace {

constexpr int kKeys = 16;  // cached rows of a warp's turn
constexpr long long kWaitLimit = 10000000000ll;

struct Maps {
    CUtensorMap k, v;
};

// A bounded wait by the whole warp.  After one has given up (or another warp's) every further wait returns at once, and
// the caller goes on to its end with whatever is there: the status word says that the results do not count.
__device__ __forceinline__ void warp_wait(uint32_t bar, uint32_t parity, const WaitCtl& ctl)
{
    if (!mbar_try_wait(bar, parity)) {
        const long long t0 = clock64();
        while (!mbar_try_wait(bar, parity)) {
            if (*ctl.abort) break;
            if (clock64() - t0 > kWaitLimit) {
                *ctl.abort = 1;
                atomicOr(ctl.status, kStatusTimeout);
                break;
            }
        }
    }
    __syncwarp();
}

__device__ __forceinline__ void drain_wait(uint32_t bar, uint32_t parity)
{
    const uint64_t t0 = global_timer_ns();
    while (!mbar_try_wait(bar, parity)) {
        if (global_timer_ns() - t0 > 1000000000ull) return;
    }
}

// Rows g of an 8 x 8 matrix of 16-bit values, two columns 2t, 2t + 1 per thread: its transpose in the same places.
__device__ __forceinline__ uint32_t transpose8(uint32_t x)
{
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

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
