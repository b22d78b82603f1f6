// cache.cu -- the key/value cache: rows quantised as they are written, and read back (HBM-bound).
//
// A cache holds k and v as [B][Hkv][cap][d] in the model's dtype, or in e4m3 with one power-of-two
// scale per row (one token of one kv head): the smallest 2^e, e >= -126, with amax <= 448 * 2^e (448
// is e4m3's largest value), stored as the byte e + 127.  Element x is stored as the e4m3 value
// nearest to x 2^-e (ties to even) and stands for that value times 2^e.  A power of two costs no
// accuracy against amax / 448 as the scale (e4m3 is a floating-point format: only the range below
// its smallest normal value moves, by less than a binade) and keeps the scaling and the reading back
// exact: the row's rounding is the conversion to e4m3 alone, at most 2^-4 of an element that is a
// normal e4m3 value after scaling.  amax passes over NaN, which is stored as NaN; an infinite amax
// takes e = 120, under which 448 * 2^e reads back as infinity.
//
// What bounds it: each element is read once and written once.  d / 8 lanes hold a row (8 elements a
// lane: 16 or 32 bytes in, 8 out; read back 16 elements), its largest magnitude is a shuffle
// reduction in that group, and kUnroll rows are loaded before the first is used.
//
// Measured, 131072 rows of 8 kv heads of 128 between bf16 and e4m3 (0.81 GB): written in 123 us (6.55 TB/s, 0.96 of the
// copy rate), read back in 130 us (6.2 TB/s, 0.91).  With one division per row, in a grid over all rows, it
// was 236 and 152 us.  Reading back with 8 bytes a lane and row: 134 us; with two or eight rows ahead, in place of four:
// 140, 130.
#include <cuda_bf16.h>

#include "ra_internal.h"
#include "ra_ptx.cuh"

namespace ra {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;      // rows per group and turn, written
constexpr int kUnrollRead = 4;  // and read back: 16 bytes a lane and row come in

template <typename T>
struct Eight {  // eight consecutive elements of T
    uint4 v[sizeof(T) / 2];
    __device__ __forceinline__ void load(const T* p)
    {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) v[i] = reinterpret_cast<const uint4*>(p)[i];
    }
    __device__ __forceinline__ void store(T* p) const
    {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) reinterpret_cast<uint4*>(p)[i] = v[i];
    }
    __device__ __forceinline__ void get(float (&f)[8]) const;
    __device__ __forceinline__ void set(const float (&f)[8]);
};

template <>
__device__ __forceinline__ void Eight<float>::get(float (&f)[8]) const
{
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        f[4 * i] = __uint_as_float(v[i].x);
        f[4 * i + 1] = __uint_as_float(v[i].y);
        f[4 * i + 2] = __uint_as_float(v[i].z);
        f[4 * i + 3] = __uint_as_float(v[i].w);
    }
}
template <>
__device__ __forceinline__ void Eight<float>::set(const float (&f)[8])
{
#pragma unroll
    for (int i = 0; i < 2; ++i)
        v[i] = make_uint4(__float_as_uint(f[4 * i]), __float_as_uint(f[4 * i + 1]), __float_as_uint(f[4 * i + 2]),
                          __float_as_uint(f[4 * i + 3]));
}
template <>
__device__ __forceinline__ void Eight<__nv_bfloat16>::get(float (&f)[8]) const
{
    const uint32_t w[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
template <>
__device__ __forceinline__ void Eight<__nv_bfloat16>::set(const float (&f)[8])
{
    v[0] = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
}

// The row's exponent from its largest magnitude, by its bits: amax = 1.f * 2^E, 448 = 1.75 * 2^8.
__device__ __forceinline__ int row_exponent(float amax)
{
    const uint32_t bits = __float_as_uint(amax);
    const int e = (int)(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
    return e < -126 ? -126 : (e > 120 ? 120 : e);
}

struct WriteArgs {
    int B, Hkv, T, cap;
    const void *k, *v;
    long long ks[3], vs[3];  // element strides: batch, head, row
    void *k_out, *v_out;
    uint8_t *k_exp, *v_exp;  // null: the cache holds the inputs' dtype
    const int *lens, *ntok;  // either may be null: 0, T
    unsigned int* status;
};

// Grid: blocks of rows, heads of all sequences, k or v.  A block stays with one head, so that a row costs no division.
template <typename T, int D, bool QUANT>
__global__ void __launch_bounds__(kThreads) cache_write_kernel(const WriteArgs a)
{
    constexpr int LPR = D / 8, kGroups = kThreads / LPR;
    const int ch = threadIdx.x % LPR, grp = threadIdx.x / LPR;
    const unsigned mask = ((1u << LPR) - 1u) << (threadIdx.x & 31 & ~(LPR - 1));
    const bool is_v = blockIdx.z != 0;
    const long long s0 = is_v ? a.vs[0] : a.ks[0], s1 = is_v ? a.vs[1] : a.ks[1], s2 = is_v ? a.vs[2] : a.ks[2];
    for (int bh = blockIdx.y; bh < a.B * a.Hkv; bh += gridDim.y) {
        const int b = bh / a.Hkv, h = bh - b * a.Hkv;
        const int len = a.lens ? a.lens[b] : 0, given = a.ntok ? a.ntok[b] : a.T;
        int n = given < 0 ? 0 : (given > a.T ? a.T : given);
        const int fit = len < 0 || len > a.cap ? 0 : (n < a.cap - len ? n : a.cap - len);
        if ((n != given || fit != n) && blockIdx.x == 0 && h == 0 && !is_v && threadIdx.x == 0) atomicOr(a.status, kStatusRange);
        n = fit;
        const T* src = static_cast<const T*>(is_v ? a.v : a.k) + b * s0 + h * s1 + ch * 8;
        const long long row0 = (long long)bh * a.cap + len;
        for (int t0 = blockIdx.x * (kGroups * kUnroll) + grp; t0 < n; t0 += gridDim.x * (kGroups * kUnroll)) {
            Eight<T> x[kUnroll];
#pragma unroll
            for (int u = 0; u < kUnroll; ++u)
                if (t0 + u * kGroups < n) x[u].load(src + (long long)(t0 + u * kGroups) * s2);
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                if (t0 + u * kGroups >= n) break;  // the same for every lane of a row
                const long long dst = row0 + t0 + u * kGroups;
                if constexpr (!QUANT) {
                    x[u].store(static_cast<T*>(is_v ? a.v_out : a.k_out) + dst * D + ch * 8);
                } else {
                    float f[8], m = 0.f;
                    x[u].get(f);
#pragma unroll
                    for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(f[e]));
#pragma unroll
                    for (int o = LPR / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(mask, m, o));
                    const int e = row_exponent(m);
                    const float down = __uint_as_float((uint32_t)(127 - e) << 23);  // 2^-e
                    uint2 w;
                    w.x = (uint32_t)e4m3x2(f[0] * down, f[1] * down) | (uint32_t)e4m3x2(f[2] * down, f[3] * down) << 16;
                    w.y = (uint32_t)e4m3x2(f[4] * down, f[5] * down) | (uint32_t)e4m3x2(f[6] * down, f[7] * down) << 16;
                    *reinterpret_cast<uint2*>(static_cast<uint8_t*>(is_v ? a.v_out : a.k_out) + dst * D + ch * 8) = w;
                    if (ch == 0) (is_v ? a.v_exp : a.k_exp)[dst] = (uint8_t)(e + 127);
                }
            }
        }
    }
}

// 32 bytes at p, in one store where p allows it (`wide`: a 32-byte boundary).
__device__ __forceinline__ void store32(void* p, const uint32_t (&v)[8], bool wide)
{
    if (wide) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]),
                     "r"(v[5]), "r"(v[6]), "r"(v[7])
                     : "memory");
    } else {
        reinterpret_cast<uint4*>(p)[0] = make_uint4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<uint4*>(p)[1] = make_uint4(v[4], v[5], v[6], v[7]);
    }
}

struct ReadArgs {
    bool wide;                   // the outputs lie on 32-byte boundaries
    int heads, cap, row0, rows;  // heads of all sequences
    const void *k, *v;
    const uint8_t *k_exp, *v_exp;
    void *k_out, *v_out;
};

// Quantised rows: 16 elements a lane, 16 bytes in and 32 (bf16) or 64 out.  Rows in the outputs' dtype are copied, 16
// bytes a lane.
template <typename T, int D, bool QUANT>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(const ReadArgs a)
{
    constexpr int E = QUANT ? 16 : 16 / sizeof(T), LPR = D / E, kGroups = kThreads / LPR;
    const int ch = threadIdx.x % LPR, grp = threadIdx.x / LPR;
    const bool is_v = blockIdx.z != 0;
    for (int bh = blockIdx.y; bh < a.heads; bh += gridDim.y) {
        const long long in0 = (long long)bh * a.cap + a.row0, out0 = (long long)bh * a.rows;
        const uint8_t* exps = is_v ? a.v_exp : a.k_exp;
        const uint8_t* in = static_cast<const uint8_t*>(is_v ? a.v : a.k) + ch * 16;
        T* out = static_cast<T*>(is_v ? a.v_out : a.k_out) + out0 * D + ch * E;
        for (int t0 = blockIdx.x * (kGroups * kUnrollRead) + grp; t0 < a.rows; t0 += gridDim.x * (kGroups * kUnrollRead)) {
            uint4 w[kUnrollRead];
            uint32_t e[kUnrollRead];
#pragma unroll
            for (int u = 0; u < kUnrollRead; ++u) {
                if (t0 + u * kGroups >= a.rows) break;
                const long long src = in0 + t0 + u * kGroups;
                w[u] = *reinterpret_cast<const uint4*>(in + src * (D / E * 16));
                if constexpr (QUANT) e[u] = exps[src];
            }
#pragma unroll
            for (int u = 0; u < kUnrollRead; ++u) {
                if (t0 + u * kGroups >= a.rows) break;
                T* dst = out + (long long)(t0 + u * kGroups) * D;
                if constexpr (QUANT) {
                    const float up = __uint_as_float(e[u] << 23);  // 2^(byte - 127), byte 1 .. 247
                    const uint32_t x[4] = {w[u].x, w[u].y, w[u].z, w[u].w};
                    uint32_t o[4 * sizeof(T)];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        float f[4];
                        e4m3x4_to_float(x[j], f[0], f[1], f[2], f[3]);
#pragma unroll
                        for (int i = 0; i < 4; ++i) f[i] *= up;
                        if constexpr (sizeof(T) == 4) {
#pragma unroll
                            for (int i = 0; i < 4; ++i) o[4 * j + i] = __float_as_uint(f[i]);
                        } else {
                            o[2 * j] = pack_bf16x2(f[0], f[1]);
                            o[2 * j + 1] = pack_bf16x2(f[2], f[3]);
                        }
                    }
#pragma unroll
                    for (int i = 0; i < (int)sizeof(T) / 2; ++i) {
                        const uint32_t part[8] = {o[8 * i], o[8 * i + 1], o[8 * i + 2], o[8 * i + 3], o[8 * i + 4], o[8 * i + 5], o[8 * i + 6], o[8 * i + 7]};
                        store32(reinterpret_cast<uint8_t*>(dst) + 32 * i, part, a.wide);
                    }
                } else {
                    *reinterpret_cast<uint4*>(dst) = w[u];
                }
            }
        }
    }
}

// Blocks for `rows` rows of every head: enough for all of them, at most eight per SM over k and v and the heads.
dim3 cache_grid(long long heads, long long rows, int lanes, int unroll)
{
    const long long per = (long long)(kThreads / lanes) * unroll;
    const long long y = heads < 65535 ? heads : 65535;
    long long most = (long long)device_sm_count() * 8 / (2 * y);
    if (most < 1) most = 1;
    const long long x = (rows + per - 1) / per;
    return dim3((unsigned)(x < most ? x : most), (unsigned)y, 2);
}

template <typename T, int D>
void write_as(const WriteArgs& a, bool quant, dim3 grid, cudaStream_t s)
{
    if (quant)
        cache_write_kernel<T, D, true><<<grid, kThreads, 0, s>>>(a);
    else
        cache_write_kernel<T, D, false><<<grid, kThreads, 0, s>>>(a);
}

template <typename T, int D>
void read_as(const ReadArgs& a, bool quant, dim3 grid, cudaStream_t s)
{
    if (quant)
        cache_read_kernel<T, D, true><<<grid, kThreads, 0, s>>>(a);
    else
        cache_read_kernel<T, D, false><<<grid, kThreads, 0, s>>>(a);
}

}  // namespace

cudaError_t launch_cache_write(const Cache& c, int T, const void* k, const long long* ks, const void* v, const long long* vs,
                               const int* lens, const int* ntok, int dtype, unsigned int* status, cudaStream_t s)
{
    WriteArgs a;
    a.B = c.B;
    a.Hkv = c.Hkv;
    a.T = T;
    a.cap = c.cap;
    a.k = k;
    a.v = v;
    for (int i = 0; i < 3; ++i) {
        a.ks[i] = ks[i];
        a.vs[i] = vs[i];
    }
    a.k_out = c.k;
    a.v_out = c.v;
    a.k_exp = c.k_exp;
    a.v_exp = c.v_exp;
    a.lens = lens;
    a.ntok = ntok;
    a.status = status;
    const bool quant = c.dtype != dtype;
    const dim3 grid = cache_grid((long long)c.B * c.Hkv, T, c.d / 8, kUnroll);
    if (dtype == 1)
        c.d == 128 ? write_as<__nv_bfloat16, 128>(a, quant, grid, s) : write_as<__nv_bfloat16, 64>(a, quant, grid, s);
    else
        c.d == 128 ? write_as<float, 128>(a, quant, grid, s) : write_as<float, 64>(a, quant, grid, s);
    return cudaGetLastError();
}

cudaError_t launch_cache_read(const Cache& c, int row0, int rows, void* k, void* v, int dtype, cudaStream_t s)
{
    ReadArgs a;
    a.wide = ((reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v)) & 31) == 0;
    a.heads = c.B * c.Hkv;
    a.cap = c.cap;
    a.row0 = row0;
    a.rows = rows;
    a.k = c.k;
    a.v = c.v;
    a.k_exp = c.k_exp;
    a.v_exp = c.v_exp;
    a.k_out = k;
    a.v_out = v;
    const bool quant = c.dtype != dtype;
    const dim3 grid = cache_grid((long long)c.B * c.Hkv, rows, quant || dtype == 1 ? c.d / (quant ? 16 : 8) : c.d / 4, kUnrollRead);
    if (dtype == 1)
        c.d == 128 ? read_as<__nv_bfloat16, 128>(a, quant, grid, s) : read_as<__nv_bfloat16, 64>(a, quant, grid, s);
    else
        c.d == 128 ? read_as<float, 128>(a, quant, grid, s) : read_as<float, 64>(a, quant, grid, s);
    return cudaGetLastError();
}

}  // namespace ra
