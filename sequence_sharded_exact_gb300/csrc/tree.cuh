// tree.cuh -- attention of a few new (drafted) tokens per sequence over a key/value cache: what the
// kernels share.
//
// Sequence b has a prefix of len = lens[b] cached rows, which every query sees, and cnt = ntok[b] <= T
// drafted tokens whose keys and values are the rows len .. len + cnt - 1; token t sees drafted token j
// where mask[b][t][j] (without a mask: j <= t).  For query row x of head h (kv head h / G):
//   s_j = x . k_j / sqrt(d),  out = sum_j exp(s_j - m) v_j / l,  l = sum_j exp(s_j - m),  lse = m + ln l
// over the rows j it sees.  A row that sees none, and a token t >= cnt, gets out = 0, lse = -infinity,
// as a ring step's rows do; so (out, lse) in float32 folds into other parts of a sequence that is
// sharded over devices (ring_attn_lse_merge).  A row that a query does not see takes no part in its
// result whatever it holds; rows from len + cnt on are not used at all.
//
// What bounds it: each cached row is needed once, by the G * T query rows of its kv head together, so
// the least traffic is the live part of the cache, and the operations are 4 d G T per row and kv head:
// below about 128 query rows per kv head it is the memory's time, above that the products'.  A long
// cache and few sequences leave only B * Hkv independent pieces, far fewer than SMs, so the token
// axis is split: the tiles (128 or 32 cached rows of one kv head against one tile of query rows) of all
// sequences form one list, and CTA c of n takes the tiles [c total / n, (c + 1) total / n) whatever
// sequences they belong to.  Every SM gets the same work to within one tile for any mix of lengths,
// and the lengths stay on the device (a captured graph replays with new ones).  A CTA writes an item (one
// kv head's tile of query rows) that it holds whole; of one that it shares it writes the partial
// (m, l, unnormalised output) to the workspace, in slot 0 if the item is the first it works on and
// slot 1 otherwise, and a second launch joins the partials in CTA order: the result does not vary
// from run to run.  That launch takes the items that go over a border between CTAs from a list that
// the first one leaves, whatever the batch, and also writes the rows of sequences that have no tokens.
//
// Through a window (kWin): token t, at position p_t in [len, len + T), sees the prefix's rows j < sinks and those with
// p_t - j < window; without a mask the same holds of the step's rows up to its own, so that a prompt may go in by
// chunks of any size.  The rows between the sinks and the first one that a token's window reaches are left out of the list,
// by whole tiles: list tile x is the cache's tile x among the sinks', and gap tiles further on behind them.  Rows that some
// tokens see and others do not are treated as drafted tokens' are.
#pragma once

#include <math.h>

#include "ra_internal.h"

namespace ra {

constexpr int kTreeTile = 128;       // cached rows per tile of the work list on the tensor cores
constexpr int kTreeSimtTile = 32;    // and on the CUDA cores
constexpr int kTreeMaxCtas = 640;    // most CTAs of the first launch on the CUDA cores (bounds the workspace)
constexpr int kTreeMaxTcCtas = 160;  // and on the tensor cores (one per SM)

struct TreeArgs {
    int B, H, Hkv, G, T, R;  // R = G * T query rows per kv head, row x: head x / T of the group, token x % T
    int cap, rt, nrt;        // cache rows; query rows per row tile; row tiles per kv head
    int tile;                // cached rows per tile
    int ctas;                // CTAs of the first launch
    int mask_batched, bf16_out;
    const int *lens, *ntok;
    const uint8_t* mask;
    const void *q, *k, *v;
    const uint8_t *k_exp, *v_exp;
    void* out;
    float* lse;
    float* part_ml;  // [ctas][2][rt][4]: m (log2 units), l, the output's normaliser, 0
    float* part_o;   // [ctas][2][d][rt]: a warp that holds consecutive rows writes whole lines
    int4* border;    // [ctas]: the item that starts in this CTA and goes on in the next: sequence (-1: none),
                     // head * nrt + row tile, its last CTA, its slot here + 2 * its sequence's drafted tokens
    unsigned int* status;
    float scale_log2;  // log2(e) / sqrt(d)
    int window, sinks; // kWin
    const int* pos;    // kWin: [B][T] positions of the tokens, or null: lens + t
    int whole;         // kWin: CTA c takes item c alone; no item is shared and there is no second launch
};

struct TreeSeq {
    int len, cnt, end;  // prefix rows, drafted tokens, rows in all (0: no queries)
    bool bad;           // a length outside its range was clamped
};
// Through a window: the prefix's rows [lo, len) are in reach, those of [all, len) and [0, sinks) seen by every token; of the
// list's tiles the first `front` are the cache's, the others lie `gap` tiles further on.
struct TreeWinSeq : TreeSeq {
    int lo, all, sinks, front, gap;
};

template <bool kWin>
struct TreeSeqOf {
    using type = TreeSeq;
};
template <>
struct TreeSeqOf<true> {
    using type = TreeWinSeq;
};

__device__ __forceinline__ TreeSeq tree_seq(const TreeArgs& a, int b)
{
    TreeSeq s;
    const int len = a.lens[b], cnt = a.ntok ? a.ntok[b] : a.T;
    s.len = len < 0 ? 0 : (len > a.cap ? a.cap : len);
    const int room = a.T < a.cap - s.len ? a.T : a.cap - s.len;
    s.cnt = cnt < 0 ? 0 : (cnt > room ? room : cnt);
    s.bad = s.len != len || s.cnt != cnt;
    s.end = s.cnt ? s.len + s.cnt : 0;
    return s;
}

template <bool kWin>
__device__ __forceinline__ typename TreeSeqOf<kWin>::type tree_sequence(const TreeArgs& a, int b)
{
    if constexpr (!kWin) {
        return tree_seq(a, b);
    } else {
        TreeWinSeq s;
        static_cast<TreeSeq&>(s) = tree_seq(a, b);
        s.lo = s.len - a.window + 1 > 0 ? s.len - a.window + 1 : 0;
        s.all = s.len + a.T - a.window > 0 ? s.len + a.T - a.window : 0;
        s.sinks = a.sinks < s.len ? a.sinks : s.len;
        s.front = (s.sinks + a.tile - 1) / a.tile;
        s.gap = s.lo / a.tile > s.front ? s.lo / a.tile - s.front : 0;
        return s;
    }
}

// Row of the cache that row x of the list is.
__device__ __forceinline__ int tree_row(const TreeSeq&, int x, int) { return x; }
__device__ __forceinline__ int tree_row(const TreeWinSeq& s, int x, int tile) { return x >= s.front * tile ? x + s.gap * tile : x; }
__device__ __forceinline__ int tree_list_row(const TreeSeq&, int key, int) { return key; }  // and back
__device__ __forceinline__ int tree_list_row(const TreeWinSeq& s, int key, int tile) { return key >= s.front * tile ? key - s.gap * tile : key; }
__device__ __forceinline__ int tree_sinks(const TreeSeq&) { return 0; }
__device__ __forceinline__ int tree_sinks(const TreeWinSeq& s) { return s.sinks; }
// The sequence's end in the list.
__device__ __forceinline__ int tree_list_end(const TreeSeq& s, int) { return s.end; }
__device__ __forceinline__ int tree_list_end(const TreeWinSeq& s, int tile) { return s.end ? s.end - s.gap * tile : 0; }
// Rows that no query sees, and rows that some may not see (the former among them).
__device__ __forceinline__ bool tree_dead(const TreeSeq& s, int key) { return key >= s.end; }
__device__ __forceinline__ bool tree_dead(const TreeWinSeq& s, int key) { return key >= s.end || (key >= s.sinks && key < s.lo); }
__device__ __forceinline__ bool tree_partly(const TreeSeq& s, int key) { return key >= s.len; }
__device__ __forceinline__ bool tree_partly(const TreeWinSeq& s, int key) { return key >= s.len || (key >= s.sinks && key < s.all); }
// The first of those that some may not see and some see.
__device__ __forceinline__ int tree_first_partly(const TreeSeq& s) { return s.len; }
__device__ __forceinline__ int tree_first_partly(const TreeWinSeq& s) { return s.lo < s.sinks ? s.sinks : s.lo; }
// Does one of the rows [k0, k0 + n) belong to them?
__device__ __forceinline__ bool tree_masked(const TreeSeq& s, int k0, int n) { return k0 + n > s.len; }
__device__ __forceinline__ bool tree_masked(const TreeWinSeq& s, int k0, int n) { return k0 + n > s.len || (k0 < s.all && k0 + n > s.sinks); }

// First row of the prefix in the window of token t of sequence b (below 0: all are).
__device__ __forceinline__ int tree_reach(const TreeArgs& a, const TreeSeq& s, int b, int t)
{
    int p = s.len + t;
    if (a.pos) {
        p = a.pos[(long long)b * a.T + t];
        p = p < s.len ? s.len : (p > s.len + a.T - 1 ? s.len + a.T - 1 : p);
    }
    return p - a.window + 1;
}

__device__ __forceinline__ int tree_tiles(const TreeArgs& a, const TreeWinSeq& s)
{
    return s.end ? (s.end + a.tile - 1) / a.tile - s.gap : 0;
}
__device__ __forceinline__ int tree_tiles(const TreeArgs& a, const TreeSeq& s)
{
    return a.tile == kTreeTile ? (s.end + kTreeTile - 1) / kTreeTile : (s.end + kTreeSimtTile - 1) / kTreeSimtTile;
}

// First tile of CTA c, and the CTA that holds tile x.  With fewer tiles than CTAs the first `total` CTAs take
// one each, so that every CTA between an item's first and last has written a partial of it.
__device__ __forceinline__ long long tree_first(const TreeArgs& a, long long total, int c)
{
    const long long n = total < a.ctas ? total : a.ctas;
    return c < n ? total * c / n : total;
}
__device__ __forceinline__ int tree_owner(const TreeArgs& a, long long total, long long x)
{
    const long long n = total < a.ctas ? total : a.ctas;
    return (int)(((x + 1) * n - 1) / total);
}

// A CTA's walk over its items: (b, kv head g, row tile r) and the tiles [t0, t1) of it.
template <bool kWin>
struct TreeWalkOf {
    long long left;  // tiles still to do, the current item's included
    long long total; // of all CTAs
    int b, g, r, t0, t1, nt;
    bool first;
    typename TreeSeqOf<kWin>::type s;

    __device__ __forceinline__ bool whole() const { return t0 == 0 && t1 == nt; }
    // Starts here and goes on in the next CTA.
    __device__ __forceinline__ bool goes_on() const { return t0 == 0 && t1 < nt; }
    // What one thread writes for the second launch about the item.  The tiles that are left lie in the CTAs behind.
    __device__ __forceinline__ int4 border(const TreeArgs& a, int cta) const
    {
        const long long end = tree_first(a, total, cta + 1) + (nt - t1);
        return make_int4(b, g * a.nrt + r, tree_owner(a, total, end - 1), (first ? 0 : 1) + 2 * s.cnt);
    }

    __device__ __forceinline__ void take()
    {
        const long long n = nt - t0;
        t1 = n < left ? nt : t0 + (int)left;
    }
    // One warp calls these.  The walk of CTA `cta`; false if it has no tiles.
    __device__ __forceinline__ bool begin(const TreeArgs& a, int cta)
    {
        if constexpr (kWin) {
            if (a.whole) {
                const int per = a.Hkv * a.nrt, item = cta % per;
                b = cta / per;
                g = item / a.nrt;
                r = item % a.nrt;
                s = tree_sequence<kWin>(a, b);
                if (s.bad && threadIdx.x == 0) atomicOr(a.status, kStatusRange);
                t0 = 0;
                total = left = t1 = nt = tree_tiles(a, s);
                first = true;
                return nt > 0;
            }
        }
        const int mine = lengths(a);
        const long long at = tree_first(a, total, cta);
        left = tree_first(a, total, cta + 1) - at;
        first = true;
        if (left <= 0) return false;
        locate(a, at, mine);
        take();
        return true;
    }
    // All tiles, and this lane's sequence's among the first 32 (the usual batch has no more: its lengths are read once).
    __device__ __forceinline__ int lengths(const TreeArgs& a)
    {
        const int lane = threadIdx.x & 31;
        const int mine = lane < a.B ? tree_tiles(a, tree_sequence<kWin>(a, lane)) : 0;
        long long all = 0;
        for (int b0 = 0; b0 < a.B; b0 += 32) {
            int n = b0 == 0 ? mine : b0 + lane < a.B ? tree_tiles(a, tree_sequence<kWin>(a, b0 + lane)) : 0;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
            all += n;
        }
        total = all * a.Hkv * a.nrt;
        return mine;
    }
    // The item that holds tile `at` of the list, and where in it.
    __device__ __forceinline__ void locate(const TreeArgs& a, long long at, int mine32)
    {
        const int lane = threadIdx.x & 31;
        const long long items = (long long)a.Hkv * a.nrt;
        for (int b0 = 0; b0 < a.B; b0 += 32) {
            const long long mine = (b0 == 0 ? mine32 : b0 + lane < a.B ? tree_tiles(a, tree_sequence<kWin>(a, b0 + lane)) : 0) * items;
            long long upto = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long up = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += up;
            }
            const unsigned past = __ballot_sync(0xffffffffu, upto > at);
            if (past) {
                const int hit = __ffs(past) - 1;
                b = b0 + hit;
                at -= __shfl_sync(0xffffffffu, upto - mine, hit);
                break;
            }
            at -= __shfl_sync(0xffffffffu, upto, 31);
        }
        s = tree_sequence<kWin>(a, b);
        nt = tree_tiles(a, s);
        const int item = (int)(at / nt);
        t0 = (int)(at % nt);
        g = item / a.nrt;
        r = item % a.nrt;
    }
    __device__ __forceinline__ bool next(const TreeArgs& a)
    {
        left -= t1 - t0;
        first = false;
        if (left <= 0) return false;
        t0 = 0;
        if (++r == a.nrt) {
            r = 0;
            if (++g == a.Hkv) {
                g = 0;
                do {
                    s = tree_sequence<kWin>(a, ++b);
                    nt = tree_tiles(a, s);
                } while (nt == 0);  // `left` says that a later sequence has tiles
            }
        }
        take();
        return true;
    }
};
using TreeWalk = TreeWalkOf<false>;

// Zeros and -infinity for the rows of CTA `cta`'s item, whose sequence has no tokens (TreeArgs::whole); all its threads.
template <int D>
__device__ __forceinline__ void tree_clear_item(const TreeArgs& a, int cta)
{
    const int r = cta % a.nrt, rows = a.R - r * a.rt < a.rt ? a.R - r * a.rt : a.rt;
    const long long row0 = (long long)(cta / a.nrt) * a.R + (long long)r * a.rt;  // cta / nrt: b Hkv + g
    for (int e = threadIdx.x; e < rows * (D / 2); e += blockDim.x) {
        if (a.bf16_out)
            static_cast<uint32_t*>(a.out)[row0 * (D / 2) + e] = 0u;
        else
            static_cast<float2*>(a.out)[row0 * (D / 2) + e] = make_float2(0.f, 0.f);
    }
    for (int e = threadIdx.x; e < rows; e += blockDim.x) a.lse[row0 + e] = -INFINITY;
}

// Does query token t see drafted token j (both < cnt)?
template <bool kWin = false>
__device__ __forceinline__ bool tree_sees(const TreeArgs& a, const TreeSeq& s, int b, int t, int j)
{
    if (!a.mask) return j <= t && (!kWin || t - j < a.window || s.len + j < a.sinks);
    return a.mask[((a.mask_batched ? (long long)b * a.T : 0) + t) * a.T + j] != 0;
}

// Query rows of an item: a row tile's, or all of a kv head's where they are fewer.
__host__ __device__ inline int tree_item_rows(const TreeArgs& a) { return a.R < a.rt ? a.R : a.rt; }

__host__ __device__ inline size_t tree_align(size_t x) { return (x + 255) & ~size_t(255); }

// Joins the partials of shared items and writes the rows that see nothing (tree_join.cu).
cudaError_t launch_tree_join(const TreeArgs& a, int d, cudaStream_t s);
// CUDA-core path: float32 queries (tree_simt.cu).  Query rows per row tile for R query rows per kv head.
int tree_simt_rows(int R);
constexpr int kTreeSimtCtasPerSm = 4;
cudaError_t launch_tree_simt(const TreeArgs& a, int d, int cache_dtype, cudaStream_t s);

// bf16 queries, up to kTreeMmaRows query rows per kv head: one row tile; an e4m3 cache (tree_mma.cu) or a bf16 one
// (tree_mma_bf16.cu).
constexpr int kTreeMmaRows = 8, kTreeMmaE4m3Rows = 16;
// 9 to 16 rows (e4m3): CTAs of four warps per SM; at d = 128 a third would leave too few registers (one sequence of 131072
// rows, 87 us, took a tenth longer).
__host__ __device__ constexpr int tree_mma16_ctas_per_sm(int d) { return d == 128 ? 2 : 3; }
// With many items (sequences times kv heads) per SM their ends cost more than the join of more CTAs' partials, so there are
// more CTAs.  e4m3: four of four warps per SM in place of two of eight; bf16: three of four warps in place of two.
// 256 sequences of 200 rows, 8 kv heads: 43 us in place of 57 (e4m3), 48 in place of 60 (bf16); 64 of 1000 rows with
// three CTAs: 54 in place of 51 (bf16).
constexpr int kTreeMmaManyItems = 6;  // per SM
constexpr int kTreeMmaWarps = 16;     // e4m3: per SM
constexpr int kTreeMaxMmaCtas = 640;
cudaError_t launch_tree_mma(const TreeArgs& a, int d, int warps, cudaStream_t s);  // 4 or 8 warps per CTA
cudaError_t launch_tree_mma_bf16(const TreeArgs& a, int d, cudaStream_t s);

// Tensor-core path: bf16 queries, bf16 or e4m3 cache (tree_tc_body.cuh).
cudaError_t launch_tree_tc_d128(const TreeArgs& a, bool e4m3, cudaStream_t s);
cudaError_t launch_tree_tc_d64(const TreeArgs& a, bool e4m3, cudaStream_t s);
cudaError_t launch_tree_window_tc_d128(const TreeArgs& a, bool e4m3, cudaStream_t s);
cudaError_t launch_tree_window_tc_d64(const TreeArgs& a, bool e4m3, cudaStream_t s);

}  // namespace ra
