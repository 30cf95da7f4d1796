// kda_tree.cuh -- what the tree attention kernels share: the arguments, the
// drafted tree's ancestor masks, and the split of the work over the CTAs.
//
// Work split.  An item is one (sequence, cache head); its keys, the L rows of the
// context and after them the Ts drafted nodes, come in ceil((L + Ts) / KT) tiles
// of KT.  An item costs its tiles and LEAD more, for what its start and end take.
// Laid end to end in (sequence, head, tile) order, the costs are cut into equal
// ranges, one per group of CTAs, whatever the lengths are; the
// lengths stay on the device and every CTA finds its own range from them.  The
// CTAs of a group have one row tile (up to RT of the item's Ts G query rows)
// each and walk the same keys side by side, so that all but one find them in
// L2.  A range covers at most one item that began in an earlier group and one
// that goes on in the next: those pieces go to the CTA's two workspace slots as
// (unnormalised o, m, l), and a second launch joins them.  Every other item is
// finished in its CTAs.
#pragma once

#include "kda_internal.cuh"

namespace kda {

constexpr int kTreeMaxNodes = 64;     // one bit per node in a 64-bit mask
// The tensor-core kernel's KT and LEAD.  LEAD 0, 4, 8, 12 and 20, us: 32 ragged
// contexts of 0 to 16,384 rows, 16 nodes, 351, 245, 206, 192 and 193 (cut without
// it, a range of short sequences is the last to end); 4 x 32,768 rows 113, 111,
// 106, 103 and 104; 64 x 4,096 rows, one token, 179, 177, 178, 179 and 183.
constexpr int kTcKeys = 128;
constexpr int kTcLead = 12;

struct TreeArgs {
    const void *q, *k, *v;
    const int32_t* parent;            // [N, Ts], or null for a chain
    const void *k_cache, *v_cache;
    const int32_t *page_table, *lengths;
    int32_t N, Ts, Hq, Hkv, G, R;     // G = Hq / Hkv, R = Ts G rows per (sequence, cache head)
    int32_t num_pages, page_size, max_pages;
    long long page_stride;            // elements from one page to the next
    float scale_log2;                 // scale * log2(e)
    void* o;
    int32_t* status;                  // workspace words (kWsTimeoutWord is used)
    float* part;                      // 2 slots per CTA: [RT][d] o, [RT] m, [RT] l
    int32_t box, tile_pages, tile_rows;   // tensor-core kernel: rows per TMA box (0: none), and
                                      // a tile's keys as whole pages and rows
    bool starve;                      // test of the waits that give up (tensor-core kernel)
    int32_t groups, row_tiles;        // CTA b: group b / row_tiles, row tile b % row_tiles
    int32_t tile_log;                 // KT = 0 below: log2 of a tile's keys
};

__device__ __forceinline__ int tree_context(const TreeArgs& a, int n)
{
    const long long most = (long long)a.max_pages * a.page_size;
    const int len = __ldg(a.lengths + n);
    return len < 0 ? 0 : (int)(len < most ? len : most);
}

// anc[t]: bit j set when node j is t or an ancestor of t; 0 when t is unused
// (its chain of parents does not end at the context).  One warp, two nodes per
// lane; six rounds of pointer doubling cover 64 nodes.
__device__ __forceinline__ void tree_masks(const int32_t* parent, int Ts, int lane,
                                           unsigned long long* anc, int32_t* up)
{
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int t = lane + 32 * i;
        int p = -2;
        if (t < Ts) {
            p = parent ? __ldg(parent + t) : t - 1;
            if (p < -1 || p >= t) p = -2;
        }
        anc[t] = 1ull << t;
        up[t] = p;
    }
    __syncwarp();
    for (int round = 0; round < 6; ++round) {
        unsigned long long m[2];
        int32_t u[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int t = lane + 32 * i, p = up[t];
            m[i] = anc[t] | (p >= 0 ? anc[p] : 0ull);
            u[i] = p >= 0 ? up[p] : p;
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            anc[lane + 32 * i] = m[i];
            up[lane + 32 * i] = u[i];
        }
        __syncwarp();
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
        if (up[lane + 32 * i] != -1) anc[lane + 32 * i] = 0ull;
    __syncwarp();
}

// Where a group's range begins in the flattened order, in units of a tile's cost.
struct TreeSpot {
    long long total;        // of the whole launch
    long long per, more;    // each group has `per` units, the first `more` one more
    long long start;        // where sequence n begins
    int n;
};

// Tiles of KT keys (0: of 2^tile_log) of a context and the nodes.
template <int KT>
__device__ __forceinline__ int tree_tiles_of(const TreeArgs& a, int ctx)
{
    if constexpr (KT == 0) return (ctx + a.Ts + (1 << a.tile_log) - 1) >> a.tile_log;
    else return (ctx + a.Ts + KT - 1) / KT;
}
template <int KT>
__device__ __forceinline__ int tree_tiles(const TreeArgs& a, int n)
{
    return tree_tiles_of<KT>(a, tree_context(a, n));
}

template <int KT, int LEAD>
__device__ __forceinline__ long long tree_cost(const TreeArgs& a, int n)
{
    return (long long)(tree_tiles<KT>(a, n) + LEAD) * a.Hkv;
}

// Where group c's range begins.
__device__ __forceinline__ long long tree_begin(const TreeSpot& sp, int c)
{
    return sp.per * c + (c < sp.more ? c : sp.more);
}

// The sequence that group c's range begins in (c < groups).  All
// THREADS threads of the block call it; `sh` is shared scratch of THREADS / 32 +
// 2 words.  With up to THREADS sequences the lengths are read once.
template <int THREADS, int KT, int LEAD>
__device__ TreeSpot tree_locate(const TreeArgs& a, int c, long long* sh)
{
    constexpr int W = THREADS / 32;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    TreeSpot r;
    long long mine = 0;                             // the first THREADS sequences' costs
    if (tid < a.N) mine = tree_cost<KT, LEAD>(a, tid);
    long long rest = 0;
    for (int n = tid + THREADS; n < a.N; n += THREADS) rest += tree_cost<KT, LEAD>(a, n);
    if (a.N > THREADS) {
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) rest += __shfl_xor_sync(0xffffffffu, rest, off);
        if (lane == 0) sh[warp] = rest;
        __syncthreads();
        rest = 0;
#pragma unroll 1
        for (int i = 0; i < W; ++i) rest += sh[i];
        __syncthreads();
    }
    long long base = 0, at = 0;
    for (int n0 = 0; n0 < a.N; n0 += THREADS) {
        const int n = n0 + tid;
        const long long w = n0 == 0 ? mine : (n < a.N ? tree_cost<KT, LEAD>(a, n) : 0);
        long long incl = w;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const long long x = __shfl_up_sync(0xffffffffu, incl, off);
            if (lane >= off) incl += x;
        }
        if (lane == 31) sh[warp] = incl;
        __syncthreads();
        // the warps' sums, a lane each (W <= 32), added up the same way
        long long upto = lane < W ? sh[lane] : 0;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const long long x = __shfl_up_sync(0xffffffffu, upto, off);
            if (lane >= off) upto += x;
        }
        const long long chunk = __shfl_sync(0xffffffffu, upto, 31);
        const long long below = __shfl_sync(0xffffffffu, upto, warp ? warp - 1 : 0);
        const long long before = base + (warp ? below : 0);
        if (n0 == 0) {
            r.total = chunk + rest;
            r.per = r.total / a.groups;
            r.more = r.total - r.per * a.groups;
            at = tree_begin(r, c);
        }
        if (at >= before + incl - w && at < before + incl) {
            sh[W] = n;
            sh[W + 1] = before + incl - w;
        }
        base += chunk;
        __syncthreads();
        if (at < base) break;                       // uniform: the block has found it
    }
    r.n = (int)sh[W];
    r.start = sh[W + 1];
    return r;
}

// A stretch of one item's tiles in a group's range, and the walk over them:
// start() takes the first, next() moves on (only the first needs a division).
template <int KT, int LEAD>
struct TreePieces {
    int n, hk, ctx;
    int tiles, t0, t1;      // the item's tiles, and those of this piece
    long long left;         // of the range, from the item's part of it on

    __device__ __forceinline__ void enter(const TreeArgs& a)
    {
        ctx = tree_context(a, n);
        tiles = tree_tiles_of<KT>(a, ctx);
    }
    // The piece of an item of which the first `skip` units lie before the range.
    __device__ __forceinline__ bool cut(long long skip)
    {
        t0 = skip > LEAD ? (int)(skip - LEAD) : 0;
        const long long end = skip + left - LEAD;
        t1 = end < tiles ? (int)end : tiles;
        left -= tiles + LEAD - skip;
        return t1 > t0;
    }

    // False when the range has no tile.
    __device__ __forceinline__ bool start(const TreeArgs& a, const TreeSpot& sp, int group)
    {
        const long long begin = tree_begin(sp, group);
        left = tree_begin(sp, group + 1) - begin;
        if (left <= 0) return false;
        n = sp.n;
        enter(a);
        hk = (int)((begin - sp.start) / (tiles + LEAD));
        // a range that begins in an item's lead and ends there has no tile
        return cut(begin - sp.start - (long long)hk * (tiles + LEAD));
    }
    __device__ __forceinline__ bool next(const TreeArgs& a)
    {
        if (left <= 0) return false;
        if (++hk == a.Hkv) {
            hk = 0;
            ++n;
            enter(a);
        }
        return cut(0);
    }
};

struct TreePlan {
    int rt;                 // rows per row tile
    int row_tiles, groups;
    bool tc;
};
// Workspace of a call, enough for either kernel.
size_t tree_workspace_bytes(int32_t Ts, int32_t Hq, int32_t Hkv, int32_t d, kda_dtype_t dtype, int sms);

cudaError_t launch_tree_attention(TreeArgs args, int32_t d, kda_dtype_t dtype, int sms,
                                  cudaStream_t stream);
cudaError_t launch_tree_attention_tc(TreeArgs args, const TreePlan& plan, int32_t d,
                                     cudaStream_t stream);

}  // namespace kda
