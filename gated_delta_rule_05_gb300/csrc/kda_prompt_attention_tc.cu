// kda_prompt_attention_tc.cu -- causal attention over packed prompts on the tensor
// cores (bf16, d = 64 or 128): a persistent CTA per SM, tcgen05 products with TMEM
// accumulators.
//
// An item is two row tiles of 128 query rows (one, in small calls) of a (sequence, cache head); the rows
// of the G heads that share it lie token by token, row r of a tile being head r % G
// of its token r / G (128 / G tokens to a tile), so that a tile spans few positions.
// Per tile of 128 keys and row tile
//     S = Q K^T             (M = 128, N = 128, K = d; Q, K in shared memory)
//     P = 2^(c S - m)       (registers; c = scale log2 e; bf16 back over S, or beside it)
//     O += P V              (M = 128, N = d, K = 128; P in TMEM, V MN-major)
// with a reference m near the running maximum of each row that moves only when a tile
// exceeds it by more than 8: P may reach 2^8, O and l are scaled by 2^(m - m') when m
// moves, and after the first tiles of a row O is left alone.  P is rounded to
// bf16, the type of V, as one product takes one type; l sums the values before
// the rounding.
//
// Roles: four warpgroups of softmax and output, two per row tile with 64 of a tile's
// 128 keys each (their threads of one row exchange its maximum and its sum through
// shared memory); a warp that issues products, one that copies keys and values, one that
// finds the items and copies their queries, one that looks through values (below).
// The row tiles share K and V and alternate on the tensor core: one's softmax runs under
// the other's products.  Tensor memory's 512 columns hold two S, two O and, with d = 64, two P: there
// the next scores are computed while these are worked on (5 prompts of 700 to 2,048
// tokens behind prefixes, 16 heads, 129.5 us without and 121.5 with).
//
// Values that a row of the item does not see must not reach it through 0 * inf: in the
// tiles on the diagonal and at the end of a sequence the fourth warp replaces
// infinities and NaN by 0 before the product and notes their keys; the rows that do
// see such a key add its value to their output at the end.
//
// Items go to the CTAs in order, the sequences with most keys first and of each its
// last rows, one at a time from a counter in the caller's workspace: 12 prompts of 512
// to 12,288 tokens, the longest CTA has 1.001 times the mean's tiles, dealt to and fro 1.07.
// (Taken over all sequences by their length, dealt to and fro, 1.002, but the keys of
// all of them pass through the L2 again and again: 4.05 ms against 3.85.)  Where there are few
// items for a CTA they are dealt to and fro, which saves the clearing of the counter.
//
// Bound by the softmax beside the products: 32 heads on 8, d = 128, one prompt of 65,536
// tokens (8 heads) 5.4 ms, 1.63 PFLOP/s, of 8,192 0.35 ms (1.57), of 2,048 34 us (1.0); 12 of 512
// to 12,288 3.6 ms (1.49).  d = 64, 16 heads on 4, 16,384 tokens 545 us (1.0): half the products for
// as many exponentials.  Steps on the way there, 8 x 2,048 tokens: 445 us with the
// products' loop rolled up (349 without), 291 with the output in a warpgroup of its own (250);
// 8,192 tokens 394 us with 16-byte stores of rows, 372 with 32-byte ones, 363 with rows that go out
// by way of shared memory; a maximum of the tile before instead of the tile's own gains
// nothing.  Items claimed two ahead 156 us, one 129 (those 5 prompts).
//
// Against the kernel for everything else (fp16 products by mma.sync), 32 heads on 8, d = 128, us:
// one prompt of 1 token 8.3 (6.1), 16 8.8 (7.4), 128 8.9 (13.8), 512 13.2 (33.5), 8,192 353 (2,863);
// d = 64, 16 on 4, 128 tokens 7.5 (11.2), 4,096 47 (204).  The shortest are not
// given to that one: a prompt's results would depend on how it is cut.
//
// Every wait has a limit; one that gives up sets the workspace's timeout word and stops
// its CTA: the warps that start copies and products end at their next wait and wait for
// what they have started (again with a limit), and the softmax runs on without
// waiting, over whatever is there, and gives its rows a sum of NaN.  The environment
// variable KDA_TEST_STARVE_CONSUMERS, for the test of that path only, has the copying
// warps exit at once.
#include <cudaTypedefs.h>
#include <stdio.h>

#include "kda_prompt.cuh"
#include "kda_sm100.cuh"

namespace kda {

// The driver's tensor-map encoder (kda_prefill_tc.cu).
PFN_cuTensorMapEncodeTiled_v12000 tc_encode_fn();

namespace {

using namespace sm100;

constexpr int KT = 128;                    // keys per tile
constexpr int kThreads = 640;              // 16 softmax warps, 4 others
constexpr int kMmaWarp = 16, kKvWarp = 17, kQWarp = 18;
// 640 threads are launched with 96 registers: 512 x 104 + 128 x 64 = 640 x 96
constexpr int kMore = 104, kFewer = 64;
constexpr int kMaxTable = 256;             // sequences whose sizes are held in shared memory
constexpr int kItems = 4;                  // items that are known ahead
constexpr int kEdges = 4;                  // an item's tiles on its edge: 256 rows begin within one and see up to 255
                                           // keys more, 3 tiles
constexpr int kItemReaders = 16 + 3;       // warps

template <int D>
struct Shape {
    static constexpr int kQBytes = 2 * 128 * D * 2;
    static constexpr int kSlotBytes = KT * D * 2;
    static constexpr int kSlots = D == 128 ? 4 : 8;
    static constexpr int kStageBytes = 1024;       // of a warp, for its rows on their way out
    static constexpr size_t kBytes = 1024 + kQBytes + (size_t)kSlots * kSlotBytes + 16 * kStageBytes;
    static constexpr int kO = 256;         // TMEM column of the outputs; the scores are at 0 and 128
    // Whether P has columns of its own and a row tile's next scores may come once the last
    // have been read.
    static constexpr bool kOwnP = D == 64;
    static constexpr int kP = kOwnP ? kO + 2 * D : 0;      // P of row tile 0
    static constexpr int kPTile = kOwnP ? 64 : 128, kPHalf = kPTile / 2;
};

struct Seq {
    int q0, lq, k0, lk;
};

// An item: its sequence, cache head and row tiles.
struct alignas(16) Item {
    int q0, lq, k0, lk;
    int hk;                                // -1: there are no more
    int t0;                                // the first row tile's first token
    int cnt[2];                            // key tiles of the row tiles
    int all;                               // keys that every row of the item sees
    int pad[3];
    __device__ __forceinline__ int tiles() const { return max(cnt[0], cnt[1]); }
    // Whether some row of the item does not see all of key tile j.
    __device__ __forceinline__ bool edge(int j) const { return (j + 1) * KT > all; }
};

struct Shared {
    uint64_t kv_full[8], kv_land[8], kv_empty[8], q_full, q_empty, kv_started, done;
    uint64_t s_full[2], s_read[2], p_full[2], pv_done[2], o_empty[2], item_full[kItems], item_empty[kItems];
    Item item[kItems];
    uint32_t tmem;
    int dead;
    int total;                             // pairs of row tiles (see Plan::span) of all sequences, for one cache head
    int per;                               // sequences of a table entry
    float top[2][2][2][128];               // of a row tile and half of a tile's keys, by row; by turns
    float sum[2][2][128];
    // Keys with an infinity or NaN in v, of the tiles on an item's edge; they live as long as the item
    // (a row tile may look at them while the other is at the next items), and whether there are any.
    alignas(16) uint32_t bad[kItems][kEdges][4];
    int noted[kItems];
    int sums[kThreads / 32];
    int before[kMaxTable];                 // row tile pairs before a table entry
    int pairs[kMaxTable];                  // (these only where an entry is one sequence)
    alignas(16) Seq seq[kMaxTable];
};

// Waits for a phase of a barrier, for about two seconds at most and (STOP) no longer
// than until some wait of this CTA has given up; false then.  Written short: the roles
// run side by side and have to share the SM's instruction cache.
template <bool STOP>
__device__ __forceinline__ bool wait_for(Shared& sh, uint64_t* bar, uint32_t parity, int32_t* status)
{
    if (mbar_try_wait(bar, parity)) return true;
    const long long t0 = clock64();
#pragma unroll 1
    while (!mbar_try_wait(bar, parity)) {
        if (STOP && *reinterpret_cast<volatile int*>(&sh.dead)) return false;
        if (clock64() - t0 > (1ll << 32)) {
            *reinterpret_cast<volatile int*>(&sh.dead) = 1;
            atomicOr(status, 2);
            return false;
        }
    }
    return true;
}
__device__ __forceinline__ bool wait_lane(Shared& sh, uint64_t* bar, uint32_t parity, int32_t* status)
{
    return wait_for<true>(sh, bar, parity, status);
}
// The same for a warp, which goes on as one or stops as one.
__device__ __forceinline__ bool wait(Shared& sh, uint64_t* bar, uint32_t parity, int32_t* status)
{
    return __all_sync(0xffffffffu, wait_for<true>(sh, bar, parity, status));
}
// The same, of a barrier of the items, which are handed on when a wait has given up too.
__device__ __forceinline__ bool wait_item(Shared& sh, uint64_t* bar, uint32_t parity, int32_t* status)
{
    return __all_sync(0xffffffffu, wait_for<false>(sh, bar, parity, status));
}
// Waits for a copy in flight after some wait has given up.
__device__ __noinline__ void settle(uint64_t* bar, uint32_t parity)
{
    const long long t0 = clock64();
#pragma unroll 1
    while (!mbar_try_wait(bar, parity) && clock64() - t0 < (1ll << 24)) {}
}

// One box of rows [token][head][d]: 64 columns.
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int32_t x, int32_t h, int32_t row,
                                            uint64_t* bar)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(h), "r"(row), "r"(smem_u32(bar))
        : "memory");
}
__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float max3(float a, uint32_t b, uint32_t c)
{
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(__uint_as_float(b)), "f"(__uint_as_float(c)));
    return r;
}
// Pairs of fp32 for the two-wide FMA and add.
__device__ __forceinline__ uint64_t pack2u(uint32_t a, uint32_t b)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint64_t pack2(float a, float b) { return pack2u(__float_as_uint(a), __float_as_uint(b)); }
__device__ __forceinline__ void unpack2(uint64_t x, float& a, float& b)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
template <int N>
__device__ __forceinline__ void more_registers()
{
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void fewer_registers()
{
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// ------------------------------------------------------------------ the items
struct Plan {
    int tok;                               // tokens of a row tile
    int rows;                              // rows of a row tile that are used
    int span;                              // tokens of an item: two row tiles, or one where there are few
};

__device__ __forceinline__ int pairs_of(int lq, const Plan& p) { return (lq + p.span - 1) / p.span; }

// The x-th item: sequence by sequence, of a sequence its last rows, the longest work,
// first, and of those every head.  (Head by head takes the same time at 65,536 keys, 268 MB
// of keys and values.)  A whole warp calls it.
template <int D>
__device__ __noinline__ Item item_at(const Shared& sh, const PromptArgs& a, const Plan& p, long long x)
{
    const int lane = threadIdx.x & 31;
    Item it = {};
    int y = (int)(x / a.Hkv);
    const int per = sh.per, entries = (a.N + per - 1) / per;
    int lo = 0, hi = entries;              // the last entry with before <= y
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (sh.before[mid] <= y) lo = mid;
        else hi = mid;
    }
    x -= (long long)sh.before[lo] * a.Hkv; // from the entry's first item
    Seq s = {0, 0, 0, 0};
    int pairs = 0;
    if (per == 1) {
        s = sh.seq[lo];
        pairs = sh.pairs[lo];
    } else {
        // through the entry's sequences, 32 at a time
        for (int n0 = lo * per;; n0 += 32) {
            const int n = n0 + lane;
            PromptSeq ps = {0, 0, 0, 0};
            if (n < a.N) ps = prompt_seq(a, n);
            const int w = pairs_of(ps.lq, p);
            int incl = w;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int z = __shfl_up_sync(0xffffffffu, incl, off);
                if (lane >= off) incl += z;
            }
            const uint32_t past = __ballot_sync(0xffffffffu, x < (long long)incl * a.Hkv);
            if (past || n0 + 32 >= a.N) {
                const int src = past ? __ffs(past) - 1 : 31;
                x -= (long long)__shfl_sync(0xffffffffu, incl - w, src) * a.Hkv;
                s.q0 = __shfl_sync(0xffffffffu, ps.q0, src);
                s.lq = __shfl_sync(0xffffffffu, ps.lq, src);
                s.k0 = __shfl_sync(0xffffffffu, ps.k0, src);
                s.lk = __shfl_sync(0xffffffffu, ps.lk, src);
                break;
            }
            x -= (long long)__shfl_sync(0xffffffffu, incl, 31) * a.Hkv;
        }
        pairs = pairs_of(s.lq, p);
    }
    // (offsets that give rows twice may add up to anything)
    if (x < 0 || x >= (long long)pairs * a.Hkv) return it;
    y = (int)(x / a.Hkv);
    it.hk = (int)(x - (long long)y * a.Hkv);
    it.q0 = s.q0;
    it.lq = s.lq;
    it.k0 = s.k0;
    it.lk = s.lk;
    it.t0 = (pairs - 1 - y) * p.span;
    const int off = s.lk - s.lq;
    it.all = min(max(it.t0 + off + 1, 0), s.lk);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int end = min(it.t0 + (i + 1) * p.tok, s.lq);        // one past the row tile's last token
        const int most = i * p.tok < p.span && it.t0 + i * p.tok < s.lq ? min(max(end + off, 0), s.lk) : 0;
        it.cnt[i] = (most + KT - 1) / KT;
    }
    return it;
}

// A warp's way through this CTA's items, which the query warp finds out ahead of the
// others.
struct Items {
    int n = 0;
    // The next one; null: there is none.
    __device__ __forceinline__ const Item* next(Shared& sh, int32_t* status)
    {
        const Item* it = &sh.item[n % kItems];
        if (!wait_item(sh, &sh.item_full[n % kItems], (uint32_t)(n / kItems) & 1, status)) return nullptr;
        return it->hk < 0 ? nullptr : it;
    }
    // Has been read.
    __device__ __forceinline__ void release(Shared& sh, int lane)
    {
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.item_empty[n % kItems]);
        ++n;
    }
};

// Sizes of the sequences in shared memory, those with most keys first (up to
// kMaxTable); all threads call it.
__device__ void build_table(Shared& sh, const PromptArgs& a, const Plan& p)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (a.N + kMaxTable - 1) / kMaxTable, entries = (a.N + per - 1) / per;
    if (per == 1) {
#pragma unroll 1
        for (int n = tid; n < a.N; n += kThreads) {
            const PromptSeq s = prompt_seq(a, n);
            sh.seq[n] = {s.q0, s.lq, s.k0, s.lk};
            sh.pairs[n] = pairs_of(s.lq, p);
        }
        __syncthreads();
        if (a.N > 1) {
            Seq mine = {0, 0, 0, 0};
            int rank = 0, pairs = 0;
            if (tid < a.N) {
                mine = sh.seq[tid];
                pairs = sh.pairs[tid];
#pragma unroll 1
                for (int m = 0; m < a.N; ++m) {
                    const int lk = sh.seq[m].lk;
                    rank += lk > mine.lk || (lk == mine.lk && m < tid);
                }
            }
            __syncthreads();
            if (tid < a.N) {
                sh.seq[rank] = mine;
                sh.pairs[rank] = pairs;
            }
            __syncthreads();
        }
    }
    int base = 0;
#pragma unroll 1
    for (int e0 = 0; e0 < entries; e0 += kThreads) {
        const int e = e0 + tid;
        int w = 0;
        if (e < entries) {
            if (per == 1) {
                w = sh.pairs[e];
            } else {
#pragma unroll 1
                for (int n = e * per; n < min((e + 1) * per, a.N); ++n) {
                    int first, count;
                    prompt_rows(a.cu_q, n, a.T, first, count);
                    w += pairs_of(count, p);
                }
            }
        }
        int incl = w;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int z = __shfl_up_sync(0xffffffffu, incl, off);
            if (lane >= off) incl += z;
        }
        if (lane == 31) sh.sums[warp] = incl;
        __syncthreads();
        int all = 0, below = 0;
#pragma unroll 1
        for (int i = 0; i < kThreads / 32; ++i) {
            if (i < warp) below += sh.sums[i];
            all += sh.sums[i];
        }
        incl += base + below;
        if (e < entries) sh.before[e] = incl - w;
        base += all;
        __syncthreads();
    }
    if (tid == 0) {
        sh.total = base;
        sh.per = per;
    }
}

// ---------------------------------------------------------------- the copies
// The entries of an item are K_0 V_0 K_1 V_1 ...  A tile of values on an item's
// edge goes to the scanning warp first.
template <int D>
__device__ void kv_role(Shared& sh, const PromptArgs& a, const CUtensorMap* map_k, const CUtensorMap* map_v, uint32_t slots,
                        int lane)
{
    using Sh = Shape<D>;
    int slot = 0;
    uint32_t turn = 0, land_turn = 0, landed = 0, used = 0;        // bits by slot
    bool ok = !a.starve;
    Items items;
    for (const Item* at; (at = items.next(sh, a.status)); items.release(sh, lane)) {
        const Item it = *at;
        const int entries = ok ? 2 * it.tiles() : 0;
#pragma unroll 1
        for (int e = 0; e < entries; ++e) {
            if (((used >> slot) & 1) && !wait(sh, &sh.kv_empty[slot], (turn ^ 1) & 1, a.status)) {
                ok = false;
                break;
            }
            const int j = e >> 1;
            const bool scan = (e & 1) && it.edge(j);
            uint64_t* bar = scan ? &sh.kv_land[slot] : &sh.kv_full[slot];
            if (lane == 0) {
                mbar_arrive_expect_tx(bar, Sh::kSlotBytes);
#pragma unroll
                for (int h = 0; h < D / 64; ++h)
                    tma_load_3d(slots + (uint32_t)slot * Sh::kSlotBytes + h * (KT * 128), (e & 1) ? map_v : map_k, h * 64,
                                it.hk, it.k0 + j * KT, bar);
            }
            __syncwarp();
            used |= 1u << slot;
            landed = (landed & ~(1u << slot)) | ((uint32_t)scan << slot);
            if (scan) land_turn ^= 1u << slot;
            if (++slot == Sh::kSlots) {
                slot = 0;
                turn ^= 1;
            }
        }
        if (lane == 0) mbar_arrive(&sh.kv_started);
    }
    // After a wait that gave up nobody has waited for the last copies in flight.
    if (*reinterpret_cast<volatile int*>(&sh.dead)) {
#pragma unroll 1
        for (int s = 0; s < Sh::kSlots; ++s) {
            if (!((used >> s) & 1)) continue;
            // the phase of the slot's last copy
            if ((landed >> s) & 1) settle(&sh.kv_land[s], ((land_turn >> s) & 1) ^ 1);
            else settle(&sh.kv_full[s], s < slot ? turn & 1 : (turn ^ 1) & 1);
        }
    }
}

// Finds this CTA's items and copies their queries.  An item is claimed when the copies of
// the keys and values of the one before have been started: early enough for its own to
// follow those, and no earlier, so that the CTAs end together.
template <int D>
__device__ void q_role(Shared& sh, const PromptArgs& a, const Plan& p, const CUtensorMap* map_q, uint32_t q_smem, int lane)
{
    int count = 0;                                 // items with queries
    bool ok = !a.starve;
    const long long total = (long long)sh.total * a.Hkv;
    long long x = blockIdx.x;
#pragma unroll 1
    for (int n = 0;; ++n) {
        const int at = n % kItems;
        Item it = {};
        if (x < total) it = item_at<D>(sh, a, p, x);
        else it.hk = -1;
        if (n >= kItems && !wait_item(sh, &sh.item_empty[at], (uint32_t)(n / kItems - 1) & 1, a.status)) break;
        if (lane == 0) {
            sh.item[at] = it;
            mbar_arrive(&sh.item_full[at]);
        }
        __syncwarp();
        if (it.hk < 0) break;
        if (it.tiles() > 0 && ok && (count == 0 || (ok = wait(sh, &sh.q_empty, (uint32_t)(count - 1) & 1, a.status)))) {
            if (lane == 0) {
                const int nt = it.cnt[1] > 0 ? 2 : 1;
                mbar_arrive_expect_tx(&sh.q_full, (uint32_t)(nt * p.rows * D * 2));
                for (int i = 0; i < nt; ++i)
#pragma unroll
                    for (int h = 0; h < D / 64; ++h)
                        tma_load_3d(q_smem + (uint32_t)(i * 128 * D * 2 + h * (128 * 128)), map_q, h * 64, it.hk * a.G,
                                    it.q0 + it.t0 + i * p.tok, &sh.q_full);
            }
            __syncwarp();
            ++count;
        }
        if (a.counter) {
            wait_item(sh, &sh.kv_started, (uint32_t)n & 1, a.status);
            uint32_t c = 0;
            if (lane == 0) c = atomicAdd(a.counter, 1u);
            x = (long long)gridDim.x + __shfl_sync(0xffffffffu, c, 0);
        } else {
            x = (n + 1ll) * gridDim.x + ((n & 1) ? blockIdx.x : gridDim.x - 1 - blockIdx.x);       // to and fro
        }
    }
    if (count > 0 && *reinterpret_cast<volatile int*>(&sh.dead)) settle(&sh.q_full, (uint32_t)(count - 1) & 1);
}

// Looks through the tiles of values on the items' edges.  A lane has every 32nd row of
// a tile: x * 0 added up is NaN where some x is an infinity or NaN.
template <int D>
__device__ void scan_role(Shared& sh, const PromptArgs& a, uint32_t slots, int lane)
{
    using Sh = Shape<D>;
    int entry = 0;                                 // ring entries before this item
    uint32_t turn = 0;                             // of the landing barriers, bits by slot
    bool ok = true;
    Items items;
    for (const Item* at; (at = items.next(sh, a.status)); items.release(sh, lane)) {
        const Item it = *at;
        const int cnt = it.tiles(), from = it.all / KT, mine = items.n % kItems;
        uint32_t some = 0;
#pragma unroll 1
        for (int j = from; ok && j < cnt; ++j) {
            const int slot = (entry + 2 * j + 1) % Sh::kSlots;
            if (!(ok = wait(sh, &sh.kv_land[slot], (turn >> slot) & 1, a.status))) break;
            turn ^= 1u << slot;
            const uint32_t base = slots + (uint32_t)slot * Sh::kSlotBytes;
            bool wrote = false;
#pragma unroll 1
            for (int b = 0; b < 4; ++b) {
                const int r = b * 32 + lane;
                uint32_t acc[4] = {0, 0, 0, 0};
#pragma unroll
                for (int c = 0; c < D / 8; ++c) {
                    const uint32_t at = base + (c >> 3) * (KT * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4);
                    uint32_t x[4];
                    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]) : "r"(at));
#pragma unroll
                    for (int k = 0; k < 4; ++k) asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(acc[k]) : "r"(x[k]), "r"(0));
                }
                bool nan = false;
#pragma unroll
                for (int k = 0; k < 4; ++k) nan |= (acc[k] & 0x7FFFu) > 0x7F80u || (acc[k] & 0x7FFF0000u) > 0x7F800000u;
                if (nan) {
                    wrote = true;
#pragma unroll 1
                    for (int c = 0; c < D / 2; ++c) {
                        const uint32_t at = base + (c >> 5) * (KT * 128) + r * 128 + ((((c >> 2) & 7) ^ (r & 7)) << 4) + (c & 3) * 4;
                        uint32_t x;
                        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(x) : "r"(at));
                        if ((x & 0x7F80u) == 0x7F80u) x &= 0xFFFF0000u;
                        if ((x & 0x7F800000u) == 0x7F800000u) x &= 0x0000FFFFu;
                        asm volatile("st.shared.b32 [%0], %1;" ::"r"(at), "r"(x) : "memory");
                    }
                }
                const uint32_t bits = __ballot_sync(0xffffffffu, nan);
                some |= bits;
                if (lane == 0) sh.bad[mine][j - from][b] = bits;
            }
            if (lane == 0) sh.noted[mine] = some != 0;
            if (wrote) fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.kv_full[slot]);
        }
        entry = (entry + 2 * cnt) % Sh::kSlots;
    }
}

// -------------------------------------------------------------- the products
// D = Q K^T: K-major operands, d / 16 steps of 32 bytes within 64-column blocks
// 16 KB apart.  One elected lane issues all steps, if its ok is true.
template <int D>
__device__ __forceinline__ void issue_qk(uint32_t d_tmem, uint64_t q_desc, uint64_t k_desc, uint32_t idesc, bool ok)
{
#pragma unroll
    for (int b = 0; b < D / 64; ++b) {
        asm volatile(
            "{\n\t.reg .pred e, t, f;\n\t.reg .b64 x, y;\n\t"
            "elect.sync _|e, 0xffffffff;\n\t"
            "setp.ne.and.b32 e, %5, 0, e;\n\t"
            "setp.ne.b32 f, %4, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, f;\n\t"
            "add.s64 x, %1, 2;\n\tadd.s64 y, %2, 2;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, t;\n\t"
            "add.s64 x, %1, 4;\n\tadd.s64 y, %2, 4;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, t;\n\t"
            "add.s64 x, %1, 6;\n\tadd.s64 y, %2, 6;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, t;\n\t}" ::"r"(d_tmem),
            "l"(q_desc + 1024 * b), "l"(k_desc + 1024 * b), "r"(idesc), "r"(b), "r"((int)ok)
            : "memory");
    }
}

// D (+)= P V for 64 keys: P in TMEM (8 columns of bf16 pairs per step), V MN-major
// (16 keys of 128 bytes per step).
__device__ __forceinline__ void issue_pv(uint32_t d_tmem, uint32_t p_tmem, uint64_t v_desc, uint32_t idesc,
                                         uint32_t accumulate, bool ok)
{
    asm volatile(
        "{\n\t.reg .pred e, t, f;\n\t.reg .b64 y;\n\t.reg .b32 x;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "setp.ne.and.b32 e, %5, 0, e;\n\t"
        "setp.ne.b32 f, %4, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, f;\n\t"
        "add.s32 x, %1, 8;\n\tadd.s64 y, %2, 128;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], y, %3, t;\n\t"
        "add.s32 x, %1, 16;\n\tadd.s64 y, %2, 256;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], y, %3, t;\n\t"
        "add.s32 x, %1, 24;\n\tadd.s64 y, %2, 384;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], y, %3, t;\n\t}" ::"r"(d_tmem),
        "r"(p_tmem), "l"(v_desc), "r"(idesc), "r"(accumulate), "r"((int)ok)
        : "memory");
}

// mma_commit (kda_sm100.cuh), if the elected lane's ok is true.
__device__ __forceinline__ void commit_if(uint64_t* bar, bool ok)
{
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
        "setp.ne.and.b32 e, %1, 0, e;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
        "r"((int)ok)
        : "memory");
}

// For both row tiles in turn, the output of tile j and the scores of tile j + 1, which
// go where tile j's scores and P were (the tensor core runs one thread's products in
// order); with P in columns of its own each row tile's scores before its output, once the last have
// been read.  (Both row tiles' scores first and then both outputs lets them fall into step, and
// both are at their exponentials at once: 16,384 tokens, d = 64, 567 us instead of 545.)
// Once a wait has given up no product is issued and nothing signalled any
// more; that is a predicate, so that the loops have one way out.
template <int D>
__device__ void mma_role(Shared& sh, const PromptArgs& a, uint32_t q_smem, uint32_t slots, uint32_t tmem, int lane)
{
    using Sh = Shape<D>;
    constexpr uint32_t id_qk = make_idesc_bf16(128, KT, false, false);
    constexpr uint32_t id_pv = make_idesc_bf16(128, D, false, true);
    int slot = 0;                                  // of the next ring entry to take
    uint32_t turn = 0;                             // parity of its use
    int done0 = 0, done1 = 0;                      // tiles of the items before, by row tile
    int pieces0 = 0, pieces1 = 0, some = 0;        // items before with work, by row tile and in all
    bool ok = true;                                // no wait of this lane has given up
    const uint64_t q_desc = make_sdesc(q_smem, 16, 1024, kSwizzle128B);
    auto take = [&]() {
        const int mine = slot;
        ok &= wait_lane(sh, &sh.kv_full[mine], turn, a.status);
        __syncwarp();
        tc_fence_after();
        if (++slot == Sh::kSlots) {
            slot = 0;
            turn ^= 1;
        }
        return mine;
    };
    Items items;
    for (const Item* at; (at = items.next(sh, a.status)); items.release(sh, lane)) {
        const Item it = *at;
        const int cnt = it.tiles();
        if (cnt == 0) continue;
        ok &= wait_lane(sh, &sh.q_full, (uint32_t)some & 1, a.status);
#pragma unroll 1
        for (int j = -1; j < cnt; ++j) {
            // V of tile j, then K of tile j + 1
            const bool more = j + 1 < cnt;
            const int ev = j >= 0 ? take() : 0;
            int ek = -1;
            const auto scores = [&](int i, int tiles) {
                if (j + 1 >= tiles) return;
                if (ek < 0) ek = take();
                const int t = (i ? done1 : done0) + j + 1;
                if (Sh::kOwnP && t > 0) {
                    ok &= wait_lane(sh, &sh.s_read[i], (uint32_t)(t - 1) & 1, a.status);
                    __syncwarp();
                    tc_fence_after();
                }
                const uint32_t k = slots + (uint32_t)ek * Sh::kSlotBytes;
                issue_qk<D>(tmem + i * 128, q_desc + (uint64_t)(i * 128 * D * 2 / 16), make_sdesc(k, 16, 1024, kSwizzle128B), id_qk, ok);
                commit_if(&sh.s_full[i], ok);
            };
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int tiles = i ? it.cnt[1] : it.cnt[0];
                if (Sh::kOwnP) scores(i, tiles);
                if (j >= 0 && j < tiles) {
                    const uint32_t v = slots + (uint32_t)ev * Sh::kSlotBytes, pt = tmem + Sh::kP + i * Sh::kPTile;
                    const uint64_t v_desc = make_sdesc(v, KT * 128, 1024, kSwizzle128B);
                    const uint32_t o = tmem + Sh::kO + i * D;
                    ok &= wait_lane(sh, &sh.p_full[i], (uint32_t)((i ? done1 : done0) + j) & 1, a.status);
                    const int before = i ? pieces1 : pieces0;
                    if (j == 0 && before > 0) ok &= wait_lane(sh, &sh.o_empty[i], (uint32_t)(before - 1) & 1, a.status);
                    __syncwarp();
                    tc_fence_after();
                    issue_pv(o, pt, v_desc, id_pv, j > 0, ok);
                    issue_pv(o, pt + Sh::kPHalf, v_desc + 512, id_pv, 1, ok);
                    commit_if(&sh.pv_done[i], ok);
                }
                if (!Sh::kOwnP) scores(i, tiles);
            }
            if (j >= 0) commit_if(&sh.kv_empty[ev], ok);
            if (more) commit_if(&sh.kv_empty[ek], ok);
            if (j + 2 == cnt) commit_if(&sh.q_empty, ok);
        }
        done0 += it.cnt[0];
        done1 += it.cnt[1];
        pieces0 += it.cnt[0] > 0;
        pieces1 += it.cnt[1] > 0;
        ++some;
    }
    // the last products and their arrivals on the ring's barriers come before the block ends
    mma_commit(&sh.done);
    wait_for<false>(sh, &sh.done, 0, a.status);
    __syncwarp();
}

// --------------------------------------------------- the softmax and the output
// Adds to O the infinities and NaN of the keys before `lim` that the scanning warp has
// taken out.
template <int D>
__device__ __forceinline__ void add_nonfinite(Shared& sh, const PromptArgs& a, const Item& it, int mine, int lim, int half, uint32_t to)
{
    constexpr int H = D / 2;
    const int from = it.all / KT;
#pragma unroll 1
    for (int c = 0; c < H / 16; ++c) {
        uint32_t y[16];
        tmem_ld16(to + 16 * c, y);
        tmem_ld_wait();
#pragma unroll 1
        for (int k = from * KT; k < lim; ++k) {
            if (!((sh.bad[mine][k / KT - from][(k >> 5) & 3] >> (k & 31)) & 1)) continue;
            const __nv_bfloat16* v = static_cast<const __nv_bfloat16*>(a.v) + (long long)(it.k0 + k) * a.v_stride + it.hk * D +
                                     half * H + 16 * c;
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const float z = __bfloat162float(v[e]);
                if (!(fabsf(z) < INFINITY)) y[e] = __float_as_uint(__uint_as_float(y[e]) + z);
            }
        }
        __syncwarp();
        tmem_st16(to + 16 * c, y);
    }
    tmem_st_wait();
}

// A warp's 32 rows of H channels, a lane's row packed in z, to memory: through 1 KB
// of shared memory, so that a store covers whole rows.  (Stored by each lane as
// they are, 16 bytes to each of 32 lines at a time, an item's rows held up every
// access to shared memory of the CTA for some 4,000 clocks.)
template <int H>
__device__ __forceinline__ void store_rows(const uint32_t (&z)[H / 2], int place, uint4* base, uint32_t stage, int lane)
{
    constexpr int L = H / 8;                       // 16-byte pieces, and lanes, of a row
    constexpr int R = 1024 / (H * 2);              // rows at a time
    const auto at = [&](int row, int c) { return stage + row * (H * 2) + ((c ^ (H == 64 ? row & 7 : (row >> 1) & 3)) << 4); };
#pragma unroll
    for (int r0 = 0; r0 < 32; r0 += R) {
        __syncwarp();
        if (lane >= r0 && lane < r0 + R) {
#pragma unroll
            for (int c = 0; c < L; ++c)
                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at(lane - r0, c)), "r"(z[4 * c]), "r"(z[4 * c + 1]),
                             "r"(z[4 * c + 2]), "r"(z[4 * c + 3])
                             : "memory");
        }
        __syncwarp();
#pragma unroll
        for (int q = 0; q < R * L / 32; ++q) {
            const int row = q * (32 / L) + lane / L;
            const int to = __shfl_sync(0xffffffffu, place, r0 + row);
            uint4 w;
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w) : "r"(at(row, lane % L)));
            if (to >= 0) base[to + lane % L] = w;
        }
    }
}

template <int D>
__device__ void softmax_role(Shared& sh, const PromptArgs& a, const Plan& p, uint32_t stage, int warp, int lane, uint32_t tmem)
{
    using Sh = Shape<D>;
    constexpr float kSlack = 8.f;
    constexpr int H = D / 2;                       // channels of the output of one half
    const int i = warp >> 3, half = (warp >> 2) & 1;       // row tile; which 64 keys, which half of O
    const int r = (warp & 3) * 32 + lane;          // row of the row tile
    const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t ts = lanes + i * 128 + half * 64, to = lanes + Sh::kO + i * D + half * H;
    const uint32_t tp = lanes + Sh::kP + i * Sh::kPTile + half * Sh::kPHalf;
    const uint32_t bar = 1 + i * 4 + (warp & 3);   // named barrier of the two warps of these rows
    const int tok = r < p.rows ? r / a.G : 1 << 29, g = r < p.rows ? r - tok * a.G : 0;
    const uint64_t scale2 = pack2(a.scale_log2, a.scale_log2);
    int done = 0;                                  // tiles before, of this row tile
    Items items;
    for (const Item* at; (at = items.next(sh, a.status)); items.release(sh, lane)) {
        const Item& it = *at;                      // (in shared memory)
        const int cnt = it.cnt[i];
        const int first = it.t0 + i * p.tok, off = it.lk - it.lq + 1, past = min(it.t0 + p.span, it.lq);
        const int lim = first + tok < past ? min(max(first + tok + off, 0), it.lk) : 0;   // keys that this row sees
        const int all = min(max(first + off, 0), it.lk);   // and those that every row of the tile sees
        float m = -INFINITY, l = 0.f;
#pragma unroll 1
        for (int j = 0; j < cnt; ++j) {
            wait_lane(sh, &sh.s_full[i], (uint32_t)(done + j) & 1, a.status);
            __syncwarp();
            tc_fence_after();
            uint32_t x[2][32];
            tmem_ld32(ts, x[0]);
            tmem_ld32(ts + 32, x[1]);
            tmem_ld_wait();
            if (Sh::kOwnP) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.s_read[i]);
            }
            if ((j + 1) * KT > all) {
                const int left = lim - j * KT - half * 64;         // this thread's keys from here on are hidden
#pragma unroll
                for (int c = 0; c < 64; ++c)
                    if (c >= left) x[c >> 5][c & 31] = 0xff800000u;
            }
            float tops[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int at = (c & 1) * 16;
                tops[c] = fmaxf(__uint_as_float(x[c >> 1][at]), __uint_as_float(x[c >> 1][at + 1]));
#pragma unroll
                for (int e = 2; e < 16; e += 2) tops[c] = max3(tops[c], x[c >> 1][at + e], x[c >> 1][at + e + 1]);
            }
            float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
            // (by turns: with scores that come early the other half may be a tile behind)
            float(&at_top)[2][128] = sh.top[Sh::kOwnP ? j & 1 : 0][i];
            at_top[half][r] = top;
            named_bar_sync(bar, 64);
            top = fmaxf(top, at_top[half ^ 1][r]) * a.scale_log2;   // the scale is positive on this path
            const bool grow = top > m + kSlack || (m == -INFINITY && top > m);
            if (__any_sync(0xffffffffu, grow)) {
                const float m2 = grow ? top : m;
                const float f = m2 == -INFINITY ? 1.f : ex2(m - m2);
                m = m2;
                l *= f;
                if (j > 0) {
                    wait_lane(sh, &sh.pv_done[i], (uint32_t)(done + j - 1) & 1, a.status);
                    __syncwarp();
                    tc_fence_after();
#pragma unroll 1
                    for (int c = 0; c < H / 16; ++c) {
                        uint32_t y[16];
                        tmem_ld16(to + 16 * c, y);
                        tmem_ld_wait();
#pragma unroll
                        for (int e = 0; e < 16; ++e) y[e] = __float_as_uint(__uint_as_float(y[e]) * f);
                        tmem_st16(to + 16 * c, y);
                    }
                }
            }
            // masked scores stay -inf (their e is 0) unless nothing was seen so far
            const uint64_t ref2 = pack2(m == -INFINITY ? 0.f : -m, m == -INFINITY ? 0.f : -m);
            uint64_t sum[2] = {0, 0};
            uint32_t e2[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) {
                const int c = e >> 4, k = 2 * (e & 15);
                float e0, e1;
                unpack2(fma2(pack2u(x[c][k], x[c][k + 1]), scale2, ref2), e0, e1);
                e0 = ex2(e0);
                e1 = ex2(e1);
                sum[e & 1] = add2(sum[e & 1], pack2(e0, e1));
                e2[e] = pack_bf16x2(e0, e1);
            }
            if (Sh::kOwnP && j > 0) {              // P of the tile before is in use until its product is done
                wait_lane(sh, &sh.pv_done[i], (uint32_t)(done + j - 1) & 1, a.status);
                __syncwarp();
                tc_fence_after();
            }
            tmem_st32(tp, e2);                     // (d = 128: over this half's scores, all of them in registers)
            float s0, s1;
            unpack2(add2(sum[0], sum[1]), s0, s1);
            l += s0 + s1;
            if (j + 1 == cnt) sh.sum[i][half][r] = l;
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.p_full[i]);
        }
        // the output
        float scale_o = 0.f;
        if (cnt > 0) {
            wait_lane(sh, &sh.pv_done[i], (uint32_t)(done + cnt - 1) & 1, a.status);
            __syncwarp();
            tc_fence_after();
            l += sh.sum[i][half ^ 1][r];           // (written before the last product began)
            // when some wait has given up, this item and those after it are not known
            if (*reinterpret_cast<volatile int*>(&sh.dead)) l = __int_as_float(0x7fffffff);
            scale_o = lim == 0 ? 0.f : __fdividef(1.f, l);
            // (written before the last product began; of an item without an edge whatever was there, and no keys are looked at)
            const int mine = items.n % kItems;
            if (*reinterpret_cast<volatile int*>(&sh.noted[mine])) add_nonfinite<D>(sh, a, it, mine, min(lim, cnt * KT), half, to);
        }
        // this row's place, in 16-byte pieces from the item's first row; negative: none
        const int place = first + tok < past ? ((i * p.tok + tok) * a.Hq + g) * (D / 8) + half * (H / 8) : -1;
        uint4* base = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.o) +
                                               ((long long)(it.q0 + it.t0) * a.Hq + (long long)it.hk * a.G) * D);
        done += cnt;
        uint32_t z[H / 2];
#pragma unroll
        for (int c = 0; c < H / 32; ++c) {
            uint32_t y[32];
            tmem_ld32(to + 32 * c, y);             // (of no keys: whatever is there; all rows are 0 then)
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 16; ++e)
                z[16 * c + e] = lim == 0 ? 0u : pack_bf16x2(__uint_as_float(y[2 * e]) * scale_o, __uint_as_float(y[2 * e + 1]) * scale_o);
        }
        if (cnt > 0) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.o_empty[i]);
        }
        store_rows<H>(z, place, base, stage, lane);
    }
}


template <int D>
__global__ void __launch_bounds__(kThreads, 1)
prompt_attention_tc_kernel(const __grid_constant__ PromptArgs a, const __grid_constant__ Plan p,
                           const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                           const __grid_constant__ CUtensorMap map_v)
{
    using Sh = Shape<D>;
    extern __shared__ uint8_t raw[];
    __shared__ Shared sh;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t q_smem = (smem_u32(raw) + 1023u) & ~1023u;
    const uint32_t slots = q_smem + Sh::kQBytes;
    if (tid == 0) {
        for (int i = 0; i < Sh::kSlots; ++i) {
            mbar_init(&sh.kv_full[i], 1);
            mbar_init(&sh.kv_land[i], 1);
            mbar_init(&sh.kv_empty[i], 1);
        }
        mbar_init(&sh.q_full, 1);
        mbar_init(&sh.q_empty, 1);
        mbar_init(&sh.done, 1);
        mbar_init(&sh.kv_started, 1);
        for (int i = 0; i < kItems; ++i) {
            mbar_init(&sh.item_full[i], 1);
            mbar_init(&sh.item_empty[i], kItemReaders);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.s_full[i], 1);
            mbar_init(&sh.s_read[i], 8);
            mbar_init(&sh.p_full[i], 8);
            mbar_init(&sh.pv_done[i], 1);
            mbar_init(&sh.o_empty[i], 8);
        }
        sh.dead = 0;
        for (int i = 0; i < kItems; ++i) sh.noted[i] = 0;
        fence_mbar_init();
    }
    if (warp == kMmaWarp) {
        tmem_alloc(&sh.tmem, 512);
        tmem_relinquish();
    }
    build_table(sh, a, p);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(&sh.tmem);
    if (warp < kMmaWarp) {
        more_registers<kMore>();
        softmax_role<D>(sh, a, p, slots + Sh::kSlots * Sh::kSlotBytes + warp * Sh::kStageBytes, warp, lane, tmem);
    } else {
        fewer_registers<kFewer>();
        if (warp == kMmaWarp) mma_role<D>(sh, a, q_smem, slots, tmem, lane);
        else if (warp == kKvWarp) kv_role<D>(sh, a, &map_k, &map_v, slots, lane);
        else if (warp == kQWarp) q_role<D>(sh, a, p, &map_q, q_smem, lane);
        else scan_role<D>(sh, a, slots, lane);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// Rows [rows][heads][d], boxes of `tokens` rows, `group` heads and 64 columns in the
// 128-byte swizzle.
bool make_map(CUtensorMap* m, const void* base, int d, int heads, long long rows, long long stride, int group, int tokens)
{
    const auto fn = tc_encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)rows};
    const cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)stride * 2};
    const cuuint32_t boxes[3] = {64, (cuuint32_t)group, (cuuint32_t)tokens};
    const cuuint32_t steps[3] = {1, 1, 1};
    const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, boxes, steps,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS && debug_enabled())
        fprintf(stderr, "kda: cuTensorMapEncodeTiled failed (CUresult %d, prompt)\n", (int)r);
    return r == CUDA_SUCCESS;
}

template <int D>
cudaError_t launch(PromptArgs a, int sms, cudaStream_t stream)
{
    Plan p;
    p.tok = 128 / a.G;
    p.rows = p.tok * a.G;
    CUtensorMap map_q, map_k, map_v;
    if (!make_map(&map_q, a.q, D, a.Hq, a.T, a.q_stride, a.G, p.tok) || !make_map(&map_k, a.k, D, a.Hkv, a.Tk, a.k_stride, 1, KT) ||
        !make_map(&map_v, a.v, D, a.Hkv, a.Tk, a.v_stride, 1, KT))
        return cudaErrorInvalidValue;
    auto kern = prompt_attention_tc_kernel<D>;
    const size_t bytes = Shape<D>::kBytes;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e != cudaSuccess) return e;
    // Every sequence has at most one pair of row tiles that is not full.  Claimed or dealt to
    // and fro, us: one prompt of 509 tokens (64 items) 18.7 and 15.1, 3 x 3,000 (564 items) 175
    // and 214, 8,192 (1,024) 362 and 352, 65,536 (2,048) 5,385 and 6,061.
    // One row tile to an item where that leaves no CTA more than one: one prompt of 509 tokens, 32
    // heads on 8, d = 128, 13.4 us (two 15.0), of 1,024, 16 on 4, d = 64, 13.8 us (17.3).
    p.span = 2 * p.tok;
    if (((long long)a.T / p.tok + a.N) * a.Hkv <= sms) p.span = p.tok;
    const long long items = ((long long)a.T / p.span + a.N) * a.Hkv;
    if (items > 2ll * sms) {
        const cudaError_t z = cudaMemsetAsync(a.counter, 0, sizeof(uint32_t), stream);
        if (z != cudaSuccess) return z;
    } else {
        a.counter = nullptr;
    }
    kern<<<(unsigned)(items < sms ? items : sms), kThreads, bytes, stream>>>(a, p, map_q, map_k, map_v);
    return cudaGetLastError();
}

}  // namespace

bool prompt_tc_supported(const PromptArgs& a, int32_t d, kda_dtype_t dtype)
{
    // (an item takes a microsecond per 128 keys, and no wait more than two seconds; places
    // within an item are 32-bit)
    return dtype == KDA_BF16 && (d == 64 || d == 128) && a.scale_log2 > 0.f && a.G <= 128 && a.Tk > 0 && a.Tk <= (1 << 27) &&
           a.T <= (1 << 27) && a.Hq <= (1 << 16);
}

cudaError_t launch_prompt_attention_tc(PromptArgs a, int32_t d, int sms, cudaStream_t stream)
{
    a.starve = getenv("KDA_TEST_STARVE_CONSUMERS") != nullptr;
    return d == 64 ? launch<64>(a, sms, stream) : launch<128>(a, sms, stream);
}

}  // namespace kda
