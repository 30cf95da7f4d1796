// kda_tree_attention_tc.cu -- the tensor-core form of the tree attention (bf16,
// d = 64 or 128): one CTA per SM, tcgen05 products with TMEM accumulators.
//
// Per tile of 128 keys and 128 query rows (lane = row):
//     S = Q K^T             (M = 128, N = 128, K = d; Q, K in shared memory)
//     P = 2^(c S - m)       (registers; c = scale log2 e; bf16 back over S)
//     O += P V              (M = 128, N = d, K = 128; P in TMEM, V MN-major)
// with the running maximum m and sum l of each row in the registers of the
// thread that owns the row.  m moves only when a tile exceeds it by more than
// 8, i.e. P may reach 2^8: then O and l are scaled by 2^(m - m').  Any m gives
// the same quotient O / l, and after the first tiles of a row O is left alone.
// P is rounded to bf16, the type of V, as one product takes one type; l sums
// the values before the rounding.
//
// Roles: a warpgroup per 128 query rows (softmax and output), one warp that
// issues the products, four warps that copy keys and values.  With up to 128
// rows (RT = 128) S is double-buffered, so that the next tile's scores are
// computed during this tile's softmax; with more (RT = 256) two row tiles share
// every K and V tile and alternate on the tensor core.
//
// Copies run ahead through a ring of K and V tiles: TMA boxes where 32 rows in
// a row are there and the page size allows, loads by the lanes elsewhere, which
// take any page size and fill rows past the length and rows of pages that do not
// exist with zeros, so that nothing stored there can reach a product.  In drafted
// values an infinity or NaN is replaced by 0: the product's 0 * inf would reach
// rows that do not see the node.  The rows that do see it add it to their output
// at the end.
//
// Bound, for few rows per cache head, by HBM: 32 x 16 nodes over contexts of 0 to
// 16,384 rows, 64 rows per cache head, 187 us, 5.8 TB/s (86 % of a copy), 64 x
// 4,096 rows, one token, 6.0 TB/s.  For many rows by the softmax beside the
// products: 4 x 64 nodes over 32K to 64K rows, 512 rows per cache head, 352 us, 1.17
// PFLOP/s (63 % of a library product), tensor pipe 54 % busy.  TMEM has room for one
// S per row tile then, so that a row tile's softmax and products take turns; a
// polynomial on the FMA pipe for every eighth exponential makes it 6 % slower, so it
// is instructions, not the exponential unit.  Pages of 16 rows cost 3 % against
// pages of 128.
//
// Every wait has a limit; one that gives up sets the workspace's timeout word and
// stops its CTA: the warps that start copies and products end at their next wait and
// wait for what they have started (again with a limit), and the softmax runs on
// without waiting, over whatever is there, and gives its rows a sum of NaN.  (The
// softmax warps may then arrive early at each other's barriers; nothing that follows
// from it is used.)  The environment variable KDA_TEST_STARVE_CONSUMERS, for the test
// of that path only, has the copying warps exit at once.
#include <cudaTypedefs.h>
#include <stdio.h>

#include "kda_sm100.cuh"
#include "kda_tree.cuh"

namespace kda {

// The driver's tensor-map encoder (kda_prefill_tc.cu).
PFN_cuTensorMapEncodeTiled_v12000 tc_encode_fn();

namespace {

using namespace sm100;

constexpr int KT = kTcKeys;                // keys per tile
using Piece = TreePieces<KT, kTcLead>;
constexpr int kRingMeta = 16;              // tiles whose key masks are kept
constexpr int kQWarps = 2;                 // warps that copy q

template <int D, int NT>
struct TcShape {
    static constexpr int kQBytes = NT * 128 * D * 2;
    static constexpr int kSlotBytes = KT * D * 2;
    static constexpr int kSlots = (D == 128) ? (NT == 1 ? 6 : 5) : 12;
    // Warps: softmax, copies, one that issues products, filled up to whole
    // warpgroups so that registers can be moved from the latter two to the
    // softmax: 384 x 168 >= 128 x 232 + 256 x 128, 512 x 128 = 256 x 184 + 256 x 72.
    static constexpr int kThreads = NT == 1 ? 384 : 512;
    static constexpr int kCopyWarp = NT * 4;
    static constexpr int kMmaWarp = NT * 4 + 4;
    static constexpr int kMore = NT == 1 ? 232 : 184, kFewer = NT == 1 ? 128 : 72;
    static constexpr size_t kBytes = 1024 + kQBytes + (size_t)kSlots * kSlotBytes;
    // TMEM columns
    static constexpr int kS1 = 128, kO0 = 256, kO1 = 256 + D;
};

struct TcShared {
    uint64_t kv_full[12], kv_empty[12], q_full, q_empty, done;
    uint64_t s_full[2], p_full[2], pv_done[2], o_empty[2];
    uint32_t tmem;
    int dead;
    alignas(16) uint32_t keys[kRingMeta][4];           // a tile's keys that are context rows of pages that exist
    uint32_t bad[kRingMeta][4];            // a tile's keys that are drafted nodes with inf or NaN in v
    long long loc[16 + 2];
};

// Waits for a phase of a barrier, for about two seconds at most and no longer than
// until some wait of this CTA has given up; false then.  Written short: the
// roles run side by side and have to share the SM's instruction cache (with
// mbar_wait's loops at every wait and all loops below unrolled they took 242 KB,
// and a piece's start and end cost 20 us).
__device__ __forceinline__ bool wait_lane(TcShared& sh, uint64_t* bar, uint32_t parity, int32_t* status)
{
    if (mbar_try_wait(bar, parity)) return true;
    const long long t0 = clock64();
#pragma unroll 1
    while (!mbar_try_wait(bar, parity)) {
        if (*reinterpret_cast<volatile int*>(&sh.dead)) return false;
        if (clock64() - t0 > (1ll << 32)) {
            *reinterpret_cast<volatile int*>(&sh.dead) = 1;
            atomicOr(status + kWsTimeoutWord, 2);
            return false;
        }
    }
    return true;
}

// The same for a warp, which goes on as one or stops as one.
__device__ __forceinline__ bool wait(TcShared& sh, uint64_t* bar, uint32_t parity, int32_t* status)
{
    return __all_sync(0xffffffffu, wait_lane(sh, bar, parity, status));
}

// One box of a page pool [num_pages][page_size][Hkv][d]: rows of one page, 64
// columns of one head.
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int32_t x, int32_t h,
                                            int32_t row, int32_t page, uint64_t* bar)
{
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(h), "r"(row), "r"(page), "r"(smem_u32(bar))
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
__device__ __forceinline__ uint64_t pack2(float a, float b)
{
    return pack2u(__float_as_uint(a), __float_as_uint(b));
}
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

// Which of eight bf16 (four words) are inf or NaN are set to 0; returns whether any was.
__device__ __forceinline__ bool clear_nonfinite(uint4& x)
{
    uint32_t* w = reinterpret_cast<uint32_t*>(&x);
    bool any = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if ((w[i] & 0x7F80u) == 0x7F80u) { w[i] &= 0xFFFF0000u; any = true; }
        if ((w[i] & 0x7F800000u) == 0x7F800000u) { w[i] &= 0x0000FFFFu; any = true; }
    }
    return any;
}

// anc[t] of one node (see tree_masks), by a whole warp: pointer doubling in
// registers, two nodes per lane, then each lane picks its t.
__device__ __forceinline__ unsigned long long tree_mask_of(const int32_t* parent, int Ts, int lane, int t)
{
    unsigned long long m[2];
    int u[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int x = lane + 32 * i;
        int p = -2;
        if (x < Ts) {
            p = parent ? __ldg(parent + x) : x - 1;
            if (p < -1 || p >= x) p = -2;
        }
        m[i] = 1ull << x;
        u[i] = p;
    }
#pragma unroll 1
    for (int round = 0; round < 6; ++round) {
        unsigned long long m2[2];
        int u2[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int src = u[i] & 31;
            const unsigned long long a = __shfl_sync(0xffffffffu, m[0], src);
            const unsigned long long b = __shfl_sync(0xffffffffu, m[1], src);
            const int ua = __shfl_sync(0xffffffffu, u[0], src), ub = __shfl_sync(0xffffffffu, u[1], src);
            const bool up = u[i] >= 0, hi = u[i] >= 32;
            m2[i] = m[i] | (up ? (hi ? b : a) : 0ull);
            u2[i] = up ? (hi ? ub : ua) : u[i];
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            m[i] = m2[i];
            u[i] = u2[i];
        }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
        if (u[i] != -1) m[i] = 0ull;
    const unsigned long long a = __shfl_sync(0xffffffffu, m[0], t & 31);
    const unsigned long long b = __shfl_sync(0xffffffffu, m[1], t & 31);
    return t >= 32 ? b : a;
}

// ---------------------------------------------------------------- the copies
// Byte offset of 16-byte chunk c of row r in a tile of 128 rows: 128-byte rows
// with the 128-byte swizzle, one block of rows per 64 columns.
__device__ __forceinline__ uint32_t tile_at(int r, int c)
{
    return (uint32_t)(c >> 3) * (128 * 128) + (uint32_t)r * 128 + (uint32_t)(((c & 7) ^ (r & 7)) << 4);
}

// Copies 32 rows of D bf16 to rows row0 .. row0 + 31 of a tile; lane's argument
// p is the source of row row0 + lane (null: zeros).  A warp, whole rows at a time,
// BATCH loads under way.  In rows whose bit of `clear` is set infinities and NaN
// become 0; returns the bits of those that had any.  The copy is ordered before
// the asynchronous reads of whoever the caller then tells.  (The same by cp.async
// took five times as long: 650 cycles an instruction, one after the other.)
template <int D, int BATCH>
__device__ __forceinline__ uint32_t copy_rows32(uint32_t dst, int row0, const __nv_bfloat16* p, uint32_t clear,
                                                int lane)
{
    constexpr int LPR = D / 8, RPI = 32 / LPR;     // lanes per row, rows per instruction
    constexpr int B = BATCH < 32 / RPI ? BATCH : 32 / RPI;
    const int c = lane % LPR, j0 = lane / LPR;
    const unsigned long long mine = reinterpret_cast<unsigned long long>(p);
    uint32_t bad = 0;
#pragma unroll 1
    for (int i0 = 0; i0 < 32 / RPI; i0 += B) {
        uint4 x[B];
#pragma unroll
        for (int k = 0; k < B; ++k) {
            const unsigned long long src = __shfl_sync(0xffffffffu, mine, (i0 + k) * RPI + j0);
            x[k] = make_uint4(0, 0, 0, 0);
            if (src) x[k] = __ldg(reinterpret_cast<const uint4*>(src + 16ull * c));
        }
        if (clear) {
#pragma unroll
            for (int k = 0; k < B; ++k) {
                const int j = (i0 + k) * RPI + j0;
                if (((clear >> j) & 1) && clear_nonfinite(x[k])) bad |= 1u << j;
            }
        }
#pragma unroll
        for (int k = 0; k < B; ++k)
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst + tile_at(row0 + (i0 + k) * RPI + j0, c)),
                         "r"(x[k].x), "r"(x[k].y), "r"(x[k].z), "r"(x[k].w)
                         : "memory");
    }
    fence_proxy_async_smem();
    return clear ? __reduce_or_sync(0xffffffffu, bad) : 0u;
}

// Four warps, 32 rows of every tile each.  A ring entry is one K or V tile; the
// entries of a piece are K_0, then (RT = 128) K_1 V_0 K_2 V_1 ... V_last or (RT =
// 256) V_0 K_1 V_1 ..., the order in which the products take them.  Two other
// warps copy each piece's q when the products of the piece before have read
// theirs, so that the ring does not drain between pieces.
//
// Where all 32 rows are context rows of pages that exist, and the page size
// allows (a.box), the rows come as TMA boxes that complete on the entry's
// barrier.  Elsewhere (the end of a context, other page sizes) the lanes copy
// them through registers.
template <int D, int NT>
struct Copier {
    using Sh = TcShape<D, NT>;
    static constexpr int kDrafted = -2;
    TcShared& sh;
    const TreeArgs& a;
    const CUtensorMap *map_k, *map_v;
    uint32_t slots;
    int lane, warp;                                // warp 0 .. 3
    int slot = 0, round = 0;                       // of the next ring entry

    __device__ uint32_t entry() const { return slots + (uint32_t)slot * Sh::kSlotBytes; }
    __device__ uint64_t* full() const { return &sh.kv_full[slot]; }

    // Waits until the next entry's slot is free.
    __device__ bool wait_slot()
    {
        return round == 0 || wait(sh, &sh.kv_empty[slot], (uint32_t)(round - 1) & 1, a.status);
    }

    // This lane's row of a tile: its page and its place there, or kDrafted and
    // the node; page -1: no row.
    struct Row {
        int page, slot;
    };
    // Walks this lane's rows tile by tile; the page number is loaded when the
    // row is looked up, a tile before it is used.
    struct Walk {
        int pos, p, slot;
    };
    __device__ Walk walk_from(int t) const
    {
        const int pos = t * KT + warp * 32 + lane;
        const int p = pos / a.page_size;
        return {pos, p, pos - p * a.page_size};
    }
    __device__ Row look_up(const Piece& w, int t, Walk& k) const
    {
        Row r = {-1, k.slot};
        if (t >= w.t1) return r;
        if (k.pos < w.ctx) r.page = __ldg(a.page_table + (long long)w.n * a.max_pages + k.p);
        else if (k.pos - w.ctx < a.Ts) r = {kDrafted, k.pos - w.ctx};
        k.pos += KT;
        k.p += a.tile_pages;
        k.slot += a.tile_rows;
        if (k.slot >= a.page_size) {
            k.slot -= a.page_size;
            ++k.p;
        }
        return r;
    }

    __device__ bool cached(const Row& r) const { return r.page >= 0 && r.page < a.num_pages; }

    // The row's source in the cache or among the drafted rows (null: none).
    __device__ const __nv_bfloat16* source(const Piece& w, const Row& r, const void* cache,
                                           const void* drafted) const
    {
        const int row_elems = a.Hkv * D;
        if (cached(r))
            return static_cast<const __nv_bfloat16*>(cache) + (long long)r.page * a.page_stride +
                   (long long)r.slot * row_elems + (long long)w.hk * D;
        if (r.page == kDrafted)
            return static_cast<const __nv_bfloat16*>(drafted) +
                   ((long long)w.n * a.Ts + r.slot) * row_elems + (long long)w.hk * D;
        return nullptr;
    }

    // The warp's 32 rows as boxes of a.box rows and 64 columns.
    __device__ void load_boxes(const CUtensorMap* map, const Piece& w, const Row& r)
    {
        if (lane == 0) mbar_arrive_expect_tx(full(), 32 * D * 2);
#pragma unroll 1
        for (int j = 0; j < 32; j += a.box) {
            const int page = __shfl_sync(0xffffffffu, r.page, j), slot = __shfl_sync(0xffffffffu, r.slot, j);
            if (lane == 0) {
#pragma unroll
                for (int h = 0; h < D / 64; ++h)
                    tma_load_4d(entry() + h * (128 * 128) + (warp * 32 + j) * 128, map, h * 64, w.hk, slot, page, full());
            }
            __syncwarp();
        }
    }

    // The next ring entry: the K or V rows of a piece's tile, the g-th tile of
    // the CTA.  False when the CTA has stopped.
    __device__ bool load(bool is_k, const Piece& w, const Row& r, int g)
    {
        if (!wait_slot()) return false;
        const uint32_t there = __ballot_sync(0xffffffffu, cached(r));
        if (a.box > 0 && there == 0xffffffffu) {
            if (lane == 0) {
                if (is_k) sh.keys[g % kRingMeta][warp] = there;
                else sh.bad[g % kRingMeta][warp] = 0;
            }
            load_boxes(is_k ? map_k : map_v, w, r);
        } else {
            const uint32_t drafted = is_k ? 0u : __ballot_sync(0xffffffffu, r.page == kDrafted);
            const uint32_t bad = copy_rows32<D, NT == 1 ? 8 : 4>(
                entry(), warp * 32, is_k ? source(w, r, a.k_cache, a.k) : source(w, r, a.v_cache, a.v), drafted, lane);
            if (lane == 0) {
                if (is_k) sh.keys[g % kRingMeta][warp] = there;
                else sh.bad[g % kRingMeta][warp] = bad;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(full());
        }
        if (++slot == Sh::kSlots) {
            slot = 0;
            ++round;
        }
        return true;
    }
};

// Returns how many ring entries it has filled.
template <int D, int NT>
__device__ int copy_role(TcShared& sh, const TreeArgs& a, const CUtensorMap* map_k, const CUtensorMap* map_v,
                         uint32_t slots, Piece w, bool go, int warp, int lane)
{
    using Sh = TcShape<D, NT>;
    Copier<D, NT> c{sh, a, map_k, map_v, slots, lane, warp};
    int g = 0;                                     // tiles of the pieces before
    bool ok = !a.starve;
    for (; ok && go; go = w.next(a)) {
        const int cnt = w.t1 - w.t0;
        auto walk = c.walk_from(w.t0);
        // the rows of the tile whose V comes next, of the one after it, and of the
        // one after that, whose page numbers are on their way
        typename Copier<D, NT>::Row row = {-1, 0}, row1 = row, row2 = row;
        int jk = 0, jv = -3;                       // tiles whose K, V are on their way
#pragma unroll 1
        while (jv < cnt) {
            const bool is_k = jv >= 0 && jk < cnt && jk < jv + (NT == 1 ? 2 : 1);
            if (jv >= 0 && !(ok = c.load(is_k, w, is_k && jk > jv ? row1 : row, g + (is_k ? jk : jv)))) break;
            if (is_k) {
                ++jk;
            } else {
                ++jv;
                row = row1;
                row1 = row2;
                row2 = c.look_up(w, w.t0 + jv + 2, walk);
            }
        }
        g += cnt;
    }
    return c.round * Sh::kSlots + c.slot;
}

template <int D, int NT>
__device__ void q_role(TcShared& sh, const TreeArgs& a, uint32_t q_smem, Piece w, bool go, int r0,
                       int warp, int lane)
{
    int piece = 0;
    for (; go; go = w.next(a)) {
        if (piece > 0 && !wait(sh, &sh.q_empty, (uint32_t)(piece - 1) & 1, a.status)) return;
#pragma unroll 1
        for (int b = warp; b < NT * 4; b += kQWarps) {
            const int r = r0 + b * 32 + lane;
            const __nv_bfloat16* p = nullptr;
            if (r < a.R) {
                const int t = r / a.G, g = r - t * a.G;
                p = static_cast<const __nv_bfloat16*>(a.q) +
                    (((long long)w.n * a.Ts + t) * a.Hq + w.hk * a.G + g) * D;
            }
            copy_rows32<D, NT == 1 ? 8 : 4>(q_smem + (b >> 2) * 128 * D * 2, (b & 3) * 32, p, 0, lane);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.q_full);
        ++piece;
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

// Takes the ring's entries in their order.  RT = 128: the scores of tile j + 1
// before the output of tile j.  RT = 256: for both row tiles in turn, the output
// of tile j and the scores of tile j + 1 (which go where tile j's P was: the
// tensor core runs one thread's products in order).  Once a wait has given up no
// product is issued and nothing signalled any more; that is a predicate, as branches
// out of these loops cost 5 % with 512 query rows.
template <int D, int NT>
__device__ void mma_role(TcShared& sh, const TreeArgs& a, uint32_t q_smem, uint32_t slots, Piece w, bool go,
                         int r0, uint32_t tmem)
{
    using Sh = TcShape<D, NT>;
    constexpr uint32_t id_qk = make_idesc_bf16(128, KT, false, false);
    constexpr uint32_t id_pv = make_idesc_bf16(128, D, false, true);
    int slot = 0;                                  // of the next ring entry to take
    uint32_t turn = 0;                             // parity of its use
    int first = 0, piece = 0;                      // tiles of the pieces before, pieces
    const int nt = (NT == 2 && a.R - r0 > 128) ? 2 : 1;
    bool ok = true;                                // no wait of this lane has given up
    const uint64_t q_desc = make_sdesc(q_smem, 16, 1024, kSwizzle128B);

    // Waits for the next ring entry; returns its slot.
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
    auto qk = [&](int i, int e, uint32_t d_tmem) {
        const uint32_t k = slots + (uint32_t)e * Sh::kSlotBytes;
        issue_qk<D>(d_tmem, q_desc + (uint64_t)(i * 128 * D * 2 / 16), make_sdesc(k, 16, 1024, kSwizzle128B), id_qk, ok);
    };
    // the output of tile `tile`, the j-th of the piece, of row tile i
    auto pv = [&](int i, int e, int j, int tile, int buf, uint32_t phase) {
        const uint32_t v = slots + (uint32_t)e * Sh::kSlotBytes;
        const uint64_t v_desc = make_sdesc(v, KT * 128, 1024, kSwizzle128B);
        const uint32_t d_tmem = tmem + (i ? Sh::kO1 : Sh::kO0);
        ok &= wait_lane(sh, &sh.p_full[buf], phase, a.status);
        if (j == 0 && piece > 0) ok &= wait_lane(sh, &sh.o_empty[i], (uint32_t)(piece - 1) & 1, a.status);
        __syncwarp();
        tc_fence_after();
        issue_pv(d_tmem, tmem + buf * Sh::kS1, v_desc, id_pv, j > 0, ok);
        issue_pv(d_tmem, tmem + buf * Sh::kS1 + 32, v_desc + 512, id_pv, 1, ok);
        commit_if(&sh.pv_done[i], ok);
    };

    for (; go; go = w.next(a)) {
        const int cnt = w.t1 - w.t0;
        ok &= wait_lane(sh, &sh.q_full, (uint32_t)piece & 1, a.status);
        if constexpr (NT == 1) {
            int jk = 0, jv = 0;
#pragma unroll 1
            while (jv < cnt) {
                const int entry = take();
                if (jk < cnt && jk < jv + 2) {
                    const int t = first + jk;
                    qk(0, entry, tmem + (t & 1) * Sh::kS1);
                    commit_if(&sh.s_full[t & 1], ok);
                    if (++jk == cnt) commit_if(&sh.q_empty, ok);
                } else {
                    const int t = first + jv;
                    pv(0, entry, jv, t, t & 1, (uint32_t)(t >> 1) & 1);
                    ++jv;
                }
                commit_if(&sh.kv_empty[entry], ok);
            }
        } else {
#pragma unroll 1
            for (int j = -1; j < cnt; ++j) {
                // V of tile j, then K of tile j + 1
                const bool more = j + 1 < cnt;
                const int ev = j >= 0 ? take() : 0;
                int ek = 0;
#pragma unroll 1
                for (int i = 0; i < nt; ++i) {
                    if (j >= 0) pv(i, ev, j, first + j, i, (uint32_t)(first + j) & 1);
                    if (more) {
                        if (i == 0) ek = take();
                        qk(i, ek, tmem + i * Sh::kS1);
                        commit_if(&sh.s_full[i], ok);
                    }
                }
                if (j >= 0) commit_if(&sh.kv_empty[ev], ok);
                if (more) commit_if(&sh.kv_empty[ek], ok);
                if (j + 2 == cnt) commit_if(&sh.q_empty, ok);
            }
        }
        first += cnt;
        ++piece;
    }
    // the last products and their arrivals on the ring's barriers come before the block ends
    mma_commit(&sh.done);
    mbar_wait(&sh.done, 0);
    __syncwarp();
}

// --------------------------------------------------- the softmax and the output
template <int D, int NT>
__device__ void softmax_role(TcShared& sh, const TreeArgs& a, Piece w, bool go, int r0, int warp, int lane,
                             uint32_t tmem)
{
    using Sh = TcShape<D, NT>;
    constexpr int RT = NT * 128;
    constexpr float kSlack = 8.f;
    const int wg = warp >> 2;
    const int local = warp * 32 + lane;            // row within the CTA's row tile
    const int r = r0 + local;
    const int rows = a.R - r0 < RT ? a.R - r0 : RT;
    if (NT == 2 && wg * 128 >= rows) return;       // nothing in this row tile
    const bool live = warp * 32 < rows;            // some row of this warp exists
    const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t to = lanes + (wg ? Sh::kO1 : Sh::kO0);
    const int node = (r < a.R ? r : a.R - 1) / a.G;
    int tile = 0, have = -1;
    unsigned long long seen = 0;
    for (; go; go = w.next(a)) {
        if (have != w.n) {
            seen = tree_mask_of(a.parent ? a.parent + (long long)w.n * a.Ts : nullptr, a.Ts, lane, node);
            have = w.n;
        }
        float m = -INFINITY, l = 0.f;
        for (int t = w.t0; t < w.t1; ++t, ++tile) {
            const int b = NT == 1 ? tile & 1 : wg;
            const uint32_t phase = (uint32_t)(NT == 1 ? tile >> 1 : tile) & 1;
            const uint32_t ts = lanes + b * Sh::kS1;
            // Every phase of pv_done is waited for in turn (wait_last): with RT =
            // 128 the scores of this tile may be there before the last tile's
            // product, and a parity names only the phase before the current one.
            wait_lane(sh, &sh.s_full[b], phase, a.status);
            __syncwarp();
            tc_fence_after();
            auto wait_last = [&]() {
                if (tile > 0) wait_lane(sh, &sh.pv_done[NT == 1 ? 0 : wg], (uint32_t)(tile - 1) & 1, a.status);
            };
            if (live) {
                const uint4 there = *reinterpret_cast<const uint4*>(sh.keys[tile % kRingMeta]);
                if ((there.x & there.y & there.z & there.w) != 0xffffffffu) {
                    // masked scores become -inf in place, 32 keys at a time
                    const int nc = w.ctx - t * KT; // key j is drafted node j - nc from j = nc on
#pragma unroll 1
                    for (int c = 0; c < 4; ++c) {
                        uint32_t keep = sh.keys[tile % kRingMeta][c], y[32];
                        const int i = 32 * c - nc; // the node at bit 0 of this word
                        if (i >= 0) keep |= i < 64 ? (uint32_t)(seen >> i) : 0u;
                        else if (i > -32) keep |= (uint32_t)(seen << -i);
                        tmem_ld32(ts + 32 * c, y);
                        tmem_ld_wait();
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (!((keep >> j) & 1)) y[j] = 0xff800000u;
                        tmem_st32(ts + 32 * c, y);
                    }
                    tmem_st_wait();
                }
                uint32_t x[4][32];
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_ld32(ts + 32 * c, x[c]);
                tmem_ld_wait();
                float tops[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    tops[c] = fmaxf(__uint_as_float(x[c][0]), __uint_as_float(x[c][1]));
#pragma unroll
                    for (int j = 2; j < 32; j += 2) tops[c] = max3(tops[c], x[c][j], x[c][j + 1]);
                }
                float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
                top *= a.scale_log2;               // the scale is positive on this path
                const bool grow = top > m + kSlack || (m == -INFINITY && top > m);
                if (__any_sync(0xffffffffu, grow)) {
                    const float m2 = grow ? top : m;
                    const float f = m2 == -INFINITY ? 1.f : ex2(m - m2);
                    m = m2;
                    l *= f;
                    if (t > w.t0) {
                        wait_last();
                        __syncwarp();
                        tc_fence_after();
#pragma unroll 1
                        for (int c = 0; c < D / 16; ++c) {
                            uint32_t y[16];
                            tmem_ld16(to + 16 * c, y);
                            tmem_ld_wait();
#pragma unroll
                            for (int j = 0; j < 16; ++j) y[j] = __float_as_uint(__uint_as_float(y[j]) * f);
                            tmem_st16(to + 16 * c, y);
                        }
                    }
                }
                // masked scores stay -inf (their e is 0) unless nothing was seen so far
                const uint64_t ref2 = pack2(m == -INFINITY ? 0.f : -m, m == -INFINITY ? 0.f : -m);
                const uint64_t scale2 = pack2(a.scale_log2, a.scale_log2);
                uint64_t sum[4] = {0, 0, 0, 0};
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t p[32];
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        const int c = 2 * h + (j >> 4), k = 2 * (j & 15);
                        float e0, e1;
                        unpack2(fma2(pack2u(x[c][k], x[c][k + 1]), scale2, ref2), e0, e1);
                        e0 = ex2(e0);
                        e1 = ex2(e1);
                        sum[j & 3] = add2(sum[j & 3], pack2(e0, e1));
                        p[j] = pack_bf16x2(e0, e1);
                    }
                    tmem_st32(ts + 32 * h, p);     // over scores, all of them in registers
                }
                float s0, s1;
                unpack2(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])), s0, s1);
                l += s0 + s1;
                tmem_st_wait();
            }
            wait_last();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.p_full[b]);
        }
        // the output of the piece
        wait_lane(sh, &sh.pv_done[NT == 1 ? 0 : wg], (uint32_t)(tile - 1) & 1, a.status);
        __syncwarp();
        tc_fence_after();
        // when some wait has given up, this piece and those after it are not known
        if (*reinterpret_cast<volatile int*>(&sh.dead)) l = __int_as_float(0x7fffffff);
        const bool whole = w.t0 == 0 && w.t1 == w.tiles;
        if (live) {
            const bool mine = r < a.R;
            unsigned long long add = 0;            // seen nodes with inf or NaN values
#pragma unroll 1
            for (int t = w.t1 - 1, k = 1; t >= w.t0 && (t + 1) * KT > w.ctx; --t, ++k) {
#pragma unroll 1
                for (int c = 0; c < 4; ++c) {
                    const unsigned long long bits = sh.bad[(tile - k) % kRingMeta][c];
                    const int i = 32 * c - (w.ctx - t * KT);
                    if (i >= 0) add |= i < 64 ? bits << i : 0ull;
                    else if (i > -32) add |= bits >> -i;
                }
            }
            add &= seen;
            const float scale_o = seen == 0 || l == 0.f ? 0.f : 1.f / l;
            const int g = r - node * a.G;
            __nv_bfloat16* op = static_cast<__nv_bfloat16*>(a.o) +
                                (((long long)w.n * a.Ts + node) * a.Hq + w.hk * a.G + g) * D;
            float* part = a.part + ((size_t)blockIdx.x * 2 + (w.t0 == 0 ? 1 : 0)) * RT * (D + 2);
            if (__any_sync(0xffffffffu, add != 0)) {
                // O is corrected in place
#pragma unroll 1
                for (int c = 0; c < D / 16; ++c) {
                    uint32_t x[16];
                    tmem_ld16(to + 16 * c, x);
                    tmem_ld_wait();
#pragma unroll 1
                    for (unsigned long long left = add; left; left &= left - 1) {
                        const int j = __ffsll((long long)left) - 1;
                        const __nv_bfloat16* v = static_cast<const __nv_bfloat16*>(a.v) +
                            (((long long)w.n * a.Ts + j) * a.Hkv + w.hk) * D + 16 * c;
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const float y = __bfloat162float(v[i]);
                            if (!(fabsf(y) < INFINITY)) x[i] = __float_as_uint(__uint_as_float(x[i]) + y);
                        }
                    }
                    __syncwarp();
                    tmem_st16(to + 16 * c, x);
                }
                tmem_st_wait();
            }
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
                uint32_t x[32];
                tmem_ld32(to + 32 * c, x);
                tmem_ld_wait();
                if (mine && whole) {
#pragma unroll
                    for (int i = 0; i < 32; i += 8) {
                        uint32_t y[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            y[j] = pack_bf16x2(__uint_as_float(x[i + 2 * j]) * scale_o,
                                               __uint_as_float(x[i + 2 * j + 1]) * scale_o);
                        *reinterpret_cast<uint4*>(op + 32 * c + i) =
                            seen == 0 ? make_uint4(0, 0, 0, 0) : make_uint4(y[0], y[1], y[2], y[3]);
                    }
                } else if (mine) {
                    // of an unused node whatever is there: its weight is 0
#pragma unroll
                    for (int i = 0; i < 32; i += 4)
                        *reinterpret_cast<uint4*>(part + (size_t)local * D + 32 * c + i) =
                            make_uint4(x[i], x[i + 1], x[i + 2], x[i + 3]);
                }
                __syncwarp();                      // before the next collective load
            }
            if (mine && !whole) {
                part[RT * D + local] = seen == 0 ? -INFINITY : m;
                part[RT * D + RT + local] = seen == 0 ? 0.f : l;
            }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.o_empty[NT == 1 ? 0 : wg]);
    }
}

template <int D, int NT>
__global__ void __launch_bounds__(TcShape<D, NT>::kThreads, 1)
tree_attention_tc_kernel(const __grid_constant__ TreeArgs a, const __grid_constant__ CUtensorMap map_k,
                         const __grid_constant__ CUtensorMap map_v)
{
    using Sh = TcShape<D, NT>;
    extern __shared__ uint8_t raw[];
    __shared__ TcShared sh;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t q_smem = (smem_u32(raw) + 1023u) & ~1023u;
    const uint32_t slots = q_smem + Sh::kQBytes;
    if (tid == 0) {
        for (int i = 0; i < Sh::kSlots; ++i) {
            mbar_init(&sh.kv_full[i], 4);
            mbar_init(&sh.kv_empty[i], 1);
        }
        mbar_init(&sh.q_full, kQWarps);
        mbar_init(&sh.q_empty, 1);
        mbar_init(&sh.done, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.s_full[i], 1);
            mbar_init(&sh.p_full[i], 4);
            mbar_init(&sh.pv_done[i], 1);
            mbar_init(&sh.o_empty[i], 4);
        }
        sh.dead = 0;
        fence_mbar_init();
    }
    if (warp == Sh::kMmaWarp) {
        tmem_alloc(&sh.tmem, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    const int group = blockIdx.x / a.row_tiles, r0 = (blockIdx.x % a.row_tiles) * (NT * 128);
    const TreeSpot sp = tree_locate<Sh::kThreads, KT, kTcLead>(a, group, sh.loc);   // has block barriers
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(&sh.tmem);
    Piece first;
    const bool go = first.start(a, sp, group);
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    int filled = 0;
    if (warp < Sh::kCopyWarp) {
        more_registers<Sh::kMore>();
        softmax_role<D, NT>(sh, a, first, go, r0, warp, lane, tmem);
    } else if (warp < Sh::kMmaWarp) {
        fewer_registers<Sh::kFewer>();
        filled = copy_role<D, NT>(sh, a, &map_k, &map_v, slots, first, go, warp - Sh::kCopyWarp, lane);
    } else {
        fewer_registers<Sh::kFewer>();
        if (warp == Sh::kMmaWarp)
            mma_role<D, NT>(sh, a, q_smem, slots, first, go, r0, tmem);
        else if (warp <= Sh::kMmaWarp + kQWarps)
            q_role<D, NT>(sh, a, q_smem, first, go, r0, warp - Sh::kMmaWarp - 1, lane);
    }
    tc_fence_before();
    __syncthreads();
    // After a wait that gave up nobody has waited for the last copies in flight.
    if (sh.dead) {
#pragma unroll 1
        for (int e = filled > Sh::kSlots ? filled - Sh::kSlots : 0; e < filled; ++e)
            mbar_wait(&sh.kv_full[e % Sh::kSlots], (uint32_t)(e / Sh::kSlots) & 1, 1ll << 24);
    }
    if (warp == Sh::kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <int D, int NT>
cudaError_t launch_tc(const TreeArgs& a, const CUtensorMap& map_k, const CUtensorMap& map_v, cudaStream_t stream)
{
    auto kern = tree_attention_tc_kernel<D, NT>;
    const size_t bytes = TcShape<D, NT>::kBytes;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e != cudaSuccess) return e;
    kern<<<a.groups * a.row_tiles, TcShape<D, NT>::kThreads, bytes, stream>>>(a, map_k, map_v);
    return cudaGetLastError();
}

// The pool as [num_pages][page_size][Hkv][d], boxes of `box` rows of one page
// and 64 columns of one head in the 128-byte swizzle.
bool make_pool_map(CUtensorMap* m, const void* base, const TreeArgs& a, int d, int box)
{
    const auto fn = tc_encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)a.Hkv, (cuuint64_t)a.page_size, (cuuint64_t)a.num_pages};
    const cuuint64_t row = (cuuint64_t)a.Hkv * d * 2;
    const cuuint64_t page = a.num_pages > 1 ? (cuuint64_t)a.page_stride * 2 : row * a.page_size;
    const cuuint64_t strides[3] = {(cuuint64_t)d * 2, row, page};
    const cuuint32_t boxes[4] = {64, 1, (cuuint32_t)box, 1};
    const cuuint32_t steps[4] = {1, 1, 1, 1};
    const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, boxes, steps,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS && debug_enabled())
        fprintf(stderr, "kda: cuTensorMapEncodeTiled failed (CUresult %d, page pool)\n", (int)r);
    return r == CUDA_SUCCESS;
}

}  // namespace

cudaError_t launch_tree_attention_tc(TreeArgs args, const TreePlan& plan, int32_t d, cudaStream_t stream)
{
    // Boxes of up to 32 rows that a page holds whole, and no fewer than the 8
    // rows of a swizzle group; other page sizes are copied by the lanes.
    int box = 32;
    while (box >= 8 && args.page_size % box != 0) box /= 2;
    CUtensorMap map_k = {}, map_v = {};
    if (box < 8 || args.num_pages == 0 || !make_pool_map(&map_k, args.k_cache, args, d, box) ||
        !make_pool_map(&map_v, args.v_cache, args, d, box))
        box = 0;
    args.box = box;
    args.tile_pages = KT / args.page_size;
    args.tile_rows = KT % args.page_size;
    args.starve = getenv("KDA_TEST_STARVE_CONSUMERS") != nullptr;
    if (d == 64)
        return plan.rt == 128 ? launch_tc<64, 1>(args, map_k, map_v, stream)
                              : launch_tc<64, 2>(args, map_k, map_v, stream);
    return plan.rt == 128 ? launch_tc<128, 1>(args, map_k, map_v, stream)
                          : launch_tc<128, 2>(args, map_k, map_v, stream);
}

}  // namespace kda
