// kda_tree_attention.cu -- attention of drafted tree nodes to a paged cache
// and to their ancestors: the CUDA-core kernel, the join of partial results
// and the launcher.
//
// For query row r = (node t, query head) against keys j:
//     x_j = scale q . k_j,   o = sum_j e^{x_j - m} v_j / sum_j e^{x_j - m}
// over the context rows of the cache and the drafted nodes that are t or its
// ancestors.  One pass over the keys with the running maximum m and sum l: a
// new tile with maximum m' scales o and l by e^{m - m'}.  Exponentials are
// taken in base 2 with log2(e) folded into q.
#include <type_traits>

#include "kda_tree.cuh"

namespace kda {
namespace {

// The CUDA-core kernels: fp32, bf16 with small heads or fp32 output, scales that
// are not positive.

// Pairs of fp32 for the two-wide FMA.
__device__ __forceinline__ uint64_t pack2(float a, float b)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t x)
{
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// 16 bytes of values as pairs of fp32.
__device__ __forceinline__ void pairs(const float*, const uint4& a, uint64_t (&x)[2])
{
    x[0] = (uint64_t)a.y << 32 | a.x;
    x[1] = (uint64_t)a.w << 32 | a.z;
}
__device__ __forceinline__ void pairs(const __nv_bfloat16*, const uint4& a, uint64_t (&x)[4])
{
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = (uint64_t)(w[i] & 0xFFFF0000u) << 32 | (w[i] << 16);
}

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 16 bytes to shared memory, asynchronously; zeros, and no read, unless there.
__device__ __forceinline__ void copy16(void* dst, const void* src, bool there)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)),
                 "l"(src), "r"(there ? 16 : 0)
                 : "memory");
}

// Up to 8 query rows per cache head: a stream.  A group of lanes shares a key, 16
// bytes each, and the groups of a CTA take keys in turn: a lane has its channels
// of q and of the output for all eight rows in registers.  Its pieces
// of K and V come by cp.async through kAhead stages of shared memory that no
// other lane touches, page numbers two steps earlier still.  The scores of a key
// are added up across its lanes so that each lane ends with the rows it owns
// (halving the rows at every step of the butterfly), takes their exponentials,
// and the probabilities go back to all lanes.  Every group has its own running
// maximum and sum per owned row (a maximum moves when a score exceeds it by more
// than 8, in base 2); they meet at the end of a piece.  Nothing in the loop
// waits for another warp.
// The context's keys have a loop of their own, without the tests that drafted
// nodes need.  Bound by instructions between the loads (eight rows of FMAs and one
// butterfly a key; 60 % of the issue slots), not by HBM: fp32, 16 heads, 5 nodes, 8
// contexts of 10 to 4000 rows, d = 64: 46 us (3.0 TB/s), 60 with one loop for all
// keys and with selects in the butterfly instead of q's permuted places; d = 128, 8
// nodes, 8 x 4096 rows: 132 us (4.1 TB/s); bf16, 16 heads, 5 nodes, 8 x 4096 rows:
// d = 32 38 us, d = 16 34 us (1.8 and 1.0 TB/s: as many steps of less).  K and V straight to registers, one or
// two steps ahead: 1.8 times as long; 4 keys a step 1.2 times.
constexpr int kAhead = 4;            // stages of two keys; 3 cost 5 % with one row
constexpr int kStreamRows = 8;
constexpr int kStreamThreads = 128;
constexpr int kStreamKeys = 64;      // keys per tile of the work split
constexpr int kStreamLead = 2;
// Per SM, by the registers that eight rows of q and of the output take.  fp32
// (4 channels a lane): 3, 4 and 5 took 50, 50 and 83 us at 8 x 2100 rows; at 5 they
// spill.  bf16 (8 channels, fp32 output, d = 128, 8 x 4096 rows): 2 and 3 took 100
// and 127.
__host__ __device__ constexpr int stream_ctas(bool fp32) { return fp32 ? 4 : 2; }

template <typename TI, typename TO, int D>
__global__ void __launch_bounds__(kStreamThreads, stream_ctas(sizeof(TI) == 4))
tree_attention_stream_kernel(const TreeArgs a)
{
    constexpr int RT = kStreamRows, CH = 16 / (int)sizeof(TI);  // rows, channels per lane
    constexpr int CP = CH / 2, LK = D / CH, GW = 32 / LK;       // pairs, lanes per key, groups per warp
    constexpr int kWarps = kStreamThreads / 32, kStep = kWarps * GW;
    constexpr int RO = RT / LK > 0 ? RT / LK : 1;               // rows a lane owns
    constexpr float kSlack = 8.f;
    __shared__ long long sh_loc[kWarps + 2];
    __shared__ unsigned long long anc[kTreeMaxNodes];
    __shared__ int32_t up[kTreeMaxNodes];
    __shared__ float sh_m[kWarps][RT], sh_l[kWarps][RT];
    __shared__ __align__(16) float sh_o[kWarps][RT][D];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane % LK, sub = lane / LK;                   // lane of the group, group of the warp
    // the first row this lane owns; LK / RT lanes share it when LK > RT
    const int own = LK >= RT ? g / (LK / RT) : g * RO;
    const TI* q = static_cast<const TI*>(a.q);
    extern __shared__ __align__(16) uint4 ring[];               // [kAhead][2 keys][K, V][threads]

    const int group = blockIdx.x / a.row_tiles, r0 = (blockIdx.x % a.row_tiles) * RT;
    const int rows = a.R - r0 < RT ? a.R - r0 : RT;
    const TreeSpot sp = tree_locate<kStreamThreads, kStreamKeys, kStreamLead>(a, group, sh_loc);
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int row_elems = a.Hkv * D;
    const int step_pages = kStep / a.page_size, step_rows = kStep % a.page_size;
    int have = -1;                                  // the sequence anc[] is of

    TreePieces<kStreamKeys, kStreamLead> w;
    for (bool more = w.start(a, sp, group); more; more = w.next(a)) {
        const int n = w.n, ctx = w.ctx, hk = w.hk;
        const int keys_end = w.t1 == w.tiles ? ctx + a.Ts : w.t1 * kStreamKeys;
        const int32_t* table = a.page_table + (long long)n * a.max_pages;
        __syncthreads();                            // the last piece's shared arrays have been read
        if (have != n) {
            if (tid < 32)
                tree_masks(a.parent ? a.parent + (long long)n * a.Ts : nullptr, a.Ts, tid, anc, up);
            have = n;
        }
        // q, scaled, this lane's channels of every row; place r has row r ^ own, so
        // that the places that a step of the butterfly keeps are the same in all lanes
        uint64_t qr[RT][CP], acc[RT][CP];
#pragma unroll
        for (int r = 0; r < RT; ++r) {
#pragma unroll
            for (int i = 0; i < CP; ++i) qr[r][i] = acc[r][i] = 0;
            const int row = r0 + (r ^ own);
            if (row < a.R) {
                const int t = row / a.G, h = row % a.G;
                const TI* from = q + (((long long)n * a.Ts + t) * a.Hq + hk * a.G + h) * D + CH * g;
                pairs(q, *reinterpret_cast<const uint4*>(from), qr[r]);
#pragma unroll
                for (int i = 0; i < CP; ++i) qr[r][i] = mul2(qr[r][i], pack2(a.scale_log2, a.scale_log2));
            }
        }
        __syncthreads();
        unsigned long long seen[RO];
        float m[RO], l[RO];
#pragma unroll
        for (int i = 0; i < RO; ++i) {
            seen[i] = own + i < rows ? anc[(r0 + own + i) / a.G] : 0ull;
            m[i] = -INFINITY;
            l[i] = 0.f;
        }
        // This group's keys: pos, pos + kStep, ..., two at a time; at, in: the next
        // position to fetch and the next to look up.
        int pos = w.t0 * kStreamKeys + warp * GW + sub, at = pos;
        int in = pos, in_p = pos / a.page_size, in_slot = pos - in_p * a.page_size;
        const int cached_end = ctx < keys_end ? ctx : keys_end;
        int page[2], slot[2];
        auto look = [&]() {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                page[i] = -1;
                slot[i] = in_slot;
                if (in < cached_end) page[i] = __ldg(table + in_p);
                in += kStep;
                in_p += step_pages;
                in_slot += step_rows;
                if (in_slot >= a.page_size) {
                    in_slot -= a.page_size;
                    ++in_p;
                }
            }
        };
        // (a cache without pages is never read, but an address is formed)
        const TI* kc = a.num_pages > 0 ? static_cast<const TI*>(a.k_cache) + (long long)hk * D + CH * g : q;
        const TI* vc = a.num_pages > 0 ? static_cast<const TI*>(a.v_cache) + (long long)hk * D + CH * g : q;
        unsigned there = 0;                         // bit 2 s + i: key i of stage s exists
        auto fetch = [&](int stage) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                bool row = (unsigned)page[i] < (unsigned)a.num_pages;
                const long long off = row ? page[i] * a.page_stride + (long long)slot[i] * row_elems : 0;
                const TI *kp = kc + off, *vp = vc + off;
                if (at >= ctx) {
                    row = at < keys_end;
                    const long long own_off = row ? (long long)hk * D + CH * g + ((long long)n * a.Ts + at - ctx) * row_elems : 0;
                    kp = static_cast<const TI*>(a.k) + own_off;
                    vp = static_cast<const TI*>(a.v) + own_off;
                }
                const int bit = 2 * stage + i;
                there = (there & ~(1u << bit)) | ((unsigned)row << bit);
                uint4* to = ring + bit * 2 * kStreamThreads + tid;
                copy16(to, kp, row);
                copy16(to + kStreamThreads, vp, row);
                at += kStep;
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        look();
#pragma unroll 1
        for (int i = 0; i < kAhead - 1; ++i) {
            fetch(i);
            look();
        }
        const int steps = (keys_end - w.t0 * kStreamKeys + 2 * kStep - 1) / (2 * kStep);
        int stage = 0;
        auto keys = [&](auto drafted) {             // whether drafted nodes may be among the keys
            constexpr bool kTail = decltype(drafted)::value;
            // the stage used in the step before takes the next keys
            fetch(stage ? stage - 1 : kAhead - 1);
            look();
            asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
            const uint4* mine = ring + stage * 4 * kStreamThreads + tid;
            // the scores of this group's keys: partial sums of all rows
            float s[2][RT];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                uint64_t x[CP];
                pairs(q, mine[u * 2 * kStreamThreads], x);
#pragma unroll
                for (int r = 0; r < RT; ++r) {
                    uint64_t t = mul2(qr[r][0], x[0]);
#pragma unroll
                    for (int i = 1; i < CP; ++i) t = fma2(qr[r][i], x[i], t);
                    const float2 y = unpack2(t);
                    s[u][r] = y.x + y.y;
                }
            }
            // across the group's lanes, each keeping half of the rows
            int cnt = RT;
#pragma unroll
            for (int off = LK / 2; off > 0; off /= 2) {
                if (cnt > 1) {
                    cnt /= 2;
#pragma unroll
                    for (int u = 0; u < 2; ++u)
#pragma unroll
                        for (int r = 0; r < cnt; ++r)
                            s[u][r] += __shfl_xor_sync(0xffffffffu, s[u][r + cnt], off);
                } else {
#pragma unroll
                    for (int u = 0; u < 2; ++u) s[u][0] += __shfl_xor_sync(0xffffffffu, s[u][0], off);
                }
            }
            const int node = pos - ctx;             // of the first key; the second's is kStep on
            bool grow = false;
            float top[RO];
#pragma unroll
            for (int i = 0; i < RO; ++i) {
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int nd = node + u * kStep;
                    bool see = (there >> (2 * stage + u)) & 1;
                    if (kTail) see = see && (nd < 0 || ((seen[i] >> (nd & 63)) & 1ull));
                    if (!see) s[u][i] = -INFINITY;
                }
                top[i] = fmaxf(s[0][i], s[1][i]);
                grow = grow || top[i] > m[i] + kSlack || (m[i] == -INFINITY && top[i] > m[i]);
            }
            if (__any_sync(0xffffffffu, grow)) {
                float f[RO];
#pragma unroll
                for (int i = 0; i < RO; ++i) {
                    const bool up_m = top[i] > m[i] + kSlack || (m[i] == -INFINITY && top[i] > m[i]);
                    f[i] = up_m ? exp2f(m[i] - top[i]) : 1.f;
                    if (up_m) m[i] = top[i];
                    l[i] *= f[i];
                }
#pragma unroll
                for (int r = 0; r < RT; ++r) {
                    const int from = LK >= RT ? r * (LK / RT) : r / RO;
                    const float fr = __shfl_sync(0xffffffffu, f[r % RO], (lane & ~(LK - 1)) + from);
#pragma unroll
                    for (int i = 0; i < CP; ++i) acc[r][i] = mul2(acc[r][i], pack2(fr, fr));
                }
            }
            float p[2][RO];
#pragma unroll
            for (int i = 0; i < RO; ++i)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    p[u][i] = ex2(s[u][i] - (m[i] == -INFINITY ? 0.f : m[i]));
                    l[i] += p[u][i];
                }
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                uint64_t x[CP];
                pairs(q, mine[(u * 2 + 1) * kStreamThreads], x);
                const int nd = node + u * kStep;
#pragma unroll
                for (int r = 0; r < RT; ++r) {
                    const int from = LK >= RT ? r * (LK / RT) : r / RO;
                    const float pr = __shfl_sync(0xffffffffu, p[u][r % RO], (lane & ~(LK - 1)) + from);
                    // a node that row r does not see may hold inf or NaN: 0 * v would keep it
                    if (kTail && nd >= 0 && !(r < rows && nd < a.Ts && ((anc[(r0 + r) / a.G] >> nd) & 1ull)))
                        continue;
#pragma unroll
                    for (int i = 0; i < CP; ++i) acc[r][i] = fma2(pack2(pr, pr), x[i], acc[r][i]);
                }
            }
            pos += 2 * kStep;
            if (++stage == kAhead) stage = 0;
        };
        const int context = (cached_end - w.t0 * kStreamKeys) / (2 * kStep);
        int step = 0;
#pragma unroll 1
        for (; step < context; ++step) keys(std::false_type());
#pragma unroll 1
        for (; step < steps; ++step) keys(std::true_type());
        asm volatile("cp.async.wait_group 0;" ::: "memory");   // the stages are free
        // The groups' maxima, sums and outputs meet: in the warp, then in the CTA.
        float top[RO], sum[RO];
#pragma unroll
        for (int i = 0; i < RO; ++i) {
            if (seen[i] == 0ull) {                  // an unused node
                m[i] = -INFINITY;
                l[i] = 0.f;
            }
            top[i] = m[i];
#pragma unroll
            for (int off = LK; off < 32; off <<= 1) top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], off));
            if (sub == 0) sh_m[warp][own + i] = top[i];
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < RO; ++i) {
#pragma unroll
            for (int k = 0; k < kWarps; ++k) top[i] = fmaxf(top[i], sh_m[k][own + i]);
            const float f = m[i] == -INFINITY ? 0.f : exp2f(m[i] - top[i]);
            sum[i] = l[i] * f;
            m[i] = f;                               // this group's factor
#pragma unroll
            for (int off = LK; off < 32; off <<= 1) sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], off);
            if (sub == 0) sh_l[warp][own + i] = sum[i];
        }
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            const int from = LK >= RT ? r * (LK / RT) : r / RO;
            const float fr = __shfl_sync(0xffffffffu, m[r % RO], (lane & ~(LK - 1)) + from);
            float y[CH];
#pragma unroll
            for (int i = 0; i < CP; ++i) {
                const float2 z = unpack2(acc[r][i]);
                // a group that has seen nothing of a row has an output of 0
                y[2 * i] = fr == 0.f ? 0.f : z.x * fr;
                y[2 * i + 1] = fr == 0.f ? 0.f : z.y * fr;
            }
#pragma unroll
            for (int i = 0; i < CH; ++i)
#pragma unroll
                for (int off = LK; off < 32; off <<= 1) y[i] += __shfl_xor_sync(0xffffffffu, y[i], off);
            if (sub == 0) {
#pragma unroll
                for (int i = 0; i < CH; i += 4)
                    *reinterpret_cast<float4*>(&sh_o[warp][r][CH * g + i]) = make_float4(y[i], y[i + 1], y[i + 2], y[i + 3]);
            }
        }
        __syncthreads();
        // Finished here, or one of the CTA's two pieces.
        const bool whole = w.t0 == 0 && w.t1 == w.tiles;
        float* part = a.part + ((size_t)blockIdx.x * 2 + (w.t0 == 0 ? 1 : 0)) * RT * (D + 2);
        for (int e = tid; e < rows * D; e += kStreamThreads) {
            const int r = e / D, c = e % D;
            float o = 0.f, sl = 0.f, sm = -INFINITY;
#pragma unroll
            for (int k = 0; k < kWarps; ++k) {
                o += sh_o[k][r][c];
                sl += sh_l[k][r];
                sm = fmaxf(sm, sh_m[k][r]);
            }
            const int t = (r0 + r) / a.G, h = (r0 + r) % a.G;
            if (whole) {
                st_f(static_cast<TO*>(a.o) + (((long long)n * a.Ts + t) * a.Hq + hk * a.G + h) * D + c,
                     sl == 0.f ? 0.f : o / sl);     // nothing seen: an unused node
            } else {
                part[e] = o;
                if (c == 0) {
                    part[RT * D + r] = sm;
                    part[RT * D + RT + r] = sl;
                }
            }
        }
    }
}

// More rows: tiles.  128 threads as 8 row groups x 16 columns for 32 query rows:
// thread (ty, tx) owns rows 4 ty .. 4 ty + 3 throughout, their scores for keys tx
// and tx + 16 and D / 16 of their output columns, so that m, l and the rescaling
// stay in registers.  K and V come by cp.async in two stages, one tile ahead;
// page numbers are loaded two tiles before that.  Bound by shared-memory reads
// (6 words of K and q for 8 FMAs) and by the few warps that its registers leave:
// fp32, 8 x 16 nodes, 32 heads on 8, 8 x 4096 rows: d = 128 313 us (27 TFLOP/s),
// d = 64 160 us; 352 and 210 with scalar FMAs and one loop for all keys.  bf16, 16
// heads on 4, 8 x 16 nodes, 8 x 4096 rows: d = 32 64 us, d = 16 48 us.
constexpr int kTileThreads = 128;
constexpr int kTileKeys = 32;
constexpr int kTileRows = 32;
constexpr int kTileLead = 2;
// Per SM.  At d = 128 two and three took 313 and 365 us in fp32 (298 and 271 from
// bf16), at d = 64 three, four and five 172, 160 and 224; below that four to six are
// within 2 %.
__host__ __device__ constexpr int tile_ctas(int D) { return D == 128 ? 2 : (D == 64 ? 4 : 5); }

template <typename TI, int D>
struct TileShape {
    static constexpr int kLdq = D + 4;
    static constexpr int kLdk = D + 16 / (int)sizeof(TI);      // rows stay 16-byte aligned
    static constexpr int kLdp = kTileKeys + 4;
    static constexpr int kStage = kTileKeys * (kLdk + D);       // elements: K, then V
    static constexpr size_t kBytes =
        sizeof(float) * (kTileRows * kLdq + kTileRows * kLdp) + 2 * sizeof(TI) * kStage;
};

template <typename T>
__device__ __forceinline__ float4 load4(const T* p);
template <>
__device__ __forceinline__ float4 load4<float>(const float* p)
{
    return *reinterpret_cast<const float4*>(p);
}
template <>
__device__ __forceinline__ float4 load4<__nv_bfloat16>(const __nv_bfloat16* p)
{
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u),
                       __uint_as_float(u.y << 16), __uint_as_float(u.y & 0xFFFF0000u));
}

template <typename TI, typename TO, int D>
__global__ void __launch_bounds__(kTileThreads, tile_ctas(D))
tree_attention_tile_kernel(const TreeArgs a)
{
    using Sh = TileShape<TI, D>;
    constexpr int RT = kTileRows, RR = RT / 8, KR = kTileKeys / 16, CR = D / 16;
    constexpr int V4 = D / 4, VR = 16 / (int)sizeof(TI);        // elements per 16 bytes
    constexpr int kVecs = D / VR;                               // 16-byte pieces of a row
    extern __shared__ __align__(16) float smem[];
    float* sQ = smem;                               // [RT][kLdq]
    float* sP = sQ + RT * Sh::kLdq;                 // [RT][kLdp]
    TI* stages = reinterpret_cast<TI*>(sP + RT * Sh::kLdp);
    __shared__ long long sh_loc[kTileThreads / 32 + 2];
    __shared__ unsigned long long anc[kTreeMaxNodes];
    __shared__ int32_t up[kTreeMaxNodes];
    __shared__ long long sh_off[4][kTileKeys];      // a key's row in the cache (-1: none), by tile % 4
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const TI* q = static_cast<const TI*>(a.q);

    const int group = blockIdx.x / a.row_tiles, r0 = (blockIdx.x % a.row_tiles) * RT;
    const int rows = a.R - r0 < RT ? a.R - r0 : RT;
    const TreeSpot sp = tree_locate<kTileThreads, kTileKeys, kTileLead>(a, group, sh_loc);
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int row_elems = a.Hkv * D;
    int have = -1;                                  // the sequence anc[] is of

    TreePieces<kTileKeys, kTileLead> w;
    for (bool more = w.start(a, sp, group); more; more = w.next(a)) {
        const int n = w.n, ctx = w.ctx, tiles = w.tiles, t0 = w.t0, t1 = w.t1, hk = w.hk;
        const int32_t* table = a.page_table + (long long)n * a.max_pages;
        __syncthreads();                            // the last piece's tiles and masks have been read
        if (have != n) {
            if (tid < 32)
                tree_masks(a.parent ? a.parent + (long long)n * a.Ts : nullptr, a.Ts, tid, anc, up);
            have = n;
        }
        // The rows of a tile, by one warp: ask() loads their page numbers, put()
        // a tile later turns them into offsets.
        int page = -1, slot = 0;
        auto ask = [&](int t) {
            if (tid < kTileKeys && t < t1) {
                const int pos = t * kTileKeys + tid;
                page = -1;
                if (pos < ctx) {
                    const int p = pos / a.page_size;
                    page = __ldg(table + p);
                    slot = pos - p * a.page_size;
                }
            }
        };
        auto put = [&](int t) {
            if (tid < kTileKeys && t < t1) {
                const int node = t * kTileKeys + tid - ctx;
                long long off = -1;
                if (page >= 0 && page < a.num_pages) off = (long long)page * a.page_stride + (long long)slot * row_elems;
                else if (node >= 0 && node < a.Ts) off = ((long long)n * a.Ts + node) * row_elems;
                sh_off[t & 3][tid] = off;
            }
        };
        auto fetch = [&](int t) {
            if (t < t1) {
                const int nc = ctx - t * kTileKeys;
                TI* sk = stages + (t & 1) * Sh::kStage;
                TI* sv = sk + kTileKeys * Sh::kLdk;
#pragma unroll 4
                for (int e = tid; e < kTileKeys * kVecs; e += kTileThreads) {
                    const int j = e / kVecs, c = (e % kVecs) * VR;
                    const long long off = sh_off[t & 3][j];
                    const TI *kp = q, *vp = q;           // not read
                    if (off >= 0) {
                        kp = static_cast<const TI*>(j >= nc ? a.k : a.k_cache) + off + hk * D + c;
                        vp = static_cast<const TI*>(j >= nc ? a.v : a.v_cache) + off + hk * D + c;
                    }
                    copy16(sk + j * Sh::kLdk + c, kp, off >= 0);
                    copy16(sv + j * D + c, vp, off >= 0);
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        ask(t0);
        put(t0);
        ask(t0 + 1);
        put(t0 + 1);
        ask(t0 + 2);
        for (int e = tid; e < RT * V4; e += kTileThreads) {
            const int r = e / V4, c = e % V4;
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r < rows) {
                const int t = (r0 + r) / a.G, g = (r0 + r) % a.G;
                x = load4(q + (((long long)n * a.Ts + t) * a.Hq + hk * a.G + g) * D + 4 * c);
            }
            *reinterpret_cast<float4*>(sQ + r * Sh::kLdq + 4 * c) =
                make_float4(x.x * a.scale_log2, x.y * a.scale_log2, x.z * a.scale_log2,
                            x.w * a.scale_log2);
        }
        __syncthreads();
        fetch(t0);
        unsigned long long mask[RR];
        float m[RR], l[RR], acc[RR][CR];
#pragma unroll
        for (int i = 0; i < RR; ++i) {
            const int r = ty * RR + i;
            mask[i] = r < rows ? anc[(r0 + r) / a.G] : 0ull;
            m[i] = -INFINITY;
            l[i] = 0.f;
#pragma unroll
            for (int c = 0; c < CR; ++c) acc[i][c] = 0.f;
        }
        for (int t = t0; t < t1; ++t) {
            const int k0 = t * kTileKeys;
            const int nc = ctx - k0;                // key j is drafted node j - nc from j = nc on
            const int nk = nc + a.Ts < kTileKeys ? nc + a.Ts : kTileKeys;
            const bool draft = nc < kTileKeys;      // some are
            fetch(t + 1);
            put(t + 2);
            ask(t + 3);
            asm volatile("cp.async.wait_group 1;" ::: "memory");
            __syncthreads();                        // tile t, and the rows of tile t + 2
            const TI* sK = stages + (t & 1) * Sh::kStage;
            const TI* sV = sK + kTileKeys * Sh::kLdk;
            uint64_t s2[RR][KR];                    // sums of even and odd channels
#pragma unroll
            for (int i = 0; i < RR; ++i)
#pragma unroll
                for (int j = 0; j < KR; ++j) s2[i][j] = 0;
#pragma unroll 4
            for (int c = 0; c < V4; ++c) {
                uint64_t kv[KR][2];
#pragma unroll
                for (int j = 0; j < KR; ++j) {
                    const float4 x = load4(sK + (tx + 16 * j) * Sh::kLdk + 4 * c);
                    kv[j][0] = pack2(x.x, x.y);
                    kv[j][1] = pack2(x.z, x.w);
                }
#pragma unroll
                for (int i = 0; i < RR; ++i) {
                    const float4 x = *reinterpret_cast<const float4*>(sQ + (ty * RR + i) * Sh::kLdq + 4 * c);
#pragma unroll
                    for (int j = 0; j < KR; ++j)
                        s2[i][j] = fma2(pack2(x.z, x.w), kv[j][1], fma2(pack2(x.x, x.y), kv[j][0], s2[i][j]));
                }
            }
            float s[RR][KR];
#pragma unroll
            for (int i = 0; i < RR; ++i)
#pragma unroll
                for (int j = 0; j < KR; ++j) {
                    const float2 y = unpack2(s2[i][j]);
                    s[i][j] = y.x + y.y;
                }
            bool there[KR];                         // context keys whose page exists
#pragma unroll
            for (int j = 0; j < KR; ++j) there[j] = tx + 16 * j < nc && sh_off[t & 3][tx + 16 * j] >= 0;
#pragma unroll
            for (int i = 0; i < RR; ++i) {
                float top = m[i];
#pragma unroll
                for (int j = 0; j < KR; ++j) {
                    const int node = tx + 16 * j - nc;
                    const bool see = node < 0 ? mask[i] != 0ull && there[j]
                                              : node < a.Ts && ((mask[i] >> node) & 1ull);
                    if (!see) s[i][j] = -INFINITY;
                    top = fmaxf(top, s[i][j]);
                }
#pragma unroll
                for (int off = 1; off < 16; off <<= 1)
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
                const float ref = top == -INFINITY ? 0.f : top;
                const float shrink = ex2(m[i] - ref);
                float sum = 0.f;
#pragma unroll
                for (int j = 0; j < KR; ++j) {
                    const float p = ex2(s[i][j] - ref);
                    sP[(ty * RR + i) * Sh::kLdp + tx + 16 * j] = p;
                    sum += p;
                }
#pragma unroll
                for (int off = 1; off < 16; off <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
                l[i] = l[i] * shrink + sum;
                m[i] = top;
#pragma unroll
                for (int c = 0; c < CR; ++c) acc[i][c] *= shrink;
            }
            __syncwarp();                           // a row's P is written and read by one warp
            // column c of this thread: its 4-column groups are 64 apart (d >= 64)
            auto add = [&](int j, const float (&p)[RR], auto drafted) {
                float v[CR];
                if constexpr (CR % 4 == 0) {
#pragma unroll
                    for (int c = 0; c < CR; c += 4) {
                        const float4 x = load4(sV + j * D + c * 16 + tx * 4);
                        v[c] = x.x;
                        v[c + 1] = x.y;
                        v[c + 2] = x.z;
                        v[c + 3] = x.w;
                    }
                } else {
#pragma unroll
                    for (int c = 0; c < CR; ++c) v[c] = ld_f(sV + j * D + tx + 16 * c);
                }
#pragma unroll
                for (int i = 0; i < RR; ++i) {
                    // a node that this row does not see may hold inf or NaN: 0 * v would keep it
                    if (decltype(drafted)::value && j >= nc && (j >= nk || !((mask[i] >> (j - nc)) & 1ull))) continue;
                    if constexpr (CR % 2 == 0) {
#pragma unroll
                        for (int c = 0; c < CR; c += 2) {
                            const float2 y = unpack2(fma2(pack2(p[i], p[i]), pack2(v[c], v[c + 1]),
                                                          pack2(acc[i][c], acc[i][c + 1])));
                            acc[i][c] = y.x;
                            acc[i][c + 1] = y.y;
                        }
                    } else {
#pragma unroll
                        for (int c = 0; c < CR; ++c) acc[i][c] = fmaf(p[i], v[c], acc[i][c]);
                    }
                }
            };
            auto products = [&](auto drafted) {
#pragma unroll 2
                for (int j = 0; j < kTileKeys; j += 4) {
                    float p[4][RR];
#pragma unroll
                    for (int i = 0; i < RR; ++i) {
                        const float4 x = *reinterpret_cast<const float4*>(sP + (ty * RR + i) * Sh::kLdp + j);
                        p[0][i] = x.x;
                        p[1][i] = x.y;
                        p[2][i] = x.z;
                        p[3][i] = x.w;
                    }
#pragma unroll
                    for (int jj = 0; jj < 4; ++jj) add(j + jj, p[jj], drafted);
                }
            };
            if (draft) products(std::true_type());
            else products(std::false_type());
            __syncthreads();                        // tile t has been read: its stage is free
        }
        // Finished here, or one of the CTA's two pieces.
        const bool whole = t0 == 0 && t1 == tiles;
        float* part = a.part + ((size_t)blockIdx.x * 2 + (t0 == 0 ? 1 : 0)) * RT * (D + 2);
#pragma unroll
        for (int i = 0; i < RR; ++i) {
            const int r = ty * RR + i;
            if (r >= rows) continue;
            const int t = (r0 + r) / a.G, g = (r0 + r) % a.G;
            TO* op = static_cast<TO*>(a.o) + (((long long)n * a.Ts + t) * a.Hq + hk * a.G + g) * D;
            const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];
#pragma unroll
            for (int c = 0; c < CR; ++c) {
                const int col = CR % 4 == 0 ? (c / 4) * 64 + tx * 4 + c % 4 : tx + 16 * c;
                if (whole) st_f(op + col, mask[i] ? acc[i][c] * inv : 0.f);
                else part[r * D + col] = acc[i][c];
            }
            if (!whole && tx == 0) {
                part[RT * D + r] = m[i];
                part[RT * D + RT + r] = l[i];
            }
        }
    }
}

// Joins the pieces of the items that were cut between groups.  Block (c, y, z):
// the item that the boundary before group c + 1 falls into, if that is the
// item's first boundary; rows y 8 .. y 8 + 7 of row tile z.  The pieces are read
// in the order of the groups, so the result does not depend on timing.  The
// launch may start before the attention kernel has ended (its blocks fill the
// SMs that have finished) and waits for it before the first partial result.
constexpr int kJoinThreads = 256;
constexpr int kJoinRows = 8;

template <typename TO, int D, int KT, int LEAD>
__global__ void __launch_bounds__(kJoinThreads)
tree_join_kernel(const TreeArgs a, int RT)
{
    __shared__ long long sh_loc[kJoinThreads / 32 + 2];
    const int c = blockIdx.x + 1, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const TreeSpot sp = tree_locate<kJoinThreads, KT, LEAD>(a, c, sh_loc);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const long long at = tree_begin(sp, c);
    if (at >= sp.total) return;                     // an empty range at the end
    const int tiles = tree_tiles<KT>(a, sp.n);
    const int hk = (int)((at - sp.start) / (tiles + LEAD));
    // where the item's tiles begin; a boundary up to there cuts nothing
    const long long first = sp.start + (long long)hk * (tiles + LEAD) + LEAD;
    if (at <= first || tree_begin(sp, c - 1) > first) return;
    int last = c;                                   // the last group with tiles of this item
    while (last + 1 < a.groups && tree_begin(sp, last + 1) < first + tiles) ++last;
    const int r0 = blockIdx.z * RT;
    const int rows = a.R - r0 < RT ? a.R - r0 : RT;
    const int r = blockIdx.y * kJoinRows + warp;    // a warp per row
    if (r >= rows) return;
    const size_t slot = (size_t)RT * (D + 2);
    // piece p of the item: group p's first slot, but the second of group c - 1
    auto piece = [&](int p) {
        return a.part + (((size_t)p * a.row_tiles + blockIdx.z) * 2 + (p == c - 1 ? 1 : 0)) * slot;
    };
    constexpr int E = D / 32 > 0 ? D / 32 : 1;      // elements per lane
    float m = -INFINITY;
    for (int p = c - 1 + lane; p <= last; p += 32) m = fmaxf(m, piece(p)[RT * D + r]);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    const float ref = m == -INFINITY ? 0.f : m;
    float l = 0.f, o[E];
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.f;
#pragma unroll 4
    for (int p = c - 1; p <= last; ++p) {
        const float* x = piece(p);
        const float w = exp2f(x[RT * D + r] - ref);
        l = fmaf(x[RT * D + RT + r], w, l);
#pragma unroll
        for (int e = 0; e < E; ++e)
            if ((D >= 32 || lane < D) && w != 0.f)   // w = 0: o may be anything (an unused node)
                o[e] = fmaf(x[(size_t)r * D + lane + 32 * e], w, o[e]);
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;     // l = 0: an unused node; a NaN stays
    const int t = (r0 + r) / a.G, g = (r0 + r) % a.G;
    TO* op = static_cast<TO*>(a.o) + (((long long)sp.n * a.Ts + t) * a.Hq + hk * a.G + g) * D;
#pragma unroll
    for (int e = 0; e < E; ++e)
        if (D >= 32 || lane < D) st_f(op + lane + 32 * e, o[e] * inv);
}

template <typename TO, int D, int KT, int LEAD>
cudaError_t launch_join(const TreeArgs& a, int rt, cudaStream_t stream)
{
    if (a.groups < 2) return cudaSuccess;
    const int rows = a.R < rt ? a.R : rt;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.groups - 1, (rows + kJoinRows - 1) / kJoinRows, a.row_tiles);
    cfg.blockDim = dim3(kJoinThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, tree_join_kernel<TO, D, KT, LEAD>, a, rt);
}

template <typename TI, typename TO, int D>
cudaError_t launch_d(const TreeArgs& a, int rt, cudaStream_t stream)
{
    const bool stream_kernel = rt == kStreamRows;
    auto kern = stream_kernel ? tree_attention_stream_kernel<TI, TO, D> : tree_attention_tile_kernel<TI, TO, D>;
    const size_t bytes = stream_kernel ? (size_t)kAhead * 4 * kStreamThreads * 16
                                       : TileShape<TI, D>::kBytes;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e != cudaSuccess) return e;
    kern<<<a.groups * a.row_tiles, stream_kernel ? kStreamThreads : kTileThreads, bytes, stream>>>(a);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return stream_kernel ? launch_join<TO, D, kStreamKeys, kStreamLead>(a, rt, stream)
                         : launch_join<TO, D, kTileKeys, kTileLead>(a, rt, stream);
}

template <typename TI, typename TO>
cudaError_t launch_typed(const TreeArgs& a, int rt, int d, cudaStream_t stream)
{
    switch (d) {
        case 16: return launch_d<TI, TO, 16>(a, rt, stream);
        case 32: return launch_d<TI, TO, 32>(a, rt, stream);
        case 64: return launch_d<TI, TO, 64>(a, rt, stream);
        case 128: return launch_d<TI, TO, 128>(a, rt, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace

TreePlan tree_plan(int32_t Ts, int32_t Hq, int32_t Hkv, int32_t d, bool fp32, int sms, bool tc)
{
    const int R = Ts * (Hq / Hkv);
    TreePlan p;
    p.tc = tc;
    // Tensor cores: two row tiles on one CTA share its keys.  Always one and always
    // two, 4 x 65,536 rows, us: 64 rows 183 and 194, 128 rows 196 and 207, 132 rows
    // 273 and 225, 256 rows 281 and 261, 512 rows 524 and 426.  CUDA cores: the
    // stream takes what eight rows in registers allow.
    p.rt = tc ? (R <= 128 ? 128 : 256) : (R <= kStreamRows ? kStreamRows : kTileRows);
    p.row_tiles = (R + p.rt - 1) / p.rt;
    const int ctas = (sms > 0 ? sms : 1) * (tc ? 1 : p.rt == kStreamRows ? stream_ctas(fp32) : tile_ctas(d));
    p.groups = ctas / p.row_tiles > 1 ? ctas / p.row_tiles : 1;
    return p;
}

// The tensor-core kernel takes bf16 with d = 64 or 128 and bf16 output (its
// probabilities are rounded to bf16, which an fp32 output would show).  It takes
// few rows too, although most of a 128-row product is then empty: 4 rows, 64 x
// 4,096 keys, 179 us against the stream's 333, 256 x 512 146 against 222, one
// sequence of 1,023 keys 19 and 21.
bool tree_tc_supported(int32_t d, kda_dtype_t dtype)
{
    return dtype == KDA_BF16 && (d == 64 || d == 128);
}

size_t tree_workspace_bytes(int32_t Ts, int32_t Hq, int32_t Hkv, int32_t d, kda_dtype_t dtype, int sms)
{
    size_t most = 0;
    for (int tc = 0; tc <= (int)tree_tc_supported(d, dtype); ++tc) {
        const TreePlan p = tree_plan(Ts, Hq, Hkv, d, dtype == KDA_FP32, sms, tc != 0);
        const size_t b = (size_t)p.groups * p.row_tiles * 2 * p.rt * (d + 2) * sizeof(float);
        if (b > most) most = b;
    }
    return kWsHeaderBytes + most;
}

// A scale that is not positive takes the CUDA-core kernel: the tensor-core one
// finds a row's maximum before it applies the scale.
cudaError_t launch_tree_attention(TreeArgs args, int32_t d, kda_dtype_t dtype, int sms,
                                  cudaStream_t stream)
{
    const bool tc = tree_tc_supported(d, dtype) && args.scale_log2 > 0.f && getenv("KDA_FORCE_SIMT") == nullptr;
    const TreePlan plan = tree_plan(args.Ts, args.Hq, args.Hkv, d, dtype == KDA_FP32, sms, tc);
    args.groups = plan.groups;
    args.row_tiles = plan.row_tiles;
    if (plan.tc) {
        const cudaError_t e = launch_tree_attention_tc(args, plan, d, stream);
        if (e != cudaSuccess) return e;
        return d == 64 ? launch_join<__nv_bfloat16, 64, kTcKeys, kTcLead>(args, plan.rt, stream)
                       : launch_join<__nv_bfloat16, 128, kTcKeys, kTcLead>(args, plan.rt, stream);
    }
    switch (dtype) {
        case KDA_BF16: return launch_typed<__nv_bfloat16, __nv_bfloat16>(args, plan.rt, d, stream);
        case KDA_BF16_F32OUT: return launch_typed<__nv_bfloat16, float>(args, plan.rt, d, stream);
        default: return launch_typed<float, float>(args, plan.rt, d, stream);
    }
}

}  // namespace kda
