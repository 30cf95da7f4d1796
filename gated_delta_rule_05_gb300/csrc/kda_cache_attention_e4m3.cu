// kda_cache_attention_e4m3.cu -- attention of a sequence's newest tokens to a paged
// cache of 8-bit keys and values with a scale per block of rows and head.
//
// Per 16 keys and 16 query rows (the Ts G rows that share a cache head), one warp:
//     S = Q K^T, s = c ks S (c = scale log2 e, ks the key's scale)
//     P = 2^(s - m), w = P vs 2^(m - n) (vs the value's scale), O += w V
// on mma.sync m16n8k16 with K and V widened to fp16 in registers, which holds e4m3
// exactly.  m is a reference near the running maximum of s of each row, n one 2^7 below that of s + log2
// vs: P stays below 2^8 and w below 2^15, in fp16's range whatever the scales are, and w's largest is 2^7
// at least, so that the weights of many keys far below one keep their bits (kda_f16_parts.cuh); O
// is in units of 2^n, the sum l of P in units of 2^m.  They move only when a score
// exceeds them by more than 8, so that a step without that has no reduction over lanes.
// q is brought into fp16's range by a power of two per row, which is exact.  With
// fp32 queries or output, q and w are a sum of two fp16 each (22 bits, hi + 2^-11 lo), and as the tensor
// cores cut off what does not fit as they add up (1e-5 of the result over 32,000 keys), the small
// products and each group's output have sums of their own.
//
// The tensor-core instruction of one thread and TMEM is not used: with 4 to 16 rows
// most of its 128 would be empty, and 8-bit products would need q and w in 8 bits.
//
// A warp has every 8th group of 16 keys of its thread block's range and a ring of
// its own, filled by cp.async a few groups ahead: no barrier until the end of an
// item's part, where the warps' (O, m, n, l) are joined in shared memory.  The rows
// lie in the ring so that the 16-byte reads below find all banks.
//
// The work is cut into equal ranges as for the tree attention (kda_tree.cuh).
#include <cudaTypedefs.h>
#include <stdio.h>

#include "kda_f16_parts.cuh"
#include "kda_prompt.cuh"
#include "kda_sm100.cuh"

namespace kda {

// The driver's tensor-map encoder (kda_prefill_tc.cu).
PFN_cuTensorMapEncodeTiled_v12000 tc_encode_fn();

namespace {

using sm100::fence_mbar_init;
using sm100::fence_proxy_async_smem;
using sm100::mbar_arrive;
using sm100::mbar_arrive_expect_tx;
using sm100::mbar_init;
using sm100::mbar_try_wait;
using namespace f16_parts;

constexpr int kWarps = 8, kThreads = kWarps * 32;
constexpr int kKeys = 16;                          // of a warp's step
constexpr int KT = kWarps * kKeys;                 // of a tile
constexpr int kLead = 4;
constexpr int kRows = 16;
constexpr uint32_t kInfinity = 0x7F800000u;
constexpr float kNaN = __builtin_nanf("");
using Piece = TreePieces<KT, kLead>;

template <int D>
struct Shape {
    static constexpr int kStageBytes = 2 * kKeys * D + 2 * kKeys * 4 + 16;
    static constexpr int kStages = D == 128 ? 4 : 6;
    static constexpr int kRing = kWarps * kStages * kStageBytes;
    static constexpr int OP = D + 4;               // row pitch of a warp's O
    static constexpr int kJoin = kWarps * (kRows * OP + 3 * kRows) * 4;
    static constexpr size_t kBytes = kRing + kJoin;
};

__device__ __forceinline__ float lg2(float x)
{
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src, bool there)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(there ? 4 : 0) : "memory");
}
// Two e4m3 (the lower or the upper half of a word) as fp16, which holds them exactly.
__device__ __forceinline__ uint32_t widen_lo(uint32_t w)
{
    uint32_t r;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(r) : "r"(w));
    return r;
}
__device__ __forceinline__ uint32_t widen_hi(uint32_t w)
{
    uint32_t r;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(r) : "r"(w));
    return r;
}
template <int BYTES>
struct Words {
    uint32_t w[(BYTES + 3) / 4];
};
template <int BYTES>
__device__ __forceinline__ Words<BYTES> read_words(uint32_t at)
{
    Words<BYTES> r;
    if constexpr (BYTES == 16)
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3]) : "r"(at));
    else if constexpr (BYTES == 8)
        asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(r.w[0]), "=r"(r.w[1]) : "r"(at));
    else if constexpr (BYTES == 4)
        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(r.w[0]) : "r"(at));
    else
        asm volatile("{\n\t.reg .b16 h;\n\tld.shared.b16 h, [%1];\n\tmov.b32 %0, {h, 0};\n\t}" : "=r"(r.w[0]) : "r"(at));
    return r;
}
__device__ __forceinline__ float read_float(uint32_t at)
{
    float x;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(x) : "r"(at));
    return x;
}

// Byte offset of 16-byte piece c of row `key` of a step's 16 rows.
template <int D>
__device__ __forceinline__ int row_at(int key, int c)
{
    if constexpr (D == 128) return key * 128 + ((c ^ (key & 7)) << 4);
    else if constexpr (D == 64) return key * 64 + ((c ^ ((key >> 1) & 3)) << 4);
    else return key * D + (c << 4);
}
// The key of a step that is column n of the first product's 8-key half, and the
// first of the channels that are column n of the second product's D / 8 blocks.
// Column pairs (2 i, 2 i + 1) are keys i and i + 4.
__device__ __forceinline__ int key_of(int n) { return ((n & 1) << 2) | (n >> 1); }
template <int D>
__device__ __forceinline__ int channel_of(int n) { return key_of(n) * (D / 8); }

// The walk of a warp's copies over its range: a step (16 keys) at a time, this
// lane's key (lane % 16) in it; the page number is loaded when the step is entered, one
// before it is used.
struct Walk {
    Piece w;
    bool go;
    int t, pos, p, slot, page;

    __device__ __forceinline__ void look_up(const E4m3Args& a)
    {
        page = -1;
        if (go && pos < w.ctx) page = __ldg(a.split.page_table + (long long)w.n * a.split.max_pages + p);
    }
    __device__ __forceinline__ void enter(const E4m3Args& a, int warp, int lane)
    {
        if (go) {
            t = w.t0;
            pos = t * KT + warp * kKeys + (lane & 15);
            p = pos / a.split.page_size;
            slot = pos - p * a.split.page_size;
        }
        look_up(a);
    }
    __device__ __forceinline__ void step(const E4m3Args& a, int warp, int lane)
    {
        if (!go) return;
        if (++t == w.t1) {
            go = w.next(a.split);
            enter(a, warp, lane);
            return;
        }
        pos += KT;
        p += a.tile_pages;
        slot += a.tile_rows;
        if (slot >= a.split.page_size) {
            slot -= a.split.page_size;
            ++p;
        }
        look_up(a);
    }
};

// Starts the copies of the walk's step into a stage.
template <int D>
__device__ __forceinline__ void start_copies(const E4m3Args& a, const Walk& k, uint32_t stage, int lane)
{
    constexpr int CPR = D / 16;                    // 16-byte pieces of a row
    if (k.go) {
        const bool there = k.page >= 0 && k.page < a.num_pages;
        const uint32_t mask = __ballot_sync(0xffffffffu, there) & 0xFFFFu;
        long long row = 0;
        const float* scale = lane < 16 ? a.k_scales : a.v_scales;
        if (there) {
            row = k.page * a.page_stride + (long long)k.slot * (a.Hkv * D) + k.w.hk * D;
            const int b = a.block == 1 ? k.slot : (int)__umulhi((uint32_t)k.slot, a.block_magic);
            scale += ((long long)k.page * a.blocks + b) * a.Hkv + k.w.hk;
        }
        copy4(stage + 2 * kKeys * D + lane * 4, scale, there);
        if (lane == 0) asm volatile("st.shared.b32 [%0], %1;" ::"r"(stage + 2 * kKeys * D + 128), "r"(mask) : "memory");
        constexpr int N = kKeys * CPR;
#pragma unroll
        for (int e0 = 0; e0 < N; e0 += 32) {
            const int e = e0 + lane, key = e / CPR, c = e % CPR;
            const long long src = __shfl_sync(0xffffffffu, row, key & 15);
            const bool ok = (mask >> (key & 15)) & 1;
            if (N >= 32 || e < N) {
                copy16(stage + row_at<D>(key, c), a.k_cache + src + c * 16, ok);
                copy16(stage + kKeys * D + row_at<D>(key, c), a.v_cache + src + c * 16, ok);
            }
        }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
}

__device__ __forceinline__ void load4(const float* p, float (&x)[4])
{
    const float4 w = __ldg(reinterpret_cast<const float4*>(p));
    x[0] = w.x, x[1] = w.y, x[2] = w.z, x[3] = w.w;
}
__device__ __forceinline__ void load4(const __nv_bfloat16* p, float (&x)[4])
{
    const uint2 w = __ldg(reinterpret_cast<const uint2*>(p));
    x[0] = __uint_as_float(w.x << 16), x[1] = __uint_as_float(w.x & 0xFFFF0000u);
    x[2] = __uint_as_float(w.y << 16), x[3] = __uint_as_float(w.y & 0xFFFF0000u);
}

// The channel of word s (4 channels) that lane i of a row's four holds.
template <int D>
__device__ __forceinline__ int q_channel(int s, int i)
{
    return D == 128 ? 64 * (s >> 2) + 16 * i + 4 * (s & 3) : D / 4 * i + 4 * s;
}

template <class T, class O, int D>
__global__ void __launch_bounds__(kThreads, 1)
cache_attention_kernel(const __grid_constant__ E4m3Args a)
{
    using Sh = Shape<D>;
    constexpr bool QLO = sizeof(T) == 4, PLO = sizeof(O) == 4;
    constexpr int KS = D / 16;                     // steps of 16 channels of the first product
    constexpr int NT = D / 8;                      // blocks of 8 channels of the second
    extern __shared__ __align__(128) uint8_t dyn[];
    __shared__ long long sh_loc[kWarps + 2];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, i4 = lane & 3;
    const int group = blockIdx.x / a.split.row_tiles, r0 = (blockIdx.x % a.split.row_tiles) * kRows;
    const TreeSpot sp = tree_locate<kThreads, KT, kLead>(a.split, group, sh_loc);
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    Walk ahead;
    ahead.go = ahead.w.start(a.split, sp, group);
    Piece w = ahead.w;
    bool go = ahead.go;
    ahead.enter(a, warp, lane);
    const uint32_t ring = smem_at(dyn) + warp * Sh::kStages * Sh::kStageBytes;
    float* join = reinterpret_cast<float*>(dyn + Sh::kRing);
    int in = 0, out = 0;                           // stages
#pragma unroll 1
    for (int i = 0; i < Sh::kStages - 1; ++i) {
        start_copies<D>(a, ahead, ring + in * Sh::kStageBytes, lane);
        ahead.step(a, warp, lane);
        in = in + 1 == Sh::kStages ? 0 : in + 1;
    }
    const ScaleParts scale = scale_parts(a.scale_log2);
    for (; go; go = w.next(a.split)) {
        // the rows' queries, in fp16 times a power of two
        uint32_t qh[KS][4], ql[QLO ? KS : 1][4];
        float rs[2];
        int lim[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = r0 + g + 8 * h, t = r / a.G;
            const bool mine = r < a.R;
            lim[h] = mine ? w.ctx - a.Ts + t + 1 : 0;
            const T* qp = static_cast<const T*>(a.q) +
                          (((long long)w.n * a.Ts + (mine ? t : 0)) * a.Hq + w.hk * a.G + (mine ? r - t * a.G : 0)) * D;
            float x[KS][4];
            uint32_t top = 0;
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                x[s][0] = x[s][1] = x[s][2] = x[s][3] = 0.f;
                if (mine) load4(qp + q_channel<D>(s, i4), x[s]);
            }
#pragma unroll
            for (int s = 0; s < KS; ++s)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    x[s][j] *= scale.pre;
                    top = top_of(top, x[s][j]);
                }
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const int e = up_of(top);
            const float up = power(e);
            rs[h] = copysignf(scale.rest * power(-e), a.scale_log2);
            if (top >= kInfinity) rs[h] = kNaN;    // (scores of -inf alone would count as no rows)
#pragma unroll
            for (int s = 0; s < KS; ++s)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float u = x[s][2 * j] * up, v = x[s][2 * j + 1] * up;
                    qh[s][2 * j + h] = two_f16(u, v);
                    if constexpr (QLO) ql[s][2 * j + h] = two_f16_rest(u, v, qh[s][2 * j + h]);
                }
        }
        const int all = w.ctx - a.Ts + r0 / a.G + 1;           // keys that every row sees
        float o[NT][4], m[2], n[2], l[2], fac[2];
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int c = 0; c < 4; ++c) o[j][c] = 0.f;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            m[h] = n[h] = -INFINITY;
            l[h] = fac[h] = 0.f;
        }
#pragma unroll 1
        for (int t = w.t0; t < w.t1; ++t) {
            asm volatile("cp.async.wait_group %0;" ::"n"(Sh::kStages - 2) : "memory");
            __syncwarp();                          // of all lanes; and the stage before has been read
            start_copies<D>(a, ahead, ring + in * Sh::kStageBytes, lane);
            ahead.step(a, warp, lane);
            in = in + 1 == Sh::kStages ? 0 : in + 1;
            const uint32_t st = ring + out * Sh::kStageBytes, sc = st + 2 * kKeys * D;
            out = out + 1 == Sh::kStages ? 0 : out + 1;

            float c[2][4], small[2][4];
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int j = 0; j < 4; ++j) c[b][j] = small[b][j] = 0.f;
            {
                constexpr int KB = D / 4 < 16 ? D / 4 : 16;    // bytes per read of a row of K
                Words<KB> kw[2][D / 4 / KB];
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int h = 0; h < D / 4 / KB; ++h) {
                        const int at = KB * i4 + 64 * h;
                        kw[b][h] = read_words<KB>(st + row_at<D>(8 * b + key_of(g), at >> 4) + (at & 15));
                    }
#pragma unroll
                for (int s = 0; s < KS; ++s)
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        const uint32_t x = kw[b][s / (KB / 4)].w[s % (KB / 4)];
                        const uint32_t b0 = widen_lo(x), b1 = widen_hi(x);
                        mma(c[b], qh[s], b0, b1);
                        if constexpr (QLO) mma(small[b], ql[s], b0, b1);
                    }
            }
            float ks[2][2], vs[2][2];              // of keys 8 b + i4 + 4 j
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    ks[b][j] = read_float(sc + (8 * b + i4 + 4 * j) * 4);
                    vs[b][j] = read_float(sc + (16 + 8 * b + i4 + 4 * j) * 4);
                }
            uint32_t mask;
            asm volatile("ld.shared.b32 %0, [%1];" : "=r"(mask) : "r"(sc + 128));
            const int pos = t * KT + warp * kKeys;
            const bool masked = mask != 0xFFFFu || pos + kKeys > all;      // (the same for the warp)
            bool grow = false;
            float top[2], vtop[2], lv[2][2];
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int j = 0; j < 2; ++j) lv[b][j] = lg2(vs[b][j]);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                top[h] = vtop[h] = -INFINITY;
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        float& x = c[b][2 * h + j];
                        // (by both factors at once: with one of them alone it may not fit)
                        x = (QLO ? fmaf(small[b][2 * h + j], kRest, x) : x) * (ks[b][j] * rs[h]);
                        const int key = 8 * b + i4 + 4 * j;
                        if (masked && (!((mask >> key) & 1) || pos + key >= lim[h])) x = -INFINITY;
                        top[h] = fmaxf(top[h], x);
                        vtop[h] = fmaxf(vtop[h], x + lv[b][j]);
                    }
                grow |= top[h] > m[h] + kSlack || vtop[h] > n[h] + (kSlack + kHead);
            }
            if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float m2 = fmaxf(m[h], quad_max(top[h]));
                    // n is kept near m, so that 2^(m - n) is finite
                    const float n2 = fmaxf(fmaxf(n[h], quad_max(vtop[h]) - kHead), m2 - 120.f);
                    const float fl = m2 == -INFINITY ? 1.f : ex2(m[h] - m2), fo = n2 == -INFINITY ? 1.f : ex2(n[h] - n2);
                    m[h] = m2;
                    n[h] = n2;
                    l[h] *= fl;
                    fac[h] = m2 == -INFINITY ? 0.f : ex2(m2 - n2);
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
                        o[j][2 * h] *= fo;
                        o[j][2 * h + 1] *= fo;
                    }
                }
            }
            uint32_t ph[4], pl[4];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float ref = m[h] == -INFINITY ? 0.f : m[h];
                float sum = 0.f;                   // (few additions to l, which small probabilities would be lost in)
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    float y[2];
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const float x = c[b][2 * h + j];
                        const float p = ex2(x - ref);
                        sum += p;
                        y[j] = p * weight_factor(vs[b][j], fac[h]);
                        if (masked && x == -INFINITY) y[j] = 0.f;
                    }
                    ph[2 * b + h] = two_f16(y[0], y[1]);
                    if constexpr (PLO) pl[2 * b + h] = two_f16_rest(y[0], y[1], ph[2 * b + h]);
                }
                l[h] += sum;
            }
            {
                // this lane's D / 8 channels of keys i4, i4 + 4, 8 + i4, 12 + i4
                Words<NT> vw[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int at = channel_of<D>(g);
                    vw[j] = read_words<NT>(st + kKeys * D + row_at<D>(i4 + 4 * j, at >> 4) + (at & 15));
                }
#pragma unroll
                for (int x = 0; x < (NT + 3) / 4; ++x) {
                    const uint32_t lo0 = __byte_perm(vw[0].w[x], vw[1].w[x], 0x5140), hi0 = __byte_perm(vw[0].w[x], vw[1].w[x], 0x7362);
                    const uint32_t lo1 = __byte_perm(vw[2].w[x], vw[3].w[x], 0x5140), hi1 = __byte_perm(vw[2].w[x], vw[3].w[x], 0x7362);
                    const uint32_t b0[4] = {widen_lo(lo0), widen_hi(lo0), widen_lo(hi0), widen_hi(hi0)};
                    const uint32_t b1[4] = {widen_lo(lo1), widen_hi(lo1), widen_lo(hi1), widen_hi(hi1)};
#pragma unroll
                    for (int j = 0; j < (NT < 4 ? NT : 4); ++j) {
                        if constexpr (PLO) {
                            float z[4], rest[4];
                            mma0(rest, pl, b0[j], b1[j]);
                            mma0(z, ph, b0[j], b1[j]);
#pragma unroll
                            for (int e = 0; e < 4; ++e) o[4 * x + j][e] += fmaf(rest[e], kRest, z[e]);
                        } else {
                            mma(o[4 * x + j], ph, b0[j], b1[j]);
                        }
                    }
                }
            }
        }
        // the warps' results of the piece
        __syncthreads();                           // those of the piece before have been read
        float* wj = join + warp * (kRows * Sh::OP + 3 * kRows);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
            const int r = g + 8 * h;
            if (i4 == 0) {
                wj[kRows * Sh::OP + r] = m[h];
                wj[kRows * Sh::OP + kRows + r] = n[h];
                wj[kRows * Sh::OP + 2 * kRows + r] = l[h];
            }
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int e = 0; e < 2; ++e) wj[r * Sh::OP + channel_of<D>(2 * i4 + e) + j] = o[j][2 * h + e];
        }
        __syncthreads();
        const bool whole = w.t0 == 0 && w.t1 == w.tiles;
        {
            constexpr int E = D / 16;              // channels per thread
            const int r = tid >> 4, c0 = (tid & 15) * E;
            float mm = -INFINITY, nn = -INFINITY, ll = 0.f, oo[E];
#pragma unroll
            for (int e = 0; e < E; ++e) oo[e] = 0.f;
#pragma unroll
            for (int x = 0; x < kWarps; ++x) {
                const float* y = join + x * (kRows * Sh::OP + 3 * kRows) + kRows * Sh::OP;
                mm = fmaxf(mm, y[r]);
                nn = fmaxf(nn, y[kRows + r]);
            }
            const float mr = mm == -INFINITY ? 0.f : mm, nr = nn == -INFINITY ? 0.f : nn;
#pragma unroll
            for (int x = 0; x < kWarps; ++x) {
                const float* y = join + x * (kRows * Sh::OP + 3 * kRows);
                ll += y[kRows * Sh::OP + 2 * kRows + r] * ex2(y[kRows * Sh::OP + r] - mr);
                const float f = ex2(y[kRows * Sh::OP + kRows + r] - nr);
#pragma unroll
                for (int e = 0; e < E; ++e) oo[e] += y[r * Sh::OP + c0 + e] * f;
            }
            const int row = r0 + r;
            if (row < a.R) {
                if (whole) {
                    const int t = row / a.G;
                    const float f = ll == 0.f ? 0.f : ex2(nr - mr) / ll;
                    O* op = static_cast<O*>(a.o) + (((long long)w.n * a.Ts + t) * a.Hq + w.hk * a.G + row - t * a.G) * D + c0;
#pragma unroll
                    for (int e = 0; e < E; ++e) op[e] = O(oo[e] * f);
                } else {
                    float* part = a.part + ((size_t)blockIdx.x * 2 + (w.t0 == 0 ? 1 : 0)) * kRows * (D + 3);
#pragma unroll
                    for (int e = 0; e < E; ++e) part[r * D + c0 + e] = oo[e];
                    if ((tid & 15) == 0) {
                        part[kRows * D + r] = mm;
                        part[kRows * D + kRows + r] = nn;
                        part[kRows * D + 2 * kRows + r] = ll;
                    }
                }
            }
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
}

// ------------------------------------------------- whole groups of rows, one scale each
// The same where SUB = 16 or 8 rows from a multiple of SUB on lie in one page and one
// block of scales: a warp's step is two groups of 16 keys, whose keys and values come as
// TMA boxes of SUB rows with one scale each, so that s = (c ks) S is one factor per row
// and box and the step has half the instructions per key.  The pages' boxes come in the
// swizzle of their row size, which is that of row_at above.
//
// An item is a sequence and 1, 2, 4 or 8 of its cache heads, side by side: warp w has head w
// % heads and every 8 / heads-th step of 32 keys.  With 8 the thread block reads whole rows
// of the cache, and a head's sums stay in one warp: nothing to join at an item's end.  But
// there are fewer items, and each one's pieces (below) are read by the join kernel in turn: so the
// most heads with at most kMostCuts thread blocks to an item.  64 x 1 token on up to 32,000
// rows, 16 x 1 on 16,000, 256 x 1 on 100 to 900, 1 x 1 on 2,047 (8 cache heads, d = 128, us):
// one head 376, 102.8, 103.9, 12.1; this rule 344 (94 % of HBM), 95.5 (82 %), 61.5 (65 %),
// 12.4; 8 heads always 344, 98.3, 61.6, 35.2.
//
// With d = 128 the instances for an fp32 output spill 64 to 150 bytes to local memory (some 145 us for
// 16 x 1 fp32 token on 16,000 rows, where bf16 takes 96); those for bf16 do not.
//
// Against the kernel above, which takes any page and block, 414, 111, 107, 16.0; boxes of 8
// rows where 16 would do 377, 103, 66, 12.7.  More warps with shorter rings (12 x 4 slots)
// took 414 instead of 374 then, two thread blocks of 4 warps 399 instead of 377.
constexpr int kStepGroups = 2;
constexpr int kStepKeys = kStepGroups * kKeys;
// Lead of 1, 2, 4 and 8 tiles (of one head), us: 32 x 4 tokens, contexts of 100 to 16,384
// rows, 127.5, 116.3, 118.0 and 122.6; 64 x 1 token 385.6, 383.7, 387.2 and 395.8.
constexpr int kGroupLead = 2;
constexpr int kMostCuts = 4;                       // 1 and 16: 32 x 4 tokens 114 and 110 us, 4: 104
constexpr int kSlots = 6;                          // groups of a warp's ring
using GroupPiece = TreePieces<0, kGroupLead>;

template <int D>
struct GroupShape {
    static constexpr int kSlotBytes = 2 * kKeys * D;
    static constexpr int kRing = kWarps * kSlots * kSlotBytes;
    static constexpr int kFrag = 32 * (D / 2);     // floats of a warp's O
    static constexpr int kJoin = kWarps / 2 * (kFrag + 3 * kRows) * 4;
    static constexpr size_t kBytes = 1024 + kRing + kJoin;
};

__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap* map, int h, int row, int page, uint64_t* bar)
{
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(h), "r"(row), "r"(page), "r"(smem_at(bar))
        : "memory");
}

// The cache head of a warp.
__device__ __forceinline__ int head_of(const E4m3Args& a, const GroupPiece& w, int warp)
{
    return (w.hk << a.heads_log) + (warp & ((1 << a.heads_log) - 1));
}

// The walk of a warp's copies, a step at a time; a lane's part of it is box lane %
// kBoxes of the step, whose page number is loaded when the step is entered, one before
// it is used.
template <int SUB>
struct GroupWalk {
    static constexpr int kBoxes = kStepGroups * kKeys / SUB;
    GroupPiece w;
    bool go;
    int t, pos, p, slot, page;

    __device__ __forceinline__ void look_up(const E4m3Args& a)
    {
        page = -1;
        if (go && pos < w.ctx) page = __ldg(a.split.page_table + (long long)w.n * a.split.max_pages + p);
    }
    __device__ __forceinline__ void enter(const E4m3Args& a, int warp, int lane)
    {
        if (go) {
            t = w.t0;
            pos = (t << a.split.tile_log) + (warp >> a.heads_log) * kStepKeys + lane % kBoxes * SUB;
            p = pos / a.split.page_size;
            slot = pos - p * a.split.page_size;
        }
        look_up(a);
    }
    __device__ __forceinline__ void step(const E4m3Args& a, int warp, int lane)
    {
        if (!go) return;
        if (++t == w.t1) {
            go = w.next(a.split);
            enter(a, warp, lane);
            return;
        }
        pos += 1 << a.split.tile_log;
        p += a.tile_pages;
        slot += a.tile_rows;
        if (slot >= a.split.page_size) {
            slot -= a.split.page_size;
            ++p;
        }
        look_up(a);
    }
};

struct GroupShared {
    uint64_t full[kWarps][kSlots];
    int scale[kWarps][kSlots][2];                  // of a box: the place of its scales; -1: no rows
    long long loc[kWarps + 2];
    int dead;
};

// Starts the copies of the walk's step into two slots, a box by a lane.  What no row fills
// is zeros.
template <int D, int SUB>
__device__ __forceinline__ void start_groups(GroupShared& sh, const E4m3Args& a, const CUtensorMap* map_k,
                                             const CUtensorMap* map_v, const GroupWalk<SUB>& k, uint32_t ring, int first, int warp,
                                             int lane)
{
    constexpr int S = kKeys / SUB, kBoxes = GroupWalk<SUB>::kBoxes;
    if (!k.go) return;
    const int at = first + lane % kBoxes / S, sub = lane % S, hk = head_of(a, k.w, warp);
    const uint32_t dst = ring + at * GroupShape<D>::kSlotBytes + sub * SUB * D;
    uint64_t* bar = &sh.full[warp][at];
    const bool there = k.page >= 0 && k.page < a.num_pages;
    if (lane < kBoxes) {
        int place = -1;
        if (there && !a.starve) {
            const int b = (int)__umulhi((uint32_t)k.slot, a.block_magic);
            place = (k.page * a.blocks + b) * a.Hkv + hk;
            mbar_arrive_expect_tx(bar, 2 * SUB * D);
            load_box(dst, map_k, hk, k.slot, k.page, bar);
            load_box(dst + kKeys * D, map_v, hk, k.slot, k.page, bar);
        }
        sh.scale[warp][at][sub] = place;
    }
    uint32_t gone = __ballot_sync(0xffffffffu, lane < kBoxes && !there);
    if (gone) {
#pragma unroll 1
        for (uint32_t left = gone; left; left &= left - 1) {
            const uint32_t to = __shfl_sync(0xffffffffu, dst, __ffs(left) - 1);
#pragma unroll 1
            for (int e = lane; e < SUB * D / 16; e += 32) {
                asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(to + e * 16), "r"(0) : "memory");
                asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(to + kKeys * D + e * 16), "r"(0) : "memory");
            }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if ((gone >> lane) & 1) mbar_arrive(bar);
    }
    __syncwarp();
}

// Waits for a group's copies, for about two seconds at most; when a wait has given up
// the CTA goes on with what is there, marks its rows and sets the workspace's timeout
// word.
__device__ __forceinline__ void wait_group(GroupShared& sh, uint64_t* bar, uint32_t parity, int32_t* status)
{
    if (mbar_try_wait(bar, parity)) return;
    const long long t0 = clock64();
#pragma unroll 1
    while (!mbar_try_wait(bar, parity)) {
        if (*reinterpret_cast<volatile int*>(&sh.dead)) return;
        if (clock64() - t0 > (1ll << 32)) {
            *reinterpret_cast<volatile int*>(&sh.dead) = 1;
            atomicOr(status, 2);
            return;
        }
    }
}

// N neighbouring values, N of one row's channels to a lane.
template <int N>
__device__ __forceinline__ void store_run(float* p, const float (&y)[N])
{
    if constexpr (N >= 4) {
#pragma unroll
        for (int j = 0; j < N; j += 4) *reinterpret_cast<float4*>(p + j) = make_float4(y[j], y[j + 1], y[j + 2], y[j + 3]);
    } else {
        *reinterpret_cast<float2*>(p) = make_float2(y[0], y[1]);
    }
}
template <int N>
__device__ __forceinline__ void store_run(__nv_bfloat16* p, const float (&y)[N])
{
    uint32_t z[N / 2];
#pragma unroll
    for (int j = 0; j < N / 2; ++j) z[j] = sm100::pack_bf16x2(y[2 * j], y[2 * j + 1]);
    if constexpr (N >= 8) {
#pragma unroll
        for (int j = 0; j < N / 2; j += 4) *reinterpret_cast<uint4*>(p + 2 * j) = make_uint4(z[j], z[j + 1], z[j + 2], z[j + 3]);
    } else if constexpr (N == 4) {
        *reinterpret_cast<uint2*>(p) = make_uint2(z[0], z[1]);
    } else {
        *reinterpret_cast<uint32_t*>(p) = z[0];
    }
}

template <class T, class O, int D, int SUB>
__global__ void __launch_bounds__(kThreads, 1)
cache_attention_group_kernel(const __grid_constant__ E4m3Args a, const __grid_constant__ CUtensorMap map_k,
                             const __grid_constant__ CUtensorMap map_v)
{
    using Sh = GroupShape<D>;
    constexpr bool QLO = sizeof(T) == 4, PLO = sizeof(O) == 4;
    constexpr int KS = D / 16, NT = D / 8;
    constexpr int KB = D / 4 < 16 ? D / 4 : 16;    // bytes per read of a row of K
    constexpr int S = kKeys / SUB;                 // boxes, and scales, of a group
    extern __shared__ __align__(128) uint8_t dyn[];
    __shared__ GroupShared sh;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, i4 = lane & 3;
    const int group = blockIdx.x / a.split.row_tiles, r0 = (blockIdx.x % a.split.row_tiles) * kRows;
    if (lane == 0) {
        for (int i = 0; i < kSlots; ++i) {
            mbar_init(&sh.full[warp][i], S);
            sh.scale[warp][i][0] = sh.scale[warp][i][1] = -1;
        }
        if (warp == 0) sh.dead = 0;
        fence_mbar_init();
    }
    const TreeSpot sp = tree_locate<kThreads, 0, kGroupLead>(a.split, group, sh.loc);   // has block barriers
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    GroupWalk<SUB> ahead;
    ahead.go = ahead.w.start(a.split, sp, group);
    GroupPiece w = ahead.w;
    bool go = ahead.go;
    ahead.enter(a, warp, lane);
    const uint32_t base = (smem_at(dyn) + 1023u) & ~1023u;
    const uint32_t ring = base + warp * kSlots * Sh::kSlotBytes;
    float* join = reinterpret_cast<float*>(dyn + (base - smem_at(dyn)) + Sh::kRing);
    int out = 0;                                   // slot of the next step
    uint32_t turn = 0;
#pragma unroll 1
    for (int i = 0; i < kSlots; i += kStepGroups) {
        start_groups<D, SUB>(sh, a, &map_k, &map_v, ahead, ring, i, warp, lane);
        ahead.step(a, warp, lane);
    }
    // the next step's scales
    float ks[kStepGroups][S], vs[kStepGroups][S];
    auto load_scales = [&](int first) {
#pragma unroll
        for (int i = 0; i < kStepGroups; ++i)
#pragma unroll
            for (int b = 0; b < S; ++b) {
                const int at = sh.scale[warp][first + i][b];
                ks[i][b] = at >= 0 ? __ldg(a.k_scales + at) : -1.f;        // (-1: no rows)
                vs[i][b] = at >= 0 ? __ldg(a.v_scales + at) : 0.f;
            }
    };
    if (go) load_scales(0);
    const int heads = 1 << a.heads_log;
    const ScaleParts scale = scale_parts(a.scale_log2);
    for (; go; go = w.next(a.split)) {
        const int hk = head_of(a, w, warp);
        // the rows' queries, in fp16 times a power of two (and -1 for a negative scale; 0 for 0)
        uint32_t qh[KS][4], ql[QLO ? KS : 1][4];
        float rs[2];
        int lim[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = r0 + g + 8 * h, t = r / a.G;
            const bool mine = r < a.R;
            lim[h] = mine ? w.ctx - a.Ts + t + 1 : 0;
            const T* qp = static_cast<const T*>(a.q) +
                          (((long long)w.n * a.Ts + (mine ? t : 0)) * a.Hq + hk * a.G + (mine ? r - t * a.G : 0)) * D;
            float x[KS][4];
            uint32_t top = 0;
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                x[s][0] = x[s][1] = x[s][2] = x[s][3] = 0.f;
                if (mine) load4(qp + q_channel<D>(s, i4), x[s]);
            }
#pragma unroll
            for (int s = 0; s < KS; ++s)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    x[s][j] *= scale.pre;
                    top = top_of(top, x[s][j]);
                }
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const int e = up_of(top);
            float up = power(e);
            rs[h] = scale.rest * power(-e);
            if (a.scale_log2 < 0.f) up = -up;
            if (a.scale_log2 == 0.f) up = 0.f, rs[h] = 1.f;
            if (top >= kInfinity) rs[h] = kNaN;    // (scores of -inf alone would count as no rows)
#pragma unroll
            for (int s = 0; s < KS; ++s)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float u = x[s][2 * j] * up, v = x[s][2 * j + 1] * up;
                    qh[s][2 * j + h] = two_f16(u, v);
                    if constexpr (QLO) ql[s][2 * j + h] = two_f16_rest(u, v, qh[s][2 * j + h]);
                }
        }
        const int all = w.ctx - a.Ts + r0 / a.G + 1;           // keys that every row sees
        float o[NT][4], m[2], n[2], l[2], fac[2];
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int c = 0; c < 4; ++c) o[j][c] = 0.f;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            m[h] = n[h] = -INFINITY;
            l[h] = fac[h] = 0.f;
        }
#pragma unroll 1
        for (int t = w.t0; t < w.t1; ++t) {
#pragma unroll
            for (int i = 0; i < kStepGroups; ++i) wait_group(sh, &sh.full[warp][out + i], turn, a.status);
            __syncwarp();
            const uint32_t st = ring + out * Sh::kSlotBytes;
            float ksn[kStepGroups][S], vsn[kStepGroups][S];
            bool gaps = false;
#pragma unroll
            for (int i = 0; i < kStepGroups; ++i)
#pragma unroll
                for (int b = 0; b < S; ++b) {
                    ksn[i][b] = ks[i][b];
                    vsn[i][b] = vs[i][b];
                    gaps |= ks[i][b] < 0.f;
                }
            const int next = out + kStepGroups == kSlots ? 0 : out + kStepGroups;
            load_scales(next);                     // (of the last step: whatever is there)
            const int pos = (t << a.split.tile_log) + (warp >> a.heads_log) * kStepKeys;
            const bool masked = pos + kStepKeys > all || gaps;     // (the same for the warp)
            if (masked && pos + kStepKeys > w.ctx) {
                // values past the last row, whatever the page holds there
#pragma unroll
                for (int i = 0; i < kStepGroups; ++i)
#pragma unroll 1
                    for (int e = lane; e < kKeys * D / 16; e += 32)
                        if (pos + i * kKeys + e / (D / 16) >= w.ctx)
                            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(st + i * Sh::kSlotBytes + kKeys * D + e * 16), "r"(0)
                                         : "memory");
                fence_proxy_async_smem();
                __syncwarp();
            }
            float c[kStepGroups][2][4], small[kStepGroups][2][4];
            {
                Words<KB> kw[kStepGroups][2][D / 4 / KB];
#pragma unroll
                for (int h = 0; h < D / 4 / KB; ++h)
#pragma unroll
                    for (int i = 0; i < kStepGroups; ++i)
#pragma unroll
                        for (int b = 0; b < 2; ++b) {
                            const int at = KB * i4 + 64 * h;
                            kw[i][b][h] = read_words<KB>(st + i * Sh::kSlotBytes + row_at<D>(8 * b + key_of(g), at >> 4) + (at & 15));
                        }
#pragma unroll
                for (int s = 0; s < KS; ++s)
#pragma unroll
                    for (int i = 0; i < kStepGroups; ++i)
#pragma unroll
                        for (int b = 0; b < 2; ++b) {
                            const uint32_t x = kw[i][b][s / (KB / 4)].w[s % (KB / 4)];
                            const uint32_t b0 = widen_lo(x), b1 = widen_hi(x);
                            if (s == 0) mma0(c[i][b], qh[s], b0, b1);
                            else mma(c[i][b], qh[s], b0, b1);
                            if constexpr (QLO) {
                                if (s == 0) mma0(small[i][b], ql[s], b0, b1);
                                else mma(small[i][b], ql[s], b0, b1);
                            }
                        }
                if constexpr (QLO) {
#pragma unroll
                    for (int i = 0; i < kStepGroups; ++i)
#pragma unroll
                        for (int b = 0; b < 2; ++b)
#pragma unroll
                            for (int j = 0; j < 4; ++j) c[i][b][j] = fmaf(small[i][b][j], kRest, c[i][b][j]);
                }
            }
            float k1[kStepGroups][S][2], top[2], vtop[2];
            bool grow = false;
#pragma unroll
            for (int i = 0; i < kStepGroups; ++i)
#pragma unroll
                for (int b = 0; b < S; ++b)
#pragma unroll
                    for (int h = 0; h < 2; ++h) k1[i][b][h] = ksn[i][b] * rs[h];
            if (masked) {
#pragma unroll
                for (int i = 0; i < kStepGroups; ++i)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
#pragma unroll
                        for (int b = 0; b < 2; ++b)
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                float& x = c[i][b][2 * h + j];
                                x *= k1[i][b % S][h];
                                if (ksn[i][b % S] < 0.f || pos + i * kKeys + 8 * b + i4 + 4 * j >= lim[h]) x = -INFINITY;
                            }
#pragma unroll
                        for (int b = 0; b < S; ++b) k1[i][b][h] = 1.f;
                    }
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                top[h] = vtop[h] = -INFINITY;
#pragma unroll
                for (int i = 0; i < kStepGroups; ++i) {
                    float tops[2];
#pragma unroll
                    for (int b = 0; b < 2; ++b) tops[b] = fmaxf(c[i][b][2 * h], c[i][b][2 * h + 1]);
                    if (S == 1) tops[0] = fmaxf(tops[0], tops[1]);
#pragma unroll
                    for (int b = 0; b < S; ++b) {
                        const float x = tops[b] * k1[i][b][h];
                        top[h] = fmaxf(top[h], x);
                        vtop[h] = fmaxf(vtop[h], x + lg2(vsn[i][b]));
                    }
                }
                grow |= top[h] > m[h] + kSlack || vtop[h] > n[h] + (kSlack + kHead);
            }
            if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float m2 = fmaxf(m[h], quad_max(top[h]));
                    // n is kept near m, so that 2^(m - n) is finite
                    const float n2 = fmaxf(fmaxf(n[h], quad_max(vtop[h]) - kHead), m2 - 120.f);
                    const float fl = m2 == -INFINITY ? 1.f : ex2(m[h] - m2), fo = n2 == -INFINITY ? 1.f : ex2(n[h] - n2);
                    m[h] = m2;
                    n[h] = n2;
                    l[h] *= fl;
                    fac[h] = m2 == -INFINITY ? 0.f : ex2(m2 - n2);
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
                        o[j][2 * h] *= fo;
                        o[j][2 * h + 1] *= fo;
                    }
                }
            }
            uint32_t ph[kStepGroups][4], pl[kStepGroups][4];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float ref = m[h] == -INFINITY ? 0.f : m[h];
                float sum = 0.f;                   // (few additions to l, which small probabilities would be lost in)
#pragma unroll
                for (int i = 0; i < kStepGroups; ++i) {
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        const float w1 = weight_factor(vsn[i][b % S], fac[h]);
                        float y[2];
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const float x = c[i][b][2 * h + j];
                            const float p = ex2(fmaf(x, k1[i][b % S][h], -ref));
                            sum += p;
                            y[j] = p * w1;
                            if (masked && x == -INFINITY) y[j] = 0.f;
                        }
                        ph[i][2 * b + h] = two_f16(y[0], y[1]);
                        if constexpr (PLO) pl[i][2 * b + h] = two_f16_rest(y[0], y[1], ph[i][2 * b + h]);
                    }
                }
                l[h] += sum;
            }
#pragma unroll
            for (int i = 0; i < kStepGroups; ++i) {
                // this lane's D / 8 channels of keys i4, i4 + 4, 8 + i4, 12 + i4
                Words<NT> vw[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int at = channel_of<D>(g);
                    vw[j] = read_words<NT>(st + i * Sh::kSlotBytes + kKeys * D + row_at<D>(i4 + 4 * j, at >> 4) + (at & 15));
                }
#pragma unroll
                for (int x = 0; x < (NT + 3) / 4; ++x) {
                    const uint32_t lo0 = __byte_perm(vw[0].w[x], vw[1].w[x], 0x5140), hi0 = __byte_perm(vw[0].w[x], vw[1].w[x], 0x7362);
                    const uint32_t lo1 = __byte_perm(vw[2].w[x], vw[3].w[x], 0x5140), hi1 = __byte_perm(vw[2].w[x], vw[3].w[x], 0x7362);
                    const uint32_t b0[4] = {widen_lo(lo0), widen_hi(lo0), widen_lo(hi0), widen_hi(hi0)};
                    const uint32_t b1[4] = {widen_lo(lo1), widen_hi(lo1), widen_lo(hi1), widen_hi(hi1)};
#pragma unroll
                    for (int j = 0; j < (NT < 4 ? NT : 4); ++j) {
                        if constexpr (PLO) {
                            float z[4], rest[4];
                            mma0(rest, pl[i], b0[j], b1[j]);
                            mma0(z, ph[i], b0[j], b1[j]);
#pragma unroll
                            for (int e = 0; e < 4; ++e) o[4 * x + j][e] += fmaf(rest[e], kRest, z[e]);
                        } else {
                            mma(o[4 * x + j], ph[i], b0[j], b1[j]);
                        }
                    }
                }
            }
            __syncwarp();                          // the slots have been read
            start_groups<D, SUB>(sh, a, &map_k, &map_v, ahead, ring, out, warp, lane);
            ahead.step(a, warp, lane);
            out = next;
            turn ^= next == 0;
        }
        // The results of a head's warps, halved until one warp has them all: the upper
        // half writes (O, m, n, l), the lower half adds them to its own.
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
        }
#pragma unroll 1
        for (int half = kWarps / 2; half >= heads; half >>= 1) {
            __syncthreads();                       // what was there has been read
            if (warp >= half && warp < 2 * half) {
                float* y = join + (warp - half) * (Sh::kFrag + 3 * kRows);
#pragma unroll
                for (int j = 0; j < NT; ++j)
                    *reinterpret_cast<float4*>(y + j * 128 + lane * 4) = make_float4(o[j][0], o[j][1], o[j][2], o[j][3]);
                if (i4 == 0) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        y[Sh::kFrag + g + 8 * h] = m[h];
                        y[Sh::kFrag + kRows + g + 8 * h] = n[h];
                        y[Sh::kFrag + 2 * kRows + g + 8 * h] = l[h];
                    }
                }
            }
            __syncthreads();
            if (warp < half) {
                const float* y = join + warp * (Sh::kFrag + 3 * kRows);
                float f0[2], f1[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float ym = y[Sh::kFrag + g + 8 * h], yn = y[Sh::kFrag + kRows + g + 8 * h];
                    const float m2 = fmaxf(m[h], ym), n2 = fmaxf(n[h], yn);
                    const float mr = m2 == -INFINITY ? 0.f : m2, nr = n2 == -INFINITY ? 0.f : n2;
                    l[h] = l[h] * ex2(m[h] - mr) + y[Sh::kFrag + 2 * kRows + g + 8 * h] * ex2(ym - mr);
                    f0[h] = ex2(n[h] - nr);
                    f1[h] = ex2(yn - nr);
                    m[h] = m2;
                    n[h] = n2;
                }
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    const float4 z = *reinterpret_cast<const float4*>(y + j * 128 + lane * 4);
                    o[j][0] = o[j][0] * f0[0] + z.x * f1[0];
                    o[j][1] = o[j][1] * f0[0] + z.y * f1[0];
                    o[j][2] = o[j][2] * f0[1] + z.z * f1[1];
                    o[j][3] = o[j][3] * f0[1] + z.w * f1[1];
                }
            }
        }
        if (warp < heads) {
            const bool whole = w.t0 == 0 && w.t1 == w.tiles;
            float* part = a.part + ((((size_t)blockIdx.x * 2 + (w.t0 == 0 ? 1 : 0)) << a.heads_log) + warp) * kRows * (D + 3);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int r = g + 8 * h, row = r0 + r;
                if (*reinterpret_cast<volatile int*>(&sh.dead)) l[h] = __int_as_float(0x7fffffff);
                if (row >= a.R) continue;
                const int t = row / a.G;
                const float f = l[h] == 0.f ? 0.f : ex2(n[h] - m[h]) / l[h];
                O* op = static_cast<O*>(a.o) + (((long long)w.n * a.Ts + t) * a.Hq + hk * a.G + row - t * a.G) * D;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int ch = channel_of<D>(2 * i4 + e);
                    float y[NT];
#pragma unroll
                    for (int j = 0; j < NT; ++j) y[j] = o[j][2 * h + e] * (whole ? f : 1.f);
                    if (whole) store_run<NT>(op + ch, y);
                    else store_run<NT>(part + r * D + ch, y);
                }
                if (!whole && i4 == 0) {
                    part[kRows * D + r] = m[h];
                    part[kRows * D + kRows + r] = n[h];
                    part[kRows * D + 2 * kRows + r] = l[h];
                }
            }
        }
    }
    // after a wait that gave up some copies may be in flight: time for them to land
    if (*reinterpret_cast<volatile int*>(&sh.dead)) {
        const long long t0 = clock64();
        while (clock64() - t0 < (1ll << 22)) {}
    }
}

// Joins the pieces of the items that were cut between groups.  Block (c, y, z): the
// item that the boundary before group c + 1 falls into, if that is the item's first
// boundary; head y of it and then rows 8 .. of row tile z, a warp each.  The pieces are
// read in the order of the groups, so the result does not depend on timing.
// (It takes 4 to 7 us at the end of a call, 12 for 64 x 4 tokens.  Joined by the last thread block
// to have written a piece, found by counters that a kernel before clears, calls take 1 to 8 us
// longer: few thread blocks then read all pieces.)
constexpr int kJoinThreads = 256;

template <class O, int D, int KT, int kLead>
__global__ void __launch_bounds__(kJoinThreads)
cache_join_kernel(const __grid_constant__ E4m3Args a)
{
    __shared__ long long sh_loc[kJoinThreads / 32 + 2];
    const int c = blockIdx.x + 1, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const TreeArgs& s = a.split;
    const TreeSpot sp = tree_locate<kJoinThreads, KT, kLead>(s, c, sh_loc);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const long long at = tree_begin(sp, c);
    if (at >= sp.total) return;                     // an empty range at the end
    const int tiles = tree_tiles<KT>(s, sp.n), heads = 1 << a.heads_log, h = blockIdx.y & (heads - 1);
    int hk = (int)((at - sp.start) / (tiles + kLead));
    // where the item's tiles begin; a boundary up to there cuts nothing
    const long long first = sp.start + (long long)hk * (tiles + kLead) + kLead;
    if (at <= first || tree_begin(sp, c - 1) > first) return;
    int last = c;                                   // the last group with tiles of this item
    while (last + 1 < s.groups && tree_begin(sp, last + 1) < first + tiles) ++last;
    hk = hk * heads + h;
    const int r = (blockIdx.y >> a.heads_log) * (kJoinThreads / 32) + warp, row = blockIdx.z * kRows + r;
    if (r >= kRows || row >= a.R) return;
    // piece p of the item: group p's first slot, but the second of group c - 1
    auto piece = [&](int p) {
        return a.part + (((((size_t)p * s.row_tiles + blockIdx.z) * 2 + (p == c - 1 ? 1 : 0)) << a.heads_log) + h) * kRows * (D + 3);
    };
    constexpr int E = D / 32 > 0 ? D / 32 : 1;
    float m = -INFINITY, n = -INFINITY;
    for (int p = c - 1 + lane; p <= last; p += 32) {
        m = fmaxf(m, piece(p)[kRows * D + r]);
        n = fmaxf(n, piece(p)[kRows * D + kRows + r]);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
        n = fmaxf(n, __shfl_xor_sync(0xffffffffu, n, off));
    }
    const float mr = m == -INFINITY ? 0.f : m, nr = n == -INFINITY ? 0.f : n;
    float l = 0.f, o[E];
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.f;
#pragma unroll 4
    for (int p = c - 1; p <= last; ++p) {
        const float* x = piece(p);
        l += x[kRows * D + 2 * kRows + r] * ex2(x[kRows * D + r] - mr);
        const float f = ex2(x[kRows * D + kRows + r] - nr);
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (D >= 32 || lane < D) o[e] += x[r * D + lane + 32 * e] * f;
    }
    const float f = l == 0.f ? 0.f : ex2(nr - mr) / l;
    const int t = row / a.G;
    O* op = static_cast<O*>(a.o) + (((long long)sp.n * a.Ts + t) * a.Hq + hk * a.G + row - t * a.G) * D;
#pragma unroll
    for (int e = 0; e < E; ++e)
        if (D >= 32 || lane < D) op[lane + 32 * e] = O(o[e] * f);
}

template <class O, int D, int KT, int LEAD>
cudaError_t launch_join(const E4m3Args& a, cudaStream_t stream)
{
    if (a.split.groups < 2) return cudaSuccess;
    cudaLaunchConfig_t cfg = {};
    const int rows = a.R < kRows ? a.R : kRows;
    cfg.gridDim = dim3(a.split.groups - 1, ((rows + kJoinThreads / 32 - 1) / (kJoinThreads / 32)) << a.heads_log, a.split.row_tiles);
    cfg.blockDim = dim3(kJoinThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, cache_join_kernel<O, D, KT, LEAD>, a);
}

// The pool as [num_pages][page_size][Hkv][d] bytes, boxes of `box` rows of one head.
bool make_pool_map(CUtensorMap* m, const uint8_t* base, const E4m3Args& a, int d, int box)
{
    const auto fn = tc_encode_fn();
    if (!fn) return false;
    const cuuint64_t row = (cuuint64_t)a.Hkv * d, size = a.split.page_size;
    const cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)a.Hkv, size, (cuuint64_t)a.num_pages};
    const cuuint64_t strides[3] = {(cuuint64_t)d, row, a.num_pages > 1 ? (cuuint64_t)a.page_stride : row * size};
    const cuuint32_t boxes[4] = {(cuuint32_t)d, 1, (cuuint32_t)box, 1}, steps[4] = {1, 1, 1, 1};
    const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<uint8_t*>(base), dims, strides, boxes, steps,
                          CU_TENSOR_MAP_INTERLEAVE_NONE,
                          d == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : d == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_NONE,
                          // (256 bytes would fetch the next head's rows with these: 64 x 1 token 532 us)
                          d == 128 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B : CU_TENSOR_MAP_L2_PROMOTION_NONE,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS && debug_enabled())
        fprintf(stderr, "kda: cuTensorMapEncodeTiled failed (CUresult %d, 8-bit pages)\n", (int)r);
    return r == CUDA_SUCCESS;
}

template <class T, class O, int D, int SUB>
cudaError_t launch_groups(E4m3Args a, const CUtensorMap& map_k, const CUtensorMap& map_v, cudaStream_t stream)
{
    auto kern = cache_attention_group_kernel<T, O, D, SUB>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)GroupShape<D>::kBytes);
    if (e != cudaSuccess) return e;
    // (the rule at the top of this part)
    while (a.heads_log < 3 && a.Hkv % (2 << a.heads_log) == 0 &&
           (long long)a.split.N * (a.Hkv >> (a.heads_log + 1)) * kMostCuts >= a.split.groups)
        ++a.heads_log;
    a.split.Hkv = a.Hkv >> a.heads_log;
    const int keys = kWarps * kStepKeys >> a.heads_log;
    a.split.tile_log = __builtin_ctz(keys);
    a.tile_pages = keys / a.split.page_size;
    a.tile_rows = keys % a.split.page_size;
    kern<<<a.split.groups * a.split.row_tiles, kThreads, GroupShape<D>::kBytes, stream>>>(a, map_k, map_v);
    e = cudaGetLastError();
    return e != cudaSuccess ? e : launch_join<O, D, 0, kGroupLead>(a, stream);
}

template <class T, class O, int D>
cudaError_t launch(E4m3Args a, cudaStream_t stream)
{
    // 16 or 8 rows from a multiple of that on in one page and one block of scales
    const int box = a.split.page_size % 16 == 0 && a.block % 16 == 0 ? 16 : 8;
    CUtensorMap map_k, map_v;
    if (a.split.page_size % box == 0 && a.block % box == 0 && (long long)a.num_pages * a.blocks * a.Hkv <= INT32_MAX &&
        make_pool_map(&map_k, a.k_cache, a, D, box) && make_pool_map(&map_v, a.v_cache, a, D, box))
        return box == 16 ? launch_groups<T, O, D, 16>(a, map_k, map_v, stream) : launch_groups<T, O, D, 8>(a, map_k, map_v, stream);
    a.split.Hkv = a.Hkv;
    auto kern = cache_attention_kernel<T, O, D>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Shape<D>::kBytes);
    if (e != cudaSuccess) return e;
    a.tile_pages = KT / a.split.page_size;
    a.tile_rows = KT % a.split.page_size;
    kern<<<a.split.groups * a.split.row_tiles, kThreads, Shape<D>::kBytes, stream>>>(a);
    e = cudaGetLastError();
    return e != cudaSuccess ? e : launch_join<O, D, KT, kLead>(a, stream);
}

template <class T, class O>
cudaError_t launch_d(const E4m3Args& a, int32_t d, cudaStream_t stream)
{
    switch (d) {
    case 16: return launch<T, O, 16>(a, stream);
    case 32: return launch<T, O, 32>(a, stream);
    case 64: return launch<T, O, 64>(a, stream);
    default: return launch<T, O, 128>(a, stream);
    }
}

void plan(int32_t R, int sms, int32_t& groups, int32_t& row_tiles)
{
    row_tiles = (R + kRows - 1) / kRows;
    groups = sms / row_tiles > 1 ? sms / row_tiles : 1;
}

}  // namespace

size_t e4m3_workspace_bytes(int32_t Ts, int32_t Hq, int32_t Hkv, int32_t d, int sms)
{
    int32_t groups, row_tiles;
    plan(Ts * (Hq / Hkv), sms > 0 ? sms : 1, groups, row_tiles);
    const int heads = Hkv % 8 == 0 ? 8 : Hkv % 4 == 0 ? 4 : Hkv % 2 == 0 ? 2 : 1;   // the most of an item
    if (groups == 1) return kWsHeaderBytes;            // (nothing is cut)
    return kWsHeaderBytes + (size_t)groups * row_tiles * 2 * heads * kRows * (d + 3) * sizeof(float);
}

cudaError_t launch_cache_attention_e4m3(E4m3Args a, int32_t d, kda_dtype_t dtype, int sms, cudaStream_t stream)
{
    a.starve = getenv("KDA_TEST_STARVE_CONSUMERS") != nullptr;
    plan(a.R, sms > 0 ? sms : 1, a.split.groups, a.split.row_tiles);
    if (dtype == KDA_BF16) return launch_d<__nv_bfloat16, __nv_bfloat16>(a, d, stream);
    if (dtype == KDA_BF16_F32OUT) return launch_d<__nv_bfloat16, float>(a, d, stream);
    return launch_d<float, float>(a, d, stream);
}

}  // namespace kda
