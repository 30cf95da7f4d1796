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
#include "kda_tree.cuh"

namespace kda {
namespace {

constexpr int kSimtThreads = 128;
constexpr int kSimtKeys = 64;        // keys per tile (a drafted tree fits one)

template <int D, int RT>
struct SimtShape {
    static constexpr int kLdk = D + 4;
    static constexpr int kLdp = kSimtKeys + 4;
    static constexpr size_t kBytes =
        sizeof(float) * (RT * kLdk + kSimtKeys * kLdk + kSimtKeys * D + RT * kLdp);
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

// 128 threads as 8 row groups x 16 columns.  Thread (ty, tx) owns rows
// ty RR .. ty RR + RR - 1 throughout: their scores for keys tx + 16 j, and D /
// 16 of their output columns, so m, l and the rescaling stay in registers.
template <typename TI, typename TO, int D, int RT>
__global__ void __launch_bounds__(kSimtThreads)
tree_attention_simt_kernel(const TreeArgs a)
{
    using Sh = SimtShape<D, RT>;
    constexpr int RR = RT / 8, KR = kSimtKeys / 16, CR = D / 16;
    constexpr int V4 = D / 4;
    extern __shared__ __align__(16) float smem[];
    float* sQ = smem;                               // [RT][kLdk]
    float* sK = sQ + RT * Sh::kLdk;                 // [keys][kLdk]
    float* sV = sK + kSimtKeys * Sh::kLdk;          // [keys][D]
    float* sP = sV + kSimtKeys * D;                 // [RT][kLdp]
    __shared__ long long sh_loc[kSimtThreads / 32 + 2];
    __shared__ unsigned long long anc[kTreeMaxNodes];
    __shared__ int32_t up[kTreeMaxNodes];
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const TI* q = static_cast<const TI*>(a.q);

    const int group = blockIdx.x / a.row_tiles, r0 = (blockIdx.x % a.row_tiles) * RT;
    const int rows = a.R - r0 < RT ? a.R - r0 : RT;
    const TreeSpot sp = tree_locate<kSimtThreads, kSimtKeys>(a, group, sh_loc);
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int row_elems = a.Hkv * D;
    int have = -1;                                  // the sequence anc[] is of

    TreePieces<kSimtKeys> w;
    for (bool more = w.start(a, sp, group); more; more = w.next(a)) {
        const int n = w.n, ctx = w.ctx, tiles = w.tiles, t0 = w.t0, t1 = w.t1, hk = w.hk;
        const int32_t* table = a.page_table + (long long)n * a.max_pages;
        if (have != n) {
            __syncthreads();
            if (tid < 32)
                tree_masks(a.parent ? a.parent + (long long)n * a.Ts : nullptr, a.Ts, tid, anc, up);
            have = n;
        }
        __syncthreads();
        for (int e = tid; e < RT * V4; e += kSimtThreads) {
            const int r = e / V4, c = e % V4;
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r < rows) {
                const int t = (r0 + r) / a.G, g = (r0 + r) % a.G;
                x = load4(q + (((long long)n * a.Ts + t) * a.Hq + hk * a.G + g) * D + 4 * c);
            }
            *reinterpret_cast<float4*>(sQ + r * Sh::kLdk + 4 * c) =
                make_float4(x.x * a.scale_log2, x.y * a.scale_log2, x.z * a.scale_log2,
                            x.w * a.scale_log2);
        }
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
            const int k0 = t * kSimtKeys;
            const int nc = ctx - k0;                // key j is drafted node j - nc from j = nc on
            const int nk = nc + a.Ts < kSimtKeys ? nc + a.Ts : kSimtKeys;
            const bool draft = nc < kSimtKeys;      // some are
            __syncthreads();                        // the previous tile has been read
            for (int e = tid; e < kSimtKeys * V4; e += kSimtThreads) {
                const int j = e / V4, c = e % V4;
                float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
                if (j < nk) {
                    long long off;
                    const TI *kp = static_cast<const TI*>(a.k_cache), *vp = static_cast<const TI*>(a.v_cache);
                    if (j >= nc) {
                        off = ((long long)n * a.Ts + j - nc) * row_elems;
                        kp = static_cast<const TI*>(a.k);
                        vp = static_cast<const TI*>(a.v);
                    } else {
                        off = tree_cache_row(a, table, k0 + j, row_elems);
                    }
                    if (off >= 0) {
                        x = load4(kp + off + hk * D + 4 * c);
                        y = load4(vp + off + hk * D + 4 * c);
                    }
                }
                *reinterpret_cast<float4*>(sK + j * Sh::kLdk + 4 * c) = x;
                *reinterpret_cast<float4*>(sV + j * D + 4 * c) = y;
            }
            __syncthreads();
            float s[RR][KR];
#pragma unroll
            for (int i = 0; i < RR; ++i)
#pragma unroll
                for (int j = 0; j < KR; ++j) s[i][j] = 0.f;
#pragma unroll 4
            for (int c = 0; c < V4; ++c) {
                float4 kv[KR];
#pragma unroll
                for (int j = 0; j < KR; ++j)
                    kv[j] = *reinterpret_cast<const float4*>(sK + (tx + 16 * j) * Sh::kLdk + 4 * c);
#pragma unroll
                for (int i = 0; i < RR; ++i) {
                    const float4 x = *reinterpret_cast<const float4*>(sQ + (ty * RR + i) * Sh::kLdk + 4 * c);
#pragma unroll
                    for (int j = 0; j < KR; ++j) {
                        s[i][j] = fmaf(x.x, kv[j].x, s[i][j]);
                        s[i][j] = fmaf(x.y, kv[j].y, s[i][j]);
                        s[i][j] = fmaf(x.z, kv[j].z, s[i][j]);
                        s[i][j] = fmaf(x.w, kv[j].w, s[i][j]);
                    }
                }
            }
            unsigned there = 0;                     // context keys whose page exists
#pragma unroll
            for (int j = 0; j < KR; ++j) {
                const int kk = tx + 16 * j;
                if (kk < nc && tree_cache_row(a, table, k0 + kk, row_elems) >= 0) there |= 1u << j;
            }
#pragma unroll
            for (int i = 0; i < RR; ++i) {
                float top = m[i];
#pragma unroll
                for (int j = 0; j < KR; ++j) {
                    const int node = tx + 16 * j - nc;
                    const bool see = node < 0 ? mask[i] != 0ull && ((there >> j) & 1)
                                              : node < a.Ts && ((mask[i] >> node) & 1ull);
                    if (!see) s[i][j] = -INFINITY;
                    top = fmaxf(top, s[i][j]);
                }
#pragma unroll
                for (int off = 1; off < 16; off <<= 1)
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
                const float ref = top == -INFINITY ? 0.f : top;
                const float shrink = exp2f(m[i] - ref);
                float sum = 0.f;
#pragma unroll
                for (int j = 0; j < KR; ++j) {
                    const float p = exp2f(s[i][j] - ref);
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
#pragma unroll 2
            for (int j = 0; j < kSimtKeys; j += 4) {
                float4 p[RR];
#pragma unroll
                for (int i = 0; i < RR; ++i)
                    p[i] = *reinterpret_cast<const float4*>(sP + (ty * RR + i) * Sh::kLdp + j);
#pragma unroll
                for (int jj = 0; jj < 4; ++jj) {
                    float v[CR];
#pragma unroll
                    for (int c = 0; c < CR; ++c) v[c] = sV[(j + jj) * D + tx + 16 * c];
#pragma unroll
                    for (int i = 0; i < RR; ++i) {
                        const float pp = jj == 0 ? p[i].x : jj == 1 ? p[i].y : jj == 2 ? p[i].z : p[i].w;
                        // a node that this row does not see may hold inf or NaN: 0 * v would keep it
                        if (draft && j + jj >= nc && (j + jj >= nk || !((mask[i] >> (j + jj - nc)) & 1ull)))
                            continue;
#pragma unroll
                        for (int c = 0; c < CR; ++c) acc[i][c] = fmaf(pp, v[c], acc[i][c]);
                    }
                }
            }
        }
        // Finished here, or one of the CTA's two pieces.
        const bool whole = t0 == 0 && t1 == tiles;
        float* part = a.part + ((size_t)blockIdx.x * 2 + (t0 == 0 ? 1 : 0)) * RT * (D + 2);
#pragma unroll
        for (int i = 0; i < RR; ++i) {
            const int r = ty * RR + i;
            if (r >= rows) continue;
            if (whole) {
                const int t = (r0 + r) / a.G, g = (r0 + r) % a.G;
                TO* op = static_cast<TO*>(a.o) + (((long long)n * a.Ts + t) * a.Hq + hk * a.G + g) * D;
                const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];
#pragma unroll
                for (int c = 0; c < CR; ++c) st_f(op + tx + 16 * c, mask[i] ? acc[i][c] * inv : 0.f);
            } else {
#pragma unroll
                for (int c = 0; c < CR; ++c) part[r * D + tx + 16 * c] = acc[i][c];
                if (tx == 0) {
                    part[RT * D + r] = m[i];
                    part[RT * D + RT + r] = l[i];
                }
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

template <typename TO, int D, int KT>
__global__ void __launch_bounds__(kJoinThreads)
tree_join_kernel(const TreeArgs a, int RT)
{
    __shared__ long long sh_loc[kJoinThreads / 32 + 2];
    const int c = blockIdx.x + 1, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const TreeSpot sp = tree_locate<kJoinThreads, KT>(a, c, sh_loc);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const long long at = tree_begin(sp, c);
    if (at >= sp.total) return;                     // an empty range at the end
    const int tiles = (int)tree_seq_tiles<KT>(a, sp.n);
    const int hk = (int)((at - sp.start) / tiles);
    const long long first = sp.start + (long long)hk * tiles;
    if (at == first || tree_begin(sp, c - 1) > first) return;
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
            if (D >= 32 || lane < D) o[e] = fmaf(x[(size_t)r * D + lane + 32 * e], w, o[e]);
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;     // l = 0: an unused node; a NaN stays
    const int t = (r0 + r) / a.G, g = (r0 + r) % a.G;
    TO* op = static_cast<TO*>(a.o) + (((long long)sp.n * a.Ts + t) * a.Hq + hk * a.G + g) * D;
#pragma unroll
    for (int e = 0; e < E; ++e)
        if (D >= 32 || lane < D) st_f(op + lane + 32 * e, o[e] * inv);
}

template <typename TO, int D, int KT>
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
    return cudaLaunchKernelEx(&cfg, tree_join_kernel<TO, D, KT>, a, rt);
}

template <typename TI, typename TO, int D, int RT>
cudaError_t launch_simt(const TreeArgs& a, cudaStream_t stream)
{
    auto kern = tree_attention_simt_kernel<TI, TO, D, RT>;
    const size_t bytes = SimtShape<D, RT>::kBytes;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e != cudaSuccess) return e;
    kern<<<a.groups * a.row_tiles, kSimtThreads, bytes, stream>>>(a);
    return cudaGetLastError();
}

template <typename TI, typename TO, int D>
cudaError_t launch_d(const TreeArgs& a, const TreePlan& plan, cudaStream_t stream)
{
    cudaError_t e = plan.rt == 8 ? launch_simt<TI, TO, D, 8>(a, stream)
                                 : launch_simt<TI, TO, D, 32>(a, stream);
    if (e != cudaSuccess) return e;
    return launch_join<TO, D, kSimtKeys>(a, plan.rt, stream);
}

template <typename TI, typename TO>
cudaError_t launch_typed(const TreeArgs& a, const TreePlan& plan, int d, cudaStream_t stream)
{
    switch (d) {
        case 16: return launch_d<TI, TO, 16>(a, plan, stream);
        case 32: return launch_d<TI, TO, 32>(a, plan, stream);
        case 64: return launch_d<TI, TO, 64>(a, plan, stream);
        case 128: return launch_d<TI, TO, 128>(a, plan, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace

TreePlan tree_plan(int32_t Ts, int32_t Hq, int32_t Hkv, int sms, bool tc)
{
    const int R = Ts * (Hq / Hkv);
    TreePlan p;
    p.tc = tc;
    p.rt = tc ? (R <= 128 ? 128 : 256) : (R <= 8 ? 8 : 32);
    p.row_tiles = (R + p.rt - 1) / p.rt;
    const int ctas = (sms > 0 ? sms : 1) * (tc ? 1 : 2);
    p.groups = ctas / p.row_tiles > 1 ? ctas / p.row_tiles : 1;
    return p;
}

// The tensor-core kernel takes bf16 with d = 64 or 128 and bf16 output (its
// probabilities are rounded to bf16, which an fp32 output would show).
bool tree_tc_supported(int32_t d, kda_dtype_t dtype)
{
    return dtype == KDA_BF16 && (d == 64 || d == 128);
}

size_t tree_workspace_bytes(int32_t Ts, int32_t Hq, int32_t Hkv, int32_t d, kda_dtype_t dtype, int sms)
{
    size_t most = 0;
    for (int tc = 0; tc <= (int)tree_tc_supported(d, dtype); ++tc) {
        const TreePlan p = tree_plan(Ts, Hq, Hkv, sms, tc != 0);
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
    const TreePlan plan = tree_plan(args.Ts, args.Hq, args.Hkv, sms, tc);
    args.groups = plan.groups;
    args.row_tiles = plan.row_tiles;
    if (plan.tc) {
        const cudaError_t e = launch_tree_attention_tc(args, plan, d, stream);
        if (e != cudaSuccess) return e;
        return d == 64 ? launch_join<__nv_bfloat16, 64, 128>(args, plan.rt, stream)
                       : launch_join<__nv_bfloat16, 128, 128>(args, plan.rt, stream);
    }
    switch (dtype) {
        case KDA_BF16: return launch_typed<__nv_bfloat16, __nv_bfloat16>(args, plan, d, stream);
        case KDA_BF16_F32OUT: return launch_typed<__nv_bfloat16, float>(args, plan, d, stream);
        default: return launch_typed<float, float>(args, plan, d, stream);
    }
}

}  // namespace kda
