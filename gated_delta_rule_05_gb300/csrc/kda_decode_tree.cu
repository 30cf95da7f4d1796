// kda_decode_tree.cu -- the KDA step of every node of a tree of drafted tokens,
// each from the state after its parent node (parent -1: from S_in).
//
// The step is kda_decode.cu's, and so is the order of its sums, so that a chain
// gives the same bits as kda_decode_multi:
//     w = S^T (alpha .* k), p = S^T (alpha .* q), u = beta (v - w)
//     S' = Diag(alpha) S + k u^T,  o = p + (k . q) u
// Each used node's state is written once and S_in read once: 4 d_k d_v (1 +
// nodes) bytes per (sequence, head); that bounds the call.  What a tree adds is
// that a node's parent need not be the node before it.  Reading such states
// back from memory would nearly double the traffic (two thirds of the nodes of
// a tree that grows from its recent nodes need it, and a launch writes more
// than L2 holds).  So a state that still has children to come is kept in a slot
// of shared memory, or, when the slots are taken, written without the
// evict-first hint, so that the threads that wrote it find it in L2.  Which
// state goes where is settled before the first node, from the parents alone.
//
// Mapping: one CTA per (sequence, head, 64 value columns) at d = 128, 8 float4 of
// the state per thread, three CTAs (96 KB of states) on an SM.  Columns matter:
// slabs of 32 write 128 bytes here and there, 375 us instead of 340 for 64
// sequences of 16 nodes (12.25 used on average) of 32 heads, d = 128, i.e. 5,060
// GB/s of states; the whole width needs 64 registers a thread and spills, 349
// us.  A chain of the same size takes 390 us, 5,970 GB/s.  All 16 nodes used: d = 128
// 427 us, d = 64 129, d = 32 53, d = 16 23 (80, 66, 41 and 23 % of a copy: the steps
// stay as many).  Few (sequence, head)
// units (fewer than SMs) take slabs of 32, for the CTAs: one sequence of 8 nodes
// 12 us instead of 18.  The inputs of the next nodes are loaded and combined
// (alpha k, alpha q, k . q) ahead of their steps, which then touch shared memory
// alone until the state is written.  Arithmetic is two-wide.
#include "kda_tree.cuh"
#include "kda_verify.cuh"

namespace kda {
namespace {

// COLS: the value columns of a CTA.
template <int D, int COLS>
struct TreeShape {
    static constexpr int RPP = D == 128 ? 16 : 8;               // rows per pass, as in kda_decode.cu
    static constexpr int LPR = COLS / 4;                        // lanes per row
    static constexpr int kThreads = RPP * LPR;
    static constexpr int R = D / RPP;                           // float4 per thread
    // kda_decode.cu adds kSummed neighbouring rows by shuffles, then those sums in
    // order; here a warp holds kInWarp rows
    static constexpr int kSummed = 32 / ((D >= 64 ? 64 : D) / 4);
    static constexpr int kInWarp = 32 / LPR < kSummed ? 32 / LPR : kSummed;
    // Blocks per SM: 80 registers a thread hold the state and what a step needs
    // (at 64 it spills, at 128 too few steps run side by side: 64 sequences of 16
    // nodes, 435 and 376 against 340 us); narrow CTAs run where there are few, and
    // take 128.
    static constexpr int kBlocks = D == 128 && COLS == 32 ? 4 : (768 / kThreads < 12 ? 768 / kThreads : 12);
    static constexpr int kNodes = D == 128 ? 4 : 2;             // nodes whose inputs are loaded together
    static constexpr int kSlotBytes = D * COLS * 4;
    static_assert(kSummed <= 2 * kInWarp && kThreads % 32 == 0, "shape");
};

enum : int { kSkip = -3, kRegisters = -2, kMemory = -1 };       // else a slot
enum : int { kNowhere = -1, kInL2 = -2 };                       // else a slot

struct Plan {
    int8_t from[kTreeMaxNodes];            // where node t finds its parent's state
    int8_t keep[kTreeMaxNodes];            // where its own is kept
    int8_t parent[kTreeMaxNodes];
    int8_t keep_root;                      // the slot S_in goes to (-1: none)
    int8_t first;                          // the first used node (Ts: none)
};

// Where every state is found and kept.  One warp; a lane has nodes lane and lane
// + 32, and what a step needs of another node comes by a shuffle.
__device__ __forceinline__ void make_plan(const int32_t* parent, int Ts, int slots, int lane, Plan& plan)
{
    constexpr unsigned kAll = 0xffffffffu;
    int par[2], last[2] = {-1, -1}, keep[2] = {kNowhere, kNowhere};        // last: the last used child
#pragma unroll
    for (int i = 0; i < 2; ++i) par[i] = lane + 32 * i < Ts ? __ldg(parent + lane + 32 * i) : -2;
    auto of = [&](const int (&x)[2], int t) {
        const int lo = __shfl_sync(kAll, x[0], t & 31);
        return Ts <= 32 ? lo : (t < 32 ? lo : __shfl_sync(kAll, x[1], t & 31));
    };
    unsigned long long used = 0;
    int last_root = -1;
#pragma unroll 1
    for (int t = 0; t < Ts; ++t) {
        const int p = of(par, t);
        if (p != -1 && (p < 0 || p >= t || !((used >> p) & 1))) continue;
        used |= 1ull << t;
        if (p < 0) last_root = t;
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (p == lane + 32 * i) last[i] = t;
    }
    unsigned free = (1u << slots) - 1;
    int keep_root = -1, at = -1;           // at: the node whose state is in registers
    const int first = used ? __ffsll((long long)used) - 1 : Ts;
    if (last_root > first && free) {       // S_in has other children
        keep_root = 0;
        free &= free - 1;
    }
#pragma unroll 1
    for (int t = 0; t < Ts; ++t) {
        int from = kSkip, p = -1;
        if ((used >> t) & 1) {
            p = of(par, t);
            const int q = p < 0 ? 0 : p;
            const int slot_p = of(keep, q), last_p = of(last, q), last_t = of(last, t);
            const int slot = p < 0 ? keep_root : slot_p;
            from = p == at ? kRegisters : (slot >= 0 ? slot : kMemory);
            if (slot >= 0 && (p < 0 ? last_root : last_p) == t) free |= 1u << slot;
            // kept unless its only child to come is the next used node
            const unsigned long long later = t < 63 ? used >> (t + 1) : 0ull;
            const int next = later ? t + __ffsll((long long)later) : Ts;
            if (last_t > next) {
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    if (t == lane + 32 * i) keep[i] = free ? __ffs(free) - 1 : kInL2;
                free &= free - 1;
            }
            at = t;
        }
        if (lane == 0) {
            plan.from[t] = from;
            plan.parent[t] = p;
        }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) plan.keep[lane + 32 * i] = keep[i];
    if (lane == 0) {
        plan.keep_root = keep_root;
        plan.first = first;
    }
}

// Pairs of fp32: the two-wide forms round each value as fmaf and * do.
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
__device__ __forceinline__ uint64_t shfl_add2(uint64_t x, int off)
{
    const float2 v = *reinterpret_cast<const float2*>(&x);
    const float2 y = make_float2(v.x + __shfl_xor_sync(0xffffffffu, v.x, off),
                                 v.y + __shfl_xor_sync(0xffffffffu, v.y, off));
    return *reinterpret_cast<const uint64_t*>(&y);
}

template <typename TI, typename TO, int D, int COLS>
__global__ void __launch_bounds__(TreeShape<D, COLS>::kThreads, TreeShape<D, COLS>::kBlocks)
decode_tree_kernel(const TI* __restrict__ q, const TI* __restrict__ k, const TI* __restrict__ v,
                   const float* __restrict__ log_alpha, const float* __restrict__ beta,
                   const float* S_in, const int32_t* __restrict__ parent, float* states,
                   TO* __restrict__ o, int Ts, int H, int slots)
{
    using Sh = TreeShape<D, COLS>;
    constexpr int T = Sh::kThreads, LPR = Sh::LPR, RPP = Sh::RPP, R = Sh::R, kNodes = Sh::kNodes;
    constexpr int E = (kNodes * D + T - 1) / T, EV = (kNodes * COLS + T - 1) / T;
    extern __shared__ __align__(16) ulonglong2 kept[];         // [slots][R][T]
    __shared__ float4 sh_s[kNodes][D], sh_r[kNodes][D];        // a, a, k, k and a k, a k, a q, a q of a channel
    __shared__ float sh_v[kNodes][COLS], sh_beta[kNodes], sh_kq[kNodes][(D + 31) / 32];
    __shared__ ulonglong2 sh_w[RPP / Sh::kInWarp][LPR], sh_p[RPP / Sh::kInWarp][LPR];
    __shared__ __align__(16) float sh_u[COLS];
    __shared__ Plan plan;

    constexpr int kSlabs = D / COLS;
    const int slab = blockIdx.x % kSlabs;
    const long long nh = blockIdx.x / kSlabs;
    const long long n = nh / H, h = nh % H;
    const int tid = threadIdx.x, lane = tid & 31;
    const int c4 = tid % LPR, rg = tid / LPR;
    const int col = slab * COLS + c4 * 4;
    const float* Sp = S_in + nh * (long long)(D * D);

    ulonglong2 s[R];                               // four columns of R rows
#pragma unroll
    for (int r = 0; r < R; ++r) s[r] = __ldcs(reinterpret_cast<const ulonglong2*>(Sp + (rg + r * RPP) * D + col));

    // The inputs of nodes t .. t + kNodes - 1, on their way in registers while
    // the nodes before them take their steps.
    float in_a[E], in_k[E], in_q[E], in_v[EV], in_beta = 0.f;
    auto load_inputs = [&](int t) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int j = (e * T + tid) / D, i = (e * T + tid) % D;
            const long long at = ((n * Ts + t + j) * H + h) * D + i;
            const bool there = t + j < Ts;
            in_a[e] = there ? log_alpha[at] : 0.f;
            in_k[e] = there ? ld_f(k + at) : 0.f;
            in_q[e] = there ? ld_f(q + at) : 0.f;
        }
#pragma unroll
        for (int e = 0; e < EV; ++e) {
            const int j = (e * T + tid) / COLS, i = (e * T + tid) % COLS;
            in_v[e] = t + j < Ts ? ld_f(v + ((n * Ts + t + j) * H + h) * D + slab * COLS + i) : 0.f;
        }
        if (tid < kNodes && t + tid < Ts) in_beta = beta[(n * Ts + t + tid) * H + h];
    };
    load_inputs(0);
    if (tid < 32) make_plan(parent + n * Ts, Ts, slots, lane, plan);

    for (int t = 0; t < Ts; ++t) {
        const int b = t % kNodes;
        if (b == 0) {
            __syncthreads();                       // the steps before have read theirs
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const int j = (e * T + tid) / D, i = (e * T + tid) % D;
                const float a = expf(in_a[e]);
                const float ak = a * in_k[e], aq = a * in_q[e];
                sh_s[j][i] = make_float4(a, a, in_k[e], in_k[e]);
                sh_r[j][i] = make_float4(ak, ak, aq, aq);
                // k . q by the sums of kda_decode.cu: 32 channels by shuffles (its
                // other lanes hold zeros at 16), then those in order
                float kq = in_k[e] * in_q[e];
#pragma unroll
                for (int off = D >= 32 ? 16 : D / 2; off > 0; off >>= 1) kq += __shfl_xor_sync(0xffffffffu, kq, off);
                if (lane % (D >= 32 ? 32 : D) == 0) sh_kq[j][i / 32] = kq;
            }
#pragma unroll
            for (int e = 0; e < EV; ++e) sh_v[(e * T + tid) / COLS][(e * T + tid) % COLS] = in_v[e];
            if (tid < kNodes) sh_beta[tid] = in_beta;
            __syncthreads();
            if (t + kNodes < Ts) load_inputs(t + kNodes);
        }
        const long long tok = (n * Ts + t) * H + h;
        const int from = plan.from[t];
        if (from == kSkip) {
            for (int i = tid; i < COLS; i += T) st_f(o + tok * D + slab * COLS + i, 0.f);
            continue;
        }
        if (t == plan.first && plan.keep_root >= 0) {
#pragma unroll
            for (int r = 0; r < R; ++r) kept[(plan.keep_root * R + r) * T + tid] = s[r];
        }
        if (from >= 0) {
#pragma unroll
            for (int r = 0; r < R; ++r) s[r] = kept[(from * R + r) * T + tid];
        } else if (from == kMemory) {
            const int p = plan.parent[t];
            const float* Sr = p < 0 ? Sp : states + ((n * Ts + p) * H + h) * (long long)(D * D);
#pragma unroll
            for (int r = 0; r < R; ++r)
                s[r] = *reinterpret_cast<const ulonglong2*>(Sr + (long long)(rg + r * RPP) * D + col);
        }
        ulonglong2 w = make_ulonglong2(0, 0), p2 = w;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const ulonglong2 f = *reinterpret_cast<const ulonglong2*>(&sh_r[b][rg + r * RPP]);
            w.x = fma2(f.x, s[r].x, w.x);
            w.y = fma2(f.x, s[r].y, w.y);
            p2.x = fma2(f.y, s[r].x, p2.x);
            p2.y = fma2(f.y, s[r].y, p2.y);
        }
#pragma unroll
        for (int off = LPR; off < LPR * Sh::kInWarp; off <<= 1) {
            w.x = shfl_add2(w.x, off);
            w.y = shfl_add2(w.y, off);
            p2.x = shfl_add2(p2.x, off);
            p2.y = shfl_add2(p2.y, off);
        }
        if (rg % Sh::kInWarp == 0) {
            sh_w[rg / Sh::kInWarp][c4] = w;
            sh_p[rg / Sh::kInWarp][c4] = p2;
        }
        __syncthreads();
        // a thread per column sums w, another p (the same one in a narrow CTA)
        auto column = [&](const ulonglong2 (&y)[RPP / Sh::kInWarp][LPR], int i) {
            const float* x = reinterpret_cast<const float*>(y) + i;
            constexpr int per = Sh::kSummed / Sh::kInWarp;     // 1 or 2
            float sum = 0.f;
#pragma unroll
            for (int g = 0; g < RPP / Sh::kSummed; ++g)
                sum += per == 1 ? x[g * COLS] : x[2 * g * COLS] + x[(2 * g + 1) * COLS];
            return sum;
        };
        constexpr int kFirst = 2 * COLS <= T ? COLS : 0;       // the thread of p's first column
        float psum = 0.f;
        if (tid < COLS) sh_u[tid] = sh_beta[b] * (sh_v[b][tid] - column(sh_w, tid));
        if (tid >= kFirst && tid < kFirst + COLS) psum = column(sh_p, tid - kFirst);
        __syncthreads();
        if (tid >= kFirst && tid < kFirst + COLS) {
            float kqs = 0.f;
#pragma unroll
            for (int i = 0; i < (D + 31) / 32; ++i) kqs += sh_kq[b][i];
            st_f(o + tok * D + slab * COLS + tid - kFirst, fmaf(kqs, sh_u[tid - kFirst], psum));
        }
        const ulonglong2 u = *reinterpret_cast<const ulonglong2*>(&sh_u[c4 * 4]);
        const int keep = plan.keep[t];
        float* Sq = states + tok * (long long)(D * D);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int i = rg + r * RPP;
            const ulonglong2 f = *reinterpret_cast<const ulonglong2*>(&sh_s[b][i]);
            s[r].x = fma2(f.x, s[r].x, mul2(f.y, u.x));
            s[r].y = fma2(f.x, s[r].y, mul2(f.y, u.y));
            ulonglong2* to = reinterpret_cast<ulonglong2*>(Sq + (long long)i * D + col);
            if (keep == kInL2) *to = s[r];
            else __stcs(to, s[r]);
            if (keep >= 0) kept[(keep * R + r) * T + tid] = s[r];
        }
    }
}

template <typename TI, typename TO, int D, int COLS>
cudaError_t launch_cols(const void* q, const void* k, const void* v, const float* g, const float* beta,
                        const float* S_in, const int32_t* parent, float* states, int32_t N, int32_t Ts,
                        int32_t H, void* o, int slots, cudaStream_t stream)
{
    using Sh = TreeShape<D, COLS>;
    const long long blocks = (long long)N * H * (D / COLS);
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    auto kern = decode_tree_kernel<TI, TO, D, COLS>;
    const int bytes = slots * Sh::kSlotBytes;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    kern<<<(unsigned)blocks, Sh::kThreads, bytes, stream>>>(
        static_cast<const TI*>(q), static_cast<const TI*>(k), static_cast<const TI*>(v), g, beta, S_in, parent,
        states, static_cast<TO*>(o), Ts, H, slots);
    return cudaGetLastError();
}

template <typename TI, typename TO, int D>
cudaError_t launch_typed(const void* q, const void* k, const void* v, const float* g, const float* beta,
                         const float* S_in, const int32_t* parent, float* states, int32_t N, int32_t Ts,
                         int32_t H, void* o, cudaStream_t stream)
{
    if constexpr (D == 128) {
        if ((long long)N * H < device_sm_count())
            return launch_cols<TI, TO, D, 32>(q, k, v, g, beta, S_in, parent, states, N, Ts, H, o, 3, stream);
    }
    constexpr int slots = D >= 64 ? 1 : (D == 32 ? 3 : 4);
    return launch_cols<TI, TO, D, (D < 64 ? D : 64)>(q, k, v, g, beta, S_in, parent, states, N, Ts, H, o, slots, stream);
}

template <typename TI, typename TO>
cudaError_t launch_d(int32_t d, const void* q, const void* k, const void* v, const float* g, const float* beta,
                     const float* S_in, const int32_t* parent, float* states, int32_t N, int32_t Ts, int32_t H,
                     void* o, cudaStream_t stream)
{
    switch (d) {
        case 16: return launch_typed<TI, TO, 16>(q, k, v, g, beta, S_in, parent, states, N, Ts, H, o, stream);
        case 32: return launch_typed<TI, TO, 32>(q, k, v, g, beta, S_in, parent, states, N, Ts, H, o, stream);
        case 64: return launch_typed<TI, TO, 64>(q, k, v, g, beta, S_in, parent, states, N, Ts, H, o, stream);
        case 128: return launch_typed<TI, TO, 128>(q, k, v, g, beta, S_in, parent, states, N, Ts, H, o, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace

cudaError_t launch_decode_tree(const void* q, const void* k, const void* v, const float* log_alpha,
                               const float* beta, const float* S_in, const int32_t* parent, float* states,
                               int32_t N, int32_t Ts, int32_t H, int32_t d, kda_dtype_t dtype, void* o,
                               cudaStream_t stream)
{
    switch (dtype) {
        case KDA_BF16:
            return launch_d<__nv_bfloat16, __nv_bfloat16>(d, q, k, v, log_alpha, beta, S_in, parent, states, N, Ts,
                                                          H, o, stream);
        case KDA_BF16_F32OUT:
            return launch_d<__nv_bfloat16, float>(d, q, k, v, log_alpha, beta, S_in, parent, states, N, Ts, H, o,
                                                  stream);
        default:
            return launch_d<float, float>(d, q, k, v, log_alpha, beta, S_in, parent, states, N, Ts, H, o, stream);
    }
}

}  // namespace kda
