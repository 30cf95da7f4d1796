// kda_logprobs.cu -- log probabilities of given tokens, the entropy and the K
// largest alternatives of each row of logits, in one pass over the row.
//
// With m the running maximum, s = sum e^{x - m} and w = sum (x - m) e^{x - m}:
//     lse = m + log s,   log p_i = x_i - lse,   H = log s - w / s.
// A new maximum m' rescales s' = s e^{m - m'}, w' = (w + (m - m') s) e^{m - m'};
// the same rule joins the sums of threads and CTAs.
//
// The K largest come from the same pass.  Order is by value, then by the lower
// index, as one 64-bit key; a NaN ranks with -inf.  The block walks its slice
// in rounds of ascending index and keeps a bound: a key with at least K keys at
// or above it so far.  A round's candidates are its keys above the bound; they
// go to a list in shared memory, which a rank count cuts to K when it grows,
// raising the bound.  Where a round has more candidates than the list can hold
// (the first round, or rising logits), the bound is first raised to the K-th
// largest of the threads' own maxima: then at most K threads have candidates,
// and 32 K of them fit.
//
// One cluster of CTAs per row splits a row into slices when there are few
// rows; the first CTA joins the slices through distributed shared memory.
#include <cooperative_groups.h>

#include "kda_internal.cuh"

namespace kda {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kPerThread = 32;                       // logits per thread and round
constexpr int kRound = kThreads * kPerThread;
constexpr int kList = kMaxAlternatives * kPerThread + kMaxAlternatives;
constexpr int kMaxCluster = 8;
constexpr float kLog2e = 1.4426950408889634f;

typedef unsigned long long Key;                      // 0: none

__device__ __forceinline__ Key make_key(float x, int i)
{
    if (!(x == x)) x = -INFINITY;
    const uint32_t b = __float_as_uint(x + 0.f);     // -0 counts as +0
    const uint32_t o = (b & 0x80000000u) ? ~b : (b | 0x80000000u);
    return ((Key)o << 32) | (uint32_t)~(uint32_t)i;
}

__device__ __forceinline__ int key_index(Key k) { return (int)~(uint32_t)k; }


// max that keeps a NaN, so that a NaN logit shows in the row's results
__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

struct Sums {
    float m, s, w;
};

__device__ __forceinline__ Sums join(const Sums& a, const Sums& b)
{
    Sums r;
    r.m = max_nan(a.m, b.m);
    // an empty or all -inf side: s = w = 0
    const float da = a.m == -INFINITY ? -200.f : a.m - r.m;
    const float db = b.m == -INFINITY ? -200.f : b.m - r.m;
    const float ea = expf(da), eb = expf(db);
    // a difference below -200 has e = 0; the bound keeps 0 * inf out of w
    r.s = a.s * ea + b.s * eb;
    r.w = (a.w + fmaxf(da, -200.f) * a.s) * ea + (b.w + fmaxf(db, -200.f) * b.s) * eb;
    return r;
}

struct Shared {
    Key list[kList];
    Key best[kMaxAlternatives];                      // this CTA's K largest, descending
    Key tmax[kThreads];
    Key bound;
    Sums sums[kWarps];
    Sums mine;                                       // this CTA's sums
    float lse;
    int count;
};

// Cuts the list to its K largest keys, in descending order, and sets the bound
// if there are K of them.  All threads; the list has count keys.
__device__ void cut_list(Shared& sh, int K)
{
    const int n = sh.count;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kThreads) {
        const Key k = sh.list[i];
        int rank = 0;
        for (int j = 0; j < n; ++j) rank += sh.list[j] > k;
        if (rank < K) sh.best[rank] = k;
    }
    __syncthreads();
    const int kept = n < K ? n : K;
    if ((int)threadIdx.x < kept) sh.list[threadIdx.x] = sh.best[threadIdx.x];
    if (threadIdx.x == 0) {
        sh.count = kept;
        if (kept == K && sh.best[K - 1] > sh.bound) sh.bound = sh.best[K - 1];
    }
    __syncthreads();
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
token_logprobs_kernel(const T* __restrict__ logits, long long row_stride,
                      const int32_t* __restrict__ tokens, int V, int J, int K,
                      float* __restrict__ logprobs, float* __restrict__ entropy,
                      int32_t* __restrict__ top_ids, float* __restrict__ top_logprobs)
{
    __shared__ Shared sh;
    cg::cluster_group cluster = cg::this_cluster();
    const int parts = cluster.num_blocks(), part = cluster.block_rank();
    const long long row = blockIdx.x / parts;
    const T* x = logits + row * row_stride;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) {
        sh.count = 0;
        sh.bound = 0;
    }
    __syncthreads();

    const int rounds = (V + kRound - 1) / kRound;
    const int lo = (int)((long long)rounds * part / parts) * kRound;
    const int hi_r = (int)((long long)rounds * (part + 1) / parts) * kRound;
    const int hi = hi_r < V ? hi_r : V;
    Sums a;
    a.m = -INFINITY;
    a.s = a.w = 0.f;
    for (int base = lo; base < hi; base += kRound) {
        float xs[kPerThread];
        float top = -INFINITY;
#pragma unroll
        for (int j = 0; j < kPerThread; ++j) {
            const int i = base + j * kThreads + tid;
            xs[j] = i < hi ? ld_f(x + i) : -INFINITY;
        }
#pragma unroll
        for (int j = 0; j < kPerThread; ++j) top = max_nan(top, xs[j]);
        const float m = max_nan(a.m, top);
        if (m != a.m) {
            const float d = a.m == -INFINITY ? -200.f : fmaxf(a.m - m, -200.f);
            const float e = expf(d);
            a.w = (a.w + d * a.s) * e;
            a.s *= e;
            a.m = m;
        }
        if (m != -INFINITY) {
#pragma unroll
            for (int j = 0; j < kPerThread; ++j) {
                const float d = fmaxf(xs[j] - m, -200.f);
                const float e = exp2f(d * kLog2e);
                a.s += e;
                a.w = fmaf(d, e, a.w);
            }
        }
        if (K > 0) {
            for (;;) {
                const Key bound = sh.bound;
                int mine = 0;
                Key best = 0;
#pragma unroll
                for (int j = 0; j < kPerThread; ++j) {
                    const int i = base + j * kThreads + tid;
                    if (i >= hi) continue;
                    const Key k = make_key(xs[j], i);
                    mine += k > bound;
                    best = k > best ? k : best;
                }
                if (!__syncthreads_or(mine > 0)) break;
                int total = mine;
#pragma unroll
                for (int off = 16; off > 0; off >>= 1) total += __shfl_xor_sync(0xffffffffu, total, off);
                if (lane == 0) sh.tmax[warp] = (Key)total;
                __syncthreads();
                int all = 0;
#pragma unroll
                for (int i = 0; i < kWarps; ++i) all += (int)sh.tmax[i];
                const int have = sh.count;           // read before any thread adds to it
                __syncthreads();
                if (have + all > kList) {
                    // too many: cut the list, raise the bound to the K-th largest thread maximum
                    cut_list(sh, K);
                    sh.tmax[tid] = best;
                    __syncthreads();
                    int rank = 0;
                    for (int j = 0; j < kThreads; ++j) rank += sh.tmax[j] > best;
                    // the bound itself stays a candidate: one below the key
                    if (rank == K - 1 && best != 0 && best - 1 > sh.bound) sh.bound = best - 1;
                    __syncthreads();
                    continue;
                }
                if (mine > 0) {
#pragma unroll
                    for (int j = 0; j < kPerThread; ++j) {
                        const int i = base + j * kThreads + tid;
                        if (i >= hi) continue;
                        const Key k = make_key(xs[j], i);
                        if (k > bound) sh.list[atomicAdd(&sh.count, 1)] = k;
                    }
                }
                __syncthreads();
                if (sh.count > 4 * kMaxAlternatives) cut_list(sh, K);
                break;
            }
        }
    }
    // the CTA's sums
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        Sums b;
        b.m = __shfl_xor_sync(0xffffffffu, a.m, off);
        b.s = __shfl_xor_sync(0xffffffffu, a.s, off);
        b.w = __shfl_xor_sync(0xffffffffu, a.w, off);
        a = join(a, b);
    }
    if (lane == 0) sh.sums[warp] = a;
    __syncthreads();
    if (tid == 0) {
        Sums r = sh.sums[0];
        for (int i = 1; i < kWarps; ++i) r = join(r, sh.sums[i]);
        sh.mine = r;
    }
    if (K > 0) cut_list(sh, K);
    cluster.sync();
    if (part == 0) {
        if (tid == 0) {
            Sums r = sh.mine;
            for (int p = 1; p < parts; ++p) r = join(r, cluster.map_shared_rank(&sh, p)->mine);
            sh.lse = r.m + logf(r.s);
            // no mass at all (every logit -inf): H = 0; m - m is NaN for a NaN or +inf logit
            if (entropy) entropy[row] = r.m == -INFINITY ? 0.f : logf(r.s) - r.w / r.s + (r.m - r.m);
        }
        for (int p = 1; p < parts && K > 0; ++p) {
            const Shared* other = cluster.map_shared_rank(&sh, p);
            const int n = other->count;
            __syncthreads();
            if (tid < n) sh.list[sh.count + tid] = other->list[tid];
            __syncthreads();
            if (tid == 0) sh.count += n;
        }
        __syncthreads();
        const float lse = sh.lse;
        if (K > 0) {
            if (parts > 1) cut_list(sh, K);
            if (tid < K) {
                const Key k = sh.list[tid];
                const int i = key_index(k);
                top_ids[row * K + tid] = i;
                top_logprobs[row * K + tid] = lse == -INFINITY ? -INFINITY : ld_f(x + i) - lse;
            }
        }
        for (int j = tid; j < J; j += kThreads) {
            const int t = tokens[row * J + j];
            logprobs[row * J + j] = (t < 0 || t >= V || lse == -INFINITY) ? -INFINITY : ld_f(x + t) - lse;
        }
    }
    cluster.sync();                                  // the other CTAs' lists have been read
}

}  // namespace

cudaError_t launch_token_logprobs(const void* logits, long long row_stride, const int32_t* tokens,
                                  int32_t T, int32_t V, int32_t J, int32_t K, bool bf16,
                                  float* logprobs, float* entropy, int32_t* top_ids,
                                  float* top_logprobs, cudaStream_t stream)
{
    int parts = 1;
    while (parts < kMaxCluster && (long long)T * parts < 4 * 152 && (long long)parts * 2 * kRound <= V)
        parts *= 2;
    if ((long long)T * parts > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(T * parts));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)parts;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    cudaError_t e;
    if (bf16)
        e = cudaLaunchKernelEx(&cfg, token_logprobs_kernel<__nv_bfloat16>,
                               static_cast<const __nv_bfloat16*>(logits), row_stride, tokens, V, J, K,
                               logprobs, entropy, top_ids, top_logprobs);
    else
        e = cudaLaunchKernelEx(&cfg, token_logprobs_kernel<float>, static_cast<const float*>(logits),
                               row_stride, tokens, V, J, K, logprobs, entropy, top_ids, top_logprobs);
    return e;
}

}  // namespace kda
