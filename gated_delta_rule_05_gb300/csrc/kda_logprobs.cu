// kda_logprobs.cu -- log probabilities of given tokens, the entropy and the K
// largest alternatives of each row of logits, in one pass over the row.
//
// With m the running maximum, s = sum e^{x - m} and w = sum (x - m) e^{x - m}:
//     lse = m + log s,   log p_i = x_i - lse,   H = log s - w / s.
// A new maximum m' rescales s' = s e^{m - m'}, w' = (w + (m - m') s) e^{m - m'};
// the same rule joins the sums of threads and CTAs.
//
// The sums are kept in base 2: t = x log2(e) - m2 in one FMA, with m2 = m log2(e)
// rounded; what the rounding lost comes off before threads' sums meet.  It grows
// with m, and t is no smaller than that where x = m: from |m| = 3e9 on 2^t may
// overflow.  So where the maximum is above 2^20 in magnitude (a thread that has met
// nothing but masked logits of -1e10, say) t = (x - m) log2(e) instead, one more
// operation and a clamp.  512 x 131,072 bf16, nine tenths masked: 59 us with -1e9,
// 55 with -1e4.
//
// The K largest come from the same pass.  Order is by value, then by the lower
// index, as one 64-bit key; a NaN ranks with -inf.  The block walks its slice in
// rounds and keeps a bound: a key with at least K keys at or above it so far, and
// a floor, its value.  A thread whose logits of a round reach the floor puts
// those that do and lie above the bound into a list in shared memory, which a
// rank count cuts to K when it has grown, raising the bound.  The first floor is
// taken from the threads' own maxima.  Rounds that the list cannot hold
// (equal or rising logits) are read again with exact bounds: the bound is raised
// to the K-th largest of the threads' largest keys, then at most K threads have
// candidates, and K times a thread's logits fit.
//
// Rows at any stride: up to 7 logits before the first 16-byte boundary and after
// the last are taken singly; all others come in 16-byte loads, the next round's
// on their way during this one's arithmetic.
//
// Bound by HBM for long batches (4,096 x 50,257 fp32, K = 20: 148 us, 5.6 TB/s, 83 %
// of a copy); 512 x 131,072 bf16 (37 us, 3.6 TB/s) by instructions (60 % of the
// issue slots) and by 512 rows on 152 SMs: three rows on some, four on others.
//
// One cluster of CTAs per row splits a row into slices when there are few rows;
// the first CTA joins the slices through distributed shared memory.
#include <cooperative_groups.h>

#include "kda_verify.cuh"

namespace kda {
namespace {

namespace cg = cooperative_groups;

constexpr int NV = 4;                                // 16-byte loads per thread and round
constexpr int kPerThread = NV * 8;                   // at most so many logits
constexpr int kEnds = 16;                            // at most 14 logits outside whole vectors
constexpr int kList = kMaxAlternatives * kPerThread + kMaxAlternatives + kEnds;
constexpr int kMaxCluster = 8;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kFloor = -200.f;                     // 2^-200 = 0; keeps 0 * inf out of w
constexpr float kLeast = -1e30f;                     // so does this for logits, with m within kNear
constexpr float kNear = 1048576.f;                   // at most 2^-4 is lost of m log2(e) up to here

typedef unsigned long long Key;                      // 0: none

// A number that orders as x does (x is no NaN); above 0.
__device__ __forceinline__ uint32_t order_of(float x)
{
    const uint32_t b = __float_as_uint(x + 0.f);     // -0 counts as +0
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

__device__ __forceinline__ Key make_key(float x, int i)
{
    if (!(x == x)) x = -INFINITY;
    return ((Key)order_of(x) << 32) | (uint32_t)~(uint32_t)i;
}

__device__ __forceinline__ int key_index(Key k) { return (int)~(uint32_t)k; }


__device__ __forceinline__ float key_value(Key k)
{
    const uint32_t o = (uint32_t)(k >> 32);
    return __uint_as_float((o & 0x80000000u) ? (o & 0x7FFFFFFFu) : ~o);
}

// max that keeps a NaN, so that a NaN logit shows in the row's results
__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Pairs of fp32 for the two-wide FMA and add.
__device__ __forceinline__ uint64_t pack2(float a, float b)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
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

__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// m: the largest logit so far (raw); s, w: sums of 2^t and t 2^t relative to m2 =
// m log2(e) rounded, or, where m is far and from settled() on, to m log2(e) itself.
struct Sums {
    float m, s, w;
};

__device__ __forceinline__ bool near(float m) { return fabsf(m) <= kNear; }

// What the rounding of m2 left out.
__device__ __forceinline__ float lost(float m) { return near(m) ? fmaf(m, kLog2e, -(m * kLog2e)) : 0.f; }

// To another maximum, d = (a.m - m) log2(e); a sum of nothing (m = -inf) stays 0.
__device__ __forceinline__ void rescale(Sums& a, float m, float d)
{
    d = fmaxf(d, kFloor);                            // of -inf and NaN too
    const float e = ex2(d);
    a.w = (a.w + d * a.s) * e;
    a.s *= e;
    a.m = m;
}

__device__ __forceinline__ void raise(Sums& a, float m)
{
    rescale(a, m, (a.m - m) * kLog2e + (lost(m) - lost(a.m)));
}

__device__ __forceinline__ Sums settled(Sums a)
{
    rescale(a, a.m, -lost(a.m));
    return a;
}

__device__ __forceinline__ Sums join(Sums a, Sums b)
{
    const float m = max_nan(a.m, b.m);
    rescale(a, m, (a.m - m) * kLog2e);
    rescale(b, m, (b.m - m) * kLog2e);
    a.s += b.s;
    a.w += b.w;
    return a;
}

template <int kThreads>
struct Shared {
    static constexpr int kWarps = kThreads / 32;
    Key list[kList];
    Key best[kMaxAlternatives];                      // this CTA's K largest, descending
    Key tmax[kThreads];
    uint32_t wtop[kWarps];
    Key bound;
    float floor;                                     // the bound's value
    Sums sums[kWarps];
    Sums mine;                                       // this CTA's sums
    float lse;
    int count, kept;                                 // keys in the list; those of the last cut
};

// Cuts the list to its K largest keys, in descending order, and sets the bound
// if there are K of them.  All threads; the list has count keys.
template <int kThreads>
__device__ void cut_list(Shared<kThreads>& sh, int K)
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
        sh.count = sh.kept = kept;
        if (kept == K && (sh.best[K - 1] > sh.bound || sh.bound == 0)) {
            sh.bound = sh.best[K - 1];
            sh.floor = key_value(sh.bound);
        }
    }
    __syncthreads();
}

// 16 bytes of logits: their maximum, and one of them as fp32.
__device__ __forceinline__ uint32_t max2_nan(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

template <typename T>
struct Vec;
template <>
struct Vec<float> {
    static constexpr int kN = 4;
    static constexpr uint32_t kNone = 0xff800000u;   // -inf
    static __device__ __forceinline__ float max(const uint4& v)
    {
        return max_nan(max_nan(__uint_as_float(v.x), __uint_as_float(v.y)),
                       max_nan(__uint_as_float(v.z), __uint_as_float(v.w)));
    }
    static __device__ __forceinline__ float get(const uint4& v, int i)
    {
        return __uint_as_float(i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w);
    }
    // -inf (and all below kLeast) as kLeast: its 2^t is 0 and t 2^t too
    static __device__ __forceinline__ uint4 clamp(const uint4& v)
    {
        return make_uint4(__float_as_uint(max_nan(__uint_as_float(v.x), kLeast)),
                          __float_as_uint(max_nan(__uint_as_float(v.y), kLeast)),
                          __float_as_uint(max_nan(__uint_as_float(v.z), kLeast)),
                          __float_as_uint(max_nan(__uint_as_float(v.w), kLeast)));
    }
};
template <>
struct Vec<__nv_bfloat16> {
    static constexpr int kN = 8;
    static constexpr uint32_t kNone = 0xff80ff80u;   // two of -inf
    static __device__ __forceinline__ float max(const uint4& v)
    {
        const uint32_t m = max2_nan(max2_nan(v.x, v.y), max2_nan(v.z, v.w));
        return max_nan(__uint_as_float(m << 16), __uint_as_float(m & 0xFFFF0000u));
    }
    static __device__ __forceinline__ float get(const uint4& v, int i)
    {
        const uint32_t w = i < 2 ? v.x : i < 4 ? v.y : i < 6 ? v.z : v.w;
        return __uint_as_float((i & 1) ? w & 0xFFFF0000u : w << 16);
    }
    static __device__ __forceinline__ uint4 clamp(const uint4& v)
    {
        constexpr uint32_t least = 0xf149f149u;      // two of -9.95e29
        return make_uint4(max2_nan(v.x, least), max2_nan(v.y, least), max2_nan(v.z, least), max2_nan(v.w, least));
    }
};

// The candidates of one round, read again: a thread has kPerThread logits at
// most, so that with the bound at the K-th largest of the threads' largest keys
// all candidates fit the list.
template <typename Vx, int kThreads>
__device__ __noinline__ void exact_round(Shared<kThreads>& sh, const uint4* vec, int head, int vb, int v1, int K)
{
    constexpr int kWarps = kThreads / 32;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    auto each = [&](auto&& f) {
#pragma unroll 1
        for (int v = vb + tid; v < v1 && v < vb + kThreads * NV; v += kThreads) {
            const uint4 x = __ldg(vec + v);
#pragma unroll
            for (int i = 0; i < Vx::kN; ++i) f(make_key(Vx::get(x, i), head + v * Vx::kN + i));
        }
    };
    for (;;) {
        const Key bound = sh.bound;
        int mine = 0;
        Key best = 0;
        each([&](Key k) {
            mine += k > bound;
            best = k > best ? k : best;
        });
        int total = mine;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) total += __shfl_xor_sync(0xffffffffu, total, off);
        if (lane == 0) sh.tmax[warp] = (Key)total;
        __syncthreads();
        int all = sh.count;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) all += (int)sh.tmax[i];
        __syncthreads();
        if (all <= kList) {
            if (mine > 0)
                each([&](Key k) {
                    if (k > bound) sh.list[atomicAdd(&sh.count, 1)] = k;
                });
            __syncthreads();
            cut_list(sh, K);
            return;
        }
        sh.tmax[tid] = best;
        __syncthreads();
        int rank = 0;
#pragma unroll 4
        for (int j = 0; j < kThreads; ++j) rank += sh.tmax[j] > best;
        // the new bound itself stays a candidate: one below the key
        if (rank == K - 1 && best != 0 && best - 1 > bound) {
            sh.bound = best - 1;
            sh.floor = key_value(best);
        }
        __syncthreads();
    }
}

// Cuts the list after the rounds [since, to): its first `kept` keys are those of
// the cut before.  Where the rounds had more candidates than the list holds they
// are read again.
template <typename Vx, int kThreads>
__device__ __forceinline__ void settle(Shared<kThreads>& sh, const uint4* vec, int head, int since, int to, int v1, int K)
{
    __syncthreads();
    if (sh.count <= kList) {
        cut_list(sh, K);
        return;
    }
    __syncthreads();
    if (threadIdx.x == 0) sh.count = sh.kept;
    __syncthreads();
    for (int vb = since; vb < to; vb += kThreads * NV) exact_round<Vx>(sh, vec, head, vb, v1, K);
}

template <typename T, int kThreads>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads)
token_logprobs_kernel(const T* __restrict__ logits, long long row_stride,
                      const int32_t* __restrict__ tokens, int V, int J, int K,
                      float* __restrict__ logprobs, float* __restrict__ entropy,
                      int32_t* __restrict__ top_ids, float* __restrict__ top_logprobs)
{
    using Vx = Vec<T>;
    constexpr int kWarps = kThreads / 32;
    __shared__ Shared<kThreads> sh;
    cg::cluster_group cluster = cg::this_cluster();
    const int parts = cluster.num_blocks(), part = cluster.block_rank();
    const long long row = blockIdx.x / parts;
    const T* x = logits + row * row_stride;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // whole vectors from element `head` on, this CTA's slice of them [v0, v1)
    const int skew = (int)(reinterpret_cast<uintptr_t>(x) / sizeof(T)) & (Vx::kN - 1);
    const int head = skew ? (Vx::kN - skew < V ? Vx::kN - skew : V) : 0;
    const int nv = (V - head) / Vx::kN;
    const int v0 = (int)((long long)nv * part / parts), v1 = (int)((long long)nv * (part + 1) / parts);
    const uint4* vec = reinterpret_cast<const uint4*>(x + head);
    uint4 cur[NV];
    auto fetch = [&](int vb) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int v = vb + j * kThreads + tid;
            cur[j] = v < v1 ? __ldcs(vec + v) : make_uint4(Vx::kNone, Vx::kNone, Vx::kNone, Vx::kNone);
        }
    };
    fetch(v0);
    float given = -INFINITY;                         // the logit of given token tid
    bool outside = true;                             // whether there is none
    if (part == 0 && tid < J) {
        const int t = tokens[row * J + tid];
        outside = t < 0 || t >= V;
        if (!outside) given = ld_f(x + t);
    }
    if (tid == 0) {
        sh.count = sh.kept = part == 0 ? V - nv * Vx::kN : 0;
        sh.bound = 0;
        sh.floor = -INFINITY;
    }
    __syncthreads();
    Sums a;
    a.m = -INFINITY;
    a.s = a.w = 0.f;
    const int ends = part == 0 ? V - nv * Vx::kN : 0;   // the logits outside whole vectors
    if (tid < ends) {
        const int i = tid < head ? tid : tid + nv * Vx::kN;
        a.m = ld_f(x + i);
        if (a.m != -INFINITY) {
            const float t = lost(a.m);
            a.s = ex2(t);
            a.w = t * a.s;
        }
        if (K > 0) sh.list[tid] = make_key(a.m, i);
    }
    int round = 0, sync_at = 1, since = v0;          // rounds, and the first vector not settled
    float floor = -INFINITY;
    Key bound = 0;
    for (int vb = v0; vb < v1; vb += kThreads * NV) {
        uint4 now[NV];
        float top = -INFINITY;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            now[j] = cur[j];
            top = max_nan(top, Vx::max(now[j]));
        }
        if (vb + kThreads * NV < v1) fetch(vb + kThreads * NV);
        if (!(top <= a.m)) raise(a, max_nan(a.m, top));
        const uint64_t c2 = pack2(kLog2e, kLog2e);
        uint64_t s2 = 0, w2 = 0;
        if (near(a.m) || a.m == -INFINITY) {
            const float m2 = a.m == -INFINITY ? 0.f : a.m * kLog2e;
            const uint64_t b2 = pack2(-m2, -m2);
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const uint4 y = Vx::clamp(now[j]);
#pragma unroll
                for (int i = 0; i < Vx::kN; i += 2) {
                    const uint64_t t = fma2(pack2(Vx::get(y, i), Vx::get(y, i + 1)), c2, b2);
                    float t0, t1;
                    unpack2(t, t0, t1);
                    const uint64_t e = pack2(ex2(t0), ex2(t1));
                    s2 = add2(s2, e);
                    w2 = fma2(t, e, w2);
                }
            }
        } else {
            // -inf, and what overflows, as kFloor; m keeps a NaN
            const uint64_t b2 = pack2(-a.m, -a.m);
#pragma unroll
            for (int j = 0; j < NV; ++j) {
#pragma unroll
                for (int i = 0; i < Vx::kN; i += 2) {
                    float t0, t1;
                    unpack2(mul2(add2(pack2(Vx::get(now[j], i), Vx::get(now[j], i + 1)), b2), c2), t0, t1);
                    t0 = fmaxf(t0, kFloor);
                    t1 = fmaxf(t1, kFloor);
                    const uint64_t e = pack2(ex2(t0), ex2(t1));
                    s2 = add2(s2, e);
                    w2 = fma2(pack2(t0, t1), e, w2);
                }
            }
        }
        {
            float x0, x1;
            unpack2(s2, x0, x1);
            a.s += x0 + x1;
            unpack2(w2, x0, x1);
            a.w += x0 + x1;
        }
        if (K == 0) continue;
        // Candidates.  `top` is the maximum of this round alone.
        if (vb == v0) {
            // Each warp's r-th largest thread maximum, r = ceil(K / warps): the
            // least of them has at least K logits at or above it.
            uint32_t mine = order_of(top == top ? top : -INFINITY), last = 0;
            for (int r = 0; r < K; r += kWarps) {
                last = __reduce_max_sync(0xffffffffu, mine);
                const uint32_t who = __ballot_sync(0xffffffffu, mine == last);
                if (lane == __ffs(who) - 1) mine = 0;
            }
            if (lane == 0) sh.wtop[warp] = last;
            __syncthreads();
            uint32_t least = sh.wtop[0];
#pragma unroll
            for (int i = 1; i < kWarps; ++i) least = min(least, sh.wtop[i]);
            floor = least != 0 ? key_value((Key)least << 32) : -INFINITY;
        }
        if (!(top < floor)) {
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                if (Vx::max(now[j]) < floor) continue;
                const int v = vb + j * kThreads + tid;
#pragma unroll
                for (int i = 0; i < Vx::kN; ++i) {
                    const float y = Vx::get(now[j], i);
                    if (!(y < floor) && v < v1) {
                        const Key k = make_key(y, head + v * Vx::kN + i);
                        if (k > bound) {
                            const int at = atomicAdd(&sh.count, 1);
                            if (at < kList) sh.list[at] = k;
                        }
                    }
                }
            }
        }
        if (++round == sync_at) {
            // Later rounds meet fewer new candidates: the list is cut after 1,
            // 2, 4, 8, ... of them.
            sync_at *= 2;
            settle<Vx>(sh, vec, head, since, vb + kThreads * NV, v1, K);
            since = vb + kThreads * NV;
            bound = sh.bound;
            floor = sh.floor > floor ? sh.floor : floor;
        }
    }
    if (K > 0) settle<Vx>(sh, vec, head, since, v1, v1, K);
    // the CTA's sums
    a = settled(a);
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
    cluster.sync();
    if (part == 0) {
        if (tid == 0) {
            Sums r = sh.mine;
            for (int p = 1; p < parts; ++p) r = join(r, cluster.map_shared_rank(&sh, p)->mine);
            sh.lse = r.m + logf(r.s);
            // no mass at all (every logit -inf): H = 0; m - m is NaN for a NaN or +inf logit
            if (entropy)
                entropy[row] = r.m == -INFINITY ? 0.f : logf(r.s) - kLn2 * (r.w / r.s) + (r.m - r.m);
        }
        for (int p = 1; p < parts && K > 0; ++p) {
            const Shared<kThreads>* other = cluster.map_shared_rank(&sh, p);
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
                top_logprobs[row * K + tid] = lse == -INFINITY ? -INFINITY : key_value(k) - lse;
            }
        }
        if (tid < J) logprobs[row * J + tid] = outside || lse == -INFINITY ? -INFINITY : given - lse;
        for (int j = tid + kThreads; j < J; j += kThreads) {
            const int t = tokens[row * J + j];
            logprobs[row * J + j] = (t < 0 || t >= V || lse == -INFINITY) ? -INFINITY : ld_f(x + t) - lse;
        }
    }
    cluster.sync();                                  // the other CTAs' lists have been read
}

template <typename T, int kThreads>
cudaError_t launch(const void* logits, long long row_stride, const int32_t* tokens, int T_rows, int V, int J,
                   int K, int parts, float* logprobs, float* entropy, int32_t* top_ids, float* top_logprobs,
                   cudaStream_t stream)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(T_rows * parts));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)parts;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, token_logprobs_kernel<T, kThreads>, static_cast<const T*>(logits), row_stride,
                              tokens, V, J, K, logprobs, entropy, top_ids, top_logprobs);
}

}  // namespace

// Many rows: a CTA of 128 threads per row, eight on an SM, whose reductions
// hide behind one another's loads.  Few rows: 256 threads, and up to eight CTAs
// per row as long as they are not more than two per SM.  Measured on one GB300 in a
// graph (128 and 256 threads): 4,096 x 50,257 fp32, K = 20, 147 and 160 us; 2,048 x
// 131,072 bf16, K = 8, 102 and 108 us; 512 x 131,072 38 and 34 us; 1 x 131,072,
// K = 20, eight CTAs, 16 and 12 us.  Two and four parts a row at 512 rows: 41 and 56
// us, with 128 threads 35 and 46; at 200 rows one part 23, two (taken) 20, four 28.
cudaError_t launch_token_logprobs(const void* logits, long long row_stride, const int32_t* tokens,
                                  int32_t T, int32_t V, int32_t J, int32_t K, bool bf16,
                                  float* logprobs, float* entropy, int32_t* top_ids,
                                  float* top_logprobs, cudaStream_t stream)
{
    const int sms = device_sm_count() > 0 ? device_sm_count() : 1;
    const bool many = T >= 4 * (long long)sms;
    int parts = 1;
    while (parts < kMaxCluster && (long long)T * parts < 2 * sms && V / (2 * parts) >= 2048) parts *= 2;
    if ((long long)T * parts > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    const auto call = bf16 ? (many ? launch<__nv_bfloat16, 128> : launch<__nv_bfloat16, 256>)
                           : (many ? launch<float, 128> : launch<float, 256>);
    return call(logits, row_stride, tokens, T, V, J, K, parts, logprobs, entropy, top_ids, top_logprobs, stream);
}

}  // namespace kda
