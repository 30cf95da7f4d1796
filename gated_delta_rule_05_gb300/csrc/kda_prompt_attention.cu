// kda_prompt_attention.cu -- causal attention over packed prompts on the CUDA
// cores, fp32 arithmetic: every type, head size and scale.  It runs when KDA_FORCE_SIMT is
// set, as something to compare the tensor-core kernels with that shares none of their
// products.
//
// One thread block per 64 query rows of a (sequence, cache head): the rows of the
// heads that share a cache head are laid out token by token, row r being head r % G
// of token r / G, so that they share every key and value tile.  Per tile of 64 keys
//     S = Q K^T, P = 2^(c S - m), O = O 2^(m' - m) + P V       (c = scale log2 e)
// with the running maximum m and sum l of each row; a thread has 4 rows and 4 keys of
// S (16 threads to a row) and 4 rows and d / 16 channels of O.
//
// A tile that some row does not see whole is masked key by key, in the second product
// too: there a key counts only for the rows that see it, so that an infinity or
// NaN in a value stays with them.
//
// Bound by fp32 FMAs and the shared memory that feeds them: 12 prompts of 512 to 12,288
// tokens, 32 heads on 8, d = 128, bf16, 119 ms (45 TFLOP/s of 75), where tcgen05 takes 3.6 ms;
// 7 fp32 prompts of up to 1,500, 12 heads on 4, d = 64, 353 us, fp16 pairs 130.
#include "kda_prompt.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr int BM = 64, BN = 64;
constexpr int PS = BM + 4;              // row pitch of P^T

template <int D>
struct Shape {
    static constexpr int QS = D + 4;    // row pitch of Q and K
    static constexpr int VC = D >= 64 ? 4 : D / 16;     // channels in a row of a thread's vectors
    static constexpr int NV = D / 16 / VC;
    // K's place is P's after the first product
    static constexpr int kK = BN * QS > BN * PS ? BN * QS : BN * PS;
    static constexpr size_t kBytes = sizeof(float) * (BM * QS + kK + BN * D);
};

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float4 load4(const float* p) { return __ldg(reinterpret_cast<const float4*>(p)); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p)
{
    const uint2 w = __ldg(reinterpret_cast<const uint2*>(p));
    return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u), __uint_as_float(w.y << 16),
                       __uint_as_float(w.y & 0xFFFF0000u));
}

template <int VC>
struct Vec {
    float x[VC];
};
template <int VC>
__device__ __forceinline__ Vec<VC> load_vec(const float* p)
{
    Vec<VC> r;
    if constexpr (VC == 4) {
        const float4 w = *reinterpret_cast<const float4*>(p);
        r.x[0] = w.x; r.x[1] = w.y; r.x[2] = w.z; r.x[3] = w.w;
    } else if constexpr (VC == 2) {
        const float2 w = *reinterpret_cast<const float2*>(p);
        r.x[0] = w.x; r.x[1] = w.y;
    } else {
        r.x[0] = *p;
    }
    return r;
}

// Block b's sequence and the block's place among that sequence's; all threads
// call it.  False: there is none.
__device__ bool locate(const PromptArgs& a, long long b, int& seq, int& tile)
{
    __shared__ long long sh_sum[kThreads / 32];
    __shared__ int sh_seq, sh_tile;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) sh_seq = -1;
    long long base = 0;
    for (int n0 = 0; n0 < a.N; n0 += kThreads) {
        const int n = n0 + tid;
        long long w = 0;
        if (n < a.N) {
            int first, count;
            prompt_rows(a.cu_q, n, a.T, first, count);
            w = ((long long)count * a.G + BM - 1) / BM;
        }
        long long incl = w;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const long long x = __shfl_up_sync(0xffffffffu, incl, off);
            if (lane >= off) incl += x;
        }
        if (lane == 31) sh_sum[warp] = incl;
        __syncthreads();
        long long before = base, all = 0;
        for (int i = 0; i < kThreads / 32; ++i) {
            if (i < warp) before += sh_sum[i];
            all += sh_sum[i];
        }
        if (b >= before + incl - w && b < before + incl) {
            sh_seq = n;
            sh_tile = (int)(w - 1 - (b - (before + incl - w)));     // a prompt's last rows, the longest work, first
        }
        base += all;
        __syncthreads();
        if (b < base) break;
    }
    __syncthreads();
    seq = sh_seq;
    tile = sh_tile;
    return seq >= 0;
}

template <class T, class O, int D>
__global__ void __launch_bounds__(kThreads, 2)
prompt_attention_kernel(const __grid_constant__ PromptArgs a)
{
    using S = Shape<D>;
    extern __shared__ __align__(16) float dyn[];
    float* sq = dyn;
    float* sk = sq + BM * S::QS;
    float* sv = sk + S::kK;
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const int hk = blockIdx.y;
    int n, tile;
    if (!locate(a, blockIdx.x, n, tile)) return;
    const PromptSeq s = prompt_seq(a, n);
    const int off = s.lk - s.lq;                           // token t sees the keys up to t + off
    const long long rows = (long long)s.lq * a.G;
    const long long r0 = (long long)tile * BM;
    const int here = rows - r0 < BM ? (int)(rows - r0) : BM;

    // the rows' queries
    for (int e = tid; e < BM * (D / 4); e += kThreads) {
        const int r = e / (D / 4), c = e % (D / 4) * 4;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r < here) {
            const int t = (int)((r0 + r) / a.G), g = (int)((r0 + r) - (long long)t * a.G);
            x = load4(static_cast<const T*>(a.q) + (long long)(s.q0 + t) * a.q_stride + ((long long)hk * a.G + g) * D + c);
        }
        *reinterpret_cast<float4*>(sq + r * S::QS + c) = x;
    }
    int lim[4];                                            // keys that each of the thread's rows sees
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = ty * 4 + i;
        lim[i] = r < here ? min(max((int)((r0 + r) / a.G) + off + 1, 0), s.lk) : 0;
    }
    const int most = min(max((int)((r0 + here - 1) / a.G) + off + 1, 0), s.lk);
    const int all = min(max((int)(r0 / a.G) + off + 1, 0), s.lk);      // keys that every row sees

    float m[4], l[4], o[4][S::NV][S::VC];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.f;
#pragma unroll
        for (int j = 0; j < S::NV; ++j)
#pragma unroll
            for (int c = 0; c < S::VC; ++c) o[i][j][c] = 0.f;
    }
    const T* kp = static_cast<const T*>(a.k) + (long long)s.k0 * a.k_stride + (long long)hk * D;
    const T* vp = static_cast<const T*>(a.v) + (long long)s.k0 * a.v_stride + (long long)hk * D;
#pragma unroll 1
    for (int k0 = 0; k0 < most; k0 += BN) {
        __syncthreads();                                   // the last tile has been read
        for (int e = tid; e < BN * (D / 4); e += kThreads) {
            const int j = e / (D / 4), c = e % (D / 4) * 4;
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
            if (k0 + j < most) {
                x = load4(kp + (long long)(k0 + j) * a.k_stride + c);
                y = load4(vp + (long long)(k0 + j) * a.v_stride + c);
            }
            *reinterpret_cast<float4*>(sk + j * S::QS + c) = x;
            *reinterpret_cast<float4*>(sv + j * D + c) = y;
        }
        __syncthreads();
        // scores of rows ty * 4 + i and keys tx + 16 j
        float x[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) x[i][j] = 0.f;
#pragma unroll 4
        for (int c = 0; c < D; c += 4) {
            float4 q4[4], k4[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) q4[i] = *reinterpret_cast<const float4*>(sq + (ty * 4 + i) * S::QS + c);
#pragma unroll
            for (int j = 0; j < 4; ++j) k4[j] = *reinterpret_cast<const float4*>(sk + (tx + 16 * j) * S::QS + c);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    x[i][j] = fmaf(q4[i].x, k4[j].x, x[i][j]);
                    x[i][j] = fmaf(q4[i].y, k4[j].y, x[i][j]);
                    x[i][j] = fmaf(q4[i].z, k4[j].z, x[i][j]);
                    x[i][j] = fmaf(q4[i].w, k4[j].w, x[i][j]);
                }
        }
        const bool masked = k0 + BN > all;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float top = -INFINITY;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                x[i][j] *= a.scale_log2;
                if (masked && k0 + tx + 16 * j >= lim[i]) x[i][j] = -INFINITY;
                top = fmaxf(top, x[i][j]);
            }
#pragma unroll
            for (int w = 8; w > 0; w >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
            const float m2 = fmaxf(m[i], top);
            const float f = m2 == -INFINITY ? 1.f : ex2(m[i] - m2);
            const float ref = m2 == -INFINITY ? 0.f : m2;
            m[i] = m2;
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                x[i][j] = ex2(x[i][j] - ref);
                sum += x[i][j];
            }
            l[i] = l[i] * f + sum;                         // of the thread's keys; added up at the end
#pragma unroll
            for (int j = 0; j < S::NV; ++j)
#pragma unroll
                for (int c = 0; c < S::VC; ++c) o[i][j][c] *= f;
        }
        __syncthreads();                                   // the scores are there: P over K
#pragma unroll
        for (int j = 0; j < 4; ++j)
            *reinterpret_cast<float4*>(sk + (tx + 16 * j) * PS + ty * 4) = make_float4(x[0][j], x[1][j], x[2][j], x[3][j]);
        __syncthreads();
        const int keys = min(BN, most - k0);
        if (!masked) {
#pragma unroll 4
            for (int j = 0; j < BN; ++j) {
                const float4 p4 = *reinterpret_cast<const float4*>(sk + j * PS + ty * 4);
                const float p[4] = {p4.x, p4.y, p4.z, p4.w};
#pragma unroll
                for (int w = 0; w < S::NV; ++w) {
                    const Vec<S::VC> v = load_vec<S::VC>(sv + j * D + w * 16 * S::VC + tx * S::VC);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int c = 0; c < S::VC; ++c) o[i][w][c] = fmaf(p[i], v.x[c], o[i][w][c]);
                }
            }
        } else {
#pragma unroll 1
            for (int j = 0; j < keys; ++j) {
                const float4 p4 = *reinterpret_cast<const float4*>(sk + j * PS + ty * 4);
                const float p[4] = {p4.x, p4.y, p4.z, p4.w};
#pragma unroll
                for (int w = 0; w < S::NV; ++w) {
                    const Vec<S::VC> v = load_vec<S::VC>(sv + j * D + w * 16 * S::VC + tx * S::VC);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (k0 + j < lim[i])
#pragma unroll
                            for (int c = 0; c < S::VC; ++c) o[i][w][c] = fmaf(p[i], v.x[c], o[i][w][c]);
                }
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int w = 8; w > 0; w >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], w);
        const int r = ty * 4 + i;
        if (r >= here) continue;
        const float inv = lim[i] == 0 ? 0.f : 1.f / l[i];
        const int t = (int)((r0 + r) / a.G), g = (int)((r0 + r) - (long long)t * a.G);
        O* op = static_cast<O*>(a.o) + ((long long)(s.q0 + t) * a.Hq + (long long)hk * a.G + g) * D;
#pragma unroll
        for (int w = 0; w < S::NV; ++w)
#pragma unroll
            for (int c = 0; c < S::VC; ++c)
                op[w * 16 * S::VC + tx * S::VC + c] = lim[i] == 0 ? O(0.f) : O(o[i][w][c] * inv);
    }
}

template <class T, class O, int D>
cudaError_t launch(const PromptArgs& a, cudaStream_t stream)
{
    auto kern = prompt_attention_kernel<T, O, D>;
    const size_t bytes = Shape<D>::kBytes;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e != cudaSuccess) return e;
    // every sequence has at most one tile that is not full
    const long long tiles = ((long long)a.T * a.G) / BM + a.N;
    if (tiles > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    kern<<<dim3((unsigned)tiles, (unsigned)a.Hkv), kThreads, bytes, stream>>>(a);
    return cudaGetLastError();
}

template <class T, class O>
cudaError_t launch_d(const PromptArgs& a, int32_t d, cudaStream_t stream)
{
    switch (d) {
    case 16: return launch<T, O, 16>(a, stream);
    case 32: return launch<T, O, 32>(a, stream);
    case 64: return launch<T, O, 64>(a, stream);
    default: return launch<T, O, 128>(a, stream);
    }
}

}  // namespace

cudaError_t launch_prompt_attention(const PromptArgs& a, int32_t d, kda_dtype_t dtype, cudaStream_t stream)
{
    if (dtype == KDA_BF16) return launch_d<__nv_bfloat16, __nv_bfloat16>(a, d, stream);
    if (dtype == KDA_BF16_F32OUT) return launch_d<__nv_bfloat16, float>(a, d, stream);
    return launch_d<float, float>(a, d, stream);
}

}  // namespace kda
