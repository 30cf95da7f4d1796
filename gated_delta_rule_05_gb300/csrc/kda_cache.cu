// kda_cache.cu -- rows of drafted or prompt tokens into the pages of a cache:
// a gather of accepted rows (kda_cache_commit) or a packed batch
// (kda_cache_append) to positions lengths[n] + i of each sequence, for every
// layer and both of K and V in one launch.  Bound by the bytes it moves.
//
// A block moves as many rows of one layer as one pass of its threads covers, with
// kDepth 16-byte pieces of K and of V per thread in flight.  Its first threads work
// out where each row goes (sequence, position, page).  One pass per block, rather
// than 32 rows of 2 KB in four passes, took the commit of 32 x 16 rows of 8 layers
// from 6.4 to 5.3 us (in a graph) and the append of 16 prompts from 172 to 165 us,
// 100 % of the measured copy bandwidth; depths 1 and 2 took 167 and 170.
#include "kda_verify.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr int kDepth = 4;

__host__ __device__ int rows_per_block(long long row_bytes)
{
    const long long rows = kDepth * kThreads * 16 / row_bytes;
    return rows < 1 ? 1 : rows > kThreads ? kThreads : (int)rows;
}

// The packed rows of sequence n: from cu_seqlens[n] to cu_seqlens[n + 1], as far as
// they exist.
__device__ __forceinline__ int first_row(const CacheArgs& a, int n)
{
    const int r = __ldg(a.cu_seqlens + n);
    return r > 0 ? r : 0;
}
__device__ __forceinline__ int row_count(const CacheArgs& a, int n)
{
    const long long end = __ldg(a.cu_seqlens + n + 1), most = end < a.rows ? end : a.rows;
    const long long c = most - first_row(a, n);
    return c > 0 ? (int)c : 0;
}

__global__ void __launch_bounds__(kThreads)
cache_rows_kernel(const CacheArgs a)
{
    __shared__ long long sh_dst[kThreads];           // byte offset in a layer's cache; -1: not written
    __shared__ long long sh_src[kThreads];           // row of k and v
    const int tid = threadIdx.x;
    const int vecs = a.row_bytes / 16, block_rows = rows_per_block(a.row_bytes);
    const long long first = (long long)blockIdx.x * block_rows;
    if (tid < block_rows) {
        const long long r = first + tid;
        long long src = -1, dst = -1;
        if (r < a.rows) {
            int n, i;
            bool there;
            src = r;
            if (a.cu_seqlens) {
                int lo = 0, hi = a.N;                // the last n with cu[n] <= r
                while (hi - lo > 1) {
                    const int mid = (lo + hi) / 2;
                    if (__ldg(a.cu_seqlens + mid) <= r) lo = mid;
                    else hi = mid;
                }
                n = lo;
                i = (int)(r - first_row(a, n));
                there = i >= 0 && i < row_count(a, n);
            } else {
                n = (int)(r / a.Ts);
                i = (int)(r - (long long)n * a.Ts);
                there = !a.count || i < __ldg(a.count + n);
                if (there && a.path) {
                    const int t = __ldg(a.path + r);
                    there = t >= 0 && t < a.Ts;
                    src = (long long)n * a.Ts + t;
                }
            }
            const int len = __ldg(a.lengths + n);
            const long long pos = (long long)len + i;
            if (there && len >= 0 && pos < (long long)a.max_pages * a.page_size) {
                const int p = (int)(pos / a.page_size);
                const int page = __ldg(a.page_table + (long long)n * a.max_pages + p);
                if (page >= 0 && page < a.num_pages)
                    dst = page * a.page_bytes + (pos - (long long)p * a.page_size) * a.row_bytes;
            }
        }
        sh_src[tid] = src;
        sh_dst[tid] = dst;
    }
    if (a.new_lengths && blockIdx.y == 0) {
        for (long long n = (long long)blockIdx.x * kThreads + tid; n < a.N;
             n += (long long)gridDim.x * kThreads) {
            int c;
            if (a.cu_seqlens) {
                c = row_count(a, n);
            } else {
                c = a.count ? a.count[n] : a.Ts;
                c = c < 0 ? 0 : (c > a.Ts ? a.Ts : c);
            }
            a.new_lengths[n] = a.lengths[n] + c;
        }
    }
    __syncthreads();
    const long long src_layer = (long long)blockIdx.y * a.rows * a.row_bytes;
    const long long dst_layer = (long long)blockIdx.y * a.layer_bytes;
    const int count = block_rows * vecs;
    for (int e0 = tid; e0 < count; e0 += kDepth * kThreads) {
        uint4 k[kDepth], v[kDepth];
        long long to[kDepth];
#pragma unroll
        for (int i = 0; i < kDepth; ++i) {
            const int e = e0 + i * kThreads, r = e / vecs, c = e - r * vecs;
            to[i] = e < count ? sh_dst[r] : -1;
            if (to[i] < 0) continue;
            const long long s = src_layer + sh_src[r] * a.row_bytes + 16ll * c;
            to[i] += dst_layer + 16ll * c;
            k[i] = __ldcs(reinterpret_cast<const uint4*>(a.k + s));
            v[i] = __ldcs(reinterpret_cast<const uint4*>(a.v + s));
        }
#pragma unroll
        for (int i = 0; i < kDepth; ++i)
            if (to[i] >= 0) {
                *reinterpret_cast<uint4*>(a.k_cache + to[i]) = k[i];
                *reinterpret_cast<uint4*>(a.v_cache + to[i]) = v[i];
            }
    }
}

}  // namespace

cudaError_t launch_cache_rows(const CacheArgs& args, cudaStream_t stream)
{
    const int per = rows_per_block(args.row_bytes);
    long long blocks = (args.rows + per - 1) / per;
    if (blocks < 1) blocks = 1;                      // no rows: new_lengths alone
    if (blocks > 0x7fffffffLL || args.layers > 65535) return cudaErrorInvalidConfiguration;
    cache_rows_kernel<<<dim3((unsigned)blocks, (unsigned)args.layers), kThreads, 0, stream>>>(args);
    return cudaGetLastError();
}

}  // namespace kda
