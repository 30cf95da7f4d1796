// kda_prompt_attention_split.cu -- causal attention over packed prompts for whatever the
// tcgen05 kernel does not take (fp32 in or out, d = 16 and 32, scales that are not positive, more
// than 128 heads to a key head): products of fp16 pairs, summed up in fp32.
//
// fp32 keeps its accuracy as a sum of two fp16, x = hi + 2^-11 lo (22 bits), in three products
// hi hi + 2^-11 (lo hi + hi lo); bf16 is exact in one, and a bf16 output takes P in one.  fp16's
// range is met by powers of two, which are exact: one per query row, one per row of
// keys and one per row of values, from its largest finite magnitude.  With the factors
// a of the query, b of the key and c of the value
//     s = scale log2 e a b (Q K^T),  P = 2^(s - m),  w = P c 2^(m - n),  O += w V,
// m a reference near the running maximum of s of a row, n one 2^7 below that of s + log2 c: P stays
// below 2^8 and w below 2^15 whatever the values are, and w's largest is 2^7 at least, so that
// the weights of many keys far below one keep their bits (kda_f16_parts.cuh).  O is in units of 2^n, the
// sum l of P in units of 2^m.  They move only when a score exceeds them by more than 8.
//
// A thread block has 128 query rows of a (sequence, cache head), token by token (row r
// is head r % G of token r / G), 16 to a warp, and goes through 32 keys at a time: while
// the products of one tile run, the next is turned into fp16 pairs in shared memory and
// the one after that is copied by cp.async.  mma.sync m16n8k16 takes 2 clocks on an SM:
// with three products 190 TFLOP/s at most, where fp32 FMAs give 75.
//
// Values of keys that a row does not see must not reach it through 0 * inf: in the tiles
// on the diagonal infinities and NaN are replaced by 0 and their keys noted; the rows that do see
// such a key add its value at the end.
//
// The tensor cores cut off what does not fit as they add up, so the products with the small
// parts and each tile's output have sums of their own (1.2e-6 of the result otherwise,
// 2.0e-7 with them; the sums in fp32 FMAs, 3.1e-7).
//
// Thread blocks take the row tiles of all sequences and heads with most keys first.
//
// Bound by mma.sync and the conversions between the products: fp32, 4 prompts of 2,000
// tokens, 8 heads on 2, d = 128, 64, 16: 395, 196 and 105 us (CUDA cores 983, 552, 223); the first
// is 83 TFLOP/s where the three products would allow 190.  7 prompts of up to 1,500, 12 heads on
// 4, d = 64: 130 us (353).  bf16, d = 128, one prompt of 8,192 tokens, 32 heads on 8: 2.9 ms, 192
// TFLOP/s, with an fp32 output 3.5 ms (tcgen05 0.35, CUDA cores 12.4).
#include "kda_f16_parts.cuh"
#include "kda_prompt.cuh"

namespace kda {
namespace {

using namespace f16_parts;

constexpr int kWarps = 8, kThreads = kWarps * 32;
constexpr int BM = kWarps * 16, BN = 32;
constexpr int kNotes = 8;                          // tiles with rows that some query does not see, at most 6

template <class T, class O, int D>
struct Shape {
    static constexpr bool kLo = sizeof(T) == 4;    // q, k and v have a second part
    static constexpr bool kPLo = sizeof(O) == 4;   // and the probabilities
    static constexpr int kParts = kLo ? 2 : 1;
    static constexpr int kQ = kParts * BM * D * 2;
    static constexpr int kHalf = BN * D * 2;       // one part of a tile of keys or values
    static constexpr int kTile = 2 * kParts * kHalf;
    static constexpr int kRaw = 2 * BN * D * (int)sizeof(T);
    static constexpr size_t kBytes = kQ + 2 * kTile + 2 * kRaw;
};

__device__ __forceinline__ void ldmatrix(uint32_t (&r)[4], uint32_t at)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at));
}
__device__ __forceinline__ void ldmatrix_t(uint32_t (&r)[4], uint32_t at)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at));
}
// Byte offset of 16-byte piece c of row r of a tile of fp16 rows of D.
template <int D>
__device__ __forceinline__ int row_at(int r, int c)
{
    constexpr int S = D >= 64 ? 1 : D == 32 ? 2 : 4, M = D >= 64 ? 7 : D == 32 ? 3 : 1;
    return r * (D * 2) + ((c ^ ((r / S) & M)) << 4);
}

constexpr uint32_t kInfinity = 0x7F800000u;

// One 16-byte piece of a row, widened.
template <class T>
struct Piece {
    static constexpr int kN = 16 / (int)sizeof(T);
    float x[kN];
};
__device__ __forceinline__ Piece<float> widen(uint4 w, float)
{
    return {{__uint_as_float(w.x), __uint_as_float(w.y), __uint_as_float(w.z), __uint_as_float(w.w)}};
}
__device__ __forceinline__ Piece<__nv_bfloat16> widen(uint4 w, __nv_bfloat16)
{
    Piece<__nv_bfloat16> p;
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        p.x[2 * i] = __uint_as_float(u[i] << 16);
        p.x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    }
    return p;
}

// The 16-byte piece c of T of row r, times up, as fp16 into the first part of a tile and
// (LO) what that leaves into the second, `part` bytes on; odd: there may be infinities
// or NaN.
template <class T, int D, bool LO>
__device__ __forceinline__ void store_parts(uint32_t tile, int part, int r, int c, const Piece<T>& p, float up, bool odd)
{
    constexpr int N = Piece<T>::kN;
    uint32_t h[N / 2], l[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
        const float x = p.x[2 * i] * up, y = p.x[2 * i + 1] * up;
        h[i] = two_f16(x, y);
        if (LO) {
            l[i] = two_f16_rest(x, y, h[i]);
            if (odd) {                             // (an infinity or NaN has no second part)
                if (!(fabsf(x) < INFINITY)) l[i] &= 0xFFFF0000u;
                if (!(fabsf(y) < INFINITY)) l[i] &= 0x0000FFFFu;
            }
        }
    }
    if constexpr (N == 4) {
        const uint32_t at = tile + row_at<D>(r, c >> 1) + (c & 1) * 8;
        asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(at), "r"(h[0]), "r"(h[1]) : "memory");
        if (LO) asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(at + part), "r"(l[0]), "r"(l[1]) : "memory");
    } else {
        const uint32_t at = tile + row_at<D>(r, c);
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(h[0]), "r"(h[1]), "r"(h[2]), "r"(h[3]) : "memory");
    }
}

struct Shared {
    float q_down[BM];                              // a query row's factor, with scale log2 e
    float k_down[2][BN], v_down[2][BN], v_log[2][BN];      // a key's and a value's, of two tiles
    uint32_t bad[kNotes];                          // keys with an infinity or NaN in v, of the tiles from the first masked one on
    long long sum[kWarps];
    int tiles[kThreads];                           // of the sequences
    int seq, tile;
};

// The block's sequence and row tile; all threads call it.  False: there is none.  Up to
// kThreads sequences are taken in levels, the largest tile number of all first (the
// longest work of whole prompts), so that the blocks that start last are short; more
// sequences are taken one after the other.
__device__ bool locate(Shared& sh, const PromptArgs& a, long long b)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) sh.seq = -1;
    if (a.N <= kThreads) {
        int mine = 0;
        if (tid < a.N) {
            int first, count;
            prompt_rows(a.cu_q, tid, a.T, first, count);
            mine = (int)(((long long)count * a.G + BM - 1) / BM);
        }
        sh.tiles[tid] = mine;
        int top = __reduce_max_sync(0xffffffffu, mine);
        if (lane == 0) sh.sum[warp] = top;
        __syncthreads();
        for (int i = 0; i < kWarps; ++i) top = max(top, (int)sh.sum[i]);
        // the largest level v with more than b tiles of level v and above
        auto above = [&](int v) {
            int x = 0;
            for (int n = lane; n < a.N; n += 32) x += max(sh.tiles[n] - v, 0);
            return (int)__reduce_add_sync(0xffffffffu, x);
        };
        int lo = 0, hi = top;              // above(lo) > b >= above(hi)
        if (b >= above(0)) return false;
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if (above(mid) > b) lo = mid;
            else hi = mid;
        }
        int left = (int)b - above(lo + 1); // which of the sequences that have that level
        for (int n0 = 0; n0 < a.N; n0 += 32) {
            const uint32_t has = __ballot_sync(0xffffffffu, n0 + lane < a.N && sh.tiles[n0 + lane] > lo);
            if (left < __popc(has)) {
                if (warp == 0 && (has >> lane & 1) && __popc(has & ((1u << lane) - 1)) == left) {
                    sh.seq = n0 + lane;
                    sh.tile = lo;
                }
                break;
            }
            left -= __popc(has);
        }
        __syncthreads();
        return sh.seq >= 0;                // (offsets that give rows twice may add up to anything)
    }
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
        if (lane == 31) sh.sum[warp] = incl;
        __syncthreads();
        long long before = base, all = 0;
        for (int i = 0; i < kWarps; ++i) {
            if (i < warp) before += sh.sum[i];
            all += sh.sum[i];
        }
        if (b >= before + incl - w && b < before + incl) {
            sh.seq = n;
            sh.tile = (int)(w - 1 - (b - (before + incl - w)));    // a prompt's last rows, the longest work, first
        }
        base += all;
        __syncthreads();
        if (b < base) break;
    }
    __syncthreads();
    return sh.seq >= 0;
}

__device__ __forceinline__ void store2(float* p, float x, float y) { *reinterpret_cast<float2*>(p) = make_float2(x, y); }
__device__ __forceinline__ void store2(__nv_bfloat16* p, float x, float y) { *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(x, y); }

template <class T, class O, int D>
__global__ void __launch_bounds__(kThreads, D <= 64 ? 2 : 1)
prompt_attention_split_kernel(const __grid_constant__ PromptArgs a)
{
    using Sh = Shape<T, O, D>;
    constexpr int P = D * (int)sizeof(T) / 16;     // pieces of a row
    constexpr int PT = (P + 7) / 8;                // of a thread, eight to a row
    constexpr int NT = D / 8;
    extern __shared__ __align__(128) uint8_t dyn[];
    __shared__ Shared sh;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int hk = blockIdx.x % a.Hkv;
    if (tid < kNotes) sh.bad[tid] = 0;
    if (!locate(sh, a, blockIdx.x / a.Hkv)) return;
    const PromptSeq s = prompt_seq(a, sh.seq);
    const int off = s.lk - s.lq;                   // token t sees the keys up to t + off
    const long long rows = (long long)s.lq * a.G, r0 = (long long)sh.tile * BM;
    const int here = rows - r0 < BM ? (int)(rows - r0) : BM;
    const int most = min(max((int)((r0 + here - 1) / a.G) + off + 1, 0), s.lk);
    const int all = min(max((int)(r0 / a.G) + off + 1, 0), s.lk);      // keys that every row sees
    const uint32_t q_tile = smem_at(dyn), tiles = q_tile + Sh::kQ, raw = tiles + 2 * Sh::kTile;
    const T* kp = static_cast<const T*>(a.k) + (long long)s.k0 * a.k_stride + (long long)hk * D;
    const T* vp = static_cast<const T*>(a.v) + (long long)s.k0 * a.v_stride + (long long)hk * D;
    const int t8 = tid & 7, tr = tid >> 3;         // this thread's pieces and row of a tile of keys
    const int count = (most + BN - 1) / BN;

    auto copy_raw = [&](int j) {
        if (j < count) {
            const int key = j * BN + tr;
            const bool there = key < most;
            const uint32_t dst = raw + (j & 1) * Sh::kRaw + tr * (P * 16);
#pragma unroll
            for (int i = 0; i < PT; ++i) {
                const int c = t8 + 8 * i;
                if (c < P) {
                    const long long k = there ? key : 0;
                    copy16(dst + c * 16, reinterpret_cast<const uint4*>(kp + k * a.k_stride) + c, there);
                    copy16(dst + BN * P * 16 + c * 16, reinterpret_cast<const uint4*>(vp + k * a.v_stride) + c, there);
                }
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    // Tile j from the copies (each thread its own) to fp16 pairs.
    auto convert = [&](int j) {
        const uint32_t src = raw + (j & 1) * Sh::kRaw + tr * (P * 16), dst = tiles + (j & 1) * Sh::kTile;
        const bool edge = (j + 1) * BN > all;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            Piece<T> p[PT];
            uint32_t top = 0;
#pragma unroll
            for (int i = 0; i < PT; ++i) {
                const int c = t8 + 8 * i;
                uint4 w = make_uint4(0, 0, 0, 0);
                if (c < P)
                    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
                                 : "r"(src + x * (BN * P * 16) + c * 16));
                p[i] = widen(w, T());
#pragma unroll
                for (int e = 0; e < Piece<T>::kN; ++e) top = top_of(top, p[i].x[e]);
            }
#pragma unroll
            for (int d = 1; d < 8; d <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
            const bool odd = top >= kInfinity;     // (the same for the row's threads)
            if (__any_sync(0xffffffffu, odd)) {
                bool mine = false;
                if (odd) top = 0;
#pragma unroll
                for (int i = 0; i < PT; ++i)
#pragma unroll
                    for (int e = 0; e < Piece<T>::kN; ++e) {
                        const bool fine = fabsf(p[i].x[e]) < INFINITY;
                        if (odd && fine) top = top_of(top, p[i].x[e]);
                        mine |= !fine;
                        if (!fine && x == 1 && edge) p[i].x[e] = 0.f;
                    }
#pragma unroll
                for (int d = 1; d < 8; d <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
                if (mine && x == 1 && edge) atomicOr(&sh.bad[j - all / BN], 1u << tr);
            }
            const int e = up_of(top);
#pragma unroll
            for (int i = 0; i < PT; ++i)
                if (t8 + 8 * i < P) store_parts<T, D, Sh::kLo>(dst + x * (Sh::kParts * Sh::kHalf), Sh::kHalf, tr, t8 + 8 * i, p[i], power(e), odd);
            if (t8 == 0) {
                if (x == 0) {
                    sh.k_down[j & 1][tr] = power(-e);
                } else {
                    // (a row of zeros has no weight and does not move the reference of the others')
                    const bool none = top == 0 && !odd;
                    sh.v_down[j & 1][tr] = none ? 0.f : power(-e);
                    sh.v_log[j & 1][tr] = none ? -INFINITY : (float)-e;
                }
            }
        }
    };

    copy_raw(0);
    copy_raw(1);
    // the queries, 32 rows at a time; -1 for a negative scale, 0 for 0
    const ScaleParts scale = scale_parts(a.scale_log2);
#pragma unroll 1
    for (int b = 0; b < BM; b += 32) {
        const int r = b + tr;
        const T* qp = nullptr;
        if (r < here) {
            const int t = (int)((r0 + r) / a.G), g = (int)((r0 + r) - (long long)t * a.G);
            qp = static_cast<const T*>(a.q) + (long long)(s.q0 + t) * a.q_stride + ((long long)hk * a.G + g) * D;
        }
        Piece<T> p[PT];
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < PT; ++i) {
            uint4 w = make_uint4(0, 0, 0, 0);
            if (qp && t8 + 8 * i < P) w = __ldg(reinterpret_cast<const uint4*>(qp) + t8 + 8 * i);
            p[i] = widen(w, T());
#pragma unroll
            for (int e = 0; e < Piece<T>::kN; ++e) {
                p[i].x[e] *= scale.pre;
                if (fabsf(p[i].x[e]) < INFINITY) top = top_of(top, p[i].x[e]);
            }
        }
#pragma unroll
        for (int d = 1; d < 8; d <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
        const int e = up_of(top);
        const float sign = a.scale_log2 > 0.f ? 1.f : a.scale_log2 < 0.f ? -1.f : a.scale_log2;     // (0 or NaN stays)
#pragma unroll
        for (int i = 0; i < PT; ++i)
            if (t8 + 8 * i < P) store_parts<T, D, Sh::kLo>(q_tile, BM * D * 2, r, t8 + 8 * i, p[i], power(e) * sign, true);
        if (t8 == 0) sh.q_down[r] = sign == 0.f ? 1.f : scale.rest * power(-e);
    }
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    if (count > 0) convert(0);
    copy_raw(2);

    const int g = lane >> 2, i4 = lane & 3;
    float o[NT][4], m[2], n[2], l[2], fac[2], rs[2];
    int lim[2];
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int c = 0; c < 4; ++c) o[j][c] = 0.f;
    __syncthreads();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int r = warp * 16 + g + 8 * h;
        lim[h] = r < here ? min(max((int)((r0 + r) / a.G) + off + 1, 0), s.lk) : 0;
        rs[h] = sh.q_down[r];
        m[h] = n[h] = -INFINITY;
        l[h] = fac[h] = 0.f;
    }
    // the rows and pieces that this lane's ldmatrix addresses name
    const int mr = lane & 15, mc = lane >> 4;      // q, v: 16 rows, two pieces
    const int kr = (lane & 7) + ((lane >> 4) << 3), kc = (lane >> 3) & 1;  // k: two blocks of 8 rows, two pieces each
#pragma unroll 1
    for (int j = 0; j < count; ++j) {
        // the next tile, while other warps are at this one's products
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        if (j + 1 < count) convert(j + 1);
        copy_raw(j + 3);
        const uint32_t kt = tiles + (j & 1) * Sh::kTile, vt = kt + Sh::kParts * Sh::kHalf;
        // The tensor cores cut off what does not fit as they add up: the small products have
        // sums of their own, and so has each tile's output below.
        float c[4][4], small[4][4];
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
            uint32_t qh[4], ql[4], kh[2][4], kl[2][4];
            ldmatrix(qh, q_tile + row_at<D>(warp * 16 + mr, 2 * k + mc));
            if (Sh::kLo) ldmatrix(ql, q_tile + BM * D * 2 + row_at<D>(warp * 16 + mr, 2 * k + mc));
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                ldmatrix(kh[b], kt + row_at<D>(b * 16 + kr, 2 * k + kc));
                if (Sh::kLo) ldmatrix(kl[b], kt + Sh::kHalf + row_at<D>(b * 16 + kr, 2 * k + kc));
            }
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                if (k == 0) mma0(c[b], qh, kh[b >> 1][2 * (b & 1)], kh[b >> 1][2 * (b & 1) + 1]);
                else mma(c[b], qh, kh[b >> 1][2 * (b & 1)], kh[b >> 1][2 * (b & 1) + 1]);
            }
            if (Sh::kLo) {
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    if (k == 0) mma0(small[b], ql, kh[b >> 1][2 * (b & 1)], kh[b >> 1][2 * (b & 1) + 1]);
                    else mma(small[b], ql, kh[b >> 1][2 * (b & 1)], kh[b >> 1][2 * (b & 1) + 1]);
                }
#pragma unroll
                for (int b = 0; b < 4; ++b) mma(small[b], qh, kl[b >> 1][2 * (b & 1)], kl[b >> 1][2 * (b & 1) + 1]);
            }
        }
        const bool masked = (j + 1) * BN > all;
        float top[2], vtop[2], vd[4][2];
        bool grow = false;
        top[0] = top[1] = vtop[0] = vtop[1] = -INFINITY;
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const float2 kd = *reinterpret_cast<const float2*>(&sh.k_down[j & 1][8 * b + 2 * i4]);
            const float2 v2 = *reinterpret_cast<const float2*>(&sh.v_down[j & 1][8 * b + 2 * i4]);
            const float2 lv = *reinterpret_cast<const float2*>(&sh.v_log[j & 1][8 * b + 2 * i4]);
            vd[b][0] = v2.x, vd[b][1] = v2.y;
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float& x = c[b][2 * h + e];
                    // (by both factors at once: with one of them alone it may not fit)
                    x = (Sh::kLo ? fmaf(small[b][2 * h + e], kRest, x) : x) * ((e ? kd.y : kd.x) * rs[h]);
                    if (masked && j * BN + 8 * b + 2 * i4 + e >= lim[h]) x = -INFINITY;
                    top[h] = fmaxf(top[h], x);
                    vtop[h] = fmaxf(vtop[h], x + (e ? lv.y : lv.x));
                }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) grow |= top[h] > m[h] + kSlack || vtop[h] > n[h] + (kSlack + kHead);
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
                for (int x = 0; x < NT; ++x) {
                    o[x][2 * h] *= fo;
                    o[x][2 * h + 1] *= fo;
                }
            }
        }
        uint32_t ph[2][4], pl[2][4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float ref = m[h] == -INFINITY ? 0.f : m[h];
            float sum = 0.f;                       // (few additions to l, which small probabilities would be lost in)
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                float y[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float p = ex2(c[b][2 * h + e] - ref);
                    sum += p;
                    y[e] = p * weight_factor(vd[b][e], fac[h]);
                }
                const uint32_t z = two_f16(y[0], y[1]);
                ph[b >> 1][2 * (b & 1) + h] = z;
                if (Sh::kPLo) pl[b >> 1][2 * (b & 1) + h] = two_f16_rest(y[0], y[1], z);
            }
            l[h] += sum;
        }
#pragma unroll
        for (int x = 0; x < NT; x += 2) {
            uint32_t vh[2][4], vl[2][4];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                ldmatrix_t(vh[k], vt + row_at<D>(k * 16 + mr, x + mc));
                if (Sh::kLo) ldmatrix_t(vl[k], vt + Sh::kHalf + row_at<D>(k * 16 + mr, x + mc));
            }
            // the small products first, times 2^-11 (which is exact), and the large ones onto them; two sums instead of one
            // take 410 us for 4 prompts of 2,000 tokens, d = 128, this 395
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                if constexpr (Sh::kPLo) {
                    float z[4];
                    mma0(z, pl[0], vh[0][2 * y], vh[0][2 * y + 1]);
                    mma(z, pl[1], vh[1][2 * y], vh[1][2 * y + 1]);
                    if (Sh::kLo) {
                        mma(z, ph[0], vl[0][2 * y], vl[0][2 * y + 1]);
                        mma(z, ph[1], vl[1][2 * y], vl[1][2 * y + 1]);
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) z[e] *= kRest;
                    mma(z, ph[0], vh[0][2 * y], vh[0][2 * y + 1]);
                    mma(z, ph[1], vh[1][2 * y], vh[1][2 * y + 1]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[x + y][e] += z[e];
                } else {
                    mma(o[x + y], ph[0], vh[0][2 * y], vh[0][2 * y + 1]);
                    mma(o[x + y], ph[1], vh[1][2 * y], vh[1][2 * y + 1]);
                }
            }
        }
        __syncthreads();                           // the next tile is there, this one has been read
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    uint32_t any = 0;
#pragma unroll
    for (int i = 0; i < kNotes; ++i) any |= sh.bad[i];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
        l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
        const int r = warp * 16 + g + 8 * h;
        if (r >= here) continue;
        const int t = (int)((r0 + r) / a.G), q = (int)((r0 + r) - (long long)t * a.G);
        const float f = lim[h] == 0 ? 0.f : ex2(n[h] - m[h]) / l[h];
        O* op = static_cast<O*>(a.o) + ((long long)(s.q0 + t) * a.Hq + (long long)hk * a.G + q) * D;
#pragma unroll
        for (int x = 0; x < NT; ++x) {
            float y[2] = {lim[h] == 0 ? 0.f : o[x][2 * h] * f, lim[h] == 0 ? 0.f : o[x][2 * h + 1] * f};
            if (any) {
#pragma unroll 1
                for (int k = all / BN * BN; k < lim[h]; ++k) {
                    if (!((sh.bad[(k - all / BN * BN) / BN] >> (k & 31)) & 1)) continue;
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float z = (float)vp[(long long)k * a.v_stride + 8 * x + 2 * i4 + e];
                        if (!(fabsf(z) < INFINITY)) y[e] += z;
                    }
                }
            }
            store2(op + 8 * x + 2 * i4, y[0], y[1]);
        }
    }
}

template <class T, class O, int D>
cudaError_t launch(const PromptArgs& a, cudaStream_t stream)
{
    auto kern = prompt_attention_split_kernel<T, O, D>;
    const size_t bytes = Shape<T, O, D>::kBytes;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e != cudaSuccess) return e;
    // every sequence has at most one tile that is not full
    const long long tiles = ((long long)a.T * a.G) / BM + a.N;
    if (tiles * a.Hkv > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    kern<<<(unsigned)(tiles * a.Hkv), kThreads, bytes, stream>>>(a);
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

cudaError_t launch_prompt_attention_split(const PromptArgs& a, int32_t d, kda_dtype_t dtype, cudaStream_t stream)
{
    if (dtype == KDA_BF16) return launch_d<__nv_bfloat16, __nv_bfloat16>(a, d, stream);
    if (dtype == KDA_BF16_F32OUT) return launch_d<__nv_bfloat16, float>(a, d, stream);
    return launch_d<float, float>(a, d, stream);
}

}  // namespace kda
