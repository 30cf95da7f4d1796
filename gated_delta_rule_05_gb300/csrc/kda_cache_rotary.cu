// kda_cache_rotary.cu -- queries and keys rotated to their positions, keys and
// values into the pages of a cache (kda_cache_append_rotary).
//
// A pair (x, y) of a row at position p is turned by p f, f the pair's frequency:
// (x cos - y sin, x sin + y cos).  The angle is taken in turns, in fixed point:
// p * round(2^64 frac(f / 2 pi)) mod 2^64 is the fraction of a turn exactly, whatever
// p is, where fp32 would lose what matters (at position 10^6 an angle is off by
// 0.03).  Its upper 32 bits go to sincospif.
//
// A unit is the part of one block of rows (of one scale, or 16 rows of a cache in
// the model's type) that one sequence adds to; the thread block that owns the unit's
// first row tabulates the sines and cosines of the unit's rows once and its warps
// share out the heads.  A lane holds 16 channels of a row, two vectors of eight
// that belong together: the halves of eight pairs, or eight neighbouring pairs.
//
// 8 bits: a warp has a unit of one head of k or v and reads it twice, first for the
// largest magnitude (as bits, so that infinities and NaN win), then to store x / s
// (from L1 or L2 then).  s is a power of two: e4m3 is a floating type, so a finer scale
// would gain nothing, and the division, a later change of the scale and the product in
// the attention are exact but for e4m3's own rounding.  A scale of NaN marks a block
// with an infinity or NaN; its bytes are 0, so that no product of a weight of 0
// with it is NaN.
//
// Bound by the bytes moved.
#include "kda_prompt.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kHeldSeqs = 1024;        // sequences whose offsets are held in shared memory

// In place the rows are written by the lane that read them, so that no load may go
// through the read-only path.
struct Raw16 { uint4 v[1]; };
struct Raw32 { uint4 v[2]; };
template <class T> struct RawOf;
template <> struct RawOf<__nv_bfloat16> { using type = Raw16; };
template <> struct RawOf<float> { using type = Raw32; };

template <class T>
__device__ __forceinline__ typename RawOf<T>::type load_raw(const uint8_t* p)
{
    typename RawOf<T>::type r;
#pragma unroll
    for (int i = 0; i < (int)(sizeof(T) / 2); ++i) r.v[i] = *(reinterpret_cast<const uint4*>(p) + i);
    return r;
}
__device__ __forceinline__ void widen(const Raw16& r, float (&x)[8])
{
    const uint32_t w[4] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ void widen(const Raw32& r, float (&x)[8])
{
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        x[4 * i] = __uint_as_float(r.v[i].x);
        x[4 * i + 1] = __uint_as_float(r.v[i].y);
        x[4 * i + 2] = __uint_as_float(r.v[i].z);
        x[4 * i + 3] = __uint_as_float(r.v[i].w);
    }
}
__device__ __forceinline__ uint32_t two_bf16(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&x)[8])
{
    *reinterpret_cast<uint4*>(p) = make_uint4(two_bf16(x[0], x[1]), two_bf16(x[2], x[3]), two_bf16(x[4], x[5]), two_bf16(x[6], x[7]));
}
__device__ __forceinline__ void store8(float* p, const float (&x)[8])
{
    *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
    *(reinterpret_cast<float4*>(p) + 1) = make_float4(x[4], x[5], x[6], x[7]);
}

__device__ __forceinline__ uint32_t four_e4m3(float a, float b, float c, float d)
{
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return (uint32_t)lo | ((uint32_t)hi << 16);
}
__device__ __forceinline__ float2 from_e4m3(uint32_t two)
{
    uint32_t h;
    const uint16_t w = (uint16_t)two;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(w));
    return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// The bits of the smallest power of two s, at least 2^-126, with top <= 448 s; 0 for
// 0, NaN for an infinity or NaN.  448 = 1.75 * 2^8.
__device__ __forceinline__ uint32_t scale_bits(uint32_t top)
{
    if (top >= 0x7F800000u) return 0x7FC00000u;
    if (top == 0) return 0;
    const int e = (int)(top >> 23) - 8 + ((top & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return (uint32_t)(e < 1 ? 1 : e) << 23;
}

struct Unit {
    int n, first, count;               // sequence, packed rows
    long long pos;                     // of the first
};

// Sequence that owns row r and r's place in it; false: none.
__device__ __forceinline__ bool row_owner(const RotaryArgs& a, const int32_t* cu, int r, int& n, int& start, int& end)
{
    int lo = 0, hi = a.N;              // the last n with cu[n] <= r
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (cu[mid] <= r) lo = mid;
        else hi = mid;
    }
    n = lo;
    start = max(cu[n], 0);
    end = min(cu[n + 1], a.T);
    return r >= start && r < end;
}

// The two vectors of eight channels that a lane holds of a row of D: their
// channels, whether they are turned, and its place in the table.
struct Pair {
    int a, b, c;
    bool turned;
};
__device__ __forceinline__ Pair pair_of(int c, int rot, bool interleaved)
{
    Pair p;
    p.c = c;
    p.turned = 16 * c < rot;
    p.a = 16 * c;
    p.b = 16 * c + 8;
    if (p.turned && !interleaved) {
        p.a = 8 * c;
        p.b = rot / 2 + 8 * c;
    }
    return p;
}

// The table: of each row the (cos, sin) of its rot / 2 pairs, as 16-byte pieces of
// two in an order that neighbouring lanes read without bank conflicts.
__device__ __forceinline__ int table_at(int row, int j, int rot)
{
    return row * (rot / 2) + ((j & 7) >> 1) * (rot / 8) + (j >> 3) * 2 + (j & 1);
}

__device__ __forceinline__ void turn(const float2* table, int row, const Pair& p, int rot, bool interleaved,
                                     float (&x)[8], float (&y)[8])
{
    const float4* t = reinterpret_cast<const float4*>(table + row * (rot / 2)) + p.c;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float4 w = t[i * (rot / 16)];        // (cos, sin) of pairs 2 i and 2 i + 1
        if (interleaved) {
            float* z = i < 2 ? x + 4 * i : y + 4 * (i - 2);
            const float z0 = z[0], z2 = z[2];
            z[0] = z0 * w.x - z[1] * w.y;
            z[1] = z0 * w.y + z[1] * w.x;
            z[2] = z2 * w.z - z[3] * w.w;
            z[3] = z2 * w.w + z[3] * w.z;
        } else {
            const float x0 = x[2 * i], x1 = x[2 * i + 1];
            x[2 * i] = x0 * w.x - y[2 * i] * w.y;
            y[2 * i] = x0 * w.y + y[2 * i] * w.x;
            x[2 * i + 1] = x1 * w.z - y[2 * i + 1] * w.w;
            y[2 * i + 1] = x1 * w.w + y[2 * i + 1] * w.z;
        }
    }
}

__device__ __forceinline__ uint32_t top_bits(uint32_t top, const float (&x)[8])
{
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(x[i]) & 0x7FFFFFFFu);
    return top;
}

template <class T, int D>
struct Rows {
    static constexpr int kLanes = D / 16;          // lanes per row
    static constexpr int kPass = 32 / kLanes;      // rows per pass of a warp
    static constexpr int kDepth = sizeof(T) == 2 ? 4 : 2;
};

// One head of a unit's rows: src to dst (null: dropped) and to the rows of a cache
// in the same type (place[row] < 0: dropped).
template <class T, int D, bool TURN>
__device__ void plain_head(const RotaryArgs& a, const Unit& u, const float2* table, const uint8_t* src,
                           long long src_row, uint8_t* dst, long long dst_row, uint8_t* cache,
                           const long long* place, int lane)
{
    using R = Rows<T, D>;
    const Pair p = pair_of(lane % R::kLanes, TURN ? a.rot : 0, a.interleaved);
    const int r0 = lane / R::kLanes;
    const int ea = p.a * (int)sizeof(T), eb = p.b * (int)sizeof(T);
#pragma unroll 1
    for (int base = r0; base < u.count; base += R::kPass * R::kDepth) {
        typename RawOf<T>::type ra[R::kDepth], rb[R::kDepth];
#pragma unroll
        for (int i = 0; i < R::kDepth; ++i) {
            const int r = base + i * R::kPass;
            if (r < u.count) {
                const uint8_t* s = src + (u.first + r) * src_row;
                ra[i] = load_raw<T>(s + ea);
                rb[i] = load_raw<T>(s + eb);
            }
        }
#pragma unroll
        for (int i = 0; i < R::kDepth; ++i) {
            const int r = base + i * R::kPass;
            if (r >= u.count) break;
            float x[8], y[8];
            widen(ra[i], x);
            widen(rb[i], y);
            if (TURN && p.turned) turn(table, r, p, a.rot, a.interleaved, x, y);
            if (dst) {
                uint8_t* d = dst + (u.first + r) * dst_row;
                store8(reinterpret_cast<T*>(d + ea), x);
                store8(reinterpret_cast<T*>(d + eb), y);
            }
            if (cache && place[r] >= 0) {
                store8(reinterpret_cast<T*>(cache + place[r] + ea), x);
                store8(reinterpret_cast<T*>(cache + place[r] + eb), y);
            }
        }
    }
}

// One head of a unit's rows as e4m3 into its block of the cache: `block0` the
// block's first row there (null: the rows have no place), `off` the rows that it
// already has, `scale` its scale.
template <class T, int D, bool TURN>
__device__ void e4m3_head(const RotaryArgs& a, const Unit& u, const float2* table, const uint8_t* src,
                          long long src_row, uint8_t* dst, long long dst_row, uint8_t* block0, int off,
                          float* scale, int lane)
{
    using R = Rows<T, D>;
    const Pair p = pair_of(lane % R::kLanes, TURN ? a.rot : 0, a.interleaved);
    const int r0 = lane / R::kLanes;
    const int ea = p.a * (int)sizeof(T), eb = p.b * (int)sizeof(T);
    const int row_bytes = a.Hkv * D;
    uint32_t top = 0;
    if (block0) {
#pragma unroll 1
        for (int base = r0; base < u.count; base += R::kPass * R::kDepth) {
            typename RawOf<T>::type ra[R::kDepth], rb[R::kDepth];
#pragma unroll
            for (int i = 0; i < R::kDepth; ++i) {
                const int r = base + i * R::kPass;
                if (r < u.count) {
                    const uint8_t* s = src + (u.first + r) * src_row;
                    ra[i] = load_raw<T>(s + ea);
                    rb[i] = load_raw<T>(s + eb);
                }
            }
#pragma unroll
            for (int i = 0; i < R::kDepth; ++i) {
                const int r = base + i * R::kPass;
                if (r >= u.count) break;
                float x[8], y[8];
                widen(ra[i], x);
                widen(rb[i], y);
                if (TURN && p.turned) turn(table, r, p, a.rot, a.interleaved, x, y);
                top = top_bits(top_bits(top, x), y);
            }
        }
    }
    top = __reduce_max_sync(0xffffffffu, top);
    uint32_t sb = scale_bits(top);
    if (block0 && off > 0) {
        const uint32_t old = __float_as_uint(*scale) & 0x7FFFFFFFu;
        if (sb > old && old > 0 && sb < 0x7F800000u) {
            // the rows that are there, in the new scale
            const float ratio = __uint_as_float(old) * __uint_as_float(0x7F000000u - sb);
            for (int e = lane; e < off * (D / 8); e += 32) {
                uint2* w = reinterpret_cast<uint2*>(block0 + (long long)(e / (D / 8)) * row_bytes + e % (D / 8) * 8);
                const uint2 b = *w;
                const float2 b0 = from_e4m3(b.x), b1 = from_e4m3(b.x >> 16), b2 = from_e4m3(b.y), b3 = from_e4m3(b.y >> 16);
                *w = make_uint2(four_e4m3(b0.x * ratio, b0.y * ratio, b1.x * ratio, b1.y * ratio),
                                four_e4m3(b2.x * ratio, b2.y * ratio, b3.x * ratio, b3.y * ratio));
            }
        }
        sb = max(sb, old);
    }
    __syncwarp();                                  // every lane has read the old scale
    if (block0 && lane == 0) *scale = __uint_as_float(sb);
    const bool store = sb > 0 && sb < 0x7F800000u;
    const float inv = store ? __uint_as_float(0x7F000000u - sb) : 0.f;
    if (!block0 && !dst) return;
#pragma unroll 1
    for (int base = r0; base < u.count; base += R::kPass * R::kDepth) {
        typename RawOf<T>::type ra[R::kDepth], rb[R::kDepth];
#pragma unroll
        for (int i = 0; i < R::kDepth; ++i) {
            const int r = base + i * R::kPass;
            if (r < u.count) {
                const uint8_t* s = src + (u.first + r) * src_row;
                ra[i] = load_raw<T>(s + ea);
                rb[i] = load_raw<T>(s + eb);
            }
        }
#pragma unroll
        for (int i = 0; i < R::kDepth; ++i) {
            const int r = base + i * R::kPass;
            if (r >= u.count) break;
            float x[8], y[8];
            widen(ra[i], x);
            widen(rb[i], y);
            if (TURN && p.turned) turn(table, r, p, a.rot, a.interleaved, x, y);
            if (dst) {
                uint8_t* d = dst + (u.first + r) * dst_row;
                store8(reinterpret_cast<T*>(d + ea), x);
                store8(reinterpret_cast<T*>(d + eb), y);
            }
            if (block0) {
                uint8_t* c = block0 + (long long)(off + r) * row_bytes;
                uint2 wx = make_uint2(0, 0), wy = make_uint2(0, 0);
                if (store) {
                    wx = make_uint2(four_e4m3(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv),
                                    four_e4m3(x[4] * inv, x[5] * inv, x[6] * inv, x[7] * inv));
                    wy = make_uint2(four_e4m3(y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv),
                                    four_e4m3(y[4] * inv, y[5] * inv, y[6] * inv, y[7] * inv));
                }
                *reinterpret_cast<uint2*>(c + p.a) = wx;
                *reinterpret_cast<uint2*>(c + p.b) = wy;
            }
        }
    }
}

template <class T, int D, bool EIGHT>
__global__ void __launch_bounds__(kThreads, 2)
cache_rotary_kernel(const __grid_constant__ RotaryArgs a)
{
    extern __shared__ __align__(16) uint8_t dyn[];
    float2* table = reinterpret_cast<float2*>(dyn);
    __shared__ int32_t sh_cu[kHeldSeqs + 1];
    __shared__ unsigned long long sh_turns[64];    // turns per position of each pair, times 2^64
    __shared__ Unit sh_unit[kMaxScaleBlock];       // of each row of the window; count 0: no unit begins there
    __shared__ long long sh_place[kMaxScaleBlock]; // of each row of the unit, byte offset in the cache
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int32_t* cu = a.cu_seqlens;
    if (a.N <= kHeldSeqs) {
        for (int i = tid; i <= a.N; i += kThreads) sh_cu[i] = __ldg(a.cu_seqlens + i);
        cu = sh_cu;
    }
    if (tid < a.rot / 2) {
        // in fp64: 53 bits of a fraction that a position (31 bits) multiplies
        double f = (double)__ldg(a.inv_freq + tid) * 0.15915494309189533577;
        f -= floor(f);
        sh_turns[tid] = __double2ull_rn(f * 18446744073709551616.0);
    }
    __syncthreads();
    if (tid < a.window) {
        Unit u = {0, 0, 0, 0};
        const int r = blockIdx.x * a.window + tid;
        int n, start, end;
        if (r < a.T && row_owner(a, cu, r, n, start, end)) {
            const int len = __ldg(a.lengths + n);
            if (len >= 0) {
                u.n = n;
                u.first = r;
                u.pos = (long long)len + (r - start);
                const int left = a.step - (int)(u.pos % a.step);
                if (r == start || left == a.step) u.count = min(left, end - r);
            }
        }
        sh_unit[tid] = u;
    }
    if (a.new_lengths && blockIdx.y == 0) {
        for (int n = blockIdx.x * kThreads + tid; n < a.N; n += gridDim.x * kThreads)
            a.new_lengths[n] = __ldg(a.lengths + n) + max(min(cu[n + 1], a.T) - max(cu[n], 0), 0);
    }
    __syncthreads();
    const int tasks = (a.q ? a.Hq : 0) + 2 * a.Hkv;
    const int half = a.rot / 2;
#pragma unroll 1
    for (int w = 0; w < a.window; ++w) {
        const Unit u = sh_unit[w];
        if (u.count == 0) continue;                // (the same for all threads)
        for (int e = tid; e < u.count * half; e += kThreads) {
            const int r = e / half, j = e - r * half;
            const unsigned long long t = (unsigned long long)(u.pos + r) * sh_turns[j];
            float s, c;
            sincospif((float)(int32_t)(t >> 32) * 4.656612873077393e-10f, &s, &c);    // 2^-31: in half turns
            table[table_at(r, j, a.rot)] = make_float2(c, s);
        }
        if (tid < u.count) {
            const long long pos = u.pos + tid;
            long long place = -1;
            if (pos < (long long)a.max_pages * a.page_size) {
                const int at = (int)(pos / a.page_size);
                const int page = __ldg(a.page_table + (long long)u.n * a.max_pages + at);
                if (page >= 0 && page < a.num_pages) {
                    const int slot = (int)(pos - (long long)at * a.page_size);
                    // of a block of 8 bits: the page and the row in it
                    place = EIGHT ? (long long)page << 32 | slot
                                  : page * a.page_bytes + (long long)slot * a.Hkv * D * (int)sizeof(T);
                }
            }
            sh_place[tid] = place;
        }
        __syncthreads();
#pragma unroll 1
        for (int task = blockIdx.y * kWarps + warp; task < tasks; task += gridDim.y * kWarps) {
            const int h = task - 2 * a.Hkv;        // keys and values first, they take longer
            if (h >= 0) {
                const long long at = (long long)h * D * (int)sizeof(T);
                plain_head<T, D, true>(a, u, table, a.q + at, a.q_row, a.q_out + at, a.q_out_row, nullptr, sh_place, lane);
                continue;
            }
            const bool is_k = task < a.Hkv;
            const int hk = is_k ? task : task - a.Hkv;
            const long long at = (long long)hk * D * (int)sizeof(T);
            uint8_t* k_out = a.k_out ? a.k_out + at : nullptr;
            if constexpr (EIGHT) {
                const long long place = sh_place[0];
                uint8_t* block0 = nullptr;
                float* scale = nullptr;
                int off = 0;
                if (place >= 0) {
                    const int page = (int)(place >> 32), slot = (int)(place & 0xFFFFFFFF), b = slot / a.block;
                    off = slot - b * a.block;
                    block0 = (is_k ? a.k_cache : a.v_cache) + page * a.page_bytes + (long long)b * a.block * a.Hkv * D + hk * D;
                    scale = (is_k ? a.k_scales : a.v_scales) + ((long long)page * (a.page_size / a.block) + b) * a.Hkv + hk;
                }
                if (is_k)
                    e4m3_head<T, D, true>(a, u, table, a.k + at, a.k_row, k_out, a.k_out_row, block0, off, scale, lane);
                else
                    e4m3_head<T, D, false>(a, u, table, a.v + at, a.v_row, nullptr, 0, block0, off, scale, lane);
            } else {
                if (is_k)
                    plain_head<T, D, true>(a, u, table, a.k + at, a.k_row, k_out, a.k_out_row, a.k_cache + at, sh_place, lane);
                else
                    plain_head<T, D, false>(a, u, table, a.v + at, a.v_row, nullptr, 0, a.v_cache + at, sh_place, lane);
            }
        }
        __syncthreads();
    }
}

template <class T, int D, bool EIGHT>
cudaError_t launch(const RotaryArgs& a, dim3 grid, cudaStream_t stream)
{
    auto kern = cache_rotary_kernel<T, D, EIGHT>;
    const size_t bytes = (size_t)a.step * (a.rot / 2) * sizeof(float2);
    if (bytes > 32 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
        if (e != cudaSuccess) return e;
    }
    kern<<<grid, kThreads, bytes, stream>>>(a);
    return cudaGetLastError();
}

template <class T, bool EIGHT>
cudaError_t launch_d(const RotaryArgs& a, int32_t d, dim3 grid, cudaStream_t stream)
{
    switch (d) {
    case 16: return launch<T, 16, EIGHT>(a, grid, stream);
    case 32: return launch<T, 32, EIGHT>(a, grid, stream);
    case 64: return launch<T, 64, EIGHT>(a, grid, stream);
    default: return launch<T, 128, EIGHT>(a, grid, stream);
    }
}

}  // namespace

cudaError_t launch_cache_append_rotary(RotaryArgs a, int32_t d, bool bf16, int sms, cudaStream_t stream)
{
    a.step = a.block ? a.block : 16;
    // As many rows per thread block as a unit has, fewer when that would leave SMs idle
    // (one per block with few tokens); then the heads are spread over more blocks too.
    const int spread = a.T / (2 * sms);
    a.window = spread < 1 ? 1 : spread > a.step ? a.step : spread;
    const int blocks = a.T > 0 ? (a.T + a.window - 1) / a.window : 1;    // no rows: new_lengths alone
    const int rounds = ((a.q ? a.Hq : 0) + 2 * a.Hkv + kWarps - 1) / kWarps;
    int y = (4 * sms + blocks - 1) / blocks;
    y = y > rounds ? rounds : y;
    const dim3 grid((unsigned)blocks, (unsigned)(y > 65535 ? 65535 : y));
    if (bf16)
        return a.block ? launch_d<__nv_bfloat16, true>(a, d, grid, stream) : launch_d<__nv_bfloat16, false>(a, d, grid, stream);
    return a.block ? launch_d<float, true>(a, d, grid, stream) : launch_d<float, false>(a, d, grid, stream);
}

}  // namespace kda
