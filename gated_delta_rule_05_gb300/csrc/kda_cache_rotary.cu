// kda_cache_rotary.cu -- queries and keys rotated to their positions, keys and
// values into the pages of a cache (kda_cache_append_rotary).
//
// A pair (x, y) of a row at position p is turned by p f, f the pair's frequency:
// (x cos - y sin, x sin + y cos).  The angle is taken in turns, in fixed point:
// p * round(2^64 frac(f / 2 pi)) mod 2^64 is the fraction of a turn, whatever p is, but for
// the 53 bits that f / 2 pi is worked out in (p f 2^-54 of a turn), where fp32 would lose what
// matters (at position 10^6 an angle is off by 0.03).  Its upper 32 bits go to sincospif as
// fp32, which rounds them to 2^-26 of a turn.
//
// Rows that are only turned and copied (queries; in a cache of the model's type keys and
// values too): a lane holds 16 channels of a row, two vectors of eight that belong
// together, namely the halves of eight pairs or eight neighbouring pairs.  It works out its row's
// place and its eight sines and cosines once and goes through the heads with them, four
// heads under way, no shared memory and no barrier.
//
// 8 bits: a unit is the part of one block of rows that one sequence adds to.  The thread
// block that owns its first row tabulates the sines and cosines of its rows; a team of as
// many warps as hold the block in registers has a head of k or v: it reads the rows
// once, turns them, finds the largest magnitude (so that infinities and NaN win) and
// stores x / s.  s is a power of two: e4m3 is a floating type, so a finer scale would gain
// nothing, and the division, a later change of the scale and the product in the attention
// are exact but for e4m3's own rounding.  A scale of NaN marks a block with an infinity or
// NaN; its bytes are 0, so that no product of a weight of 0 with it is NaN.
//
// Bound by the bytes moved: 12 prompts of 512 to 12,288 tokens, 32 query heads on 8, d =
// 128, bf16, into a bf16 cache 305 us (the rate of a copy), into 8 bits in blocks of 64 rows 320 us
// (88 %), 8 fp32 prompts of 4,096 253 us (91 %).  Few rows are bound by the chain of loads, angles and
// the block's maximum: 64 sequences of a token 5.4 us, one prompt of 1,023 14 us.
#include "kda_prompt.cuh"
#include "kda_sm100.cuh"

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

template <class T>
struct Pieces {
    typename RawOf<T>::type a, b;
};
template <class T>
__device__ __forceinline__ void widen(const Pieces<T>& r, float (&x)[8], float (&y)[8])
{
    widen(r.a, x);
    widen(r.b, y);
}
template <class T>
__device__ __forceinline__ Pieces<T> load_pieces(const uint8_t* row, const Pair& p)
{
    return {load_raw<T>(row + p.a * (int)sizeof(T)), load_raw<T>(row + p.b * (int)sizeof(T))};
}
template <class T>
__device__ __forceinline__ void store_pieces(uint8_t* row, const Pair& p, const float (&x)[8], const float (&y)[8])
{
    store8(reinterpret_cast<T*>(row + p.a * (int)sizeof(T)), x);
    store8(reinterpret_cast<T*>(row + p.b * (int)sizeof(T)), y);
}

// (cos, sin) of pair j of a row at position pos.
__device__ __forceinline__ float2 angle(unsigned long long turns, long long pos)
{
    float s, c;
    // the upper 32 bits as a signed fraction of a turn, in half turns: times 2^-31
    sincospif((float)(int32_t)(((unsigned long long)pos * turns) >> 32) * 4.656612873077393e-10f, &s, &c);
    return make_float2(c, s);
}
// Turns per position of a pair, times 2^64.  In fp64: 53 bits of a fraction that a
// position (31 bits) multiplies.
__device__ __forceinline__ unsigned long long turns_of(float inv_freq)
{
    double f = (double)inv_freq * 0.15915494309189533577;
    f -= floor(f);
    return __double2ull_rn(f * 18446744073709551616.0);
}

// Turns a lane's 16 channels by its eight angles.
__device__ __forceinline__ void turn(const float2 (&w)[8], bool interleaved, float (&x)[8], float (&y)[8])
{
    if (interleaved) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float x0 = x[2 * i], y0 = y[2 * i];
            x[2 * i] = x0 * w[i].x - x[2 * i + 1] * w[i].y;
            x[2 * i + 1] = x0 * w[i].y + x[2 * i + 1] * w[i].x;
            y[2 * i] = y0 * w[4 + i].x - y[2 * i + 1] * w[4 + i].y;
            y[2 * i + 1] = y0 * w[4 + i].y + y[2 * i + 1] * w[4 + i].x;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float x0 = x[i];
            x[i] = x0 * w[i].x - y[i] * w[i].y;
            y[i] = x0 * w[i].y + y[i] * w[i].x;
        }
    }
}

// The same from the table of a unit's rows.
__device__ __forceinline__ void turn(const float2* table, int row, const Pair& p, int rot, bool interleaved, float (&x)[8], float (&y)[8])
{
    const float4* t = reinterpret_cast<const float4*>(table + row * (rot / 2)) + p.c;
    float2 w[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float4 z = t[i * (rot / 16)];        // (cos, sin) of pairs 2 i and 2 i + 1
        w[2 * i] = make_float2(z.x, z.y);
        w[2 * i + 1] = make_float2(z.z, z.w);
    }
    turn(w, interleaved, x, y);
}

// The larger of top and eight magnitudes; NaN when one is NaN.
__device__ __forceinline__ float top_of(float top, const float (&x)[8])
{
#pragma unroll
    for (int i = 0; i < 8; i += 2)
        asm("{\n\t.reg .f32 a, b;\n\tabs.f32 a, %1;\n\tabs.f32 b, %2;\n\tmax.NaN.f32 %0, %0, a, b;\n\t}" : "+f"(top) : "f"(x[i]), "f"(x[i + 1]));
    return top;
}

// Where position pos of sequence n lies: page and row in it; false: nowhere.
__device__ __forceinline__ bool place_of(const RotaryArgs& a, int n, long long pos, int& page, int& slot)
{
    if (pos >= (long long)a.max_pages * a.page_size) return false;
    const int at = (int)(pos / a.page_size);
    page = __ldg(a.page_table + (long long)n * a.max_pages + at);
    slot = (int)(pos - (long long)at * a.page_size);
    return page >= 0 && page < a.num_pages;
}

constexpr int kAhead = 4;              // heads under way in the rows that are only turned

// Heads h0 .. h1 - 1 of a row's tensor, `step` bytes from head to head; from src to dst and
// to cache (either may be null).
template <class T, int D, bool TURN>
__device__ __forceinline__ void row_heads(const uint8_t* src, uint8_t* dst, uint8_t* cache, int heads, const Pair& p,
                                          const float2 (&w)[8], bool interleaved)
{
    constexpr int kHead = D * (int)sizeof(T);
#pragma unroll 1
    for (int h = 0; h < heads; h += kAhead) {
        Pieces<T> r[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (h + i < heads) r[i] = load_pieces<T>(src + (h + i) * kHead, p);
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            if (h + i >= heads) break;
            float x[8], y[8];
            widen(r[i], x, y);
            if (TURN && p.turned) turn(w, interleaved, x, y);
            if (dst) store_pieces<T>(dst + (h + i) * kHead, p, x, y);
            if (cache) store_pieces<T>(cache + (h + i) * kHead, p, x, y);
        }
    }
}

// Rows that are only turned and copied: a warp has 32 / (D / 16) rows and some of
// their heads.
template <class T, int D, bool EIGHT>
__device__ __forceinline__ void rows_part(const RotaryArgs& a, const int32_t* cu, const unsigned long long* turns, int block, int warp, int lane)
{
    constexpr int L = D / 16, R = 32 / L;
    const long long id = (long long)block * kWarps + warp;
    const int chunk = (int)(id % a.chunks), h0 = chunk * a.chunk_heads;
    const long long first = id / a.chunks * R;
    const int r = (int)(first + lane / L);
    if (first >= a.T || r >= a.T) return;
    int n, start, end;
    if (!row_owner(a, cu, r, n, start, end)) return;
    const int len = __ldg(a.lengths + n);
    if (len < 0) return;
    const long long pos = (long long)len + (r - start);
    const int c = lane % L;
    const Pair p = pair_of(c, a.rot, a.interleaved);
    float2 w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = p.turned ? angle(turns[8 * c + i], pos) : make_float2(1.f, 0.f);
    const int h1 = h0 + a.chunk_heads;             // of the queries, then keys, then values
    constexpr int kHead = D * (int)sizeof(T);
    if (h0 < a.Hq) {
        const int n_q = min(h1, a.Hq) - h0;
        row_heads<T, D, true>(a.q + r * a.q_row + h0 * kHead, a.q_out + r * a.q_out_row + h0 * kHead, nullptr, n_q, p, w, a.interleaved);
    }
    if constexpr (!EIGHT) {
        if (h1 <= a.Hq) return;
        int page, slot;
        const bool there = place_of(a, n, pos, page, slot);
        const long long at = there ? page * a.page_bytes + (long long)slot * a.Hkv * kHead : 0;
        const int k0 = max(h0 - a.Hq, 0), k1 = min(h1 - a.Hq, a.Hkv);
        if (k0 < k1)
            row_heads<T, D, true>(a.k + r * a.k_row + k0 * kHead, a.k_out ? a.k_out + r * a.k_out_row + k0 * kHead : nullptr,
                                  there ? a.k_cache + at + k0 * kHead : nullptr, k1 - k0, p, w, a.interleaved);
        const int v0 = max(h0 - a.Hq - a.Hkv, 0), v1 = min(h1 - a.Hq - a.Hkv, a.Hkv);
        if (v0 < v1 && there)
            row_heads<T, D, false>(a.v + r * a.v_row + v0 * kHead, nullptr, a.v_cache + at + v0 * kHead, v1 - v0, p, w, a.interleaved);
    }
}

// Rows of a lane.  Two (twice the warps to a team) took 346 us where four took 329; loads of the
// next head before the stores of this one spill registers (408 against 342), and by cp.async
// into shared memory, without spills, they gain nothing (319.6 against 319.9); values
// read from the cache lines anew instead of kept turned in registers 329 against 320.
constexpr int kHeld = 4;

// One head of a unit's rows as e4m3 into its block of the cache, by a team of `team`
// warps: `block0` the block's first row there (null: the rows have no place), `off`
// the rows that it already has, `scale` its scale.
struct Held {
    float x[kHeld][8], y[kHeld][8];
};
template <class T, int D, bool TURN>
__device__ __forceinline__ void e4m3_head(const RotaryArgs& a, const Unit& u, const float2* table, const uint8_t* src, long long src_row,
                                          uint8_t* dst, long long dst_row, uint8_t* block0, int off, float* scale, uint32_t* tops, int team,
                                          int warp, int lane, int tl)
{
    constexpr int L = D / 16;
    const Pair p = pair_of(tl % L, TURN ? a.rot : 0, a.interleaved);
    const int r0 = tl / L, pass = team * 32 / L;
    const int row_bytes = a.Hkv * D;
    Held v;
    {
        Pieces<T> raw[kHeld];
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            raw[i] = {};
            const int r = r0 + i * pass;
            if (r < u.count) raw[i] = load_pieces<T>(src + (u.first + r) * src_row, p);
        }
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            widen(raw[i], v.x[i], v.y[i]);
            if (TURN && p.turned && r0 + i * pass < u.count) turn(table, r0 + i * pass, p, a.rot, a.interleaved, v.x[i], v.y[i]);
        }
    }
    uint32_t old = 0;
    if (block0 && off > 0) old = __float_as_uint(*reinterpret_cast<volatile float*>(scale)) & 0x7FFFFFFFu;
    float most = 0.f;
#pragma unroll
    for (int i = 0; i < kHeld; ++i) most = top_of(top_of(most, v.x[i]), v.y[i]);
    uint32_t top = __float_as_uint(most) & 0x7FFFFFFFu;
    top = __reduce_max_sync(0xffffffffu, top);
    if (team > 1) {
        const int first = warp / team * team;
        if (lane == 0) tops[warp] = top;
        sm100::named_bar_sync(1 + first, team * 32);
        for (int i = 0; i < team; ++i) top = max(top, tops[first + i]);
        // (all have read before the next head's are written)
        sm100::named_bar_sync(1 + first, team * 32);
    } else {
        __syncwarp();                              // every lane has read the old scale
    }
    uint32_t sb = scale_bits(top);
    if (block0) {
        if (sb > old && old > 0 && sb < 0x7F800000u) {
            // the rows that are there, in the new scale
            const float ratio = __uint_as_float(old) * __uint_as_float(0x7F000000u - sb);
            for (int e = tl; e < off * (D / 8); e += team * 32) {
                uint2* w = reinterpret_cast<uint2*>(block0 + (long long)(e / (D / 8)) * row_bytes + e % (D / 8) * 8);
                const uint2 b = *w;
                const float2 b0 = from_e4m3(b.x), b1 = from_e4m3(b.x >> 16), b2 = from_e4m3(b.y), b3 = from_e4m3(b.y >> 16);
                *w = make_uint2(four_e4m3(b0.x * ratio, b0.y * ratio, b1.x * ratio, b1.y * ratio),
                                four_e4m3(b2.x * ratio, b2.y * ratio, b3.x * ratio, b3.y * ratio));
            }
        }
        sb = max(sb, old);
        if (tl == 0) *scale = __uint_as_float(sb);
    }
    const bool store = sb > 0 && sb < 0x7F800000u;
    const float inv = store ? __uint_as_float(0x7F000000u - sb) : 0.f;
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
        const int r = r0 + i * pass;
        if (r >= u.count) break;
        const float(&x)[8] = v.x[i], (&y)[8] = v.y[i];
        if (dst) store_pieces<T>(dst + (u.first + r) * dst_row, p, x, y);
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

template <class T, int D>
__device__ __forceinline__ void units_part(const RotaryArgs& a, const int32_t* cu, const unsigned long long* turns, float2* table,
                                           int block, int warp, int lane)
{
    __shared__ Unit sh_unit[kMaxScaleBlock];       // of each row of the window; count 0: no unit begins there
    __shared__ uint32_t sh_tops[kWarps];
    const int tid = threadIdx.x;
    const int window = block / a.splits, split = block - window * a.splits;
    if (tid < a.window) {
        Unit u = {0, 0, 0, 0};
        const long long r = (long long)window * a.window + tid;
        int n, start, end;
        if (r < a.T && row_owner(a, cu, (int)r, n, start, end)) {
            const int len = __ldg(a.lengths + n);
            if (len >= 0) {
                u.n = n;
                u.first = (int)r;
                u.pos = (long long)len + (u.first - start);
                const int left = a.block - (int)(u.pos % a.block);
                if (u.first == start || left == a.block) u.count = min(left, end - u.first);
            }
        }
        sh_unit[tid] = u;
    }
    __syncthreads();
    const int half = a.rot / 2, teams = kWarps / a.team;
#pragma unroll 1
    for (int w = 0; w < a.window; ++w) {
        const Unit u = sh_unit[w];
        if (u.count == 0) continue;                // (the same for all threads)
        for (int e = tid; e < u.count * half; e += kThreads) {
            const int r = e / half, j = e - r * half;
            table[table_at(r, j, a.rot)] = angle(turns[j], u.pos + r);
        }
        int page, slot;
        const bool there = place_of(a, u.n, u.pos, page, slot);    // (a block lies in one page)
        const int b = there ? slot / a.block : 0, off = there ? slot - b * a.block : 0;
        const long long block_at = there ? page * a.page_bytes + (long long)b * a.block * a.Hkv * D : 0;
        const long long scale_at = there ? ((long long)page * (a.page_size / a.block) + b) * a.Hkv : 0;
        const int step = a.splits * teams, tl = (warp % a.team) * 32 + lane;
        int task = split * teams + warp / a.team;
        __syncthreads();                           // the table is there
#pragma unroll 1
        for (; task < 2 * a.Hkv; task += step) {
            const bool is_k = task < a.Hkv;
            const int hk = is_k ? task : task - a.Hkv;
            uint8_t* block0 = there ? (is_k ? a.k_cache : a.v_cache) + block_at + hk * D : nullptr;
            float* scale = (is_k ? a.k_scales : a.v_scales) + scale_at + hk;
            if (is_k)
                e4m3_head<T, D, true>(a, u, table, a.k + (long long)hk * D * (int)sizeof(T), a.k_row, a.k_out ? a.k_out + (long long)hk * D * (int)sizeof(T) : nullptr, a.k_out_row,
                                      block0, off, scale, sh_tops, a.team, warp, lane, tl);
            else
                e4m3_head<T, D, false>(a, u, table, a.v + (long long)hk * D * (int)sizeof(T), a.v_row, nullptr, 0, block0, off, scale, sh_tops, a.team, warp, lane, tl);
        }
        __syncthreads();
    }
}

// The first unit_blocks thread blocks have the units (8 bits), the others rows.
template <class T, int D, bool EIGHT>
__global__ void __launch_bounds__(kThreads, 2)
cache_rotary_kernel(const __grid_constant__ RotaryArgs a)
{
    extern __shared__ __align__(16) uint8_t dyn[];
    __shared__ int32_t sh_cu[kHeldSeqs + 1];
    __shared__ unsigned long long sh_turns[64];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int32_t* cu = a.cu_seqlens;
    if (a.N <= kHeldSeqs) {
        for (int i = tid; i <= a.N; i += kThreads) sh_cu[i] = __ldg(a.cu_seqlens + i);
        cu = sh_cu;
    }
    if (tid < a.rot / 2) sh_turns[tid] = turns_of(__ldg(a.inv_freq + tid));
    __syncthreads();
    if (a.new_lengths) {
        // (with millions of sequences of a token there are more threads than 2^31)
        for (long long n = (long long)blockIdx.x * kThreads + tid; n < a.N; n += (long long)gridDim.x * kThreads) {
            const int first = max(cu[n], 0), end = min(cu[n + 1], a.T);
            a.new_lengths[n] = __ldg(a.lengths + n) + (end > first ? end - first : 0);     // (their difference may not fit)
        }
    }
    if (EIGHT && (int)blockIdx.x < a.unit_blocks)
        units_part<T, D>(a, cu, sh_turns, reinterpret_cast<float2*>(dyn), blockIdx.x, warp, lane);
    else
        rows_part<T, D, EIGHT>(a, cu, sh_turns, blockIdx.x - a.unit_blocks, warp, lane);
}

template <class T, int D, bool EIGHT>
cudaError_t launch(const RotaryArgs& a, unsigned blocks, cudaStream_t stream)
{
    auto kern = cache_rotary_kernel<T, D, EIGHT>;
    const size_t bytes = EIGHT ? (size_t)a.block * (a.rot / 2) * sizeof(float2) : 0;
    // (the same limit from every call, as another thread may set it between these two steps)
    constexpr size_t most = (size_t)kMaxScaleBlock * (D / 2) * sizeof(float2);
    if (EIGHT && most > 32 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
        if (e != cudaSuccess) return e;
    }
    kern<<<blocks, kThreads, bytes, stream>>>(a);
    return cudaGetLastError();
}

template <class T, bool EIGHT>
cudaError_t launch_d(const RotaryArgs& a, int32_t d, unsigned blocks, cudaStream_t stream)
{
    switch (d) {
    case 16: return launch<T, 16, EIGHT>(a, blocks, stream);
    case 32: return launch<T, 32, EIGHT>(a, blocks, stream);
    case 64: return launch<T, 64, EIGHT>(a, blocks, stream);
    default: return launch<T, 128, EIGHT>(a, blocks, stream);
    }
}

}  // namespace

cudaError_t launch_cache_append_rotary(RotaryArgs a, int32_t d, bool bf16, int sms, cudaStream_t stream)
{
    long long units = 0;
    if (a.block) {
        // As many rows per thread block as a unit has on the average (every sequence may begin one
        // in the middle of a block); with few units their heads are spread over more blocks, each
        // of which tabulates the angles anew.  32 query heads on 8, d = 128, blocks of 64 rows, 1, 2,
        // 4 and 8 parts, us: 17 windows 23.9, 17.0, 14.0, 13.8; 64 windows 31.4, 24.2, 27.6, 33.3; 164
        // windows 53.1, 36.6, 42.5, 55.9; 254 windows 74.4, 79.2, 90.2, 117.3.  Windows of one row
        // take 725 us instead of 320 for 12 prompts of 512 to 12,288 rows, windows of a whole block
        // 34 instead of 5.4 for 64 sequences of a token each.
        const long long rows = a.T / ((long long)a.T / a.block + a.N);
        a.window = rows < 1 ? 1 : rows > a.block ? a.block : (int)rows;
        const int lanes = a.block * (d / 16);      // of a block's rows
        a.team = 1;
        while (a.team * 32 * kHeld < lanes) a.team *= 2;
        const long long windows = ((long long)a.T + a.window - 1) / a.window;
        const int rounds = (2 * a.Hkv * a.team + kWarps - 1) / kWarps;
        const long long most = windows > 0 ? (5ll * sms / 4 + windows - 1) / windows : 1;
        a.splits = (int)(most < 1 ? 1 : most > rounds ? rounds : most);
        units = windows * a.splits;
    }
    // the rows, in groups of a warp's, and a part of their heads each, where all would
    // leave SMs idle (one prompt of 1,000 rows 9.2 us, with all heads 13.8; 64 rows 5.0 and 13.7)
    const int per = 32 / (d / 16), heads = a.Hq + (a.block ? 0 : 2 * a.Hkv);
    const long long groups = heads ? ((long long)a.T + per - 1) / per : 0;
    a.chunks = 1;
    while (a.chunks < heads / kAhead && groups * a.chunks < 2ll * kWarps * sms) a.chunks *= 2;
    a.chunk_heads = (heads + a.chunks - 1) / a.chunks;
    const long long blocks = units + (groups * a.chunks + kWarps - 1) / kWarps;
    if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
    a.unit_blocks = (int32_t)units;
    const unsigned grid = blocks > 0 ? (unsigned)blocks : 1;       // no rows: new_lengths alone
    if (bf16)
        return a.block ? launch_d<__nv_bfloat16, true>(a, d, grid, stream) : launch_d<__nv_bfloat16, false>(a, d, grid, stream);
    return a.block ? launch_d<float, true>(a, d, grid, stream) : launch_d<float, false>(a, d, grid, stream);
}

}  // namespace kda
