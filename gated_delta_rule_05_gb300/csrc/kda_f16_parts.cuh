// kda_f16_parts.cuh -- products of fp16 parts on mma.sync, as the attention kernels
// for whatever tcgen05 does not take share them.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

namespace kda {
namespace f16_parts {

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t smem_at(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool there)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The same onto nothing.
__device__ __forceinline__ void mma0(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%10, %10, %10, %10};"
                 : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ uint32_t two_f16(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// What two_f16 leaves of the pair, times 2^11, as fp16: next to its first part, the second has all
// of its bits then wherever the first is a normal number, and reaches down to 2^-36 below that.
// Products with it have sums of their own, which count 2^-11 (kRest).
constexpr float kRest = 1.f / 2048.f;
__device__ __forceinline__ uint32_t two_f16_rest(float lo, float hi, uint32_t taken)
{
    const float2 t = __half22float2(*reinterpret_cast<const __half2*>(&taken));
    return two_f16((lo - t.x) * 2048.f, (hi - t.y) * 2048.f);
}
// The references of a softmax: m near the maximum of a row's scores moves when one exceeds it by more
// than kSlack; n lies kHead below the one of the scores with their values' factors, so that a row's
// largest weight is 2^7 to 2^15 in fp16, whose normal numbers reach down to 2^-14: a weight has its 11
// bits down to 2^-21 of the largest, and is off by 2^-32 of that at most below.
constexpr float kSlack = 8.f, kHead = 7.f;

__device__ __forceinline__ float quad_max(float x)
{
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
    return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
}

// Bits of the largest magnitude.
__device__ __forceinline__ uint32_t top_of(uint32_t top, float x) { return max(top, __float_as_uint(x) & 0x7FFFFFFFu); }
// The power of two that brings that magnitude to 2^14 or a little more; for the smallest, some of them
// subnormal, the one whose inverse is still a normal number.
__device__ __forceinline__ int up_of(uint32_t top) { return top == 0 ? 0 : min(14 + 127 - (int)(top >> 23), 126); }
__device__ __forceinline__ float power(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }

// What a value's probability is multiplied by to become its weight: the value's factor times 2^(m - n),
// but finite, so that a probability of 0 (of a hidden key, or of one far below the maximum) gives a
// weight of 0.  Where this cuts off, the probability is 2^-112 at most.  NaN stays NaN.
__device__ __forceinline__ float weight_factor(float down, float fac)
{
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(down * fac), "f"(1.7014118e38f));
    return r;
}

// A scale's magnitude as pre * rest: pre, a power of two up to 1, goes to the queries before their rows'
// factors are found, so that rest times the inverse of such a factor is a normal number however small
// the scale is.
struct ScaleParts {
    float pre, rest;
};
__device__ __forceinline__ ScaleParts scale_parts(float scale)
{
    const int e = max(min((int)((__float_as_uint(scale) >> 23) & 255) - 127, 0), -126);
    return {power(e), fabsf(scale) * power(-e)};
}

}  // namespace f16_parts
}  // namespace kda
