// kda_args.cuh -- checks of arguments that the calls around the softmax layers
// share (host code).
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "kda.h"

namespace kda {
namespace args {

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline bool supported_d(int32_t d) { return d == 16 || d == 32 || d == 64 || d == 128; }

inline bool overlaps(const void* a, size_t na, const void* b, size_t nb)
{
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + nb && y < x + na;
}

inline bool valid_dtype(kda_dtype_t t) { return t == KDA_BF16 || t == KDA_FP32 || t == KDA_BF16_F32OUT; }

inline size_t in_bytes(kda_dtype_t t) { return t == KDA_FP32 ? 4 : 2; }
inline size_t out_bytes(kda_dtype_t t) { return t == KDA_BF16 ? 2 : 4; }

// Bytes from the first to the last element of a layer's pages, and whether the
// strides are ones that the kernels take.
inline bool cache_shape(int32_t num_pages, int32_t page_size, int32_t Hkv, int32_t d, int64_t page_stride,
                 size_t elem, size_t* bytes)
{
    const int64_t page_elems = (int64_t)page_size * Hkv * d;
    if (num_pages > 1 && (page_stride < page_elems || (page_stride * (int64_t)elem) % 16 != 0)) return false;
    *bytes = ((size_t)(num_pages - 1) * (size_t)(num_pages > 1 ? page_stride : 0) + (size_t)page_elems) * elem;
    return true;
}

}  // namespace args
}  // namespace kda
