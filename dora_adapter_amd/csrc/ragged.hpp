// ragged.hpp - 16-byte loads at any element, for rows whose width leaves them
// unaligned: a load that runs past the end of its row, or of its matrix, is put
// right in registers.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace dora {

typedef unsigned int u32x4_a1_t __attribute__((ext_vector_type(4), aligned(1)));

__device__ __forceinline__ uint4 load16_any(const void *p)
{
    const u32x4_a1_t v = *static_cast<const u32x4_a1_t *>(p);
    return make_uint4(v.x, v.y, v.z, v.w);
}

// What is left of 16 bytes that were loaded `back` bytes early and of which
// `left` bytes belong to the row (the rest zeros): the row's last chunk.
__device__ __forceinline__ uint4 row_end16(uint4 v, int back, int64_t left)
{
    uint64_t lo = v.x | static_cast<uint64_t>(v.y) << 32;
    uint64_t hi = v.z | static_cast<uint64_t>(v.w) << 32;
    if (back >= 8) {
        lo = hi >> (8 * (back - 8));
        hi = 0;
    } else if (back > 0) {
        lo = lo >> (8 * back) | hi << (64 - 8 * back);
        hi >>= 8 * back;
    }
    const int n = left < 0 ? 0 : (left < 16 ? static_cast<int>(left) : 16);
    lo = n >= 8 ? lo : lo & ((1ull << (8 * n)) - 1);
    hi = n >= 16 ? hi : (n > 8 ? hi & ((1ull << (8 * (n - 8))) - 1) : 0);
    return make_uint4(static_cast<unsigned int>(lo), static_cast<unsigned int>(lo >> 32),
                      static_cast<unsigned int>(hi), static_cast<unsigned int>(hi >> 32));
}

}  // namespace dora
