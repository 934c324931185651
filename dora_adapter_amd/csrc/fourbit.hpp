// fourbit.hpp - 4-bit rows: e2m1 codes (0, 0.5, 1, 1.5, 2, 3, 4, 6 with a sign, the type that
// gfx950 converts by itself) with one scale for each `group` consecutive columns.
#pragma once

#include "rows8.hpp"

namespace dora {

typedef unsigned int u32x2_a2_t __attribute__((ext_vector_type(2), aligned(2)));
typedef unsigned int u32_a2_t __attribute__((aligned(2)));

// The scale of a group from its largest |v|: top / 6 at six significant bits (ties to even), so
// that a code's two bits times it are a bf16 number exactly.  0 for a group of zeros, NaN where
// the group holds an infinity or a NaN (their bit patterns sort above every number), else
// between 2^-125 (half of it, the smallest value but zero, is a normal number) and the largest
// with 6 s finite in bf16.  The fp32 quotient decides the rounding as the exact one would: at
// a tie top = 6 s' it is exact, and next to one it is off the tie by 2/3 of its last place.
__device__ __forceinline__ float fourbit_scale(unsigned int top)
{
    if (top == 0u)
        return 0.f;
    if (top >= 0x7f800000u)
        return __uint_as_float(0x7fc00000u);
    const unsigned int q = __float_as_uint(__uint_as_float(top) / 6.f);
    const float s = __uint_as_float((q + 0x1ffffu + ((q >> 18) & 1u)) & ~0x3ffffu);
    return fminf(fmaxf(s, 0x1p-125f), 0x1.5p+125f);
}

}  // namespace dora
