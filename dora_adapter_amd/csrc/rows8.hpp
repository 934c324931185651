// rows8.hpp - rows of bf16 or fp32 elements in groups of eight, and their
// 8-bit form: int8 values with one fp32 scale per row or per group of
// columns.  Shared by the row kernels (rows8.hip) and the kernels that read
// the 8-bit form.
#pragma once

#include "dora_internal.hpp"
#include "epilogue.hpp"

#include <type_traits>

namespace dora {

// 16 bytes at any element boundary: rows of an odd width start anywhere, and
// gfx950 serves a 16-byte access at any address (a crossed cache line costs
// one more request), so one code path covers every width.
typedef unsigned int u32x4_a2_t __attribute__((ext_vector_type(4), aligned(2)));
typedef unsigned int u32x4_a4_t __attribute__((ext_vector_type(4), aligned(4)));
typedef unsigned int u32x2_a1_t __attribute__((ext_vector_type(2), aligned(1)));

// Eight consecutive elements, as they are stored.  load() takes the first
// `cnt` of them (the rest read as zero), store() writes the first `cnt`.
template <typename T>
struct Raw8;

template <>
struct Raw8<uint16_t> {
    unsigned int w[4];
    // KEEP: the data is read again soon (by the other rows), leave it in the caches
    template <bool KEEP = false>
    __device__ __forceinline__ void load(const uint16_t *p, int cnt)
    {
        if (cnt >= 8) {
            const u32x4_a2_t *u = reinterpret_cast<const u32x4_a2_t *>(p);
            const u32x4_a2_t v = KEEP ? *u : __builtin_nontemporal_load(u);
            w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
        } else {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const unsigned int lo = 2 * q < cnt ? p[2 * q] : 0u;
                const unsigned int hi = 2 * q + 1 < cnt ? p[2 * q + 1] : 0u;
                w[q] = lo | (hi << 16);
            }
        }
    }
    __device__ __forceinline__ void store(uint16_t *p, int cnt) const
    {
        if (cnt >= 8) {
            const u32x4_a2_t v = {w[0], w[1], w[2], w[3]};
            __builtin_nontemporal_store(v, reinterpret_cast<u32x4_a2_t *>(p));
        } else {
#pragma unroll
            for (int q = 0; q < 8; ++q)
                if (q < cnt)
                    p[q] = static_cast<uint16_t>(w[q >> 1] >> (16 * (q & 1)));
        }
    }
    __device__ __forceinline__ void get(float (&v)[8]) const
    {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            v[2 * q] = __uint_as_float(w[q] << 16);
            v[2 * q + 1] = __uint_as_float(w[q] & 0xffff0000u);
        }
    }
    // rounded once, to nearest even
    __device__ __forceinline__ void set(const float (&v)[8])
    {
#pragma unroll
        for (int q = 0; q < 4; ++q)
            w[q] = pack_bf16x2(v[2 * q], v[2 * q + 1]);
    }
};

template <>
struct Raw8<float> {
    unsigned int w[8];
    template <bool KEEP = false>
    __device__ __forceinline__ void load(const float *p, int cnt)
    {
        if (cnt >= 8) {
            const u32x4_a4_t *u = reinterpret_cast<const u32x4_a4_t *>(p);
            const u32x4_a4_t a = KEEP ? u[0] : __builtin_nontemporal_load(u);
            const u32x4_a4_t b = KEEP ? u[1] : __builtin_nontemporal_load(u + 1);
            w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
            w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
        } else {
#pragma unroll
            for (int q = 0; q < 8; ++q)
                w[q] = q < cnt ? __float_as_uint(p[q]) : 0u;
        }
    }
    __device__ __forceinline__ void store(float *p, int cnt) const
    {
        if (cnt >= 8) {
            const u32x4_a4_t a = {w[0], w[1], w[2], w[3]}, b = {w[4], w[5], w[6], w[7]};
            __builtin_nontemporal_store(a, reinterpret_cast<u32x4_a4_t *>(p));
            __builtin_nontemporal_store(b, reinterpret_cast<u32x4_a4_t *>(p + 4));
        } else {
#pragma unroll
            for (int q = 0; q < 8; ++q)
                if (q < cnt)
                    p[q] = __uint_as_float(w[q]);
        }
    }
    __device__ __forceinline__ void get(float (&v)[8]) const
    {
#pragma unroll
        for (int q = 0; q < 8; ++q)
            v[q] = __uint_as_float(w[q]);
    }
    __device__ __forceinline__ void set(const float (&v)[8])
    {
#pragma unroll
        for (int q = 0; q < 8; ++q)
            w[q] = __float_as_uint(v[q]);
    }
};

// The same vector, its values to be formed again from here on: what was unpacked
// from it earlier is then not kept in registers for the next use.
template <typename T>
__device__ __forceinline__ void forget(Raw8<T> &r)
{
#pragma unroll
    for (unsigned int &w : r.w)
        __asm__ volatile("" : "+v"(w));
}

// Eight int8 values.
struct Raw8i {
    unsigned int w[2];
    __device__ __forceinline__ void load(const int8_t *p, int cnt)
    {
        if (cnt >= 8) {
            const u32x2_a1_t v = __builtin_nontemporal_load(reinterpret_cast<const u32x2_a1_t *>(p));
            w[0] = v.x; w[1] = v.y;
        } else {
            w[0] = w[1] = 0u;
#pragma unroll
            for (int q = 0; q < 8; ++q)
                if (q < cnt)
                    w[q >> 2] |= static_cast<unsigned int>(static_cast<uint8_t>(p[q])) << (8 * (q & 3));
        }
    }
    __device__ __forceinline__ void store(int8_t *p, int cnt) const
    {
        if (cnt >= 8) {
            const u32x2_a1_t v = {w[0], w[1]};
            __builtin_nontemporal_store(v, reinterpret_cast<u32x2_a1_t *>(p));
        } else {
#pragma unroll
            for (int q = 0; q < 8; ++q)
                if (q < cnt)
                    p[q] = static_cast<int8_t>(w[q >> 2] >> (8 * (q & 3)));
        }
    }
    __device__ __forceinline__ float value(int q) const
    {
        return static_cast<float>(static_cast<int8_t>(w[q >> 2] >> (8 * (q & 3))));
    }
};

// ------------------------------------------------------------ the 8-bit form
// A group of values v_j (a row, or `group` consecutive columns of one) is held
// as q_j = rint(v_j / s) with s = max_j |v_j| / 127.  The maximum is taken on
// the bit patterns of |v_j|, which order like the values and put infinities
// and NaN above every number, so that a group holding one of those gets a NaN
// scale and restores as NaN throughout instead of as plausible numbers.
__device__ __forceinline__ unsigned int abs_bits(float v)
{
    return __float_as_uint(v) & 0x7fffffffu;
}

// s from the largest |v_j|: 0 for a group of zeros, else between 2^-126 (so
// that 1 / s is finite; smaller values lose at most 2^-127) and the largest s
// with 127 s finite.
__device__ __forceinline__ float scale_of(unsigned int top)
{
    if (top == 0u)
        return 0.f;
    if (top >= 0x7f800000u)
        return __uint_as_float(0x7fc00000u);
    const float s = __uint_as_float(top) / 127.f;
    return fminf(fmaxf(s, 0x1p-126f), 0x1.020406p+121f);
}

// 1 / s, and 0 where nothing is to be scaled (s = 0 or NaN: q = 0).
__device__ __forceinline__ float inverse_scale(float s) { return s > 0.f ? 1.f / s : 0.f; }

// rint(v / s), ties to even, for a quotient v inv near a tie: the remainder
// v - q s of the nearest integer q, which one fma forms without rounding,
// decides (both v and q s are multiples of the smaller one's last place, and
// the difference is about s / 2).
__device__ __forceinline__ float quantize_near_tie(float v, float s, float q)
{
    const float rem2 = 2.f * __fmaf_rn(-q, s, v);
    const bool odd = (static_cast<int>(q) & 1) != 0;
    if (rem2 > s || (rem2 == s && odd))
        return q + 1.f;
    if (-rem2 > s || (-rem2 == s && odd))
        return q - 1.f;
    return q;
}

// Eight quotients rint(v / s).  Adding 1.5 * 2^23 rounds v inv to an integer
// whose two's complement byte is the sum's lowest.  inv is 1 / s to 2^-24, so v
// inv is off by at most 127 * 2^-24 < 8e-6 (|v / s| <= 127 but for a capped
// scale, a hair over): only what lies within 1e-5 of a tie takes the exact
// path, about one vector of 64 lanes in a hundred.
__device__ __forceinline__ Raw8i quantize8(const float (&v)[8], float s, float inv)
{
    constexpr float MAGIC = 12582912.f;
    float f[8], worst = 0.f;
#pragma unroll
    for (int q = 0; q < 8; ++q) {
        f[q] = __fmaf_rn(v[q], inv, MAGIC);
        worst = fmaxf(worst, fabsf(__fmaf_rn(v[q], inv, MAGIC - f[q])));
    }
    if (worst > 0.49999f) {
#pragma unroll
        for (int q = 0; q < 8; ++q)
            f[q] = quantize_near_tie(v[q], s, f[q] - MAGIC) + MAGIC;
    }
    Raw8i r;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const unsigned int lo = __builtin_amdgcn_perm(
            __float_as_uint(f[4 * k + 1]), __float_as_uint(f[4 * k]), 0x0c0c0400u);
        const unsigned int hi = __builtin_amdgcn_perm(
            __float_as_uint(f[4 * k + 3]), __float_as_uint(f[4 * k + 2]), 0x04000c0cu);
        // (a NaN or zero scale: all zeros)
        r.w[k] = s > 0.f ? lo | hi : 0u;
    }
    return r;
}

// ---------------------------------------------------------------- reductions
// Over 64 lanes in a fixed order (every lane gets the result).
__device__ __forceinline__ float wave_sum(float v)
{
#pragma unroll
    for (int d = 32; d > 0; d >>= 1)
        v += __shfl_xor(v, d);
    return v;
}

// The largest over aligned runs of `lanes` lanes (a power of two up to 64, the
// same for the whole wave), for N values at once: the exchanges of one step
// are independent of each other, and a step's distance is a constant.
template <int N>
__device__ __forceinline__ void lanes_max(unsigned int (&v)[N], int lanes)
{
    auto step = [&](auto dist) {
        constexpr int D = decltype(dist)::value;
        if (lanes > D) {
            unsigned int o[N];
#pragma unroll
            for (int i = 0; i < N; ++i)
                o[i] = __shfl_xor(v[i], D);
#pragma unroll
            for (int i = 0; i < N; ++i)
                v[i] = v[i] > o[i] ? v[i] : o[i];
        }
    };
    step(std::integral_constant<int, 1>{});
    step(std::integral_constant<int, 2>{});
    step(std::integral_constant<int, 4>{});
    step(std::integral_constant<int, 8>{});
    step(std::integral_constant<int, 16>{});
    step(std::integral_constant<int, 32>{});
}

__device__ __forceinline__ unsigned int lane_max(unsigned int v, int lanes)
{
    unsigned int a[1] = {v};
    lanes_max(a, lanes);
    return a[0];
}

// Over a workgroup of `waves` waves in a fixed order; `red` holds one value a
// wave (and may be used again by the next call: its writes follow a barrier).
__device__ __forceinline__ float block_sum(float v, float *red, int waves)
{
    v = wave_sum(v);
    if (waves == 1)
        return v;
    __syncthreads();
    if ((threadIdx.x & 63) == 0)
        red[threadIdx.x >> 6] = v;
    __syncthreads();
    float s = red[0];
    for (int k = 1; k < waves; ++k)
        s += red[k];
    return s;
}

__device__ __forceinline__ unsigned int block_max(unsigned int v, unsigned int *red, int waves)
{
    v = lane_max(v, 64);
    if (waves == 1)
        return v;
    __syncthreads();
    if ((threadIdx.x & 63) == 0)
        red[threadIdx.x >> 6] = v;
    __syncthreads();
    unsigned int s = red[0];
    for (int k = 1; k < waves; ++k)
        s = s > red[k] ? s : red[k];
    return s;
}

// y = c xs wscale for an int32 sum c, as (c xs) wscale: c xs leaves fp32's range only
// where xs is so large that c xs wscale need not (2^97 and 2^-97 in front of 1e9), and
// loses no bit below 2^-126, where it is a multiple of 2^-149 like xs.  (The scales' own
// product would leave it far sooner.)  A token scale from 2^96 on is taken 2^64 smaller,
// which the result gets back: c xs wscale is then between 2^-117 and what overflows
// in any case, so that every finite scale gives a y that is right to its own rounding.
// Costs one product an output (by 1, for all but such tokens).
struct I8Scale {
    float by, after;
};
__device__ __forceinline__ I8Scale i8_xs(float xs)
{
    const bool big = fabsf(xs) >= 0x1p96f;
    return {big ? xs * 0x1p-64f : xs, big ? 0x1p64f : 1.f};
}
__device__ __forceinline__ float i8_scaled(int c, I8Scale xs, float ws)
{
    return static_cast<float>(c) * xs.by * ws * xs.after;
}

}  // namespace dora
