// rows8.hpp - rows of bf16 or fp32 elements in groups of eight, and their
// 8-bit form: int8 values with one fp32 scale per row or per group of
// columns.  Shared by the row kernels (rows8.hip) and the kernels that read
// the 8-bit form.
#pragma once

#include "dora_internal.hpp"
#include "epilogue.hpp"

namespace dora {

// 16 bytes at any element boundary: rows of an odd width start anywhere, and
// gfx950 serves a 16-byte access at any address (a crossed cache line costs
// one more request), so one code path covers every width.
typedef unsigned int u32x4_a2_t __attribute__((ext_vector_type(4), aligned(2)));
typedef unsigned int u32x4_a4_t __attribute__((ext_vector_type(4), aligned(4)));
typedef unsigned int u32x2_a1_t __attribute__((ext_vector_type(2), aligned(1)));
typedef unsigned int u32x4_a1_t __attribute__((ext_vector_type(4), aligned(1)));

// Eight consecutive elements, as they are stored.  load() takes the first
// `cnt` of them (the rest read as zero), store() writes the first `cnt`.
template <typename T>
struct Raw8;

template <>
struct Raw8<uint16_t> {
    unsigned int w[4];
    __device__ __forceinline__ void load(const uint16_t *p, int cnt)
    {
        if (cnt >= 8) {
            const u32x4_a2_t v = __builtin_nontemporal_load(reinterpret_cast<const u32x4_a2_t *>(p));
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
    __device__ __forceinline__ void load(const float *p, int cnt)
    {
        if (cnt >= 8) {
            const u32x4_a4_t a = __builtin_nontemporal_load(reinterpret_cast<const u32x4_a4_t *>(p));
            const u32x4_a4_t b =
                __builtin_nontemporal_load(reinterpret_cast<const u32x4_a4_t *>(p + 4));
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

// rint(v / s), ties to even, exactly: v inv is off by less than 2e-5 (|v / s|
// <= 127, two roundings of 2^-24), so only quotients within that of a tie
// need the remainder v - q s, which one fma forms without rounding.
__device__ __forceinline__ int quantize1(float v, float s, float inv)
{
    const float t = v * inv;
    float q = rintf(t);
    if (fabsf(t - q) > 0.4999f) {
        const float rem2 = 2.f * __fmaf_rn(-q, s, v);
        const bool odd = (static_cast<int>(q) & 1) != 0;
        if (rem2 > s || (rem2 == s && odd))
            q += 1.f;
        else if (-rem2 > s || (-rem2 == s && odd))
            q -= 1.f;
    }
    // a scale capped from above leaves |v / s| a hair over 127
    return static_cast<int>(fminf(fmaxf(q, -127.f), 127.f));
}

__device__ __forceinline__ Raw8i quantize8(const float (&v)[8], float s, float inv)
{
    Raw8i r;
    r.w[0] = r.w[1] = 0u;
#pragma unroll
    for (int q = 0; q < 8; ++q)
        r.w[q >> 2] |= (static_cast<unsigned int>(quantize1(v[q], s, inv)) & 0xffu) << (8 * (q & 3));
    // (an infinity times an inverse of 0 is a NaN, not 0)
    const unsigned int some = s > 0.f ? 0xffffffffu : 0u;
    r.w[0] &= some;
    r.w[1] &= some;
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

// The largest over aligned runs of `lanes` lanes (a power of two up to 64).
__device__ __forceinline__ unsigned int lanes_max(unsigned int v, int lanes)
{
    for (int d = lanes >> 1; d > 0; d >>= 1) {
        const unsigned int o = __shfl_xor(v, d);
        v = v > o ? v : o;
    }
    return v;
}

// Over a workgroup of NW waves; `red` holds NW values and is free again after
// the call's second barrier.
template <int NW>
__device__ __forceinline__ float block_sum(float v, float *red)
{
    v = wave_sum(v);
    __syncthreads();
    if ((threadIdx.x & 63) == 0)
        red[threadIdx.x >> 6] = v;
    __syncthreads();
    float s = red[0];
#pragma unroll
    for (int k = 1; k < NW; ++k)
        s += red[k];
    return s;
}

template <int NW>
__device__ __forceinline__ unsigned int block_max(unsigned int v, unsigned int *red)
{
    v = lanes_max(v, 64);
    __syncthreads();
    if ((threadIdx.x & 63) == 0)
        red[threadIdx.x >> 6] = v;
    __syncthreads();
    unsigned int s = red[0];
#pragma unroll
    for (int k = 1; k < NW; ++k)
        s = s > red[k] ? s : red[k];
    return s;
}

}  // namespace dora
