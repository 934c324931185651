// fourbit.hip - rows to 4 bits and back (gfx950).  Both are bound by memory traffic, a thread
// takes eight consecutive columns at a time: 16 bytes of bf16, four of codes.  28672 x 8192 in
// bf16: 108 us to codes (5.5 TB/s), 102 back (5.8).
#include "around.hpp"
#include "fourbit.hpp"

namespace dora {
namespace {

constexpr int THREADS = 256;
constexpr int VPT = 4;  // vectors of eight columns a thread

// Threads along a row and rows a workgroup: a workgroup takes `rows` rows by VPT * along vectors.
// No more threads along a row than its vectors have work for, VPT each (28672 x 384 in bf16 to
// codes: 8.8 us, 22 with a thread a vector).
struct Shape {
    unsigned along, rows, shares;
    int64_t groups;  // workgroups along the rows
};
Shape shape_of(int64_t rows, int64_t vecs, int lanes)
{
    Shape s;
    s.along = static_cast<unsigned>(lanes);
    while (s.along < THREADS && s.along * VPT < vecs)
        s.along *= 2;
    s.rows = THREADS / s.along;
    const int64_t shares = (vecs + s.along * VPT - 1) / (s.along * VPT);
    s.shares = static_cast<unsigned>(shares < 4096 ? shares : 4096);
    // (2^23 workgroups at most: the rest by a loop)
    const int64_t most = (int64_t(1) << 23) / s.shares, all = (rows + s.rows - 1) / s.rows;
    s.groups = all < most ? all : most;
    return s;
}

// Eight quotients v / s to e2m1, ties to even, the first in the lowest four bits.
//
// bf16: v times 1 / s is off by 2^-22 of it, and rounding to a multiple of 2^-16 (by adding 192,
// whose last place that is) restores every tie (a multiple of 1/4) and makes none: v has eight
// bits and s six, so that v / s is a tie or at least 2^-13 away from one.
// fp32: the correctly rounded quotient is a tie exactly where v / s is one (v differs from a tie
// times s by its last place or not at all, which moves the quotient by more than half of its).
template <typename T>
__device__ __forceinline__ unsigned int to_codes(const float (&v)[8], float s, float inv)
{
    float t[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) {
        if constexpr (sizeof(T) == 2)
            t[q] = __fmaf_rn(v[q], inv, 192.f) - 192.f;
        else
            t[q] = v[q] / s;
        t[q] = __builtin_amdgcn_fmed3f(t[q], -6.f, 6.f);
    }
    unsigned int c = 0u;
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, t[0], t[1], 1.f, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, t[2], t[3], 1.f, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, t[4], t[5], 1.f, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, t[6], t[7], 1.f, 3);
    return s > 0.f ? c : 0u;
}

template <typename T>
__global__ void __launch_bounds__(THREADS)
    quantize_fourbit_kernel(const T *x, int64_t rows, int64_t d, int64_t groups, int group,
                            uint8_t *codes, uint16_t *scale)
{
    const int lanes = group / 8, shift = 31 - __clz(lanes);
    const int64_t vecs = groups * lanes;  // of a row, its last group whole
    for (int64_t t = blockIdx.x * static_cast<int64_t>(blockDim.y) + threadIdx.y;
         t - threadIdx.y < rows; t += gridDim.x * static_cast<int64_t>(blockDim.y)) {
        // (whole waves walk on together: their lanes meet in the group maximum)
        const bool in = t < rows;
        for (int64_t v0 = blockIdx.y * static_cast<int64_t>(blockDim.x * VPT); v0 < vecs;
             v0 += gridDim.y * static_cast<int64_t>(blockDim.x * VPT)) {
            Raw8<T> r[VPT];
            unsigned int top[VPT];
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int64_t j = (v0 + threadIdx.x + i * blockDim.x) * 8;
                r[i].load(x + t * d + j, in ? count8(d, j) : 0);
            }
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                float f[8];
                r[i].get(f);
                top[i] = 0u;
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    const unsigned int b = abs_bits(f[q]);
                    top[i] = top[i] > b ? top[i] : b;
                }
            }
            lanes_max(top, lanes);
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int64_t v = v0 + threadIdx.x + i * blockDim.x;
                if (!in || v >= vecs)
                    continue;
                const float s = fourbit_scale(top[i]);
                if ((v & (lanes - 1)) == 0)
                    scale[t * groups + (v >> shift)] = static_cast<uint16_t>(__float_as_uint(s) >> 16);
                float f[8];
                r[i].get(f);
                const unsigned int c = to_codes<T>(f, s, inverse_scale(s));
                __builtin_nontemporal_store(c, reinterpret_cast<unsigned int *>(codes) + t * vecs + v);
            }
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(THREADS)
    dequantize_fourbit_kernel(const uint8_t *codes, const uint16_t *scale, int64_t rows, int64_t d,
                              int64_t groups, int group, T *out)
{
    const int lanes = group / 8, shift = 31 - __clz(lanes);
    const int64_t row_vecs = groups * lanes, vecs = (d + 7) / 8;
    for (int64_t t = blockIdx.x * static_cast<int64_t>(blockDim.y) + threadIdx.y; t < rows;
         t += gridDim.x * static_cast<int64_t>(blockDim.y)) {
        for (int64_t v0 = blockIdx.y * static_cast<int64_t>(blockDim.x * VPT) + threadIdx.x; v0 < vecs;
             v0 += gridDim.y * static_cast<int64_t>(blockDim.x * VPT)) {
            unsigned int c[VPT];
            uint16_t s[VPT];
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int64_t v = v0 + i * blockDim.x;
                const bool in = v < vecs;
                c[i] = in ? __builtin_nontemporal_load(reinterpret_cast<const unsigned int *>(codes) +
                                                       t * row_vecs + v)
                          : 0u;
                s[i] = in ? scale[t * groups + (v >> shift)] : 0;
            }
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int64_t v = v0 + i * blockDim.x;
                const float by = __uint_as_float(static_cast<unsigned int>(s[i]) << 16);
                const auto a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[i], 1.f, 0);
                const auto b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[i], 1.f, 1);
                const auto e = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[i], 1.f, 2);
                const auto g = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[i], 1.f, 3);
                const float f[8] = {a[0] * by, a[1] * by, b[0] * by, b[1] * by,
                                    e[0] * by, e[1] * by, g[0] * by, g[1] * by};
                Raw8<T> o;
                o.set(f);
                o.store(out + t * d + v * 8, count8(d, v * 8));
            }
        }
    }
}

// out[m, n] = sum_z part[z, m, n], in order, rounded once; rows of `out` ldo apart.
template <typename T>
__global__ void __launch_bounds__(THREADS)
    sum_splits_kernel(const float *part, int splits, int64_t M, int64_t N, T *out, int64_t ldo)
{
    const int64_t vecs = (N + 7) / 8, total = vecs * M;
    for (int64_t i = blockIdx.x * static_cast<int64_t>(THREADS) + threadIdx.x; i < total;
         i += gridDim.x * static_cast<int64_t>(THREADS)) {
        const int64_t m = i / vecs, n = i % vecs * 8;
        const int cnt = count8(N, n);
        float acc[8];
#pragma unroll
        for (int q = 0; q < 8; ++q)
            acc[q] = 0.f;
#pragma unroll 4
        for (int z = 0; z < splits; ++z) {
            Raw8<float> r;
            r.load(part + (z * M + m) * N + n, cnt);
            float f[8];
            r.get(f);
#pragma unroll
            for (int q = 0; q < 8; ++q)
                acc[q] += f[q];
        }
        Raw8<T> o;
        o.set(acc);
        o.store(out + m * ldo + n, cnt);
    }
}

}  // namespace

hipError_t launch_quantize_fourbit(int bf16, const void *x, int64_t rows, int64_t d, int group,
                                   uint8_t *codes, uint16_t *scale, hipStream_t st)
{
    if (rows == 0)
        return hipSuccess;
    const int64_t groups = (d + group - 1) / group;
    const Shape s = shape_of(rows, groups * (group / 8), group / 8);
    const dim3 grid(static_cast<unsigned>(s.groups), s.shares), block(s.along, s.rows);
    if (bf16)
        hipLaunchKernelGGL((quantize_fourbit_kernel<uint16_t>), grid, block, 0, st,
                           static_cast<const uint16_t *>(x), rows, d, groups, group, codes, scale);
    else
        hipLaunchKernelGGL((quantize_fourbit_kernel<float>), grid, block, 0, st,
                           static_cast<const float *>(x), rows, d, groups, group, codes, scale);
    return hipGetLastError();
}

hipError_t launch_dequantize_fourbit(int bf16, const uint8_t *codes, const uint16_t *scale,
                                     int64_t rows, int64_t d, int group, void *out, hipStream_t st)
{
    if (rows == 0)
        return hipSuccess;
    const int64_t groups = (d + group - 1) / group;
    const Shape s = shape_of(rows, (d + 7) / 8, 4);
    const dim3 grid(static_cast<unsigned>(s.groups), s.shares), block(s.along, s.rows);
    if (bf16)
        hipLaunchKernelGGL((dequantize_fourbit_kernel<uint16_t>), grid, block, 0, st, codes, scale,
                           rows, d, groups, group, static_cast<uint16_t *>(out));
    else
        hipLaunchKernelGGL((dequantize_fourbit_kernel<float>), grid, block, 0, st, codes, scale, rows,
                           d, groups, group, static_cast<float *>(out));
    return hipGetLastError();
}

hipError_t launch_sum_splits(int bf16, const float *part, int splits, int64_t M, int64_t N, void *out,
                             int64_t ldo, hipStream_t st)
{
    const int64_t groups = ((N + 7) / 8 * M + THREADS - 1) / THREADS;
    const dim3 grid(static_cast<unsigned>(groups < (1 << 20) ? groups : 1 << 20));
    if (bf16)
        hipLaunchKernelGGL((sum_splits_kernel<uint16_t>), grid, dim3(THREADS), 0, st, part, splits, M,
                           N, static_cast<uint16_t *>(out), ldo);
    else
        hipLaunchKernelGGL((sum_splits_kernel<float>), grid, dim3(THREADS), 0, st, part, splits, M, N,
                           static_cast<float *>(out), ldo);
    return hipGetLastError();
}

}  // namespace dora
