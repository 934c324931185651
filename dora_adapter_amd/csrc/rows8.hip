// rows8.hip - the row kernels around a DoRA module (gfx950):
//
//   rmsnorm     h = x + residual, y = w h / sqrt(mean(h^2) + eps), with y in
//               the element type, in the 8-bit form, or both
//   its gradient
//   quantize    rows to the 8-bit form, and back
//
// All are bound by memory traffic.  A workgroup takes whole rows, a thread
// eight consecutive columns at a time (16 bytes of bf16).
#include "dora_internal.hpp"
#include "rows8.hpp"

namespace dora {
namespace {

constexpr int ROW_THREADS = 256;
constexpr int ROW_WAVES = ROW_THREADS / 64;
constexpr int64_t MAX_ROW_GROUPS = 1 << 20;  // workgroups of a row launch

__device__ __forceinline__ int count8(int64_t d, int64_t j)
{
    return d - j < 8 ? static_cast<int>(d - j > 0 ? d - j : 0) : 8;
}

// h of eight columns: x + residual summed in fp32 and rounded to the element
// type, because that is what the residual stream keeps and what the backward
// pass reads (the norm is then a function of the stored h).
template <typename T>
__device__ __forceinline__ Raw8<T> load_h(const NormArgs &a, int64_t at, int cnt)
{
    Raw8<T> x;
    x.load(static_cast<const T *>(a.x) + at, cnt);
    if (a.res != nullptr) {
        Raw8<T> r;
        r.load(static_cast<const T *>(a.res) + at, cnt);
        float u[8], v[8];
        x.get(u);
        r.get(v);
#pragma unroll
        for (int q = 0; q < 8; ++q)
            u[q] += v[q];
        x.set(u);
    }
    return x;
}

// y of eight columns (zero past the row's end).
template <typename T>
__device__ __forceinline__ void norm_y(const Raw8<T> &h, const T *w, int cnt, float rstd,
                                       float (&y)[8])
{
    Raw8<T> wr;
    wr.load(w, cnt);
    float hv[8], wv[8];
    h.get(hv);
    wr.get(wv);
#pragma unroll
    for (int q = 0; q < 8; ++q)
        y[q] = hv[q] * rstd * wv[q];
}

__device__ __forceinline__ unsigned int top8(const float (&v)[8])
{
    unsigned int t = 0u;
#pragma unroll
    for (int q = 0; q < 8; ++q) {
        const unsigned int b = abs_bits(v[q]);
        t = t > b ? t : b;
    }
    return t;
}

// Rows of any width: every pass reads the row again.  A thread meets the same
// columns in each pass and writes them only in the last, so that h may be x
// or the residual, and y may be x.
template <typename T>
__global__ void __launch_bounds__(ROW_THREADS) rmsnorm_kernel(NormArgs a)
{
    __shared__ float red[ROW_WAVES];
    __shared__ unsigned int redu[ROW_WAVES];
    const int64_t groups = a.group ? (a.d + a.group - 1) / a.group : 1;
    const int lanes = a.group / 8;
    // whole waves walk the row together (their lanes meet in the group maximum)
    const int64_t vecs = ((a.d + 7) / 8 + 63) / 64 * 64;
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        const int64_t row = t * a.d;
        float ss = 0.f;
        for (int64_t v = threadIdx.x; v < vecs; v += ROW_THREADS) {
            const int cnt = count8(a.d, v * 8);
            const Raw8<T> h = load_h<T>(a, row + v * 8, cnt);
            float f[8];
            h.get(f);
#pragma unroll
            for (int q = 0; q < 8; ++q)
                ss = __fmaf_rn(f[q], f[q], ss);
        }
        ss = block_sum<ROW_WAVES>(ss, red);
        const float rstd = 1.f / sqrtf(ss / static_cast<float>(a.d) + a.eps);
        if (a.rstd != nullptr && threadIdx.x == 0)
            a.rstd[t] = rstd;
        float s = 0.f;
        if (a.q != nullptr && a.group == 0) {
            unsigned int top = 0u;
            for (int64_t v = threadIdx.x; v < vecs; v += ROW_THREADS) {
                const int cnt = count8(a.d, v * 8);
                const Raw8<T> h = load_h<T>(a, row + v * 8, cnt);
                float y[8];
                norm_y<T>(h, static_cast<const T *>(a.w) + v * 8, cnt, rstd, y);
                const unsigned int b = top8(y);
                top = top > b ? top : b;
            }
            s = scale_of(block_max<ROW_WAVES>(top, redu));
            if (threadIdx.x == 0)
                a.scale[t] = s;
        }
        for (int64_t v = threadIdx.x; v < vecs; v += ROW_THREADS) {
            const int cnt = count8(a.d, v * 8);
            const Raw8<T> h = load_h<T>(a, row + v * 8, cnt);
            float y[8];
            norm_y<T>(h, static_cast<const T *>(a.w) + v * 8, cnt, rstd, y);
            if (a.h != nullptr)
                h.store(static_cast<T *>(a.h) + row + v * 8, cnt);
            if (a.y != nullptr) {
                Raw8<T> o;
                o.set(y);
                o.store(static_cast<T *>(a.y) + row + v * 8, cnt);
            }
            if (a.q != nullptr) {
                if (a.group != 0) {
                    s = scale_of(lanes_max(top8(y), lanes));
                    if (v % lanes == 0 && v / lanes < groups)
                        a.scale[t * groups + v / lanes] = s;
                }
                quantize8(y, s, inverse_scale(s)).store(a.q + row + v * 8, cnt);
            }
        }
    }
}

// The gradient with respect to h:
//   dx = dres + rstd (w dy) - h rstd^3 / d * sum_j w_j dy_j h_j
// (dres: the gradient that reaches h along the residual stream).  dx may be
// dres.
template <typename T>
__global__ void __launch_bounds__(ROW_THREADS) rmsnorm_dx_kernel(NormGradArgs a)
{
    __shared__ float red[ROW_WAVES];
    const T *w = static_cast<const T *>(a.w);
    const int64_t vecs = (a.d + 7) / 8;
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        const int64_t row = t * a.d;
        float dot = 0.f;
        for (int64_t v = threadIdx.x; v < vecs; v += ROW_THREADS) {
            const int cnt = count8(a.d, v * 8);
            Raw8<T> hr, gr, wr;
            hr.load(static_cast<const T *>(a.h) + row + v * 8, cnt);
            gr.load(static_cast<const T *>(a.dy) + row + v * 8, cnt);
            wr.load(w + v * 8, cnt);
            float h[8], g[8], wv[8];
            hr.get(h);
            gr.get(g);
            wr.get(wv);
#pragma unroll
            for (int q = 0; q < 8; ++q)
                dot = __fmaf_rn(wv[q] * g[q], h[q], dot);
        }
        dot = block_sum<ROW_WAVES>(dot, red);
        const float rstd = a.rstd[t];
        const float c = -(dot / static_cast<float>(a.d)) * rstd * rstd * rstd;
        for (int64_t v = threadIdx.x; v < vecs; v += ROW_THREADS) {
            const int cnt = count8(a.d, v * 8);
            Raw8<T> hr, gr, wr, rr;
            hr.load(static_cast<const T *>(a.h) + row + v * 8, cnt);
            gr.load(static_cast<const T *>(a.dy) + row + v * 8, cnt);
            wr.load(w + v * 8, cnt);
            float h[8], g[8], wv[8], o[8];
            hr.get(h);
            gr.get(g);
            wr.get(wv);
#pragma unroll
            for (int q = 0; q < 8; ++q)
                o[q] = 0.f;
            if (a.dres != nullptr) {
                rr.load(static_cast<const T *>(a.dres) + row + v * 8, cnt);
                rr.get(o);
            }
#pragma unroll
            for (int q = 0; q < 8; ++q)
                o[q] += __fmaf_rn(c, h[q], rstd * (wv[q] * g[q]));
            rr.set(o);
            rr.store(static_cast<T *>(a.dx) + row + v * 8, cnt);
        }
    }
}

// dw_j = sum_t dy_tj h_tj rstd_t: workgroup (i, p) sums rows p, p + P, ... of
// its 2048 columns; the finish adds the P partial sums in order.
template <typename T>
__global__ void __launch_bounds__(ROW_THREADS) rmsnorm_dw_kernel(NormGradArgs a)
{
    const int64_t j = (static_cast<int64_t>(blockIdx.x) * ROW_THREADS + threadIdx.x) * 8;
    if (j >= a.d)
        return;
    const int cnt = count8(a.d, j);
    float acc[8];
#pragma unroll
    for (int q = 0; q < 8; ++q)
        acc[q] = 0.f;
    for (int64_t t = blockIdx.y; t < a.T; t += a.parts) {
        Raw8<T> hr, gr;
        hr.load(static_cast<const T *>(a.h) + t * a.d + j, cnt);
        gr.load(static_cast<const T *>(a.dy) + t * a.d + j, cnt);
        float h[8], g[8];
        hr.get(h);
        gr.get(g);
        const float rstd = a.rstd[t];
#pragma unroll
        for (int q = 0; q < 8; ++q)
            acc[q] = __fmaf_rn(g[q], h[q] * rstd, acc[q]);
    }
    for (int q = 0; q < cnt; ++q)
        a.dw_part[static_cast<int64_t>(blockIdx.y) * a.d + j + q] = acc[q];
}

__global__ void __launch_bounds__(ROW_THREADS) sum_parts_kernel(const float *__restrict__ part,
                                                                int parts, int64_t d,
                                                                float *__restrict__ out)
{
    const int64_t j = static_cast<int64_t>(blockIdx.x) * ROW_THREADS + threadIdx.x;
    if (j >= d)
        return;
    float acc = 0.f;
    for (int p = 0; p < parts; ++p)
        acc += part[static_cast<int64_t>(p) * d + j];
    out[j] = acc;
}

template <typename T>
__global__ void __launch_bounds__(ROW_THREADS) quantize_kernel(const T *x, int64_t rows, int64_t d,
                                                               int group, int8_t *q, float *scale)
{
    __shared__ unsigned int redu[ROW_WAVES];
    const int64_t groups = group ? (d + group - 1) / group : 1;
    const int lanes = group / 8;
    const int64_t vecs = ((d + 7) / 8 + 63) / 64 * 64;
    for (int64_t t = blockIdx.x; t < rows; t += gridDim.x) {
        const int64_t row = t * d;
        float s = 0.f;
        if (group == 0) {
            unsigned int top = 0u;
            for (int64_t v = threadIdx.x; v < vecs; v += ROW_THREADS) {
                Raw8<T> r;
                r.load(x + row + v * 8, count8(d, v * 8));
                float f[8];
                r.get(f);
                const unsigned int b = top8(f);
                top = top > b ? top : b;
            }
            s = scale_of(block_max<ROW_WAVES>(top, redu));
            if (threadIdx.x == 0)
                scale[t] = s;
        }
        for (int64_t v = threadIdx.x; v < vecs; v += ROW_THREADS) {
            const int cnt = count8(d, v * 8);
            Raw8<T> r;
            r.load(x + row + v * 8, cnt);
            float f[8];
            r.get(f);
            if (group != 0) {
                s = scale_of(lanes_max(top8(f), lanes));
                if (v % lanes == 0 && v / lanes < groups)
                    scale[t * groups + v / lanes] = s;
            }
            quantize8(f, s, inverse_scale(s)).store(q + row + v * 8, cnt);
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(ROW_THREADS) dequantize_kernel(const int8_t *q,
                                                                 const float *scale, int64_t rows,
                                                                 int64_t d, int group, T *out)
{
    const int64_t groups = group ? (d + group - 1) / group : 1;
    const int64_t vecs = (d + 7) / 8;
    for (int64_t t = blockIdx.x; t < rows; t += gridDim.x) {
        for (int64_t v = threadIdx.x; v < vecs; v += ROW_THREADS) {
            const int cnt = count8(d, v * 8);
            Raw8i r;
            r.load(q + t * d + v * 8, cnt);
            const float s = scale[t * groups + (group ? v * 8 / group : 0)];
            float f[8];
#pragma unroll
            for (int k = 0; k < 8; ++k)
                f[k] = r.value(k) * s;
            Raw8<T> o;
            o.set(f);
            o.store(out + t * d + v * 8, cnt);
        }
    }
}

// dh = g dy and dm partial sums, as the pass over a stored y makes them: thread
// (column group c, first row t0) sums dy (q scale) over rows t0, t0 + R, ...
template <typename T>
__global__ void __launch_bounds__(ROW_THREADS)
    dh_dm_rows8_kernel(const T *__restrict__ dy, const int8_t *__restrict__ yq,
                       const float *__restrict__ ys, int group, const float *__restrict__ m,
                       const float *__restrict__ n, int64_t Tn, int64_t d, int64_t R,
                       T *__restrict__ dh, float *__restrict__ dm_part)
{
    const int64_t gpr = (d + 7) / 8;
    const int64_t gi = static_cast<int64_t>(blockIdx.x) * ROW_THREADS + threadIdx.x;
    const int64_t c = gi % gpr, t0 = gi / gpr;
    if (t0 >= R)
        return;
    const int64_t i0 = c * 8;
    const int cnt = count8(d, i0);
    const int64_t groups = group ? (d + group - 1) / group : 1;
    const int64_t gc = group ? i0 / group : 0;
    float g[8], acc[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) {
        g[q] = q < cnt ? m[i0 + q] / n[i0 + q] : 0.f;
        acc[q] = 0.f;
    }
    for (int64_t t = t0; t < Tn; t += R) {
        const int64_t off = t * d + i0;
        Raw8<T> ar, o;
        Raw8i b;
        ar.load(dy + off, cnt);
        b.load(yq + off, cnt);
        const float s = ys[t * groups + gc];
        float a[8], h[8];
        ar.get(a);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            h[q] = g[q] * a[q];
            acc[q] = __fmaf_rn(a[q], b.value(q) * s, acc[q]);
        }
        o.set(h);
        o.store(dh + off, cnt);
    }
    for (int q = 0; q < cnt; ++q)
        dm_part[t0 * d + i0 + q] = acc[q];
}

unsigned row_groups(int64_t rows)
{
    return static_cast<unsigned>(rows < MAX_ROW_GROUPS ? rows : MAX_ROW_GROUPS);
}

}  // namespace

int rmsnorm_parts(int64_t T, int64_t d)
{
    // about 2048 workgroups over column blocks and row shares, 16 rows each
    // at least
    const int64_t blocks = ((d + 7) / 8 + ROW_THREADS - 1) / ROW_THREADS;
    int64_t p = 2048 / blocks;
    p = p < (T + 15) / 16 ? p : (T + 15) / 16;
    return static_cast<int>(p < 1 ? 1 : (p > 512 ? 512 : p));
}

hipError_t launch_rmsnorm(int bf16, const NormArgs &a, hipStream_t st)
{
    if (a.T == 0)
        return hipSuccess;
    const dim3 grid(row_groups(a.T)), block(ROW_THREADS);
    if (bf16)
        hipLaunchKernelGGL((rmsnorm_kernel<uint16_t>), grid, block, 0, st, a);
    else
        hipLaunchKernelGGL((rmsnorm_kernel<float>), grid, block, 0, st, a);
    return hipGetLastError();
}

hipError_t launch_rmsnorm_grad(int bf16, const NormGradArgs &a, float *dw, hipStream_t st)
{
    const dim3 block(ROW_THREADS);
    const unsigned cols = static_cast<unsigned>(((a.d + 7) / 8 + ROW_THREADS - 1) / ROW_THREADS);
    if (a.T > 0) {
        const dim3 rows(row_groups(a.T));
        if (bf16)
            hipLaunchKernelGGL((rmsnorm_dx_kernel<uint16_t>), rows, block, 0, st, a);
        else
            hipLaunchKernelGGL((rmsnorm_dx_kernel<float>), rows, block, 0, st, a);
    }
    if (dw != nullptr) {
        // (T = 0: the partial sums are zeros)
        const dim3 grid(cols, static_cast<unsigned>(a.parts));
        if (bf16)
            hipLaunchKernelGGL((rmsnorm_dw_kernel<uint16_t>), grid, block, 0, st, a);
        else
            hipLaunchKernelGGL((rmsnorm_dw_kernel<float>), grid, block, 0, st, a);
        hipLaunchKernelGGL(sum_parts_kernel,
                           dim3(static_cast<unsigned>((a.d + ROW_THREADS - 1) / ROW_THREADS)), block,
                           0, st, a.dw_part, a.parts, a.d, dw);
    }
    return hipGetLastError();
}

hipError_t launch_quantize_rows(int bf16, const void *x, int64_t rows, int64_t d, int group,
                                int8_t *q, float *scale, hipStream_t st)
{
    if (rows == 0)
        return hipSuccess;
    const dim3 grid(row_groups(rows)), block(ROW_THREADS);
    if (bf16)
        hipLaunchKernelGGL((quantize_kernel<uint16_t>), grid, block, 0, st,
                           static_cast<const uint16_t *>(x), rows, d, group, q, scale);
    else
        hipLaunchKernelGGL((quantize_kernel<float>), grid, block, 0, st,
                           static_cast<const float *>(x), rows, d, group, q, scale);
    return hipGetLastError();
}

hipError_t launch_dequantize_rows(int bf16, const int8_t *q, const float *scale, int64_t rows,
                                  int64_t d, int group, void *out, hipStream_t st)
{
    if (rows == 0)
        return hipSuccess;
    const dim3 grid(row_groups(rows)), block(ROW_THREADS);
    if (bf16)
        hipLaunchKernelGGL((dequantize_kernel<uint16_t>), grid, block, 0, st, q, scale, rows, d,
                           group, static_cast<uint16_t *>(out));
    else
        hipLaunchKernelGGL((dequantize_kernel<float>), grid, block, 0, st, q, scale, rows, d, group,
                           static_cast<float *>(out));
    return hipGetLastError();
}

hipError_t launch_dh_dm_rows8(int bf16, const void *dy, const int8_t *yq, const float *ys,
                              int group, const float *m, const float *n, int64_t T, int64_t d_out,
                              int64_t sweep, void *dh, float *dm_part, hipStream_t st)
{
    if (T == 0)
        return hipSuccess;
    const int64_t threads = (d_out + 7) / 8 * sweep;
    const dim3 grid(static_cast<unsigned>((threads + ROW_THREADS - 1) / ROW_THREADS));
    if (bf16)
        hipLaunchKernelGGL((dh_dm_rows8_kernel<uint16_t>), grid, dim3(ROW_THREADS), 0, st,
                           static_cast<const uint16_t *>(dy), yq, ys, group, m, n, T, d_out, sweep,
                           static_cast<uint16_t *>(dh), dm_part);
    else
        hipLaunchKernelGGL((dh_dm_rows8_kernel<float>), grid, dim3(ROW_THREADS), 0, st,
                           static_cast<const float *>(dy), yq, ys, group, m, n, T, d_out, sweep,
                           static_cast<float *>(dh), dm_part);
    return hipGetLastError();
}

}  // namespace dora
