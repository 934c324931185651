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
    wr.template load<true>(w, cnt);
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

// The 8-bit form of row t, held as VPT vectors a thread (zeros past its end):
// thread i holds the vectors k0 + i, k0 + i + threads, ... (k0 a multiple of
// 64; 0 where the row has one scale); value(i, v) gives its i-th.
template <int VPT, typename F>
__device__ __forceinline__ void quantize_held(F &&value, int k0, int d, int group, int64_t t,
                                              int8_t *q, float *scale, unsigned int *redu)
{
    const int threads = static_cast<int>(blockDim.x);
    unsigned int top[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        float v[8];
        value(i, v);
        top[i] = top8(v);
    }
    float s = 0.f, inv = 0.f;
    const int lanes = group / 8, shift = 31 - __clz(lanes | 1);
    const int groups = group ? (d + group - 1) / group : 1;
    if (group == 0) {
        unsigned int all = top[0];
#pragma unroll
        for (int i = 1; i < VPT; ++i)
            all = all > top[i] ? all : top[i];
        s = scale_of(block_max(all, redu, threads >> 6));
        inv = inverse_scale(s);
        if (threadIdx.x == 0)
            scale[t] = s;
    } else {
        lanes_max(top, lanes);
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int k = k0 + static_cast<int>(threadIdx.x) + i * threads;
        if (group != 0) {
            s = scale_of(top[i]);
            inv = inverse_scale(s);
            if ((k & (lanes - 1)) == 0 && (k >> shift) < groups)
                scale[t * groups + (k >> shift)] = s;
        }
        float v[8];
        value(i, v);
        quantize8(v, s, inv).store(q + t * d + k * 8, count8(d, k * 8));
    }
}

// 1 / sqrt(ss / d + eps) of a row whose squares sum to ss (the same in every thread).
// The squares leave fp32's range long before h and rstd do (overflow from 2^64 on,
// lost bits below 2^-50 where eps is as small): such a row's are summed again, of
// k h with a power of two k that puts them inside (every |h| < 2^128, d < 2^31: k h to
// 2^48; the mean below 2^-100: k h to 2^56, denormal h from 2^-59 on), and the root
// gets it back.  rstd is a number for rows whose root mean square lies from 2^-127 to
// the largest value (denormal from 2^126 on).
template <typename F>
__device__ __forceinline__ float rstd_of(float ss, float d, float eps, F &&sum_squares_of)
{
    const float ms = ss / d + eps;
    if (ms >= 0x1p-100f && ms < __builtin_inff())
        return 1.f / sqrtf(ms);
    const float k = ms > 1.f ? 0x1p-80f : 0x1p90f;
    return k / sqrtf(sum_squares_of(k) / d + eps * k * k);
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
        auto sum_squares = [&](float k) {
            float ss = 0.f;
            for (int64_t v = threadIdx.x; v < vecs; v += ROW_THREADS) {
                const int cnt = count8(a.d, v * 8);
                const Raw8<T> h = load_h<T>(a, row + v * 8, cnt);
                float f[8];
                h.get(f);
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    ss = __fmaf_rn(k * f[q], k * f[q], ss);
            }
            return block_sum(ss, red, ROW_WAVES);
        };
        const float rstd = rstd_of(sum_squares(1.f), static_cast<float>(a.d), a.eps, sum_squares);
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
            s = scale_of(block_max(top, redu, ROW_WAVES));
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
                    s = scale_of(lane_max(top8(y), lanes));
                    if (v % lanes == 0 && v / lanes < groups)
                        a.scale[t * groups + v / lanes] = s;
                }
                quantize8(y, s, inverse_scale(s)).store(a.q + row + v * 8, cnt);
            }
        }
    }
}

// Rows that fit a workgroup's registers: thread i holds the vectors i, i +
// threads, ... (VPT of them), so x, the residual and w are read once (w before
// the first reduction, whose wait covers it) and everything is written once.
// h goes out as soon as it is formed.
template <typename T, int VPT>
__global__ void __launch_bounds__(1024) rmsnorm_held_kernel(NormArgs a)
{
    __shared__ float red[16];
    __shared__ unsigned int redu[16];
    const int threads = static_cast<int>(blockDim.x), waves = threads >> 6;
    const int d = static_cast<int>(a.d);
    const int64_t row = static_cast<int64_t>(blockIdx.x) * a.d;
    Raw8<T> h[VPT], w[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int j = (static_cast<int>(threadIdx.x) + i * threads) * 8;
        h[i] = load_h<T>(a, row + j, count8(d, j));
    }
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int j = (static_cast<int>(threadIdx.x) + i * threads) * 8;
        w[i].template load<true>(static_cast<const T *>(a.w) + j, count8(d, j));
        if (a.h != nullptr)
            h[i].store(static_cast<T *>(a.h) + row + j, count8(d, j));
        float f[8];
        h[i].get(f);
#pragma unroll
        for (int q = 0; q < 8; ++q)
            ss = __fmaf_rn(f[q], f[q], ss);
    }
    ss = block_sum(ss, red, waves);
    const float rstd = rstd_of(ss, static_cast<float>(d), a.eps, [&](float k) {
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            float f[8];
            h[i].get(f);
#pragma unroll
            for (int q = 0; q < 8; ++q)
                sum = __fmaf_rn(k * f[q], k * f[q], sum);
        }
        return block_sum(sum, red, waves);
    });
    if (a.rstd != nullptr && threadIdx.x == 0)
        a.rstd[blockIdx.x] = rstd;
    auto value = [&](int i, float (&y)[8]) {
        float wv[8];
        h[i].get(y);
        w[i].get(wv);
#pragma unroll
        for (int q = 0; q < 8; ++q)
            y[q] = y[q] * rstd * wv[q];
    };
    if (a.y != nullptr) {
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int j = (static_cast<int>(threadIdx.x) + i * threads) * 8;
            float y[8];
            value(i, y);
            Raw8<T> o;
            o.set(y);
            o.store(static_cast<T *>(a.y) + row + j, count8(d, j));
        }
    }
    if (a.q != nullptr)
        quantize_held<VPT>(value, 0, d, a.group, blockIdx.x, a.q, a.scale, redu);
}

// The gradient with respect to h:
//   dx = dres + rstd (w dy - hat * mean_j(w_j dy_j hat_j)),  hat = h rstd
// (dres: the gradient that reaches h along the residual stream).  dx may be
// dres.  Every h meets rstd first: hat is of the order of one, where sums of
// w dy h, and rstd^3, leave fp32's range for rows of 2^-43 or 2^43 already.
template <typename T>
__global__ void __launch_bounds__(ROW_THREADS) rmsnorm_dx_kernel(NormGradArgs a)
{
    __shared__ float red[ROW_WAVES];
    const T *w = static_cast<const T *>(a.w);
    const int64_t vecs = (a.d + 7) / 8;
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        const int64_t row = t * a.d;
        const float rstd = a.rstd[t];
        float dot = 0.f;
        for (int64_t v = threadIdx.x; v < vecs; v += ROW_THREADS) {
            const int cnt = count8(a.d, v * 8);
            Raw8<T> hr, gr, wr;
            hr.load(static_cast<const T *>(a.h) + row + v * 8, cnt);
            gr.load(static_cast<const T *>(a.dy) + row + v * 8, cnt);
            wr.template load<true>(w + v * 8, cnt);
            float h[8], g[8], wv[8];
            hr.get(h);
            gr.get(g);
            wr.get(wv);
#pragma unroll
            for (int q = 0; q < 8; ++q)
                dot = __fmaf_rn(wv[q] * g[q], h[q] * rstd, dot);
        }
        const float mean = block_sum(dot, red, ROW_WAVES) / static_cast<float>(a.d);
        for (int64_t v = threadIdx.x; v < vecs; v += ROW_THREADS) {
            const int cnt = count8(a.d, v * 8);
            Raw8<T> hr, gr, wr, rr;
            hr.load(static_cast<const T *>(a.h) + row + v * 8, cnt);
            gr.load(static_cast<const T *>(a.dy) + row + v * 8, cnt);
            wr.template load<true>(w + v * 8, cnt);
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
                o[q] += rstd * __fmaf_rn(-mean, h[q] * rstd, wv[q] * g[q]);
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

// dx and dw in one pass over dy, h and dres, for rows that fit a workgroup's
// registers: workgroup b takes rows b, b + parts, ...; a thread keeps its
// columns' w and running dw.  PRE: the next row's loads go out before this
// row's reduction, and cover it.
// LDW: the running dw in LDS (four floats a thread and half vector, dynamic,
// 32 VPT bytes a thread) where the registers have no room for it.
template <typename T, int VPT, bool PRE, bool LDW>
__global__ void __launch_bounds__(1024) rmsnorm_grad_held_kernel(NormGradArgs a)
{
    extern __shared__ __align__(16) float4 ldw[];
    __shared__ float red[2][16];
    const int threads = static_cast<int>(blockDim.x), waves = threads >> 6;
    const int d = static_cast<int>(a.d);
    // column col(i) of a row that starts at `base`: a scalar base and a 32-bit
    // offset (one register for all arrays, not two for each)
    auto in_row = [](auto *base, unsigned int c) {
        using P = decltype(base);
        using B = std::conditional_t<std::is_const_v<std::remove_pointer_t<P>>, const char *, char *>;
        return reinterpret_cast<P>(reinterpret_cast<B>(base) + c * static_cast<unsigned int>(sizeof(T)));
    };
    const float inv_d = 1.f / static_cast<float>(d);
    const bool with_res = a.dres != nullptr;
    auto col = [&](int i) { return (threadIdx.x + i * blockDim.x) * 8u; };
    Raw8<T> w[VPT];
    float dw[LDW ? 1 : VPT][8];
    auto place = [&](int i, int half) -> float4 & {
        return ldw[(2 * i + half) * threads + static_cast<int>(threadIdx.x)];
    };
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        w[i].template load<true>(in_row(static_cast<const T *>(a.w), col(i)), count8(d, col(i)));
        if constexpr (LDW) {
            place(i, 0) = place(i, 1) = make_float4(0.f, 0.f, 0.f, 0.f);
        } else {
#pragma unroll
            for (int q = 0; q < 8; ++q)
                dw[i][q] = 0.f;
        }
    }
    struct Row {
        Raw8<T> h[VPT], g[VPT], r[VPT];
        float rstd;
    };
    auto fetch = [&](Row &o, int64_t t) {
        const int64_t at = t * a.d;
        o.rstd = a.rstd[t];
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int cnt = count8(d, col(i));
            o.h[i].load(in_row(static_cast<const T *>(a.h) + at, col(i)), cnt);
            o.g[i].load(in_row(static_cast<const T *>(a.dy) + at, col(i)), cnt);
            if (with_res)
                o.r[i].load(in_row(static_cast<const T *>(a.dres) + at, col(i)), cnt);
        }
    };
    Row cur, nxt;
    int64_t t = blockIdx.x;
    if (t < a.T)
        fetch(cur, t);
    for (int par = 0; t < a.T; par ^= 1) {
        const int64_t tn = t + gridDim.x;
        float dot = 0.f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            float h[8], g[8], wv[8];
            cur.h[i].get(h);
            cur.g[i].get(g);
            w[i].get(wv);
#pragma unroll
            for (int q = 0; q < 8; ++q)
                dot = __fmaf_rn(wv[q] * g[q], h[q] * cur.rstd, dot);
            __builtin_amdgcn_sched_barrier(0);
        }
        if (PRE && tn < a.T)
            fetch(nxt, tn);
        dot = wave_sum(dot);
        if (waves > 1) {
            // one barrier a row: the next row writes the other half of `red`
            if ((threadIdx.x & 63) == 0)
                red[par][threadIdx.x >> 6] = dot;
            __syncthreads();
            dot = red[par][0];
            for (int k = 1; k < waves; ++k)
                dot += red[par][k];
        }
        const float mean = dot * inv_d;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            // (what the dot product made of them would not leave the registers else)
            forget(cur.h[i]);
            forget(cur.g[i]);
            float h[8], g[8], wv[8], o[8];
            cur.h[i].get(h);
            cur.g[i].get(g);
            w[i].get(wv);
            if (with_res) {
                cur.r[i].get(o);
            } else {
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    o[q] = 0.f;
            }
#pragma unroll
            for (int q = 0; q < 8; ++q)
                o[q] += cur.rstd * __fmaf_rn(-mean, h[q] * cur.rstd, wv[q] * g[q]);
            if constexpr (LDW) {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    float4 p = place(i, k);
                    p.x = __fmaf_rn(g[4 * k], h[4 * k] * cur.rstd, p.x);
                    p.y = __fmaf_rn(g[4 * k + 1], h[4 * k + 1] * cur.rstd, p.y);
                    p.z = __fmaf_rn(g[4 * k + 2], h[4 * k + 2] * cur.rstd, p.z);
                    p.w = __fmaf_rn(g[4 * k + 3], h[4 * k + 3] * cur.rstd, p.w);
                    place(i, k) = p;
                }
            } else {
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    dw[i][q] = __fmaf_rn(g[q], h[q] * cur.rstd, dw[i][q]);
            }
            Raw8<T> out;
            out.set(o);
            out.store(in_row(static_cast<T *>(a.dx) + t * a.d, col(i)), count8(d, col(i)));
            // one vector at a time (left free, the scheduler unpacks them all)
            __builtin_amdgcn_sched_barrier(0);
        }
        t = tn;
        if (PRE)
            cur = nxt;
        else if (t < a.T)
            fetch(cur, t);
    }
    if (a.dw_part != nullptr) {
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int cnt = count8(d, col(i));
            float *p = a.dw_part + static_cast<int64_t>(blockIdx.x) * a.d + col(i);
            if constexpr (LDW) {
                const float4 u = place(i, 0), v = place(i, 1);
                const float o[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    if (q < cnt)
                        p[q] = o[q];
            } else {
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    if (q < cnt)
                        p[q] = dw[i][q];
            }
        }
    }
}

// Sums of `parts` rows, each divided by its column's `over` (or 1): 64 columns a
// workgroup, its 16 waves taking every 16th row each, then the 16 sums in order.
__global__ void __launch_bounds__(1024) sum_parts_kernel(const float *__restrict__ part, int parts,
                                                         int64_t d, const float *__restrict__ over,
                                                         float *__restrict__ out)
{
    __shared__ float sums[16][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int64_t j0 = static_cast<int64_t>(blockIdx.x) * 64; j0 < d;
         j0 += static_cast<int64_t>(gridDim.x) * 64) {
        const int64_t j = j0 + lane;
        float acc = 0.f;
        if (j < d) {
#pragma unroll 8
            for (int p = wave; p < parts; p += 16)
                acc += part[static_cast<int64_t>(p) * d + j];
        }
        __syncthreads();  // the last columns' sums have been read
        sums[wave][lane] = acc;
        __syncthreads();
        if (wave == 0 && j < d) {
            acc = sums[0][lane];
#pragma unroll
            for (int k = 1; k < 16; ++k)
                acc += sums[k][lane];
            out[j] = over != nullptr ? acc / over[j] : acc;
        }
    }
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
            s = scale_of(block_max(top, redu, ROW_WAVES));
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
                s = scale_of(lane_max(top8(f), lanes));
                if (v % lanes == 0 && v / lanes < groups)
                    scale[t * groups + v / lanes] = s;
            }
            quantize8(f, s, inverse_scale(s)).store(q + row + v * 8, cnt);
        }
    }
}

// A row (or, with scales in groups, blockIdx.y's share of one) a workgroup.
template <typename T, int VPT>
__global__ void __launch_bounds__(1024)
    quantize_held_kernel(const T *x, int64_t width, int group, int8_t *q, float *scale)
{
    __shared__ unsigned int redu[16];
    const int d = static_cast<int>(width);
    const int k0 = static_cast<int>(blockIdx.y * blockDim.x) * VPT;
    const T *row = x + static_cast<int64_t>(blockIdx.x) * width;
    Raw8<T> r[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int j = (k0 + static_cast<int>(threadIdx.x + i * blockDim.x)) * 8;
        r[i].load(row + j, count8(d, j));
    }
    quantize_held<VPT>([&](int i, float (&v)[8]) { r[i].get(v); }, k0, d, group, blockIdx.x, q,
                       scale, redu);
}

// Rows blockIdx.x + k gridDim.x, shares (8192 columns) blockIdx.y + k gridDim.y.
template <typename T>
__global__ void __launch_bounds__(ROW_THREADS) dequantize_kernel(const int8_t *q,
                                                                 const float *scale, int64_t rows,
                                                                 int64_t d, int group, T *out)
{
    constexpr int VPT = 4;
    const int64_t groups = group ? (d + group - 1) / group : 1;
    const int shift = group ? 31 - __clz(group) : 63;
    constexpr int SHARE = ROW_THREADS * VPT * 8;
    for (int64_t c = blockIdx.y * static_cast<int64_t>(SHARE); c < d;
         c += gridDim.y * static_cast<int64_t>(SHARE)) {
        for (int64_t t = blockIdx.x; t < rows; t += gridDim.x) {
            const int64_t j0 = c + threadIdx.x * 8;
            Raw8i r[VPT];
            float s[VPT];
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int64_t j = j0 + i * (ROW_THREADS * 8);
                r[i].load(q + t * d + j, count8(d, j));
                s[i] = j < d ? scale[t * groups + (j >> shift)] : 0.f;
            }
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int64_t j = j0 + i * (ROW_THREADS * 8);
                float f[8];
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    f[k] = r[i].value(k) * s[i];
                Raw8<T> o;
                o.set(f);
                o.store(out + t * d + j, count8(d, j));
            }
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

// A launch holds fewer than 2^32 threads.
bool launchable(int64_t groups, int64_t threads) { return groups < (int64_t(1) << 32) / threads; }

// Rows held in registers: vectors a thread and threads a row.  Up to two rows a
// CU: as many threads as the row has vectors, so that one row's latency is
// short; more rows: `most` vectors a thread.  vpt = 0: the row is too long, or
// the rows too many for one launch of a workgroup each.
struct RowShape {
    int vpt, threads;
};
RowShape held_shape(int64_t T, int64_t d, int most)
{
    const int64_t vecs = (d + 7) / 8;
    if (vecs > 4096)
        return {0, 0};
    int vpt = T <= 512 ? 1 : most;
    while (vecs > 1024 * static_cast<int64_t>(vpt))
        vpt *= 2;
    const int64_t threads = ((vecs + vpt - 1) / vpt + 63) / 64 * 64;
    return {launchable(T, threads) ? vpt : 0, static_cast<int>(threads)};
}

template <typename T>
void rmsnorm_launch(const NormArgs &a, hipStream_t st)
{
    // two vectors a thread: 91 us at 8192 x 8192 to int8, against 117 (one) and
    // 100 (four)
    const RowShape s = held_shape(a.T, a.d, 2);
    const dim3 grid(static_cast<unsigned>(a.T)), block(static_cast<unsigned>(s.threads));
    if (s.vpt == 1)
        hipLaunchKernelGGL((rmsnorm_held_kernel<T, 1>), grid, block, 0, st, a);
    else if (s.vpt == 2)
        hipLaunchKernelGGL((rmsnorm_held_kernel<T, 2>), grid, block, 0, st, a);
    else if (s.vpt == 4)
        hipLaunchKernelGGL((rmsnorm_held_kernel<T, 4>), grid, block, 0, st, a);
    else
        hipLaunchKernelGGL((rmsnorm_kernel<T>), dim3(row_groups(a.T)), dim3(ROW_THREADS), 0, st, a);
}

template <typename T>
void quantize_launch(const T *x, int64_t rows, int64_t d, int group, int8_t *q, float *scale,
                     hipStream_t st)
{
    // four vectors a thread: 35 us at 8192 x 8192, against 58 (one) and 40 (two)
    RowShape s = held_shape(rows, d, 4);
    int64_t shares = 1;
    if (group != 0 && d <= (int64_t(1) << 30)) {
        // no reduction over the row: 8192 columns a workgroup (2048 with few rows)
        const int64_t vecs = (d + 7) / 8;
        s.vpt = rows <= 512 ? 1 : 4;
        s.threads = static_cast<int>(vecs < 256 * s.vpt ? ((vecs + s.vpt - 1) / s.vpt + 63) / 64 * 64
                                                       : 256);
        shares = (vecs + s.vpt * s.threads - 1) / (s.vpt * s.threads);
        if (shares > 65535 || !launchable(rows * shares, s.threads))
            s.vpt = 0;
    }
    const dim3 grid(static_cast<unsigned>(rows), static_cast<unsigned>(s.vpt ? shares : 1)),
        block(static_cast<unsigned>(s.threads));
    if (s.vpt == 1)
        hipLaunchKernelGGL((quantize_held_kernel<T, 1>), grid, block, 0, st, x, d, group, q, scale);
    else if (s.vpt == 2)
        hipLaunchKernelGGL((quantize_held_kernel<T, 2>), grid, block, 0, st, x, d, group, q, scale);
    else if (s.vpt == 4)
        hipLaunchKernelGGL((quantize_held_kernel<T, 4>), grid, block, 0, st, x, d, group, q, scale);
    else
        hipLaunchKernelGGL((quantize_kernel<T>), dim3(row_groups(rows)), dim3(ROW_THREADS), 0, st, x,
                           rows, d, group, q, scale);
}

// Rows whose gradient is formed in one pass, held in a workgroup's registers.
bool grad_held(int64_t d, bool wide) { return (d + 7) / 8 <= (wide ? 2048 : 4096); }
}  // namespace

int rmsnorm_parts(int64_t T, int64_t d, int bf16)
{
    const int64_t vecs = (d + 7) / 8;
    int64_t p;
    if (grad_held(d, !bf16)) {
        // a workgroup a CU as soon as there are rows for them, and the shorter the
        // rows the more, of eight rows at least (four of up to 1024 columns).  us
        // with 256, 512, 1024, 2048 workgroups (bf16): 8192 x 8192 94, 101, 110, 128;
        // 16384 x 4096 92, 94, 104, 108; 8192 x 2048 45, 33, 36, 44; 32768 x 1024 131,
        // 78, 53, 58; 32768 x 512 91, 54, 38, 35 (4096: 43); 65536 x 128 381, 229, 128,
        // 77 (4096: 55); 4096 x 768 41, 27, 21, 24
        const int most = vecs > 512 ? 1 : vecs > 128 ? 2 : vecs > 64 ? 4 : vecs > 32 ? 8 : 16;
        const int64_t share = vecs > 128 ? T / 8 : T / 4;
        p = share > 256 ? share : 256;
        p = p < 256 * most ? p : 256 * most;
        p = p < T ? p : T;
    } else {
        // about 2048 workgroups over column blocks and row shares, 16 rows each
        // at least
        p = 2048 / ((vecs + ROW_THREADS - 1) / ROW_THREADS);
        p = p < (T + 15) / 16 ? p : (T + 15) / 16;
    }
    return static_cast<int>(p < 1 ? 1 : p);
}

hipError_t launch_rmsnorm(int bf16, const NormArgs &a, hipStream_t st)
{
    if (a.T == 0)
        return hipSuccess;
    if (bf16)
        rmsnorm_launch<uint16_t>(a, st);
    else
        rmsnorm_launch<float>(a, st);
    return hipGetLastError();
}

hipError_t launch_sum_parts(const float *part, int parts, int64_t d, const float *over, float *out,
                            hipStream_t st)
{
    const int64_t blocks = (d + 63) / 64;
    hipLaunchKernelGGL(sum_parts_kernel, dim3(static_cast<unsigned>(blocks < 65536 ? blocks : 65536)),
                       dim3(1024), 0, st, part, parts, d, over, out);
    return hipGetLastError();
}

namespace {
template <typename T>
hipError_t rmsnorm_grad_launch(NormGradArgs a, float *dw, hipStream_t st)
{
    constexpr bool WIDE = sizeof(T) == 4;
    const int64_t vecs = (a.d + 7) / 8;
    const unsigned parts = static_cast<unsigned>(a.parts);
    float *const part = a.dw_part;
    // one part is the sum itself
    a.dw_part = dw == nullptr ? nullptr : (parts == 1 ? dw : part);
    if (a.T > 0 && grad_held(a.d, WIDE)) {
        // the fewest vectors a thread that 1024 threads allow, two at least
        // where the registers take two rows of them (bf16)
        const int vpt = vecs <= 64 ? 1 : (WIDE && vecs <= 1024 ? 1 : (vecs <= 2048 ? 2 : 4));
        const dim3 grid(parts), block(static_cast<unsigned>(((vecs + vpt - 1) / vpt + 63) / 64 * 64));
        if (vpt == 1)
            hipLaunchKernelGGL((rmsnorm_grad_held_kernel<T, 1, true, false>), grid, block, 0, st, a);
        else if (vpt == 2)
            hipLaunchKernelGGL((rmsnorm_grad_held_kernel<T, 2, !WIDE, false>), grid, block, 0, st, a);
        else if constexpr (!WIDE)
            hipLaunchKernelGGL((rmsnorm_grad_held_kernel<T, 4, false, true>), grid, block,
                               block.x * 4 * 32, st, a);
    } else {
        const dim3 block(ROW_THREADS);
        if (a.T > 0) {
            hipLaunchKernelGGL((rmsnorm_dx_kernel<T>), dim3(row_groups(a.T)), block, 0, st, a);
            const hipError_t e = hipGetLastError();
            if (e != hipSuccess)
                return e;
        }
        // (T = 0: the partial sums are zeros)
        if (dw != nullptr)
            hipLaunchKernelGGL((rmsnorm_dw_kernel<T>),
                               dim3(static_cast<unsigned>((vecs + ROW_THREADS - 1) / ROW_THREADS),
                                    parts),
                               block, 0, st, a);
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || dw == nullptr || parts == 1)
        return e;
    return launch_sum_parts(part, a.parts, a.d, nullptr, dw, st);
}
}  // namespace

hipError_t launch_rmsnorm_grad(int bf16, const NormGradArgs &a, float *dw, hipStream_t st)
{
    return bf16 ? rmsnorm_grad_launch<uint16_t>(a, dw, st) : rmsnorm_grad_launch<float>(a, dw, st);
}

hipError_t launch_quantize_rows(int bf16, const void *x, int64_t rows, int64_t d, int group,
                                int8_t *q, float *scale, hipStream_t st)
{
    if (rows == 0)
        return hipSuccess;
    if (bf16)
        quantize_launch(static_cast<const uint16_t *>(x), rows, d, group, q, scale, st);
    else
        quantize_launch(static_cast<const float *>(x), rows, d, group, q, scale, st);
    return hipGetLastError();
}

hipError_t launch_dequantize_rows(int bf16, const int8_t *q, const float *scale, int64_t rows,
                                  int64_t d, int group, void *out, hipStream_t st)
{
    if (rows == 0)
        return hipSuccess;
    int64_t shares = (d + ROW_THREADS * 32 - 1) / (ROW_THREADS * 32);
    shares = shares < 4096 ? shares : 4096;
    // (2^23 workgroups at most)
    const int64_t groups = (int64_t(1) << 23) / shares;
    const dim3 grid(static_cast<unsigned>(rows < groups ? rows : groups),
                    static_cast<unsigned>(shares)),
        block(ROW_THREADS);
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

int64_t dm_rows8_sweep(int64_t T, int64_t d_out)
{
    // as the pass over a stored y, but at least two rows a thread: one leaves
    // more bytes of partial sums than the pass reads
    const int64_t r = dm_sweep_rows(T, d_out), most = (T + 1) / 2;
    return r < most ? r : most;
}

}  // namespace dora
