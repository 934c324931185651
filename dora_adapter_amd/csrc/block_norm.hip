// block_norm.hip - the norms on both sides of a residual addition (gfx950):
//
//   u = w_post (.) x / rms(x)              the block's output normed (or x itself)
//   h = a residual + b gate (.) u          rounded to the element type, as it is stored
//   y = w_pre (.) h / rms(h)               normed for the block behind it
//
// and the gradients, with hat(v) = v / rms(v) and m1, m2 means over a row's columns:
//
//   dh        = dh_in + (w_pre dy - m1 hat(h)) / rms(h),   m1 = mean(w_pre dy hat(h))
//   dresidual = a dh,  db = b dh,  dgate = sum db u,  du = gate db
//   dx        = (w_post du - m2 hat(x)) / rms(x),          m2 = mean(w_post du hat(x))
//   dw_pre    = sum dy hat(h),  dw_post = sum du hat(x)
//
// Both are bound by memory traffic: two matrices in and two out forward, four in and two out
// backward, each once.  A workgroup takes whole rows, a thread eight consecutive columns at a
// time (16 bytes of bf16).  8192 x 8192 in bf16: 94 us forward (5.7 TB/s), 145 + 10 backward (5.7).
#include "around.hpp"
#include "rows8.hpp"

namespace dora {
namespace {

typedef float f32x4_a4_t __attribute__((ext_vector_type(4), aligned(4)));

constexpr int LOOP_THREADS = 256;
constexpr int LOOP_WAVES = LOOP_THREADS / 64;

// Sums over aligned runs of 16 lanes, and over the wave, in a fixed order (every lane gets the
// result): lane exchanges of the vector ALU, a few cycles each, where the ones through LDS take
// about a hundred (the forward at 8192 x 8192 in bf16: 101 -> 95 us).
template <int CTRL>
__device__ __forceinline__ float add_dpp(float v)
{
    return v + __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), CTRL, 0xf, 0xf, true));
}
__device__ __forceinline__ float row16_sum(float v)
{
    v = add_dpp<0xb1>(v);    // lanes 1 apart (quad_perm 1 0 3 2)
    v = add_dpp<0x4e>(v);    // 2 apart (quad_perm 2 3 0 1)
    v = add_dpp<0x141>(v);   // the other quad of eight (row_half_mirror)
    return add_dpp<0x140>(v);  // the other eight (row_mirror)
}
__device__ __forceinline__ float lanes_sum(float v)
{
    v = row16_sum(v);
    auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(p[0]) + __uint_as_float(p[1]);
    p = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(p[0]) + __uint_as_float(p[1]);
}

// N sums over a workgroup of up to 16 waves with one barrier; red [N][16] may be written again
// behind a further one.
template <int N>
__device__ __forceinline__ void group_sums(float (&v)[N], float (*red)[16], int waves)
{
#pragma unroll
    for (int i = 0; i < N; ++i)
        v[i] = lanes_sum(v[i]);
    if (waves == 1)
        return;
    const int lane = threadIdx.x & 63;
    if (lane == 0)
#pragma unroll
        for (int i = 0; i < N; ++i)
            red[i][threadIdx.x >> 6] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i)
        v[i] = row16_sum((lane & 15) < waves ? red[i][lane & 15] : 0.f);
}

// gate row of row t (no gate, or one for all rows: 0)
__device__ __forceinline__ int64_t gate_row(int64_t t, int64_t gate_rows, int64_t T)
{
    return gate_rows == 1 ? t : (gate_rows == 0 || gate_rows >= T ? 0 : t / gate_rows);
}

// h of eight columns from x, the residual, and what x is scaled by (b / rms(x), or b)
template <typename T>
__device__ __forceinline__ Raw8<T> block_h(const BlockNormArgs &a, const Raw8<T> &x,
                                           const Raw8<T> &res, const Raw8<T> &w, const Raw8<T> &gate,
                                           float rstd)
{
    float u[8], r[8];
    x.get(u);
    res.get(r);
    if (a.w_post != nullptr) {
        float v[8];
        w.get(v);
#pragma unroll
        for (int q = 0; q < 8; ++q)
            u[q] = u[q] * rstd * v[q];
    }
    if (a.gate != nullptr) {
        float v[8];
        gate.get(v);
#pragma unroll
        for (int q = 0; q < 8; ++q)
            u[q] *= v[q];
    }
#pragma unroll
    for (int q = 0; q < 8; ++q)
        u[q] = __fmaf_rn(a.branch_scale, u[q], a.res_scale * r[q]);
    Raw8<T> h;
    h.set(u);
    return h;
}

template <typename T>
__device__ __forceinline__ float squares8(const Raw8<T> &v, float k, float acc)
{
    float f[8];
    v.get(f);
#pragma unroll
    for (int q = 0; q < 8; ++q)
        acc = __fmaf_rn(k * f[q], k * f[q], acc);
    return acc;
}

// 1 / rms of a row held as VPT vectors a thread.  red [2][16] is of this call alone: neither row is
// written again by another one, whose waves might be ahead of those that still read it (there
// is no barrier behind the last read; group_sums has none in front of its writes).
template <typename T, int VPT>
__device__ __forceinline__ float row_rstd(const Raw8<T> (&v)[VPT], const BlockNormArgs &a,
                                          float (*red)[16], int waves)
{
    float ss[1] = {0.f};
#pragma unroll
    for (int i = 0; i < VPT; ++i)
        ss[0] = squares8(v[i], 1.f, ss[0]);
    group_sums(ss, red, waves);
    return rstd_of(ss[0], static_cast<float>(a.d), a.eps, [&](float k) {
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            sum = squares8(v[i], k, sum);
        return block_sum(sum, red[1], waves);
    });
}

// Rows that fit a workgroup's registers, VPT vectors a thread: everything is read before the
// first reduction, whose wait covers it, and written once.  h may be the residual, y may be x.
template <typename T, int VPT>
__global__ void __launch_bounds__(1024) block_norm_held_kernel(BlockNormArgs a)
{
    __shared__ float red[4][16];  // two rows for each row_rstd
    const int threads = static_cast<int>(blockDim.x), waves = threads >> 6;
    const int d = static_cast<int>(a.d);
    const int64_t row = static_cast<int64_t>(blockIdx.x) * a.d;
    const T *const gate = static_cast<const T *>(a.gate) + gate_row(blockIdx.x, a.gate_rows, a.T) * a.d;
    auto col = [&](int i) { return (static_cast<int>(threadIdx.x) + i * threads) * 8; };
    Raw8<T> x[VPT], h[VPT], w1[VPT], g[VPT], w2[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        x[i].load(static_cast<const T *>(a.x) + row + col(i), count8(d, col(i)));
        h[i].load(static_cast<const T *>(a.res) + row + col(i), count8(d, col(i)));
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        if (a.w_post != nullptr)
            w1[i].template load<true>(static_cast<const T *>(a.w_post) + col(i), count8(d, col(i)));
        if (a.gate != nullptr)
            g[i].template load<true>(gate + col(i), count8(d, col(i)));
        w2[i].template load<true>(static_cast<const T *>(a.w_pre) + col(i), count8(d, col(i)));
    }
    float r1 = 1.f;
    if (a.w_post != nullptr) {
        r1 = row_rstd(x, a, red, waves);
        if (a.rstd_post != nullptr && threadIdx.x == 0)
            a.rstd_post[blockIdx.x] = r1;
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        h[i] = block_h(a, x[i], h[i], w1[i], g[i], r1);
        h[i].store(static_cast<T *>(a.h) + row + col(i), count8(d, col(i)));
    }
    const float r2 = row_rstd(h, a, red + 2, waves);
    if (a.rstd_pre != nullptr && threadIdx.x == 0)
        a.rstd_pre[blockIdx.x] = r2;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        float f[8], w[8];
        h[i].get(f);
        w2[i].get(w);
#pragma unroll
        for (int q = 0; q < 8; ++q)
            f[q] = f[q] * r2 * w[q];
        Raw8<T> o;
        o.set(f);
        o.store(static_cast<T *>(a.y) + row + col(i), count8(d, col(i)));
    }
}

// Rows of any width: every pass reads the row again, the same columns by the same thread.
template <typename T>
__global__ void __launch_bounds__(LOOP_THREADS) block_norm_kernel(BlockNormArgs a)
{
    __shared__ float red[LOOP_WAVES];
    const int64_t vecs = (a.d + 7) / 8;
    const float d = static_cast<float>(a.d);
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        const int64_t row = t * a.d, grow = gate_row(t, a.gate_rows, a.T) * a.d;
        auto squares = [&](const void *m) {
            return [&, m](float k) {
                float ss = 0.f;
                for (int64_t v = threadIdx.x; v < vecs; v += LOOP_THREADS) {
                    Raw8<T> r;
                    r.load(static_cast<const T *>(m) + row + v * 8, count8(a.d, v * 8));
                    ss = squares8(r, k, ss);
                }
                return block_sum(ss, red, LOOP_WAVES);
            };
        };
        float r1 = 1.f;
        if (a.w_post != nullptr) {
            const auto sum = squares(a.x);
            r1 = rstd_of(sum(1.f), d, a.eps, sum);
            if (a.rstd_post != nullptr && threadIdx.x == 0)
                a.rstd_post[t] = r1;
        }
        float ss = 0.f;
        for (int64_t v = threadIdx.x; v < vecs; v += LOOP_THREADS) {
            const int cnt = count8(a.d, v * 8);
            Raw8<T> x, r, w1, g;
            x.load(static_cast<const T *>(a.x) + row + v * 8, cnt);
            r.load(static_cast<const T *>(a.res) + row + v * 8, cnt);
            if (a.w_post != nullptr)
                w1.template load<true>(static_cast<const T *>(a.w_post) + v * 8, cnt);
            if (a.gate != nullptr)
                g.template load<true>(static_cast<const T *>(a.gate) + grow + v * 8, cnt);
            r = block_h(a, x, r, w1, g, r1);
            r.store(static_cast<T *>(a.h) + row + v * 8, cnt);
            ss = squares8(r, 1.f, ss);
        }
        // (a thread reads back only what it wrote)
        const float r2 = rstd_of(block_sum(ss, red, LOOP_WAVES), d, a.eps, squares(a.h));
        if (a.rstd_pre != nullptr && threadIdx.x == 0)
            a.rstd_pre[t] = r2;
        for (int64_t v = threadIdx.x; v < vecs; v += LOOP_THREADS) {
            const int cnt = count8(a.d, v * 8);
            Raw8<T> h, w2;
            h.load(static_cast<const T *>(a.h) + row + v * 8, cnt);
            w2.template load<true>(static_cast<const T *>(a.w_pre) + v * 8, cnt);
            float f[8], w[8];
            h.get(f);
            w2.get(w);
#pragma unroll
            for (int q = 0; q < 8; ++q)
                f[q] = f[q] * r2 * w[q];
            h.set(f);
            h.store(static_cast<T *>(a.y) + row + v * 8, cnt);
        }
    }
}

// --------------------------------------------------------------- the gradients
// A row's eight columns as the gradient reads them.
template <typename T>
struct GradVec {
    Raw8<T> dy, dh, x, h, gate;  // gate: where every row has its own
};
// A thread's columns: w_pre, and what scales Dh: c = b w_post gate (the gate where rows share
// it, w_post and gate 1 where there are none).
template <typename T>
struct GradWeights {
    Raw8<T> pre;
    float c[8];
};
// What the sums need of the scalars.
struct GradScalars {
    float r1, r2;
    bool with_dh;
};

// Column j of a row that starts at `base`: a scalar base and a 32-bit offset (rows of under
// 2^30 columns).
template <typename P>
__device__ __forceinline__ P *in_row(P *base, unsigned int j)
{
    using B = std::conditional_t<std::is_const_v<P>, const char, char>;
    return reinterpret_cast<P *>(reinterpret_cast<B *>(base) + j * static_cast<unsigned int>(sizeof(P)));
}

// GATE: 0 none, 1 rows share gate rows, 2 a gate row of its own each.
template <bool POST, int GATE, typename T>
__device__ __forceinline__ GradWeights<T> grad_weights(const BlockNormGradArgs &a, int64_t grow,
                                                       int64_t j, int cnt)
{
    GradWeights<T> w;
    w.pre.template load<true>(static_cast<const T *>(a.w_pre) + j, cnt);
#pragma unroll
    for (int q = 0; q < 8; ++q)
        w.c[q] = a.branch_scale;
    auto times = [&](const T *m) {
        Raw8<T> r;
        r.template load<true>(m + j, cnt);
        float f[8];
        r.get(f);
#pragma unroll
        for (int q = 0; q < 8; ++q)
            w.c[q] *= f[q];
    };
    if constexpr (POST)
        times(static_cast<const T *>(a.w_post));
    if constexpr (GATE == 1)
        times(static_cast<const T *>(a.gate) + grow * a.d);
    return w;
}

template <bool POST, int GATE, typename T>
__device__ __forceinline__ void grad_load(GradVec<T> &v, const BlockNormGradArgs &a, int64_t row,
                                          unsigned int j, int cnt)
{
    v.dy.load(in_row(static_cast<const T *>(a.dy) + row, j), cnt);
    v.h.load(in_row(static_cast<const T *>(a.h) + row, j), cnt);
    if constexpr (POST || GATE != 0)
        v.x.load(in_row(static_cast<const T *>(a.x) + row, j), cnt);
    if (a.dh != nullptr)
        v.dh.load(in_row(static_cast<const T *>(a.dh) + row, j), cnt);
    if constexpr (GATE == 2)
        v.gate.load(in_row(static_cast<const T *>(a.gate) + row, j), cnt);
}

// Dh before m1 is known: dh_in + w_pre dy / rms(h); and hat(h).
template <typename T>
__device__ __forceinline__ void grad_front(const GradVec<T> &v, const GradWeights<T> &w,
                                           const GradScalars &k, float (&dy)[8], float (&hh)[8],
                                           float (&e)[8], float &s1)
{
    float wp[8];
    v.dy.get(dy);
    v.h.get(hh);
    w.pre.get(wp);
    if (k.with_dh) {
        v.dh.get(e);
    } else {
#pragma unroll
        for (int q = 0; q < 8; ++q)
            e[q] = 0.f;
    }
#pragma unroll
    for (int q = 0; q < 8; ++q) {
        hh[q] *= k.r2;
        const float wdy = dy[q] * wp[q];
        s1 = __fmaf_rn(wdy, hh[q], s1);
        e[q] = __fmaf_rn(k.r2, wdy, e[q]);
    }
}

// The row's three sums, from which m1 and m2 follow in one reduction: with
// k = c gate hat(x), m2 is the mean of k Dh, and Dh is linear in m1:
//   s1 = sum w_pre dy hat(h),  sa = sum k (dh_in + w_pre dy / rms(h)),  sb = sum k hat(h),
//   m1 = s1 / d,  m2 = (sa - m1 sb / rms(h)) / d
struct GradSums {
    float s1, sa, sb;
};

template <bool POST, int GATE, typename T>
__device__ __forceinline__ void grad_sums(GradSums &s, const GradVec<T> &v, const GradWeights<T> &w,
                                          const GradScalars &sc)
{
    float dy[8], hh[8], e[8];
    grad_front(v, w, sc, dy, hh, e, s.s1);
    if constexpr (POST) {
        float k[8], g[8];
        v.x.get(k);
        if constexpr (GATE == 2)
            v.gate.get(g);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            k[q] *= sc.r1;
            k[q] *= GATE == 2 ? w.c[q] * g[q] : w.c[q];
            s.sa = __fmaf_rn(k[q], e[q], s.sa);
            s.sb = __fmaf_rn(k[q], hh[q], s.sb);
        }
    }
}

// What is left of eight columns once m1 and m2 are known: dx and dresidual, dw_pre's terms,
// and z = sum Dh hat(x), from which the gradients of the gate and of w_post both follow while
// rows share the gate: dgate = b w_post z, dw_post = b gate z.  With a gate row for
// each row (GATE 2), z = sum gate Dh hat(x) and dgate is the row's own.
template <bool POST, int GATE, typename T>
__device__ __forceinline__ void grad_apply(const GradVec<T> &v, const GradWeights<T> &w,
                                           const GradScalars &sc, float a, float m1, float m2,
                                           Raw8<T> &dx, Raw8<T> &dres, Raw8<T> &dgate,
                                           float (&dw2)[8], float (&z)[8])
{
    float dy[8], hh[8], o[8], f[8], unused = 0.f;
    grad_front(v, w, sc, dy, hh, o, unused);
    const float back = -sc.r2 * m1;
#pragma unroll
    for (int q = 0; q < 8; ++q) {
        dw2[q] = __fmaf_rn(dy[q], hh[q], dw2[q]);
        o[q] = __fmaf_rn(back, hh[q], o[q]);
        f[q] = a * o[q];
    }
    dres.set(f);
    float x[8], g[8];
    if constexpr (POST || GATE != 0)
        v.x.get(x);
    if constexpr (GATE == 2)
        v.gate.get(g);
#pragma unroll
    for (int q = 0; q < 8; ++q) {
        if constexpr (POST || GATE != 0) {
            if constexpr (POST)
                x[q] *= sc.r1;
            if constexpr (GATE == 2) {
                const float t = o[q] * x[q];
                z[q] = __fmaf_rn(g[q], t, z[q]);
                f[q] = w.c[q] * t;
                o[q] *= g[q];
            } else {
                z[q] = __fmaf_rn(o[q], x[q], z[q]);
            }
        }
        o[q] *= w.c[q];
        if constexpr (POST)
            o[q] = sc.r1 * __fmaf_rn(-m2, x[q], o[q]);
    }
    if constexpr (GATE == 2)
        dgate.set(f);
    dx.set(o);
}

// m2 from the row's sums
__device__ __forceinline__ float grad_m2(const GradSums &s, float m1, float r2, float inv_d)
{
    return __fmaf_rn(-m1 * r2, s.sb, s.sa) * inv_d;
}

// The first cnt of eight sums, as whole vectors where they all are there (single values 32 bytes
// apart a lane took most of a short call's time: 8192 x 8192 in bf16 161 -> 154 us, 512 x 4096 27 -> 22).
__device__ __forceinline__ void put8(float *p, const float (&v)[8], int cnt)
{
    if (cnt >= 8) {
#pragma unroll
        for (int k = 0; k < 2; ++k)
            reinterpret_cast<f32x4_a4_t *>(p)[k] =
                f32x4_a4_t{v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]};
    } else {
#pragma unroll
        for (int q = 0; q < 8; ++q)
            if (q < cnt)
                p[q] = v[q];
    }
}

struct GradOut {  // partial sums (or, where there is one part, the sums)
    float *pre, *post, *gate;
    float *mean;  // rows of any width: m1 and m2 of each row
    int64_t chunk;  // rows a workgroup
    int direct;
    // 0: workgroup b's rows are b chunk and on; else b, b + stride, ..., so that the rows in
    // work at one time lie next to each other (chunks start a power of two apart, and their
    // lines in the same memory channels: 16384 x 4096 in bf16 171 -> 158 us)
    int64_t stride;
    __device__ __forceinline__ int64_t first(int64_t b) const { return stride ? b : b * chunk; }
    __device__ __forceinline__ int64_t end(int64_t b, int64_t T) const
    {
        return !stride && (b + 1) * chunk < T ? (b + 1) * chunk : T;
    }
    __device__ __forceinline__ int64_t step() const { return stride ? stride : 1; }
};

// The end of a run of rows that share gate row `grow`, in workgroup `part`: the gate's gradient
// goes out (rounded, or to slot part + grow of the partial sums, which no other pair has, both
// indices growing along the rows), f becomes dw_post's share of z, and z is cleared.
template <bool POST, typename T>
__device__ __forceinline__ void grad_gate_end(const BlockNormGradArgs &a, const GradOut &out,
                                              int64_t part, int64_t grow, int64_t j, int cnt,
                                              float (&z)[8], float (&f)[8])
{
    Raw8<T> r;
    float g[8];
#pragma unroll
    for (int q = 0; q < 8; ++q)
        g[q] = a.branch_scale * z[q];
    if constexpr (POST) {
        r.template load<true>(static_cast<const T *>(a.gate) + grow * a.d + j, cnt);
        r.get(f);
#pragma unroll
        for (int q = 0; q < 8; ++q)
            f[q] *= g[q];
        r.template load<true>(static_cast<const T *>(a.w_post) + j, cnt);
        float w[8];
        r.get(w);
#pragma unroll
        for (int q = 0; q < 8; ++q)
            g[q] *= w[q];
    }
    if (a.dgate != nullptr) {
        if (out.direct) {
            r.set(g);
            r.store(static_cast<T *>(a.dgate) + grow * a.d + j, cnt);
        } else {
            put8(out.gate + (part + grow) * a.d + j, g, cnt);
        }
    }
#pragma unroll
    for (int q = 0; q < 8; ++q)
        z[q] = 0.f;
}

// One pass over rows that fit a workgroup's registers; a thread keeps its eight columns' weights and sums.
template <typename T, bool POST, int GATE, int THREADS>
__global__ void __launch_bounds__(THREADS) block_norm_grad_held_kernel(BlockNormGradArgs a, GradOut out)
{
    constexpr bool FOLD = POST && GATE == 1;  // dw_post is gathered where gate rows end
    __shared__ float red[2][3][16];
    __shared__ float4 fold[2][FOLD ? THREADS : 1];
    const int waves = static_cast<int>(blockDim.x) >> 6;
    const float inv_d = 1.f / static_cast<float>(a.d);
    const unsigned int j = threadIdx.x * 8;
    const int cnt = count8(a.d, j);
    GradWeights<T> w;
    float dw2[8], z[8];
    if constexpr (GATE != 1)
        w = grad_weights<POST, GATE, T>(a, 0, j, cnt);
    if constexpr (FOLD)
        fold[0][threadIdx.x] = fold[1][threadIdx.x] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int q = 0; q < 8; ++q)
        dw2[q] = z[q] = 0.f;
    int64_t t = out.first(blockIdx.x);
    const int64_t end = out.end(blockIdx.x, a.T), step = out.step();
    int64_t grow = 0, gend = 0;  // GATE 1: the gate row held, and the row behind its last
    auto gate_end = [&]() {
        float f[8];
        grad_gate_end<POST, T>(a, out, blockIdx.x, grow, j, cnt, z, f);
        if constexpr (FOLD) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                float4 p = fold[k][threadIdx.x];
                p.x += f[4 * k];
                p.y += f[4 * k + 1];
                p.z += f[4 * k + 2];
                p.w += f[4 * k + 3];
                fold[k][threadIdx.x] = p;
            }
        }
    };
    for (int par = 0; t < end; t += step, par ^= 1) {
        GradVec<T> v;
        grad_load<POST, GATE>(v, a, t * a.d, j, cnt);
        const GradScalars sc{POST ? a.rstd_post[t] : 1.f, a.rstd_pre[t], a.dh != nullptr};
        if constexpr (GATE == 1) {
            if (t >= gend) {
                if (gend != 0)
                    gate_end();
                grow = gate_row(t, a.gate_rows, a.T);
                gend = (grow + 1) * a.gate_rows;
                w = grad_weights<POST, GATE, T>(a, grow, j, cnt);
            }
        }
        GradSums s{0.f, 0.f, 0.f};
        grad_sums<POST, GATE>(s, v, w, sc);
        // one barrier a row: the next row writes the other half of `red`
        if constexpr (POST) {
            float all[3] = {s.s1, s.sa, s.sb};
            group_sums(all, red[par], waves);
            s = GradSums{all[0], all[1], all[2]};
        } else {
            float all[1] = {s.s1};
            group_sums(all, red[par], waves);
            s.s1 = all[0];
        }
        const float m1 = s.s1 * inv_d;
        const float m2 = POST ? grad_m2(s, m1, sc.r2, inv_d) : 0.f;
        // (what the sums made of them would not leave the registers else)
        forget(v.dy);
        forget(v.h);
        if constexpr (POST)
            forget(v.x);
        Raw8<T> dx, dres, dgate;
        grad_apply<POST, GATE>(v, w, sc, a.res_scale, m1, m2, dx, dres, dgate, dw2, z);
        dx.store(in_row(static_cast<T *>(a.dx) + t * a.d, j), cnt);
        dres.store(in_row(static_cast<T *>(a.dres) + t * a.d, j), cnt);
        if (GATE == 2 && a.dgate != nullptr)
            dgate.store(in_row(static_cast<T *>(a.dgate) + t * a.d, j), cnt);
    }
    if (GATE == 1 && gend != 0)
        gate_end();
    const int64_t o = blockIdx.x * a.d + j;
    float f[8];
    if constexpr (FOLD) {
        const float4 u = fold[0][threadIdx.x], v = fold[1][threadIdx.x];
        const float all[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
#pragma unroll
        for (int q = 0; q < 8; ++q)
            f[q] = all[q];
    } else {
#pragma unroll
        for (int q = 0; q < 8; ++q)
            f[q] = a.branch_scale * z[q];
    }
    if (out.pre != nullptr)
        put8(out.pre + o, dw2, cnt);
    if (POST && out.post != nullptr)
        put8(out.post + o, f, cnt);
}

// Rows of any width, first pass: m1 and m2 of every row.
template <typename T, bool POST, int GATE>
__global__ void __launch_bounds__(LOOP_THREADS) block_norm_mean_kernel(BlockNormGradArgs a, float *mean)
{
    __shared__ float red[LOOP_WAVES];
    const int64_t vecs = (a.d + 7) / 8;
    const float inv_d = 1.f / static_cast<float>(a.d);
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        const int64_t grow = GATE == 1 ? gate_row(t, a.gate_rows, a.T) : 0;
        GradSums s{0.f, 0.f, 0.f};
        const GradScalars sc{POST ? a.rstd_post[t] : 1.f, a.rstd_pre[t], a.dh != nullptr};
        for (int64_t i = threadIdx.x; i < vecs; i += LOOP_THREADS) {
            const int cnt = count8(a.d, i * 8);
            GradVec<T> v;
            grad_load<POST, POST ? GATE : 0>(v, a, t * a.d + i * 8, 0u, cnt);
            grad_sums<POST, GATE>(s, v, grad_weights<POST, GATE, T>(a, grow, i * 8, cnt), sc);
        }
        const float m1 = block_sum(s.s1, red, LOOP_WAVES) * inv_d;
        float m2 = 0.f;
        if constexpr (POST) {
            s.sa = block_sum(s.sa, red, LOOP_WAVES);
            s.sb = block_sum(s.sb, red, LOOP_WAVES);
            m2 = grad_m2(s, m1, sc.r2, inv_d);
        }
        if (threadIdx.x == 0) {
            mean[2 * t] = m1;
            mean[2 * t + 1] = m2;
        }
    }
}

// Second pass: workgroup (i, b) walks its rows at 2048 columns.
template <typename T, bool POST, int GATE>
__global__ void __launch_bounds__(LOOP_THREADS) block_norm_grad_kernel(BlockNormGradArgs a, GradOut out)
{
    const int64_t j = (static_cast<int64_t>(blockIdx.x) * LOOP_THREADS + threadIdx.x) * 8;
    if (j >= a.d)
        return;
    const int cnt = count8(a.d, j);
    GradWeights<T> w;
    if constexpr (GATE != 1)
        w = grad_weights<POST, GATE, T>(a, 0, j, cnt);
    float dw2[8], z[8], dw1[8];
#pragma unroll
    for (int q = 0; q < 8; ++q)
        dw2[q] = z[q] = dw1[q] = 0.f;
    int64_t t = out.first(blockIdx.y);
    const int64_t end = out.end(blockIdx.y, a.T), step = out.step();
    int64_t grow = 0, gend = 0;
    auto gate_end = [&]() {
        float f[8];
        grad_gate_end<POST, T>(a, out, blockIdx.y, grow, j, cnt, z, f);
        if constexpr (POST) {
#pragma unroll
            for (int q = 0; q < 8; ++q)
                dw1[q] += f[q];
        }
    };
    for (; t < end; t += step) {
        if (GATE == 1 && t >= gend) {
            if (gend != 0)
                gate_end();
            grow = gate_row(t, a.gate_rows, a.T);
            gend = (grow + 1) * a.gate_rows;
            w = grad_weights<POST, GATE, T>(a, grow, j, cnt);
        }
        const int64_t at = t * a.d + j;
        GradVec<T> v;
        grad_load<POST, GATE>(v, a, at, 0u, cnt);
        const GradScalars sc{POST ? a.rstd_post[t] : 1.f, a.rstd_pre[t], a.dh != nullptr};
        Raw8<T> dx, dres, dgate;
        grad_apply<POST, GATE>(v, w, sc, a.res_scale, out.mean[2 * t], out.mean[2 * t + 1], dx, dres,
                               dgate, dw2, z);
        dx.store(static_cast<T *>(a.dx) + at, cnt);
        dres.store(static_cast<T *>(a.dres) + at, cnt);
        if (GATE == 2 && a.dgate != nullptr)
            dgate.store(static_cast<T *>(a.dgate) + at, cnt);
    }
    if (GATE == 1) {
        if (gend != 0)
            gate_end();
    } else {
#pragma unroll
        for (int q = 0; q < 8; ++q)
            dw1[q] = a.branch_scale * z[q];
    }
    const int64_t o = static_cast<int64_t>(blockIdx.y) * a.d + j;
    if (out.pre != nullptr)
        put8(out.pre + o, dw2, cnt);
    if (POST && out.post != nullptr)
        put8(out.post + o, dw1, cnt);
}

// The partial sums in a fixed order: blockIdx.y 0 dw_pre, 1 dw_post, then the gate rows, one at a
// time or, where they have few slots (a slot at least a chunk of rows, see the plan), 16 of them,
// a wave each; 16, 32 or 64 columns a workgroup (`cols`), whose 16 waves take every 16th part, or
// group of 2 or 4 of them, each.
template <typename T>
__global__ void __launch_bounds__(1024)
    block_norm_finish_kernel(GradOut part, int parts, int64_t Tn, int64_t d, int64_t gate_rows,
                             int cols, float *dw_pre, float *dw_post, T *dgate)
{
    __shared__ float sums[16][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const bool few = gate_rows <= 16 * part.chunk && gate_rows < Tn;
    const int64_t g = blockIdx.y < 2 ? -1 : few ? (blockIdx.y - 2ll) * 16 + wave : blockIdx.y - 2ll;
    const bool alone = few && g >= 0;  // the wave sums by itself
    const float *from = blockIdx.y == 0 ? part.pre : part.post;
    int64_t count = parts;
    if (g >= 0) {
        if (dgate == nullptr || (alone && g * gate_rows >= Tn))
            return;
        const int64_t first = g * gate_rows;
        const int64_t last = (first + gate_rows < Tn ? first + gate_rows : Tn) - 1;
        from = part.gate + (first / part.chunk + g) * d;
        count = Tn == 0 ? 0 : last / part.chunk - first / part.chunk + 1;
    } else if ((blockIdx.y == 0 ? dw_pre : dw_post) == nullptr) {
        return;
    }
    const int at_once = 64 / cols, part_of = lane / cols, column = lane & (cols - 1);
    for (int64_t j0 = static_cast<int64_t>(blockIdx.x) * cols; j0 < d;
         j0 += static_cast<int64_t>(gridDim.x) * cols) {
        const int64_t j = j0 + column;
        float acc = 0.f;
        if (j < d) {
#pragma unroll 8
            for (int64_t p = (alone ? 0 : wave * at_once) + part_of; p < count;
                 p += alone ? at_once : 16 * at_once)
                acc += from[p * d + j];
        }
        for (int m = cols; m < 64; m *= 2)
            acc += __shfl_xor(acc, m);
        if (!alone) {
            __syncthreads();  // the last columns' sums have been read
            sums[wave][lane] = acc;
            __syncthreads();
            acc = sums[0][lane];
#pragma unroll
            for (int k = 1; k < 16; ++k)
                acc += sums[k][lane];
        }
        if ((alone || wave == 0) && part_of == 0 && j < d) {
            if (g >= 0) {
                if constexpr (sizeof(T) == 2)
                    dgate[g * d + j] = f32_to_bf16(acc);
                else
                    dgate[g * d + j] = acc;
            } else {
                (blockIdx.y == 0 ? dw_pre : dw_post)[j] = acc;
            }
        }
    }
}

constexpr int64_t MAX_ROW_GROUPS = 1 << 20;  // workgroups of a row launch

template <typename T>
hipError_t forward(const BlockNormArgs &a, hipStream_t st)
{
    const int64_t vecs = (a.d + 7) / 8;
    int vpt = a.T <= 512 ? 1 : 2;
    while (vecs > 1024 * static_cast<int64_t>(vpt) && vpt < 4)
        vpt *= 2;
    const int64_t threads = ((vecs + vpt - 1) / vpt + 63) / 64 * 64;
    const dim3 grid(static_cast<unsigned>(a.T)), block(static_cast<unsigned>(threads));
    // (a launch holds fewer than 2^32 threads)
    if (vecs > 1024 * static_cast<int64_t>(vpt) || a.T >= (int64_t(1) << 32) / threads)
        hipLaunchKernelGGL((block_norm_kernel<T>),
                           dim3(static_cast<unsigned>(a.T < MAX_ROW_GROUPS ? a.T : MAX_ROW_GROUPS)),
                           dim3(LOOP_THREADS), 0, st, a);
    else if (vpt == 1)
        hipLaunchKernelGGL((block_norm_held_kernel<T, 1>), grid, block, 0, st, a);
    else if (vpt == 2)
        hipLaunchKernelGGL((block_norm_held_kernel<T, 2>), grid, block, 0, st, a);
    else
        hipLaunchKernelGGL((block_norm_held_kernel<T, 4>), grid, block, 0, st, a);
    return hipGetLastError();
}

// Rows held in registers: eight columns of each of 1024 threads.
bool grad_held(int64_t d) { return d <= 8192; }

template <typename T, bool POST, int GATE>
hipError_t backward(const BlockNormGradArgs &a, const BlockNormPlan &p, const GradOut &out, hipStream_t st)
{
    const int64_t vecs = (a.d + 7) / 8;
    if (p.held) {
        const dim3 grid(static_cast<unsigned>(p.parts)),
            block(static_cast<unsigned>((vecs + 63) / 64 * 64));
        if (vecs <= 512)
            hipLaunchKernelGGL((block_norm_grad_held_kernel<T, POST, GATE, 512>), grid, block, 0, st, a,
                               out);
        else
            hipLaunchKernelGGL((block_norm_grad_held_kernel<T, POST, GATE, 1024>), grid, block, 0, st,
                               a, out);
        return hipGetLastError();
    }
    hipLaunchKernelGGL((block_norm_mean_kernel<T, POST, GATE>),
                       dim3(static_cast<unsigned>(a.T < MAX_ROW_GROUPS ? a.T : MAX_ROW_GROUPS)),
                       dim3(LOOP_THREADS), 0, st, a, out.mean);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess)
        return e;
    hipLaunchKernelGGL((block_norm_grad_kernel<T, POST, GATE>),
                       dim3(static_cast<unsigned>((vecs + LOOP_THREADS - 1) / LOOP_THREADS),
                            static_cast<unsigned>(p.parts)),
                       dim3(LOOP_THREADS), 0, st, a, out);
    return hipGetLastError();
}

template <typename T>
hipError_t backward_any(const BlockNormGradArgs &a, const BlockNormPlan &p, char *ws, hipStream_t st)
{
    const bool one = p.parts <= 1;  // one part is the sum itself
    auto at = [&](size_t o) { return reinterpret_cast<float *>(ws + o); };
    const GradOut out{a.dw_pre == nullptr ? nullptr : (one ? a.dw_pre : at(p.o_pre)),
                      a.dw_post == nullptr ? nullptr : (one ? a.dw_post : at(p.o_post)),
                      at(p.o_gate), at(p.o_mean), p.chunk, p.direct,
                      a.gate_rows > 1 && a.gate_rows < a.T ? 0 : p.parts};
    const int gate = a.gate == nullptr ? 0 : (a.gate_rows == 1 ? 2 : 1);
    hipError_t e = hipSuccess;
    if (a.T == 0)
        ;  // (no partial sums: the finish writes zeros)
    else if (a.w_post != nullptr)
        e = gate == 0   ? backward<T, true, 0>(a, p, out, st)
            : gate == 1 ? backward<T, true, 1>(a, p, out, st)
                        : backward<T, true, 2>(a, p, out, st);
    else
        e = gate == 0   ? backward<T, false, 0>(a, p, out, st)
            : gate == 1 ? backward<T, false, 1>(a, p, out, st)
                        : backward<T, false, 2>(a, p, out, st);
    const bool slots = a.dgate != nullptr && (a.T == 0 || (gate == 1 && !p.direct));
    const bool sums = (!one || a.T == 0) && (a.dw_pre != nullptr || a.dw_post != nullptr);
    if (e != hipSuccess || (!slots && !sums))
        return e;
    const int64_t rows = !slots ? 0 : a.T == 0 ? 1 : (a.T + a.gate_rows - 1) / a.gate_rows;
    const bool few = a.gate_rows <= 16 * p.chunk && a.gate_rows < a.T;
    const int64_t arrays = 2 + (few ? (rows + 15) / 16 : rows);
    // the widest columns that make 256 workgroups, but a line's half at least (the sums of 256
    // parts of 4096 columns: 32 columns 2 us less than 64; with eight gates' 4 us more)
    int cols = 64;
    while (cols > 16 && (a.d + cols - 1) / cols * arrays < 256)
        cols /= 2;
    const int64_t blocks = (a.d + cols - 1) / cols;
    hipLaunchKernelGGL((block_norm_finish_kernel<T>),
                       dim3(static_cast<unsigned>(blocks < 65536 ? blocks : 65536),
                            static_cast<unsigned>(arrays)),
                       dim3(1024), 0, st, out, p.parts, a.T, a.d, a.gate_rows, cols,
                       sums ? a.dw_pre : nullptr, sums ? a.dw_post : nullptr,
                       slots ? static_cast<T *>(a.dgate) : nullptr);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_block_norm(int bf16, const BlockNormArgs &a, hipStream_t st)
{
    if (a.T == 0)
        return hipSuccess;
    return bf16 ? forward<uint16_t>(a, st) : forward<float>(a, st);
}

BlockNormPlan plan_block_norm_grad(int64_t T, int64_t d, int64_t gate_rows)
{
    BlockNormPlan p;
    p.held = grad_held(d);
    const int64_t vecs = (d + 7) / 8;
    int64_t parts;
    if (p.held) {
        // A workgroup a CU, and the shorter the rows the more of them from eight rows each on (2048 x
        // 4096 in bf16: 42 us, from four on 47); of wide rows fewer, down to 128, before
        // they have less than four, since each leaves a row of sums (512 x 8192: 39 us, 256 of
        // them 41; 256 x 8192: 32 and 37).
        const int most = vecs > 512 ? 1 : vecs > 128 ? 2 : vecs > 64 ? 4 : 8;
        const int64_t share = T / 8, few = T / 4 < 128 ? 128 : T / 4 < 256 ? T / 4 : 256;
        const int64_t least = vecs > 512 ? few : 256;
        parts = share > least ? share : least;
        parts = parts < 256 * most ? parts : 256 * most;
        parts = parts < T ? parts : T;
    } else {
        // about 2048 workgroups over column blocks and chunks, 16 rows each at least
        parts = 2048 / ((vecs + LOOP_THREADS - 1) / LOOP_THREADS);
        parts = parts < (T + 15) / 16 ? parts : (T + 15) / 16;
    }
    parts = parts < 1 ? 1 : parts;
    p.chunk = (T + parts - 1) / parts;
    p.chunk = p.chunk < 1 ? 1 : p.chunk;
    // Whole gate rows in a chunk, where that makes it longer by a quarter at most, leave no
    // partial sums; else the slots are at most five a workgroup.
    p.direct = gate_rows > 1 && (gate_rows >= T ? p.chunk >= T : 4 * gate_rows <= p.chunk);
    if (p.direct && gate_rows < T)
        p.chunk = (p.chunk + gate_rows - 1) / gate_rows * gate_rows;
    p.parts = static_cast<int>((T + p.chunk - 1) / p.chunk);
    p.slots = gate_rows > 1 && !p.direct && T > 0 ? p.parts + (T + gate_rows - 1) / gate_rows : 0;
    auto take = [off = size_t(0)](size_t bytes) mutable {
        const size_t at = off;
        off += (bytes + 255) / 256 * 256;
        return at;
    };
    const size_t row = static_cast<size_t>(d) * sizeof(float);
    const size_t sums = p.parts > 1 ? p.parts * row : 0;
    p.o_pre = take(sums);
    p.o_post = take(sums);
    p.o_gate = take(p.slots * row);
    p.o_mean = take(p.held ? 0 : static_cast<size_t>(T) * 2 * sizeof(float));
    p.bytes = take(0);
    return p;
}

hipError_t launch_block_norm_grad(int bf16, const BlockNormGradArgs &a, const BlockNormPlan &p,
                                  void *ws, hipStream_t st)
{
    char *const w = static_cast<char *>(ws);
    return bf16 ? backward_any<uint16_t>(a, p, w, st) : backward_any<float>(a, p, w, st);
}

}  // namespace dora
