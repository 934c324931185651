// gemm_fourbit.hip - y = x W^T for a few tokens and a weight held as 4-bit rows (gfx950).
//
// Bound by reading the codes once (half a byte a weight).  A workgroup takes 16 NT output
// channels and up to 16 TM tokens; its waves split K, wave w taking the lines (256 columns, the
// 128 bytes of codes that one cache line holds) w, w + W, ...  A lane loads 16 bytes of its
// channel's codes at a time, D lines ahead, straight into registers; exchanges between the lane
// groups turn four such registers into four MFMA operands of 32 consecutive columns each, and
// one conversion instruction makes two bf16 weights of two codes.  The weights enter the
// products as the codes' own values, exact in bf16, and the fp32 sums over a group's columns
// meet its scale, so that nothing is rounded before the sums.  fp32 tokens enter as three bf16
// numbers each, which hold all 24 bits.  The waves' sums meet in LDS, in order.
#include "around.hpp"
#include "fourbit.hpp"

namespace dora {
namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef unsigned int u32x4_t __attribute__((ext_vector_type(4)));

constexpr int LINE = 256;          // columns of a line
constexpr int STEPS = LINE / 32;   // MFMA steps of a line

// Exchanges register index and lane group (16 lanes): afterwards register s holds, in group
// k, what register k held in group s.
__device__ __forceinline__ void exchange4(unsigned int (&r)[4])
{
    auto p = __builtin_amdgcn_permlane32_swap(r[0], r[2], false, false);
    r[0] = p[0];
    r[2] = p[1];
    p = __builtin_amdgcn_permlane32_swap(r[1], r[3], false, false);
    r[1] = p[0];
    r[3] = p[1];
    p = __builtin_amdgcn_permlane16_swap(r[0], r[1], false, false);
    r[0] = p[0];
    r[1] = p[1];
    p = __builtin_amdgcn_permlane16_swap(r[2], r[3], false, false);
    r[2] = p[0];
    r[3] = p[1];
}

// Eight codes as bf16.
__device__ __forceinline__ bf16x8_t weights8(unsigned int c)
{
    const auto a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, 1.f, 0);
    const auto b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, 1.f, 1);
    const auto e = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, 1.f, 2);
    const auto g = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, 1.f, 3);
    return bf16x8_t{a[0], a[1], b[0], b[1], e[0], e[1], g[0], g[1]};
}

// Eight elements of x as P operands whose sum they are (1: bf16; 3: fp32, each the leading
// eight bits of what the ones before it leave; infinities and NaN in the first alone).
template <typename T>
constexpr int planes = sizeof(T) == 2 ? 1 : 3;
template <typename T>
__device__ __forceinline__ void split8(const Raw8<T> &v, unsigned int (&w)[planes<T>][4])
{
    if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
            w[0][q] = v.w[q];
    } else {
        unsigned int p[3][8];
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            const unsigned int b = v.w[q];
            p[0][q] = b & 0xffff0000u;
            const bool finite = (b & 0x7f800000u) != 0x7f800000u;
            const float r = finite ? __uint_as_float(b) - __uint_as_float(p[0][q]) : 0.f;
            p[1][q] = __float_as_uint(r) & 0xffff0000u;
            p[2][q] = __float_as_uint(r - __uint_as_float(p[1][q]));
            // (a NaN whose bits all lie in the lower half stays one)
            if ((b & 0x7fffffffu) > 0x7f800000u)
                p[0][q] |= 0x400000u;
        }
#pragma unroll
        for (int k = 0; k < 3; ++k)
#pragma unroll
            for (int q = 0; q < 4; ++q)
                w[k][q] = (p[k][2 * q] >> 16) | (p[k][2 * q + 1] & 0xffff0000u);
    }
}

// The scales of a line's groups: PER of them (8, 4, 2 for groups of 32, 64, 128; else one).
template <int PER>
struct LineScales {
    unsigned int w[(PER + 1) / 2];
    __device__ __forceinline__ void load(const uint16_t *p)
    {
        if constexpr (PER == 8) {
            const u32x4_a2_t v = *reinterpret_cast<const u32x4_a2_t *>(p);
            w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
        } else if constexpr (PER == 4) {
            const u32x2_a2_t v = *reinterpret_cast<const u32x2_a2_t *>(p);
            w[0] = v.x; w[1] = v.y;
        } else if constexpr (PER == 2) {
            w[0] = *reinterpret_cast<const u32_a2_t *>(p);
        } else {
            w[0] = *p;
        }
    }
    // the first `cnt` of them
    __device__ __forceinline__ void load_some(const uint16_t *p, int64_t cnt)
    {
#pragma unroll
        for (int q = 0; q < (PER + 1) / 2; ++q) {
            w[q] = 2 * q < cnt ? p[2 * q] : 0u;
            if (PER > 1 && 2 * q + 1 < cnt)
                w[q] |= static_cast<unsigned int>(p[2 * q + 1]) << 16;
        }
    }
    __device__ __forceinline__ float get(int k) const
    {
        return __uint_as_float(k & 1 ? w[k >> 1] & 0xffff0000u : w[k >> 1] << 16);
    }
};

template <int NT, int PER>
struct Line {
    unsigned int c[NT][2][4];
    LineScales<PER> s[NT];
};

// XLDS: the tokens' rows lie whole in LDS (dynamic: planes x T x pitch elements); else every
// lane reads its own operands from memory, half a line ahead of their use.
template <typename T, int TM, int NT, int PER, bool XLDS, int W, int D>
__global__ void __launch_bounds__(W * 64) linear_fourbit_kernel(FourbitArgs a)
{
    constexpr int P = planes<T>, HALF = STEPS / 2;
    constexpr int PITCH = 16 * NT + 4;
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ __align__(16) float sums[W][16 * TM][PITCH];
    const int lane = static_cast<int>(threadIdx.x) & 63, nl = lane & 15, kq = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6);
    const int64_t n0 = static_cast<int64_t>(blockIdx.x) * (16 * NT);
    const int64_t t0 = static_cast<int64_t>(blockIdx.y) * (16 * TM);
    const int64_t lines = a.d_in / LINE;
    const int64_t code_pitch = a.groups * (a.group / 2);
    const int line_groups_shift = PER > 1 ? 0 : 31 - __clz(a.group / LINE);  // lines a group, its log

    const uint8_t *code_row[NT];
    const uint16_t *scale_row[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        const int64_t n = n0 + 16 * i + nl < a.d_out ? n0 + 16 * i + nl : a.d_out - 1;
        code_row[i] = a.codes + n * code_pitch + 16 * kq;
        scale_row[i] = a.scale + n * a.groups;
    }
    auto load = [&](Line<NT, PER> &l, int64_t line) {
#pragma unroll
        for (int i = 0; i < NT; ++i) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const u32x4_t v = __builtin_nontemporal_load(
                    reinterpret_cast<const u32x4_t *>(code_row[i] + line * (LINE / 2) + 64 * h));
                l.c[i][h][0] = v.x; l.c[i][h][1] = v.y; l.c[i][h][2] = v.z; l.c[i][h][3] = v.w;
            }
            l.s[i].load(scale_row[i] + (PER > 1 ? line * PER : line >> line_groups_shift));
        }
    };
    // the line that the row ends in: nothing past the row's codes and scales
    auto load_tail = [&](Line<NT, PER> &l) {
#pragma unroll
        for (int i = 0; i < NT; ++i) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                u32x4_t v = {0u, 0u, 0u, 0u};
                if (lines * (LINE / 2) + 64 * h + 16 * kq < code_pitch)
                    v = *reinterpret_cast<const u32x4_t *>(code_row[i] + lines * (LINE / 2) + 64 * h);
                l.c[i][h][0] = v.x; l.c[i][h][1] = v.y; l.c[i][h][2] = v.z; l.c[i][h][3] = v.w;
            }
            if constexpr (PER > 1)
                l.s[i].load_some(scale_row[i] + lines * PER, a.groups - lines * PER);
            else
                l.s[i].load(scale_row[i] + (lines >> line_groups_shift));
        }
    };

    Line<NT, PER> ring[D];
    const int64_t mine = lines > wave ? (lines - wave + W - 1) / W : 0;
#pragma unroll
    for (int k = 0; k < D; ++k)
        if (k < mine)
            load(ring[k], wave + static_cast<int64_t>(k) * W);

    // the tokens
    const int64_t xpitch = (a.d_in + LINE - 1) / LINE * LINE + 8;  // in LDS
    const int tokens = static_cast<int>(a.T - t0 < 16 * TM ? a.T - t0 : 16 * TM);
    if constexpr (XLDS) {
        const int64_t vecs = xpitch / 8;
        for (int t = 0; t < tokens; ++t)
            for (int64_t v = threadIdx.x; v < vecs; v += W * 64) {
                Raw8<T> r;
                r.template load<true>(static_cast<const T *>(a.x) + (t0 + t) * a.d_in + v * 8,
                                      count8(a.d_in, v * 8));
                unsigned int w[P][4];
                split8(r, w);
#pragma unroll
                for (int p = 0; p < P; ++p)
                    *reinterpret_cast<u32x4_t *>(smem + ((p * tokens + t) * xpitch + v * 8) * 2) =
                        u32x4_t{w[p][0], w[p][1], w[p][2], w[p][3]};
            }
        __syncthreads();
    }
    const T *x_row[TM];
    const unsigned char *x_lds[TM];
#pragma unroll
    for (int i = 0; i < TM; ++i) {
        const int t = 16 * i + nl < tokens ? 16 * i + nl : tokens - 1;
        x_row[i] = static_cast<const T *>(a.x) + (t0 + t) * a.d_in + 8 * kq;
        x_lds[i] = smem + (t * xpitch + 8 * kq) * 2;
    }

    f32x4_t acc[TM][NT], part[TM][NT];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
            acc[i][j] = part[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};

    struct Half {
        Raw8<T> x[HALF][TM];
    };
    auto fetch = [&](Half &o, int64_t line, int h, bool tail) {
        if constexpr (!XLDS) {
#pragma unroll
            for (int s = 0; s < HALF; ++s)
#pragma unroll
                for (int i = 0; i < TM; ++i) {
                    const int64_t k = line * LINE + (h * HALF + s) * 32;
                    o.x[s][i].template load<true>(x_row[i] + k, tail ? count8(a.d_in, k + 8 * kq) : 8);
                }
        }
    };
    // half a line: the codes of register quad c, scales from the line's
    auto products = [&](Line<NT, PER> &l, const Half &x, int64_t line, int h) {
#pragma unroll
        for (int j = 0; j < NT; ++j)
            exchange4(l.c[j][h]);
#pragma unroll
        for (int s = 0; s < HALF; ++s) {
            bf16x8_t xs[TM][P];
#pragma unroll
            for (int i = 0; i < TM; ++i) {
                if constexpr (XLDS) {
                    const int64_t at = (line * LINE + (h * HALF + s) * 32) * 2;
#pragma unroll
                    for (int p = 0; p < P; ++p)
                        xs[i][p] = __builtin_bit_cast(
                            bf16x8_t, *reinterpret_cast<const u32x4_t *>(
                                          x_lds[i] + p * tokens * xpitch * 2 + at));
                } else {
                    unsigned int w[P][4];
                    split8(x.x[s][i], w);
#pragma unroll
                    for (int p = 0; p < P; ++p)
                        xs[i][p] = __builtin_bit_cast(bf16x8_t,
                                                      u32x4_t{w[p][0], w[p][1], w[p][2], w[p][3]});
                }
            }
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const bf16x8_t w = weights8(l.c[j][h][s]);
#pragma unroll
                for (int i = 0; i < TM; ++i)
#pragma unroll
                    for (int p = P - 1; p >= 0; --p)  // the smallest parts first
                        part[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xs[i][p], w, part[i][j],
                                                                             0, 0, 0);
            }
            // the end of a group (or of the line): its sums meet its scale
            constexpr int EVERY = STEPS / PER;
            const int step = h * HALF + s;
            if ((step + 1) % EVERY == 0) {
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    const float by = l.s[j].get(step / EVERY);
#pragma unroll
                    for (int i = 0; i < TM; ++i)
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            acc[i][j][q] = __fmaf_rn(by, part[i][j][q], acc[i][j][q]);
                            part[i][j][q] = 0.f;
                        }
                }
            }
        }
    };

    Half xa, xb;
    if (mine > 0)
        fetch(xa, wave, 0, false);
    for (int64_t k0 = 0; k0 < mine; k0 += D) {
#pragma unroll
        for (int d = 0; d < D; ++d) {
            const int64_t k = k0 + d;
            if (k < mine) {
                const int64_t line = wave + k * W;
                fetch(xb, line, 1, false);
                products(ring[d], xa, line, 0);
                if (k + 1 < mine)
                    fetch(xa, line + W, 0, false);
                products(ring[d], xb, line, 1);
                if (k + D < mine)
                    load(ring[d], line + static_cast<int64_t>(D) * W);
            }
        }
    }
    if (lines * LINE < a.d_in && lines % W == wave) {
        Line<NT, PER> l;
        load_tail(l);
        fetch(xa, lines, 0, true);
        products(l, xa, lines, 0);
        fetch(xb, lines, 1, true);
        products(l, xb, lines, 1);
    }

#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q)
                sums[wave][16 * i + 4 * kq + q][16 * j + nl] = acc[i][j][q];
    __syncthreads();
    for (int e = static_cast<int>(threadIdx.x); e < tokens * 16 * NT; e += W * 64) {
        const int m = e / (16 * NT), n = e % (16 * NT);
        if (n0 + n >= a.d_out)
            continue;
        float v = sums[0][m][n];
#pragma unroll
        for (int w = 1; w < W; ++w)
            v += sums[w][m][n];
        T *out = static_cast<T *>(a.y) + (t0 + m) * a.d_out + n0 + n;
        if constexpr (sizeof(T) == 2)
            *out = f32_to_bf16(v);
        else
            *out = v;
    }
}

template <typename T, int TM, int NT, int PER, bool XLDS, int W, int D>
hipError_t launch(const FourbitArgs &a, hipStream_t st)
{
    const int64_t xpitch = (a.d_in + LINE - 1) / LINE * LINE + 8;
    const size_t lds = XLDS ? static_cast<size_t>(planes<T> * a.T * xpitch * 2) : 0;
    const dim3 grid(static_cast<unsigned>((a.d_out + 16 * NT - 1) / (16 * NT)),
                    static_cast<unsigned>((a.T + 16 * TM - 1) / (16 * TM)));
    hipLaunchKernelGGL((linear_fourbit_kernel<T, TM, NT, PER, XLDS, W, D>), grid, dim3(W * 64), lds, st,
                       a);
    return hipGetLastError();
}

template <typename T, int PER>
hipError_t launch_per(const FourbitArgs &a, hipStream_t st)
{
    const int64_t xpitch = (a.d_in + LINE - 1) / LINE * LINE + 8;
    if (planes<T> * a.T * xpitch * 2 <= 64 * 1024 && a.T <= 4)
        return launch<T, 1, 2, PER, true, 4, 3>(a, st);
    if (a.T <= 16)
        return launch<T, 1, 4, PER, false, 4, 2>(a, st);
    return launch<T, 2, 2, PER, false, 4, 2>(a, st);
}

template <typename T>
hipError_t launch_any(const FourbitArgs &a, hipStream_t st)
{
    switch (a.group) {
    case 32: return launch_per<T, 8>(a, st);
    case 64: return launch_per<T, 4>(a, st);
    case 128: return launch_per<T, 2>(a, st);
    default: return launch_per<T, 1>(a, st);
    }
}

}  // namespace

hipError_t launch_linear_fourbit(int bf16, const FourbitArgs &a, hipStream_t st)
{
    if (a.T == 0)
        return hipSuccess;
    return bf16 ? launch_any<uint16_t>(a, st) : launch_any<float>(a, st);
}

}  // namespace dora
