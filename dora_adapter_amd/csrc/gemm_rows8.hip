// gemm_rows8.hip - dA = Q^T x of a bf16 module's backward from x's int8 rows
// (gfx950), with nothing rounded to bf16 on the way:
//   dA[i, j] = sum_t (Q[t, i] m) (2^e xq[t, j]),  xs[t, g(j)] = m 2^e
// An int8 value times a power of two is exact in bf16; what the token's scale has beside
// that, 1 to 2, goes to Q, which is still in fp32, and the product to a pair of bf16 (16
// bits of it).  Either operand keeps its own range.  Restoring x and storing Q
// in bf16 first, as the backward from a bf16 x does, rounds both: dA is then 0.0032
// of its norm off against 0.0024 here, where 0.0017 is its own last rounding
// and the rest dh's.
//
// The scale has to be one for all columns of a tile: one scale a row, or groups of
// whole tiles of 128 columns.
//
// 64 x 128 tiles of four waves (32 x 64 each), 64 tokens a step in two LDS buffers, the
// next step's loads in flight (two steps' took half as long again).  Both operands
// come MN-major; a thread writes two tokens of eight columns of Q, or four of x, as
// K-consecutive pairs.  K is split over workgroups; the fp32 sums go to slots that the
// caller adds in order.  r 384, 8192 tokens, 8192 columns: 204 us (505 TFLOP/s of the
// pair's products), bound by the conversions on the way to LDS (vector ALUs busy 0.6
// of the time, matrix cores a quarter), against 80 from an x and a Q in bf16 and 35
// for restoring that x: 2% of that backward, for 0.7 of dA's error.  r 37, 509 tokens,
// 1027 columns: 7 us.
#include "gemm_bf16_dma.hpp"
#include "gemm_rows8.hpp"
#include "rows8.hpp"

namespace dora {
namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

constexpr int BM = 64, BN = 128, BK = 64, NT = 256;
constexpr int AROWS = 2, BROWS = 4;  // tokens a thread holds of either operand
static_assert(BM / 8 * BK / AROWS == NT && BN / 8 * BK / BROWS == NT, "a chunk column a thread");
static_assert(BN == ROWS8_TILE, "a scale a tile");

// chunk c (8 K values) of row r of an operand: distinct banks for the reads of one
// chunk column and for the writes eight rows apart
__device__ __forceinline__ int place(int row, int c)
{
    return row * 8 + (c ^ ((row ^ (row >> 3)) & 7));
}

// A pair of bf16: v rounded, and what that left (at most 2^-8 of v; some number where
// v, or its rounding, is infinite or NaN, which the first of the pair then says).
__device__ __forceinline__ float rest_of(float v, float hi)
{
    return __builtin_amdgcn_fmed3f(v - hi, -0x1p121f, 0x1p121f);
}

// A scale as a number from 1 to 2 (0, NaN and infinities: itself) times a power of two.
__device__ __forceinline__ float mantissa(float s)
{
    return 2.f * __builtin_amdgcn_frexp_mantf(s);
}
__device__ __forceinline__ float power(float s)
{
    return __builtin_amdgcn_ldexpf(0.5f, __builtin_amdgcn_frexp_expf(s));
}

__global__ void __launch_bounds__(NT, 2) gemm_rows8_kernel(Rows8Args g)
{
    __shared__ __align__(16) uint4 lds[2][2 * BM * 8 + BN * 8];  // Q's pair, x
    const int tid = static_cast<int>(threadIdx.x), lane = tid & 63, wave = tid >> 6;
    const int wm = (wave >> 1) * 32, wn = (wave & 1) * 64;
    int tm, tn;
    tile_coords(g.r, g.d, BM, BN, tm, tn);
    const int64_t m0 = static_cast<int64_t>(tm) * BM, n0 = static_cast<int64_t>(tn) * BN;
    const int64_t groups = g.group ? (g.d + g.group - 1) / g.group : 1;
    const float *const xs = g.xs + (g.group ? n0 / g.group : 0);
    const int64_t kb = static_cast<int64_t>(blockIdx.y) * g.t_per_split;
    const int64_t ke = kb + g.t_per_split < g.T ? kb + g.t_per_split : g.T;

    // thread: columns 8 am .. of tokens AROWS ak .. of Q, 8 bm .. of BROWS bk .. of x
    const int am = tid & 7, ak = tid >> 3, bm = tid & 15, bk = tid >> 4;
    // columns past the end: a row's last eight, shifted into place (past all of them: any)
    const bool inside = n0 + BN <= g.d, tiny = g.d < 8;
    const int64_t col = n0 + bm * 8, from = col + 8 <= g.d || tiny ? col : g.d - 8;
    const int shift = 8 * static_cast<int>(col - from < 7 ? col - from : 7);
    struct Regs {
        float4 q[AROWS][2];
        float s[AROWS], sx[BROWS];
        Raw8i x[BROWS];
    } regs;
    // offsets of the thread's rows from a step's first
    int64_t qo[AROWS], xo[BROWS];
#pragma unroll
    for (int i = 0; i < AROWS; ++i)
        qo[i] = (ak * AROWS + i) * g.ldq + m0 + am * 8;
#pragma unroll
    for (int i = 0; i < BROWS; ++i)
        xo[i] = (bk * BROWS + i) * g.d + from;
    auto load = [&](int64_t k0) {
        if (!tiny && k0 + BK <= g.T) {
            const float *const q0 = g.q + k0 * g.ldq, *const s0 = xs + k0 * groups;
            const int8_t *const x0 = g.xq + k0 * g.d;
#pragma unroll
            for (int i = 0; i < AROWS; ++i) {
                regs.q[i][0] = reinterpret_cast<const float4 *>(q0 + qo[i])[0];
                regs.q[i][1] = reinterpret_cast<const float4 *>(q0 + qo[i])[1];
                regs.s[i] = s0[(ak * AROWS + i) * groups];
            }
#pragma unroll
            for (int i = 0; i < BROWS; ++i) {
                const u32x2_a1_t v = *reinterpret_cast<const u32x2_a1_t *>(x0 + xo[i]);
                regs.x[i].w[0] = v.x;
                regs.x[i].w[1] = v.y;
                regs.sx[i] = s0[(bk * BROWS + i) * groups];
            }
            return;
        }
        // (tokens past the end: the last one, whose Q is then taken as zeros)
#pragma unroll
        for (int i = 0; i < AROWS; ++i) {
            const int64_t k = k0 + ak * AROWS + i, t = k < g.T ? k : g.T - 1;
            const float4 *q = reinterpret_cast<const float4 *>(g.q + t * g.ldq + m0 + am * 8);
            regs.q[i][0] = q[0];
            regs.q[i][1] = q[1];
            regs.s[i] = xs[t * groups];
        }
#pragma unroll
        for (int i = 0; i < BROWS; ++i) {
            const int64_t k = k0 + bk * BROWS + i, t = k < g.T ? k : g.T - 1;
            const int8_t *x = g.xq + t * g.d + from;
            if (tiny) {
                regs.x[i].load(x, static_cast<int>(g.d - col));
            } else {
                const u32x2_a1_t v = *reinterpret_cast<const u32x2_a1_t *>(x);
                regs.x[i].w[0] = v.x;
                regs.x[i].w[1] = v.y;
            }
            regs.sx[i] = xs[t * groups];
        }
    };
    f32x4_t acc[2][4];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};

    int at = 0;
    if (kb < ke)
        load(kb);
    for (int64_t k0 = kb; k0 < ke; k0 += BK) {
        uint4 *const Hi = lds[at], *const Lo = Hi + BM * 8, *const X = Lo + BM * 8;
        float v[AROWS][8];
#pragma unroll
        for (int i = 0; i < AROWS; ++i) {
            const float m = mantissa(regs.s[i]);
            const float q[8] = {regs.q[i][0].x, regs.q[i][0].y, regs.q[i][0].z, regs.q[i][0].w,
                                regs.q[i][1].x, regs.q[i][1].y, regs.q[i][1].z, regs.q[i][1].w};
#pragma unroll
            for (int c = 0; c < 8; ++c)
                v[i][c] = q[c] * m;
        }
        if (k0 + BK > g.T) {
#pragma unroll
            for (int i = 0; i < AROWS; ++i)
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    v[i][c] = k0 + ak * AROWS + i < g.T ? v[i][c] : 0.f;
        }
        if (!inside && !tiny) {
#pragma unroll
            for (int i = 0; i < BROWS; ++i) {
                const uint64_t x = (static_cast<uint64_t>(regs.x[i].w[1]) << 32 | regs.x[i].w[0]) >> shift;
                regs.x[i].w[0] = static_cast<unsigned int>(x);
                regs.x[i].w[1] = static_cast<unsigned int>(x >> 32);
            }
        }
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            const uint32_t hi = pack_bf16x2(v[0][c], v[1][c]);
            const uint32_t lo = pack_bf16x2(rest_of(v[0][c], __uint_as_float(hi << 16)),
                                            rest_of(v[1][c], __uint_as_float(hi & 0xffff0000u)));
            const int to = place(am * 8 + c, ak / 4);
            reinterpret_cast<uint32_t *>(Hi + to)[ak % 4] = hi;
            reinterpret_cast<uint32_t *>(Lo + to)[ak % 4] = lo;
        }
        float p2[BROWS];
#pragma unroll
        for (int i = 0; i < BROWS; ++i)
            p2[i] = power(regs.sx[i]);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            const uint2 x = make_uint2(
                pack_bf16x2(regs.x[0].value(c) * p2[0], regs.x[1].value(c) * p2[1]),
                pack_bf16x2(regs.x[2].value(c) * p2[2], regs.x[3].value(c) * p2[3]));
            reinterpret_cast<uint2 *>(X + place(bm * 8 + c, bk / 2))[bk % 2] = x;
        }
        // (one barrier a step, bare: a wave past it is done with the other buffer, and
        // __syncthreads would wait for loads in flight as well)
        dma::wait_lgkm0();
        dma::stage_barrier();
        if (k0 + BK < ke)
            load(k0 + BK);
#pragma unroll
        for (int h = 0; h < BK / 32; ++h) {
            const int c = h * 4 + (lane >> 4);
            bf16x8_t fh[2], fl[2], fx[4];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                fh[i] = __builtin_bit_cast(bf16x8_t, Hi[place(wm + i * 16 + (lane & 15), c)]);
                fl[i] = __builtin_bit_cast(bf16x8_t, Lo[place(wm + i * 16 + (lane & 15), c)]);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
                fx[j] = __builtin_bit_cast(bf16x8_t, X[place(wn + j * 16 + (lane & 15), c)]);
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    acc[i][j] =
                        __builtin_amdgcn_mfma_f32_16x16x32_bf16(fh[i], fx[j], acc[i][j], 0, 0, 0);
                    acc[i][j] =
                        __builtin_amdgcn_mfma_f32_16x16x32_bf16(fl[i], fx[j], acc[i][j], 0, 0, 0);
                }
        }
        at ^= 1;
    }
    float *const out = g.slots + static_cast<int64_t>(blockIdx.y) * g.r * g.d;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            const int64_t m = m0 + wm + i * 16 + (lane >> 4) * 4 + v;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int64_t n = n0 + wn + j * 16 + (lane & 15);
                if (m < g.r && n < g.d)
                    out[m * g.d + n] = acc[i][j][v];
            }
        }
}

// Q = alpha sum_z part[z] ([splits][T, r]) in bf16 and, for the product above, in
// fp32 with zeros up to its pitch.  The sum and rounding of a Q stored in bf16 alone.
// A wave a row.
__global__ void __launch_bounds__(NT) q_rows8_kernel(const float *__restrict__ part, int splits,
                                                     int64_t T, int64_t r, int64_t ldq, float alpha,
                                                     uint16_t *__restrict__ Q,
                                                     float *__restrict__ Qf)
{
    const int lane = static_cast<int>(threadIdx.x) & 63;
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * (NT / 64) + (threadIdx.x >> 6); t < T;
         t += static_cast<int64_t>(gridDim.x) * (NT / 64))
        for (int64_t c = lane; c < ldq; c += 64) {
            float v = 0.f;
            if (c < r) {
                float acc = part[t * r + c];
                for (int z = 1; z < splits; ++z)
                    acc += part[(z * T + t) * r + c];
                v = alpha * acc;
                Q[t * r + c] = f32_to_bf16(v);
            }
            Qf[t * ldq + c] = v;
        }
}

}  // namespace

Rows8Plan plan_rows8(int64_t T, int64_t r, int64_t d)
{
    // rounds of two workgroups a CU, about 1.6 us a step, and the slots' writing and
    // reading; two steps a split at least
    const int64_t tiles = ((r + BM - 1) / BM) * ((d + BN - 1) / BN), steps = (T + BK - 1) / BK;
    int64_t per = steps;
    double best = -1.0;
    for (int64_t z = 1; z <= 32 && (z == 1 || 2 * z <= steps); ++z) {
        const int64_t n = (steps + z - 1) / z;
        const double us = 1.6 * static_cast<double>((tiles * z + 511) / 512 * n) +
                          static_cast<double>(z * r * d) * 8 / 4.0e6;
        if (best < 0 || us < best) {
            best = us;
            per = n;
        }
    }
    Rows8Plan p;
    p.splits = steps > 0 ? static_cast<int>((steps + per - 1) / per) : 0;
    p.t_per_split = per * BK;
    p.ldq = (r + BM - 1) / BM * BM;
    return p;
}

hipError_t launch_q_rows8(const float *part, int splits, int64_t T, int64_t r, int64_t ldq,
                          float alpha, void *Q, float *Qf, hipStream_t st)
{
    if (T == 0)
        return hipSuccess;
    const int64_t blocks = (T + NT / 64 - 1) / (NT / 64);
    hipLaunchKernelGGL(q_rows8_kernel, dim3(static_cast<unsigned>(blocks < 65536 ? blocks : 65536)),
                       dim3(NT), 0, st, part, splits, T, r, ldq, alpha, static_cast<uint16_t *>(Q), Qf);
    return hipGetLastError();
}

hipError_t launch_gemm_rows8(const Rows8Args &g, int splits, hipStream_t st)
{
    const int64_t tiles = ((g.r + BM - 1) / BM) * ((g.d + BN - 1) / BN);
    if (g.T == 0 || splits == 0)
        return hipSuccess;
    if (g.group % BN != 0 || tiles >= (int64_t(1) << 32) / NT)
        return hipErrorInvalidValue;
    hipLaunchKernelGGL(gemm_rows8_kernel,
                       dim3(static_cast<unsigned>(tiles), static_cast<unsigned>(splits)), dim3(NT), 0,
                       st, g);
    return hipGetLastError();
}

}  // namespace dora
