// newton_schulz.hip - matrices orthogonalised by Newton-Schulz steps, and the optimiser's step
// along them (gfx950).
//
// With X = U / (|U|_F + eps) (U or its transpose, so that X is [n, L] with n <= L) a step is
//     X <- P(G) X,   G = X X^T,   P(G) = a I + b G + c G^2.
// Every factor is a polynomial of the first G, so the steps run on n x n matrices alone,
//     Q <- P(G) Q,   G <- P(G) G P(G),
// between one product along L, G = U U^T, and another, O = Q U / (|U|_F + eps), whose epilogue is
// the update: 4 n^2 L flops instead of 4 n^2 L a step, and U is read twice.
//
// The n x n part is in 64 bits: G holds squares of singular values, so that an error of 2^-24 of
// its largest one would move the small ones' directions by 2^-24 / (2 sigma^2), where the
// literal steps in fp32 move them by about 2^-24 / sigma; with 2^-53 the fp32 product at
// the end is all that is left (measured against 64 bits: as far off as the literal steps).
// That product takes its operands as two bf16 numbers each (three for fp32 matrices), which
// hold 16 (24) bits, on the bf16 matrix cores with fp32 sums; so does G of bf16 matrices, whose
// output's 8 bits leave room for that (about 1e-4 of its norm), while G of fp32 matrices is formed
// in 64 bits.
//
// Up to 16 matrices share each launch.
#include "around.hpp"
#include "rows8.hpp"

namespace dora {
namespace {

typedef double f64x4_t __attribute__((ext_vector_type(4)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef unsigned int u32x4_t __attribute__((ext_vector_type(4)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef short s16x8_t __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) s16x4_t lds_s16x4;

constexpr int THREADS = 256;
constexpr int TILE = 64;       // Gram tile
constexpr int SMALL = 64;      // n x n matrices of one workgroup's LDS
constexpr int POLY = 32;       // tile of the n x n products
constexpr int POLY_WAVES = 8;  // which split their K

struct NsItem {
    NsMatrix m;
    int tall, np;        // rows > cols; the shorter side padded to 64 or to 128s
    int64_t rp, cp, lp;  // rows, columns and the longer side as padded (128s)
    char *u;             // U padded with zeros, [rp, cp]: bf16 hi and lo, or fp32
    unsigned int *tops;  // bf16: the largest |U| of each workgroup that wrote it, as bits
    int top_count;
    void *part;          // Gram partials [splits, np, np], tiles on and below the diagonal:
                         // fp32 (bf16 matrices) or fp64
    double *mat;         // G, P, Q, H [np, np] (larger matrices)
    double *scal;        // 1 / (|U|_F + eps)
    uint16_t *q;         // planes of Q / (|U|_F + eps), [planes, np, np]
    int splits;
    int64_t per_split;   // of L, a multiple of 128
};
constexpr int MAX_ITEMS = 16;
struct NsGroup {
    NsItem it[MAX_ITEMS];
    int start[MAX_ITEMS + 1];  // workgroups of the items before
    int count;
    NsParams p;
};
static_assert(sizeof(NsGroup) <= 4032, "a group must fit the kernel argument space");

__device__ __forceinline__ int find_item(const NsGroup &g, int block)
{
    int i = 0;
    while (i + 1 < g.count && block >= g.start[i + 1])
        ++i;
    return i;
}

// v as P bf16 numbers whose sum it is (to 16 bits with two of them, 24 with three)
template <int P>
__device__ __forceinline__ void split_planes(const float (&v)[8], u32x4_t (&w)[P])
{
    float r[8];
#pragma unroll
    for (int q = 0; q < 8; ++q)
        r[q] = v[q];
#pragma unroll
    for (int p = 0; p < P; ++p) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
            w[p][q] = pack_bf16x2(r[2 * q], r[2 * q + 1]);
        if (p + 1 < P) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                r[2 * q] -= __uint_as_float(w[p][q] << 16);
                r[2 * q + 1] -= __uint_as_float(w[p][q] & 0xffff0000u);
            }
        }
    }
}

// ------------------------------------------------------------- U and the momentum
constexpr int PREP_VPT = 4;
template <typename T>
__global__ void __launch_bounds__(THREADS) ns_prepare_kernel(NsGroup g)
{
    const NsItem &it = g.it[find_item(g, blockIdx.x)];
    const unsigned int block = blockIdx.x - g.start[find_item(g, blockIdx.x)];
    __shared__ unsigned int wave_top[THREADS / 64];
    unsigned int top = 0u;
    const unsigned int along = static_cast<unsigned int>(it.cp / 8);
    const unsigned int total = static_cast<unsigned int>(it.rp * it.cp / 8);
#pragma unroll
    for (int i = 0; i < PREP_VPT; ++i) {
        const unsigned int v = block * (THREADS * PREP_VPT) + i * THREADS + threadIdx.x;
        if (v >= total)
            break;
        const int64_t r = v / along, c = static_cast<int64_t>(v % along) * 8;
        float u[8];
#pragma unroll
        for (int q = 0; q < 8; ++q)
            u[q] = 0.f;
        const int cnt = r < it.m.rows ? count8(it.m.cols, c) : 0;
        if (cnt > 0) {
            const int64_t at = r * it.m.cols + c;
            Raw8<T> gr;
            gr.load(static_cast<const T *>(it.m.g) + at, cnt);
            gr.get(u);
            if (it.m.m != nullptr) {
                Raw8<float> mr;
                mr.load(it.m.m + at, cnt);
                float m[8];
                mr.get(m);
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    m[q] = __fmaf_rn(g.p.mu, m[q], u[q]);
                    u[q] = g.p.nesterov ? __fmaf_rn(g.p.mu, m[q], u[q]) : m[q];
                }
                mr.set(m);
                mr.store(it.m.m_out + at, cnt);
            }
        }
        const int64_t at = static_cast<int64_t>(v) * 8;
        if constexpr (sizeof(T) == 2) {
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                const unsigned int b = abs_bits(u[q]);
                top = top > b ? top : b;
            }
            u32x4_t w[2];
            split_planes(u, w);
            uint16_t *const h = reinterpret_cast<uint16_t *>(it.u) + at;
            *reinterpret_cast<u32x4_t *>(h) = w[0];
            *reinterpret_cast<u32x4_t *>(h + it.rp * it.cp) = w[1];
        } else {
            float *const o = reinterpret_cast<float *>(it.u) + at;
#pragma unroll
            for (int k = 0; k < 2; ++k)
                *reinterpret_cast<f32x4_t *>(o + 4 * k) =
                    f32x4_t{u[4 * k], u[4 * k + 1], u[4 * k + 2], u[4 * k + 3]};
        }
    }
    if constexpr (sizeof(T) == 2) {
        top = lane_max(top, 64);
        if ((threadIdx.x & 63) == 0)
            wave_top[threadIdx.x >> 6] = top;
        __syncthreads();
        if (threadIdx.x == 0) {
            for (int w = 1; w < THREADS / 64; ++w)
                top = top > wave_top[w] ? top : wave_top[w];
            it.tops[block] = top;
        }
    }
}

// The power of two that brings a bf16 matrix's largest |U| near one, where its squares (or theirs
// of what is 2^-24 as large) would leave fp32's range; else 1.  Called by whole workgroups.
__device__ __forceinline__ float range_scale(const NsItem &it, unsigned int *red)
{
    unsigned int top = 0u;
    for (int i = threadIdx.x; i < it.top_count; i += blockDim.x) {
        const unsigned int b = it.tops[i];
        top = top > b ? top : b;
    }
    top = block_max(top, red, static_cast<int>(blockDim.x) >> 6);
    const int e = static_cast<int>(top >> 23) - 127;
    if (top == 0u || e == 128 || (e > -30 && e < 40))
        return 1.f;
    // (2^-e; |e| is at most 127)
    return __uint_as_float(static_cast<unsigned int>(e == 127 ? 1 : 127 - e) << 23);
}

// ------------------------------------------------------------------- G = U U^T
// fp32 matrices: 64 x 64 tiles on and below the diagonal, four waves of 32 x 32, 32 values of L
// at a time straight into registers.  An MFMA takes four of them: of a wide matrix a lane's
// eight consecutive ones give it one each time, of a tall one they are four rows.
__global__ void __launch_bounds__(THREADS) ns_gram_f64_kernel(NsGroup g)
{
    const int item = find_item(g, blockIdx.x);
    const NsItem &it = g.it[item];
    const int nt = it.np / TILE, tiles = nt * (nt + 1) / 2;
    const int block = static_cast<int>(blockIdx.x) - g.start[item];
    const int z = block / tiles;
    int t = block % tiles, ti = 0;
    while (t > ti) {
        t -= ti + 1;
        ++ti;
    }
    const int tj = t;  // t <= ti
    const int lane = static_cast<int>(threadIdx.x) & 63, wave = static_cast<int>(threadIdx.x) >> 6;
    const int lr = lane & 15, kq = lane >> 4;
    const int i0 = ti * TILE + 32 * (wave >> 1), j0 = tj * TILE + 32 * (wave & 1);
    const int64_t k0 = z * it.per_split, k1 = k0 + it.per_split < it.lp ? k0 + it.per_split : it.lp;
    const float *const f = reinterpret_cast<const float *>(it.u);

    f64x4_t acc[2][2];
#pragma unroll
    for (int a = 0; a < 2; ++a)
#pragma unroll
        for (int b = 0; b < 2; ++b)
            acc[a][b] = f64x4_t{0., 0., 0., 0.};
    // the operand of 16 rows from r0: v[s] for MFMA step s of the 32 values from k
    auto operand = [&](float (&v)[8], int r0, int64_t k) {
        if (!it.tall) {
            const int64_t at = (r0 + lr) * it.cp + k + 8 * kq;
            const f32x4_t x = *reinterpret_cast<const f32x4_t *>(f + at),
                          y = *reinterpret_cast<const f32x4_t *>(f + at + 4);
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                v[s] = x[s];
                v[4 + s] = y[s];
            }
        } else {
#pragma unroll
            for (int s = 0; s < 8; ++s)
                v[s] = f[(k + 4 * s + kq) * it.cp + r0 + lr];
        }
    };
    // (the next 32 values on their way)
    float a[2][2][8], b[2][2][8];
    auto fetch = [&](int to, int64_t k) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            operand(a[to][q], i0 + 16 * q, k);
            operand(b[to][q], j0 + 16 * q, k);
        }
    };
    fetch(0, k0);
    for (int64_t k = k0; k < k1; k += 64) {  // (whole 128s)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int64_t next = k + 32 * half + 32;
            fetch(half ^ 1, next < k1 ? next : k0);
#pragma unroll
            for (int s = 0; s < 8; ++s)
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int y = 0; y < 2; ++y)
                        acc[x][y] = __builtin_amdgcn_mfma_f64_16x16x4f64(
                            static_cast<double>(a[half][x][s]), static_cast<double>(b[half][y][s]),
                            acc[x][y], 0, 0, 0);
        }
    }
    double *const out = static_cast<double *>(it.part) + static_cast<int64_t>(z) * it.np * it.np;
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int y = 0; y < 2; ++y)
#pragma unroll
            for (int q = 0; q < 4; ++q)
                out[static_cast<int64_t>(i0 + 16 * x + 4 * q + kq) * it.np + j0 + 16 * y + lr] =
                    acc[x][y][q];
}

// LDS tiles of one plane: 64 K values of R rows of the shorter side, as rows of K values 144 bytes
// apart (16 of them at one chunk on distinct banks), or, where the matrix lies the other way,
// as 64 rows of R values (four rows of 32 bytes on distinct banks), read by transposing loads.
template <int R>
struct Tiles {
    static constexpr int KP = 144, MP = R == 128 ? 288 : 160;
    static constexpr int K_BYTES = R * KP, M_BYTES = 64 * MP;
    // operands of 32 K values (h: the first or the second half of the stage) of 16 rows from r0
    __device__ __forceinline__ static bf16x8_t rows16(const unsigned char *tile, int r0, int h, int lane)
    {
        return __builtin_bit_cast(bf16x8_t, *reinterpret_cast<const u32x4_t *>(
                                                tile + (r0 + (lane & 15)) * KP + 64 * h + 16 * (lane >> 4)));
    }
    __device__ __forceinline__ static bf16x8_t columns16(const unsigned char *tile, int c0, int h, int lane)
    {
        const int lr = lane & 15, kq = lane >> 4;
        const unsigned char *const p =
            tile + (32 * h + 8 * kq + (lr >> 2)) * MP + (c0 + 4 * (lr & 3)) * 2;
        const s16x4_t x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(p));
        const s16x4_t y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(p + 4 * MP));
        return __builtin_bit_cast(bf16x8_t, __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7));
    }
};

// bf16 matrices: both planes of both operands, all four products, in fp32 over a share of L (the
// shares are added in 64 bits).  NB x NB tiles on and below the diagonal, eight waves (4 x 2),
// 64 values of L a stage, the next one on its way.
constexpr int WAVES8 = 512;
template <bool TALL, int NB>
__global__ void __launch_bounds__(WAVES8) ns_gram_kernel(NsGroup g)
{
    using Tl = Tiles<NB>;
    constexpr int BYTES = TALL ? Tl::M_BYTES : Tl::K_BYTES;
    constexpr int TM = NB / 64, TN = NB / 32;       // 16 x 16 blocks of a wave
    constexpr int V = NB * 8 / WAVES8;              // 16-byte chunks of a plane a thread
    __shared__ __align__(16) unsigned char sa[2][BYTES], sb[2][BYTES];
    __shared__ unsigned int red[WAVES8 / 64];
    const int item = find_item(g, blockIdx.x);
    const NsItem &it = g.it[item];
    const int nt = it.np / NB, tiles = nt * (nt + 1) / 2;
    const int block = static_cast<int>(blockIdx.x) - g.start[item];
    const int z = block / tiles;
    int t = block % tiles, ti = 0;
    while (t > ti) {
        t -= ti + 1;
        ++ti;
    }
    const int i0 = ti * NB, j0 = t * NB;
    const bool diagonal = i0 == j0;
    const int tid = static_cast<int>(threadIdx.x), lane = tid & 63, wave = tid >> 6;
    const int wm = wave >> 1, wn = wave & 1;
    const int64_t k0 = z * it.per_split, k1 = k0 + it.per_split < it.lp ? k0 + it.per_split : it.lp;
    const int64_t usize = it.rp * it.cp;
    const float scale = range_scale(it, red);

    u32x4_t ra[V][2], rb[V][2];
    auto fetch = [&](u32x4_t (&r)[V][2], int r0, int64_t k) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int v = tid + i * WAVES8;
            const int64_t at = TALL ? (k + v / (NB / 8)) * it.cp + r0 + v % (NB / 8) * 8
                                    : (r0 + v / 8) * it.cp + k + v % 8 * 8;
#pragma unroll
            for (int p = 0; p < 2; ++p)
                r[i][p] = *reinterpret_cast<const u32x4_t *>(reinterpret_cast<const uint16_t *>(it.u) +
                                                             p * usize + at);
        }
    };
    auto keep = [&](const u32x4_t (&r)[V][2], unsigned char (&to)[2][BYTES]) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int v = tid + i * WAVES8;
            const int at = TALL ? v / (NB / 8) * Tl::MP + v % (NB / 8) * 16 : v / 8 * Tl::KP + v % 8 * 16;
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                u32x4_t w = r[i][p];
                if (scale != 1.f) {
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        w[q] = pack_bf16x2(scale * __uint_as_float(w[q] << 16),
                                           scale * __uint_as_float(w[q] & 0xffff0000u));
                }
                *reinterpret_cast<u32x4_t *>(&to[p][at]) = w;
            }
        }
    };
    f32x4_t acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
            acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    auto operand = [&](const unsigned char *tile, int r0, int h) {
        if constexpr (TALL)
            return Tl::columns16(tile, r0, h, lane);
        else
            return Tl::rows16(tile, r0, h, lane);
    };
    unsigned char(*const other)[BYTES] = diagonal ? sa : sb;
    fetch(ra, i0, k0);
    if (!diagonal)
        fetch(rb, j0, k0);
    for (int64_t k = k0; k < k1; k += 64) {
        __syncthreads();
        keep(ra, sa);
        if (!diagonal)
            keep(rb, sb);
        __syncthreads();
        if (k + 64 < k1) {
            fetch(ra, i0, k + 64);
            if (!diagonal)
                fetch(rb, j0, k + 64);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            bf16x8_t a[TM][2], b[TN][2];
#pragma unroll
            for (int p = 0; p < 2; ++p) {
#pragma unroll
                for (int i = 0; i < TM; ++i)
                    a[i][p] = operand(sa[p], wm * (NB / 4) + 16 * i, h);
#pragma unroll
                for (int j = 0; j < TN; ++j)
                    b[j][p] = operand(other[p], wn * (NB / 2) + 16 * j, h);
            }
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int j = 0; j < TN; ++j)
#pragma unroll
                    for (int s = 3; s >= 0; --s)  // the small products first
                        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[j][s & 1], a[i][s >> 1],
                                                                            acc[i][j], 0, 0, 0);
        }
    }
    // a lane holds row lr and four consecutive columns of each block
    float *const out = static_cast<float *>(it.part) + static_cast<int64_t>(z) * it.np * it.np;
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
            *reinterpret_cast<f32x4_t *>(
                out + static_cast<int64_t>(i0 + wm * (NB / 4) + 16 * i + (lane & 15)) * it.np + j0 +
                wn * (NB / 2) + 16 * j + 4 * (lane >> 4)) = acc[i][j];
}

// The sum of the Gram partials at place e, and what a range scale took from it.
template <bool F32>
__device__ __forceinline__ double gram_at(const NsItem &it, int64_t size, int64_t e, double back)
{
    double s = 0.;
    if constexpr (F32) {
        const double *const p = static_cast<const double *>(it.part);
#pragma unroll 8
        for (int z = 0; z < it.splits; ++z)
            s += p[z * size + e];
    } else {
        const float *const p = static_cast<const float *>(it.part);
#pragma unroll 8
        for (int z = 0; z < it.splits; ++z)
            s += static_cast<double>(p[z * size + e]);
    }
    return s * back;
}

// ------------------------------------------------------- the n x n part, n <= 64
// One workgroup a matrix, everything in LDS: bound by one CU's 64-bit matrix rate, so that only
// tiles on and below the diagonal are formed (16 x 16, as many as n has), and a single product's
// waves split K in two, which balances them over the SIMDs.
constexpr int SP = SMALL + 4;  // pitch
template <int PLANES>
__global__ void __launch_bounds__(1024) ns_small_kernel(NsGroup g)
{
    constexpr bool F32 = PLANES == 3;
    constexpr int UNITS = 20;  // tiles of two products, or of one by half its K
    __shared__ double m[4][SMALL][SP];
    __shared__ double half[10][16][17];
    __shared__ unsigned int red[16];
    double(*G)[SP] = m[0], (*P)[SP] = m[1], (*Q)[SP] = m[2], (*H)[SP] = m[3];
    const NsItem &it = g.it[blockIdx.x];
    const int tid = static_cast<int>(threadIdx.x), lane = tid & 63, wave = tid >> 6;
    const int lr = lane & 15, kq = lane >> 4;
    const int n = static_cast<int>(it.tall ? it.m.cols : it.m.rows);
    const int nt = (n + 15) / 16, tiles = nt * (nt + 1) / 2, K = 16 * nt;
    double back = 1.;
    if constexpr (!F32) {
        const double scale = range_scale(it, red);
        back = 1. / (scale * scale);
    }
    {
        double v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            v[i] = gram_at<F32>(it, SMALL * SMALL, tid + i * 1024, back);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            G[(tid + i * 1024) / SMALL][tid % SMALL] = v[i];
    }
    __syncthreads();
    double trace = 0.;
    for (int i = 0; i < K; ++i)
        trace += G[i][i];
    const double inv = 1. / (sqrt(trace) + static_cast<double>(g.p.eps));
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i)
        G[(tid + i * 1024) / SMALL][tid % SMALL] *= inv * inv;
    __syncthreads();
    auto tile_of = [](int t, int &i0, int &j0) {
        int ti = 0;
        while (t > ti) {
            t -= ti + 1;
            ++ti;
        }
        i0 = 16 * ti;
        j0 = 16 * t;
    };
    // rows i0.. of X against rows j0.. of Y (symmetric), K values from k0 to k1
    auto product = [&](double(*X)[SP], double(*Y)[SP], int i0, int j0, int k0, int k1) {
        f64x4_t acc = {0., 0., 0., 0.};
        for (int k = k0; k < k1; k += 8) {
#pragma unroll
            for (int s = 0; s < 8; s += 4)
                acc = __builtin_amdgcn_mfma_f64_16x16x4f64(X[i0 + lr][k + s + kq], Y[j0 + lr][k + s + kq],
                                                           acc, 0, 0, 0);
        }
        return acc;
    };
    auto place = [&](double(*Z)[SP], int i0, int j0, const f64x4_t &v) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int i = i0 + 4 * q + kq, j = j0 + lr;
            if (j <= i) {
                Z[i][j] = v[q];
                Z[j][i] = v[q];
            }
        }
    };
    // (a wave takes units wave and wave + 16)
    auto one = [&](double(*X)[SP], double(*Y)[SP], double(*Z)[SP], bool poly) {
        f64x4_t acc[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int u = wave + 16 * r;
            int i0, j0;
            tile_of(u < tiles ? u : u - tiles, i0, j0);
            if (u < 2 * tiles)
                acc[r] = product(X, Y, i0, j0, u < tiles ? 0 : K / 2, u < tiles ? K / 2 : K);
            if (u >= tiles && u < 2 * tiles)
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    half[u - tiles][4 * q + kq][lr] = acc[r][q];
        }
        __syncthreads();
        if (wave < tiles) {
            int i0, j0;
            tile_of(wave, i0, j0);
            f64x4_t v;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                v[q] = acc[0][q] + half[wave][4 * q + kq][lr];
                if (poly) {
                    const int i = i0 + 4 * q + kq, j = j0 + lr;
                    v[q] = (i == j ? static_cast<double>(g.p.a) : 0.) +
                           static_cast<double>(g.p.b) * X[i][j] + static_cast<double>(g.p.c) * v[q];
                }
            }
            place(Z, i0, j0, v);
        }
        __syncthreads();
    };
    auto copy = [&](double(*from)[SP], double(*to)[SP]) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            to[(tid + i * 1024) / SMALL][tid % SMALL] = from[(tid + i * 1024) / SMALL][tid % SMALL];
        __syncthreads();
    };
    for (int step = 0; step < g.p.steps; ++step) {
        const bool first = step == 0, last = step + 1 == g.p.steps;
        one(G, G, P, true);
        if (first) {
            copy(P, Q);
            if (!last)
                one(P, G, H, false);
        } else if (last) {
            one(P, Q, H, false);
            copy(H, Q);
        } else {
            // H = P G and Q = P Q at once
            f64x4_t acc[2];
            static_assert(UNITS <= 32, "two units a wave");
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int u = wave + 16 * r;
                int i0, j0;
                tile_of(u < tiles ? u : u - tiles, i0, j0);
                if (u < 2 * tiles)
                    acc[r] = product(P, u < tiles ? G : Q, i0, j0, 0, K);
            }
            __syncthreads();
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int u = wave + 16 * r;
                int i0, j0;
                tile_of(u < tiles ? u : u - tiles, i0, j0);
                if (u < 2 * tiles)
                    place(u < tiles ? H : Q, i0, j0, acc[r]);
            }
            __syncthreads();
        }
        if (!last)
            one(H, P, G, false);
    }
    if (tid < SMALL * SMALL / 8) {
        const int i = tid / (SMALL / 8), j = tid % (SMALL / 8) * 8;
        float v[8];
#pragma unroll
        for (int q = 0; q < 8; ++q)  // (zeros past n's tiles: U is zero there, too)
            v[q] = i < K && j + q < K ? static_cast<float>(Q[i][j + q] * inv) : 0.f;
        u32x4_t w[PLANES];
        split_planes(v, w);
#pragma unroll
        for (int p = 0; p < PLANES; ++p)
            *reinterpret_cast<u32x4_t *>(it.q + (p * SMALL + i) * SMALL + j) = w[p];
    }
}

// ------------------------------------------------------- the n x n part, larger
template <bool F32>
__global__ void __launch_bounds__(THREADS) ns_gram_sum_kernel(NsGroup g)
{
    __shared__ unsigned int red[THREADS / 64];
    const int item = find_item(g, blockIdx.x);
    const NsItem &it = g.it[item];
    const int64_t size = static_cast<int64_t>(it.np) * it.np;
    double back = 1.;
    if constexpr (!F32) {
        const double scale = range_scale(it, red);
        back = 1. / (scale * scale);
    }
    const int64_t e = (static_cast<int64_t>(blockIdx.x) - g.start[item]) * THREADS + threadIdx.x;
    const int i = static_cast<int>(e / it.np), j = static_cast<int>(e % it.np);
    if (i >= it.np || j > i)
        return;
    const double s = gram_at<F32>(it, size, e, back);
    it.mat[e] = s;
    it.mat[static_cast<int64_t>(j) * it.np + i] = s;
}

// One product of symmetric matrices, 32 x 32 tiles on and below the diagonal, mirrored:
//   0  P = a I + b G + c G G    1  H = P G, and Q = P Q    2  G = H P    3  Q = P Q
// (Q in the first step: P).  G is not scaled in place: the first step's products take it by
// 1 / |U|^2, which is formed from its diagonal.  Matrices 4 and 5 are the other G and Q.
template <int OP>
__global__ void __launch_bounds__(POLY_WAVES * 64) ns_poly_kernel(NsGroup g, int step)
{
    __shared__ double red[POLY_WAVES][POLY][POLY + 1];
    __shared__ double tr[POLY_WAVES];
    const int item = find_item(g, blockIdx.x);
    const NsItem &it = g.it[item];
    const int np = it.np, nt = np / POLY, tiles = nt * (nt + 1) / 2;
    int tj = static_cast<int>(blockIdx.x) - g.start[item];
    const bool second = tj >= tiles;  // Q's tiles behind H's
    tj -= second ? tiles : 0;
    int ti = 0;
    while (tj > ti) {
        tj -= ti + 1;
        ++ti;
    }
    const int64_t size = static_cast<int64_t>(np) * np;
    double *const G = it.mat + (step & 1 ? 4 * size : 0), *const G2 = it.mat + (step & 1 ? 0 : 4 * size);
    double *const P = it.mat + size, *const H = it.mat + 3 * size;
    double *const Q = it.mat + (step & 1 ? 5 : 2) * size, *const Q2 = it.mat + (step & 1 ? 2 : 5) * size;
    const double *X, *Y;
    double *out;
    if constexpr (OP == 0) {
        X = Y = G;
        out = P;
    } else if constexpr (OP == 1) {
        X = P;
        Y = second ? Q : G;
        out = second ? Q2 : H;
    } else if constexpr (OP == 2) {
        X = H;
        Y = P;
        out = G2;
    } else {
        X = P;
        Y = Q;
        out = Q2;
    }
    const int tid = static_cast<int>(threadIdx.x), lane = tid & 63, wave = tid >> 6;
    const int lr = lane & 15, kq = lane >> 4, i0 = ti * POLY, j0 = tj * POLY;

    // the first G's scale
    double inv = 1.;
    if (step == 0 && OP == 0) {
        double s = 0.;
        for (int i = tid; i < np; i += POLY_WAVES * 64)
            s += G[static_cast<int64_t>(i) * np + i];
#pragma unroll
        for (int d = 32; d > 0; d >>= 1)
            s += __shfl_xor(s, d);
        if (lane == 0)
            tr[wave] = s;
        __syncthreads();
        s = tr[0];
        for (int w = 1; w < POLY_WAVES; ++w)
            s += tr[w];
        inv = 1. / (sqrt(s) + static_cast<double>(g.p.eps));
        if (ti == 0 && tid == 0)
            *it.scal = inv;
    } else if (step == 0) {
        inv = *it.scal;
    }

    f64x4_t acc[2][2];
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int y = 0; y < 2; ++y)
            acc[x][y] = f64x4_t{0., 0., 0., 0.};
    // 16 values of K a turn (np is whole turns of the waves), four consecutive ones a lane; three
    // turns' loads at once: another CU wrote them, and each wait is one for its cache
    constexpr int TURN = 16 * POLY_WAVES, AHEAD = 3;
    for (int k0 = 16 * wave; k0 < np; k0 += AHEAD * TURN) {
        f64x4_t a[AHEAD][2], b[AHEAD][2];
#pragma unroll
        for (int t = 0; t < AHEAD; ++t) {
            const int k = k0 + t * TURN < np ? k0 + t * TURN : k0;
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                a[t][q] = *reinterpret_cast<const f64x4_t *>(
                    X + static_cast<int64_t>(i0 + 16 * q + lr) * np + k + 4 * kq);
                b[t][q] = *reinterpret_cast<const f64x4_t *>(
                    Y + static_cast<int64_t>(j0 + 16 * q + lr) * np + k + 4 * kq);
            }
        }
#pragma unroll
        for (int t = 0; t < AHEAD; ++t) {
            if (k0 + t * TURN >= np)
                break;
#pragma unroll
            for (int s = 0; s < 4; ++s)
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int y = 0; y < 2; ++y)
                        acc[x][y] = __builtin_amdgcn_mfma_f64_16x16x4f64(a[t][x][s], b[t][y][s],
                                                                         acc[x][y], 0, 0, 0);
        }
    }
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int y = 0; y < 2; ++y)
#pragma unroll
            for (int q = 0; q < 4; ++q)
                red[wave][16 * x + 4 * q + kq][16 * y + lr] = acc[x][y][q];
    __syncthreads();
    for (int e = tid; e < POLY * POLY; e += POLY_WAVES * 64) {
        const int i = e / POLY, j = e % POLY;
        double s = red[0][i][j];
#pragma unroll
        for (int w = 1; w < POLY_WAVES; ++w)
            s += red[w][i][j];
        const int64_t at = static_cast<int64_t>(i0 + i) * np + j0 + j;
        if constexpr (OP == 0) {
            const double i2 = inv * inv;
            s = static_cast<double>(g.p.b) * (i2 * G[at]) + static_cast<double>(g.p.c) * (i2 * i2 * s);
            if (i0 + i == j0 + j)
                s += static_cast<double>(g.p.a);
        } else if constexpr (OP == 1) {
            if (!second)
                s *= inv * inv;
        }
        if (j0 + j <= i0 + i) {
            out[at] = s;
            out[static_cast<int64_t>(j0 + j) * np + i0 + i] = s;
            if constexpr (OP == 0) {
                if (step == 0) {  // the first Q
                    Q2[at] = s;
                    Q2[static_cast<int64_t>(j0 + j) * np + i0 + i] = s;
                }
            }
        }
    }
}

// the planes of Q / (|U|_F + eps)
template <int PLANES>
__global__ void __launch_bounds__(THREADS) ns_q_planes_kernel(NsGroup g)
{
    const int item = find_item(g, blockIdx.x);
    const NsItem &it = g.it[item];
    const int64_t size = static_cast<int64_t>(it.np) * it.np;
    const double *const Q = it.mat + ((g.p.steps & 1) ? 5 : 2) * size, inv = *it.scal;
    const int64_t e = ((static_cast<int64_t>(blockIdx.x) - g.start[item]) * THREADS + threadIdx.x) * 8;
    if (e >= size)
        return;
    float v[8];
#pragma unroll
    for (int q = 0; q < 8; ++q)
        v[q] = static_cast<float>(Q[e + q] * inv);
    u32x4_t w[PLANES];
    split_planes(v, w);
#pragma unroll
    for (int p = 0; p < PLANES; ++p)
        *reinterpret_cast<u32x4_t *>(it.q + p * size + e) = w[p];
}

// ------------------------------------------------------------- O = Q U (or U Q)
// Tiles of NB values of the shorter side by 128 of the longer one, eight waves (4 x 2), 64 values
// of K (the shorter side) a stage, the next one on its way.
template <typename T, bool TALL, int NB>
__global__ void __launch_bounds__(WAVES8) ns_final_kernel(NsGroup g)
{
    constexpr int P = sizeof(T) == 2 ? 2 : 3;
    constexpr int BM = TALL ? 128 : NB, BN = TALL ? NB : 128;
    using Tq = Tiles<NB>;
    using Tu = Tiles<128>;
    constexpr int KP = Tu::KP, MP = Tu::MP;
    constexpr int Q_ROWS = NB, Q_BYTES = Tq::K_BYTES, U_BYTES = TALL ? Tu::K_BYTES : Tu::M_BYTES;
    constexpr int TM = BM / 64, TN = BN / 32;  // 16 x 16 blocks of a wave
    __shared__ __align__(16) unsigned char qs[P][Q_BYTES], us[P][U_BYTES];
    const int item = find_item(g, blockIdx.x);
    const NsItem &it = g.it[item];
    const int block = static_cast<int>(blockIdx.x) - g.start[item];
    const int nb = it.np / NB;
    // (the tiles of one stretch of the longer side next to each other: they read the same U)
    const int n0 = (block % nb) * NB;
    const int64_t l0 = static_cast<int64_t>(block / nb) * 128;
    const int tid = static_cast<int>(threadIdx.x), lane = tid & 63, wave = tid >> 6;
    const int lr = lane & 15, kq = lane >> 4, wm = wave >> 1, wn = wave & 1;
    const int np = it.np;
    const int64_t qsize = static_cast<int64_t>(np) * np, usize = it.rp * it.cp;

    constexpr int QV = Q_ROWS * 8 / WAVES8, UV = 128 * 8 / WAVES8;  // 16-byte chunks a thread
    u32x4_t qr[QV][P];
    Raw8<float> uf[UV];
    u32x4_t up[UV][2];
    auto u_at = [&](int v, int k) {  // row-major place of chunk v of the stage at k
        if constexpr (TALL)
            return (l0 + v / 8) * it.cp + k + v % 8 * 8;
        else
            return static_cast<int64_t>(k + v / 16) * it.cp + l0 + v % 16 * 8;
    };
    auto fetch = [&](int k) {
#pragma unroll
        for (int i = 0; i < QV; ++i) {
            const int v = tid + i * WAVES8;
#pragma unroll
            for (int p = 0; p < P; ++p)
                qr[i][p] = *reinterpret_cast<const u32x4_t *>(
                    it.q + p * qsize + static_cast<int64_t>(n0 + v / 8) * np + k + v % 8 * 8);
        }
#pragma unroll
        for (int i = 0; i < UV; ++i) {
            const int64_t at = u_at(tid + i * WAVES8, k);
            if constexpr (P == 3) {
                uf[i].template load<true>(reinterpret_cast<const float *>(it.u) + at, 8);
            } else {
#pragma unroll
                for (int p = 0; p < 2; ++p)
                    up[i][p] = *reinterpret_cast<const u32x4_t *>(
                        reinterpret_cast<const uint16_t *>(it.u) + p * usize + at);
            }
        }
    };
    auto keep = [&]() {
#pragma unroll
        for (int i = 0; i < QV; ++i) {
            const int v = tid + i * WAVES8;
#pragma unroll
            for (int p = 0; p < P; ++p)
                *reinterpret_cast<u32x4_t *>(&qs[p][v / 8 * KP + v % 8 * 16]) = qr[i][p];
        }
#pragma unroll
        for (int i = 0; i < UV; ++i) {
            const int v = tid + i * WAVES8;
            u32x4_t w[P];
            if constexpr (P == 3) {
                float f[8];
                uf[i].get(f);
                split_planes(f, w);
            } else {
                w[0] = up[i][0];
                w[1] = up[i][1];
            }
#pragma unroll
            for (int p = 0; p < P; ++p)
                *reinterpret_cast<u32x4_t *>(
                    &us[p][TALL ? v / 8 * KP + v % 8 * 16 : v / 16 * MP + v % 16 * 16]) = w[p];
        }
    };
    f32x4_t acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
            acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    fetch(0);
    for (int k = 0; k < np; k += 64) {
        __syncthreads();
        keep();
        __syncthreads();
        if (k + 64 < np)
            fetch(k + 64);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            bf16x8_t a[TM][P], b[TN][P];
#pragma unroll
            for (int p = 0; p < P; ++p) {
#pragma unroll
                for (int i = 0; i < TM; ++i)
                    a[i][p] = TALL ? Tu::rows16(us[p], wm * (BM / 4) + 16 * i, h, lane)
                                   : Tq::rows16(qs[p], wm * (BM / 4) + 16 * i, h, lane);
#pragma unroll
                for (int j = 0; j < TN; ++j)
                    b[j][p] = TALL ? Tq::rows16(qs[p], wn * (BN / 2) + 16 * j, h, lane)
                                   : Tu::columns16(us[p], wn * (BN / 2) + 16 * j, h, lane);
            }
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int j = 0; j < TN; ++j)
#pragma unroll
                    for (int s = P - 1; s >= 0; --s)  // planes x and s - x, the small ones first
#pragma unroll
                        for (int x = 0; x <= s; ++x)
                            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[j][s - x], a[i][x],
                                                                                acc[i][j], 0, 0, 0);
        }
    }
    // a lane holds row lr and four consecutive columns of each block
    const int64_t m0 = (TALL ? l0 : n0) + wm * (BM / 4), c0 = (TALL ? n0 : l0) + wn * (BN / 2);
    const bool aligned = it.m.cols % 4 == 0;
#pragma unroll
    for (int i = 0; i < TM; ++i) {
        const int64_t r = m0 + 16 * i + lr;
        if (r >= it.m.rows)
            continue;
#pragma unroll
        for (int j = 0; j < TN; ++j) {
            const int64_t c = c0 + 16 * j + 4 * kq, at = r * it.m.cols + c;
            const T *const p = static_cast<const T *>(it.m.p) + at;
            T *const o = static_cast<T *>(it.m.out) + at;
            float v[4], w[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                v[q] = acc[i][j][q];
                w[q] = 0.f;
            }
            if (aligned && c < it.m.cols) {
                if constexpr (sizeof(T) == 2) {
                    if (it.m.p != nullptr) {
                        const uint2 u = *reinterpret_cast<const uint2 *>(p);
                        w[0] = __uint_as_float(u.x << 16);
                        w[1] = __uint_as_float(u.x & 0xffff0000u);
                        w[2] = __uint_as_float(u.y << 16);
                        w[3] = __uint_as_float(u.y & 0xffff0000u);
                    }
                } else if (it.m.p != nullptr) {
                    const f32x4_t u = *reinterpret_cast<const f32x4_t *>(p);
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        w[q] = u[q];
                }
            } else if (it.m.p != nullptr) {
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    if (c + q < it.m.cols) {
                        if constexpr (sizeof(T) == 2)
                            w[q] = __uint_as_float(static_cast<unsigned int>(p[q]) << 16);
                        else
                            w[q] = p[q];
                    }
            }
            if (it.m.p != nullptr) {
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    v[q] = __fmaf_rn(-it.m.step, v[q], it.m.keep * w[q]);
            }
            if (aligned && c < it.m.cols) {
                if constexpr (sizeof(T) == 2)
                    *reinterpret_cast<uint2 *>(o) =
                        make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
                else
                    *reinterpret_cast<f32x4_t *>(o) = f32x4_t{v[0], v[1], v[2], v[3]};
            } else {
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    if (c + q < it.m.cols) {
                        if constexpr (sizeof(T) == 2)
                            o[q] = f32_to_bf16(v[q]);
                        else
                            o[q] = v[q];
                    }
            }
        }
    }
}

// ------------------------------------------------------------------- planning
int64_t up_to(int64_t v, int64_t of) { return (v + of - 1) / of * of; }

// The padded sides of a matrix.
struct Sides {
    bool tall;
    int64_t np, lp, rp, cp;
};
Sides sides(int64_t rows, int64_t cols)
{
    Sides s;
    s.tall = rows > cols;
    const int64_t n = s.tall ? cols : rows, l = s.tall ? rows : cols;
    s.np = n <= SMALL ? SMALL : up_to(n, 128);
    s.lp = up_to(l, 128);
    s.rp = s.tall ? s.lp : s.np;
    s.cp = s.tall ? s.np : s.lp;
    return s;
}

// Matrices [first, first + count) of one set of launches: up to 16, in 256 MiB (or one).
struct Chunk {
    int first, count;
    size_t bytes;
    NsItem it[MAX_ITEMS];
};
constexpr size_t CHUNK_BYTES = size_t(256) << 20;

int64_t gram_tile(int bf16, int64_t np) { return bf16 && np > SMALL ? 128 : 64; }
int64_t prepare_groups(int64_t rp, int64_t cp)
{
    return (rp * cp / 8 + THREADS * PREP_VPT - 1) / (THREADS * PREP_VPT);
}

Chunk plan_chunk(int bf16, const NsMatrix *mats, int count, int first, char *ws)
{
    Chunk c;
    c.first = first;
    c.count = 0;
    c.bytes = 0;
    auto fill = [&](NsItem &it, const NsMatrix &m, size_t off, int share) {
        const Sides s = sides(m.rows, m.cols);
        it.m = m;
        it.tall = s.tall;
        it.np = static_cast<int>(s.np);
        it.rp = s.rp;
        it.cp = s.cp;
        it.lp = s.lp;
        // about 512 workgroups for the Gram products of the set (1024 in 64 bits, of four
        // waves), of 128 values of L each at least
        const int64_t nt = s.np / gram_tile(bf16, s.np), tiles = nt * (nt + 1) / 2;
        int64_t z = (bf16 ? 512 : 1024) / (tiles * share);
        z = z < 1 ? 1 : z > 32 ? 32 : z;
        it.per_split = up_to((s.lp + z - 1) / z, 128);
        it.splits = static_cast<int>((s.lp + it.per_split - 1) / it.per_split);
        auto take = [&](size_t bytes) {
            const size_t at = off;
            off += (bytes + 255) / 256 * 256;
            return ws + at;
        };
        const size_t square = static_cast<size_t>(s.np) * s.np;
        it.u = take(static_cast<size_t>(s.rp) * s.cp * 4);
        it.top_count = bf16 ? static_cast<int>(prepare_groups(s.rp, s.cp)) : 0;
        it.tops = reinterpret_cast<unsigned int *>(take(it.top_count * sizeof(unsigned int)));
        it.part = take(it.splits * square * (bf16 ? 4 : 8));
        it.mat = reinterpret_cast<double *>(take(s.np > SMALL ? 6 * square * 8 : 0));
        it.scal = reinterpret_cast<double *>(take(8));
        it.q = reinterpret_cast<uint16_t *>(take((bf16 ? 2 : 3) * square * 2));
        return off;
    };
    // how many matrices share the set decides their splits: count them at the most splits first
    size_t off = 0;
    while (first + c.count < count && c.count < MAX_ITEMS) {
        NsItem it;
        const size_t next = fill(it, mats[first + c.count], off, 1);
        if (c.count > 0 && next > CHUNK_BYTES)
            break;
        off = next;
        ++c.count;
    }
    off = 0;
    for (int i = 0; i < c.count; ++i)
        off = fill(c.it[i], mats[first + i], off, c.count);
    c.bytes = off;
    return c;
}

// The items of a chunk that `take` picks, with `blocks` workgroups each.
template <typename Take, typename Blocks>
int group_of(NsGroup &g, const Chunk &c, Take &&take, Blocks &&blocks)
{
    g.count = 0;
    int at = 0;
    for (int i = 0; i < c.count; ++i) {
        if (!take(c.it[i]))
            continue;
        g.it[g.count] = c.it[i];
        g.start[g.count++] = at;
        at += static_cast<int>(blocks(c.it[i]));
    }
    g.start[g.count] = at;
    return at;
}

template <typename T>
hipError_t run_chunk(const Chunk &c, const NsParams &p, hipStream_t st)
{
    constexpr bool F32 = sizeof(T) == 4;
    constexpr int PLANES = F32 ? 3 : 2;
    NsGroup g;
    g.p = p;
    auto all = [](const NsItem &) { return true; };
    auto small = [](const NsItem &i) { return i.np == SMALL; };
    auto large = [](const NsItem &i) { return i.np > SMALL; };
#define NS_LAUNCH(...)                         \
    do {                                       \
        hipLaunchKernelGGL(__VA_ARGS__);       \
        const hipError_t e_ = hipGetLastError(); \
        if (e_ != hipSuccess)                  \
            return e_;                         \
    } while (0)
    int n = group_of(g, c, all, [](const NsItem &i) { return prepare_groups(i.rp, i.cp); });
    NS_LAUNCH((ns_prepare_kernel<T>), dim3(n), dim3(THREADS), 0, st, g);
    auto gram_groups = [](const NsItem &i) {
        const int64_t nt = i.np / gram_tile(!F32, i.np);
        return nt * (nt + 1) / 2 * i.splits;
    };
    if constexpr (F32) {
        n = group_of(g, c, all, gram_groups);
        NS_LAUNCH(ns_gram_f64_kernel, dim3(n), dim3(THREADS), 0, st, g);
    } else {
        for (int kind = 0; kind < 4; ++kind) {
            const bool tall = kind & 1, big = kind & 2;
            n = group_of(g, c, [&](const NsItem &i) { return (i.tall != 0) == tall && (i.np > SMALL) == big; },
                         gram_groups);
            if (n == 0)
                continue;
            if (tall && big)
                NS_LAUNCH((ns_gram_kernel<true, 128>), dim3(n), dim3(WAVES8), 0, st, g);
            else if (tall)
                NS_LAUNCH((ns_gram_kernel<true, 64>), dim3(n), dim3(WAVES8), 0, st, g);
            else if (big)
                NS_LAUNCH((ns_gram_kernel<false, 128>), dim3(n), dim3(WAVES8), 0, st, g);
            else
                NS_LAUNCH((ns_gram_kernel<false, 64>), dim3(n), dim3(WAVES8), 0, st, g);
        }
    }
    n = group_of(g, c, small, [](const NsItem &) { return 1; });
    if (n > 0)
        NS_LAUNCH((ns_small_kernel<PLANES>), dim3(n), dim3(1024), 0, st, g);
    n = group_of(g, c, large, [](const NsItem &i) {
        return (static_cast<int64_t>(i.np) * i.np + THREADS - 1) / THREADS;
    });
    if (n > 0) {
        NS_LAUNCH((ns_gram_sum_kernel<F32>), dim3(n), dim3(THREADS), 0, st, g);
        auto tiles = [](const NsItem &i) {
            return static_cast<int64_t>(i.np / POLY) * (i.np / POLY + 1) / 2;
        };
        const dim3 block(POLY_WAVES * 64);
        for (int s = 0; s < p.steps; ++s) {
            const bool first = s == 0, last = s + 1 == p.steps;
            n = group_of(g, c, large, tiles);
            NS_LAUNCH((ns_poly_kernel<0>), dim3(n), block, 0, st, g, s);
            if (last) {
                if (!first)
                    NS_LAUNCH((ns_poly_kernel<3>), dim3(n), block, 0, st, g, s);
                continue;
            }
            // (the first Q is P)
            const int each = first ? 1 : 2;
            n = group_of(g, c, large, [&](const NsItem &i) { return each * tiles(i); });
            NS_LAUNCH((ns_poly_kernel<1>), dim3(n), block, 0, st, g, s);
            n = group_of(g, c, large, tiles);
            NS_LAUNCH((ns_poly_kernel<2>), dim3(n), block, 0, st, g, s);
        }
        n = group_of(g, c, large, [](const NsItem &i) {
            return (static_cast<int64_t>(i.np) * i.np / 8 + THREADS - 1) / THREADS;
        });
        NS_LAUNCH((ns_q_planes_kernel<PLANES>), dim3(n), dim3(THREADS), 0, st, g);
    }
    for (int tall = 0; tall < 2; ++tall)
        for (int wide_n = 0; wide_n < 2; ++wide_n) {
            n = group_of(g, c,
                         [&](const NsItem &i) { return i.tall == tall && (i.np > SMALL) == wide_n; },
                         [](const NsItem &i) {
                             return i.lp / 128 * (i.np > SMALL ? i.np / 128 : 1);
                         });
            if (n == 0)
                continue;
            if (tall && wide_n)
                NS_LAUNCH((ns_final_kernel<T, true, 128>), dim3(n), dim3(WAVES8), 0, st, g);
            else if (tall)
                NS_LAUNCH((ns_final_kernel<T, true, 64>), dim3(n), dim3(WAVES8), 0, st, g);
            else if (wide_n)
                NS_LAUNCH((ns_final_kernel<T, false, 128>), dim3(n), dim3(WAVES8), 0, st, g);
            else
                NS_LAUNCH((ns_final_kernel<T, false, 64>), dim3(n), dim3(WAVES8), 0, st, g);
        }
#undef NS_LAUNCH
    return hipSuccess;
}

}  // namespace

bool newton_schulz_fits(int64_t rows, int64_t cols)
{
    const Sides s = sides(rows, cols);
    // (32-bit places of eight values, and workgroups of a launch)
    return s.np <= NS_MAX_SHORT && s.rp <= (int64_t(1) << 33) / s.cp;
}

size_t newton_schulz_workspace(int bf16, const NsMatrix *mats, int count)
{
    size_t most = 0;
    for (int first = 0; first < count;) {
        const Chunk c = plan_chunk(bf16, mats, count, first, nullptr);
        most = c.bytes > most ? c.bytes : most;
        first += c.count;
    }
    return most;
}

hipError_t launch_newton_schulz(int bf16, const NsMatrix *mats, int count, const NsParams &p, void *ws,
                                hipStream_t st)
{
    for (int first = 0; first < count;) {
        const Chunk c = plan_chunk(bf16, mats, count, first, static_cast<char *>(ws));
        const hipError_t e = bf16 ? run_chunk<uint16_t>(c, p, st) : run_chunk<float>(c, p, st);
        if (e != hipSuccess)
            return e;
        first += c.count;
    }
    return hipSuccess;
}

}  // namespace dora
