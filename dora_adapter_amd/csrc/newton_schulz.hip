// newton_schulz.hip - matrices orthogonalised by Newton-Schulz steps, and the optimiser's step
// along them (gfx950).
//
// With X = U / (|U|_F + eps) (U or its transpose, so that X is [n, L] with n <= L) a step is
//     X <- P(G) X,   G = X X^T,   P(G) = a I + b G + c G^2.
// Every factor is a polynomial of the first G, so the steps run on n x n matrices alone,
//     Q <- P(G) Q,   G <- P(G) G P(G),
// between one product along L, G = U U^T, and another, O = Q U / (|U|_F + eps), whose epilogue is
// the update: 4 n^2 L flops instead of 4 n^2 L a step, and U is read twice.  Where n comes near L
// that is a loss (4096 x 4096, five steps: 28.9 ms, the literal steps in fp32 14.5; 1024 x 8192 1.0
// against 1.6).
//
// G holds squares of singular values, so that an error of 2^-24 of its largest one would move the
// small ones' directions by 2^-24 / (2 sigma^2), where the literal steps in fp32 move them by
// about 2^-24 / sigma.  Worse, an eigenvalue that it takes below zero is multiplied by a^2 a
// step, as U U^T's cannot be, and leaves the range where the polynomial is bounded: with G in
// 32 bits that is seven steps of the quintic for a matrix of low rank.  So G and the n x n part
// are in 64 bits, for matrices of either type, and the product at the end is all that is left
// (against 64 bits a quarter of the literal fp32 steps' error at full rank, 0.6 to 0.85 of it at low
// ones); it takes Q and U as three bf16 numbers each, which hold 24 bits, on the bf16 matrix cores with
// fp32 sums.
//
// Up to 40 matrices share each launch.  Measured: a step of the factors 384 x 8192 and 28672 x 384
// in bf16 432 us (eighteen launches), of fourteen 64 x 4096 and fourteen 4096 x 64 98 us
// (three), 37 x 1027 in fp32 37 us (three).  (G, the n x n part and the planes of bf16 matrices at
// 16 to 24 bits took 229 and 90 us, and are not right for a low rank: see above.)
#include <algorithm>
#include <climits>
#include <cmath>
#include <type_traits>

#include "around.hpp"
#include "rows8.hpp"

namespace dora {
namespace {

typedef double f64x4_t __attribute__((ext_vector_type(4)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef unsigned int u32x4_t __attribute__((ext_vector_type(4)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4_t lds_s16x4;

constexpr int THREADS = 256;
constexpr int TILE = 64;       // Gram tiles
constexpr int SMALL = 64;      // n x n matrices of one workgroup's LDS
constexpr int POLY = 32;       // tile of the n x n products
constexpr int POLY_WAVES = 8;  // which split their K

// A matrix as its kernels see it.
struct NsItem {
    float *u;      // U padded with zeros, [rp, cp]
    double *part;  // Gram partials [splits, np, np], tiles on and below the diagonal
    double *mat;   // G, P, Q, H and the other G and Q [np, np] (larger matrices)
    double *scal;  // what makes the planes of Q, the first G of U U^T, and what U meets
    uint16_t *q;   // planes of Q / (|U|_F + eps) times a power of two, [3, np, np]
    int n, np;     // the shorter side, padded to 64 or to 128s
    int tall;      // rows > cols
    int rp, cp;    // rows and columns as padded (the longer side to 128s)
    int splits, per_split;  // of the longer side, a multiple of 64
    float lift;             // of G's diagonal
};
struct NsInput {  // what the first kernel reads and writes
    float *u;
    double *part;
    const void *g;
    const float *m;
    float *m_out;
    int64_t rows, cols;
    int rp, cp, tall, per_split;
};
struct NsOutput {  // what the last kernel reads and writes
    const float *u;
    const uint16_t *q;
    const double *scal;
    const void *p;
    void *out;
    int64_t rows, cols;
    float step, keep;
    int np, tall, rp, cp;
};
constexpr int MAX_ITEMS = 40;
template <typename I>
struct NsGroup {
    I it[MAX_ITEMS];
    int start[MAX_ITEMS];  // workgroups of the items before; behind the last item INT_MAX
    NsParams p;
};
static_assert(sizeof(NsGroup<NsItem>) <= 4000 && sizeof(NsGroup<NsInput>) <= 4000 &&
                  sizeof(NsGroup<NsOutput>) <= 4000,
              "a group must fit the kernel argument space");

// The item of a workgroup and its place among that item's workgroups.  Each lane reads one item and
// where it starts, so that there is one round trip to the arguments, which no cache holds yet
// (a scalar search makes two, and 1.2 us of a kernel's 7).
template <typename I>
struct Found {
    I it;
    int block;
};
template <typename I>
__device__ __forceinline__ Found<I> find_item(const NsGroup<I> &g, int block)
{
    constexpr int WORDS = sizeof(I) / 4;
    struct Words {
        int w[WORDS];
    };
    const int lane = static_cast<int>(threadIdx.x) & 63, k = lane < MAX_ITEMS ? lane : MAX_ITEMS - 1;
    const int start = g.start[k];
    const Words mine = *reinterpret_cast<const Words *>(&g.it[k]);
    const int i = __popcll(__ballot(lane < MAX_ITEMS && block >= start)) - 1;
    Words one;
#pragma unroll
    for (int q = 0; q < WORDS; ++q)
        one.w[q] = __builtin_amdgcn_readlane(mine.w[q], i);
    return Found<I>{__builtin_bit_cast(I, one), block - __builtin_amdgcn_readlane(start, i)};
}

// A launch's workgroups go round the eight XCDs.  This gives each of them consecutive places, so
// that the tiles that read the same stretch of U share an L2.
__device__ __forceinline__ int place_on_xcd()
{
    const int n = static_cast<int>(gridDim.x), b = static_cast<int>(blockIdx.x);
    const int xcd = b & 7, each = n >> 3, more = n & 7;
    return xcd * each + (xcd < more ? xcd : more) + (b >> 3);
}

// 1 / (|U|_F + eps), and the power of two that goes from it to U where one of them is so far from
// one that its planes would leave fp32's range (O is Q times it times U): half of the way from
// one to the other, so that both keep their bits where U lies far below eps, too.  Of zeros O is
// zeros whatever eps, 0 too.
struct NormScale {
    double inv;  // of |U|_F + eps
    int s;
    __device__ __forceinline__ static double power(int e)
    {
        return __hiloint2double((1023 + e) << 20, 0);
    }
    __device__ __forceinline__ double for_q() const { return inv * power(s); }
    __device__ __forceinline__ double for_u() const { return power(-s); }
};
__device__ __forceinline__ NormScale norm_scale(double norm, double eps)
{
    // (zero -1023, infinity and NaN 1024)
    auto exponent = [](double v) { return ((__double2hiint(v) >> 20) & 0x7ff) - 1023; };
    const double t = norm + eps;
    const int en = exponent(norm), et = exponent(t), e = (en + et) / 2;
    NormScale n;
    n.inv = norm == 0. ? 0. : 1. / t;
    n.s = en < -1000 || et > 1000 || (en > -60 && et < 60) ? 0 : e < -126 ? -126 : e > 126 ? 126 : e;
    return n;
}

// the row of an fp64 product's register q (its column is lane % 16)
__device__ __forceinline__ int d_row(int q, int lane) { return 4 * q + (lane >> 4); }
__device__ __forceinline__ f64x4_t mfma4(double a, double b, f64x4_t c)
{
    return __builtin_amdgcn_mfma_f64_16x16x4f64(a, b, c, 0, 0, 0);
}

// v as three bf16 numbers whose sum it is, to 24 bits
constexpr int PLANES = 3;
__device__ __forceinline__ void split_planes(const float (&v)[8], u32x4_t (&w)[PLANES])
{
    float r[8];
#pragma unroll
    for (int q = 0; q < 8; ++q)
        r[q] = v[q];
#pragma unroll
    for (int p = 0; p < PLANES; ++p) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
            w[p][q] = pack_bf16x2(r[2 * q], r[2 * q + 1]);
        if (p + 1 < PLANES) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                r[2 * q] -= __uint_as_float(w[p][q] << 16);
                r[2 * q + 1] -= __uint_as_float(w[p][q] & 0xffff0000u);
            }
        }
    }
}

// the next eight of the fp32 numbers of U
__device__ __forceinline__ void put_u(float *o, const float (&u)[8])
{
#pragma unroll
    for (int k = 0; k < 2; ++k)
        *reinterpret_cast<f32x4_t *>(o + 4 * k) = f32x4_t{u[4 * k], u[4 * k + 1], u[4 * k + 2], u[4 * k + 3]};
}

// ------------------------------------------------------------- U and the momentum
// Bound by memory traffic: 6 bytes an element in, 8 out (14.2 million in bf16: 42 us, 4.7 TB/s).
constexpr int PREP_VPT = 4;
template <typename T>
__global__ void __launch_bounds__(THREADS) ns_prepare_kernel(NsGroup<NsInput> g)
{
    const Found<NsInput> found = find_item(g, blockIdx.x);
    const NsInput &it = found.it;
    const unsigned int block = found.block;
    const unsigned int along = static_cast<unsigned int>(it.cp / 8);
    const int64_t usize = static_cast<int64_t>(it.rp) * it.cp;
    const unsigned int total = static_cast<unsigned int>(usize / 8);
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
        const int cnt = r < it.rows ? count8(it.cols, c) : 0;
        if (cnt > 0) {
            const int64_t at = r * it.cols + c;
            Raw8<T> gr;
            gr.load(static_cast<const T *>(it.g) + at, cnt);
            gr.get(u);
            if (it.m != nullptr) {
                Raw8<float> mr;
                mr.load(it.m + at, cnt);
                float m[8];
                mr.get(m);
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    m[q] = __fmaf_rn(g.p.mu, m[q], u[q]);
                    u[q] = g.p.nesterov ? __fmaf_rn(g.p.mu, m[q], u[q]) : m[q];
                }
                mr.set(m);
                mr.store(it.m_out + at, cnt);
            }
        }
        put_u(it.u + static_cast<int64_t>(v) * 8, u);
    }
}

// ------------------------------------------------------------------- G = U U^T
// 64 x 64 tiles on and below the diagonal, four waves of 32 x 32, 32 values of L
// at a time straight into registers.  An MFMA takes four of them: of a wide matrix a lane's
// eight consecutive ones give it one each time, of a tall one they are four rows.  Bound by the
// matrix cores' 64-bit rate (72 TFLOP/s in a large product; 384 x 8192 and 28672 x 384: 6.3 GFLOP of
// tiles in 152 us).
__global__ void __launch_bounds__(THREADS) ns_gram_kernel(NsGroup<NsItem> g)
{
    const Found<NsItem> found = find_item(g, place_on_xcd());
    const NsItem &it = found.it;
    const int nt = it.np / TILE, tiles = nt * (nt + 1) / 2;
    const int block = found.block;
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
    const int64_t lp = it.tall ? it.rp : it.cp, k0 = static_cast<int64_t>(z) * it.per_split,
                  k1 = k0 + it.per_split < lp ? k0 + it.per_split : lp;
    const float *const f = it.u;

    f64x4_t acc[2][2];
#pragma unroll
    for (int a = 0; a < 2; ++a)
#pragma unroll
        for (int b = 0; b < 2; ++b)
            acc[a][b] = f64x4_t{0., 0., 0., 0.};
    // the operand of 16 rows from r0: v[s] for MFMA step s of the 32 values from k
    auto operand = [&](float (&v)[8], int r0, int64_t k) {
        if (!it.tall) {
            const int64_t at = static_cast<int64_t>(r0 + lr) * it.cp + k + 8 * kq;
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
    for (int64_t k = k0; k < k1; k += 64) {  // (whole 64s)
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
                        acc[x][y] = mfma4(static_cast<double>(a[half][x][s]),
                                          static_cast<double>(b[half][y][s]), acc[x][y]);
        }
    }
    double *const out = it.part + static_cast<int64_t>(z) * it.np * it.np;
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int y = 0; y < 2; ++y)
#pragma unroll
            for (int q = 0; q < 4; ++q)
                out[static_cast<int64_t>(i0 + 16 * x + d_row(q, lane)) * it.np + j0 + 16 * y + lr] =
                    acc[x][y][q];
}

// ------------------------------------------------- U and its Gram partial, n <= 64
// A workgroup has all rows of a stretch of the longer side, so that it forms U, writes it for the
// last kernel and multiplies it from LDS at once; 128 values of the longer side a turn.  28
// matrices of 64 x 4096 in bf16: 35 us for 103 MB, the 64-bit products between the turns' loads.
struct FrontLds {
    static constexpr int K = 128;
    // rows of K values (four places of 16 rows on distinct banks) or K rows of n values (four
    // rows of 16)
    static constexpr int KP = K + 4, MP = SMALL + 16;
    static constexpr int BYTES = (SMALL * KP > K * MP ? SMALL * KP : K * MP) * 4;
};
constexpr int FRONT = 512;
template <typename T, bool TALL>
__device__ __forceinline__ void front_stretch(const NsInput &it, const NsParams &p, int block,
                                              float *lds)
{
    using L = FrontLds;
    constexpr int V = SMALL * L::K / 8 / FRONT;
    const int tid = static_cast<int>(threadIdx.x), lane = tid & 63, wave = tid >> 6;
    const int lr = lane & 15, kq = lane >> 4;
    const int64_t lp = TALL ? it.rp : it.cp, k0 = static_cast<int64_t>(block) * it.per_split,
                  k1 = k0 + it.per_split < lp ? k0 + it.per_split : lp;
    const int n = static_cast<int>(TALL ? it.cols : it.rows), nt = (n + 15) / 16;
    const int64_t l = TALL ? it.rows : it.cols;

    // tiles wave and wave + 8 on and below the diagonal
    f64x4_t acc[2];
#pragma unroll
    for (int r = 0; r < 2; ++r)
        acc[r] = f64x4_t{0., 0., 0., 0.};
    auto tile_of = [](int t, int &i0, int &j0) {
        const int ti = (t >= 1 ? 1 : 0) + (t >= 3 ? 1 : 0) + (t >= 6 ? 1 : 0);
        i0 = 16 * ti;
        j0 = 16 * (t - ti * (ti + 1) / 2);
    };
    for (int64_t k = k0; k < k1; k += L::K) {
        const int kc = static_cast<int>(k1 - k < L::K ? k1 - k : L::K);  // whole 64s
        // place of chunk v of eight: row and column in the matrix
        auto place = [&](int v, int64_t &r, int64_t &c) {
            r = TALL ? k + v / 8 : v / (L::K / 8);
            c = TALL ? v % 8 * 8 : k + v % (L::K / 8) * 8;
        };
        auto inside = [&](int v) { return TALL ? v / 8 < kc : v % (L::K / 8) * 8 < kc; };
        auto lds_at = [&](int v) {
            return TALL ? v / 8 * L::MP + v % 8 * 8 : v / (L::K / 8) * L::KP + v % (L::K / 8) * 8;
        };
        Raw8<T> gr[V];
        Raw8<float> mr[V];
        int cnt[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int v = tid + i * FRONT;
            int64_t r, c;
            place(v, r, c);
            cnt[i] = inside(v) && r < it.rows ? count8(it.cols, c) : 0;
        }
        // no chunk that a row's end cuts: all loads at once (no branch round one), from the
        // matrix's start where there is nothing
        const bool whole = TALL ? n % 8 == 0 : k + kc <= l || l % 8 == 0;
        if (whole) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                int64_t r, c;
                place(tid + i * FRONT, r, c);
                const int64_t at = cnt[i] > 0 ? r * it.cols + c : 0;
                gr[i].load(static_cast<const T *>(it.g) + at, 8);
                if (it.m != nullptr)
                    mr[i].load(it.m + at, 8);
            }
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                int64_t r, c;
                place(tid + i * FRONT, r, c);
                const int64_t at = r * it.cols + c;
                gr[i].load(static_cast<const T *>(it.g) + at, cnt[i]);
                if (it.m != nullptr)
                    mr[i].load(it.m + at, cnt[i]);
            }
        }
        if (k > k0)
            __syncthreads();  // (the last turn's tiles)
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int v = tid + i * FRONT;
            if (!inside(v))
                continue;
            int64_t r, c;
            place(v, r, c);
            float u[8];
            gr[i].get(u);
            if (it.m != nullptr) {
                float m[8];
                mr[i].get(m);
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    m[q] = __fmaf_rn(p.mu, m[q], u[q]);
                    u[q] = p.nesterov ? __fmaf_rn(p.mu, m[q], u[q]) : m[q];
                }
                if (cnt[i] > 0) {
                    mr[i].set(m);
                    mr[i].store(it.m_out + r * it.cols + c, cnt[i]);
                }
            }
            if (cnt[i] <= 0)
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    u[q] = 0.f;
            put_u(it.u + r * it.cp + c, u);
            put_u(lds + lds_at(v), u);
        }
        __syncthreads();
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int t = wave + 8 * r;
            if (t >= nt * (nt + 1) / 2)
                continue;
            int i0, j0;
            tile_of(t, i0, j0);
            for (int kk = 0; kk < kc; kk += 16) {
                float a[4], b[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int at = kk + 4 * q + kq;
                    a[q] = TALL ? lds[at * L::MP + i0 + lr] : lds[(i0 + lr) * L::KP + at];
                    b[q] = TALL ? lds[at * L::MP + j0 + lr] : lds[(j0 + lr) * L::KP + at];
                }
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    acc[r] = mfma4(static_cast<double>(a[q]), static_cast<double>(b[q]), acc[r]);
            }
        }
    }
    double *const out = it.part + block * SMALL * SMALL;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const int t = wave + 8 * r;
        if (t >= nt * (nt + 1) / 2)
            continue;
        int i0, j0;
        tile_of(t, i0, j0);
#pragma unroll
        for (int q = 0; q < 4; ++q)
            out[(i0 + d_row(q, lane)) * SMALL + j0 + lr] = acc[r][q];
    }
}

template <typename T>
__global__ void __launch_bounds__(FRONT, 2) ns_front_kernel(NsGroup<NsInput> g)
{
    __shared__ __align__(16) float lds[FrontLds::BYTES / 4];
    const Found<NsInput> found = find_item(g, blockIdx.x);
    if (found.it.tall)
        front_stretch<T, true>(found.it, g.p, found.block, lds);
    else
        front_stretch<T, false>(found.it, g.p, found.block, lds);
}

// The sums of the Gram partials at N places from e, in row i from column j on.  The diagonal is
// lifted by more than G's own rounding may take from its eigenvalues: 64 bits leave some of a
// matrix of low rank at -2^-56 or so of its norm, and sixteen steps take those out of the
// polynomial's range (16 x 333 of rank 1: O 180 times its size).  The rounding of a row and a column
// goes by the root of their diagonal elements' product, so that a share of each of those makes up
// for it, however far apart they are.  (An O that depends on singular values so small is
// lost to 24 bits of U in any case.)
template <int N>
__device__ __forceinline__ void gram_at(const NsItem &it, int64_t e, int i, int j, double (&s)[N])
{
    typedef double vec_t __attribute__((ext_vector_type(N)));
    const double *const p = it.part + e;
    const int64_t size = static_cast<int64_t>(it.np) * it.np;
#pragma unroll
    for (int q = 0; q < N; ++q)
        s[q] = 0.;
#pragma unroll 8
    for (int z = 0; z < it.splits; ++z) {
        const vec_t v = *reinterpret_cast<const vec_t *>(p + z * size);
#pragma unroll
        for (int q = 0; q < N; ++q)
            s[q] += v[q];
    }
#pragma unroll
    for (int q = 0; q < N; ++q)
        s[q] += i == j + q ? s[q] * static_cast<double>(it.lift) : 0.;
}

// ------------------------------------------------------- the n x n part, n <= 64
// One workgroup a matrix, everything in LDS; a wave for each 16 x 16 tile on and below the
// diagonal, whose operands are all on their way before the first product.  Bound by the latency of
// the chain, 14 products of five steps: 1.4 us each at n = 37; 28 matrices of n = 64 in 41 us.
template <int NT>
struct SmallLds {
    static constexpr int PITCH = 16 * NT + 2;  // 16 bytes of 16 rows on distinct banks
    alignas(16) double m[4][16 * NT][PITCH];
};
template <int NT>
__device__ __forceinline__ void small_steps(const NsItem &it, const NsParams &p, unsigned char *lds,
                                            double *diagonal)
{
    constexpr int K = 16 * NT, TILES = NT * (NT + 1) / 2;
    auto &m = reinterpret_cast<SmallLds<NT> *>(lds)->m;
    const int tid = static_cast<int>(threadIdx.x), lane = tid & 63, wave = tid >> 6;
    const int lr = lane & 15, kq = lane >> 4;

    const int gi = tid >> 4, gj = 4 * (tid & 15);
    const bool below = gi < K && gj >> 4 <= gi >> 4;  // in a tile on or below the diagonal
    double v[4] = {0., 0., 0., 0.};
    if (below)
        gram_at(it, gi * SMALL + gj, gi, gj, v);
    if (gi < K && gj == (gi & ~3))
        diagonal[gi] = v[gi & 3];
    __syncthreads();
    double trace = lane < K ? diagonal[lane] : 0.;
#pragma unroll
    for (int d = 32; d > 0; d >>= 1)
        trace += __shfl_xor(trace, d);
    const NormScale norm = norm_scale(sqrt(trace), static_cast<double>(p.eps));
    const double inv = norm.inv;
    if (tid == 0)
        it.scal[2] = norm.for_u();
    if (below)
#pragma unroll
        for (int q = 0; q < 4; ++q)
            if (gj + q <= gi) {
                const double x = v[q] * inv * inv;
                m[0][gi][gj + q] = x;
                m[0][gj + q][gi] = x;
            }
    __syncthreads();

    // Matrices 0 to 3: G, P, Q and H = P G.  Three stages a step,
    //   P = a + b G + c G G    H = P G and Q = P Q    G = H P,
    // in one piece of code, which is short enough to be fetched once.  (The first Q is P; after
    // the last one nothing is to follow.)
    constexpr int ROUNDS = (2 * TILES + 15) / 16;
    const int unit = __builtin_amdgcn_readfirstlane(wave);
    for (int step = 0, stage = 0;; stage = stage == 2 ? 0 : stage + 1) {
        const bool first = step == 0, last = step + 1 == p.steps;
        const int from = stage == 1 && last ? TILES : 0, to = stage == 1 && !first ? 2 * TILES : TILES;
        f64x4_t x[ROUNDS];
        int i0[ROUNDS], j0[ROUNDS], into[ROUNDS];
#pragma unroll
        for (int r = 0; r < ROUNDS; ++r) {
            const int u = from + unit + 16 * r;
            into[r] = -1;
            if (u >= to)
                continue;
            const bool second = u >= TILES;
            int t = second ? u - TILES : u, ti = 0;
#pragma unroll
            for (int k = 1; k < NT; ++k)
                ti += t >= k * (k + 1) / 2 ? 1 : 0;
            i0[r] = 16 * ti;
            j0[r] = 16 * (t - ti * (ti + 1) / 2);
            into[r] = stage == 0 ? 1 : stage == 1 ? (second ? 2 : 3) : 0;
            // rows i0.. of X against rows j0.. of Y (symmetric)
            // (a lane's four consecutive values of 16 are four products' share)
            const double *const X = &m[stage == 0 ? 0 : stage == 1 ? 1 : 3][i0[r] + lr][4 * kq];
            const double *const Y = &m[stage == 0 ? 0 : stage == 1 ? (second ? 2 : 0) : 1][j0[r] + lr][4 * kq];
            typedef double pair_t __attribute__((ext_vector_type(2)));
            pair_t v1[2 * NT], v2[2 * NT];
#pragma unroll
            for (int k = 0; k < 2 * NT; ++k) {
                const int at = 16 * (k / 2) + 2 * (k % 2);
                v1[k] = *reinterpret_cast<const pair_t *>(X + at);
                v2[k] = *reinterpret_cast<const pair_t *>(Y + at);
            }
            f64x4_t acc = {0., 0., 0., 0.};
#pragma unroll
            for (int k = 0; k < 4 * NT; ++k)
                acc = mfma4(v1[k / 2][k % 2], v2[k / 2][k % 2], acc);
            if (stage == 0) {
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int i = i0[r] + d_row(q, lane), j = j0[r] + lr;
                    acc[q] = (i == j ? static_cast<double>(p.a) : 0.) +
                             static_cast<double>(p.b) * m[0][i][j] + static_cast<double>(p.c) * acc[q];
                }
            }
            x[r] = acc;
        }
        if (stage == 1)
            __syncthreads();  // (Q is read and written)
#pragma unroll
        for (int r = 0; r < ROUNDS; ++r) {
            if (into[r] < 0)
                continue;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int i = i0[r] + d_row(q, lane), j = j0[r] + lr;
                if (j <= i) {
                    m[into[r]][i][j] = x[r][q];
                    m[into[r]][j][i] = x[r][q];
                    if (stage == 0 && first) {
                        m[2][i][j] = x[r][q];
                        m[2][j][i] = x[r][q];
                    }
                }
            }
        }
        __syncthreads();
        if (stage == 1 && last)
            break;
        step += stage == 2 ? 1 : 0;
    }
    auto &Q = m[2];
    if (tid < SMALL * SMALL / 8) {
        const int i = tid / (SMALL / 8), j = tid % (SMALL / 8) * 8;
        float w[8];
#pragma unroll
        for (int q = 0; q < 8; ++q)  // (zeros past n's tiles: U is zero there, too)
            w[q] = i < K && j < K ? static_cast<float>(Q[i][j + q] * norm.for_q()) : 0.f;
        u32x4_t planes[PLANES];
        split_planes(w, planes);
#pragma unroll
        for (int k = 0; k < PLANES; ++k)
            *reinterpret_cast<u32x4_t *>(it.q + (k * SMALL + i) * SMALL + j) = planes[k];
    }
}

__global__ void __launch_bounds__(1024) ns_small_kernel(NsGroup<NsItem> g)
{
    __shared__ __align__(16) unsigned char lds[sizeof(SmallLds<SMALL / 16>)];
    __shared__ double diagonal[SMALL];
    const NsItem &it = g.it[blockIdx.x];
    if (it.n > 48)
        small_steps<4>(it, g.p, lds, diagonal);
    else if (it.n > 32)
        small_steps<3>(it, g.p, lds, diagonal);
    else if (it.n > 16)
        small_steps<2>(it, g.p, lds, diagonal);
    else
        small_steps<1>(it, g.p, lds, diagonal);
}

// ------------------------------------------------------- the n x n part, larger
__global__ void __launch_bounds__(THREADS) ns_gram_sum_kernel(NsGroup<NsItem> g)
{
    const Found<NsItem> found = find_item(g, blockIdx.x);
    const NsItem &it = found.it;
    const int64_t e = static_cast<int64_t>(found.block) * THREADS + threadIdx.x;
    const int i = static_cast<int>(e / it.np), j = static_cast<int>(e % it.np);
    if (i >= it.np || j > i)
        return;
    double s[1];
    gram_at(it, e, i, j, s);
    it.mat[e] = s[0];
    it.mat[static_cast<int64_t>(j) * it.np + i] = s[0];
}

// One product of symmetric matrices, 32 x 32 tiles on and below the diagonal, mirrored:
//   0  P = a I + b G + c G G    1  H = P G, and Q = P Q    2  G = H P    3  Q = P Q
// (Q in the first step: P).  G is not scaled in place: the first step's products take it by
// 1 / |U|^2, which is formed from its diagonal.  Matrices 4 and 5 are the other G and Q.  The last
// Q goes into planes.  Bound by latency and the 64-bit rate where n is a few hundred (two of 384:
// 8.5 us a product, 13.2 for two).
template <int OP>
__global__ void __launch_bounds__(POLY_WAVES * 64) ns_poly_kernel(NsGroup<NsItem> g, int step)
{
    using R = double;
    constexpr int OPERANDS = POLY_WAVES * 2 * POLY * 144, SUMS = POLY_WAVES * POLY * (POLY + 1) * sizeof(R);
    __shared__ __align__(16) unsigned char lds[OPERANDS > SUMS ? OPERANDS : SUMS];
    auto &red = *reinterpret_cast<R(*)[POLY_WAVES][POLY][POLY + 1]>(lds);
    __shared__ double tr[POLY_WAVES];
    const Found<NsItem> found = find_item(g, place_on_xcd());
    const NsItem &it = found.it;
    const int np = it.np, nt = np / POLY, tiles = nt * (nt + 1) / 2;
    int tj = found.block;
    const bool second = tj >= tiles;  // Q's tiles behind H's
    tj -= second ? tiles : 0;
    int ti = 0;
    while (tj > ti) {
        tj -= ti + 1;
        ++ti;
    }
    const int64_t size = static_cast<int64_t>(np) * np;
    R *const mat = it.mat;
    R *const G = mat + (step & 1 ? 4 * size : 0), *const G2 = mat + (step & 1 ? 0 : 4 * size);
    R *const P = mat + size, *const H = mat + 3 * size;
    R *const Q = mat + (step & 1 ? 5 : 2) * size, *const Q2 = mat + (step & 1 ? 2 : 5) * size;
    const R *X, *Y;
    R *out;
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
    double scaled = 1., for_q = 1.;
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
        const NormScale norm = norm_scale(sqrt(s), static_cast<double>(g.p.eps));
        scaled = norm.inv * norm.inv;
        for_q = norm.for_q();
        if (ti == 0 && tid == 0) {
            it.scal[0] = for_q;
            it.scal[1] = scaled;
            it.scal[2] = norm.for_u();
        }
    } else if (step == 0) {
        scaled = it.scal[1];
    }

    f64x4_t acc[2][2];
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int y = 0; y < 2; ++y)
            acc[x][y] = f64x4_t{0., 0., 0., 0.};
    // Each wave takes every eighth 128-byte line of the 32 rows and the 32 columns' rows: whole lines
    // (half of them an instruction took 3 us longer to come, from caches that other CUs wrote), two
    // turns' on their way at once, turned in LDS of the wave's own into operands of 16 rows.
    constexpr int LINE = 128 / sizeof(R), PITCH = 144;  // (16 bytes of 16 rows on distinct banks)
    unsigned char *const mine = lds + wave * 64 * PITCH;
    const int lines = np / LINE;
    const int own = __builtin_amdgcn_readfirstlane(wave);
    const unsigned int in_line = (lane >> 3) * np + (lane & 7) * (16 / sizeof(R));
    u32x4_t v[2][8];
    auto fetch = [&](u32x4_t (&to)[8], int line) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {  // (uniform addresses and the lane's place: fewer registers)
            const R *const from = (i < 4 ? X + static_cast<int64_t>(i0 + 8 * i) * np
                                         : Y + static_cast<int64_t>(j0 + 8 * (i - 4)) * np) + line * LINE;
            to[i] = *reinterpret_cast<const u32x4_t *>(from + in_line);
        }
    };
    auto use = [&](const u32x4_t (&from)[8]) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            *reinterpret_cast<u32x4_t *>(mine + (8 * i + (lane >> 3)) * PITCH + (lane & 7) * 16) = from[i];
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int t = 0; t < LINE / 16; ++t) {  // 16 values of K, four consecutive ones a lane
            f64x4_t a[2], b[2];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int at = (16 * t + 4 * kq) * static_cast<int>(sizeof(R));
                a[q] = *reinterpret_cast<const f64x4_t *>(mine + (16 * q + lr) * PITCH + at);
                b[q] = *reinterpret_cast<const f64x4_t *>(mine + (32 + 16 * q + lr) * PITCH + at);
            }
#pragma unroll
            for (int s = 0; s < 4; ++s)
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int y = 0; y < 2; ++y)
                        acc[x][y] = mfma4(a[x][s], b[y][s], acc[x][y]);
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    };
    if (own < lines) {
        fetch(v[0], own);
        fetch(v[1], own + POLY_WAVES < lines ? own + POLY_WAVES : own);
    }
    for (int line = own; line < lines; line += 2 * POLY_WAVES) {
        use(v[0]);
        if (line + 2 * POLY_WAVES < lines)
            fetch(v[0], line + 2 * POLY_WAVES);
        if (line + POLY_WAVES < lines)
            use(v[1]);
        if (line + 3 * POLY_WAVES < lines)
            fetch(v[1], line + 3 * POLY_WAVES);
    }
    __syncthreads();  // (the sums lie where the operands were)
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int y = 0; y < 2; ++y)
#pragma unroll
            for (int q = 0; q < 4; ++q)
                red[wave][16 * x + d_row(q, lane)][16 * y + lr] = acc[x][y][q];
    __syncthreads();
    const bool planes = (OP == 3 || OP == 0) && step + 1 == g.p.steps && (OP == 3 || step == 0);
    // the values of the tile, and a second time transposed
    auto put = [&](int i, int j, R x) {
        const int64_t at = static_cast<int64_t>(i) * np + j;
        if (planes) {
            float r = static_cast<float>(x * (OP == 0 ? for_q : it.scal[0]));
#pragma unroll
            for (int k = 0; k < PLANES; ++k) {
                const uint16_t w = f32_to_bf16(r);
                it.q[k * size + at] = w;
                r -= __uint_as_float(static_cast<unsigned int>(w) << 16);
            }
            return;
        }
        out[at] = x;
        if constexpr (OP == 0) {
            if (step == 0)  // the first Q
                Q2[at] = x;
        }
    };
    for (int e = tid; e < POLY * POLY; e += POLY_WAVES * 64) {
        const int i = e / POLY, j = e % POLY;
        R s = red[0][i][j];
#pragma unroll
        for (int w = 1; w < POLY_WAVES; ++w)
            s += red[w][i][j];
        if constexpr (OP == 0) {
            const double x = G[static_cast<int64_t>(i0 + i) * np + j0 + j];
            s = (i0 + i == j0 + j ? static_cast<double>(g.p.a) : 0.) +
                static_cast<double>(g.p.b) * (scaled * x) +
                static_cast<double>(g.p.c) * (scaled * (scaled * s));
        } else if constexpr (OP == 1) {
            if (!second)
                s *= scaled;
        }
        red[0][i][j] = s;  // (no other thread reads it before the barrier)
        if (j0 + j <= i0 + i)
            put(i0 + i, j0 + j, s);
    }
    __syncthreads();
    for (int e = tid; e < POLY * POLY; e += POLY_WAVES * 64) {
        const int i = e % POLY, j = e / POLY;
        if (j0 + j < i0 + i)
            put(j0 + j, i0 + i, red[0][i][j]);
    }
}

// ------------------------------------------------------------- O = Q U (or U Q)
// Tiles of NB values of the shorter side by 128 of the longer one, eight waves (4 x 2), 64 values
// of K (the shorter side) a stage, the next one on its way.  The tile goes through LDS, so that
// the update reads and writes whole lines.  Bound by its loads' round trips, the splitting and the
// products in turn, at one workgroup a CU (384 x 8192 and 28672 x 384 in bf16: 98 us for 85 MB read,
// 28 written and six products of 11 GFLOP).
constexpr int FINAL_WAVES = 8;  // two in each row

// LDS tiles of one plane: 64 K values of R rows, as rows of K values 160 bytes apart (a 16-byte
// read takes lanes 0-3, 12-15 and 20-27 at once, and so on: sixteen chunks of two neighbouring
// columns, which lie on distinct banks; 144 bytes: two on each), or, where the matrix lies the
// other way, as 64 rows of R values, read by transposing loads.
template <int R>
struct Tiles {
    static constexpr int KP = 160, MP = 2 * R + 32;
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
        const unsigned char *const p = tile + (32 * h + 8 * kq + (lr >> 2)) * MP + (c0 + 4 * (lr & 3)) * 2;
        const s16x4_t x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(p));
        const s16x4_t y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(p + 4 * MP));
        return __builtin_bit_cast(bf16x8_t, __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7));
    }
};
template <int NB>
struct FinalLds {
    static constexpr int U_BYTES = Tiles<128>::K_BYTES > Tiles<128>::M_BYTES ? Tiles<128>::K_BYTES
                                                                             : Tiles<128>::M_BYTES;
    static constexpr int STAGE = PLANES * (Tiles<NB>::K_BYTES + U_BYTES);
    static constexpr int OUT = 128 * (NB + 4) * 4 > NB * (128 + 4) * 4 ? 128 * (NB + 4) * 4
                                                                       : NB * (128 + 4) * 4;
    static constexpr int BYTES = STAGE > OUT ? STAGE : OUT;
};
template <typename T, bool TALL, int NB>
__device__ __forceinline__ void final_tile(const NsOutput &it, int block, unsigned char *lds)
{
    constexpr int P = PLANES;
    constexpr int BM = TALL ? 128 : NB, BN = TALL ? NB : 128;
    using Tq = Tiles<NB>;
    using Tu = Tiles<128>;
    constexpr int KP = Tu::KP, MP = Tu::MP;
    constexpr int Q_ROWS = NB;
    constexpr int TM = BM / (8 * FINAL_WAVES), TN = BN / 32;  // 16 x 16 blocks of a wave
    unsigned char *qs[P], *us[P];
#pragma unroll
    for (int p = 0; p < P; ++p) {
        qs[p] = lds + p * Tq::K_BYTES;
        us[p] = lds + P * Tq::K_BYTES + p * FinalLds<NB>::U_BYTES;
    }
    const int nb = it.np / NB;
    // (the tiles of one stretch of the longer side next to each other: they read the same U)
    const int n0 = (block % nb) * NB;
    const int64_t l0 = static_cast<int64_t>(block / nb) * 128;
    const int tid = static_cast<int>(threadIdx.x), lane = tid & 63, wave = tid >> 6;
    const int lr = lane & 15, kq = lane >> 4, wm = wave >> 1, wn = wave & 1;
    const int np = it.np;
    const int64_t qsize = static_cast<int64_t>(np) * np;
    const float scale = static_cast<float>(it.scal[2]);

    // 16-byte chunks a thread
    constexpr int QV = Q_ROWS * 8 / (64 * FINAL_WAVES), UV = 128 * 8 / (64 * FINAL_WAVES);
    u32x4_t qr[QV][P];
    Raw8<float> uf[UV];
    auto u_at = [&](int v, int k) {  // row-major place of chunk v of the stage at k
        if constexpr (TALL)
            return (l0 + v / 8) * it.cp + k + v % 8 * 8;
        else
            return static_cast<int64_t>(k + v / 16) * it.cp + l0 + v % 16 * 8;
    };
    auto fetch = [&](int k) {
#pragma unroll
        for (int i = 0; i < QV; ++i) {
            const int v = tid + i * (64 * FINAL_WAVES);
#pragma unroll
            for (int p = 0; p < P; ++p)
                qr[i][p] = *reinterpret_cast<const u32x4_t *>(
                    it.q + p * qsize + static_cast<int64_t>(n0 + v / 8) * np + k + v % 8 * 8);
        }
#pragma unroll
        for (int i = 0; i < UV; ++i)
            uf[i].template load<true>(it.u + u_at(tid + i * (64 * FINAL_WAVES), k), 8);
    };
    auto keep = [&]() {
#pragma unroll
        for (int i = 0; i < QV; ++i) {
            const int v = tid + i * (64 * FINAL_WAVES);
#pragma unroll
            for (int p = 0; p < P; ++p)
                *reinterpret_cast<u32x4_t *>(qs[p] + v / 8 * KP + v % 8 * 16) = qr[i][p];
        }
#pragma unroll
        for (int i = 0; i < UV; ++i) {
            const int v = tid + i * (64 * FINAL_WAVES);
            u32x4_t w[P];
            float f[8];
            uf[i].get(f);
#pragma unroll
            for (int q = 0; q < 8; ++q)
                f[q] *= scale;
            split_planes(f, w);
#pragma unroll
            for (int p = 0; p < P; ++p)
                *reinterpret_cast<u32x4_t *>(
                    us[p] + (TALL ? v / 8 * KP + v % 8 * 16 : v / 16 * MP + v % 16 * 16)) = w[p];
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
        fetch(k + 64 < np ? k + 64 : 0);  // (no branch round a load, as above)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            bf16x8_t a[TM][P];
#pragma unroll
            for (int p = 0; p < P; ++p)
#pragma unroll
                for (int i = 0; i < TM; ++i)
                    a[i][p] = TALL ? Tu::rows16(us[p], wm * (16 * TM) + 16 * i, h, lane)
                                   : Tq::rows16(qs[p], wm * (16 * TM) + 16 * i, h, lane);
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                bf16x8_t b[P];
#pragma unroll
                for (int p = 0; p < P; ++p)
                    b[p] = TALL ? Tq::rows16(qs[p], wn * (BN / 2) + 16 * j, h, lane)
                                : Tu::columns16(us[p], wn * (BN / 2) + 16 * j, h, lane);
#pragma unroll
                for (int i = 0; i < TM; ++i)
#pragma unroll
                    for (int s = P - 1; s >= 0; --s)  // planes x and s - x, the small ones first
#pragma unroll
                        for (int x = 0; x <= s; ++x)
                            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[s - x], a[i][x],
                                                                                acc[i][j], 0, 0, 0);
            }
        }
    }
    // a lane holds row lr and four consecutive columns of each block
    constexpr int OP = BN + 4, ROW = BN / 8, OV = BM * ROW / (64 * FINAL_WAVES);
    const int64_t m0 = TALL ? l0 : n0, c0 = TALL ? n0 : l0;
    Raw8<T> raw[OV];
    int cnt[OV];
#pragma unroll
    for (int i = 0; i < OV; ++i) {
        const int v = tid + i * (64 * FINAL_WAVES);
        const int64_t r = m0 + v / ROW, c = c0 + v % ROW * 8;
        cnt[i] = r < it.rows ? count8(it.cols, c) : 0;
        if (it.p != nullptr && cnt[i] > 0)
            raw[i].load(static_cast<const T *>(it.p) + r * it.cols + c, cnt[i]);
    }
    float *const tile = reinterpret_cast<float *>(lds);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
            *reinterpret_cast<f32x4_t *>(tile + (wm * (16 * TM) + 16 * i + lr) * OP + wn * (BN / 2) +
                                         16 * j + 4 * kq) = acc[i][j];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < OV; ++i) {
        const int v = tid + i * (64 * FINAL_WAVES);
        const int64_t r = m0 + v / ROW, c = c0 + v % ROW * 8;
        if (cnt[i] <= 0)
            continue;
        float x[8];
        const float *const from = tile + v / ROW * OP + v % ROW * 8;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const f32x4_t y = *reinterpret_cast<const f32x4_t *>(from + 4 * q);
#pragma unroll
            for (int k = 0; k < 4; ++k)
                x[4 * q + k] = y[k];
        }
        if (it.p != nullptr) {
            float w[8];
            raw[i].get(w);
#pragma unroll
            for (int q = 0; q < 8; ++q)
                x[q] = __fmaf_rn(-it.step, x[q], it.keep * w[q]);
        }
        raw[i].set(x);
        raw[i].store(static_cast<T *>(it.out) + r * it.cols + c, cnt[i]);
    }
}

template <typename T, int NB>
__global__ void __launch_bounds__(64 * FINAL_WAVES, FINAL_WAVES / 4) ns_final_kernel(NsGroup<NsOutput> g)
{
    __shared__ __align__(16) unsigned char lds[FinalLds<NB>::BYTES];
    const Found<NsOutput> found = find_item(g, place_on_xcd());
    if (found.it.tall)
        final_tile<T, true, NB>(found.it, found.block, lds);
    else
        final_tile<T, false, NB>(found.it, found.block, lds);
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

int64_t gram_tiles(int64_t np) { return np / TILE * (np / TILE + 1) / 2; }
int64_t prepare_groups(int64_t rp, int64_t cp)
{
    return (rp * cp / 8 + THREADS * PREP_VPT - 1) / (THREADS * PREP_VPT);
}

// Matrices [first, first + count) of one set of launches: up to 40, in 256 MiB (or one).
struct Chunk {
    int first, count;
    size_t bytes;
    NsItem it[MAX_ITEMS];
};
constexpr size_t CHUNK_BYTES = size_t(256) << 20;

Chunk plan_chunk(const NsMatrix *mats, int count, int first, char *ws)
{
    Chunk c;
    c.first = first;
    int64_t per_split = 0, per_front = 0;
    auto fill = [&](NsItem &it, const NsMatrix &m, size_t off) {
        const Sides s = sides(m.rows, m.cols);
        it.tall = s.tall;
        it.n = static_cast<int>(s.tall ? m.cols : m.rows);
        it.np = static_cast<int>(s.np);
        it.rp = static_cast<int>(s.rp);
        it.cp = static_cast<int>(s.cp);
        // (a product's n terms a row, and the sums over a share of the longer side before that)
        it.lift = static_cast<float>((16. + 4. * it.n) * std::max(1., std::sqrt(double(s.lp)) / 64.) * 0x1p-53);
        const int64_t share = s.np > SMALL ? per_split : per_front;
        it.per_split = static_cast<int>(share < s.lp ? share : s.lp);
        it.splits = static_cast<int>((s.lp + it.per_split - 1) / it.per_split);
        auto take = [&](size_t bytes) {
            const size_t at = off;
            off += (bytes + 255) / 256 * 256;
            return ws + at;
        };
        const size_t square = static_cast<size_t>(s.np) * s.np;
        it.u = reinterpret_cast<float *>(take(static_cast<size_t>(s.rp) * s.cp * sizeof(float)));
        it.part = reinterpret_cast<double *>(take(it.splits * square * sizeof(double)));
        it.mat = reinterpret_cast<double *>(take(s.np > SMALL ? 6 * square * sizeof(double) : 0));
        it.scal = reinterpret_cast<double *>(take(3 * sizeof(double)));
        it.q = reinterpret_cast<uint16_t *>(take(PLANES * square * sizeof(uint16_t)));
        return off;
    };
    // The Gram products of the set as about 1024 workgroups of equal length (512 where one forms U,
    // too), of 64 values of the longer side each at least; a matrix has at most 32 shares.
    auto split = [&](int n) {
        int64_t work = 0, longest = 0, work_front = 0, longest_front = 0;
        for (int i = first; i < first + n; ++i) {
            const Sides s = sides(mats[i].rows, mats[i].cols);
            if (s.np > SMALL) {
                work += gram_tiles(s.np) * s.lp;
                longest = s.lp > longest ? s.lp : longest;
            } else {
                work_front += s.lp;
                longest_front = s.lp > longest_front ? s.lp : longest_front;
            }
        }
        auto share = [](int64_t even, int64_t least) { return up_to(even > least ? even : least, 64); };
        per_split = share(work / 1024, (longest + 31) / 32);
        per_front = share(work_front / 512, (longest_front + 31) / 32);
        size_t off = 0;
        for (int i = 0; i < n; ++i)
            off = fill(c.it[i], mats[first + i], off);
        return off;
    };
    c.count = count - first < MAX_ITEMS ? count - first : MAX_ITEMS;
    while ((c.bytes = split(c.count)) > CHUNK_BYTES && c.count > 1)
        c.count -= (c.count + 7) / 8;
    return c;
}

// The items that `take` picks as a launch's group, with `blocks` workgroups each.
template <typename I, typename Take, typename Blocks>
int group_of(NsGroup<I> &g, const I *items, const Chunk &c, Take &&take, Blocks &&blocks)
{
    int n = 0, at = 0;
    for (int i = 0; i < c.count; ++i) {
        if (!take(c.it[i]))
            continue;
        g.it[n] = items[i];
        g.start[n++] = at;
        at += static_cast<int>(blocks(c.it[i]));
    }
    for (; n < MAX_ITEMS; ++n)
        g.start[n] = INT_MAX;
    return at;
}

template <typename T>
hipError_t run_chunk(const Chunk &c, const NsMatrix *mats, const NsParams &p, hipStream_t st)
{
#define NS_LAUNCH(...)                         \
    do {                                       \
        hipLaunchKernelGGL(__VA_ARGS__);       \
        const hipError_t e_ = hipGetLastError(); \
        if (e_ != hipSuccess)                  \
            return e_;                         \
    } while (0)
    auto small = [](const NsItem &i) { return i.np == SMALL; };
    auto large = [](const NsItem &i) { return i.np > SMALL; };
    int n;
    {
        NsInput in[MAX_ITEMS];
        for (int i = 0; i < c.count; ++i) {
            const NsItem &it = c.it[i];
            const NsMatrix &m = mats[c.first + i];
            in[i] = NsInput{it.u,   it.part, m.g,   m.m,   m.m_out, m.rows,
                            m.cols, it.rp,   it.cp, it.tall, it.per_split};
        }
        NsGroup<NsInput> g;
        g.p = p;
        n = group_of(g, in, c, small, [](const NsItem &i) { return i.splits; });
        if (n > 0)
            NS_LAUNCH((ns_front_kernel<T>), dim3(n), dim3(FRONT), 0, st, g);
        n = group_of(g, in, c, large, [](const NsItem &i) { return prepare_groups(i.rp, i.cp); });
        if (n > 0)
            NS_LAUNCH((ns_prepare_kernel<T>), dim3(n), dim3(THREADS), 0, st, g);
    }
    NsGroup<NsItem> g;
    g.p = p;
    n = group_of(g, c.it, c, large, [](const NsItem &i) { return gram_tiles(i.np) * i.splits; });
    if (n > 0)
        NS_LAUNCH(ns_gram_kernel, dim3(n), dim3(THREADS), 0, st, g);
    n = group_of(g, c.it, c, small, [](const NsItem &) { return 1; });
    if (n > 0)
        NS_LAUNCH(ns_small_kernel, dim3(n), dim3(1024), 0, st, g);
    n = group_of(g, c.it, c, large, [](const NsItem &i) {
        return (static_cast<int64_t>(i.np) * i.np + THREADS - 1) / THREADS;
    });
    if (n > 0) {
        NS_LAUNCH(ns_gram_sum_kernel, dim3(n), dim3(THREADS), 0, st, g);
        auto tiles = [](const NsItem &i) {
            return static_cast<int64_t>(i.np / POLY) * (i.np / POLY + 1) / 2;
        };
        const dim3 block(POLY_WAVES * 64);
        for (int s = 0; s < p.steps; ++s) {
            const bool first = s == 0, last = s + 1 == p.steps;
            n = group_of(g, c.it, c, large, tiles);
            NS_LAUNCH((ns_poly_kernel<0>), dim3(n), block, 0, st, g, s);
            if (last) {
                if (!first)
                    NS_LAUNCH((ns_poly_kernel<3>), dim3(n), block, 0, st, g, s);
                continue;
            }
            // (the first Q is P)
            const int each = first ? 1 : 2;
            n = group_of(g, c.it, c, large, [&](const NsItem &i) { return each * tiles(i); });
            NS_LAUNCH((ns_poly_kernel<1>), dim3(n), block, 0, st, g, s);
            n = group_of(g, c.it, c, large, tiles);
            NS_LAUNCH((ns_poly_kernel<2>), dim3(n), block, 0, st, g, s);
        }
    }
    NsOutput to[MAX_ITEMS];
    for (int i = 0; i < c.count; ++i) {
        const NsItem &it = c.it[i];
        const NsMatrix &m = mats[c.first + i];
        to[i] = NsOutput{it.u,   it.q,   it.scal, m.p,   m.out,   m.rows, m.cols,
                         m.step, m.keep, it.np,   it.tall, it.rp, it.cp};
    }
    NsGroup<NsOutput> o;
    o.p = p;
    n = group_of(o, to, c, small, [](const NsItem &i) { return (i.tall ? i.rp : i.cp) / 128; });
    if (n > 0)
        NS_LAUNCH((ns_final_kernel<T, 64>), dim3(n), dim3(64 * FINAL_WAVES), 0, st, o);
    n = group_of(o, to, c, large, [](const NsItem &i) {
        return static_cast<int64_t>(i.tall ? i.rp : i.cp) / 128 * (i.np / 128);
    });
    if (n > 0)
        NS_LAUNCH((ns_final_kernel<T, 128>), dim3(n), dim3(64 * FINAL_WAVES), 0, st, o);
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

size_t newton_schulz_workspace(const NsMatrix *mats, int count)
{
    size_t most = 0;
    for (int first = 0; first < count;) {
        const Chunk c = plan_chunk(mats, count, first, nullptr);
        most = c.bytes > most ? c.bytes : most;
        first += c.count;
    }
    return most;
}

hipError_t launch_newton_schulz(int bf16, const NsMatrix *mats, int count, const NsParams &p, void *ws,
                                hipStream_t st)
{
    for (int first = 0; first < count;) {
        const Chunk c = plan_chunk(mats, count, first, static_cast<char *>(ws));
        const hipError_t e = bf16 ? run_chunk<uint16_t>(c, mats, p, st)
                                  : run_chunk<float>(c, mats, p, st);
        if (e != hipSuccess)
            return e;
        first += c.count;
    }
    return hipSuccess;
}

}  // namespace dora
