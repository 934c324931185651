// gemm_fourbit.hip - y = x W^T for a few tokens and a weight held as 4-bit rows (gfx950).
//
// Bound by reading the codes once (half a byte a weight), as whole cache lines: a line is 256
// columns, the 128 bytes of codes that one cache line holds.  A wave loads eight rows of a line
// an instruction into registers (16 rows of half a line are 64-byte requests: 30 us against 24.5
// for one token over 28672 channels of 8192, on one weight in a graph; 25.9 on six weights in turn,
// 26.2 by the profiler, 27.3 as a call), turns them in LDS, and exchanges between the
// lane groups make four MFMA operands of 32 consecutive columns each of four registers; one
// conversion instruction makes two bf16 weights of two codes.  The weights enter the products as
// the codes' own values, exact in bf16, and the fp32 sums over a group's columns meet its
// scale, so that nothing is rounded before the sums.  fp32 tokens enter as three bf16 numbers
// each, which hold all 24 bits.  The sums of waves that split K meet in LDS, in order.
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
    // (rows of an odd number of scales start at any 2 bytes)
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, uint32_t v, int s)
    {
        if constexpr (PER == 8) {
            const auto q = __builtin_amdgcn_raw_buffer_load_b128(r, v, s, 0);
            w[0] = q[0]; w[1] = q[1]; w[2] = q[2]; w[3] = q[3];
        } else if constexpr (PER == 4) {
            const auto q = __builtin_amdgcn_raw_buffer_load_b64(r, v, s, 0);
            w[0] = q[0]; w[1] = q[1];
        } else if constexpr (PER == 2) {
            w[0] = __builtin_amdgcn_raw_buffer_load_b32(r, v, s, 0);
        } else {
            w[0] = __builtin_amdgcn_raw_buffer_load_b16(r, v, s, 0);
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
    u32x4_t c[NT][2];
    LineScales<PER> s[NT];
};

// A descriptor of `bytes` bytes (under 2^31) from `p`, in scalar registers.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_rsrc(const void *p, int64_t bytes)
{
    const uint64_t at = reinterpret_cast<uint64_t>(p);
    const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(at));
    const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(at >> 32));
    return __builtin_amdgcn_make_buffer_rsrc(
        reinterpret_cast<void *>((static_cast<uint64_t>(hi) << 32) | lo), static_cast<short>(0),
        __builtin_amdgcn_readfirstlane(static_cast<int>(bytes)), 0x00020000);
}
constexpr int AUX_NT = 2;  // non-temporal

// 16-byte chunk c of row r of a tile in LDS lies at c ^ swizzle(r): neither 8 rows written whole
// nor 16 rows read at one chunk meet on a bank.
__device__ __forceinline__ int swizzle(int r) { return ((r >> 1) ^ ((r & 1) << 2)) & 7; }

// The same for rows of 512 bytes, whose chunks all lie on the same banks: a 16-byte read takes
// lanes 0-3, 12-15 and 20-27 at once (and so on), eight rows at one chunk and the other eight at
// the next one.
__device__ __forceinline__ int swizzle_line(int r)
{
    return swizzle(r) | ((((r >> 2) ^ (r >> 3)) & 1) << 3);
}

// Orders the wave's LDS accesses around it: to the compiler, for which accesses of one lane to
// different places could change places, though other lanes meet them (LDS itself takes a wave's in order).
__device__ __forceinline__ void wave_lds_order()
{
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
    __builtin_amdgcn_wave_barrier();
}

// A wave's reader of the codes of tiles of 16 NT channels.
template <int NT, int PER>
struct Codes {
    const FourbitArgs &a;
    unsigned char *turned;  // the wave's LDS, NT x 2 KiB
    int lane, nl, kq, lrow, lchunk, per_shift;
    int64_t whole, pitch;  // lines that lie inside the row; bytes of a row
    uint32_t code_off[NT][2], scale_off[NT];

    __device__ __forceinline__ Codes(const FourbitArgs &args, unsigned char *lds, int l)
        : a(args), turned(lds), lane(l), nl(l & 15), kq(l >> 4), lrow(l >> 3), lchunk(l & 7),
          per_shift(PER > 1 ? 0 : 31 - __clz(args.group / LINE)), whole(args.d_in / LINE),
          pitch(args.groups * (args.group / 2))
    {
#pragma unroll
        for (int i = 0; i < NT; ++i) {
#pragma unroll
            for (int u = 0; u < 2; ++u)
                code_off[i][u] =
                    (16 * i + 8 * u + lrow) * static_cast<uint32_t>(pitch) + 16 * lchunk;
            scale_off[i] = (16 * i + nl) * static_cast<uint32_t>(a.groups) * 2;
        }
    }
    __device__ __forceinline__ int64_t row_of(int64_t n) const { return n < a.d_out ? n : a.d_out - 1; }

    // Line `line` of tile `tile`: eight rows of whole cache lines an instruction, lane l the
    // l & 7th 16 bytes of rows l >> 3 and 8 + (l >> 3).  Through descriptors of the tile's
    // rows: channels past the last one read zeros, and everything does unless `any`, with no
    // branch: around a branch the compiler cannot count the loads in flight, and waits for all
    // of them at each use.
    __device__ __forceinline__ void load(Line<NT, PER> &l, int64_t tile, int64_t line, bool any) const
    {
        const int64_t n0 = tile * (16 * NT), left = a.d_out - n0 < 16 * NT ? a.d_out - n0 : 16 * NT;
        const auto rc = rows_rsrc(a.codes + n0 * pitch, any ? left * pitch : 0);
        const auto rs = rows_rsrc(a.scale + n0 * a.groups, any ? left * a.groups * 2 : 0);
        const int co = static_cast<int>(line * (LINE / 2));
        const int so = static_cast<int>(PER > 1 ? line * PER : line >> per_shift) * 2;
#pragma unroll
        for (int i = 0; i < NT; ++i) {
#pragma unroll
            for (int u = 0; u < 2; ++u)
                l.c[i][u] = __builtin_bit_cast(
                    u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rc, code_off[i][u], co, AUX_NT));
            l.s[i].load(rs, scale_off[i], so);
        }
    }
    // the line that the row ends in, nothing past its end
    __device__ __forceinline__ void load_tail(Line<NT, PER> &l, int64_t tile) const
    {
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            const int64_t n0 = (tile * NT + i) * 16, at = whole * (LINE / 2) + 16 * lchunk;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                l.c[i][u] = u32x4_t{0u, 0u, 0u, 0u};
                if (at < pitch)
                    l.c[i][u] = *reinterpret_cast<const u32x4_t *>(
                        a.codes + row_of(n0 + 8 * u + lrow) * pitch + at);
            }
            const uint16_t *s = a.scale + row_of(n0 + nl) * a.groups;
            if constexpr (PER > 1)
                l.s[i].load_some(s + whole * PER, a.groups - whole * PER);
            else
                l.s[i].load_some(s + (whole >> per_shift), 1);
        }
    }
    // a line into the wave's LDS, and the four operand registers of its half h from there
    __device__ __forceinline__ void turn(const Line<NT, PER> &l) const
    {
        wave_lds_order();  // (the line before it has been read)
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int r = 8 * u + lrow;
                *reinterpret_cast<u32x4_t *>(turned + i * 2048 + r * 128 + 16 * (lchunk ^ swizzle(r))) =
                    l.c[i][u];
            }
        wave_lds_order();
    }
    __device__ __forceinline__ void half(unsigned int (&c)[NT][4], int h) const
    {
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            const u32x4_t v = *reinterpret_cast<const u32x4_t *>(
                turned + i * 2048 + nl * 128 + 16 * ((4 * h + kq) ^ swizzle(nl)));
            c[i][0] = v.x; c[i][1] = v.y; c[i][2] = v.z; c[i][3] = v.w;
            exchange4(c[i]);
        }
    }
};

// A wave's sums: of the group under way, and of those whose scale has been met.
template <int TM, int NT>
struct Sums {
    f32x4_t acc[TM][NT], part[TM][NT];
    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < NT; ++j)
                acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    }
    // step `step` of a line: the products of 32 columns, and the scale where a group ends
    template <int PER, int P>
    __device__ __forceinline__ void step(const bf16x8_t (&x)[TM][P], const unsigned int (&c)[NT][4],
                                         const Line<NT, PER> &l, int step)
    {
        constexpr int EVERY = STEPS / PER;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const bf16x8_t w = weights8(c[j][step % 4]);
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int p = P - 1; p >= 0; --p)  // the smallest parts first
                    part[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                        x[i][p], w, step % EVERY == 0 && p == P - 1 ? f32x4_t{0.f, 0.f, 0.f, 0.f} : part[i][j],
                        0, 0, 0);
        }
        if ((step + 1) % EVERY == 0) {
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const float by = l.s[j].get(step / EVERY);
#pragma unroll
                for (int i = 0; i < TM; ++i)
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        acc[i][j][q] = __fmaf_rn(by, part[i][j][q], acc[i][j][q]);
            }
        }
    }
};

template <typename T>
__device__ __forceinline__ void put(T *p, float v)
{
    if constexpr (sizeof(T) == 2)
        *p = f32_to_bf16(v);
    else
        *p = v;
}

// Up to FEW tokens (a block of them, blockIdx.y), whose rows lie whole in LDS (dynamic: planes x
// tokens x pitch elements).  The W waves split K; a workgroup walks the tiles blockIdx.x,
// blockIdx.x + gridDim.x, ... of 16 channels and keeps its waves' loads going across them, so
// that the workgroups at work read rows that lie close to each other (one workgroup a CU over
// 28672 channels of 8192, on one weight in a graph: 24.5 us, two 28, a workgroup a tile 38).
constexpr int FEW = 4;
template <typename T, int PER, int W>
__global__ void __launch_bounds__(W * 64) linear_fourbit_kernel(FourbitArgs a)
{
    constexpr int P = planes<T>, PITCH = 20;
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ __align__(16) float sums[2][W][FEW][PITCH];  // (two buffers: one barrier a tile)
    __shared__ __align__(16) unsigned char turned[W][2048];
    const int lane = static_cast<int>(threadIdx.x) & 63, nl = lane & 15, kq = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6);
    const int64_t t0 = static_cast<int64_t>(blockIdx.y) * FEW;
    const int tokens = static_cast<int>(a.T - t0 < FEW ? a.T - t0 : FEW);
    const Codes<1, PER> codes(a, turned[wave], lane);
    const int64_t whole = codes.whole, lines = (a.d_in + LINE - 1) / LINE;
    const int64_t rounds = whole > 0 ? (whole + W - 1) / W : 1;
    const int64_t tiles = (a.d_out + 15) / 16;

    // the wave's whole lines in order, over all its tiles: where the next load stands
    Line<1, PER> ring;
    int64_t ltile = blockIdx.x, lround = 0;
    auto load_next = [&]() {
        const int64_t line = wave + lround * W;
        codes.load(ring, ltile < tiles ? ltile : 0, line, ltile < tiles && line < whole);
        if (++lround == rounds) {
            lround = 0;
            ltile += gridDim.x;
        }
    };
    load_next();

    const int64_t xpitch = lines * LINE + 8, vecs = xpitch / 8;
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
    const unsigned char *const x = smem + ((nl < tokens ? nl : tokens - 1) * xpitch + 8 * kq) * 2;

    Sums<1, 1> sum;
    sum.clear();
    auto products = [&](const Line<1, PER> &l, int64_t line) {
        codes.turn(l);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            unsigned int c[1][4];
            codes.half(c, h);
#pragma unroll
            for (int s = 4 * h; s < 4 * h + 4; ++s) {
                bf16x8_t xs[1][P];
#pragma unroll
                for (int p = 0; p < P; ++p)
                    xs[0][p] = __builtin_bit_cast(
                        bf16x8_t, *reinterpret_cast<const u32x4_t *>(
                                      x + (p * tokens * xpitch + line * LINE + s * 32) * 2));
                sum.step(xs, c, l, s);
            }
        }
    };
    // the end of a tile: the waves' sums, in order (the tokens are rows 0 to 3, lanes 0 to 15)
    int buf = 0;
    auto finish = [&](int64_t tile) {
        if (kq == 0)
#pragma unroll
            for (int q = 0; q < FEW; ++q)
                sums[buf][wave][q][nl] = sum.acc[0][0][q];
        sum.clear();
        __syncthreads();
        const int e = static_cast<int>(threadIdx.x), m = e / 16, n = e % 16;
        if (m < tokens && tile * 16 + n < a.d_out) {
            float v = sums[buf][0][m][n];
#pragma unroll
            for (int w = 1; w < W; ++w)
                v += sums[buf][w][m][n];
            put(static_cast<T *>(a.y) + (t0 + m) * a.d_out + tile * 16 + n, v);
        }
        buf ^= 1;
    };
    for (int64_t tile = blockIdx.x, round = 0; tile < tiles;) {
        const int64_t line = wave + round * W;
        if (line < whole)
            products(ring, line);
        load_next();
        if (++round == rounds) {
            if (whole < lines && whole % W == wave) {
                Line<1, PER> l;
                codes.load_tail(l, tile);
                products(l, whole);
            }
            finish(tile);
            round = 0;
            tile += gridDim.x;
        }
    }
}

// More tokens: CW waves a K group take 16 NT channels each and share the tokens' line, which lies
// in LDS, the next one on its way; KG such groups split K.  (d_in of a line at least.)
template <typename T, int TM, int NT, int PER, int CW, int KG, int D, int XD>
__global__ void __launch_bounds__(CW *KG * 64) linear_fourbit_shared_kernel(FourbitArgs a)
{
    constexpr int P = planes<T>;
    constexpr int ROW = LINE * 2;                    // bytes of a token's line
    constexpr int XBYTES = P * 16 * TM * ROW;        // a line of the tokens
    constexpr int LOADS = 16 * TM * (LINE / 8) / (CW * 64);  // vectors of eight a thread
    static_assert(LOADS * CW * 64 == 16 * TM * (LINE / 8), "whole vectors a thread");
    constexpr int PITCH = CW * 16 * NT + 4;
    static_assert(KG * 16 * TM * PITCH * 4 <= 2 * KG * XBYTES, "the sums lie where the tokens lay");
    __shared__ __align__(16) unsigned char xs[KG][2][XBYTES];
    __shared__ __align__(16) unsigned char turned[KG * CW][NT * 2048];
    const int lane = static_cast<int>(threadIdx.x) & 63, nl = lane & 15, kq = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6);
    const int cw = wave % CW, kg = wave / CW, tid = static_cast<int>(threadIdx.x) % (CW * 64);
    const int64_t t0 = static_cast<int64_t>(blockIdx.y) * (16 * TM);
    const int tokens = static_cast<int>(a.T - t0 < 16 * TM ? a.T - t0 : 16 * TM);
    const Codes<NT, PER> codes(a, turned[wave], lane);
    const int64_t whole = codes.whole, lines = (a.d_in + LINE - 1) / LINE;
    const int64_t rounds = (lines + KG - 1) / KG;
    const int64_t tile = static_cast<int64_t>(blockIdx.x) * CW + cw;
    const bool mine = tile * (16 * NT) < a.d_out;

    Line<NT, PER> ring[D];
#pragma unroll
    for (int k = 0; k < D; ++k)
        codes.load(ring[k], mine ? tile : 0, kg + k * KG, mine && kg + k * KG < whole);

    // the tokens' line: thread i takes chunks i, i + threads, ... (32 a token)
    struct Tokens {
        Raw8<T> v[LOADS];
    };
    // (uniform addresses and the thread's place in bytes, of 32 bits: 64 rows below 2^23 at most)
    const T *const xrows = static_cast<const T *>(a.x) + t0 * a.d_in;
    unsigned int place[LOADS];
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
        const int v = tid + i * CW * 64, r = v / 32;
        place[i] = sizeof(T) * ((r < tokens ? r : tokens - 1) * static_cast<unsigned int>(a.d_in) +
                                8 * (v % 32));
    }
    auto fetch = [&](Tokens &x, int64_t line, auto WHOLE) {
#pragma unroll
        for (int i = 0; i < LOADS; ++i)
            x.v[i].template load<true>(reinterpret_cast<const T *>(
                                           reinterpret_cast<const unsigned char *>(xrows + line * LINE) +
                                           place[i]),
                                       WHOLE() ? 8 : count8(a.d_in, line * LINE + 8 * (tid % 32)));
    };
    using Yes = std::true_type;
    // (the next whole line, or the last one again, with no branch; the row's end apart)
    auto fetch_next = [&](Tokens &x, int64_t line) {
        fetch(x, line < whole ? line : whole - 1, Yes());
        if (line == whole && whole < lines)
            fetch(x, line, std::false_type());
    };
    auto keep = [&](const Tokens &x, int buf) {
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            const int v = tid + i * CW * 64, r = v / 32, c = v % 32;
            unsigned int w[P][4];
            split8(x.v[i], w);
#pragma unroll
            for (int p = 0; p < P; ++p)
                *reinterpret_cast<u32x4_t *>(&xs[kg][buf][(p * 16 * TM + r) * ROW +
                                                          16 * (c ^ swizzle_line(r))]) =
                    u32x4_t{w[p][0], w[p][1], w[p][2], w[p][3]};
        }
    };
    Sums<TM, NT> sum;
    sum.clear();
    auto products = [&](const Line<NT, PER> &l, int buf) {
        codes.turn(l);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            unsigned int c[NT][4];
            codes.half(c, h);
#pragma unroll
            for (int s = 4 * h; s < 4 * h + 4; ++s) {
                bf16x8_t x[TM][P];
#pragma unroll
                for (int i = 0; i < TM; ++i)
#pragma unroll
                    for (int p = 0; p < P; ++p)
                        x[i][p] = __builtin_bit_cast(
                            bf16x8_t, *reinterpret_cast<const u32x4_t *>(
                                          &xs[kg][buf][(p * 16 * TM + 16 * i + nl) * ROW +
                                                       16 * ((4 * s + kq) ^ swizzle_line(nl))]));
                sum.step(x, c, l, s);
            }
        }
    };
    // XD lines of the tokens are on their way.  Loads return in order, so that a wait for them is one
    // for all codes loaded before them too: two lines where few waves are there to fill it, one
    // where the registers of more waves are worth more.
    Tokens x[XD];
    fetch_next(x[0], kg);
    if constexpr (XD == 2)
        fetch_next(x[1], kg + KG);
    keep(x[0], 0);
    __syncthreads();
    for (int64_t r0 = 0; r0 < rounds; r0 += 2) {
#pragma unroll
        for (int d = 0; d < 2; ++d) {
            const int64_t line = kg + (r0 + d) * KG;
            fetch_next(x[d % XD], line + XD * KG);
            if (line < whole) {
                products(ring[d % D], d);
            } else if (line < lines && mine) {
                Line<NT, PER> l;
                codes.load_tail(l, tile);
                products(l, d);
            }
            const int64_t ahead = line + static_cast<int64_t>(D) * KG;
            codes.load(ring[d % D], mine ? tile : 0, ahead, mine && ahead < whole);
            keep(x[(d ^ 1) % XD], d ^ 1);
            __syncthreads();
        }
    }
    float *const sums = reinterpret_cast<float *>(&xs[0][0][0]);
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q)
                sums[(kg * 16 * TM + 16 * i + 4 * kq + q) * PITCH + 16 * (cw * NT + j) + nl] =
                    sum.acc[i][j][q];
    __syncthreads();
    const int64_t n0 = static_cast<int64_t>(blockIdx.x) * (CW * 16 * NT);
    for (int e = static_cast<int>(threadIdx.x); e < tokens * CW * 16 * NT; e += CW * KG * 64) {
        const int m = e / (CW * 16 * NT), n = e % (CW * 16 * NT);
        if (n0 + n >= a.d_out)
            continue;
        float v = sums[m * PITCH + n];
#pragma unroll
        for (int g = 1; g < KG; ++g)
            v += sums[(g * 16 * TM + m) * PITCH + n];
        put(static_cast<T *>(a.y) + (t0 + m) * a.d_out + n0 + n, v);
    }
}

constexpr int FEW_WAVES = 16;
template <typename T>
size_t few_lds(const FourbitArgs &a)
{
    const int64_t xpitch = (a.d_in + LINE - 1) / LINE * LINE + 8;
    return static_cast<size_t>(planes<T> * (a.T < FEW ? a.T : FEW) * xpitch * 2);
}

template <typename T, int PER>
hipError_t launch_few(const FourbitArgs &a, hipStream_t st)
{
    // (with 43 KiB of the waves' sums and lines)
    if (few_lds<T>(a) > 64 * 1024)
        return hipErrorInvalidValue;
    const int64_t tiles = (a.d_out + 15) / 16, rounds = (tiles + 255) / 256;
    const dim3 grid(static_cast<unsigned>((tiles + rounds - 1) / rounds),
                    static_cast<unsigned>((a.T + FEW - 1) / FEW));
    hipLaunchKernelGGL((linear_fourbit_kernel<T, PER, FEW_WAVES>), grid, dim3(FEW_WAVES * 64),
                       few_lds<T>(a), st, a);
    return hipGetLastError();
}

template <typename T, int TM, int NT, int PER, int CW, int KG, int D, int XD = 2>
hipError_t launch_shared(const FourbitArgs &a, hipStream_t st)
{
    constexpr size_t LDS = 2 * KG * planes<T> * 16 * TM * LINE * 2 + KG * CW * NT * 2048;
    static_assert(LDS <= 160 * 1024, "LDS");
    const dim3 grid(static_cast<unsigned>((a.d_out + CW * 16 * NT - 1) / (CW * 16 * NT)),
                    static_cast<unsigned>((a.T + 16 * TM - 1) / (16 * TM)));
    hipLaunchKernelGGL((linear_fourbit_shared_kernel<T, TM, NT, PER, CW, KG, D, XD>), grid,
                       dim3(CW * KG * 64), 0, st, a);
    return hipGetLastError();
}

// Up to four tokens whose rows fit in LDS, and rows of less than a line, take the first kernel.
// The other one's tile is the widest that makes 192 workgroups (us at 14336 channels of 4096, 24
// tokens: 64 channels 14, 128 19, 32 20; at 8192 of 8192: 32 channels 18, 64 23, 128 34), with
// the K groups that LDS holds (64 channels of 14336, 32 tokens: four 36 us, two 40; 128 channels of
// 8192, 24 tokens, eight waves of 16 channels in two groups 39.5, four of 32 in two 42); 33 to
// 64 tokens over many channels share a read of the codes (28672 of 8192, 48 tokens: four waves of
// 32 channels in two groups 53, eight of 16 in one 59, two blocks of 32 tokens 74).
template <typename T, int PER>
hipError_t launch_per(const FourbitArgs &a, hipStream_t st)
{
    if (a.d_in < LINE || (a.T <= FEW && few_lds<T>(a) <= 64 * 1024))
        return launch_few<T, PER>(a, st);
    auto fills = [&](int channels, int tokens) {
        return (a.d_out + channels - 1) / channels * ((a.T + tokens - 1) / tokens) >= 192;
    };
    if constexpr (sizeof(T) == 4) {
        // (three planes of the tokens: 16 of them at a time)
        if (fills(64, 16))
            return launch_shared<T, 1, 1, PER, 4, 2, 2>(a, st);
        return launch_shared<T, 1, 1, PER, 2, 2, 2>(a, st);
    } else {
        if (a.T <= 16)
            return fills(64, 16) ? launch_shared<T, 1, 1, PER, 4, 2, 2>(a, st)
                                 : launch_shared<T, 1, 1, PER, 2, 4, 1>(a, st);
        if (a.T > 32 && fills(128, 64))
            return launch_shared<T, 4, 2, PER, 4, 2, 1, 1>(a, st);
        if (fills(128, 32))
            return launch_shared<T, 2, 1, PER, 8, 2, 1, 1>(a, st);
        if (fills(64, 32))
            return launch_shared<T, 2, 1, PER, 4, 4, 1, 1>(a, st);
        return launch_shared<T, 2, 1, PER, 2, 4, 1>(a, st);
    }
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
