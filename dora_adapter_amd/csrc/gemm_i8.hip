// gemm_i8.hip - y = (xq wq^T) scaled by token and output channel (gfx950):
// y[t, i] = xs[t] ws[i] sum_k xq[t, k] wq[i, k], int8 operands, int32 sums
// (exact: the width is at most 131071, and 128 * 128 * 131071 < 2^31), scaled
// in fp32 and rounded once.
//
// v_mfma_i32_16x16x64_i8 reads 16 bytes of a row per lane, as the bf16
// 16 x 16 x 32 form does, so an int8 row of K bytes moves and lies in LDS
// exactly like a bf16 row of K / 2 elements.  W's fragment goes first: lane l
// of an accumulator block then holds output row l & 15 and the four
// consecutive columns 4 (l >> 4) + 0..3.
//
// The general kernel: any width and alignment, operands staged through
// registers.  128 x 128 tiles of four waves (64 x 64 each), 64 bytes of K a
// step; the next step's loads are in flight during this one's products.
#include "dora_internal.hpp"
#include "rows8.hpp"

namespace dora {
namespace {

typedef int i32x4_t __attribute__((ext_vector_type(4)));

constexpr int GB = 128;           // tile rows and columns
constexpr int GK = 64;            // bytes of K a step
constexpr int GPITCH = GK + 16;   // LDS row: 8 rows of a 16-byte read phase on distinct banks
constexpr int GTHREADS = 256;

// 16 bytes of a row from byte k on, zeros past the width K.
__device__ __forceinline__ i32x4_t load_k16(const int8_t *row, int64_t k, int64_t K)
{
    i32x4_t v = {0, 0, 0, 0};
    if (k + 16 <= K) {
        const u32x4_a1_t u = *reinterpret_cast<const u32x4_a1_t *>(row + k);
        v[0] = static_cast<int>(u.x);
        v[1] = static_cast<int>(u.y);
        v[2] = static_cast<int>(u.z);
        v[3] = static_cast<int>(u.w);
    } else if (k < K) {
        unsigned int w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int b = 0; b < 15; ++b)
            if (k + b < K)
                w[b >> 2] |= static_cast<unsigned int>(static_cast<uint8_t>(row[k + b]))
                             << (8 * (b & 3));
#pragma unroll
        for (int q = 0; q < 4; ++q)
            v[q] = static_cast<int>(w[q]);
    }
    return v;
}

// Four consecutive outputs of row m from column n on.
template <typename T>
__device__ __forceinline__ void store_scaled(const I8GemmArgs &g, int64_t m, int64_t n,
                                             const int (&c)[4], float sx)
{
    T *out = static_cast<T *>(g.y) + m * g.N + n;
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (n + e < g.N) {
            const float v = static_cast<float>(c[e]) * (sx * g.ws[n + e]);
            if constexpr (sizeof(T) == 2)
                out[e] = f32_to_bf16(v);
            else
                out[e] = v;
        }
}

template <typename T>
__global__ void __launch_bounds__(GTHREADS) gemm_i8_general_kernel(I8GemmArgs g)
{
    __shared__ __align__(16) unsigned char As[GB * GPITCH];
    __shared__ __align__(16) unsigned char Bs[GB * GPITCH];
    const int tid = static_cast<int>(threadIdx.x), lane = tid & 63, wave = tid >> 6;
    const int wm = (wave >> 1) * 64, wn = (wave & 1) * 64;
    const int64_t num_n = (g.N + GB - 1) / GB;
    const int64_t m0 = static_cast<int64_t>(blockIdx.x / num_n) * GB;
    const int64_t n0 = static_cast<int64_t>(blockIdx.x % num_n) * GB;
    const int64_t k_end_all = (g.K + GK - 1) / GK * GK;
    const int64_t kb = static_cast<int64_t>(blockIdx.y) * g.k_per_split;
    const int64_t ke = kb + g.k_per_split < k_end_all ? kb + g.k_per_split : k_end_all;

    // thread: chunk tid & 3 of rows tid >> 2 and 64 + (tid >> 2) of either
    // operand (rows past the end: the last one, never stored)
    const int lr = tid >> 2, lc = (tid & 3) * 16;
    const int8_t *ap[2], *bp[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int64_t m = m0 + lr + 64 * i, n = n0 + lr + 64 * i;
        ap[i] = g.x + (m < g.M ? m : g.M - 1) * g.K;
        bp[i] = g.w + (n < g.N ? n : g.N - 1) * g.K;
    }
    i32x4_t ra[2], rb[2];
    auto fetch = [&](int64_t k) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            ra[i] = load_k16(ap[i], k + lc, g.K);
            rb[i] = load_k16(bp[i], k + lc, g.K);
        }
    };
    i32x4_t acc[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            acc[i][j] = i32x4_t{0, 0, 0, 0};
    if (kb < ke)
        fetch(kb);
    for (int64_t k = kb; k < ke; k += GK) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            *reinterpret_cast<i32x4_t *>(As + (lr + 64 * i) * GPITCH + lc) = ra[i];
            *reinterpret_cast<i32x4_t *>(Bs + (lr + 64 * i) * GPITCH + lc) = rb[i];
        }
        __syncthreads();
        if (k + GK < ke)
            fetch(k + GK);
        i32x4_t fa[4], fb[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = 16 * i + (lane & 15), c = (lane >> 4) * 16;
            fa[i] = *reinterpret_cast<const i32x4_t *>(As + (wm + r) * GPITCH + c);
            fb[i] = *reinterpret_cast<const i32x4_t *>(Bs + (wn + r) * GPITCH + c);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                acc[i][j] =
                    __builtin_amdgcn_mfma_i32_16x16x64_i8(fb[j], fa[i], acc[i][j], 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t m = m0 + wm + 16 * i + (lane & 15);
        if (m >= g.M)
            continue;
        const float sx = g.xs[m];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t n = n0 + wn + 16 * j + 4 * (lane >> 4);
            const int c[4] = {acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]};
            if (g.part == nullptr) {
                store_scaled<T>(g, m, n, c, sx);
            } else {
                int *p = g.part + (static_cast<int64_t>(blockIdx.y) * g.M + m) * g.N + n;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (n + e < g.N)
                        p[e] = c[e];
            }
        }
    }
}

// The split products' sums, scaled (int32 sums are exact in any order).
template <typename T>
__global__ void __launch_bounds__(GTHREADS) i8_finish_kernel(I8GemmArgs g, int splits)
{
    const int64_t MN = g.M * g.N;
    for (int64_t e = static_cast<int64_t>(blockIdx.x) * GTHREADS + threadIdx.x; e < MN;
         e += static_cast<int64_t>(gridDim.x) * GTHREADS) {
        int c = 0;
        for (int z = 0; z < splits; ++z)
            c += g.part[static_cast<int64_t>(z) * MN + e];
        const float v = static_cast<float>(c) * (g.xs[e / g.N] * g.ws[e % g.N]);
        if constexpr (sizeof(T) == 2)
            static_cast<T *>(g.y)[e] = f32_to_bf16(v);
        else
            static_cast<T *>(g.y)[e] = v;
    }
}

}  // namespace

namespace {

constexpr int64_t I8_STAGE_K = 128;                  // bytes of K a stage of the pipelined kernel
constexpr int64_t I8_MAX_BYTES = (1LL << 31) - 8192;  // 32-bit buffer offsets
struct I8Tile {
    int bm, bn, resident;  // workgroups a CU
    double rate;           // relative rate of a full tile
};
constexpr I8Tile I8_TILES[] = {{256, 256, 1, 1.0}, {128, 128, 2, 0.8}};

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace

I8Plan plan_gemm_i8(int64_t M, int64_t N, int64_t K, int bf16)
{
    I8Plan p{I8Plan::GENERAL, 1, 0, 0};
    const int64_t elt = bf16 ? 2 : 4;
    if (M <= I8_ROWS_MOST && K % 16 == 0 && M * K < I8_MAX_BYTES && N * K < I8_MAX_BYTES) {
        p.cfg = I8Plan::ROWS;
    } else if (K % 16 == 0 && N % (16 / elt) == 0 && M * K < I8_MAX_BYTES && N * K < I8_MAX_BYTES &&
        M * N * 4 < I8_MAX_BYTES) {
        // Time of a configuration: rounds of resident workgroups, each its
        // products at the rate a full GPU sustains plus a fill and an epilogue;
        // a split writes and reads int32 partial sums and launches once more.
        const int64_t stages = ceil_div(K, I8_STAGE_K);
        double best = -1.0;
        for (int c = 0; c < 2; ++c) {
            const I8Tile &t = I8_TILES[c];
            const int64_t tiles = ceil_div(M, t.bm) * ceil_div(N, t.bn);
            for (int64_t z = 1; z <= 16 && (z == 1 || stages / z >= 4); ++z) {
                const int64_t sps = ceil_div(stages, z);
                const int64_t used = ceil_div(stages, sps);
                if (used != z || (z > 1 && z * M * N * 4 >= I8_MAX_BYTES))
                    continue;
                const int64_t slots = 256 * t.resident;
                const int64_t rounds = ceil_div(tiles * z, slots);
                const int64_t busy = tiles * z < slots ? ceil_div(tiles * z, 256) : t.resident;
                double s = static_cast<double>(rounds) *
                           (2.0 * t.bm * t.bn * sps * I8_STAGE_K * static_cast<double>(busy) /
                                (9.0e12 * t.rate) +
                            4e-6);
                if (z > 1)
                    s += 8.0 * z * M * N / 4.0e12 + 5e-6;
                if (best < 0 || s < best) {
                    best = s;
                    p.cfg = c;
                    p.splits = static_cast<int>(z);
                    p.k_per_split = sps * I8_STAGE_K;
                }
            }
        }
    } else {
        const int64_t tiles = ceil_div(M, GB) * ceil_div(N, GB);
        const int64_t steps = ceil_div(K, GK);
        // split K until two workgroups a CU are reached, eight steps a split at
        // least
        int64_t z = tiles > 0 ? 512 / tiles : 1;
        z = z < steps / 8 ? z : steps / 8;
        z = z < 1 ? 1 : (z > 32 ? 32 : z);
        const int64_t per = ceil_div(steps, z);
        p.splits = static_cast<int>(ceil_div(steps, per));
        p.k_per_split = per * GK;
    }
    p.part_bytes = p.splits > 1 ? static_cast<size_t>(p.splits) * M * N * 4 : 0;
    return p;
}

hipError_t launch_gemm_i8(int bf16, I8GemmArgs g, const I8Plan &p, void *ws, hipStream_t st)
{
    if (g.M == 0)
        return hipSuccess;
    g.part = p.splits > 1 ? static_cast<int *>(ws) : nullptr;
    g.k_per_split = p.k_per_split;
    g.splits = p.splits;
    hipError_t e = hipSuccess;
    if (p.cfg == I8Plan::ROWS) {
        e = launch_gemm_i8_rows(bf16, g, st);
    } else if (p.cfg != I8Plan::GENERAL) {
        e = launch_gemm_i8_dma(bf16, g, p.cfg, st);
    } else {
        const int64_t tiles = ceil_div(g.M, GB) * ceil_div(g.N, GB);
        if (tiles > 0x7fffffff)
            return hipErrorInvalidConfiguration;
        const dim3 grid(static_cast<unsigned>(tiles), static_cast<unsigned>(p.splits));
        if (bf16)
            hipLaunchKernelGGL((gemm_i8_general_kernel<uint16_t>), grid, dim3(GTHREADS), 0, st, g);
        else
            hipLaunchKernelGGL((gemm_i8_general_kernel<float>), grid, dim3(GTHREADS), 0, st, g);
        e = hipGetLastError();
    }
    if (e != hipSuccess || p.splits == 1)
        return e;
    int64_t blocks = ceil_div(g.M * g.N, GTHREADS);
    blocks = blocks < 8192 ? blocks : 8192;
    if (bf16)
        hipLaunchKernelGGL((i8_finish_kernel<uint16_t>), dim3(static_cast<unsigned>(blocks)),
                           dim3(GTHREADS), 0, st, g, p.splits);
    else
        hipLaunchKernelGGL((i8_finish_kernel<float>), dim3(static_cast<unsigned>(blocks)),
                           dim3(GTHREADS), 0, st, g, p.splits);
    return hipGetLastError();
}

}  // namespace dora
