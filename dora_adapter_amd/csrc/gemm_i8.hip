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
// registers.  256 x 256 (eight waves), 128 x 128 or 64 x 64 (four) tiles, 128 bytes of K
// a step in two LDS buffers; the next step's loads are in flight during this
// one's products.
#include "dora_internal.hpp"
#include "gemm_bf16_dma.hpp"
#include "ragged.hpp"
#include "rows8.hpp"

namespace dora {
namespace {

typedef int i32x4_t __attribute__((ext_vector_type(4)));

constexpr int GK = 128;          // bytes of K a step
constexpr int GPITCH = GK + 16;  // LDS row: 8 rows of a 16-byte read phase on distinct banks
constexpr int GTHREADS = 256;

// The first `left` bytes at p, one by one (operands of fewer than 16 bytes).
__device__ __forceinline__ i32x4_t load_bytes(const int8_t *p, int64_t left)
{
    unsigned int w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int b = 0; b < 15; ++b)
        if (b < left)
            w[b >> 2] |= static_cast<unsigned int>(static_cast<uint8_t>(p[b])) << (8 * (b & 3));
    return i32x4_t{static_cast<int>(w[0]), static_cast<int>(w[1]), static_cast<int>(w[2]),
                   static_cast<int>(w[3])};
}

// Four consecutive outputs of row m from column n on.
template <typename T>
__device__ __forceinline__ void store_scaled(const I8GemmArgs &g, int64_t m, int64_t n,
                                             const int (&c)[4], I8Scale sx)
{
    T *out = static_cast<T *>(g.y) + m * g.N + n;
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (n + e < g.N) {
            const float v = i8_scaled(c[e], sx, g.ws[n + e]);
            if constexpr (sizeof(T) == 2)
                out[e] = f32_to_bf16(v);
            else
                out[e] = v;
        }
}

// B x B tiles of 2 x WN waves (B / 2 rows x B / WN columns each); AHEAD: steps
// whose loads are in flight in registers; TINY: an operand of fewer than 16 bytes.
template <int B, int WN, int AHEAD, bool TINY, typename T>
__global__ void __launch_bounds__(128 * WN, 2) gemm_i8_general_kernel(I8GemmArgs g)
{
    constexpr int NT = 128 * WN, ROWS = NT / 8;  // threads; rows they load at a time
    constexpr int WTN = B / WN, TM = B / 32, TN = WTN / 16, PER = B / ROWS;
    __shared__ __align__(16) unsigned char lds[2][2][B * GPITCH];
    const int tid = static_cast<int>(threadIdx.x), lane = tid & 63, wave = tid >> 6;
    const int wm = (wave / WN) * (B / 2), wn = (wave % WN) * WTN;
    int tm, tn;
    tile_coords(g.M, g.N, B, B, tm, tn);
    const int64_t m0 = static_cast<int64_t>(tm) * B, n0 = static_cast<int64_t>(tn) * B;
    const int64_t kb = static_cast<int64_t>(blockIdx.y) * g.k_per_split;
    const int64_t ke = kb + g.k_per_split < g.K ? kb + g.k_per_split : g.K;

    // thread: chunk tid & 7 of rows (tid >> 3) + ROWS i of either operand (rows
    // past the end: the last one, never stored), as offsets of their first byte
    const int lr = tid >> 3, lc = (tid & 7) * 16;
    int64_t ao[PER], bo[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int64_t m = m0 + lr + ROWS * i, n = n0 + lr + ROWS * i;
        ao[i] = (m < g.M ? m : g.M - 1) * g.K + lc;
        bo[i] = (n < g.N ? n : g.N - 1) * g.K + lc;
    }
    struct Regs {
        i32x4_t a[PER], b[PER];
    } regs[AHEAD];
    // The loads of K values k .. k + GK - 1: whole chunks, without a branch or a
    // wait among them.  Where the row ends they run into the next one, and at the
    // operand's end they start early; the last step's are put right when they
    // go to LDS (row_end16).
    const int64_t alim = g.M * g.K - 16, blim = g.N * g.K - 16;
    auto load16 = [](const int8_t *p) {
        return __builtin_bit_cast(i32x4_t, load16_any(p));
    };
    auto ended = [](i32x4_t v, int back, int64_t left) {
        return __builtin_bit_cast(i32x4_t, row_end16(__builtin_bit_cast(uint4, v), back, left));
    };
    auto fetch = [&](Regs &r, int64_t k) {
        if constexpr (TINY) {
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                r.a[i] = load_bytes(g.x + ao[i] + k, g.K - k - lc);
                r.b[i] = load_bytes(g.w + bo[i] + k, g.K - k - lc);
            }
        } else if (k + GK <= g.K) {
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                r.a[i] = load16(g.x + ao[i] + k);
                r.b[i] = load16(g.w + bo[i] + k);
            }
        } else {
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                r.a[i] = load16(g.x + (ao[i] + k < alim ? ao[i] + k : alim));
                r.b[i] = load16(g.w + (bo[i] + k < blim ? bo[i] + k : blim));
            }
        }
    };
    auto row_ends = [&](Regs &r, int64_t k) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int64_t ab = ao[i] + k - alim, bb = bo[i] + k - blim, left = g.K - k - lc;
            r.a[i] = ended(r.a[i], ab > 0 && left > 0 ? static_cast<int>(ab) : 0, left);
            r.b[i] = ended(r.b[i], bb > 0 && left > 0 ? static_cast<int>(bb) : 0, left);
        }
    };
    i32x4_t acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
            acc[i][j] = i32x4_t{0, 0, 0, 0};
    int at = 0;
    const int64_t steps = kb < ke ? (ke - kb + GK - 1) / GK : 0;
    auto k_of = [&](int64_t s) { return kb + (s < steps ? s : steps - 1) * GK; };
    // step s from the registers r, which then take step s + AHEAD (past the end
    // the last one again: the loads in flight are always the same number, which
    // the waits before their use count on).  One barrier a step: a wave past it
    // is done with the other buffer's fragments, which the next step overwrites.
    auto step = [&](Regs &r, int64_t s) {
        if (!TINY && k_of(s) + GK > g.K)
            row_ends(r, k_of(s));
        unsigned char *const As = lds[at][0], *const Bs = lds[at][1];
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            *reinterpret_cast<i32x4_t *>(As + (lr + ROWS * i) * GPITCH + lc) = r.a[i];
            *reinterpret_cast<i32x4_t *>(Bs + (lr + ROWS * i) * GPITCH + lc) = r.b[i];
        }
        // (a bare barrier behind this wave's LDS writes: __syncthreads would wait
        // for the loads in flight as well)
        dma::wait_lgkm0();
        dma::stage_barrier();
        fetch(r, k_of(s + AHEAD));
#pragma unroll
        for (int h = 0; h < GK / 64; ++h) {
            i32x4_t fa[TM], fb[TN];
            const int c = h * 64 + (lane >> 4) * 16;
#pragma unroll
            for (int i = 0; i < TM; ++i)
                fa[i] = *reinterpret_cast<const i32x4_t *>(
                    As + (wm + 16 * i + (lane & 15)) * GPITCH + c);
#pragma unroll
            for (int j = 0; j < TN; ++j)
                fb[j] = *reinterpret_cast<const i32x4_t *>(
                    Bs + (wn + 16 * j + (lane & 15)) * GPITCH + c);
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int j = 0; j < TN; ++j)
                    acc[i][j] =
                        __builtin_amdgcn_mfma_i32_16x16x64_i8(fb[j], fa[i], acc[i][j], 0, 0, 0);
        }
        at ^= 1;
    };
    if (steps > 0) {
#pragma unroll
        for (int p = 0; p < AHEAD; ++p)
            fetch(regs[p], k_of(p));
        int64_t s = 0;
        for (; s + AHEAD <= steps; s += AHEAD) {
#pragma unroll
            for (int p = 0; p < AHEAD; ++p)
                step(regs[p], s + p);
        }
#pragma unroll
        for (int p = 0; p < AHEAD - 1; ++p)
            if (s + p < steps)
                step(regs[p], s + p);
    }
#pragma unroll
    for (int i = 0; i < TM; ++i) {
        const int64_t m = m0 + wm + 16 * i + (lane & 15);
        if (m >= g.M)
            continue;
        const I8Scale sx = i8_xs(g.xs[m]);
#pragma unroll
        for (int j = 0; j < TN; ++j) {
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
        const float v = i8_scaled(c, i8_xs(g.xs[e / g.N]), g.ws[e % g.N]);
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

// The pipelined kernel's tiles: microseconds a stage takes an item with one
// and with all of its workgroups resident on a CU, and microseconds an item
// takes beside its stages (epilogue, drain).  Fitted to measurements between
// 128 and 8192 tokens, 512 and 8192 wide, 4096 and 28672 channels; for
// instance (us, tile and slots in LDS): 128 tokens, 4096 -> 14336: 128 x 64 of
// four 20, 128 x 128 of four 25, of two 33, 64 x 64 24, 256 x 256 54; 512 tokens,
// 8192 -> 8192: 128 x 128 of four 43, 128 x 64 58, 128 x 128 of two 60; 2048
// tokens, 4096 -> 4096: 128 x 128 of two 36, of four 42, 256 x 256 51.
struct I8Tile {
    int bm, bn, resident;
    double stage_one, stage_all, item;
};
constexpr I8Tile I8_TILES[] = {{256, 256, 1, 1.5, 1.5, 8.0},
                               {128, 128, 2, 0.7, 0.95, 2.5},
                               {128, 128, 1, 0.56, 0.56, 1.5},
                               {128, 64, 1, 0.43, 0.43, 1.0},
                               {64, 64, 2, 0.34, 0.5, 1.0}};
constexpr int I8_NUM_TILES = sizeof(I8_TILES) / sizeof(I8_TILES[0]);

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// The general kernel's tile: 256 x 256 where there is one for every CU (its steps
// have the products to cover their loads: 8192 tokens, 8190 -> 28672 2.9 ms, 128 x
// 128 3.8), 64 x 64 where there is no 128 x 128 one for every CU.
int64_t general_tile(int64_t M, int64_t N, int64_t K)
{
    if (M * K < 16 || N * K < 16)
        return 64;
    if (ceil_div(M, 256) * ceil_div(N, 256) >= 256)
        return 256;
    return ceil_div(M, 128) * ceil_div(N, 128) < 256 ? 64 : 128;
}

}  // namespace

I8Plan plan_gemm_i8(int64_t M, int64_t N, int64_t K)
{
    I8Plan p{I8Plan::GENERAL, 1, 0, 0};
    const bool dma = K % 16 == 0 && M * K < I8_MAX_BYTES && N * K < I8_MAX_BYTES;
    if (dma && gemm_i8_rows_ok(M, N)) {
        p.cfg = I8Plan::ROWS;
    } else if (dma && M * N * 4 < I8_MAX_BYTES) {
        // (four bytes an output whichever its type: a y of 1 to 2 GiB in bf16 takes the
        // general kernel, at half the rate)
        // rounds of resident workgroups, each its items' stages; a split writes
        // and reads int32 partial sums and launches once more
        const int64_t stages = ceil_div(K, I8_STAGE_K);
        double best = -1.0;
        for (int c = 0; c < I8_NUM_TILES; ++c) {
            const I8Tile &t = I8_TILES[c];
            const int64_t tiles = ceil_div(M, t.bm) * ceil_div(N, t.bn);
            for (int64_t z = 1; z <= 16 && (z == 1 || stages / z >= 4); ++z) {
                const int64_t sps = ceil_div(stages, z);
                if (ceil_div(stages, sps) != z || z * M * N * 4 >= I8_MAX_BYTES)
                    continue;
                const int64_t rounds = ceil_div(tiles * z, 256 * t.resident);
                const double stage = tiles * z <= 256 ? t.stage_one : t.stage_all;
                double us = 5.0 + static_cast<double>(rounds) * (sps * stage + t.item);
                if (z > 1)
                    us += 8.0 * z * M * N / 4.0e6 + 5.0;
                if (best < 0 || us < best) {
                    best = us;
                    p.cfg = c;
                    p.splits = static_cast<int>(z);
                    p.k_per_split = sps * I8_STAGE_K;
                }
            }
        }
    } else {
        // split K until two workgroups a CU are reached, four steps a split at
        // least
        const int64_t b = general_tile(M, N, K), tiles = ceil_div(M, b) * ceil_div(N, b);
        const int64_t steps = ceil_div(K, GK);
        int64_t z = b < 256 && tiles > 0 ? 512 / tiles : 1;
        z = z < steps / 4 ? z : steps / 4;
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
        const int64_t b = general_tile(g.M, g.N, g.K), tiles = ceil_div(g.M, b) * ceil_div(g.N, b);
        const dim3 grid(static_cast<unsigned>(tiles), static_cast<unsigned>(p.splits));
        const dim3 block(b == 256 ? 512 : 256);
        if (tiles >= (int64_t(1) << 32) / block.x)  // a launch holds fewer than 2^32 threads
            return hipErrorInvalidConfiguration;
        if (b == 64 && (g.M * g.K < 16 || g.N * g.K < 16)) {
            if (bf16)
                hipLaunchKernelGGL((gemm_i8_general_kernel<64, 2, 1, true, uint16_t>), grid, block, 0,
                                   st, g);
            else
                hipLaunchKernelGGL((gemm_i8_general_kernel<64, 2, 1, true, float>), grid, block, 0, st,
                                   g);
        } else if (b == 256 && bf16)
            hipLaunchKernelGGL((gemm_i8_general_kernel<256, 4, 1, false, uint16_t>), grid, block, 0, st, g);
        else if (b == 256)
            hipLaunchKernelGGL((gemm_i8_general_kernel<256, 4, 1, false, float>), grid, block, 0, st, g);
        else if (b == 128 && bf16)
            hipLaunchKernelGGL((gemm_i8_general_kernel<128, 2, 2, false, uint16_t>), grid, block, 0, st, g);
        else if (b == 128)
            hipLaunchKernelGGL((gemm_i8_general_kernel<128, 2, 2, false, float>), grid, block, 0, st, g);
        else if (bf16)
            hipLaunchKernelGGL((gemm_i8_general_kernel<64, 2, 3, false, uint16_t>), grid, block, 0, st, g);
        else
            hipLaunchKernelGGL((gemm_i8_general_kernel<64, 2, 3, false, float>), grid, block, 0, st, g);
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
