// gemm_i8_rows.hip - the int8 product for a few tokens (gfx950): y = xq wq^T
// scaled by token and output channel, up to 64 tokens, widths d_in of whole
// 16-byte chunks.
//
// Bound by reading wq once.  A workgroup takes BN output channels; its four
// waves split K, wave w taking the 128-byte stages w, w + 4, ... (so the
// workgroup reads 512 consecutive bytes of each row at a time).  A wave streams
// its stages of wq and of the tokens through an LDS ring of its own, loaded
// directly from memory (buffer_load ... lds: 8 rows x 128 bytes an instruction,
// whole lines) D - 1 stages ahead, and needs no barrier until the end, where
// the four waves' int32 sums (exact in any order) meet in LDS, are scaled,
// rounded once and stored.  The layout in LDS and the fragments are those of
// the pipelined kernel.
#include "gemm_dma_launch.hpp"
#include "rows8.hpp"

namespace dora {
namespace dma {

typedef int i32x4_t __attribute__((ext_vector_type(4)));

constexpr int ROWS_WAVES = 4;

// TM: blocks of 16 tokens; D: ring slots of a wave.
template <int TM, int BN, int D, typename T>
__global__ void __launch_bounds__(ROWS_WAVES * 64) gemm_i8_rows_kernel(I8GemmArgs g)
{
    constexpr int TN = BN / 16;
    constexpr int G = BN / 8 % 4 == 0 && TM % 2 == 0 ? 4 : 2;
    using DA = OperandDma<true, 16 * TM, 1, G>;
    using DB = OperandDma<true, BN, 1, G>;
    constexpr int LPS = DA::PER + DB::PER;  // loads of a stage
    constexpr int A_BYTES = 16 * TM * ROW_BYTES, SLOT = A_BYTES + BN * ROW_BYTES;
    static_assert((D - 1) * LPS < 64, "vmcnt range");
    constexpr int PITCH = BN + 4;  // int32 sums of a token
    constexpr int SUMS = ROWS_WAVES * 16 * TM * PITCH * 4;
    constexpr int SMEM = ROWS_WAVES * D * SLOT > SUMS ? ROWS_WAVES * D * SLOT : SUMS;
    static_assert(SMEM <= 160 * 1024, "LDS");
    __shared__ __align__(1024) unsigned char smem[SMEM];

    const int lane = static_cast<int>(threadIdx.x) & 63;
    const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6);
    const int64_t n0 = static_cast<int64_t>(blockIdx.x) * BN;
    const int64_t ld = g.K / 2;  // the rows as 2-byte elements
    const int nst = static_cast<int>((g.K + 2 * BK - 1) / (2 * BK));
    const int mine = nst > wave ? (nst - wave + ROWS_WAVES - 1) / ROWS_WAVES : 0;
    DA da;
    DB db;
    da.init(g.M, ld, 0, 0, lane);
    db.init(g.N, ld, n0, 0, lane);
    const int na = range_bytes(g.M * g.K), nb = range_bytes(g.N * g.K);
    unsigned char *const ring = smem + wave * (D * SLOT);

    // the loads of the wave's stage s into its slot
    auto load = [&](int s, int at) {
        const int kd = (wave + s * ROWS_WAVES) * BK;
        const uint32_t lds = __builtin_amdgcn_readfirstlane(
            static_cast<uint32_t>(reinterpret_cast<uintptr_t>((lds_void *)(ring + at * SLOT))));
        const uint32_t soff = static_cast<uint32_t>(kd * 2);
        const __amdgpu_buffer_rsrc_t ra = scalar_rsrc(g.x, na), rb = scalar_rsrc(g.w, nb);
        static_for<LPS / G>([&](auto gc) {
            constexpr int d = decltype(gc)::value;
            constexpr bool isa = d < DA::PER / G;
            constexpr int i0 = (isa ? d : d - DA::PER / G) * G;
            uint32_t v[G];
#pragma unroll
            for (int j = 0; j < G; ++j) {
                const uint32_t kc = isa ? DA::kchunk(0, i0 + j, lane) : DB::kchunk(0, i0 + j, lane);
                v[j] = kd + static_cast<int>(kc) < static_cast<int>(ld)
                           ? (isa ? da.off[i0 + j] : db.off[i0 + j])
                           : OOB_OFFSET;
            }
            set_m0(lds + (isa ? 0 : A_BYTES) + i0 * 1024);
            static_for<G>([&](auto jc) {
                constexpr int J = decltype(jc)::value;
                lds_dma16<J>(isa ? ra : rb, v[J], soff);
            });
        });
    };

    i32x4_t acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
            acc[i][j] = i32x4_t{0, 0, 0, 0};
    auto products = [&](int at) {
        const unsigned char *As = ring + at * SLOT, *Bs = As + A_BYTES;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            i32x4_t fa[TM], fb[TN];
#pragma unroll
            for (int i = 0; i < TM; ++i)
                fa[i] = __builtin_bit_cast(i32x4_t, read_frag16(As, 16 * i, h, lane));
#pragma unroll
            for (int j = 0; j < TN; ++j)
                fb[j] = __builtin_bit_cast(i32x4_t, read_frag16(Bs, 16 * j, h, lane));
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int j = 0; j < TN; ++j)
                    acc[i][j] =
                        __builtin_amdgcn_mfma_i32_16x16x64_i8(fb[j], fa[i], acc[i][j], 0, 0, 0);
        }
    };

#pragma unroll
    for (int s = 0; s < D - 1; ++s)
        if (s < mine)
            load(s, s);
    int at = 0, fill = D - 1;  // the slot read next, the slot filled next
#pragma unroll 1
    for (int s = 0; s < mine; ++s) {
        // the previous stage's fragments are in registers: its slot is free
        wait_lgkm0();
        if (s + D - 1 < mine) {
            load(s + D - 1, fill);
            wait_vmcnt<(D - 1) * LPS>();
        } else {
            wait_vmcnt<0>();
        }
        __asm__ volatile("" ::: "memory");
        products(at);
        __asm__ volatile("" ::: "memory");
        at = at + 1 == D ? 0 : at + 1;
        fill = fill + 1 == D ? 0 : fill + 1;
    }
    __syncthreads();  // every wave is done with its ring

    int *const sums = reinterpret_cast<int *>(smem);
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
            *reinterpret_cast<i32x4_t *>(sums + (wave * 16 * TM + 16 * i + (lane & 15)) * PITCH +
                                         16 * j + 4 * (lane >> 4)) = acc[i][j];
    __syncthreads();
    const int tokens = static_cast<int>(g.M);
    for (int e = static_cast<int>(threadIdx.x); e < tokens * BN; e += ROWS_WAVES * 64) {
        const int m = e / BN, n = e % BN;
        if (n0 + n >= g.N)
            continue;
        int c = 0;
#pragma unroll
        for (int w = 0; w < ROWS_WAVES; ++w)
            c += sums[(w * 16 * TM + m) * PITCH + n];
        const float v = i8_scaled(c, i8_xs(g.xs[m]), g.ws[n0 + n]);
        T *out = static_cast<T *>(g.y) + m * g.N + n0 + n;
        if constexpr (sizeof(T) == 2)
            *out = f32_to_bf16(v);
        else
            *out = v;
    }
}

template <int TM, int BN, int D>
hipError_t launch_rows(int bf16, const I8GemmArgs &g, hipStream_t st)
{
    const dim3 grid(static_cast<unsigned>((g.N + BN - 1) / BN)), block(ROWS_WAVES * 64);
    if (bf16)
        hipLaunchKernelGGL((gemm_i8_rows_kernel<TM, BN, D, uint16_t>), grid, block, 0, st, g);
    else
        hipLaunchKernelGGL((gemm_i8_rows_kernel<TM, BN, D, float>), grid, block, 0, st, g);
    return hipGetLastError();
}

}  // namespace dma

// Which products run here, and how many channels a workgroup takes and slots a
// ring has.  More channels read the tokens' rows less often; fewer make more
// workgroups.  Measured (us, d_in -> d_out):
//   up to 16 tokens   16 channels, two workgroups a CU (8192 -> 28672: 42 at one
//                     token, 46 at 16; 32 channels 54, 57; the pipelined kernel
//                     51), but 32 where they make one round of the CUs and 16 make
//                     two (4096 -> 14336: 14 against 17)
//   up to 32          64 channels (8192 -> 28672: 51, 32 channels 60; 8192 -> 8192:
//                     19, 21), 16 where that is one round (14336 -> 4096: 16, 64
//                     channels 28)
//   up to 64          while one round of the CUs takes them: 16 channels up to 4096
//                     (14336 -> 4096: 24, 32 channels 28), 32 up to 8192 (8192 ->
//                     8192: 23, 64 channels 25); beyond, the pipelined kernel is as
//                     fast (4096 -> 14336: 16, 64 channels here 17; 8192 -> 28672: 51,
//                     56)
bool gemm_i8_rows_ok(int64_t M, int64_t N) { return M <= 32 || (M <= 64 && N <= 8192); }

hipError_t launch_gemm_i8_rows(int bf16, const I8GemmArgs &g, hipStream_t st)
{
    if (!gemm_i8_rows_ok(g.M, g.N))
        return hipErrorInvalidValue;
    const bool few = g.N <= 4096;
    if (g.M <= 16)
        return g.N > 8192 && g.N <= 16384 ? dma::launch_rows<1, 32, 3>(bf16, g, st)
                                          : dma::launch_rows<1, 16, 4>(bf16, g, st);
    if (g.M <= 32)
        return few ? dma::launch_rows<2, 16, 4>(bf16, g, st) : dma::launch_rows<2, 64, 3>(bf16, g, st);
    return few ? dma::launch_rows<4, 16, 3>(bf16, g, st) : dma::launch_rows<4, 32, 2>(bf16, g, st);
}

}  // namespace dora
