// gemm_f32.hip - true-fp32 GEMM on the matrix cores for fp32 DoRA modules.
//
// Same contract as the bf16 MFMA GEMM (GemmArgs: up to two K segments,
// split-K, store / row-dot epilogues, optional row sums of squares of A) so
// that the fp32 module runs the identical factored-norm, forward and
// backward pipeline; no operand is ever rounded below fp32.
//
// v_mfma_f32_32x32x2_f32 adds its two products to the accumulator one after
// the other, each with a single rounding: bit for bit the chain of fmas in
// ascending K that a vector-ALU loop makes (tests/test_gpu_f32_sums.py holds it to that
// on ordinary, cancelling and denormal operands), at twice the rate those reach.  A sum's order
// is thus K ascending within its split, and does not depend on the tile.
//
// 64 x 64 tiles of four waves (32 x 32 each), K in granules of 16 (the unit of
// the splits; each segment's last one is filled with zeros), two granules a
// step, double-buffered in LDS, the next two steps' loads in flight.  A
// K-major operand lies in LDS as rows of K with the even K values of every
// eight before the odd ones, so that one 16-byte read gives a lane (the lower
// 32 lanes hold even K, the upper odd) its operand of four MFMAs; an MN-major
// one lies as it comes, [K][64], read four bytes at a time.  x W^T of 4096 tokens,
// 4096 -> 4096: 1.46 ms (94 TFLOP/s; the vendor library 0.92), against 2.34 on the
// vector ALUs; 1024 tokens, 2048 -> 4096: 0.19 against 0.39.
#include "dora_internal.hpp"
#include "epilogue.hpp"
#include "gemm_bf16_dma.hpp"

#include <type_traits>

namespace dora {
namespace {

constexpr int BM = GEMM_F32_BM, BN = GEMM_F32_BN, BK = GEMM_F32_BK, NT = 256;
static_assert(BM == 64 && BN == 64 && BK == 16, "thread and wave layout");
constexpr int STEP = 2;                  // granules a step
constexpr int AHEAD = 2;                 // steps whose loads are in flight
constexpr int KPITCH = STEP * BK + 4;    // floats of a K-major LDS row
constexpr int MPITCH = 64 + 4;           // floats of an MN-major LDS row

typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef float f32x4_a4_t __attribute__((ext_vector_type(4), aligned(4)));

// One operand's share of a granule: four floats a thread, consecutive in
// memory (K-major: row tid / 4, K 4 (tid % 4) ...; MN-major: K tid / 16, M or N
// 4 (tid % 16) ...), zeros past K and past the last row or column.
template <bool KMAJ>
__device__ __forceinline__ float4 load4(const float *__restrict__ p, int64_t ld, int64_t MN,
                                        int64_t K, int64_t mn0, int64_t k0, int tid)
{
    const int64_t row = KMAJ ? mn0 + (tid >> 2) : k0 + (tid >> 4);
    const int64_t col = KMAJ ? k0 + (tid & 3) * 4 : mn0 + (tid & 15) * 4;
    const int64_t left = (row < (KMAJ ? MN : K) ? (KMAJ ? K : MN) : 0) - col;
    const float *q = p + row * ld + col;
    if (left >= 4) {
        const f32x4_a4_t v = *reinterpret_cast<const f32x4_a4_t *>(q);
        return make_float4(v.x, v.y, v.z, v.w);
    }
    return make_float4(left > 0 ? q[0] : 0.f, left > 1 ? q[1] : 0.f, left > 2 ? q[2] : 0.f, 0.f);
}

// The same for a granule that lies wholly inside the operand: no branch.
template <bool KMAJ>
__device__ __forceinline__ float4 load4_whole(const float *__restrict__ p, int64_t ld, int64_t mn0,
                                              int64_t k0, int tid)
{
    const float *q = KMAJ ? p + (mn0 + (tid >> 2)) * ld + k0 + (tid & 3) * 4
                          : p + (k0 + (tid >> 4)) * ld + mn0 + (tid & 15) * 4;
    const f32x4_a4_t v = *reinterpret_cast<const f32x4_a4_t *>(q);
    return make_float4(v.x, v.y, v.z, v.w);
}

// Where K value k (of a step) of a K-major row lies: evens, then odds of every 8.
__device__ __forceinline__ int place_k(int k) { return (k & ~7) + ((k & 1) << 2) + ((k & 7) >> 1); }

template <bool KMAJ>
__device__ __forceinline__ void store4(float *__restrict__ S, float4 v, int j, int tid)
{
    if constexpr (KMAJ) {
        const int k = j * BK + (tid & 3) * 4;
        float *q = S + (tid >> 2) * KPITCH + place_k(k);
        *reinterpret_cast<float2 *>(q) = make_float2(v.x, v.z);
        *reinterpret_cast<float2 *>(q + 4) = make_float2(v.y, v.w);
    } else {
        *reinterpret_cast<float4 *>(S + (j * BK + (tid >> 4)) * MPITCH + (tid & 15) * 4) = v;
    }
}

// The operand of lane `lane` for the four MFMAs of K values 8 e .. 8 e + 7 of a
// step, rows (or columns) mn .. mn + 31.
template <bool KMAJ>
__device__ __forceinline__ float4 frag4(const float *__restrict__ S, int mn, int e, int lane)
{
    if constexpr (KMAJ) {
        return *reinterpret_cast<const float4 *>(S + (mn + (lane & 31)) * KPITCH + 8 * e +
                                                 4 * (lane >> 5));
    } else {
        const float *q = S + (8 * e + (lane >> 5)) * MPITCH + mn + (lane & 31);
        return make_float4(q[0], q[2 * MPITCH], q[4 * MPITCH], q[6 * MPITCH]);
    }
}

template <bool AK, bool BKM, bool ROWSQ>
__global__ void __launch_bounds__(NT) gemm_f32_kernel(GemmArgs g)
{
    constexpr int AF = AK ? BM * KPITCH : STEP * BK * MPITCH;
    constexpr int BF = BKM ? BN * KPITCH : STEP * BK * MPITCH;
    constexpr int CF = BM * (BN + 4);
    __shared__ __align__(16) float lds[2 * (AF + BF) > CF ? 2 * (AF + BF) : CF];

    const int tid = static_cast<int>(threadIdx.x);
    const int lane = tid & 63, wave = tid >> 6;
    const int wm = (wave >> 1) * 32, wn = (wave & 1) * 32;
    int tm, tn;
    tile_coords(g.M, g.N, BM, BN, tm, tn);
    const int64_t m0 = static_cast<int64_t>(tm) * BM, n0 = static_cast<int64_t>(tn) * BN;
    const int z = static_cast<int>(blockIdx.y);

    const int64_t st1 = (g.seg[0].K + BK - 1) / BK;
    const int64_t st_total = st1 + (g.nseg > 1 ? (g.seg[1].K + BK - 1) / BK : 0);
    int64_t s_begin = static_cast<int64_t>(z) * g.steps_per_split;
    if (s_begin > st_total)
        s_begin = st_total;
    int64_t s_end = s_begin + g.steps_per_split;
    if (s_end > st_total)
        s_end = st_total;

    f32x16_t acc;
#pragma unroll
    for (int i = 0; i < 16; ++i)
        acc[i] = 0.f;
    float sq = 0.f;

    struct Regs {
        float4 a[STEP], b[STEP];
    } regs[AHEAD];
    const bool inside = m0 + BM <= g.M && n0 + BN <= g.N;
    // the loads of step s (granules past the split's end: its last one again, so
    // that every step has the same number of loads in flight; none in a lone step)
    auto fetch = [&](Regs &r, int64_t s) {
#pragma unroll
        for (int j = 0; j < STEP; ++j) {
            if (j > 0 && s_end - s_begin == 1)
                break;
            const int64_t gr = s + j < s_end ? s + j : s_end - 1;
            const bool first = gr < st1;
            const GemmSeg &sg = first ? g.seg[0] : g.seg[1];
            const int64_t k0 = (first ? gr : gr - st1) * BK;
            const float *pa = static_cast<const float *>(sg.a);
            const float *pb = static_cast<const float *>(sg.b);
            if (inside && k0 + BK <= sg.K) {
                r.a[j] = load4_whole<AK>(pa, sg.lda, m0, k0, tid);
                r.b[j] = load4_whole<BKM>(pb, sg.ldb, n0, k0, tid);
            } else {
                r.a[j] = load4<AK>(pa, sg.lda, g.M, sg.K, m0, k0, tid);
                r.b[j] = load4<BKM>(pb, sg.ldb, g.N, sg.K, n0, k0, tid);
            }
        }
    };
    int at = 0;
    // One barrier a step (a wave past it is done with the other buffer), bare:
    // __syncthreads would wait for the loads in flight as well.
    auto step = [&](Regs &r, int64_t s, auto more) {
        float *const As = lds + at * (AF + BF), *const Bs = As + AF;
#pragma unroll
        for (int j = 0; j < STEP; ++j) {
            store4<AK>(As, r.a[j], j, tid);
            store4<BKM>(Bs, r.b[j], j, tid);
        }
        dma::wait_lgkm0();
        dma::stage_barrier();
        if constexpr (decltype(more)::value)
            fetch(r, s + AHEAD * STEP);
#pragma unroll
        for (int j = 0; j < STEP; ++j) {
            if (s + j >= s_end)
                break;
#pragma unroll
            for (int e = 2 * j; e < 2 * j + 2; ++e) {
                const float4 a = frag4<AK>(As, wm, e, lane), b = frag4<BKM>(Bs, wn, e, lane);
                acc = __builtin_amdgcn_mfma_f32_32x32x2f32(a.x, b.x, acc, 0, 0, 0);
                acc = __builtin_amdgcn_mfma_f32_32x32x2f32(a.y, b.y, acc, 0, 0, 0);
                acc = __builtin_amdgcn_mfma_f32_32x32x2f32(a.z, b.z, acc, 0, 0, 0);
                acc = __builtin_amdgcn_mfma_f32_32x32x2f32(a.w, b.w, acc, 0, 0, 0);
            }
            if constexpr (ROWSQ) {
                if (tid < BM) {
#pragma unroll
                    for (int kk = 0; kk < BK; ++kk) {
                        const float v = As[tid * KPITCH + place_k(j * BK + kk)];
                        sq += v * v;
                    }
                }
            }
        }
        at ^= 1;
    };
    if (s_begin + AHEAD * STEP < s_end) {
#pragma unroll
        for (int p = 0; p < AHEAD; ++p)
            fetch(regs[p], s_begin + p * STEP);
        for (int64_t s = s_begin; s < s_end; s += AHEAD * STEP) {
#pragma unroll
            for (int p = 0; p < AHEAD; ++p)
                if (s + p * STEP < s_end)
                    step(regs[p], s + p * STEP, std::true_type{});
        }
    } else {
        // few steps: no loads but theirs (the epilogue's barrier would wait for more:
        // a norm of 16 x 16, r 2, 21 us with them, 15 without)
#pragma unroll
        for (int p = 0; p < AHEAD; ++p)
            if (s_begin + p * STEP < s_end)
                fetch(regs[p], s_begin + p * STEP);
#pragma unroll
        for (int p = 0; p < AHEAD; ++p)
            if (s_begin + p * STEP < s_end)
                step(regs[p], s_begin + p * STEP, std::false_type{});
    }

    if constexpr (ROWSQ) {
        if (g.rowsq != nullptr && tn == 0 && tid < BM && m0 + tid < g.M)
            g.rowsq[static_cast<int64_t>(z) * g.M + m0 + tid] = sq;
    }

    __syncthreads();  // the tile takes the operands' place
    float *const Cs = lds;
#pragma unroll
    for (int i = 0; i < 16; ++i)
        Cs[(wm + (i & 3) + 8 * (i >> 2) + 4 * (lane >> 5)) * (BN + 4) + wn + (lane & 31)] = acc[i];
    __syncthreads();
    epilogue_rows<BM, BN, BN + 4, NT, float>(Cs, g, m0, n0, z, tn, tid);
}

template <bool AK, bool BKM, bool RS>
hipError_t launch_one(const GemmArgs &a, hipStream_t st)
{
    const int64_t tiles = ((a.M + BM - 1) / BM) * ((a.N + BN - 1) / BN);
    if (tiles == 0 || a.splits == 0)
        return hipSuccess;
    dim3 grid(static_cast<unsigned>(tiles), static_cast<unsigned>(a.splits));
    hipLaunchKernelGGL((gemm_f32_kernel<AK, BKM, RS>), grid, dim3(NT), 0, st, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_gemm_f32(const GemmArgs &a, int layout, bool rowsq, hipStream_t st)
{
    switch (layout) {
    case 0:
        return rowsq ? launch_one<true, true, true>(a, st) : launch_one<true, true, false>(a, st);
    case 1:
        return launch_one<true, false, false>(a, st);
    case 2:
        return launch_one<false, false, false>(a, st);
    default:
        return hipErrorInvalidValue;
    }
}

}  // namespace dora
