// gemm_bf16_any.hip - the bf16 product for operands of any width (gfx950):
// rows start at any element.  Same contract, K steps, order of sums and
// epilogues as gemm_bf16.hip's kernel, with 128 x 128 or 64 x 64 tiles.
//
// Operands are staged through registers by 16-byte loads at whatever element.
// A load that runs past its row's end takes in the next row's values, and at the
// matrix's end it starts early; the last K steps' are put right on the way into
// LDS, so that there is no branch and no wait among the loads.
//   K-major: a thread holds chunk tid & 7 of rows (tid >> 3) + 32 i (rows past
//     the end: the last one, never stored);
//   MN-major: KR = B / 32 consecutive K rows of eight columns, written to LDS as
//     2 KR bytes of each of the eight rows there.  The chunk in which rows of at
//     least eight columns end is taken from their last eight instead: those
//     columns are written twice, with the same values.  Columns past the end
//     are never stored.
// LDS rows hold 64 K values as eight 16-byte chunks, chunk c of row r at
// c ^ (r & 7) ^ (r / 8 & 7): fragment reads, and the writes of one chunk column
// by threads eight rows apart, meet distinct banks.
//
// Most of these products are small, and a step's time is its loads' round trip:
// 64 x 64 tiles, with AHEAD = 2 steps' loads in flight, serve where there are few
// 128 x 128 ones (whose accumulators leave registers for one step's).  The nine
// products of a backward through the norm from a bf16 x, 509 tokens, 1027 -> 1411, r 37,
// call included: 148 us, with one step ahead 170, three 155, 128 x 128 tiles alone 245.
#include "dora_internal.hpp"
#include "epilogue.hpp"
#include "gemm_bf16_dma.hpp"
#include "ragged.hpp"

#include <type_traits>

namespace dora {
namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

constexpr int BK = GEMM_BK, NT = 256;
static_assert(BK == 64, "eight chunks a row");

// Eight values p[0 .. 8), those at or past `live` zero, one by one (products with
// a matrix of fewer than eight values).
__device__ __forceinline__ uint4 load8_masked(const uint16_t *p, int64_t live)
{
    uint32_t w[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const uint32_t lo = 2 * q < live ? p[2 * q] : 0u;
        const uint32_t hi = 2 * q + 1 < live ? p[2 * q + 1] : 0u;
        w[q] = lo | (hi << 16);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ uint32_t word(const uint4 &v, int w)
{
    return w == 0 ? v.x : (w == 1 ? v.y : (w == 2 ? v.z : v.w));
}

__device__ __forceinline__ int place(int row, int c) { return row * 8 + (c ^ ((row ^ (row >> 3)) & 7)); }

// One operand's share of a step: B rows (of M or N) x 64 K values, rows from mn0.
template <bool KMAJ, int B, bool TINY>
struct Operand {
    static constexpr int PER = B / 32;  // chunks a thread
    static constexpr int CB = B / 8;    // column chunks of an MN-major tile

    // MN-major: the first column, from the tile's, of the eight that chunk mb holds
    static __device__ __forceinline__ int first(int64_t MN, int64_t mn0, int mb)
    {
        const int64_t c = mn0 + mb * 8;
        return static_cast<int>((MN >= 8 && c + 8 > MN ? MN - 8 : c) - mn0);
    }

    // the matrix's last eight values
    static __device__ __forceinline__ int64_t last(int64_t ld, int64_t MN, int64_t K)
    {
        return KMAJ ? (MN - 1) * ld + K - 8 : (K - 1) * ld + MN - 8;
    }

    // where chunk i of a step starts, from the step's first K value on: its row
    // (K-major), its K value and its first column (MN-major)
    static __device__ __forceinline__ int64_t start(int64_t ld, int64_t MN, int64_t mn0, int tid,
                                                    int i)
    {
        if constexpr (KMAJ) {
            const int64_t mn = mn0 + (tid >> 3) + 32 * i;
            return (mn < MN ? mn : MN - 1) * ld + (tid & 7) * 8;
        } else {
            const int mb = tid % CB;
            return (tid / CB * PER + i) * ld + (mn0 + mb * 8 < MN ? mn0 + first(MN, mn0, mb) : 0);
        }
    }
    int64_t from[PER];  // those of the segment that is being loaded
    __device__ __forceinline__ void init(int64_t ld, int64_t MN, int64_t mn0, int tid)
    {
#pragma unroll
        for (int i = 0; i < PER; ++i)
            from[i] = start(ld, MN, mn0, tid, i);
    }

    __device__ __forceinline__ void load(uint4 (&v)[PER], const uint16_t *p, int64_t ld, int64_t MN,
                                         int64_t K, int64_t mn0, int64_t k0, int tid) const
    {
        const int64_t end = last(ld, MN, K), step = KMAJ ? k0 : k0 * ld;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int64_t at = from[i] + step;
            if constexpr (TINY) {
                const int64_t k = k0 + (KMAJ ? (tid & 7) * 8 : tid / CB * PER + i);
                const int64_t c = mn0 + tid % CB * 8;
                v[i] = k < K ? load8_masked(p + at, KMAJ ? K - k : (c < MN ? MN - mn0 - first(MN, mn0, tid % CB) : 0))
                             : make_uint4(0, 0, 0, 0);
            } else {
                v[i] = load16_any(p + (at < end ? at : end));
            }
        }
    }

    // What of the loads near the K range's end belongs there (`tail`).
    static constexpr int TAIL = KMAJ ? 0 : 8;  // MN-major rows of fewer than eight columns
    static __device__ __forceinline__ void tail(uint4 (&v)[PER], int64_t ld, int64_t MN, int64_t K,
                                                int64_t mn0, int64_t k0, int tid)
    {
        const int64_t end = last(ld, MN, K);
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int64_t k = k0 + (KMAJ ? (tid & 7) * 8 : tid / CB * PER + i), left = K - k;
            const int64_t back = start(ld, MN, mn0, tid, i) + (KMAJ ? k0 : k0 * ld) - end;
            v[i] = row_end16(v[i], !TINY && back > 0 && left > 0 ? static_cast<int>(2 * back) : 0,
                             KMAJ ? 2 * left : (left > 0 ? 16 : 0));
        }
    }

    static __device__ __forceinline__ void store(uint4 *S, const uint4 (&v)[PER], int64_t MN,
                                                 int64_t mn0, int tid)
    {
        if constexpr (KMAJ) {
#pragma unroll
            for (int i = 0; i < PER; ++i)
                S[place((tid >> 3) + 32 * i, tid & 7)] = v[i];
        } else {
            const int mb = tid % CB, kg = tid / CB;
            if (mn0 + mb * 8 >= MN)
                return;
            const int row0 = first(MN, mn0, mb);
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                uint32_t o[PER / 2];
#pragma unroll
                for (int h = 0; h < PER / 2; ++h) {
                    const uint32_t a = word(v[2 * h], q >> 1), b = word(v[2 * h + 1], q >> 1);
                    o[h] = q & 1 ? (a >> 16) | (b & 0xffff0000u) : (a & 0xffffu) | (b << 16);
                }
                const int row = row0 + q;
                if (row < 0)  // a column of the tile before
                    continue;
                uint32_t *s = reinterpret_cast<uint32_t *>(S + place(row, kg * PER / 8)) +
                              kg % (8 / PER) * (PER / 2);
                if constexpr (PER == 4)
                    *reinterpret_cast<uint2 *>(s) = make_uint2(o[0], o[1]);
                else
                    *s = o[0];
            }
        }
    }
};

// TINY: a matrix of fewer than eight values
template <int B, int AHEAD, bool TINY, bool AK, bool BKM, bool ROWSQ>
__global__ void __launch_bounds__(NT, 2) gemm_bf16_any_kernel(GemmArgs g)
{
    constexpr int WT = B / 2, TT = WT / 16, PER = B / 32;
    constexpr int CST = B + 4;  // floats of an epilogue row
    constexpr int OPS = 2 * 2 * B * BK * 2, EPI = WT * CST * 4;
    using OA = Operand<AK, B, TINY>;
    using OB = Operand<BKM, B, TINY>;
    static_assert(!ROWSQ || AK, "row sums of squares need a K-major A");
    __shared__ __align__(16) unsigned char smem[OPS > EPI ? OPS : EPI];
    uint4 *const lds = reinterpret_cast<uint4 *>(smem);  // [2][A, B][B * 8]

    const int tid = static_cast<int>(threadIdx.x), lane = tid & 63, wave = tid >> 6;
    const int wm = (wave >> 1) * WT, wn = (wave & 1) * WT;
    int tm, tn;
    tile_coords(g.M, g.N, B, B, tm, tn);
    const int64_t m0 = static_cast<int64_t>(tm) * B, n0 = static_cast<int64_t>(tn) * B;
    const int z = static_cast<int>(blockIdx.y);

    const int64_t st1 = (g.seg[0].K + BK - 1) / BK;
    const int64_t st_total = st1 + (g.nseg > 1 ? (g.seg[1].K + BK - 1) / BK : 0);
    int64_t s_begin = static_cast<int64_t>(z) * g.steps_per_split;
    s_begin = s_begin < st_total ? s_begin : st_total;
    int64_t s_end = s_begin + g.steps_per_split;
    s_end = s_end < st_total ? s_end : st_total;

    f32x4_t acc[TT][TT];
#pragma unroll
    for (int i = 0; i < TT; ++i)
#pragma unroll
        for (int j = 0; j < TT; ++j)
            acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    float sq[ROWSQ ? PER : 1];
#pragma unroll
    for (int i = 0; i < (ROWSQ ? PER : 1); ++i)
        sq[i] = 0.f;

    struct Regs {
        uint4 a[PER], b[PER];
    } regs[AHEAD];
    // the loads of step s (past the split's end its last one again: the loads in
    // flight are always the same number)
    OA oa;
    OB ob;
    int64_t seg_end = -1;  // the loads' segment ends here
    auto load = [&](Regs &r, int64_t s) {
        s = s < s_end ? s : s_end - 1;
        const bool one = s < st1;
        const GemmSeg &sg = one ? g.seg[0] : g.seg[1];
        if (s >= seg_end) {
            seg_end = one ? st1 : st_total;
            oa.init(sg.lda, g.M, m0, tid);
            ob.init(sg.ldb, g.N, n0, tid);
        }
        const int64_t k0 = (one ? s : s - st1) * BK;
        oa.load(r.a, static_cast<const uint16_t *>(sg.a), sg.lda, g.M, sg.K, m0, k0, tid);
        ob.load(r.b, static_cast<const uint16_t *>(sg.b), sg.ldb, g.N, sg.K, n0, k0, tid);
    };
    int at = 0;
    // One barrier a step (a wave past it is done with the other buffer), bare:
    // __syncthreads would wait for the loads in flight as well.
    auto step = [&](Regs &r, int64_t s, auto more) {
        const bool one = s < st1;
        const GemmSeg &sg = one ? g.seg[0] : g.seg[1];
        const int64_t k0 = (one ? s : s - st1) * BK;
        if (k0 + BK + OA::TAIL > sg.K)
            OA::tail(r.a, sg.lda, g.M, sg.K, m0, k0, tid);
        if (k0 + BK + OB::TAIL > sg.K)
            OB::tail(r.b, sg.ldb, g.N, sg.K, n0, k0, tid);
        if constexpr (ROWSQ) {
#pragma unroll
            for (int i = 0; i < PER; ++i)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const float lo = __uint_as_float(word(r.a[i], q) << 16);
                    const float hi = __uint_as_float(word(r.a[i], q) & 0xffff0000u);
                    sq[i] += lo * lo;
                    sq[i] += hi * hi;
                }
        }
        uint4 *const As = lds + at * 2 * B * 8, *const Bs = As + B * 8;
        OA::store(As, r.a, g.M, m0, tid);
        OB::store(Bs, r.b, g.N, n0, tid);
        dma::wait_lgkm0();
        dma::stage_barrier();
        if constexpr (decltype(more)::value)
            load(r, s + AHEAD);
#pragma unroll
        for (int h = 0; h < BK / 32; ++h) {
            const int c = h * 4 + (lane >> 4);
            bf16x8_t fa[TT], fb[TT];
#pragma unroll
            for (int i = 0; i < TT; ++i)
                fa[i] = __builtin_bit_cast(bf16x8_t, As[place(wm + i * 16 + (lane & 15), c)]);
#pragma unroll
            for (int j = 0; j < TT; ++j)
                fb[j] = __builtin_bit_cast(bf16x8_t, Bs[place(wn + j * 16 + (lane & 15), c)]);
#pragma unroll
            for (int i = 0; i < TT; ++i)
#pragma unroll
                for (int j = 0; j < TT; ++j)
                    acc[i][j] =
                        __builtin_amdgcn_mfma_f32_16x16x32_bf16(fa[i], fb[j], acc[i][j], 0, 0, 0);
        }
        at ^= 1;
    };
    if (s_begin + 1 == s_end) {
        // (no load but this step's: the epilogue's barrier would wait for more)
        load(regs[0], s_begin);
        step(regs[0], s_begin, std::false_type{});
    } else if (s_begin < s_end) {
#pragma unroll
        for (int p = 0; p < AHEAD; ++p)
            load(regs[p], s_begin + p);
        int64_t s = s_begin;
        for (; s + AHEAD <= s_end; s += AHEAD) {
#pragma unroll
            for (int p = 0; p < AHEAD; ++p)
                step(regs[p], s + p, std::true_type{});
        }
#pragma unroll
        for (int p = 0; p < AHEAD - 1; ++p)
            if (s + p < s_end)
                step(regs[p], s + p, std::true_type{});
    }

    if constexpr (ROWSQ) {
        if (g.rowsq != nullptr && tn == 0) {
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                float v = sq[i];
                v += __shfl_xor(v, 1);
                v += __shfl_xor(v, 2);
                v += __shfl_xor(v, 4);
                const int64_t m = m0 + (tid >> 3) + 32 * i;
                if ((tid & 7) == 0 && m < g.M)
                    g.rowsq[static_cast<int64_t>(z) * g.M + m] = v;
            }
        }
    }

    // Epilogue: half the tile's rows at a time through LDS.
    __syncthreads();
    float *const Cs = reinterpret_cast<float *>(smem);
#pragma unroll 1
    for (int h = 0; h < 2; ++h) {
        if (wm == h * WT) {
#pragma unroll
            for (int i = 0; i < TT; ++i)
#pragma unroll
                for (int j = 0; j < TT; ++j)
#pragma unroll
                    for (int v = 0; v < 4; ++v)
                        Cs[(i * 16 + (lane >> 4) * 4 + v) * CST + wn + j * 16 + (lane & 15)] =
                            acc[i][j][v];
        }
        __syncthreads();
        epilogue_rows<WT, B, CST, NT, uint16_t>(Cs, g, m0 + h * WT, n0, z, tn, tid);
        __syncthreads();
    }
}

template <int B, int AHEAD, bool TINY = false>
hipError_t launch_any(const GemmArgs &a, int layout, bool rowsq, hipStream_t st)
{
    const int64_t tiles = ((a.M + B - 1) / B) * ((a.N + B - 1) / B);
    if (tiles == 0 || a.splits == 0)
        return hipSuccess;
    const dim3 grid(static_cast<unsigned>(tiles), static_cast<unsigned>(a.splits)), block(NT);
    if (layout == 0 && rowsq)
        hipLaunchKernelGGL((gemm_bf16_any_kernel<B, AHEAD, TINY, true, true, true>), grid, block, 0, st, a);
    else if (layout == 0)
        hipLaunchKernelGGL((gemm_bf16_any_kernel<B, AHEAD, TINY, true, true, false>), grid, block, 0, st, a);
    else if (layout == 1)
        hipLaunchKernelGGL((gemm_bf16_any_kernel<B, AHEAD, TINY, true, false, false>), grid, block, 0, st, a);
    else if (layout == 2)
        hipLaunchKernelGGL((gemm_bf16_any_kernel<B, AHEAD, TINY, false, false, false>), grid, block, 0, st, a);
    else
        return hipErrorInvalidValue;
    return hipGetLastError();
}

// Whether a matrix holds fewer than the eight values of one load.
bool tiny(const GemmArgs &a, int layout)
{
    for (int q = 0; q < a.nseg; ++q) {
        const GemmSeg &sg = a.seg[q];
        if (sg.K > 0 && ((layout < 2 ? (a.M - 1) * sg.lda + sg.K : (sg.K - 1) * sg.lda + a.M) < 8 ||
                         (layout == 0 ? (a.N - 1) * sg.ldb + sg.K : (sg.K - 1) * sg.ldb + a.N) < 8))
            return true;
    }
    return false;
}

}  // namespace

// The planner counts 128 x 128 tiles, whose columns also number the row-dot
// partial sums; stored products take 64 x 64 ones, with the same bits, where
// those are fewer than the CUs (x W^T, 1027 -> 1411 at 509 tokens, 48 tiles of
// 128 x 128: 18 us, by those 26; 4097 -> 4096 at 2048, 512 of them: 178 us, by
// those 103).
hipError_t launch_gemm_bf16_any(const GemmArgs &a, int layout, bool rowsq, hipStream_t st)
{
    const int64_t tiles = ((a.M + 127) / 128) * ((a.N + 127) / 128) * a.splits;
    if (tiny(a, layout))
        return a.mode == EPI_ROWDOT ? launch_any<128, 1, true>(a, layout, rowsq, st)
                                    : launch_any<64, 1, true>(a, layout, rowsq, st);
    if (a.mode != EPI_ROWDOT && tiles < 256)
        return launch_any<64, 2>(a, layout, rowsq, st);
    return launch_any<128, 1>(a, layout, rowsq, st);
}

}  // namespace dora
