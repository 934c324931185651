// gemm_i8_dma.hip - the pipelined int8 product (gfx950): y = xq wq^T scaled by
// token and output channel, for widths d_in of whole 16-byte chunks.
//
// v_mfma_i32_16x16x64_i8 takes 16 bytes of a row per lane like the bf16
// 16 x 16 x 32 form, so an int8 matrix of width K is loaded and laid out in
// LDS as a bf16 matrix of width K / 2: the stages (128 bytes of K), the
// direct-to-LDS load plan, the chunk swizzle and the two half stages are those
// of the bf16 kernels, at twice the products per byte and per instruction.
//
// A workgroup walks its share of the work items (an output tile, or one K
// range of it) as one unbroken stream of stages: while the products of stage
// S run, stage S + SLOTS loads, whichever item it belongs to, so that the pipeline
// does not drain between items.  Item order: XCD x owns a contiguous run of
// items, its workgroups take them in turn.
//
// The sums are exact in int32, so a product may be split over K into any
// number of ranges without changing its bits.  Epilogue, per wave: sums times
// token scale times channel scale in fp32, rounded once, through the wave's
// own LDS rows into 16-byte stores of whole 128-byte lines.
#include "gemm_dma_launch.hpp"
#include "rows8.hpp"

namespace dora {
namespace dma {

typedef int i32x4_t __attribute__((ext_vector_type(4)));

template <int TM, int TN>
struct FragsI8 {
    i32x4_t a[TM], b[TN];
};

// Output kinds: the element types of y, or int32 partial sums.
constexpr int OUT_BF16 = 0, OUT_F32 = 1, OUT_PART = 2;

constexpr int I8_STAGE_ROWS = 32;  // rows of a wave's staging area, 128 bytes each at most

// Fragment read number O of half `h`: A fragments, then B.
template <int TM, int TN, int WTM, int WTN, int O>
__device__ __forceinline__ void read_one_i8(FragsI8<TM, TN> &f, const unsigned char *As,
                                            const unsigned char *Bs, int h, int wm, int wn,
                                            int lane)
{
    if constexpr (O < TM)
        f.a[O] = __builtin_bit_cast(i32x4_t, read_frag16(As, wm * WTM + O * 16, h, lane));
    else
        f.b[O - TM] =
            __builtin_bit_cast(i32x4_t, read_frag16(Bs, wn * WTN + (O - TM) * 16, h, lane));
}

// SLOTS: stages held in LDS (a power of two); PERCU: workgroups resident on a CU
// (the register budget).
template <int BM, int BN, int WM, int WN, int SLOTS, int PERCU, int OUT>
__global__ void __launch_bounds__(WM *WN * 64, WM *WN *PERCU / 4)
    gemm_i8_dma_kernel(I8GemmArgs g)
{
    using C = DmaCfg<BM, BN, WM, WN>;
    constexpr int G = group_size<(BM * ROW_BYTES / 1024) / (WM * WN),
                                 (BN * ROW_BYTES / 1024) / (WM * WN)>();
    using DA = OperandDma<true, BM, WM * WN, G>;
    using DB = OperandDma<true, BN, WM * WN, G>;
    constexpr int NW = WM * WN;
    constexpr int WTM = BM / WM, WTN = BN / WN;
    constexpr int TM = WTM / 16, TN = WTN / 16;
    constexpr int ELT = OUT == OUT_BF16 ? 2 : 4;
    constexpr int SLAB = WTN < 128 / ELT ? WTN : 128 / ELT;  // columns of a staging pass
    constexpr int SROW = SLAB * ELT;                         // bytes of a staging row
    constexpr int SCH = SROW / 16;                           // its 16-byte chunks
    constexpr int STAGE = I8_STAGE_ROWS * SROW;
    static_assert(WTM % I8_STAGE_ROWS == 0 && WTN % SLAB == 0, "whole staging passes");
    static_assert(DA::PER + DB::PER == C::LPS, "load count");
    // scales of the wave's rows and columns: in LDS where the accumulators leave
    // no registers for them
    constexpr bool LDS_SCALES = TM * TN > 32 && OUT != OUT_PART;
    constexpr int WAVE_BYTES = STAGE + (LDS_SCALES ? (WTM + WTN) * 4 : 0);
    constexpr int OPS = SLOTS * C::STAGE_BYTES;
    constexpr int SMEM = OPS + NW * WAVE_BYTES;
    static_assert(SMEM * PERCU <= 160 * 1024, "LDS");
    __shared__ __align__(1024) unsigned char smem[SMEM];

    const int tid = static_cast<int>(threadIdx.x);
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WN, wn = wave % WN;

    // this workgroup's items: first + k * per, k < count
    const int num_m = static_cast<int>((g.M + BM - 1) / BM);
    const int num_n = static_cast<int>((g.N + BN - 1) / BN);
    const int ntiles = num_m * num_n;
    const int nitems = ntiles * g.splits;
    int first, count, per;
    {
        const int nb = static_cast<int>(gridDim.x), b = static_cast<int>(blockIdx.x);
        const int xcd = b & 7, local = b >> 3;
        per = nb >> 3;
        const int q = nitems >> 3, rem = nitems & 7;
        const int start = xcd < rem ? xcd * (q + 1) : rem * (q + 1) + (xcd - rem) * q;
        const int len = q + (xcd < rem ? 1 : 0);
        first = start + local;
        count = local < len ? (len - local + per - 1) / per : 0;
    }
    if (count == 0)
        return;
    // item k: its K range z, tile (tm, tn) and number of stages
    const int nst = static_cast<int>((g.K + 2 * BK - 1) / (2 * BK));
    const int sps = static_cast<int>(g.k_per_split / (2 * BK));
    struct Item {
        int z, tm, tn, stages;
    };
    auto item = [&](int k) {
        const int L = first + k * per;
        Item it;
        it.z = L / ntiles;
        tile_in_order(L - it.z * ntiles, g.M, g.N, BM, BN, it.tm, it.tn);
        const int left = nst - it.z * sps;
        it.stages = left < sps ? left : sps;
        return it;
    };

    const int64_t ld = g.K / 2;  // the rows as 2-byte elements
    const int na = range_bytes(g.M * g.K), nb = range_bytes(g.N * g.K);
    DA da;
    DB db;
    // the load cursor: item lk, its stage ls of ln, from K stage lbase on
    int lk = 0, ls = 0, ln = 0, lbase = 0;
    auto plan = [&]() {
        const Item it = item(lk);
        int lane_here;
        // (an opaque copy: the plan is formed here each time, not from terms
        // kept live across the stage loop)
        __asm__ volatile("v_mov_b32 %0, %1" : "=v"(lane_here) : "v"(lane));
        da.init(g.M, ld, static_cast<int64_t>(it.tm) * BM, wave, lane_here);
        db.init(g.N, ld, static_cast<int64_t>(it.tn) * BN, wave, lane_here);
        ln = it.stages;
        lbase = it.z * sps;
        ls = 0;
    };
    // to the next stage to be loaded (past the last item: loads of nothing)
    auto advance = [&]() {
        if (++ls >= ln && lk < count) {
            ++lk;
            if (lk < count)
                plan();
        }
    };
    plan();

    auto slot = [&](int S) { return smem + (S & (SLOTS - 1)) * C::STAGE_BYTES; };
    unsigned char *const stg = smem + OPS + wave * WAVE_BYTES;

    constexpr int GA = DA::PER / G, NG = C::LPS / G;
    struct Group {
        __amdgpu_buffer_rsrc_t rs;
        uint32_t soff;
        uint32_t v[G];
    };
    // load group d of the cursor's stage into the slot of running stage S
    auto dma_prep = [&](int S, int d) {
        const bool live = lk < count;
        const int kd = (lbase + ls) * BK;
        const bool isa = d < GA;
        const int i0 = (isa ? d : d - GA) * G;
        const uint32_t lds = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(
            reinterpret_cast<uintptr_t>((lds_void *)(slot(S) + (isa ? 0 : C::A_BYTES) +
                                                     (wave * (isa ? DA::PER : DB::PER) + i0) *
                                                         1024))));
        Group grp;
        grp.rs = scalar_rsrc(isa ? g.x : g.w, live ? (isa ? na : nb) : 0);
#pragma unroll
        for (int j = 0; j < G; ++j) {
            const uint32_t off = isa ? da.off[i0 + j] : db.off[i0 + j];
            const uint32_t kc =
                isa ? DA::kchunk(wave, i0 + j, lane) : DB::kchunk(wave, i0 + j, lane);
            grp.v[j] = kd + static_cast<int>(kc) < static_cast<int>(ld) ? off : OOB_OFFSET;
        }
        grp.soff = static_cast<uint32_t>(kd * 2);
        set_m0(lds);
        return grp;
    };
    auto issue = [&](const Group &grp, auto j_c) {
        constexpr int J = decltype(j_c)::value;
        lds_dma16<J>(grp.rs, grp.v[J], grp.soff);
    };

    constexpr int NMF = TM * TN, NRD = TM + TN;
    using FR = FragsI8<TM, TN>;
    using ACC = i32x4_t[TM][TN];

    // One half stage: the products of `cur`, the fragment reads of the next
    // half into `nxt` (READS), and in half 1 the loads of the cursor's stage
    // into this stage's slot, for running stage S + SLOTS.
    auto half = [&](ACC &acc, auto h_c, int S, FR &cur, FR &nxt, auto reads_c) {
        constexpr int H = decltype(h_c)::value;
        constexpr bool READS = decltype(reads_c)::value;
        constexpr int NLH = H == 1 ? NG * G : 0;
        constexpr int NOPS = (READS ? NRD : 0) + NLH;
        wait_lgkm0();
        if constexpr (H == 1) {
            // stage S + 1 has landed (the loads of SLOTS - 2 stages may still be
            // under way), and every wave is done with this slot's fragments
            wait_vmcnt<(SLOTS - 2) * C::LPS>();
            stage_barrier();
        }
        const unsigned char *An = slot(H == 0 ? S : S + 1);
        const unsigned char *Bn = An + C::A_BYTES;
        Group grp;
        static_for<NMF>([&](auto qc) {
            constexpr int q = decltype(qc)::value;
            constexpr int i = q / TN, j = q % TN;
            acc[i][j] =
                __builtin_amdgcn_mfma_i32_16x16x64_i8(cur.b[j], cur.a[i], acc[i][j], 0, 0, 0);
            constexpr int cnt = (q + 1) * NOPS / NMF - q * NOPS / NMF;
            static_for<cnt>([&](auto oc) {
                constexpr int o = q * NOPS / NMF + decltype(oc)::value;
                constexpr int li = NLH > 0 && (o * NLH) % NOPS < NLH ? (o * NLH) / NOPS : -1;
                constexpr int rd = o - (o * NLH + NOPS - 1) / NOPS;
                if constexpr (li >= 0) {
                    if constexpr (li % G == 0)
                        grp = dma_prep(S + SLOTS, li / G);
                    issue(grp, std::integral_constant<int, li % G>{});
                } else if constexpr (READS) {
                    read_one_i8<TM, TN, WTM, WTN, rd>(nxt, An, Bn, 1 - H, wm, wn, lane);
                }
            });
            __builtin_amdgcn_sched_barrier(0);
        });
    };

    const __amdgpu_buffer_rsrc_t out_rs = __builtin_amdgcn_make_buffer_rsrc(
        OUT == OUT_PART ? static_cast<void *>(g.part) : g.y, static_cast<short>(0),
        __builtin_amdgcn_readfirstlane(static_cast<int>(
            g.M * g.N * ELT * (OUT == OUT_PART ? static_cast<int64_t>(g.splits) : 1))),
        0x00020000);

    // Accumulator block (i, j): lane l holds row 16 i + (l & 15), columns
    // 16 j + 4 (l >> 4) + 0..3 of the wave's tile.  16-byte chunk c of staging
    // row r sits at c ^ swz(r) (of as many bits as a row has chunks).
    auto chunk = [](int r, int c) { return (c ^ (swz(r) & (SCH - 1))) << 4; };
    auto epilogue = [&](ACC &acc, const Item &it) {
        const int64_t m0 = static_cast<int64_t>(it.tm) * BM + wm * WTM;
        const int64_t n0 = static_cast<int64_t>(it.tn) * BN + wn * WTN;
        const int q4 = lane >> 4;
        // rows of y in whole 16-byte chunks; else element by element
        const bool whole = g.N % (16 / ELT) == 0;
        float4 swr[LDS_SCALES ? 1 : TN];
        float sxr[LDS_SCALES ? 1 : TM];
        float *const lsx = reinterpret_cast<float *>(stg + STAGE), *const lsw = lsx + WTM;
        if constexpr (LDS_SCALES) {
#pragma unroll
            for (int b = 0; b < WTM; b += 64) {
                const int64_t m = m0 + b + lane;
                lsx[b + lane] = g.xs[m < g.M ? m : g.M - 1];
            }
#pragma unroll
            for (int b = 0; b < WTN; b += 64) {
                const int64_t n = n0 + b + lane;
                lsw[b + lane] = g.ws[n < g.N ? n : g.N - 1];
            }
        } else if constexpr (OUT != OUT_PART) {
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                const int64_t n = n0 + 16 * j + 4 * q4, last = g.N - 1;
                if (whole)
                    swr[j] = n < g.N ? *reinterpret_cast<const float4 *>(g.ws + n)
                                     : make_float4(0.f, 0.f, 0.f, 0.f);
                else
                    swr[j] = make_float4(g.ws[n < last ? n : last], g.ws[n + 1 < last ? n + 1 : last],
                                         g.ws[n + 2 < last ? n + 2 : last],
                                         g.ws[n + 3 < last ? n + 3 : last]);
            }
#pragma unroll
            for (int i = 0; i < TM; ++i) {
                const int64_t m = m0 + 16 * i + (lane & 15);
                sxr[i] = g.xs[m < g.M ? m : g.M - 1];
            }
        }
        auto scale_x = [&](int i) {
            if constexpr (LDS_SCALES)
                return i8_xs(lsx[16 * i + (lane & 15)]);
            else
                return i8_xs(sxr[i]);
        };
        auto scale_w = [&](int j) {
            if constexpr (LDS_SCALES)
                return *reinterpret_cast<const float4 *>(lsw + 16 * j + 4 * q4);
            else
                return swr[j];
        };
#pragma unroll
        for (int i2 = 0; i2 < WTM / 32; ++i2) {
#pragma unroll
            for (int hf = 0; hf < WTN / SLAB; ++hf) {
#pragma unroll
                for (int ii = 0; ii < 2; ++ii) {
                    const int i = 2 * i2 + ii;
                    const int rr = 16 * ii + (lane & 15);
                    I8Scale sx;
                    if constexpr (OUT != OUT_PART)
                        sx = scale_x(i);
#pragma unroll
                    for (int jj = 0; jj < SLAB / 16; ++jj) {
                        const int j = hf * (SLAB / 16) + jj;
                        const i32x4_t c = acc[i][j];
                        if constexpr (OUT == OUT_PART) {
                            *reinterpret_cast<i32x4_t *>(
                                stg + rr * SROW + chunk(rr, 4 * jj + q4)) = c;
                        } else {
                            const float4 sw = scale_w(j);
                            const float4 v = make_float4(i8_scaled(c[0], sx, sw.x), i8_scaled(c[1], sx, sw.y),
                                                         i8_scaled(c[2], sx, sw.z), i8_scaled(c[3], sx, sw.w));
                            if constexpr (OUT == OUT_F32)
                                *reinterpret_cast<float4 *>(
                                    stg + rr * SROW + chunk(rr, 4 * jj + q4)) = v;
                            else
                                *reinterpret_cast<uint2 *>(
                                    stg + rr * SROW + chunk(rr, 2 * jj + (q4 >> 1)) +
                                    8 * (q4 & 1)) =
                                    make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
                        }
                    }
                }
#pragma unroll
                for (int ps = 0; ps < STAGE / 1024; ++ps) {
                    const int rr = ps * (64 / SCH) + lane / SCH, c = lane % SCH;
                    const i32x4_t v =
                        *reinterpret_cast<const i32x4_t *>(stg + rr * SROW + chunk(rr, c));
                    const int64_t m = m0 + i2 * 32 + rr;
                    const int64_t n = n0 + hf * SLAB + c * (16 / ELT);
                    const int64_t at =
                        ((OUT == OUT_PART ? static_cast<int64_t>(it.z) * g.M : 0) + m) * g.N + n;
                    if (whole) {
                        const uint32_t off =
                            m < g.M && n < g.N ? static_cast<uint32_t>(at * ELT) : OOB_OFFSET;
                        __builtin_amdgcn_raw_buffer_store_b128(v, out_rs, off, 0, 0);
                    } else if (m < g.M) {
                        using E = std::conditional_t<ELT == 2, uint16_t, int>;
                        E *const out = reinterpret_cast<E *>(OUT == OUT_PART
                                                                 ? static_cast<void *>(g.part)
                                                                 : g.y) + at;
#pragma unroll
                        for (int e = 0; e < 16 / ELT; ++e)
                            if (n + e < g.N)
                                out[e] = static_cast<E>(
                                    ELT == 2 ? static_cast<unsigned int>(v[e / 2]) >> (16 * (e & 1))
                                             : static_cast<unsigned int>(v[e & 3]));
                    }
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    };

    FR fa, fb;
    // prologue: running stages 0 .. SLOTS - 1
#pragma unroll 1
    for (int p = 0; p < SLOTS; ++p) {
#pragma unroll
        for (int d = 0; d < NG; ++d) {
            const Group grp = dma_prep(p, d);
            static_for<G>([&](auto jc) { issue(grp, jc); });
        }
        advance();
    }
    wait_vmcnt<(SLOTS - 1) * C::LPS>();
    stage_barrier();
    static_for<NRD>([&](auto oc) {
        read_one_i8<TM, TN, WTM, WTN, decltype(oc)::value>(fa, slot(0), slot(0) + C::A_BYTES, 0, wm,
                                                           wn, lane);
    });

    int S = 0;  // running stage
#pragma unroll 1
    for (int k = 0; k < count; ++k) {
        const Item it = item(k);
        ACC acc;
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j)
                acc[i][j] = i32x4_t{0, 0, 0, 0};
#pragma unroll 1
        for (int D = 0; D + 1 < it.stages; ++D, ++S) {
            half(acc, std::integral_constant<int, 0>{}, S, fa, fb, std::true_type{});
            half(acc, std::integral_constant<int, 1>{}, S, fb, fa, std::true_type{});
            advance();
        }
        // the item's last stage: the next item's first fragments are read
        // after the epilogue, which then needs fewer registers
        half(acc, std::integral_constant<int, 0>{}, S, fa, fb, std::true_type{});
        half(acc, std::integral_constant<int, 1>{}, S, fb, fa, std::false_type{});
        advance();
        ++S;
        epilogue(acc, it);
        static_for<NRD>([&](auto oc) {
            read_one_i8<TM, TN, WTM, WTN, decltype(oc)::value>(fa, slot(S), slot(S) + C::A_BYTES, 0,
                                                               wm, wn, lane);
        });
    }
    wait_vmcnt<0>();  // the last loads (of nothing) have deposited their zeros
}

template <int BM, int BN, int WM, int WN, int SLOTS, int PERCU>
hipError_t launch_i8(int bf16, const I8GemmArgs &g, hipStream_t st)
{
    const int64_t items = ((g.M + BM - 1) / BM) * ((g.N + BN - 1) / BN) * g.splits;
    const int64_t per = std::min<int64_t>(cus_per_xcd() * PERCU, (items + 7) / 8);
    const dim3 grid(static_cast<unsigned>(8 * per)), block(WM * WN * 64);
    if (g.part != nullptr)
        hipLaunchKernelGGL((gemm_i8_dma_kernel<BM, BN, WM, WN, SLOTS, PERCU, OUT_PART>), grid, block, 0, st,
                           g);
    else if (bf16)
        hipLaunchKernelGGL((gemm_i8_dma_kernel<BM, BN, WM, WN, SLOTS, PERCU, OUT_BF16>), grid, block, 0, st,
                           g);
    else
        hipLaunchKernelGGL((gemm_i8_dma_kernel<BM, BN, WM, WN, SLOTS, PERCU, OUT_F32>), grid, block, 0, st,
                           g);
    return hipGetLastError();
}

}  // namespace dma

hipError_t launch_gemm_i8_dma(int bf16, const I8GemmArgs &g, int cfg, hipStream_t st)
{
    switch (cfg) {  // in the order of I8_TILES
    case 0:
        return dma::launch_i8<256, 256, 2, 2, 2, 1>(bf16, g, st);
    case 1:
        return dma::launch_i8<128, 128, 2, 2, 2, 2>(bf16, g, st);
    case 2:
        return dma::launch_i8<128, 128, 2, 2, 4, 1>(bf16, g, st);
    case 3:
        return dma::launch_i8<128, 64, 2, 2, 4, 1>(bf16, g, st);
    case 4:
        return dma::launch_i8<64, 64, 2, 2, 4, 2>(bf16, g, st);
    default:
        return hipErrorInvalidValue;
    }
}

}  // namespace dora
