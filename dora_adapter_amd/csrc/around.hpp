// around.hpp - the operators that stand around a module, as dora_api.cpp plans and launches
// them: the norms on both sides of a residual addition (block_norm.hip), 4-bit weights
// (fourbit.hip, gemm_fourbit.hip) and orthogonalised updates (newton_schulz.hip).
#pragma once

#include "dora_internal.hpp"

namespace dora {

// ------------------------------------------------------------ block_norm.hip
// Row t of x uses row t / gate_rows of the gate (gate_rows 0: no gate).
struct BlockNormArgs {
    const void *x, *res, *w_post, *gate, *w_pre;  // w_post, gate may be null
    float res_scale, branch_scale, eps;
    int64_t T, d, gate_rows;
    void *h, *y;
    float *rstd_post, *rstd_pre;  // each may be null
};
hipError_t launch_block_norm(int bf16, const BlockNormArgs &a, hipStream_t st);

// How the rows are dealt to the gradient's workgroups, and what it keeps in its workspace.
struct BlockNormPlan {
    bool held;         // rows held in a workgroup's registers, one pass
    int64_t chunk;     // consecutive rows a workgroup
    int parts;         // of them
    bool direct;       // a gate row's rows all lie in one chunk: its sum is final there
    int64_t slots;     // partial sums of gate rows otherwise
    size_t o_pre, o_post, o_gate, o_mean, bytes;
};
BlockNormPlan plan_block_norm_grad(int64_t T, int64_t d, int64_t gate_rows);
struct BlockNormGradArgs {
    const void *dy, *dh, *x, *h, *w_pre, *w_post, *gate;  // dh, w_post, gate may be null
    const float *rstd_pre, *rstd_post;
    float res_scale, branch_scale;
    int64_t T, d, gate_rows;
    void *dx, *dres, *dgate;   // dgate may be null
    float *dw_pre, *dw_post;   // each may be null
};
hipError_t launch_block_norm_grad(int bf16, const BlockNormGradArgs &a, const BlockNormPlan &p,
                                  void *ws, hipStream_t st);

// --------------------------------------------------- fourbit.hip, gemm_fourbit.hip
// 4-bit rows: e2m1 codes two a byte, rows of whole groups (`groups` of them), bf16 scales.
hipError_t launch_quantize_fourbit(int bf16, const void *x, int64_t rows, int64_t d, int group,
                                   uint8_t *codes, uint16_t *scale, hipStream_t st);
hipError_t launch_dequantize_fourbit(int bf16, const uint8_t *codes, const uint16_t *scale,
                                     int64_t rows, int64_t d, int group, void *out, hipStream_t st);
// out[m, n] = sum_z part[z, m, n] in order, rounded once; ldo elements between rows of `out`.
hipError_t launch_sum_splits(int bf16, const float *part, int splits, int64_t M, int64_t N, void *out,
                             int64_t ldo, hipStream_t st);
struct FourbitArgs {
    const void *x;  // [T, d_in]
    const uint8_t *codes;
    const uint16_t *scale;
    void *y;  // [T, d_out]
    int64_t T, d_in, d_out;
    int64_t groups;
    int group;
};
hipError_t launch_linear_fourbit(int bf16, const FourbitArgs &a, hipStream_t st);

// --------------------------------------------------------------- newton_schulz.hip
// One matrix U [rows, cols]: the gradient g alone, or, with a momentum, g + mu M' or M' for
// M' = mu M + g.  Its orthogonalised form O goes to `out`, or out = keep p - step O.
struct NsMatrix {
    const void *g, *p;  // p may be null
    const float *m;     // may be null
    float *m_out;
    void *out;
    int64_t rows, cols;
    float step, keep;
};
struct NsParams {
    float mu;
    int nesterov, steps;
    float a, b, c, eps;
};
constexpr int NS_MAX_STEPS = 16;
constexpr int64_t NS_MAX_SHORT = 8192;  // the shorter side
bool newton_schulz_fits(int64_t rows, int64_t cols);
size_t newton_schulz_workspace(const NsMatrix *mats, int count);
hipError_t launch_newton_schulz(int bf16, const NsMatrix *mats, int count, const NsParams &p, void *ws,
                                hipStream_t st);

}  // namespace dora
