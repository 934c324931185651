// gemm_rows8.hpp - the product Q^T x from x's int8 rows (gemm_rows8.hip), as dora_api.cpp
// plans and launches it.
#pragma once

#include "dora_internal.hpp"

namespace dora {

// slots[z] = Q^T x over tokens z t_per_split ..., x as int8 rows with one scale a row or
// in groups of whole tiles' columns, Q in fp32 [T, ldq] (gemm_rows8.hip).
constexpr int ROWS8_TILE = 128;
struct Rows8Args {
    const float *q;
    int64_t ldq;  // a multiple of the kernel's 64 rows of r
    const int8_t *xq;
    const float *xs;
    int group;
    int64_t T, r, d;
    int64_t t_per_split;
    float *slots;  // [splits][r, d]
};
struct Rows8Plan {
    int splits;  // 0 without tokens
    int64_t t_per_split, ldq;
};
Rows8Plan plan_rows8(int64_t T, int64_t r, int64_t d);
hipError_t launch_gemm_rows8(const Rows8Args &g, int splits, hipStream_t st);
// Q = alpha sum_z part[z], [T, r], in bf16 and (zeros up to ldq) in fp32.
hipError_t launch_q_rows8(const float *part, int splits, int64_t T, int64_t r, int64_t ldq,
                          float alpha, void *Q, float *Qf, hipStream_t st);

}  // namespace dora
