// fp32 grouped products on the CUDA cores and the fp32 hidden gradients of the
// expert FFNs: the training calls of the fp32 layer.
#pragma once

#include "grouped.cuh"

namespace moe {
namespace grp {

// C[g][m][n] = (add[g][m][n] +) sum_k A[g](m, k) B[g](n, k), any strides:
// A(m, k) = a[g a_group + m a_m + k a_k], likewise B.  Modes as in Set: the
// ragged extent's rows are consecutive in A (RAGGED_M), or in A and B
// (RAGGED_K), from offsets[g] on; group strides are then 0 where the buffer is
// shared by all groups.
struct Simt {
    int mode, groups, M, N, K;
    const float *a, *b, *add;
    float *c;
    int64_t a_m, a_k, a_group, b_n, b_k, b_group, c_m, c_group;
    const int32_t *offsets, *rows;
    int n_rows;
    int32_t *clear;   // nullable: the status word, set to 0
};

cudaError_t launch_simt(const Simt &p, cudaStream_t s);

// h, du (and dv) of n elements from u, (v,) dh; in place allowed.
cudaError_t launch_act_grad(int act, int64_t n, const float *u, const float *v, const float *dh,
                            float *h, float *du, float *dv, cudaStream_t s);

}  // namespace grp
}  // namespace moe
