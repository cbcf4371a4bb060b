// linear.cuh -- arguments of the linear-attention kernels (k_linear.cu, k_linear_tc.cu).
#pragma once

#include "stree_internal.cuh"

namespace stree {

struct LinearArgs {
    const void *q, *k, *v;             // [total or batch, heads, d]
    const float *alpha, *beta, *skip;  // beta NULL: ones; skip NULL: none
    const float *S0;                   // NULL (prompt): zeros
    const int32_t *cu;                 // prompt: packed offsets
    void *o;
    float *S_new;                      // NULL (prompt): not wanted
    int32_t *err;
    int total, batch, heads_v, heads_k, dk, dv;
    stree_dtype dtype;
};

// The tensor-core prompt pass: whether it takes the shape, the workspace in which it
// splits long sequences over CTAs, and the launch (one CTA per item without enough of it).
bool linear_tc_supported(int heads_v, int heads_k, int dk, int dv, stree_dtype dtype);
cudaError_t linear_tc_workspace(int batch, int total, int heads_v, int dv, size_t *bytes);
cudaError_t launch_linear_tc(const LinearArgs &a, void *workspace, size_t workspace_bytes, cudaStream_t s);

}  // namespace stree
