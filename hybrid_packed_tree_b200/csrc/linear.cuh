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

}  // namespace stree
