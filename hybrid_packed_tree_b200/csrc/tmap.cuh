// tmap.cuh -- tensor maps of the packed and paged attention tensors.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

namespace stree {

// Rows of 128 bf16 (or 128 one-byte values) as a 2-D map with boxes of `box_rows` rows x
// 128 bytes, 128-byte swizzle.
bool encode_rows(CUtensorMap *m, const void *base, bool bytes, long long rows, int box_rows);

// A [rows, heads, 128] bf16 tensor as a 3-D map with boxes of 64 columns x `box_heads`
// heads x `box_rows` rows, 128-byte swizzle.
bool encode_heads(CUtensorMap *m, const void *base, long long rows, int heads, int box_heads, int box_rows);

}  // namespace stree
