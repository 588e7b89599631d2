// products.cuh -- matrix products inside the operators of a layer's training
// step (not part of the public C ABI).
#pragma once

#include "oop_internal.cuh"
#include "rows.cuh"

namespace oop {

// Rows of any oop_type as floats, `pitch` elements apart.
cudaError_t launch_to_f32(const void *src, int type, int64_t nb, int64_t cols, int64_t rows, float *dst,
                          int64_t pitch, cudaStream_t st);

// c[i, j] = alpha * sum_k a[i, k] b[j, k] + beta * c[i, j], batched; strides in elements.
struct Product {
    const float *a, *b;
    float *c;
    int64_t M, N, K, batch;
    int64_t a_row, a_col, a_mat, b_row, b_col, b_mat, c_row, c_mat;
    float alpha, beta;
};
cudaError_t launch_product(const Product &p, cudaStream_t st);

}  // namespace oop
