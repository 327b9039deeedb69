// Entry points of products.hip for the library's own callers (the step's
// 8-bit preconditioning products).
#pragma once

#include <hip/hip_runtime.h>

#include "shampoo.h"

namespace shampoo {

shampoo_status quantize_f8_impl(const void* x, int x_dt, int64_t n, int64_t rows, int64_t cols, int64_t ld, int64_t stride, int fmt,
                                int32_t block_rows, void* q, void* s, void* qt, void* st, hipStream_t stream);
size_t matmul_f8_bytes(int64_t n, int64_t M, int64_t N, int64_t K);
// exact: products feeding a float32 result are summed to float32 accuracy
shampoo_status matmul_f8_impl(const void* a, int a_dt, const void* a_scale, int32_t a_block_rows, const void* b, int b_dt,
                              const void* b_scale, int32_t b_block_rows, int64_t n, int64_t M, int64_t N, int64_t K, void* c, int c_dt, bool exact,
                              void* ws, size_t ws_bytes, hipStream_t stream);

}  // namespace shampoo
