// Passes over memory around the products of product_core.hpp (gfx950): sums of
// partial results, operands copied to rows that start on 16 bytes.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gemm_common.hpp"

namespace shampoo {

// C = alpha x the sum of `splits` float32 partial results (+ beta C), any output type
// (0 float32, 1 half, 2 bfloat16); rows of N elements, ldc apart, batches of M
// rows.  2^tx threads of a workgroup go along a row, 4 columns each (vec: N
// and the rows' starts allow 16-byte accesses); the others take further rows.
static __global__ __launch_bounds__(256) void sum_splits_kernel(const float* __restrict__ part, int splits, int64_t split_stride,
                                                         void* __restrict__ C, int64_t ldc, int64_t strideC, int M, int N,
                                                         int c_dt, float alpha, const float* __restrict__ alpha_dev, float beta, int tx,
                                                         int vec) {
  if (alpha_dev) alpha *= *alpha_dev;
  const int64_t b = blockIdx.z;
  const int n = 4 * ((int)(threadIdx.x & ((1 << tx) - 1)) + ((int)blockIdx.x << tx));
  if (n >= N) return;
  for (int m = (blockIdx.y << (8 - tx)) + (threadIdx.x >> tx); m < M; m += gridDim.y << (8 - tx)) {
    const float* p = part + (b * M + m) * (int64_t)N + n;
    float a[4] = {0.f, 0.f, 0.f, 0.f};
    if (vec) {
#pragma unroll 4
      for (int s = 0; s < splits; ++s) {
        const floatx4 v = *reinterpret_cast<const floatx4*>(p + s * split_stride);
#pragma unroll
        for (int e = 0; e < 4; ++e) a[e] += v[e];
      }
    } else {
      for (int s = 0; s < splits; ++s)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (n + e < N) a[e] += p[s * split_stride + e];
    }
    const int64_t at = b * strideC + m * ldc + n;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (n + e >= N) break;
      if (c_dt == 0) {
        float* o = reinterpret_cast<float*>(C) + at + e;
        *o = alpha * a[e] + (beta != 0.f ? beta * *o : 0.f);
      } else if (c_dt == 1) {
        _Float16* o = reinterpret_cast<_Float16*>(C) + at + e;
        *o = (_Float16)(alpha * a[e] + (beta != 0.f ? beta * (float)*o : 0.f));
      } else {
        __bf16* o = reinterpret_cast<__bf16*>(C) + at + e;
        *o = (__bf16)(alpha * a[e] + (beta != 0.f ? beta * (float)*o : 0.f));
      }
    }
  }
}

// Rows of `cols` elements, ld apart, as rows of ldo elements (a multiple of
// 8) with zeros behind: an operand whose rows do not start on 16 bytes, or a
// float32 weight rounded to bfloat16.  TI, TO: float, or uint16_t for
// bfloat16.  A wave takes a row at a time, 4 elements a lane.
template <typename TI, typename TO>
__global__ __launch_bounds__(256) void pad_rows_kernel(const TI* __restrict__ x, int64_t ld, int64_t rows, int cols, TO* __restrict__ o,
                                                       int ldo, int vec) {
  struct Four { TI v[4]; };
  struct Out { TO v[4]; };
  auto turn = [](TI v) -> TO {
    if constexpr (sizeof(TI) == sizeof(TO)) return v;
    else return __builtin_bit_cast(uint16_t, (__bf16)v);
  };
  const int lane = threadIdx.x & 63;
  for (int64_t r = blockIdx.x * (int64_t)4 + (threadIdx.x >> 6); r < rows; r += (int64_t)gridDim.x * 4) {
    const TI* from = x + r * ld;
    TO* to = o + r * ldo;
    for (int c = 4 * lane; c < ldo; c += 256) {
      Out w;
      if (vec && c + 4 <= cols) {
        const Four f = *reinterpret_cast<const Four*>(from + c);
#pragma unroll
        for (int e = 0; e < 4; ++e) w.v[e] = turn(f.v[e]);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) w.v[e] = c + e < cols ? turn(from[c + e]) : TO(0);
      }
      *reinterpret_cast<Out*>(to + c) = w;
    }
  }
}

}  // namespace shampoo
