// 8-bit block-scaled product for few rows (serving: one to four tokens).
//
// With so few rows the product is a read of B: N x K bytes once.  A wave
// takes 4 rows of B, its lanes 16 consecutive bytes of each in turn, so that
// a 1 KB run of every row is one load and four are in flight; A's runs come
// from cache.  Operands are widened to float32 (exactly), 16 products are
// summed and scaled by the block's power of two, and the lanes' sums are
// joined at the end.  No matrix cores, no split of k: one launch.
// One row, N = 4096, K = 1024: 4.1 us against 11.0 on the 128-tiles (32
// workgroups, each alone with its latency); N = K = 8192: 14.6 against 19.6
// (4.6 TB/s).  Every row of A adds its own widening and sums: at N = K = 4096
// two rows take 9.4 us and four 11.1 against the tiles' 14.1, eight 24.4.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gemm_common.hpp"
#include "product_core.hpp"

namespace shampoo {

constexpr int F8_ROWS_MAX = 4;  // rows of A

template <int F> __device__ __forceinline__ void widen16(u32x4 q, float* o) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    floatx2 lo, hi;
    if constexpr (F == 0) {
      lo = __builtin_amdgcn_cvt_pk_f32_fp8(q[i], false);
      hi = __builtin_amdgcn_cvt_pk_f32_fp8(q[i], true);
    } else {
      lo = __builtin_amdgcn_cvt_pk_f32_bf8(q[i], false);
      hi = __builtin_amdgcn_cvt_pk_f32_bf8(q[i], true);
    }
    o[4 * i] = lo[0];
    o[4 * i + 1] = lo[1];
    o[4 * i + 2] = hi[0];
    o[4 * i + 3] = hi[1];
  }
}

// MB: rows of A, at most; grid (N / 16, batch), 256 threads
template <int MB, int FA, int FB>
__global__ __launch_bounds__(256) void f8_rows_kernel(ProductArgs g) {
  constexpr int NR = 4;
  const int lane = threadIdx.x & 63, n0 = (blockIdx.x * 4 + (threadIdx.x >> 6)) * NR;
  if (n0 >= g.N) return;
  const int64_t batch = blockIdx.y;
  const uint8_t* A = reinterpret_cast<const uint8_t*>(g.A) + batch * g.strideA;
  const uint8_t* sa = g.sa + batch * g.strideSa;
  const uint8_t* B[NR];
  const uint8_t* sb[NR];
#pragma unroll
  for (int r = 0; r < NR; ++r) {
    const int n = min(n0 + r, g.N - 1);
    B[r] = reinterpret_cast<const uint8_t*>(g.B) + batch * g.strideB + (int64_t)n * g.ldb;
    sb[r] = g.sb + batch * g.strideSb + (int64_t)(n >> g.sb_shift) * g.ldsb;
  }
  float acc[MB][NR];
#pragma unroll
  for (int m = 0; m < MB; ++m)
#pragma unroll
    for (int r = 0; r < NR; ++r) acc[m][r] = 0.f;
#pragma unroll 2
  for (int c = lane; c < g.K / 16; c += 64) {
    u32x4 q[NR];
    int eb[NR];
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      q[r] = *reinterpret_cast<const u32x4*>(B[r] + 16 * c);
      eb[r] = sb[r][c >> 3];
    }
    float b[NR][16];
#pragma unroll
    for (int r = 0; r < NR; ++r) widen16<FB>(q[r], b[r]);
#pragma unroll
    for (int m = 0; m < MB; ++m) {
      const int row = min(m, g.M - 1);
      float a[16];
      widen16<FA>(*reinterpret_cast<const u32x4*>(A + row * g.lda + 16 * c), a);
      const int ea = (int)sa[(row >> g.sa_shift) * g.ldsa + (c >> 3)] - 254;
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        float s = a[0] * b[r][0];
#pragma unroll
        for (int e = 1; e < 16; ++e) s = __builtin_fmaf(a[e], b[r][e], s);
        acc[m][r] += ldexpf(s, ea + eb[r]);
      }
    }
  }
#pragma unroll
  for (int m = 0; m < MB; ++m)
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      float s = acc[m][r];
#pragma unroll
      for (int d = 1; d < 64; d *= 2) s += __shfl_xor(s, d);
      if (lane == m * NR + r && m < g.M && n0 + r < g.N) {
        const int64_t at = batch * g.strideC + m * g.ldc + n0 + r;
        if (g.c_dt == 0) reinterpret_cast<float*>(g.C)[at] = s;
        else if (g.c_dt == 1) reinterpret_cast<_Float16*>(g.C)[at] = (_Float16)s;
        else reinterpret_cast<__bf16*>(g.C)[at] = (__bf16)s;
      }
    }
}

}  // namespace shampoo
