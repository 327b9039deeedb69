// Quantisation to 8-bit floating point with a power-of-two scale for each
// block of 128 (gfx950).
//
// For a block with largest finite magnitude a, 2^e is the least power of two
// with a <= L 2^e (L = 448 for e4m3, 57344 for e5m2; e = 0 for a = 0), and
// the block holds x 2^-e rounded to nearest even.  Both the scale and the
// scaling are exact, so the only rounding is the one to 8 bits, at most half
// a step, and no order of work changes a bit.  A power of two costs a
// floating format no precision (its steps are relative) and is what the
// matrix cores scale by.  NaN stays NaN; an infinity stays one in e5m2 and
// becomes NaN in e4m3, which has none; neither takes part in a.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gemm_common.hpp"

namespace shampoo {

struct QuantArgs {
  const void* x;             // [n][rows][ld]
  int64_t ld, stride;        // elements
  uint8_t* q;                // [n][rows][Kp], Kp = cols rounded up to 128 (may be null)
  uint8_t* s;                // [n][ceil(rows / rb)][Ks], Ks = Kp / 128 rounded up to 4
  uint8_t* qt;               // [n][cols][Rp], the transpose's (may be null)
  uint8_t* st;
  int rows, cols;
};

// e + 127 of a block whose largest magnitude has the bits `a` (finite, sign
// clear).  a = f 2^k with 1 <= f < 2; L = 1.75 2^top.
template <int FMT> __device__ __forceinline__ int scale_byte(uint32_t a) {
  constexpr int TOP = FMT == 0 ? 8 : 15;
  if (a == 0) return 127;
  if (a < 0x00800000u) return 0;  // below 2^-126: the clamp decides
  const int k = (int)(a >> 23);   // exponent + 127
  return max(k - TOP + ((a & 0x7fffffu) > 0x600000u ? 1 : 0), 0);
}
__device__ __forceinline__ uint32_t finite_bits(float v) {
  const uint32_t b = __builtin_bit_cast(uint32_t, v) & 0x7fffffffu;
  return b < 0x7f800000u ? b : 0u;
}
// 2^-e from the scale byte (e <= 120, so the exponent field is at least 7)
__device__ __forceinline__ float inverse_scale(int byte) { return __builtin_bit_cast(float, (uint32_t)(254 - byte) << 23); }

// four values, already scaled, as four bytes: the conversion instructions
// round to nearest even, keep NaN, and turn an infinity into e5m2's infinity
// or e4m3's NaN
template <int FMT> __device__ __forceinline__ uint32_t to_f8x4(float a, float b, float c, float d) {
  uint32_t r = 0;
  if constexpr (FMT == 0) {
    r = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, r, false);
    r = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, r, true);
  } else {
    r = __builtin_amdgcn_cvt_pk_bf8_f32(a, b, r, false);
    r = __builtin_amdgcn_cvt_pk_bf8_f32(c, d, r, true);
  }
  return r;
}
template <typename T> __device__ __forceinline__ float wide(T v) { return (float)v; }
template <> __device__ __forceinline__ float wide<uint16_t>(uint16_t v) { return __builtin_bit_cast(float, (uint32_t)v << 16); }

// One 128 x 128 tile of one matrix per workgroup of 256 threads: thread t
// holds rows 8 (t / 16) .. + 7 of columns 8 (t % 16) .. + 7, read once in 16-byte
// runs, and serves the matrix, its transpose, or both from registers.  The
// transpose goes through LDS in runs of 8 bytes so that it too is stored 16
// bytes a lane.  T: float, _Float16, or uint16_t for bfloat16.
//
// Bound by memory: 8192 x 4096 bfloat16 to 8 bits (101 MB) 20.3 us = 5.0 TB/s,
// transposed 20.9 us, float32 50001 x 1024 in 128 x 128 blocks (256 MB) 44 us =
// 5.8 TB/s; a plain copy reaches 5.2.  Rows to lanes with the columns' maxima
// across lanes, the first form, took 64 us for the transpose.
template <typename T, int FMT, int RB>
__global__ __launch_bounds__(256) void quantize_tile_kernel(QuantArgs g) {
  __shared__ uint32_t col_part[4][128];
  __shared__ uint32_t tile_part[4];
  __shared__ __attribute__((aligned(16))) uint8_t tr[128 * 128];
  const int tid = threadIdx.x, cg = tid & 15, rg = tid >> 4, wave = tid >> 6;
  const int row0 = blockIdx.y * 128, col0 = blockIdx.x * 128;
  const int row1 = row0 + 8 * rg, col1 = col0 + 8 * cg;  // this thread's first row and column
  const int Kp = (g.cols + 127) / 128 * 128, Rp = (g.rows + 127) / 128 * 128;
  const int Ks = (Kp / 128 + 3) / 4 * 4, Rs = (Rp / 128 + 3) / 4 * 4;
  const T* x = reinterpret_cast<const T*>(g.x) + blockIdx.z * g.stride + (int64_t)row1 * g.ld + col1;
  constexpr int VE = 16 / sizeof(T);
  float v[8][8];
  if (col1 + 8 <= g.cols && (g.ld % VE | g.stride % VE) == 0 && ((uintptr_t)g.x & 15) == 0) {
    struct Pack { T e[VE]; };
    u32x4 w[8][8 / VE];
#pragma unroll
    for (int r = 0; r < 8; ++r)
#pragma unroll
      for (int i = 0; i < 8 / VE; ++i)
        w[r][i] = row1 + r < g.rows ? *reinterpret_cast<const u32x4*>(x + r * g.ld + VE * i) : u32x4{0, 0, 0, 0};
#pragma unroll
    for (int r = 0; r < 8; ++r)
#pragma unroll
      for (int i = 0; i < 8 / VE; ++i) {
        const Pack p = __builtin_bit_cast(Pack, w[r][i]);
#pragma unroll
        for (int e = 0; e < VE; ++e) v[r][VE * i + e] = wide<T>(p.e[e]);
      }
  } else {
#pragma unroll
    for (int r = 0; r < 8; ++r)
#pragma unroll
      for (int i = 0; i < 8; ++i) v[r][i] = row1 + r < g.rows && col1 + i < g.cols ? wide<T>(x[r * g.ld + i]) : 0.f;
  }
  // magnitudes as integers; a wave that holds a NaN or an infinity filters
  uint32_t row_max[8], col_max[8], raw = 0;
#pragma unroll
  for (int r = 0; r < 8; ++r)
#pragma unroll
    for (int i = 0; i < 8; ++i) raw = max(raw, __builtin_bit_cast(uint32_t, v[r][i]) & 0x7fffffffu);
  const bool odd = __any(raw >= 0x7f800000u);
  auto maxima = [&](auto bits) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      uint32_t a = 0, b = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        a = max(a, bits(v[k][i]));
        b = max(b, bits(v[i][k]));
      }
      row_max[k] = a;
      col_max[k] = b;
    }
  };
  if (odd) maxima([](float f) { return finite_bits(f); });
  else maxima([](float f) { return __builtin_bit_cast(uint32_t, f) & 0x7fffffffu; });
  auto over = [](uint32_t a, int d) { return max(a, (uint32_t)__shfl_xor((int)a, d)); };
  uint32_t tile_max = 0;
  if constexpr (RB == 128) {
#pragma unroll
    for (int k = 0; k < 8; ++k) tile_max = max(tile_max, row_max[k]);
#pragma unroll
    for (int d = 1; d < 64; d *= 2) tile_max = over(tile_max, d);
    if ((tid & 63) == 0) tile_part[wave] = tile_max;
    __syncthreads();
    tile_max = max(max(tile_part[0], tile_part[1]), max(tile_part[2], tile_part[3]));
  }
  if (g.q) {
    const int nrs = RB == 128 ? (g.rows + 127) / 128 : g.rows;
    uint8_t* q = g.q + ((int64_t)blockIdx.z * g.rows + row1) * Kp + col1;
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      uint32_t mx = RB == 128 ? tile_max : row_max[r];
      if constexpr (RB == 1) {
#pragma unroll
        for (int d = 1; d < 16; d *= 2) mx = over(mx, d);
      }
      const int byte = scale_byte<FMT>(mx);
      const float inv = inverse_scale(byte);
      u32x2 o;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        uint32_t w = to_f8x4<FMT>(v[r][4 * k] * inv, v[r][4 * k + 1] * inv, v[r][4 * k + 2] * inv, v[r][4 * k + 3] * inv);
        o[k] = w;
      }
      if (row1 + r < g.rows) {
        *reinterpret_cast<u32x2*>(q + (int64_t)r * Kp) = o;
        if (cg == 0 && (RB == 1 || (rg == 0 && r == 0))) {
          uint8_t* s = g.s + ((int64_t)blockIdx.z * nrs + (RB == 128 ? (int)blockIdx.y : row1 + r)) * Ks;
          s[blockIdx.x] = (uint8_t)byte;
          if ((int)blockIdx.x == Kp / 128 - 1)
            for (int k = blockIdx.x + 1; k < Ks; ++k) s[k] = 127;
        }
      }
    }
  }
  if (g.qt) {
    if constexpr (RB == 1) {
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        col_max[c] = over(over(col_max[c], 16), 32);
        if ((tid & 48) == 0) col_part[wave][8 * cg + c] = col_max[c];
      }
      __syncthreads();
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const int at = 8 * cg + c;
        col_max[c] = max(max(col_part[0][at], col_part[1][at]), max(col_part[2][at], col_part[3][at]));
      }
    }
    const int nrs = RB == 128 ? (g.cols + 127) / 128 : g.cols;
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const int byte = scale_byte<FMT>(RB == 128 ? tile_max : col_max[c]);
      const float inv = inverse_scale(byte);
      u32x2 o;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        uint32_t w = to_f8x4<FMT>(v[4 * k][c] * inv, v[4 * k + 1][c] * inv, v[4 * k + 2][c] * inv, v[4 * k + 3][c] * inv);
        o[k] = w;
      }
      // rows of 128 bytes, run rg of transposed row 8 cg + c at rg ^ 2 (cg % 8)
      *reinterpret_cast<u32x2*>(tr + (8 * cg + c) * 128 + 8 * (rg ^ (2 * (cg & 7)))) = o;
      if (rg == 0 && col1 + c < g.cols && (RB == 1 || (cg == 0 && c == 0))) {
        uint8_t* s = g.st + ((int64_t)blockIdx.z * nrs + (RB == 128 ? (int)blockIdx.x : col1 + c)) * Rs;
        s[blockIdx.y] = (uint8_t)byte;
        if ((int)blockIdx.y == Rp / 128 - 1)
          for (int k = blockIdx.y + 1; k < Rs; ++k) s[k] = 127;
      }
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int at = k * 256 + tid, line = at >> 3, run = at & 7;  // 16 bytes: runs 2 run and 2 run + 1
      if (col0 + line < g.cols)
        *reinterpret_cast<u32x4*>(g.qt + ((int64_t)blockIdx.z * g.cols + col0 + line) * Rp + row0 + 16 * run) =
            *reinterpret_cast<const u32x4*>(tr + line * 128 + 16 * (run ^ ((line >> 3) & 7)));
    }
  }
}

}  // namespace shampoo
