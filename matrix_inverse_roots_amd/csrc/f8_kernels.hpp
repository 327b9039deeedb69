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

// four values, already scaled, as four bytes; the conversion instructions
// round to nearest even, and what is not finite is put in by hand
template <int FMT> __device__ __forceinline__ uint32_t to_f8x4(float a, float b, float c, float d) {
  uint32_t r = 0;
  if constexpr (FMT == 0) {
    r = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, r, false);
    r = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, r, true);
  } else {
    r = __builtin_amdgcn_cvt_pk_bf8_f32(a, b, r, false);
    r = __builtin_amdgcn_cvt_pk_bf8_f32(c, d, r, true);
  }
  const float m = fmaxf(fmaxf(fabsf(a), fabsf(b)), fmaxf(fabsf(c), fabsf(d)));
  if (!(m < INFINITY) || a != a || b != b || c != c || d != d) {
    const float v[4] = {a, b, c, d};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t bits = __builtin_bit_cast(uint32_t, v[i]), mag = bits & 0x7fffffffu;
      if (mag < 0x7f800000u) continue;
      const uint32_t code = ((bits >> 24) & 0x80u) | (FMT == 1 && mag == 0x7f800000u ? 0x7cu : 0x7fu);
      r = (r & ~(0xffu << (8 * i))) | (code << (8 * i));
    }
  }
  return r;
}

template <typename T> __device__ __forceinline__ float wide(T v) { return (float)v; }
template <> __device__ __forceinline__ float wide<uint16_t>(uint16_t v) { return __builtin_bit_cast(float, (uint32_t)v << 16); }

// Tile form: 256 threads, one 128 x 128 tile of one matrix.  Thread t holds
// row t / 2, columns 64 (t & 1) .. + 63 of the tile.  Serves every
// combination of outputs; T: float, _Float16, or uint16_t for bfloat16.
template <typename T, int FMT, int RB>
__global__ __launch_bounds__(256) void quantize_tile_kernel(QuantArgs g) {
  __shared__ uint32_t col_max[2][128];
  __shared__ uint32_t tile_max[4];
  __shared__ __attribute__((aligned(16))) uint8_t tr[128][144];
  const int tid = threadIdx.x, r = tid >> 1, c0 = 64 * (tid & 1);
  const int row0 = blockIdx.y * 128, col0 = blockIdx.x * 128;
  const int row = row0 + r;
  const T* x = reinterpret_cast<const T*>(g.x) + blockIdx.z * g.stride + (int64_t)row * g.ld + col0 + c0;
  const int Kp = (g.cols + 127) / 128 * 128, Rp = (g.rows + 127) / 128 * 128;
  const int Ks = (Kp / 128 + 3) / 4 * 4, Rs = (Rp / 128 + 3) / 4 * 4;
  float v[64];
  const int left = row < g.rows ? g.cols - col0 - c0 : 0;
  constexpr int VE = 16 / sizeof(T);
  if (left >= 64 && (g.ld % VE | g.stride % VE) == 0 && ((uintptr_t)g.x & 15) == 0) {
#pragma unroll
    for (int i = 0; i < 64 / VE; ++i) {
      const u32x4 w = *reinterpret_cast<const u32x4*>(x + VE * i);
      struct Pack { T v[VE]; };
      const Pack p = __builtin_bit_cast(Pack, w);
#pragma unroll
      for (int e = 0; e < VE; ++e) v[VE * i + e] = wide<T>(p.v[e]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 64; ++i) v[i] = i < left ? wide<T>(x[i]) : 0.f;
  }
  uint32_t mx = 0;
#pragma unroll
  for (int i = 0; i < 64; ++i) mx = max(mx, finite_bits(v[i]));
  mx = max(mx, (uint32_t)__shfl_xor((int)mx, 1));  // the row's 128 columns
  if constexpr (RB == 128) {
    uint32_t w = mx;
#pragma unroll
    for (int d = 2; d < 64; d *= 2) w = max(w, (uint32_t)__shfl_xor((int)w, d));
    if ((tid & 63) == 0) tile_max[tid >> 6] = w;
    __syncthreads();
    mx = max(max(tile_max[0], tile_max[1]), max(tile_max[2], tile_max[3]));
  }
  if (g.q) {
    const int byte = scale_byte<FMT>(mx);
    const float inv = inverse_scale(byte);
    if (row < g.rows) {
      uint8_t* o = g.q + ((int64_t)blockIdx.z * g.rows + row) * Kp + col0 + c0;
#pragma unroll
      for (int i = 0; i < 64; i += 16) {
        u32x4 w;
#pragma unroll
        for (int k = 0; k < 4; ++k)
          w[k] = to_f8x4<FMT>(v[i + 4 * k] * inv, v[i + 4 * k + 1] * inv, v[i + 4 * k + 2] * inv, v[i + 4 * k + 3] * inv);
        *reinterpret_cast<u32x4*>(o + i) = w;
      }
    }
    const int rs = RB == 128 ? blockIdx.y : row;
    const int nrs = RB == 128 ? (g.rows + 127) / 128 : g.rows;
    uint8_t* s = g.s + ((int64_t)blockIdx.z * nrs + rs) * Ks;
    if (c0 == 0 && (RB == 128 ? r == 0 : row < g.rows)) {
      s[blockIdx.x] = (uint8_t)byte;
      if ((int)blockIdx.x == Kp / 128 - 1)
        for (int k = blockIdx.x + 1; k < Ks; ++k) s[k] = 127;
    }
  }
  if (g.qt) {
    uint32_t byte_of[1];
    if constexpr (RB == 1) {
      // largest magnitude of each column: over the wave's 32 rows, then the
      // four waves
      __shared__ uint32_t part[4][128];
#pragma unroll
      for (int i = 0; i < 64; ++i) {
        uint32_t w = finite_bits(v[i]);
#pragma unroll
        for (int d = 2; d < 64; d *= 2) w = max(w, (uint32_t)__shfl_xor((int)w, d));
        if ((tid & 63) < 2) part[tid >> 6][c0 + i] = w;
      }
      __syncthreads();
      if (tid < 128) col_max[0][tid] = scale_byte<FMT>(max(max(part[0][tid], part[1][tid]), max(part[2][tid], part[3][tid])));
    } else {
      if (tid < 128) col_max[0][tid] = scale_byte<FMT>(mx);
    }
    byte_of[0] = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 64; ++i) {
      const float inv = inverse_scale((int)col_max[0][c0 + i]);
      tr[c0 + i][r] = (uint8_t)to_f8x4<FMT>(v[i] * inv, 0.f, 0.f, 0.f);
    }
    __syncthreads();
    // thread t: transposed row t / 2, bytes 64 (t & 1) .. + 63
    const int col = col0 + r;
    if (col < g.cols) {
      uint8_t* o = g.qt + ((int64_t)blockIdx.z * g.cols + col) * Rp + row0 + c0;
#pragma unroll
      for (int i = 0; i < 64; i += 16) *reinterpret_cast<u32x4*>(o + i) = *reinterpret_cast<const u32x4*>(&tr[r][c0 + i]);
    }
    const int rs = RB == 128 ? (int)blockIdx.x : col;
    const int nrs = RB == 128 ? (g.cols + 127) / 128 : g.cols;
    uint8_t* s = g.st + ((int64_t)blockIdx.z * nrs + rs) * Rs;
    if (c0 == 0 && (RB == 128 ? r == 0 : col < g.cols)) {
      s[blockIdx.y] = (uint8_t)col_max[0][r];
      if ((int)blockIdx.y == Rp / 128 - 1)
        for (int k = blockIdx.y + 1; k < Rs; ++k) s[k] = 127;
    }
  }
}

}  // namespace shampoo
