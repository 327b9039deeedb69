// Epilogues of the feed-forward layers on a product's tile (gfx950).
//
//   LINEAR      z = acc + bias, y = act(z) + residual; z may be kept
//   GATED       g, u in two fragments of one lane: h = act(g) u; g, u may be kept
//   GATED_GRAD  dh = acc with g, u as kept: du = dh act(g), dg = dh u act'(g),
//               and h = act(g) u again for the down projection's gradient
//
// What is kept stays in the operands' type, or in 8 bits (e4m3) with a power
// of two for each 32 columns of a row.  32 columns of a row are what two lanes
// hold of one matrix-core block, so the scale is one exchange between the
// halves of the wave; 128, the block of quantised operands, would take the
// gated form an exchange between waves, and a coarser scale.  As there, 2^e is
// the least power of two that keeps the block's largest finite magnitude
// within 448 (e = 0 for zeros), and a value has one rounding.
//
// Layout of a block (see product_core.hpp): lane l holds row l % 32 and, in
// value v, column 8 (v / 4) + 4 (l / 32) + v % 4.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "activation.hpp"
#include "f8_kernels.hpp"
#include "product_types.hpp"

namespace shampoo {

constexpr int KEEP_BLOCK = 32;  // columns of a kept block

// A 32 x 32 block from column nb on, of a row: `row` is where the lane's row
// starts, `ok` whether it is one, `cols` where the rows end.  vec: rows start
// on 16 bytes.
__device__ __forceinline__ floatx16 load_block(const float* row, bool ok, int nb, int half, int cols, int vec) {
  floatx16 r;
  if (vec && nb + 32 <= cols) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const floatx4 v = ok ? *reinterpret_cast<const floatx4*>(row + nb + 8 * q + 4 * half) : floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int e = 0; e < 4; ++e) r[4 * q + e] = v[e];
    }
  } else {
#pragma unroll
    for (int v = 0; v < 16; ++v) {
      const int n = nb + 8 * (v >> 2) + 4 * half + (v & 3);
      r[v] = ok && n < cols ? row[n] : 0.f;
    }
  }
  return r;
}
__device__ __forceinline__ floatx16 load_block(const uint16_t* row, bool ok, int nb, int half, int cols, int vec) {
  floatx16 r;
  auto put = [&](int v, uint32_t two) {
    r[v] = bits_float(two << 16);
    r[v + 1] = bits_float(two & 0xffff0000u);
  };
  if (vec && nb + 32 <= cols) {
    // 8 columns a lane; the halves of the wave swap 4 of them
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const u32x4 w = ok ? *reinterpret_cast<const u32x4*>(row + nb + 16 * q + 8 * half) : u32x4{0, 0, 0, 0};
      const auto a = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
      const auto b = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
      put(8 * q, a[0]);
      put(8 * q + 2, b[0]);
      put(8 * q + 4, a[1]);
      put(8 * q + 6, b[1]);
    }
  } else {
#pragma unroll
    for (int v = 0; v < 16; ++v) {
      const int n = nb + 8 * (v >> 2) + 4 * half + (v & 3);
      r[v] = ok && n < cols ? bits_float((uint32_t)row[n] << 16) : 0.f;
    }
  }
  return r;
}

__device__ __forceinline__ void store_block(float* row, bool ok, int nb, int half, int cols, int vec, const floatx16& x) {
  if (!ok) return;
  if (vec && nb + 32 <= cols) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      *reinterpret_cast<floatx4*>(row + nb + 8 * q + 4 * half) = floatx4{x[4 * q], x[4 * q + 1], x[4 * q + 2], x[4 * q + 3]};
  } else {
#pragma unroll
    for (int v = 0; v < 16; ++v) {
      const int n = nb + 8 * (v >> 2) + 4 * half + (v & 3);
      if (n < cols) row[n] = x[v];
    }
  }
}
__device__ __forceinline__ void store_block(uint16_t* row, bool ok, int nb, int half, int cols, int vec, const floatx16& x) {
  uint32_t two[8];
#pragma unroll
  for (int v = 0; v < 8; ++v) two[v] = pack_bf16(x[2 * v], x[2 * v + 1]);
  if (vec && nb + 32 <= cols) {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const auto a = __builtin_amdgcn_permlane32_swap(two[4 * q], two[4 * q + 2], false, false);
      const auto b = __builtin_amdgcn_permlane32_swap(two[4 * q + 1], two[4 * q + 3], false, false);
      if (ok) *reinterpret_cast<u32x4*>(row + nb + 16 * q + 8 * half) = u32x4{a[0], b[0], a[1], b[1]};
    }
  } else if (ok) {
#pragma unroll
    for (int v = 0; v < 16; ++v) {
      const int n = nb + 8 * (v >> 2) + 4 * half + (v & 3);
      if (n < cols) row[n] = (uint16_t)(two[v >> 1] >> (16 * (v & 1)));
    }
  }
}

// Rows `ld` elements apart, of float32 (dt 0) or bfloat16 (dt 2).
__device__ __forceinline__ floatx16 load_rows(const void* p, int dt, int64_t ld, int m, bool ok, int nb, int half, int cols, int vec) {
  if (dt == 0) return load_block(reinterpret_cast<const float*>(p) + m * ld, ok, nb, half, cols, vec);
  return load_block(reinterpret_cast<const uint16_t*>(p) + m * ld, ok, nb, half, cols, vec);
}
__device__ __forceinline__ void store_rows(void* p, int dt, int64_t ld, int m, bool ok, int nb, int half, int cols, int vec, const floatx16& x) {
  if (dt == 0) store_block(reinterpret_cast<float*>(p) + m * ld, ok, nb, half, cols, vec, x);
  else store_block(reinterpret_cast<uint16_t*>(p) + m * ld, ok, nb, half, cols, vec, x);
}

// 2^(byte - 127), byte 0 included
__device__ __forceinline__ float scale_value(uint32_t byte) { return bits_float(byte ? byte << 23 : 0x00400000u); }

// Largest finite magnitude's bits among 16 values of this lane and of its
// partner in the other half of the wave.
__device__ __forceinline__ uint32_t block_max(const floatx16& x) {
  uint32_t a = 0;
#pragma unroll
  for (int v = 0; v < 16; ++v) a = max(a, float_bits(x[v]) & 0x7fffffffu);
  if (__any(a >= 0x7f800000u)) {
    a = 0;
#pragma unroll
    for (int v = 0; v < 16; ++v) a = max(a, finite_bits(x[v]));
  }
  const auto s = __builtin_amdgcn_permlane32_swap(a, a, false, false);
  return max(s[0], s[1]);
}

// A block to 8 bits: 16 bytes a lane, the first half of the wave the first 16
// columns.  Rows of `ld` bytes (cols rounded up to 32), their scales behind
// one another; columns past `cols` become zeros.
__device__ __forceinline__ void keep_f8(uint8_t* q, uint8_t* s, int64_t ld, int m, bool ok, int nb, int half, int cols, floatx16 x) {
  if (nb + 32 > cols) {
#pragma unroll
    for (int v = 0; v < 16; ++v)
      if (nb + 8 * (v >> 2) + 4 * half + (v & 3) >= cols) x[v] = 0.f;
  }
  const int byte = scale_byte<0>(block_max(x));
  const float inv = inverse_scale(byte);
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = to_f8x4<0>(x[4 * i] * inv, x[4 * i + 1] * inv, x[4 * i + 2] * inv, x[4 * i + 3] * inv);
  const auto a = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
  const auto b = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
  if (ok && nb < cols) {
    *reinterpret_cast<u32x4*>(q + m * ld + nb + 16 * half) = u32x4{a[0], a[1], b[0], b[1]};
    if (half == 0) s[m * (ld / KEEP_BLOCK) + nb / KEEP_BLOCK] = (uint8_t)byte;
  }
}
__device__ __forceinline__ floatx16 kept_f8(const uint8_t* q, const uint8_t* s, int64_t ld, int m, bool ok, int nb, int half, int cols) {
  u32x4 w = u32x4{0, 0, 0, 0};
  uint32_t byte = 127;
  if (ok && nb < cols) {
    w = *reinterpret_cast<const u32x4*>(q + m * ld + nb + 16 * half);
    byte = s[m * (ld / KEEP_BLOCK) + nb / KEEP_BLOCK];
  }
  const float scale = scale_value(byte);
  const auto a = __builtin_amdgcn_permlane32_swap(w[0], w[1], false, false);
  const auto b = __builtin_amdgcn_permlane32_swap(w[2], w[3], false, false);
  const uint32_t four[4] = {a[0], b[0], a[1], b[1]};
  floatx16 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const floatx2 lo = __builtin_amdgcn_cvt_pk_f32_fp8(four[i], false), hi = __builtin_amdgcn_cvt_pk_f32_fp8(four[i], true);
    r[4 * i] = lo[0] * scale;
    r[4 * i + 1] = lo[1] * scale;
    r[4 * i + 2] = hi[0] * scale;
    r[4 * i + 3] = hi[1] * scale;
  }
  return r;
}

__device__ __forceinline__ void keep_block(const FfnArgs& e, int which, int m, bool ok, int nb, int half, int cols, const floatx16& x) {
  if (e.keep_dt == 4) keep_f8((uint8_t*)e.keep[which], e.keep_scale[which], e.ld_keep, m, ok, nb, half, cols, x);
  else store_rows(e.keep[which], e.keep_dt, e.ld_keep, m, ok, nb, half, cols, e.keep_vec, x);
}
__device__ __forceinline__ floatx16 kept_block(const FfnArgs& e, int which, int m, bool ok, int nb, int half, int cols) {
  if (e.keep_dt == 4) return kept_f8((const uint8_t*)e.keep[which], e.keep_scale[which], e.ld_keep, m, ok, nb, half, cols);
  return load_rows(e.keep[which], e.keep_dt, e.ld_keep, m, ok, nb, half, cols, e.keep_vec);
}

template <int FM, int FN>
__device__ __forceinline__ void linear_epilogue(const ProductArgs& g, floatx16 (&acc)[FM][FN], int m0, int n0, int l32, int half) {
  const FfnArgs& e = g.ffn;
  if (e.bias) {
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) {
        const int n = min(n0 + 32 * j + 8 * (v >> 2) + 4 * half + (v & 3), g.N - 1);
        const float b = e.bias_bf16 ? bits_float((uint32_t)reinterpret_cast<const uint16_t*>(e.bias)[n] << 16) : reinterpret_cast<const float*>(e.bias)[n];
#pragma unroll
        for (int i = 0; i < FM; ++i) acc[i][j][v] += b;
      }
  }
  if (e.keep[0]) {
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) keep_block(e, 0, m0 + 32 * i + l32, m0 + 32 * i + l32 < g.M, n0 + 32 * j, half, g.N, acc[i][j]);
  }
  if (e.act) {
    with_activation(e.act, [&](auto act) {
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
          for (int v = 0; v < 16; ++v) acc[i][j][v] = act.value(acc[i][j][v]);
    });
  }
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    const int m = m0 + 32 * i + l32;
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      const int nb = n0 + 32 * j;
      if (nb >= g.N) continue;
      if (e.residual) {
        const floatx16 r = load_rows(e.residual, g.c_dt, e.ld_residual, m, m < g.M, nb, half, g.N, e.residual_vec);
#pragma unroll
        for (int v = 0; v < 16; ++v) acc[i][j][v] += r[v];
      }
      store_rows(g.C, g.c_dt, g.ldc, m, m < g.M, nb, half, g.N, g.vec, acc[i][j]);
    }
  }
}

// C receives h: rows of ldc, zeros behind the columns
template <int FM>
__device__ __forceinline__ void gated_epilogue(const ProductArgs& g, floatx16 (&acc)[FM][4], int m0, int n0, int l32, int half, int range) {
  const FfnArgs& e = g.ffn;
  if (g.splits > 1) {
    float* part = e.part + (int64_t)range * g.M * 2 * g.N;
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      const int m = m0 + 32 * i + l32;
      float* row = part + m * (int64_t)(2 * g.N);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        store_block(row + (j >> 1) * g.N, m < g.M, n0 + 32 * (j & 1), half, g.N, g.N % 4 == 0, acc[i][j]);
    }
    return;
  }
  if (e.keep[0]) {
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        keep_block(e, j >> 1, m0 + 32 * i + l32, m0 + 32 * i + l32 < g.M, n0 + 32 * (j & 1), half, g.N, acc[i][j]);
  }
  with_activation(e.act, [&](auto act) {
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int v = 0; v < 16; ++v) acc[i][j][v] = act.value(acc[i][j][v]) * acc[i][j + 2][v];
  });
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    const int m = m0 + 32 * i + l32;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int nb = n0 + 32 * j;
      if (nb + 32 > g.N) {
#pragma unroll
        for (int v = 0; v < 16; ++v)
          if (nb + 8 * (v >> 2) + 4 * half + (v & 3) >= g.N) acc[i][j][v] = 0.f;
      }
      store_rows(g.C, g.c_dt, g.ldc, m, m < g.M, nb, half, (int)g.ldc, g.vec, acc[i][j]);
    }
  }
}

// ES: bytes of an element of dg, du (rows of ldc) and h (rows of ldc / 2), zeros behind the columns
template <int FM, int FN, int ES>
__device__ __forceinline__ void gated_grad_epilogue(const ProductArgs& g, floatx16 (&acc)[FM][FN], int m0, int n0, int l32, int half) {
  const FfnArgs& e = g.ffn;
  constexpr int DT = ES == 4 ? 0 : 2;
  const int wide = (int)(g.ldc / 2);
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    const int m = m0 + 32 * i + l32;
    const bool ok = m < g.M;
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      const int nb = n0 + 32 * j;
      if (nb >= wide) continue;
      floatx16 gate = kept_block(e, 0, m, ok, nb, half, g.N), up = kept_block(e, 1, m, ok, nb, half, g.N);
      floatx16 dg, h;
      with_activation(e.act, [&](auto act) {
#pragma unroll
        for (int v = 0; v < 16; ++v) {
          float slope;
          const float a = act.both(gate[v], slope), dh = acc[i][j][v];
          h[v] = a * up[v];
          dg[v] = dh * up[v] * slope;
          acc[i][j][v] = dh * a;
        }
      });
      if (nb + 32 > g.N) {
#pragma unroll
        for (int v = 0; v < 16; ++v)
          if (nb + 8 * (v >> 2) + 4 * half + (v & 3) >= g.N) h[v] = dg[v] = acc[i][j][v] = 0.f;
      }
      store_rows(g.C, DT, g.ldc, m, ok, nb, half, wide, 1, dg);
      store_rows(e.du, DT, g.ldc, m, ok, nb, half, wide, 1, acc[i][j]);
      store_rows(e.h, DT, wide, m, ok, nb, half, wide, 1, h);
    }
  }
}

}  // namespace shampoo
