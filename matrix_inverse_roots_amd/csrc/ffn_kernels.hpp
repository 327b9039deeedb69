// Kernels of the feed-forward layers beside the products (gfx950): layers of
// one to four rows, sums of partial results with the layers' epilogues, the
// activation's gradient with the bias's, operands kept in 8 bits.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "activation.hpp"
#include "ffn_epilogue.hpp"
#include "product_types.hpp"

namespace shampoo {

constexpr int FFN_ROWS_MAX = 4;

__device__ __forceinline__ float load_one(const void* p, int dt, int64_t at) {
  return dt == 0 ? reinterpret_cast<const float*>(p)[at] : bits_float((uint32_t)reinterpret_cast<const uint16_t*>(p)[at] << 16);
}
__device__ __forceinline__ void store_one(void* p, int dt, int64_t at, float v) {
  if (dt == 0) reinterpret_cast<float*>(p)[at] = v;
  else reinterpret_cast<__bf16*>(p)[at] = (__bf16)v;
}
__device__ __forceinline__ float round_bf16(float v) { return (float)(__bf16)v; }

// ---------------------------------------------------------------------------
// few rows
// ---------------------------------------------------------------------------
struct RowsArgs {
  const void* x;          // [M][ldx]
  const void* w;          // [N][ldw]
  const void* w2;         // GATED: the up projection
  const void* bias;
  const void* residual;
  void* y;                // [M][ldy]; GATED: h
  void* keep[2];
  int64_t ldx, ldw, ldw2, ld_residual, ldy, ld_keep;
  int M, N, K;
  int act, y_dt, keep_dt, bias_bf16;
  int kw;                 // waves that share a row's k: 1, 2 or 4
  int vec;                // rows of x and w start on 16 bytes
};

// 8 consecutive elements, as float32 (those from `left` on as zeros).  ROUND: to bfloat16 on the way.
template <typename T, bool ROUND> __device__ __forceinline__ void load8(const T* p, bool vec, int left, float* o) {
  if (vec && left >= 8) {
    if constexpr (sizeof(T) == 2) {
      const u32x4 w = *reinterpret_cast<const u32x4*>(p);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        o[2 * i] = bits_float(w[i] << 16);
        o[2 * i + 1] = bits_float(w[i] & 0xffff0000u);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const floatx4 v = *reinterpret_cast<const floatx4*>(p + 4 * i);
#pragma unroll
        for (int e = 0; e < 4; ++e) o[4 * i + e] = ROUND ? round_bf16(v[e]) : v[e];
      }
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float v = 0.f;
      if (e < left) {
        if constexpr (sizeof(T) == 2) v = bits_float((uint32_t)p[e] << 16);
        else v = ROUND ? round_bf16(p[e]) : p[e];
      }
      o[e] = v;
    }
  }
}

// A read of the weights: with so few rows the products are N x K values once,
// in 16-byte loads of 4 columns at a time (GATED: 4 of either projection), all
// of a wave's share of k in flight.  kw waves of a workgroup share a column's
// k, 512 elements each at a time, and meet in LDS, so that short and long sums
// both fill the chip.  Products and sums are float32.
// One row, 4096 x 1024 bfloat16 (8.4 MB): 3.7-4.0 us; both projections (16.8 MB)
// 6.6 us = 2.5 TB/s, 1024 x 4096 5.0 us: bound by the latency of the loads and of
// the launch.  Against the 128-tiles with their ranges of k: 4096 x 1024, one row
// 3.7 and 10.2 us, four 5.1 and 10.2; 1024 x 4096, four rows 6.3 and 10.4; 8192 x
// 8192, four rows 40 and 39: from there on the widening of more rows costs more
// than a second launch, so four rows are the most.
// MB: rows, at most.  TX, TW: float, or uint16_t for bfloat16.  ROUND: a
// float32 weight enters as bfloat16.
template <typename TX, typename TW, bool ROUND, int MB, bool GATED>
__global__ __launch_bounds__(256) void ffn_rows_kernel(RowsArgs g) {
  constexpr int NC = 4, NW = GATED ? 2 * NC : NC;
  __shared__ float red[4][MB * NW];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int ks = wave % g.kw, group = wave / g.kw;
  const int n0 = (blockIdx.x * (4 / g.kw) + group) * NC;
  const TX* x = reinterpret_cast<const TX*>(g.x);
  float acc[MB][NW];
#pragma unroll
  for (int m = 0; m < MB; ++m)
#pragma unroll
    for (int r = 0; r < NW; ++r) acc[m][r] = 0.f;
  const TW* w[NW];
#pragma unroll
  for (int r = 0; r < NW; ++r)
    w[r] = reinterpret_cast<const TW*>(r < NC ? g.w : g.w2) + min(n0 + r % NC, g.N - 1) * (r < NC ? g.ldw : g.ldw2);
#pragma unroll 2
  for (int k = (ks * 64 + lane) * 8; k < g.K; k += g.kw * 512) {
    float b[NW][8];
#pragma unroll
    for (int r = 0; r < NW; ++r) load8<TW, ROUND>(w[r] + k, g.vec, g.K - k, b[r]);
#pragma unroll
    for (int m = 0; m < MB; ++m) {
      float a[8];
      load8<TX, false>(x + min(m, g.M - 1) * g.ldx + k, g.vec, g.K - k, a);
#pragma unroll
      for (int r = 0; r < NW; ++r)
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[m][r] = __builtin_fmaf(a[e], b[r][e], acc[m][r]);
    }
  }
  // sums over the wave: halves of it, then quarters, take a value each, so that
  // a register serves four values when 16 lanes are left to join
#pragma unroll
  for (int m = 0; m < MB; ++m)
#pragma unroll
    for (int r = 0; r < NW; r += 4) {
      float two[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const auto w = __builtin_amdgcn_permlane32_swap(float_bits(acc[m][r + 2 * i]), float_bits(acc[m][r + 2 * i + 1]), false, false);
        two[i] = bits_float(w[0]) + bits_float(w[1]);
      }
      const auto w = __builtin_amdgcn_permlane16_swap(float_bits(two[0]), float_bits(two[1]), false, false);
      float t = bits_float(w[0]) + bits_float(w[1]);
#pragma unroll
      for (int d = 1; d < 16; d *= 2) t += __shfl_xor(t, d);
      // quarters: value 0 of r, 2, 1, 3
      if ((lane & 15) == 0) red[wave][m * NW + r + ((lane >> 4 & 1) << 1 | lane >> 5)] = t;
    }
  __syncthreads();
  if (ks != 0) return;
  const int m = lane / NC, c = lane % NC, n = n0 + c;
  if (m >= MB || m >= g.M || n >= g.N) return;
  float z = 0.f, u = 0.f;
  for (int s = 0; s < g.kw; ++s) {
    z += red[wave + s][m * NW + c];
    if (GATED) u += red[wave + s][m * NW + NC + c];
  }
  if (g.bias) z += load_one(g.bias, g.bias_bf16 ? 2 : 0, n);
  if (g.keep[0]) store_one(g.keep[0], g.keep_dt, m * g.ld_keep + n, z);
  if (GATED && g.keep[1]) store_one(g.keep[1], g.keep_dt, m * g.ld_keep + n, u);
  float y = z;
  with_activation(g.act, [&](auto act) { y = act.value(z); });
  if (GATED) y *= u;
  if (g.residual) y += load_one(g.residual, g.y_dt, m * g.ld_residual + n);
  store_one(g.y, g.y_dt, m * g.ldy + n, y);
}

// ---------------------------------------------------------------------------
// partial results of a product split along k
// ---------------------------------------------------------------------------
struct FinishArgs {
  const float* part;      // [range][M][P], GATED: [range][M][2 P], P: N rounded up to 4
  int64_t range_stride;
  int splits, M, N, wide; // wide: GATED: h's padded width
  void* y;
  int64_t ldy;
  int y_dt;
  FfnArgs ffn;
};

// Sums the ranges and applies the layer's epilogue.  A thread takes 4 columns,
// 8 threads a kept block.  Grid (column blocks of 1024, rows).  Bound by the
// latency of its loads: 4 ranges of 77 x 2 x 2731 (6.7 MB) 3.0 us, 77 x 1000 3.2.
template <bool GATED>
static __global__ __launch_bounds__(256) void ffn_finish_kernel(FinishArgs g) {
  const FfnArgs& e = g.ffn;
  const int n = (blockIdx.x * 256 + threadIdx.x) * 4;
  const int P = (g.N + 3) & ~3;
  const int64_t row = GATED ? 2 * (int64_t)P : P;
  for (int m = blockIdx.y; m < g.M; m += gridDim.y) {
    float z[GATED ? 2 : 1][4];
#pragma unroll
    for (int p = 0; p < (GATED ? 2 : 1); ++p) {
#pragma unroll
      for (int c = 0; c < 4; ++c) z[p][c] = 0.f;
      const float* from = g.part + m * row + p * P + n;
      if (n < g.N) {
#pragma unroll 8
        for (int s = 0; s < g.splits; ++s) {
          const floatx4 v = *reinterpret_cast<const floatx4*>(from + s * g.range_stride);
#pragma unroll
          for (int c = 0; c < 4; ++c) z[p][c] += n + c < g.N ? v[c] : 0.f;  // columns from N on hold anything
        }
      }
    }
    if (e.bias) {
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (n + c < g.N) z[0][c] += load_one(e.bias, e.bias_bf16 ? 2 : 0, n + c);
    }
    if (e.keep[0]) {
#pragma unroll
      for (int p = 0; p < (GATED ? 2 : 1); ++p) {
        if (e.keep_dt == 4) {
          uint32_t a = 0;
#pragma unroll
          for (int c = 0; c < 4; ++c) a = max(a, finite_bits(z[p][c]));
#pragma unroll
          for (int d = 1; d < 8; d *= 2) a = max(a, (uint32_t)__shfl_xor((int)a, d));
          const int byte = scale_byte<0>(a);
          const float inv = inverse_scale(byte);
          if (n < e.ld_keep) {
            *reinterpret_cast<uint32_t*>((uint8_t*)e.keep[p] + m * e.ld_keep + n) =
                to_f8x4<0>(z[p][0] * inv, z[p][1] * inv, z[p][2] * inv, z[p][3] * inv);
            if ((threadIdx.x & 7) == 0) e.keep_scale[p][m * (e.ld_keep / KEEP_BLOCK) + n / KEEP_BLOCK] = (uint8_t)byte;
          }
        } else {
#pragma unroll
          for (int c = 0; c < 4; ++c)
            if (n + c < g.N) store_one(e.keep[p], e.keep_dt, m * e.ld_keep + n + c, z[p][c]);
        }
      }
    }
    float y[4] = {z[0][0], z[0][1], z[0][2], z[0][3]};
    with_activation(e.act, [&](auto act) {
#pragma unroll
      for (int c = 0; c < 4; ++c) y[c] = act.value(y[c]);
    });
    if constexpr (GATED) {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        y[c] *= z[1][c];
        if (n + c < g.wide) store_one(g.y, g.y_dt, m * g.ldy + n + c, n + c < g.N ? y[c] : 0.f);
      }
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (n + c < g.N) {
          if (e.residual) y[c] += load_one(e.residual, g.y_dt, m * e.ld_residual + n + c);
          store_one(g.y, g.y_dt, m * g.ldy + n + c, y[c]);
        }
    }
  }
}

// ---------------------------------------------------------------------------
// the activation's gradient and the bias's
// ---------------------------------------------------------------------------
constexpr int GRAD_ROWS = 128;  // rows of a workgroup of act_grad_kernel

struct ActGradArgs {
  const void* dy;
  const void* z;            // as kept; null without an activation
  const uint8_t* z_scale;
  void* dz;                 // rows of ld_dz elements, zeros behind the columns; or null
  float* sums;              // [row chunks][N]: the chunk's sums of dz; or null
  int64_t ld_dy, ld_z, ld_dz;
  int M, N, act, z_dt;
  int dy_vec, z_vec;
  int blocks;               // of 128 columns
};

// dz = dy act'(z) and its sums over 128 rows, from the float32 values.  A
// thread takes 8 columns of every 16th row; 16 threads a row.  One pass serves
// both products and the bias.  8192 x 4096 bfloat16 with gelu: 39 us, from z in
// bfloat16 (201 MB, 5.1 TB/s) and from 8 bits (168 MB) alike: the memory and the
// derivative's arithmetic (some 45 instructions an element) take as long.
template <typename T>
__global__ __launch_bounds__(256) void act_grad_kernel(ActGradArgs g) {
  __shared__ float red[16][128 + 4];
  const int cg = threadIdx.x & 15, rg = threadIdx.x >> 4;
  const int col0 = (int)(blockIdx.x % g.blocks) * 128;
  const int64_t chunk = blockIdx.x / g.blocks;
  const int n = col0 + 8 * cg, left = g.N - n;
  const T* dy = reinterpret_cast<const T*>(g.dy);
  float sum[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) sum[e] = 0.f;
#pragma unroll 2
  for (int r = 0; r < GRAD_ROWS / 16; ++r) {
    const int m = (int)chunk * GRAD_ROWS + 16 * r + rg;
    if (m >= g.M || left <= 0) break;
    float d[8];
    load8<T, false>(dy + m * g.ld_dy + n, g.dy_vec, left, d);
    if (g.act) {
      float z[8];
      if (g.z_dt == 4) {
        // rows of whole blocks: 8 columns start inside them wherever n < N
        const u32x2 w = *reinterpret_cast<const u32x2*>(reinterpret_cast<const uint8_t*>(g.z) + m * g.ld_z + n);
        const float scale = scale_value(g.z_scale[m * (g.ld_z / KEEP_BLOCK) + n / KEEP_BLOCK]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const floatx2 lo = __builtin_amdgcn_cvt_pk_f32_fp8(w[i], false), hi = __builtin_amdgcn_cvt_pk_f32_fp8(w[i], true);
          z[4 * i] = lo[0] * scale;
          z[4 * i + 1] = lo[1] * scale;
          z[4 * i + 2] = hi[0] * scale;
          z[4 * i + 3] = hi[1] * scale;
        }
      } else {
        load8<T, false>(reinterpret_cast<const T*>(g.z) + m * g.ld_z + n, g.z_vec, left, z);
      }
      with_activation(g.act, [&](auto act) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float slope;
          act.both(z[e], slope);
          d[e] = e < left ? d[e] * slope : 0.f;
        }
      });
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) sum[e] += d[e];
    if (g.dz) {
      T* to = reinterpret_cast<T*>(g.dz) + m * g.ld_dz + n;
      if constexpr (sizeof(T) == 2) {
        *reinterpret_cast<u32x4*>(to) = u32x4{pack_bf16(d[0], d[1]), pack_bf16(d[2], d[3]), pack_bf16(d[4], d[5]), pack_bf16(d[6], d[7])};
      } else {
        *reinterpret_cast<floatx4*>(to) = floatx4{d[0], d[1], d[2], d[3]};
        *reinterpret_cast<floatx4*>(to + 4) = floatx4{d[4], d[5], d[6], d[7]};
      }
    }
  }
  if (!g.sums) return;
#pragma unroll
  for (int e = 0; e < 8; ++e) red[rg][8 * cg + e] = sum[e];
  __syncthreads();
  const int c = threadIdx.x;
  if (c < 128 && col0 + c < g.N) {
    float s = 0.f;
#pragma unroll
    for (int r = 0; r < 16; ++r) s += red[r][c];
    g.sums[chunk * g.N + col0 + c] = s;
  }
}

// dbias from the chunks' sums: a column per thread of a wave, chunks dealt to
// the 16 waves (+ dbias where accumulated).  Bound by latency: 64 x 4096 4.7 us.
static __global__ __launch_bounds__(1024) void bias_grad_kernel(const float* __restrict__ sums, int chunks, int N, void* __restrict__ out,
                                                                int dt, int accumulate) {
  __shared__ float red[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, n = blockIdx.x * 64 + lane;
  float s = 0.f;
  if (n < N) {
#pragma unroll 4
    for (int c = wave; c < chunks; c += 16) s += sums[(int64_t)c * N + n];
  }
  red[wave][lane] = s;
  __syncthreads();
  if (wave != 0 || n >= N) return;
  s = 0.f;
#pragma unroll
  for (int w = 0; w < 16; ++w) s += red[w][lane];
  if (accumulate) s += load_one(out, dt, n);
  store_one(out, dt, n, s);
}

// ---------------------------------------------------------------------------
// operands whose rows do not start on 16 bytes
// ---------------------------------------------------------------------------
// Rows of `cols` elements, ld apart, as rows of ldo (a multiple of 8) with zeros
// behind; float32 to bfloat16 on the way where TI and TO say so.  A wave takes
// 512 elements of a row, 8 a lane, in 16-byte loads at any element's address: 1000
// rows of 2731 bfloat16 (11 MB) 5.4 us, against 9.4 in loads of single elements.
template <typename TI, typename TO>
__global__ __launch_bounds__(256) void copy_rows_kernel(const TI* __restrict__ x, int64_t ld, int64_t rows, int cols, TO* __restrict__ o, int64_t ldo) {
  struct Eight { TI v[8]; };
  const int lane = threadIdx.x & 63;
  for (int64_t r = blockIdx.x * (int64_t)4 + (threadIdx.x >> 6); r < rows; r += (int64_t)gridDim.x * 4) {
    const TI* row = x + r * ld;
    TO* to = o + r * ldo;
    const int c = blockIdx.y * 512 + 8 * lane;
    if (c < (int)ldo) {
      Eight w;
      if (c + 8 <= cols) {
        __builtin_memcpy(&w, row + c, sizeof(w));
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) w.v[e] = c + e < cols ? row[c + e] : TI(0);
      }
      if constexpr (sizeof(TO) == 4) {
#pragma unroll
        for (int e = 0; e < 8; e += 4) *reinterpret_cast<floatx4*>(to + c + e) = floatx4{w.v[e], w.v[e + 1], w.v[e + 2], w.v[e + 3]};
      } else if constexpr (sizeof(TI) == 4) {
        *reinterpret_cast<u32x4*>(to + c) = u32x4{pack_bf16(w.v[0], w.v[1]), pack_bf16(w.v[2], w.v[3]), pack_bf16(w.v[4], w.v[5]), pack_bf16(w.v[6], w.v[7])};
      } else {
        *reinterpret_cast<u32x4*>(to + c) = __builtin_bit_cast(u32x4, w);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// operands kept in 8 bits
// ---------------------------------------------------------------------------
// Rows quantised in blocks of 128 columns (e4m3) to T: exactly, an 8-bit value
// times a power of two is a bfloat16 number (unless it leaves that type's
// range).  A thread takes 16 columns; zeros behind `cols` up to ldo.  Bound by
// memory: 8192 x 4096 (101 MB) 20.8 us = 4.8 TB/s, beside products of a millisecond.
template <typename T>
__global__ __launch_bounds__(256) void widen_rows_kernel(const uint8_t* __restrict__ q, const uint8_t* __restrict__ s, int64_t ldq, int64_t lds,
                                                         int64_t rows, int cols, T* __restrict__ o, int64_t ldo) {
  const int per = (int)((ldo + 15) / 16);
  const int64_t total = rows * per;
  for (int64_t i = blockIdx.x * (int64_t)256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t r = i / per;
    const int c = (int)(i - r * per) * 16;
    const u32x4 w = *reinterpret_cast<const u32x4*>(q + r * ldq + c);
    const float scale = scale_value(s[r * lds + (c >> 7)]);
    float v[16];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const floatx2 lo = __builtin_amdgcn_cvt_pk_f32_fp8(w[k], false), hi = __builtin_amdgcn_cvt_pk_f32_fp8(w[k], true);
      v[4 * k] = lo[0] * scale;
      v[4 * k + 1] = lo[1] * scale;
      v[4 * k + 2] = hi[0] * scale;
      v[4 * k + 3] = hi[1] * scale;
    }
    if (c + 16 > cols) {
#pragma unroll
      for (int e = 0; e < 16; ++e)
        if (c + e >= cols) v[e] = 0.f;
    }
    T* to = o + r * ldo + c;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (c + 8 * k >= ldo) break;  // rows of a multiple of 8
      if constexpr (sizeof(T) == 2) {
        *reinterpret_cast<u32x4*>(to + 8 * k) = u32x4{pack_bf16(v[8 * k], v[8 * k + 1]), pack_bf16(v[8 * k + 2], v[8 * k + 3]),
                                                      pack_bf16(v[8 * k + 4], v[8 * k + 5]), pack_bf16(v[8 * k + 6], v[8 * k + 7])};
      } else {
        *reinterpret_cast<floatx4*>(to + 8 * k) = floatx4{v[8 * k], v[8 * k + 1], v[8 * k + 2], v[8 * k + 3]};
        *reinterpret_cast<floatx4*>(to + 8 * k + 4) = floatx4{v[8 * k + 4], v[8 * k + 5], v[8 * k + 6], v[8 * k + 7]};
      }
    }
  }
}

}  // namespace shampoo
