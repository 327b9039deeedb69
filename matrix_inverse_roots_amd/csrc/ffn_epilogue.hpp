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
// What bounds them: one workgroup holds a unit's LDS, so a tile's epilogue and
// products take turns, and every instruction and byte here shows.  8191 x 4096
// x 1024 with gelu and z in 8 bits: 108 us, of which 26% of the cycles are the
// matrix cores', 35% this arithmetic (some 35 instructions an element), the rest
// waits; without activation and kept values the product takes 81.  8192 x 10240 x
// 4096 with the gated block's gradients from 8 bits: 810-830 us against 533 for
// the product alone, for 168 MB read, 503 MB written and the arithmetic.
// Blocks are done one after another (apart()), what was kept of the next one
// loaded ahead: all at once they spilled up to 300 registers, which cost the
// gated block's gradients 8%.  Now none spills but 8 in GATED_GRAD's 256 x 256
// tile of bfloat16 (36 bytes of scratch a lane).
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

template <int ES> struct KeptType;
template <> struct KeptType<2> { typedef uint16_t type; };
template <> struct KeptType<4> { typedef float type; };

// f(0), f(1), ... f(N - 1) with constants: the blocks' loop bodies are too large
// for the compiler to unroll them, and a block indexed at run time would put the
// tile's results into scratch memory.
template <int I> struct Index { static constexpr int value = I; };
template <int N, int I = 0, typename F> __device__ __forceinline__ void for_each(F f) {
  if constexpr (I < N) {
    f(Index<I>{});
    for_each<N, I + 1>(f);
  }
}

// Nothing in memory moves over it: the loads of several blocks at a time would
// not fit the registers beside a tile's results.
__device__ __forceinline__ void apart() { asm volatile("" ::: "memory"); }

// A 32 x 32 block from column nb on, of a row: `row` is where the lane's row
// starts, `ok` whether it is one, `cols` where the rows end.  Accesses are 16
// bytes wherever rows start; only a block over the rows' end goes by elements.
__device__ __forceinline__ floatx16 load_block(const float* row, bool ok, int nb, int half, int cols) {
  floatx16 r;
  if (nb + 32 <= cols) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const floatx4 v = ok ? *reinterpret_cast<const floatx4_any*>(row + nb + 8 * q + 4 * half) : floatx4{0.f, 0.f, 0.f, 0.f};
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
__device__ __forceinline__ floatx16 load_block(const uint16_t* row, bool ok, int nb, int half, int cols) {
  floatx16 r;
  auto put = [&](int v, uint32_t two) {
    r[v] = bits_float(two << 16);
    r[v + 1] = bits_float(two & 0xffff0000u);
  };
  if (nb + 32 <= cols) {
    // 8 columns a lane; the halves of the wave swap 4 of them
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const u32x4 w = ok ? *reinterpret_cast<const u32x4_any*>(row + nb + 16 * q + 8 * half) : u32x4{0, 0, 0, 0};
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

// FULL: the whole block lies within the rows.
template <bool FULL = false>
__device__ __forceinline__ void store_block(float* row, bool ok, int nb, int half, int cols, const floatx16& x) {
  if (!ok) return;
  if (FULL || nb + 32 <= cols) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      *reinterpret_cast<floatx4_any*>(row + nb + 8 * q + 4 * half) = floatx4{x[4 * q], x[4 * q + 1], x[4 * q + 2], x[4 * q + 3]};
  } else {
#pragma unroll
    for (int v = 0; v < 16; ++v) {
      const int n = nb + 8 * (v >> 2) + 4 * half + (v & 3);
      if (n < cols) row[n] = x[v];
    }
  }
}
template <bool FULL = false>
__device__ __forceinline__ void store_block(uint16_t* row, bool ok, int nb, int half, int cols, const floatx16& x) {
  uint32_t two[8];
#pragma unroll
  for (int v = 0; v < 8; ++v) two[v] = pack_bf16(x[2 * v], x[2 * v + 1]);
  if (FULL || nb + 32 <= cols) {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const auto a = __builtin_amdgcn_permlane32_swap(two[4 * q], two[4 * q + 2], false, false);
      const auto b = __builtin_amdgcn_permlane32_swap(two[4 * q + 1], two[4 * q + 3], false, false);
      if (ok) *reinterpret_cast<u32x4_any*>(row + nb + 16 * q + 8 * half) = u32x4{a[0], b[0], a[1], b[1]};
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
__device__ __forceinline__ floatx16 load_rows(const void* p, int dt, int64_t ld, int m, bool ok, int nb, int half, int cols) {
  if (dt == 0) return load_block(reinterpret_cast<const float*>(p) + m * ld, ok, nb, half, cols);
  return load_block(reinterpret_cast<const uint16_t*>(p) + m * ld, ok, nb, half, cols);
}
__device__ __forceinline__ void store_rows(void* p, int dt, int64_t ld, int m, bool ok, int nb, int half, int cols, const floatx16& x) {
  if (dt == 0) store_block(reinterpret_cast<float*>(p) + m * ld, ok, nb, half, cols, x);
  else store_block(reinterpret_cast<uint16_t*>(p) + m * ld, ok, nb, half, cols, x);
}

// 2^(byte - 127), byte 0 included
__device__ __forceinline__ float scale_value(uint32_t byte) { return bits_float(byte ? byte << 23 : 0x00400000u); }

// Largest finite magnitude's bits among 16 values of this lane and of its
// partner in the other half of the wave.  The maximum passes over NaN by
// itself; a wave that meets an infinity filters.
__device__ __forceinline__ uint32_t block_max(const floatx16& x) {
  float f = 0.f;
#pragma unroll
  for (int v = 0; v < 16; ++v) f = fmaxf(f, fabsf(x[v]));
  uint32_t a = float_bits(f);
  if (__any(a >= 0x7f800000u)) {
    a = 0;
#pragma unroll
    for (int v = 0; v < 16; ++v) a = max(a, finite_bits(x[v]));
  }
  const auto s = __builtin_amdgcn_permlane32_swap(a, a, false, false);
  return max(s[0], s[1]);
}

// A block to 8 bits: 16 bytes a lane, the first half of the wave the first 16
// columns; rows of `ld` bytes (cols rounded up to 32); columns past `cols`
// become zeros.  Returns the scale's byte, which store_scales takes.
__device__ __forceinline__ uint32_t keep_f8(uint8_t* q, int64_t ld, int m, bool ok, int nb, int half, int cols, floatx16 x) {
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
  if (ok && nb < cols) *reinterpret_cast<u32x4*>(q + m * ld + nb + 16 * half) = u32x4{a[0], a[1], b[0], b[1]};
  return (uint32_t)byte;
}
__device__ __forceinline__ uint32_t keep_block(const FfnArgs& e, int which, int m, bool ok, int nb, int half, int cols, const floatx16& x) {
  if (e.keep_dt == 4) return keep_f8((uint8_t*)e.keep[which], e.ld_keep, m, ok, nb, half, cols, x);
  store_rows(e.keep[which], e.keep_dt, e.ld_keep, m, ok, nb, half, cols, x);
  return 0;
}

// The scales of COUNT neighbouring blocks of a row, a byte each of `word`, in one
// store (a byte for each block at a time was half of all the epilogue's line
// accesses).
template <int COUNT> __device__ __forceinline__ void store_scales(const FfnArgs& e, int which, int m, bool ok, int n0, int cols, uint32_t word) {
  if (!ok) return;
  uint8_t* s = e.keep_scale[which] + m * (e.ld_keep / KEEP_BLOCK) + n0 / KEEP_BLOCK;
  if (COUNT > 1 && e.scale_vec && n0 + COUNT * KEEP_BLOCK <= cols) {
    if constexpr (COUNT == 4) *reinterpret_cast<uint32_t*>(s) = word;
    else if constexpr (COUNT == 2) *reinterpret_cast<uint16_t*>(s) = (uint16_t)word;
  } else {
#pragma unroll
    for (int c = 0; c < COUNT; ++c)
      if (n0 + c * KEEP_BLOCK < cols) s[c] = (uint8_t)(word >> (8 * c));
  }
}
template <int COUNT> __device__ __forceinline__ uint32_t load_scales(const FfnArgs& e, int which, int m, bool ok, int n0, int cols) {
  uint32_t word = 0x7f7f7f7fu;
  if (!ok) return word;
  const uint8_t* s = e.keep_scale[which] + m * (e.ld_keep / KEEP_BLOCK) + n0 / KEEP_BLOCK;
  if (COUNT > 1 && e.scale_vec && n0 + COUNT * KEEP_BLOCK <= cols) {
    if constexpr (COUNT == 4) word = *reinterpret_cast<const uint32_t*>(s);
    else if constexpr (COUNT == 2) word = *reinterpret_cast<const uint16_t*>(s);
  } else {
    word = 0;
#pragma unroll
    for (int c = 0; c < COUNT; ++c) word |= (n0 + c * KEEP_BLOCK < cols ? (uint32_t)s[c] : 127u) << (8 * c);
  }
  return word;
}

// Half a block (values 8 q to 8 q + 7 of the lane, columns 16 q to 16 q + 15 of the
// block): what an epilogue holds beside a tile's results and the next tile's
// first fragments.
struct Half {
  float v[8];
};
__device__ __forceinline__ Half load_half(const float* row, bool ok, int n0, int half, int cols) {
  Half r;
  if (n0 + 16 <= cols) {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const floatx4 w = ok ? *reinterpret_cast<const floatx4_any*>(row + n0 + 8 * q + 4 * half) : floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int e = 0; e < 4; ++e) r.v[4 * q + e] = w[e];
    }
  } else {
#pragma unroll
    for (int v = 0; v < 8; ++v) {
      const int n = n0 + 8 * (v >> 2) + 4 * half + (v & 3);
      r.v[v] = ok && n < cols ? row[n] : 0.f;
    }
  }
  return r;
}
__device__ __forceinline__ Half load_half(const uint16_t* row, bool ok, int n0, int half, int cols) {
  Half r;
  if (n0 + 16 <= cols) {
    const u32x4 w = ok ? *reinterpret_cast<const u32x4_any*>(row + n0 + 8 * half) : u32x4{0, 0, 0, 0};
    const auto a = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
    const auto b = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
    const uint32_t two[4] = {a[0], b[0], a[1], b[1]};
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      r.v[2 * v] = bits_float(two[v] << 16);
      r.v[2 * v + 1] = bits_float(two[v] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int v = 0; v < 8; ++v) {
      const int n = n0 + 8 * (v >> 2) + 4 * half + (v & 3);
      r.v[v] = ok && n < cols ? bits_float((uint32_t)row[n] << 16) : 0.f;
    }
  }
  return r;
}
// wholly within rows that start on 16 bytes
__device__ __forceinline__ void store_half(float* row, bool ok, int n0, int half, const Half& x) {
  if (!ok) return;
#pragma unroll
  for (int q = 0; q < 2; ++q)
    *reinterpret_cast<floatx4*>(row + n0 + 8 * q + 4 * half) = floatx4{x.v[4 * q], x.v[4 * q + 1], x.v[4 * q + 2], x.v[4 * q + 3]};
}
__device__ __forceinline__ void store_half(uint16_t* row, bool ok, int n0, int half, const Half& x) {
  const auto a = __builtin_amdgcn_permlane32_swap(pack_bf16(x.v[0], x.v[1]), pack_bf16(x.v[4], x.v[5]), false, false);
  const auto b = __builtin_amdgcn_permlane32_swap(pack_bf16(x.v[2], x.v[3]), pack_bf16(x.v[6], x.v[7]), false, false);
  if (ok) *reinterpret_cast<u32x4*>(row + n0 + 8 * half) = u32x4{a[0], b[0], a[1], b[1]};
}

// A kept block in 8 bits, as it lies in memory, and its values 8 q to 8 q + 7.
struct KeptF8 {
  u32x4 w;
  uint32_t byte;
  __device__ __forceinline__ void load(const FfnArgs& e, int which, int m, bool ok, int nb, int half, int cols, uint32_t scale) {
    w = u32x4{0, 0, 0, 0};
    byte = scale;
    if (ok && nb < cols) w = *reinterpret_cast<const u32x4*>((const uint8_t*)e.keep[which] + m * e.ld_keep + nb + 16 * half);
  }
  __device__ __forceinline__ void swap() {
    const auto a = __builtin_amdgcn_permlane32_swap(w[0], w[1], false, false);
    const auto b = __builtin_amdgcn_permlane32_swap(w[2], w[3], false, false);
    w = u32x4{a[0], b[0], a[1], b[1]};
  }
  __device__ __forceinline__ Half values(int q) const {
    const float scale = scale_value(byte);
    Half r;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t four = i == 0 ? (q == 0 ? w[0] : w[2]) : (q == 0 ? w[1] : w[3]);
      const floatx2 lo = __builtin_amdgcn_cvt_pk_f32_fp8(four, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8(four, true);
      r.v[4 * i] = lo[0] * scale;
      r.v[4 * i + 1] = lo[1] * scale;
      r.v[4 * i + 2] = hi[0] * scale;
      r.v[4 * i + 3] = hi[1] * scale;
    }
    return r;
  }
};

// Loads that a block's epilogue will need, issued a block ahead: blocks of
// bfloat16 rows, wholly inside.
struct Ahead {
  u32x4 w[2];
  __device__ __forceinline__ void load(const uint16_t* row, bool ok, int nb, int half) {
#pragma unroll
    for (int q = 0; q < 2; ++q) w[q] = ok ? *reinterpret_cast<const u32x4_any*>(row + nb + 16 * q + 8 * half) : u32x4{0, 0, 0, 0};
  }
  __device__ __forceinline__ Half values(int q) const {
    const auto a = __builtin_amdgcn_permlane32_swap(w[q][0], w[q][2], false, false);
    const auto b = __builtin_amdgcn_permlane32_swap(w[q][1], w[q][3], false, false);
    const uint32_t two[4] = {a[0], b[0], a[1], b[1]};
    Half r;
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      r.v[2 * v] = bits_float(two[v] << 16);
      r.v[2 * v + 1] = bits_float(two[v] & 0xffff0000u);
    }
    return r;
  }
};

__device__ __forceinline__ floatx16 bias_block(const FfnArgs& e, int nb, int half, int cols) {
  floatx16 b;
  if (nb + 32 <= cols) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int n = nb + 8 * q + 4 * half;
      if (e.bias_bf16) {
        const u32x2 w = *reinterpret_cast<const u32x2_any*>(reinterpret_cast<const uint16_t*>(e.bias) + n);
#pragma unroll
        for (int c = 0; c < 4; ++c) b[4 * q + c] = bits_float(c & 1 ? w[c >> 1] & 0xffff0000u : w[c >> 1] << 16);
      } else {
        const floatx4 w = *reinterpret_cast<const floatx4_any*>(reinterpret_cast<const float*>(e.bias) + n);
#pragma unroll
        for (int c = 0; c < 4; ++c) b[4 * q + c] = w[c];
      }
    }
  } else {
#pragma unroll
    for (int v = 0; v < 16; ++v) {
      const int n = min(nb + 8 * (v >> 2) + 4 * half + (v & 3), cols - 1);
      b[v] = e.bias_bf16 ? bits_float((uint32_t)reinterpret_cast<const uint16_t*>(e.bias)[n] << 16) : reinterpret_cast<const float*>(e.bias)[n];
    }
  }
  return b;
}

template <int FM, int FN>
__device__ __forceinline__ void linear_epilogue(const ProductArgs& g, floatx16 (&acc)[FM][FN], int m0, int n0, int l32, int half) {
  const FfnArgs& e = g.ffn;
  const bool early = e.residual && g.c_dt == 2 && n0 + 32 * FN <= g.N;
  const auto residual_row = [&](int i) __attribute__((always_inline)) {
    return reinterpret_cast<const uint16_t*>(e.residual) + (m0 + 32 * i + l32) * e.ld_residual;
  };
  Ahead next;
  if (early) next.load(residual_row(0), m0 + l32 < g.M, n0, half);
  uint32_t scales[FM] = {};
  for_each<FN>([&](auto J) __attribute__((always_inline)) {
    const int nb = n0 + 32 * J.value;
    if (nb >= g.N) return;
    apart();
    floatx16 b;
    if (e.bias) b = bias_block(e, nb, half, g.N);
    for_each<FM>([&](auto I) __attribute__((always_inline)) {
      const int m = m0 + 32 * I.value + l32;
      const bool ok = m < g.M;
      apart();
      const Ahead now = next;
      if (early && !(I.value == FM - 1 && J.value == FN - 1)) {
        constexpr int i = I.value == FM - 1 ? 0 : I.value + 1, j = I.value == FM - 1 ? J.value + 1 : J.value;
        next.load(residual_row(i), m0 + 32 * i + l32 < g.M, n0 + 32 * j, half);
      }
      apart();
      floatx16 z = acc[I.value][J.value];
      if (e.bias) {
#pragma unroll
        for (int v = 0; v < 16; ++v) z[v] += b[v];
      }
      if (e.keep[0]) scales[I.value] |= keep_block(e, 0, m, ok, nb, half, g.N, z) << (8 * J.value);
      if (e.act) {
        with_activation(e.act, [&](auto act) __attribute__((always_inline)) {
#pragma unroll
          for (int v = 0; v < 16; ++v) z[v] = act.value(z[v]);
        });
      }
      if (early) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const Half r = now.values(q);
#pragma unroll
          for (int v = 0; v < 8; ++v) z[8 * q + v] += r.v[v];
        }
      } else if (e.residual) {
        const floatx16 r = load_rows(e.residual, g.c_dt, e.ld_residual, m, ok, nb, half, g.N);
#pragma unroll
        for (int v = 0; v < 16; ++v) z[v] += r[v];
      }
      store_rows(g.C, g.c_dt, g.ldc, m, ok, nb, half, g.N, z);
    });
  });
  if (e.keep[0] && e.keep_dt == 4) {
#pragma unroll
    for (int i = 0; i < FM; ++i) store_scales<FN>(e, 0, m0 + 32 * i + l32, m0 + 32 * i + l32 < g.M && half == 0, n0, g.N, scales[i]);
  }
}

// C receives h: rows of ldc, zeros behind the columns.  Blocks j and j + FN / 2
// are the same columns of the gate and of the up projection.
template <int FM, int FN>
__device__ __forceinline__ void gated_epilogue(const ProductArgs& g, floatx16 (&acc)[FM][FN], int m0, int n0, int l32, int half, int range) {
  constexpr int HF = FN / 2;
  const FfnArgs& e = g.ffn;
  if (g.splits > 1) {
    const int P = (g.N + 3) & ~3;
    float* part = e.part + (int64_t)range * g.M * 2 * P;
    for_each<FM * FN>([&](auto K) __attribute__((always_inline)) {
      constexpr int I = K.value / FN, J = K.value % FN;
      const int m = m0 + 32 * I + l32;
      store_block(part + m * (int64_t)(2 * P) + J / HF * P, m < g.M, n0 + 32 * (J % HF), half, g.N, acc[I][J]);
    });
    return;
  }
  uint32_t scales[FM][2] = {};
  for_each<FM * HF>([&](auto K) __attribute__((always_inline)) {
    constexpr int I = K.value / HF, J = K.value % HF;
    const int m = m0 + 32 * I + l32, nb = n0 + 32 * J;
    const bool ok = m < g.M;
    if (nb >= g.ldc) return;
    apart();
    floatx16 h = acc[I][J];
    const floatx16 up = acc[I][J + HF];
    if (e.keep[0]) {
      scales[I][0] |= keep_block(e, 0, m, ok, nb, half, g.N, h) << (8 * J);
      scales[I][1] |= keep_block(e, 1, m, ok, nb, half, g.N, up) << (8 * J);
    }
    with_activation(e.act, [&](auto act) __attribute__((always_inline)) {
#pragma unroll
      for (int v = 0; v < 16; ++v) h[v] = act.value(h[v]) * up[v];
    });
    if (nb + 32 > g.N) {
#pragma unroll
      for (int v = 0; v < 16; ++v)
        if (nb + 8 * (v >> 2) + 4 * half + (v & 3) >= g.N) h[v] = 0.f;
    }
    if (g.c_dt == 0) store_block<true>(reinterpret_cast<float*>(g.C) + m * g.ldc, ok, nb, half, 0, h);
    else store_block<true>(reinterpret_cast<uint16_t*>(g.C) + m * g.ldc, ok, nb, half, 0, h);
  });
  if (e.keep[0] && e.keep_dt == 4) {
#pragma unroll
    for (int i = 0; i < FM; ++i)  // the gate's from one half of the wave, the up projection's from the other
      store_scales<HF>(e, half, m0 + 32 * i + l32, m0 + 32 * i + l32 < g.M, n0, g.N, half ? scales[i][1] : scales[i][0]);
  }
}

// ES: bytes of an element of dg, du (rows of ldc) and h (rows of ldc / 2), zeros behind the columns
template <int FM, int FN, int ES>
__device__ __forceinline__ void gated_grad_epilogue(const ProductArgs& g, floatx16 (&acc)[FM][FN], int m0, int n0, int l32, int half) {
  using T = typename KeptType<ES>::type;
  const FfnArgs& e = g.ffn;
  const int wide = (int)(g.ldc / 2);
  const bool f8 = e.keep_dt == 4;
  // what was kept of the next block is loaded before this one is computed
  const bool early = ES == 2 && !f8 && n0 + 32 * FN <= g.N;
  uint32_t scales[FM][2];
  if (f8) {
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int p = 0; p < 2; ++p) scales[i][p] = load_scales<FN>(e, p, m0 + 32 * i + l32, m0 + 32 * i + l32 < g.M, n0, g.N);
  }
  KeptF8 next8[2];
  Ahead next[2];
  const auto load = [&](int i, int j) __attribute__((always_inline)) {
    const int m = m0 + 32 * i + l32, nb = n0 + 32 * j;
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      if (f8) next8[p].load(e, p, m, m < g.M, nb, half, g.N, scales[i][p] >> (8 * j) & 255);
      else if (early) next[p].load(reinterpret_cast<const uint16_t*>(e.keep[p]) + m * e.ld_keep, m < g.M, nb, half);
    }
  };
  load(0, 0);
  for_each<FM * FN>([&](auto K) __attribute__((always_inline)) {
    constexpr int I = K.value / FN, J = K.value % FN;
    const int m = m0 + 32 * I + l32, nb = n0 + 32 * J;
    const bool ok = m < g.M;
    apart();
    KeptF8 gate8 = next8[0], up8 = next8[1];
    const Ahead gate16 = next[0], up16 = next[1];
    if constexpr (K.value + 1 < FM * FN) load((K.value + 1) / FN, (K.value + 1) % FN);
    if (nb >= wide) return;
    if (f8) {
      gate8.swap();
      up8.swap();
    }
    for_each<2>([&](auto Q) __attribute__((always_inline)) {
      constexpr int q = Q.value;
      const int n = nb + 16 * q;
      apart();
      Half gate, up, h;
      if (f8) {
        gate = gate8.values(q);
        up = up8.values(q);
      } else if (early) {
        gate = gate16.values(q);
        up = up16.values(q);
      } else {
        gate = load_half(reinterpret_cast<const T*>(e.keep[0]) + m * e.ld_keep, ok, n, half, g.N);
        up = load_half(reinterpret_cast<const T*>(e.keep[1]) + m * e.ld_keep, ok, n, half, g.N);
      }
      // gate becomes dg, up du
      with_activation(e.act, [&](auto act) __attribute__((always_inline)) {
#pragma unroll
        for (int v = 0; v < 8; ++v) {
          float slope;
          const float a = act.both(gate.v[v], slope), dh = acc[I][J][8 * q + v];
          h.v[v] = a * up.v[v];
          gate.v[v] = dh * up.v[v] * slope;
          up.v[v] = dh * a;
        }
      });
      if (n + 16 > g.N) {
#pragma unroll
        for (int v = 0; v < 8; ++v)
          if (n + 8 * (v >> 2) + 4 * half + (v & 3) >= g.N) h.v[v] = gate.v[v] = up.v[v] = 0.f;
      }
      store_half(reinterpret_cast<T*>(g.C) + m * g.ldc, ok, n, half, gate);
      store_half(reinterpret_cast<T*>(e.du) + m * g.ldc, ok, n, half, up);
      store_half(reinterpret_cast<T*>(e.h) + m * (int64_t)wide, ok, n, half, h);
    });
  });
}

}  // namespace shampoo
