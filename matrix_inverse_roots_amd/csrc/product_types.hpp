// Types and arguments of the rectangular product (product_core.hpp) and of its
// epilogues.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gemm_common.hpp"

namespace shampoo {

typedef float floatx16 __attribute__((ext_vector_type(16)));
typedef int intx8 __attribute__((ext_vector_type(8)));
typedef short shortx4_t __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef float floatx2 __attribute__((ext_vector_type(2)));

// 16 and 8 bytes at an element's address: one access wherever it lies.
typedef u32x4 u32x4_any __attribute__((aligned(2)));
typedef u32x2 u32x2_any __attribute__((aligned(2)));
typedef floatx4 floatx4_any __attribute__((aligned(4)));

enum class Elem { BF16, F32, F8, F8W };
// What becomes of a tile.  STORE: C = alpha acc + beta C.  STORE2: the same, B's
// rows of k continued in a second matrix.  SOFTMAX: the projection's loss.
// LINEAR, GATED, GATED_GRAD: the feed-forward layers (ffn_epilogue.hpp); GATED
// takes two matrices B1, B2 and finds both products of a column in one lane.
enum class Epi { STORE, STORE2, SOFTMAX, LINEAR, GATED, GATED_GRAD };

// Epilogues of the feed-forward layers.
struct FfnArgs {
  const void* bias;       // LINEAR: [N] or null
  const void* residual;   // LINEAR: rows of N in C's type, or null
  int64_t ld_residual;
  // z (LINEAR) or g and u: written by LINEAR and GATED (null: not), read by GATED_GRAD
  void* keep[2];
  uint8_t* keep_scale[2];
  int64_t ld_keep;        // elements; 8 bits: N rounded up to 32
  float* part;            // GATED with ranges of k: partial results [range][M][2 P], P: N rounded up to 4
  void* du;               // GATED_GRAD: rows of ldc (C receives dg)
  void* h;                // GATED_GRAD: rows of ldc / 2
  int bias_bf16, act, keep_dt, scale_vec;  // keep_dt: 0 float32, 2 bfloat16, 4 e4m3; scale_vec: rows of scales start on 4 bytes
};

struct ProductArgs {
  const void* A;
  const void* B;
  const uint8_t* sa;  // F8: scales, [rows >> sa_shift][ldsa] bytes, 4-byte aligned rows
  const uint8_t* sb;
  void* C;            // STORE: float32, bfloat16 or half by c_dt; SOFTMAX: exponentials (may be null)
  int64_t lda, ldb, ldc;              // elements
  int64_t strideA, strideB, strideC;  // elements between the matrices of a batch
  int64_t ldsa, ldsb, strideSa, strideSb;
  int64_t split_stride;               // STORE: elements between the partial results of two k-ranges
  int M, N, K;
  int sa_shift, sb_shift;             // 0: a scale per row; 7: per 128 rows
  int mt, nt;                         // tiles along M and N
  int nst;                            // k-stages of 128 bytes
  int splits, split_stages;           // ranges of k; stages of each but the last (F8: a multiple of 4)
  int c_dt;                           // 0 float32, 1 half, 2 bfloat16
  int vec;                            // whole runs of C in 16-byte accesses
  float alpha, beta;                  // STORE: C = alpha acc + beta C
  const float* alpha_dev;             // times this, or null
  int64_t items;                      // batch * splits * mt * nt
  // SOFTMAX
  floatx2* stats;                     // [pieces][M]: (max, sum of exp(z - max)) of 128 columns
  const int64_t* targets;             // [M]
  float* target_logit;                // [M]: the logit at each row's target, where that is a column
  // STORE2, GATED
  const void* B2;                     // rows of ldb
  int kswitch, kpart;                 // STORE2: B2 begins with this stage; k of either matrix
  FfnArgs ffn;
};

template <Elem E> struct ElemTraits;
template <> struct ElemTraits<Elem::BF16> { static constexpr int size = 2; };
template <> struct ElemTraits<Elem::F32> { static constexpr int size = 4; };
template <> struct ElemTraits<Elem::F8> { static constexpr int size = 1; };
template <> struct ElemTraits<Elem::F8W> { static constexpr int size = 1; };

// By value: __builtin_bit_cast of a vector's element reads element 0.
__device__ __forceinline__ float bits_float(uint32_t b) { return __builtin_bit_cast(float, b); }
__device__ __forceinline__ uint32_t float_bits(float f) { return __builtin_bit_cast(uint32_t, f); }

__device__ __forceinline__ uint32_t pack_bf16(float x, float y) {
  typedef __bf16 b2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, b2{(__bf16)x, (__bf16)y});
}
__device__ __forceinline__ uint32_t pack_f16(float x, float y) {
  typedef _Float16 h2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, h2{(_Float16)x, (_Float16)y});
}

}  // namespace shampoo
