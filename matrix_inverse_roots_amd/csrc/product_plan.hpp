// Host side of product_core.hpp, shared by the translation units that launch
// it: checks of a call's memory, tile and split plans, launches.
#pragma once

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "host_common.hpp"
#include "product_core.hpp"
#include "product_passes.hpp"
#include "product_shapes.hpp"
#include "shampoo.h"

namespace shampoo {

inline bool aligned(const void* p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
inline size_t size_of(int dt) { return dt == SHAMPOO_F32 ? 4 : dt == SHAMPOO_E4M3 || dt == SHAMPOO_E5M2 ? 1 : 2; }

// Memory of a call: `rows` of `width` bytes, `apart` bytes from one to the next.
struct Span {
  const char* name;
  const void* p;
  int64_t rows, width, apart;
};
inline Span run_of(const char* name, const void* p, int64_t bytes) { return {name, p, 1, bytes, bytes}; }
inline Span rows_of(const char* name, const void* p, int64_t rows, int64_t cols, int64_t ld, int dt) {
  const int64_t es = (int64_t)size_of(dt);
  return {name, p, rows, cols * es, rows > 1 ? ld * es : cols * es};
}
// Rows of the same distance may lie between one another (views of one wider
// matrix); otherwise the spans' whole extents count.
inline bool overlap(const Span& a, const Span& b) {
  if (!a.p || !b.p || a.rows <= 0 || b.rows <= 0 || a.width <= 0 || b.width <= 0) return false;
  const uintptr_t pa = (uintptr_t)a.p, pb = (uintptr_t)b.p;
  const uintptr_t ea = pa + (uintptr_t)((a.rows - 1) * a.apart + a.width), eb = pb + (uintptr_t)((b.rows - 1) * b.apart + b.width);
  if (ea <= pb || eb <= pa) return false;
  if (a.rows > 1 && b.rows > 1 && a.apart != b.apart) return true;
  const int64_t apart = a.rows > 1 ? a.apart : b.apart;
  const int64_t at = pb >= pa ? (int64_t)((pb - pa) % (uintptr_t)apart) : (apart - (int64_t)((pa - pb) % (uintptr_t)apart)) % apart;
  return at < a.width || at + b.width > apart;
}
// What a call writes (the first `written` spans) may overlap nothing else of it.
template <size_t COUNT> shampoo_status check_apart(const Span (&spans)[COUNT], size_t written) {
  for (size_t i = 0; i < written; ++i)
    for (size_t j = i + 1; j < COUNT; ++j)
      if (overlap(spans[i], spans[j])) return fail(SHAMPOO_E_INVALID, "%s overlaps %s", spans[i].name, spans[j].name);
  return SHAMPOO_OK;
}

// ---------------------------------------------------------------------------
// products
// ---------------------------------------------------------------------------
template <Elem E, int FM, int FN, int WM, int WN, int NB, int PER_CU, bool AS, bool BS, Epi EPI, int FA, int FB>
hipError_t launch_tiles(ProductArgs g, int64_t batch, hipStream_t st) {
  constexpr int TM = 32 * FM * WM, TN = 32 * FN * WN;
  constexpr int LDS = NB * (TM + TN) * 128 +  // stages, groups of scales, groups of targets
                      4 * scale_groups(NB) * ((E == Elem::F8 || E == Elem::F8W ? TM + TN : 0) + (EPI == Epi::SOFTMAX ? TM : 0));
  const auto kernel = product_kernel<E, FM, FN, WM, WN, NB, AS, BS, EPI, FA, FB>;
  static bool ready[MAX_DEVICES] = {false};
  int dev = 0, cus = 0;
  HIP_TRY_ERR(hipGetDevice(&dev));
  if (!(dev >= 0 && dev < MAX_DEVICES && ready[dev])) {
    HIP_TRY_ERR(hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, LDS));
    if (dev >= 0 && dev < MAX_DEVICES) ready[dev] = true;
  }
  HIP_TRY_ERR(cu_count(&cus));
  g.mt = (g.M + TM - 1) / TM;
  constexpr int TNO = EPI == Epi::GATED ? TN / 2 : TN;
  g.nt = (g.N + TNO - 1) / TNO;
  g.items = batch * g.splits * (int64_t)g.mt * g.nt;
  const int64_t grid = std::min<int64_t>(up(g.items, 8), std::max(8, cus * PER_CU / 8 * 8));
  hipLaunchKernelGGL(kernel, dim3((unsigned)grid), dim3(64 * WM * WN), LDS, st, g);
  return hipGetLastError();
}

template <Elem E, bool AS, bool BS, Epi EPI, int FA = 0, int FB = 0>
hipError_t launch_product(const ProductArgs& g, bool large, int64_t batch, hipStream_t st) {
  if (large) return launch_tiles<E, 2, 4, 4, 2, 2, 1, AS, BS, EPI, FA, FB>(g, batch, st);
  const int64_t items = batch * g.splits * ((g.M + 127) / 128) * ((g.N + 127) / 128);
  if (items <= CUS) return launch_tiles<E, 1, 4, 4, 1, 4, 1, AS, BS, EPI, FA, FB>(g, batch, st);
  return launch_tiles<E, 1, 4, 4, 1, 2, 2, AS, BS, EPI, FA, FB>(g, batch, st);
}

// A feed-forward layer's product on the tile that its plan chose.  Only the
// tiles that some plan reaches are built: float32 has no 256 x 128, GATED none of
// 64 x 64 (it needs two fragments of columns), and a forward product over ranges of
// k (STORE without strided operands), which has few tiles, no large ones.
template <Elem E, bool AS, bool BS, Epi EPI>
hipError_t launch_layer(const ProductArgs& g, const Shape& s, int64_t batch, hipStream_t st) {
  constexpr bool RANGES_ONLY = EPI == Epi::STORE && !AS && !BS;
  if constexpr (E == Elem::F32 && EPI != Epi::GATED) {
    if (s.tile == TILE_64) return launch_tiles<E, 1, 1, 2, 2, 3, 3, AS, BS, EPI, 0, 0>(g, batch, st);
  }
  if constexpr (!RANGES_ONLY) {
    if constexpr (E == Elem::BF16) {
      if (s.tile == TILE_MEDIUM) return launch_tiles<E, 2, 2, 4, 2, 3, 1, AS, BS, EPI, 0, 0>(g, batch, st);
    }
    if (s.tile == TILE_LARGE) return launch_tiles<E, 2, 4, 4, 2, 2, 1, AS, BS, EPI, 0, 0>(g, batch, st);
    if (s.tile == TILE_128_TWO) return launch_tiles<E, 1, 4, 4, 1, 2, 2, AS, BS, EPI, 0, 0>(g, batch, st);
  }
  if (s.tile == TILE_128) return launch_tiles<E, 1, 4, 4, 1, 4, 1, AS, BS, EPI, 0, 0>(g, batch, st);
  return hipErrorInvalidValue;
}

inline void set_shape(ProductArgs& g, const Shape& s) {
  g.nst = s.nst;
  g.splits = s.splits;
  g.split_stages = s.split_stages;
}

inline size_t partial_bytes(const Shape& s, int64_t batch, int64_t M, int64_t N) {
  return s.splits > 1 ? align_up((size_t)s.splits * batch * M * N * 4) : 0;
}

// Points a split product at its partial results; finish_split sums them.
struct Out {
  void* C;
  int64_t ldc, strideC;
  int c_dt, vec;
  float beta;
  float alpha = 1.f;
  const float* alpha_dev = nullptr;
};
inline void point_output(ProductArgs& g, const Shape& s, const Out& o, float* part, int64_t batch) {
  if (s.splits > 1) {
    g.C = part;
    g.ldc = g.N;
    g.strideC = (int64_t)g.M * g.N;
    g.split_stride = batch * g.strideC;
    g.c_dt = 0;
    g.vec = g.N % 4 == 0;
    g.alpha = 1.f;
    g.beta = 0.f;
  } else {
    g.C = o.C;
    g.ldc = o.ldc;
    g.strideC = o.strideC;
    g.c_dt = o.c_dt;
    g.vec = o.vec;
    g.alpha = o.alpha;
    g.alpha_dev = o.alpha_dev;
    g.beta = o.beta;
  }
}
inline hipError_t sum_splits(const float* part, int splits, int64_t split_stride, const Out& o, int64_t batch, int M, int N, hipStream_t st) {
  int tx = 0;
  while (tx < 8 && (4 << tx) < N) ++tx;
  const int gx = (N + (4 << tx) - 1) / (4 << tx);
  const int gy = (int)std::max<int64_t>(1, std::min<int64_t>(((int64_t)M + (256 >> tx) - 1) / (256 >> tx), 65535));
  hipLaunchKernelGGL(sum_splits_kernel, dim3(gx, gy, (unsigned)batch), dim3(256), 0, st, part, splits, split_stride, o.C, o.ldc, o.strideC, M,
                     N, o.c_dt, o.alpha, o.alpha_dev, o.beta, tx, N % 4 == 0 ? 1 : 0);
  return hipGetLastError();
}
inline hipError_t finish_split(const ProductArgs& g, const Shape& s, const Out& o, const float* part, int64_t batch, hipStream_t st) {
  if (s.splits == 1) return hipSuccess;
  return sum_splits(part, s.splits, g.split_stride, o, batch, g.M, g.N, st);
}

inline int out_code(int dt) { return dt == SHAMPOO_F32 ? 0 : dt == SHAMPOO_F16 ? 1 : 2; }
// rows that allow the epilogue's 16-byte stores
inline int rows_vec(const void* C, int64_t ldc, int64_t strideC, int dt) {
  const int64_t ve = 16 / (int64_t)size_of(dt);
  return aligned(C, 16) && ldc % ve == 0 && strideC % ve == 0;
}

}  // namespace shampoo
