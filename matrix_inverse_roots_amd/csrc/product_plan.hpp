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
#include "shampoo.h"

namespace shampoo {

inline int64_t up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }
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
// Tile of a product and its split of k.  LARGE: 256 x 256, one workgroup of
// 8 waves per CU; SMALL: 128 x 128, two workgroups of 4 waves.
struct Shape {
  bool large;
  int splits, split_stages, nst;
  int tile = 0;  // Tile, where plan_layer chose
};

constexpr int CUS = 256;  // planning only; the grid follows the device

inline Shape plan_shape(int64_t batch, int64_t M, int64_t N, int64_t K, int es, bool may_split) {
  Shape s;
  s.nst = (int)((K * es + 127) / 128);
  const int64_t tl = batch * ((M + 255) / 256) * ((N + 255) / 256);
  const int64_t ts = batch * ((M + 127) / 128) * ((N + 127) / 128);
  // Tiles of the busiest compute unit, in large tiles' time.  A small tile is
  // a quarter of the work, at 84% of the rate of a large one (8-bit 4096^3,
  // 4 small per unit against 1 large: 80 and 71 us; bfloat16 8192 x 65536 x
  // 1024: 1190 and 980 us), or 95% in float32, whose matrix instructions
  // outlast the loads (2048 x 16384 x 1024: 543 and 522 us).  So small tiles
  // win where they divide among the units better (8-bit 6144^2 x 2048, 9 small
  // against 3 large: 95 and 102 us; float32 10007 x 1024 x 999: 617 and 727 us
  // for the loss with both gradients).
  const double large_cost = (double)((tl + CUS - 1) / CUS);
  const double small_cost = (double)((ts + CUS - 1) / CUS) * 0.25 / (es == 4 ? 0.95 : 0.84);
  s.large = large_cost <= small_cost;
  s.splits = 1;
  s.split_stages = s.nst;
  const int64_t items = s.large ? tl : ts, slots = CUS;
  if (may_split && items * 2 <= slots) {
    // at least 4 stages a range
    const int64_t want = std::min<int64_t>(slots / items, s.nst / 4);
    if (want >= 2) {
      s.split_stages = (int)up((s.nst + want - 1) / want, 4);
      s.splits = (s.nst + s.split_stages - 1) / s.split_stages;
    }
  }
  return s;
}

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
  const int64_t items = batch * g.splits * ((g.M + 127) / 128) * (EPI == Epi::GATED ? (g.N + 63) / 64 : (g.N + 127) / 128);
  if (items <= CUS) return launch_tiles<E, 1, 4, 4, 1, 4, 1, AS, BS, EPI, FA, FB>(g, batch, st);
  return launch_tiles<E, 1, 4, 4, 1, 2, 2, AS, BS, EPI, FA, FB>(g, batch, st);
}

// Tiles of the feed-forward layers' products: 64 x 64 (float32 only), 128 x 128,
// 256 x 128 (bfloat16 only; three buffers, since its stages are half as long as a large
// tile's and loads take as long), 256 x 256.
enum Tile { TILE_64 = 1, TILE_128, TILE_MEDIUM, TILE_LARGE };

template <Elem E, bool AS, bool BS, Epi EPI>
hipError_t launch_layer(const ProductArgs& g, const Shape& s, int64_t batch, hipStream_t st) {
  if constexpr (E == Elem::F32 && EPI != Epi::GATED) {  // GATED needs two fragments of columns
    if (s.tile == TILE_64) return launch_tiles<E, 1, 1, 2, 2, 3, 3, AS, BS, EPI, 0, 0>(g, batch, st);
  }
  if constexpr (E == Elem::BF16) {
    if (s.tile == TILE_MEDIUM) return launch_tiles<E, 2, 2, 4, 2, 3, 1, AS, BS, EPI, 0, 0>(g, batch, st);
  }
  return launch_product<E, AS, BS, EPI>(g, s.tile == TILE_LARGE, batch, st);
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
