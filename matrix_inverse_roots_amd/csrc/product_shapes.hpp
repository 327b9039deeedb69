// Tiles and ranges of k of the rectangular products (product_core.hpp): host
// arithmetic alone, which needs neither HIP nor a GPU.
#pragma once

#include <algorithm>
#include <cstdint>

namespace shampoo {

inline int64_t up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }

// Tile of a product and its split of k.  LARGE: 256 x 256, one workgroup of
// 8 waves per CU; SMALL: 128 x 128, two workgroups of 4 waves.
struct Shape {
  bool large;
  int splits, split_stages, nst;
  int tile = 0;  // Tile, where plan_layer chose
};

// Tiles of the feed-forward layers' products: 64 x 64 (float32 only), 128 x 128
// alone on a unit (four buffers) or two of them, 256 x 128 (bfloat16 only; three
// buffers, since its stages are half as long as a large tile's and loads take as
// long), 256 x 256.
enum Tile { TILE_64 = 1, TILE_128, TILE_128_TWO, TILE_MEDIUM, TILE_LARGE };

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

// Tile and ranges of k of a layer's product: the least of the tiles' costs.
//
// Costs in the time of one 256 x 256 tile (bfloat16) where the chip is full and
// power holds its clock: 256 x 256 1, 256 x 128 0.54, two 128 x 128 on a unit 0.60
// (8192 x 10240 x 4096: 533, 585 and 644 us; 4096^3: 115, 122 and 138), one alone
// 0.33.  Where it is not, the clock rises and a tile is faster: 0.63, 0.40, 0.45,
// so that a last round which few units take costs less than a full one (4096 x
// 10240 x 8192, 2.5 rounds of large tiles, 5 of medium: 575 and 585 us; 8192 x
// 1024 x 4096, half a round and one: 88 and 65).  The epilogue of a large tile
// leaves the matrix cores waiting for longer: `epilogue` counts it in columns of
// k (150 for bias, activation, residual or kept values, 300 for the gated block's
// gradients; 8192 x 4096 x 1024 with gelu and kept values: 103 us large, 95
// medium, 100 small; with k 4096 and 10240 columns 598, 665, 775).
// float32 (matrix instructions, not loads, bound it): a 128 x 128 tile 0.26, a 64
// x 64 one 0.073 (777 x 2731 x 1000, 154 tiles or 559: 73 and 57 us; 1000 x 1000 x
// 1000, 64 or 256: 69 and 26; 2048 x 2048 x 1024, 256 or 1024: 72-78 and 75-79).
inline Shape plan_layer(int64_t batch, int64_t M, int64_t N, int64_t K, int es, bool may_split, int epilogue, bool dual = false) {
  if (M == 0 || K == 0) return Shape{};  // an empty batch, which launches none
  Shape s = plan_shape(batch, M, N, K, es, may_split);
  s.tile = s.large ? TILE_LARGE : TILE_128;
  auto tiles = [&](int64_t m, int64_t n) { return batch * ((M + m - 1) / m) * ((N + n - 1) / n); };
  if (es == 4) {
    // Ranges of k cost a launch that sums them, some 5 us, 0.3 us a range and 8 bytes
    // of traffic for each of its values, at 6.5 TB/s; a large tile takes 0.245 us for
    // each k, so in its time 20 / K, 1.2 / K and 5e-6 / K.  With all of the epilogue,
    // whole and in 2, 3, 5 ranges: 777 x 2731 x 1000 58, 59, 60, 64 us; 2048 x 2048 x
    // 1024 77, 93, 99, 110; 1100 x 1300 x 3000 104, 88, 99, 97; 497 x 434 x 3980 79, 45, 34,
    // 37 and, in 9, 28.  8 x 64 x 8000 in 16 ranges of 64-tiles 15.5 us, in 62 of one
    // 128-tile 20.
    auto ranges = [&](int64_t n, double tile, int r) {
      return (double)((n * r + CUS - 1) / CUS) * tile / r + (r > 1 ? (20.0 + (1.2 + 5e-6 * batch * M * N) * r) / K : 0.0);
    };
    double now = s.large ? (double)((tiles(256, 256) + CUS - 1) / CUS) : ranges(tiles(128, 128), 0.26, s.splits);
    for (int r = 1; !dual && r <= (may_split ? 16 : 1) && (r == 1 || r <= s.nst / 4); ++r) {
      const int stages = (s.nst + r - 1) / r;
      if ((s.nst + stages - 1) / stages != r) continue;
      const double c = ranges(tiles(64, 64), 0.073, r);
      if (c >= now) continue;
      now = c;
      s.large = false;
      s.tile = TILE_64;
      s.splits = r;
      s.split_stages = stages;
    }
    if (s.tile == TILE_128 && tiles(128, 128) * s.splits > CUS) s.tile = TILE_128_TWO;
    return s;
  }
  if (s.splits > 1) return s;
  auto cost = [&](int64_t n, int64_t slots, double full, double alone) {
    return std::max((double)n / slots * full, (double)((n + slots - 1) / slots) * alone);
  };
  const double e = 1.0 + (double)epilogue / K;
  const int64_t small = tiles(128, 128);
  const double large = cost(tiles(256, 256), CUS, 1.0, 0.63) * e;
  const double medium = cost(tiles(256, 128), CUS, 0.54, 0.40);
  const double least = small <= CUS ? 0.33 : cost(small, 2 * CUS, 0.60, 0.45);
  s.large = large <= medium && large <= least;
  s.tile = s.large ? TILE_LARGE : medium <= least ? TILE_MEDIUM : small > CUS ? TILE_128_TWO : TILE_128;
  return s;
}

// The layers' products; es: bytes of an element.  `epilogue`: whether the layer's
// has anything to do.
inline Shape plan_linear(int64_t M, int64_t N, int64_t K, int es, bool epilogue) { return plan_layer(1, M, N, K, es, true, epilogue ? 150 : 0); }
inline Shape plan_linear_dx(int64_t M, int64_t N, int64_t K, int es) { return plan_layer(1, M, K, N, es, true, 0); }
inline Shape plan_linear_dw(int64_t M, int64_t N, int64_t K, int es) { return plan_layer(1, N, K, M, es, true, 0); }
// rows of h, dg and du: whole stages of k for the products that read them
inline int64_t gated_width(int64_t f) { return up(f, 64); }
inline Shape plan_gated_in(int64_t T, int64_t d, int64_t f, int es) { return plan_layer(1, T, 2 * f, d, es, true, 0, true); }
inline Shape plan_gated_out(int64_t T, int64_t d, int64_t f, int es, bool epilogue) { return plan_linear(T, d, f, es, epilogue); }
inline Shape plan_gated_dh(int64_t T, int64_t d, int64_t f, int es) { return plan_layer(1, T, gated_width(f), d, es, false, 300); }
inline Shape plan_gated_dx(int64_t T, int64_t d, int64_t f, int es) { return plan_layer(1, T, d, 2 * gated_width(f), es, true, 0); }
inline Shape plan_gated_dw_down(int64_t T, int64_t d, int64_t f, int es) { return plan_layer(1, d, f, T, es, true, 0); }
// of the gate's or the up projection's weights, or of both in one launch
inline Shape plan_gated_dw(int64_t T, int64_t d, int64_t f, int es, bool pair) { return plan_layer(pair ? 2 : 1, f, d, T, es, true, 0); }

}  // namespace shampoo
