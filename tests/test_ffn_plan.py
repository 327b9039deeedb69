"""Host-only checks of the feed-forward layers' plans: which tiles they reach,
and that the sizes of the GPU tests reach all of them."""

import os
import subprocess

import pytest

import ffn_shapes

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# Prints one line for each product of the sizes given as arguments, or of many
# that it draws: layer, product, bytes of an element, tile, ranges of k.
SOURCE = r"""
#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <random>
#include <set>
#include <string>
#include "product_shapes.hpp"
using namespace shampoo;
std::set<std::string> lines;
void put(const char* layer, const char* what, int es, const Shape& s) {
  char b[99];
  snprintf(b, sizeof(b), "%s %s %d %d %s%s", layer, what, es, s.tile, s.splits > 1 ? "ranges" : "whole", s.splits > 1 && s.large ? " large" : "");
  lines.insert(b);
}
void layer(int64_t M, int64_t K, int64_t N, int es) {
  for (int e = 0; e < 2; ++e) put("linear", "y", es, plan_linear(M, N, K, es, e));
  put("linear", "dx", es, plan_linear_dx(M, N, K, es));
  put("linear", "dw", es, plan_linear_dw(M, N, K, es));
}
void block(int64_t T, int64_t d, int64_t f, int es) {
  put("gated", "in", es, plan_gated_in(T, d, f, es));
  for (int e = 0; e < 2; ++e) put("gated", "out", es, plan_gated_out(T, d, f, es, e));
  put("gated", "dh", es, plan_gated_dh(T, d, f, es));
  put("gated", "dx", es, plan_gated_dx(T, d, f, es));
  put("gated", "dw_down", es, plan_gated_dw_down(T, d, f, es));
  put("gated", "pair", es, plan_gated_dw(T, d, f, es, true));
}
int main(int argc, char** argv) {
  for (int i = 1; i + 4 < argc; i += 5) (argv[i][0] == 'l' ? layer : block)(atol(argv[i + 2]), atol(argv[i + 3]), atol(argv[i + 4]), atoi(argv[i + 1]));
  std::mt19937 rng(1);
  std::uniform_real_distribution<double> u(0, 1);
  auto size = [&](double hi) { return (int64_t)std::exp(u(rng) * std::log(hi)); };
  for (int i = 0; argc == 1 && i < 300000; ++i) {
    const int64_t a = 5 + size(60000), b = size(30000), c = size(60000);
    if ((double)a * b * c > 4e12) continue;
    for (int es = 2; es <= 4; es += 2) layer(a, b, c, es), block(a, b, c, es);
  }
  for (const auto& l : lines) puts(l.c_str());
}
"""


def lines_of(exe, sizes):
    """Lines of these (layer, bytes of an element, sizes)."""
    args = [str(v) for name, es, size in sizes for v in (name, es) + tuple(size)]
    return subprocess.run([str(exe)] + args, check=True, capture_output=True, text=True).stdout.splitlines()


@pytest.fixture(scope="module")
def exe(tmp_path_factory):
    at = tmp_path_factory.mktemp("plans")
    src, exe = at / "plans.cpp", at / "plans"
    src.write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-O2", "-I", os.path.join(ROOT, "matrix_inverse_roots_amd", "csrc"), str(src), "-o", str(exe)],
                   check=True, capture_output=True)
    return exe


@pytest.fixture(scope="module")
def reachable(exe):
    return lines_of(exe, [])


def test_sizes_reach_every_tile(exe, reachable):
    """Each product's kernels, of each type: what any size reaches, the tests' sizes reach too."""
    tested = lines_of(exe, [(name, es, size) for name, sizes in (("linear", ffn_shapes.LINEAR), ("gated", ffn_shapes.GATED))
                            for dt, es in (("bfloat16", 2), ("float32", 4)) for size in sizes[dt]])
    assert len(reachable) >= 80
    assert sorted(set(reachable) - set(tested)) == []


def test_only_built_tiles_are_chosen(reachable):
    """What launch_layer builds: no 256 x 128 of float32, no 64 x 64 of bfloat16 or for the two projections, over ranges of k
    only 64 x 64 and 128 x 128 alone on a unit; and each of the others by some plan."""
    t64, t128, two, medium, large = 1, 2, 3, 4, 5
    tiles = {}
    for line in reachable:
        layer, what, es, tile, how = line.split()
        tiles.setdefault((layer, what, int(es), how), set()).add(int(tile))
    for (layer, what, es, how), got in tiles.items():
        small = {t64} if es == 4 and what != "in" else set()
        if how == "ranges":
            assert got == small | {t128}, (layer, what, es, how)
        else:
            assert got == small | {t128, two, large} | ({medium} if es == 2 else set()), (layer, what, es, how)


@pytest.mark.parametrize("size,ranges", [
    # each range of a large result is written and read again: measured, whole against 2 and 5 ranges,
    # 58, 59, 64 us; 77, 93, 110; 26, 32, 35
    ((777, 1000, 2731), False), ((2048, 1024, 2048), False), ((1000, 1000, 1000), False),
    # few results of a long sum, whole against 4: 79, 30; 44, 21; 25, 17; and 104 against 88 in 2
    ((497, 3980, 434), True), ((434, 2048, 497), True), ((64, 1024, 4096), True), ((1100, 3000, 1300), True)])
def test_float32_ranges_where_they_pay(exe, size, ranges):
    (y,) = {l.split()[-1] for l in lines_of(exe, [("linear", 4, size)]) if l.startswith("linear y ")}
    assert (y == "ranges") == ranges
