// 8-bit block-scaled products and the projection's softmax cross entropy
// (see include/shampoo.h): argument checks, workspace carving, launches.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "f8_kernels.hpp"
#include "f8_rows.hpp"
#include "host_common.hpp"
#include "product_plan.hpp"
#include "shampoo.h"
#include "xent_kernels.hpp"

using namespace shampoo;

namespace {

constexpr int64_t F8_MAX = (int64_t(1) << 23) - 128;

shampoo_status check_f8_sizes(int64_t n, int64_t M, int64_t N, int64_t K) {
  if (n < 0 || M < 0 || N < 0) return fail(SHAMPOO_E_INVALID, "negative size");
  if (K < 128 || K % 128 != 0) return fail(SHAMPOO_E_INVALID, "K = %lld: must be a positive multiple of 128", (long long)K);
  if (n > 65535 || M > F8_MAX || N > F8_MAX || K > F8_MAX)
    return fail(SHAMPOO_E_UNSUPPORTED, "product too large (%lld of %lld x %lld x %lld)", (long long)n, (long long)M, (long long)N,
                (long long)K);
  if (((M + 127) / 128) * ((N + 127) / 128) > INT32_MAX / 2) return fail(SHAMPOO_E_UNSUPPORTED, "too many tiles");
  return SHAMPOO_OK;
}

shampoo_status quantize_f8_impl(const void* x, int x_dt, int64_t n, int64_t rows, int64_t cols, int64_t ld, int64_t stride, int fmt,
                                int32_t block_rows, void* q, void* s, void* qt, void* st_, hipStream_t st) {
  if (n < 0 || rows < 0 || cols < 0) return fail(SHAMPOO_E_INVALID, "negative size");
  if (x_dt != SHAMPOO_F32 && x_dt != SHAMPOO_F16 && x_dt != SHAMPOO_BF16)
    return fail(SHAMPOO_E_UNSUPPORTED, "dtype %d to quantise (F32, F16, BF16)", x_dt);
  if (fmt != SHAMPOO_E4M3 && fmt != SHAMPOO_E5M2) return fail(SHAMPOO_E_UNSUPPORTED, "8-bit format %d (E4M3, E5M2)", fmt);
  if (block_rows != 1 && block_rows != 128) return fail(SHAMPOO_E_UNSUPPORTED, "block_rows = %d (1, 128)", block_rows);
  if (n > 65535 || rows > F8_MAX || cols > F8_MAX) return fail(SHAMPOO_E_UNSUPPORTED, "matrix too large to quantise");
  if (n == 0 || rows == 0 || cols == 0) return SHAMPOO_OK;
  if ((q == nullptr) != (s == nullptr) || (qt == nullptr) != (st_ == nullptr))
    return fail(SHAMPOO_E_INVALID, "values and scales are given together");
  if (!q && !qt) return fail(SHAMPOO_E_INVALID, "no output");
  if (!x) return fail(SHAMPOO_E_INVALID, "null pointer argument");
  if (ld < cols || (n > 1 && stride < 0)) return fail(SHAMPOO_E_INVALID, "row stride %lld < %lld columns", (long long)ld, (long long)cols);
  if (!aligned(q, 16) || !aligned(qt, 16) || !aligned(s, 4) || !aligned(st_, 4) || !aligned(x, size_of(x_dt)))
    return fail(SHAMPOO_E_INVALID, "misaligned pointer");
  if ((rows + 127) / 128 > 65535) return fail(SHAMPOO_E_UNSUPPORTED, "matrix too large to quantise");
  const int64_t Kp = up(cols, 128), Rp = up(rows, 128), part = n * (block_rows == 1 ? rows : Rp / 128), part_t = n * (block_rows == 1 ? cols : Kp / 128);
  const Span spans[] = {run_of("q", q, n * rows * Kp), run_of("s", s, part * up(Kp / 128, 4)), run_of("qt", qt, n * cols * Rp),
                        run_of("st", st_, part_t * up(Rp / 128, 4)),
                        run_of("x", x, (((n - 1) * stride) + (rows - 1) * ld + cols) * (int64_t)size_of(x_dt))};
  const shampoo_status apart = check_apart(spans, 4);
  if (apart != SHAMPOO_OK) return apart;
  QuantArgs g;
  g.x = x; g.ld = ld; g.stride = n > 1 ? stride : 0;
  g.q = (uint8_t*)q; g.s = (uint8_t*)s; g.qt = (uint8_t*)qt; g.st = (uint8_t*)st_;
  g.rows = (int)rows; g.cols = (int)cols;
  const dim3 grid((unsigned)((cols + 127) / 128), (unsigned)((rows + 127) / 128), (unsigned)n);
#define SHAMPOO_QUANT(T, F, R) hipLaunchKernelGGL((quantize_tile_kernel<T, F, R>), grid, dim3(256), 0, st, g)
#define SHAMPOO_QUANT_T(T)                                                     \
  do {                                                                         \
    if (fmt == SHAMPOO_E4M3) {                                                 \
      if (block_rows == 1) SHAMPOO_QUANT(T, 0, 1); else SHAMPOO_QUANT(T, 0, 128); \
    } else {                                                                   \
      if (block_rows == 1) SHAMPOO_QUANT(T, 1, 1); else SHAMPOO_QUANT(T, 1, 128); \
    }                                                                          \
  } while (0)
  if (x_dt == SHAMPOO_F32) SHAMPOO_QUANT_T(float);
  else if (x_dt == SHAMPOO_F16) SHAMPOO_QUANT_T(_Float16);
  else SHAMPOO_QUANT_T(uint16_t);
#undef SHAMPOO_QUANT_T
#undef SHAMPOO_QUANT
  LAUNCH_CHECK("quantize_f8");
  return SHAMPOO_OK;
}

template <Elem E>
hipError_t launch_f8(const ProductArgs& g, int a_dt, int b_dt, bool large, int64_t n, hipStream_t st) {
  const bool a5 = a_dt == SHAMPOO_E5M2, b5 = b_dt == SHAMPOO_E5M2;
  if (!a5 && !b5) return launch_product<E, false, false, Epi::STORE, 0, 0>(g, large, n, st);
  if (!b5) return launch_product<E, false, false, Epi::STORE, 1, 0>(g, large, n, st);
  if (!a5) return launch_product<E, false, false, Epi::STORE, 0, 1>(g, large, n, st);
  return launch_product<E, false, false, Epi::STORE, 1, 1>(g, large, n, st);
}

// Few rows: f8_rows_kernel.  Measured against the tiles: see there.
bool few_rows(int64_t M) { return M <= F8_ROWS_MAX; }

template <int MB>
hipError_t launch_rows(const ProductArgs& g, int a_dt, int b_dt, int64_t n, hipStream_t st) {
  const dim3 grid((unsigned)((g.N + 15) / 16), (unsigned)n);
  const bool a5 = a_dt == SHAMPOO_E5M2, b5 = b_dt == SHAMPOO_E5M2;
  const auto kernel = a5 ? (b5 ? f8_rows_kernel<MB, 1, 1> : f8_rows_kernel<MB, 1, 0>) : (b5 ? f8_rows_kernel<MB, 0, 1> : f8_rows_kernel<MB, 0, 0>);
  hipLaunchKernelGGL(kernel, grid, dim3(256), 0, st, g);
  return hipGetLastError();
}

size_t matmul_f8_bytes(int64_t n, int64_t M, int64_t N, int64_t K) {
  if (n == 0 || M == 0 || N == 0 || few_rows(M)) return 0;
  return partial_bytes(plan_shape(n, M, N, K, 1, true), n, M, N);
}

shampoo_status matmul_f8_impl(const void* a, int a_dt, const void* sa, int32_t arb, const void* b, int b_dt, const void* sb, int32_t brb,
                              int64_t n, int64_t M, int64_t N, int64_t K, void* c, int c_dt, void* ws, size_t ws_bytes, hipStream_t st) {
  shampoo_status r = check_f8_sizes(n, M, N, K);
  if (r != SHAMPOO_OK) return r;
  for (int dt : {a_dt, b_dt})
    if (dt != SHAMPOO_E4M3 && dt != SHAMPOO_E5M2) return fail(SHAMPOO_E_UNSUPPORTED, "operand dtype %d (E4M3, E5M2)", dt);
  if (c_dt != SHAMPOO_F32 && c_dt != SHAMPOO_F16 && c_dt != SHAMPOO_BF16)
    return fail(SHAMPOO_E_UNSUPPORTED, "result dtype %d (F32, F16, BF16)", c_dt);
  for (int rb : {arb, brb})
    if (rb != 1 && rb != 128) return fail(SHAMPOO_E_UNSUPPORTED, "block_rows = %d (1, 128)", rb);
  if (n == 0 || M == 0 || N == 0) return SHAMPOO_OK;
  if (!a || !b || !sa || !sb || !c) return fail(SHAMPOO_E_INVALID, "null pointer argument");
  if (!aligned(a, 16) || !aligned(b, 16) || !aligned(sa, 4) || !aligned(sb, 4) || !aligned(c, size_of(c_dt)))
    return fail(SHAMPOO_E_INVALID, "misaligned pointer");
  const Shape s = plan_shape(n, M, N, K, 1, true);
  const size_t need = matmul_f8_bytes(n, M, N, K);
  if (need && (!ws || ws_bytes < need || !aligned(ws, 256)))
    return fail(SHAMPOO_E_WORKSPACE, "workspace %zu bytes < %zu needed (256-byte aligned)", ws ? ws_bytes : 0, need);
  ProductArgs g{};
  g.A = a; g.B = b; g.sa = (const uint8_t*)sa; g.sb = (const uint8_t*)sb;
  g.M = (int)M; g.N = (int)N; g.K = (int)K;
  g.lda = g.ldb = K;
  g.strideA = M * K; g.strideB = N * K;
  g.ldsa = g.ldsb = up(K / 128, 4);
  g.sa_shift = arb == 128 ? 7 : 0;
  g.sb_shift = brb == 128 ? 7 : 0;
  g.strideSa = (arb == 128 ? (M + 127) / 128 : M) * g.ldsa;
  g.strideSb = (brb == 128 ? (N + 127) / 128 : N) * g.ldsb;
  const Span spans[] = {run_of("c", c, n * M * N * (int64_t)size_of(c_dt)), run_of("the workspace", ws, (int64_t)need), run_of("a", a, n * M * K),
                        run_of("b", b, n * N * K), run_of("a_scale", sa, n * g.strideSa), run_of("b_scale", sb, n * g.strideSb)};
  r = check_apart(spans, 2);
  if (r != SHAMPOO_OK) return r;
  if (few_rows(M)) {
    g.C = c; g.ldc = N; g.strideC = M * N; g.c_dt = out_code(c_dt);
    HIP_TRY(M == 1 ? launch_rows<1>(g, a_dt, b_dt, n, st) : M == 2 ? launch_rows<2>(g, a_dt, b_dt, n, st)
            : launch_rows<4>(g, a_dt, b_dt, n, st));
    return SHAMPOO_OK;
  }
  set_shape(g, s);
  const Out o{c, N, M * N, out_code(c_dt), rows_vec(c, N, n > 1 ? M * N : 0, c_dt), 0.f};
  point_output(g, s, o, (float*)ws, n);
  HIP_TRY(c_dt == SHAMPOO_F32 ? launch_f8<Elem::F8W>(g, a_dt, b_dt, s.large, n, st)
                              : launch_f8<Elem::F8>(g, a_dt, b_dt, s.large, n, st));
  HIP_TRY(finish_split(g, s, o, (const float*)ws, n, st));
  return SHAMPOO_OK;
}

// ---------------------------------------------------------------------------
// softmax cross entropy
// ---------------------------------------------------------------------------
constexpr int64_t XENT_MAX_ROW = int64_t(1) << 20;  // elements: 256 rows stay within 32-bit offsets
// The default panel's exponentials.  Every further panel reads and writes the
// weight's float32 gradient again.  From 2 to 1 GiB a call with both gradients
// loses 7-13% (8192 x 4096 x 131072 21.6 to 23.0 ms, 16384 x 2048 x 131072 23.6 to
// 26.5, 16384 x 1024 x 65536 6.5 to 7.1), from 4 to 2 GiB 2% (16384 x 2048 x
// 131072) and from 6 to 3 GiB 4% (32768 x 512 x 100003).
constexpr int64_t XENT_PANEL_BYTES = int64_t(1) << 31;
constexpr int64_t XENT_STATS_BYTES = int64_t(1) << 28;

struct XentLayout {
  int64_t panel, pieces, ldE, dp;
  int64_t Kp, Ks;  // 8-bit logits: padded width, scales of a row
  bool f8, grads, copy_hidden, copy_weight, dw_sum;  // dw_sum: float32 sum of the panels' bfloat16 gradients
  size_t count, stats, nll, norm, rows, E, hidden, kept, weight, hq, hs, wq, wsc, part, dw, total;
  Shape dx, dwp;
};

int64_t row_elems(int dt) { return dt == SHAMPOO_F32 ? 4 : 8; }

shampoo_status xent_layout(const shampoo_xent_args* a, XentLayout* L) {
  if (!a) return fail(SHAMPOO_E_INVALID, "null arguments");
  if (a->N < 0 || a->V < 1 || a->d < 1) return fail(SHAMPOO_E_INVALID, "N = %lld, V = %lld, d = %lld", (long long)a->N, (long long)a->V, (long long)a->d);
  if (a->dt != SHAMPOO_F32 && a->dt != SHAMPOO_BF16) return fail(SHAMPOO_E_UNSUPPORTED, "dtype %d (F32, BF16)", (int)a->dt);
  if (a->weight_dt != a->dt && a->weight_dt != SHAMPOO_F32)
    return fail(SHAMPOO_E_UNSUPPORTED, "weight dtype %d for dtype %d", (int)a->weight_dt, (int)a->dt);
  if (a->logits_dt != a->dt && !(a->logits_dt == SHAMPOO_E4M3 && a->dt == SHAMPOO_BF16))
    return fail(SHAMPOO_E_UNSUPPORTED, "logits dtype %d for dtype %d", (int)a->logits_dt, (int)a->dt);
  if (a->dweight && a->dweight_dt != SHAMPOO_F32 && !(a->dweight_dt == SHAMPOO_BF16 && a->dt == SHAMPOO_BF16))
    return fail(SHAMPOO_E_UNSUPPORTED, "weight gradient dtype %d for dtype %d", (int)a->dweight_dt, (int)a->dt);
  if (a->reduction < 0 || a->reduction > 2) return fail(SHAMPOO_E_INVALID, "reduction %d", a->reduction);
  if (a->N > (a->logits_dt == SHAMPOO_E4M3 ? F8_MAX : INT32_MAX / 4) || a->V > XENT_MAX_ROW || a->d > XENT_MAX_ROW / 4 || a->ld_hidden > XENT_MAX_ROW || a->ld_weight > XENT_MAX_ROW)
    return fail(SHAMPOO_E_UNSUPPORTED, "N = %lld, V = %lld, d = %lld too large", (long long)a->N, (long long)a->V, (long long)a->d);
  if (a->panel_rows < 0) return fail(SHAMPOO_E_INVALID, "panel_rows < 0");
  const int64_t es = a->dt == SHAMPOO_F32 ? 4 : 2, ve = row_elems(a->dt);
  L->grads = a->dhidden || a->dweight;
  L->pieces = (a->V + 127) / 128;
  L->ldE = L->pieces * 128;
  // rows a multiple of 128 KiB apart fall on the same cache channels when the
  // weight's gradient reads them across (131072 bfloat16 columns: 15.9 instead
  // of 23.5 GB fetched).  The call, apart against not, in bfloat16: 131072 columns
  // 6.84 and 7.07 ms (8192 rows, d 1024), 1.90 and 1.98 (2048, 1024), 21.39 and
  // 21.50 (8192, 4096); 196608: 9.29 and 9.40; 65536: 3.43 and 3.45, 10.74 and
  // 10.79; 262144: 7.46 and 7.42; float32 at 32768 to 131072 within 0.5%.
  if (L->ldE * es % 131072 == 0) L->ldE += 128;
  int64_t rows = a->panel_rows;
  if (rows == 0) {
    rows = XENT_STATS_BYTES / (L->pieces * 8);
    if (L->grads) rows = std::min(rows, XENT_PANEL_BYTES / (L->pieces * 128 * es));
    rows = std::min<int64_t>(std::max<int64_t>(rows / 256 * 256, 256), 131072);
    // panels of one size rather than a short last one
    const int64_t count = (a->N + rows - 1) / rows;
    if (count > 1) rows = up((a->N + count - 1) / count, 256);
  }
  rows = std::min<int64_t>(rows, 131072);
  L->panel = std::max<int64_t>(std::min(rows, a->N), 1);
  // the products read 16-byte runs of rows: others are copied into rows that
  // start on 16 bytes
  L->dp = up(a->d, 8);
  L->f8 = a->logits_dt == SHAMPOO_E4M3;
  L->Kp = up(a->d, 128);
  L->Ks = up(L->Kp / 128, 4);
  const bool needed = L->grads || !L->f8;
  L->copy_hidden = needed && (a->d % ve || a->ld_hidden % ve || !aligned(a->hidden, 16));
  L->copy_weight = needed && (a->weight_dt != a->dt || a->d % ve || a->ld_weight % ve || !aligned(a->weight, 16));
  L->dw_sum = a->dweight && a->dweight_dt == SHAMPOO_BF16 && L->panel < a->N;
  L->dx = plan_shape(1, L->panel, a->d, a->V, (int)es, true);
  L->dwp = plan_shape(1, a->V, a->d, L->panel, (int)es, true);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t p = at;
    at += align_up(bytes);
    return p;
  };
  L->count = take(4);
  L->stats = take((size_t)L->pieces * L->panel * 8);
  L->nll = take((size_t)L->panel * 4);
  L->norm = take((size_t)L->panel * 8);
  L->rows = take((size_t)std::max<int64_t>(a->N, 1) * 4);
  L->E = take(L->grads ? (size_t)L->panel * L->ldE * es : 0);
  L->hidden = take(L->copy_hidden ? (size_t)a->N * L->dp * es : 0);
  // hidden's rows with the ignored ones zeroed: a panel's, or the copy in place
  L->kept = take(a->dweight && !L->copy_hidden ? (size_t)L->panel * L->dp * es : 0);
  L->weight = take(L->copy_weight ? (size_t)a->V * L->dp * es : 0);
  L->hq = take(L->f8 ? a->N * L->Kp : 0);
  L->hs = take(L->f8 ? a->N * L->Ks : 0);
  L->wq = take(L->f8 ? a->V * L->Kp : 0);
  L->wsc = take(L->f8 ? a->V * L->Ks : 0);
  size_t part = 0;
  if (a->dhidden) part = std::max(part, partial_bytes(L->dx, 1, L->panel, a->d));
  if (a->dweight) part = std::max(part, partial_bytes(L->dwp, 1, a->V, a->d));
  L->part = take(part);
  L->dw = take(L->dw_sum ? (size_t)a->V * a->d * 4 : 0);
  L->total = at;
  return SHAMPOO_OK;
}

template <Elem E, bool AS, bool BS, Epi EPI>
hipError_t product(ProductArgs& g, const Shape& s, hipStream_t st) {
  set_shape(g, s);
  return launch_product<E, AS, BS, EPI>(g, s.large, 1, st);
}

template <Elem E, typename T>
shampoo_status run_xent(const shampoo_xent_args* a, const XentLayout& L, hipStream_t st) {
  using TE = typename std::conditional<E == Elem::F32, float, uint16_t>::type;
  unsigned char* w = (unsigned char*)a->ws;
  const int64_t N = a->N, V = a->V, d = a->d;
  const int64_t es = sizeof(T);
  float* inv_count = (float*)(w + L.count);
  floatx2* stats = (floatx2*)(w + L.stats);
  float* nll = (float*)(w + L.nll);
  floatx2_t* norm = (floatx2_t*)(w + L.norm);
  const bool mean = a->reduction == SHAMPOO_REDUCE_MEAN, each = a->reduction == SHAMPOO_REDUCE_NONE;
  float* rows = each ? a->loss : (float*)(w + L.rows);
  const unsigned char* hidden = (const unsigned char*)a->hidden;
  const unsigned char* weight = (const unsigned char*)a->weight;
  int64_t ldh = a->ld_hidden, ldw = a->ld_weight;
  auto pad = [&](const void* from, int dt, int64_t ld, int64_t count, unsigned char* to) -> hipError_t {
    const int wgs = (int)std::max<int64_t>(1, std::min<int64_t>((count + 3) / 4, 8192));
    const int vec = ld % 4 == 0 && aligned(from, 4 * size_of(dt));
    if (sizeof(T) == 2 && dt == SHAMPOO_F32)
      hipLaunchKernelGGL((pad_rows_kernel<float, T>), dim3(wgs), dim3(256), 0, st, (const float*)from, ld, count, (int)d, (T*)to, (int)L.dp, vec);
    else
      hipLaunchKernelGGL((pad_rows_kernel<T, T>), dim3(wgs), dim3(256), 0, st, (const T*)from, ld, count, (int)d, (T*)to, (int)L.dp, vec);
    return hipGetLastError();
  };
  if (N > 0 && L.copy_hidden) {
    HIP_TRY(pad(a->hidden, a->dt, ldh, N, w + L.hidden));
    hidden = w + L.hidden;
    ldh = L.dp;
  }
  if (N > 0 && L.copy_weight) {
    HIP_TRY(pad(a->weight, a->weight_dt, ldw, V, w + L.weight));
    weight = w + L.weight;
    ldw = L.dp;
  }
  if (N > 0 && L.f8) {
    shampoo_status r = quantize_f8_impl(a->hidden, a->dt, 1, N, d, a->ld_hidden, 0, SHAMPOO_E4M3, 1, w + L.hq, w + L.hs, nullptr, nullptr, st);
    if (r == SHAMPOO_OK)
      r = quantize_f8_impl(a->weight, a->weight_dt, 1, V, d, a->ld_weight, 0, SHAMPOO_E4M3, 1, w + L.wq, w + L.wsc, nullptr, nullptr, st);
    if (r != SHAMPOO_OK) return r;
  }
  // one panel: the reduction counts, ahead of the gradients' products (an
  // empty batch has none, and nothing in it is read)
  const bool single = N > 0 && N <= L.panel;
  auto reduce = [&]() -> hipError_t {
    hipLaunchKernelGGL(xent_reduce_kernel, dim3(1), dim3(1024), 0, st, rows, mean && single ? a->targets : nullptr, (int)N, a->ignore_index,
                       mean ? inv_count : nullptr, a->loss);
    return hipGetLastError();
  };
  if (mean && !single) {
    hipLaunchKernelGGL(xent_count_kernel, dim3(1), dim3(1024), 0, st, a->targets, (int)N, a->ignore_index, inv_count);
    LAUNCH_CHECK("xent_count");
  }
  const Out dw{a->dweight, a->ld_dweight, 0, out_code(a->dweight_dt),
               a->dweight ? rows_vec(a->dweight, a->ld_dweight, 0, a->dweight_dt) : 0, a->accumulate ? 1.f : 0.f,
               a->scale, mean ? inv_count : nullptr};
  const Out dw32{w + L.dw, d, 0, 0, d % 4 == 0, 0.f};
  for (int64_t r0 = 0; r0 < N; r0 += L.panel) {
    const int64_t M = std::min(L.panel, N - r0);
    // logits, consumed where they are made
    ProductArgs g{};
    g.A = hidden + r0 * ldh * es; g.B = weight;
    g.lda = ldh; g.ldb = ldw;
    g.M = (int)M; g.N = (int)V; g.K = (int)d;
    g.C = L.grads ? w + L.E : nullptr;
    g.ldc = L.ldE;
    g.stats = stats;
    g.targets = a->targets + r0;
    g.target_logit = nll;
    if (L.f8) {
      g.A = w + L.hq + r0 * L.Kp; g.sa = w + L.hs + r0 * L.Ks;
      g.B = w + L.wq; g.sb = w + L.wsc;
      g.lda = g.ldb = L.Kp;
      g.ldsa = g.ldsb = L.Ks;
      g.K = (int)L.Kp;
      HIP_TRY((product<Elem::F8, false, false, Epi::SOFTMAX>(g, plan_shape(1, M, V, L.Kp, 1, false), st)));
    } else {
      HIP_TRY((product<E, false, false, Epi::SOFTMAX>(g, plan_shape(1, M, V, d, (int)es, false), st)));
    }
    RowArgs ra{(const floatx2_t*)stats, nll, a->targets + r0, a->row_scale && !each ? a->row_scale + r0 : nullptr, norm,
               a->lse ? a->lse + r0 : nullptr, rows + r0, a->ignore_index, (int)M, (int)V, (int)L.pieces, each ? 1.f : a->scale};
    if (M <= 256) hipLaunchKernelGGL(xent_rows_kernel<1>, dim3((unsigned)M), dim3(1024), 0, st, ra);
    else hipLaunchKernelGGL(xent_rows_kernel<32>, dim3((unsigned)((M + 31) / 32)), dim3(1024), 0, st, ra);
    LAUNCH_CHECK("xent_rows");
    if (single && !each) HIP_TRY(reduce());
    if (!L.grads) continue;
    const int first = (int)((L.ldE + 2047) / 2048), more = a->dweight ? (int)((d + 2047) / 2048) : 0;
    unsigned char* kept = L.copy_hidden ? w + L.hidden + r0 * L.dp * es : w + L.kept;
    GradArgs ga{w + L.E, L.ldE, (const floatx2_t*)stats, nll, norm, a->targets + r0, a->row_scale ? a->row_scale + r0 : nullptr,
                a->ignore_index, (int)M, (int)V, (int)L.pieces, hidden + r0 * ldh * es, ldh, kept, L.dp, (int)d, first};
    hipLaunchKernelGGL((xent_grad_kernel<TE>), dim3((unsigned)(first + more), (unsigned)((M + 3) / 4)), dim3(256), 0, st, ga);
    LAUNCH_CHECK("xent_grad");
    float* part = (float*)(w + L.part);
    if (a->dhidden) {
      unsigned char* C = (unsigned char*)a->dhidden + r0 * a->ld_dhidden * es;
      const Out o{C, a->ld_dhidden, 0, out_code(a->dt), rows_vec(C, a->ld_dhidden, 0, a->dt), 0.f, a->scale, mean ? inv_count : nullptr};
      // a shorter last panel keeps the full panel's split, which the workspace holds
      const Shape s = L.dx;
      ProductArgs p{};
      p.A = w + L.E; p.B = weight; p.lda = L.ldE; p.ldb = ldw;
      p.M = (int)M; p.N = (int)d; p.K = (int)V;
      point_output(p, s, o, part, 1);
      HIP_TRY((product<E, false, true, Epi::STORE>(p, s, st)));
      HIP_TRY(finish_split(p, s, o, part, 1, st));
    }
    if (a->dweight) {
      Out o = L.dw_sum ? dw32 : dw;
      if (r0 > 0) o.beta = 1.f;
      Shape s = plan_shape(1, V, d, M, (int)es, true);
      if (partial_bytes(s, 1, V, d) > partial_bytes(L.dwp, 1, V, d)) s = plan_shape(1, V, d, M, (int)es, false);
      ProductArgs p{};
      p.A = w + L.E; p.B = kept; p.lda = L.ldE; p.ldb = L.dp;
      p.M = (int)V; p.N = (int)d; p.K = (int)M;
      point_output(p, s, o, part, 1);
      HIP_TRY((product<E, true, true, Epi::STORE>(p, s, st)));
      HIP_TRY(finish_split(p, s, o, part, 1, st));
    }
  }
  if (L.dw_sum) HIP_TRY(sum_splits((const float*)(w + L.dw), 1, 0, dw, 1, (int)V, (int)d, st));
  if (N == 0 && a->dweight) {  // zeros (or unchanged)
    Out none = dw;
    none.alpha_dev = nullptr;
    HIP_TRY(sum_splits(nullptr, 0, 0, none, 1, (int)V, (int)d, st));
  }
  if (!each && !single) HIP_TRY(reduce());
  return SHAMPOO_OK;
}

}  // namespace

extern "C" {

shampoo_status shampoo_quantize_f8(const void* x, shampoo_dtype x_dt, int64_t n, int64_t rows, int64_t cols, int64_t ld, int64_t stride,
                                   shampoo_dtype fmt, int32_t block_rows, void* q, void* s, void* qt, void* st, hipStream_t stream) {
  return quantize_f8_impl(x, x_dt, n, rows, cols, ld, stride, fmt, block_rows, q, s, qt, st, stream);
}

shampoo_status shampoo_matmul_f8_workspace(int64_t n, int64_t M, int64_t N, int64_t K, size_t* bytes) {
  if (!bytes) return fail(SHAMPOO_E_INVALID, "null pointer argument");
  const shampoo_status r = check_f8_sizes(n, M, N, K);
  if (r != SHAMPOO_OK) return r;
  *bytes = matmul_f8_bytes(n, M, N, K);
  return SHAMPOO_OK;
}

shampoo_status shampoo_matmul_f8(const void* a, shampoo_dtype a_dt, const void* a_scale, int32_t a_block_rows, const void* b,
                                 shampoo_dtype b_dt, const void* b_scale, int32_t b_block_rows, int64_t n, int64_t M, int64_t N,
                                 int64_t K, void* c, shampoo_dtype c_dt, void* ws, size_t ws_bytes, hipStream_t stream) {
  return matmul_f8_impl(a, a_dt, a_scale, a_block_rows, b, b_dt, b_scale, b_block_rows, n, M, N, K, c, c_dt, ws, ws_bytes, stream);
}

shampoo_status shampoo_linear_xent_workspace(const shampoo_xent_args* args, size_t* bytes) {
  if (!bytes) return fail(SHAMPOO_E_INVALID, "null pointer argument");
  XentLayout L;
  const shampoo_status r = xent_layout(args, &L);
  if (r != SHAMPOO_OK) return r;
  *bytes = L.total;
  return SHAMPOO_OK;
}

shampoo_status shampoo_linear_xent(const shampoo_xent_args* a, hipStream_t stream) {
  XentLayout L;
  const shampoo_status r = xent_layout(a, &L);
  if (r != SHAMPOO_OK) return r;
  if (!a->weight || (a->N > 0 && (!a->hidden || !a->targets)) || (!a->loss && (a->N > 0 || a->reduction != SHAMPOO_REDUCE_NONE)))
    return fail(SHAMPOO_E_INVALID, "null pointer argument");
  const size_t es = size_of(a->dt);
  if (a->ld_hidden < a->d || a->ld_weight < a->d || (a->dhidden && a->ld_dhidden < a->d) || (a->dweight && a->ld_dweight < a->d))
    return fail(SHAMPOO_E_INVALID, "row stride below d = %lld", (long long)a->d);
  if (!aligned(a->hidden, es) || !aligned(a->weight, size_of(a->weight_dt)) || !aligned(a->dhidden, es) || !aligned(a->targets, 8) || !aligned(a->loss, 4) ||
      (a->dweight && !aligned(a->dweight, size_of(a->dweight_dt))) || !aligned(a->row_scale, 4) || !aligned(a->lse, 4))
    return fail(SHAMPOO_E_INVALID, "misaligned pointer");
  if (!a->ws || a->ws_bytes < L.total || !aligned(a->ws, 256))
    return fail(SHAMPOO_E_WORKSPACE, "workspace %zu bytes < %zu needed (256-byte aligned)", a->ws ? a->ws_bytes : 0, L.total);
  // a later panel reads what an earlier one's gradients would have replaced
  const Span spans[] = {rows_of("dhidden", a->dhidden, a->N, a->d, a->ld_dhidden, a->dt),
                        rows_of("dweight", a->dweight, a->V, a->d, a->ld_dweight, a->dweight_dt),
                        run_of("loss", a->loss, a->reduction == SHAMPOO_REDUCE_NONE ? 4 * a->N : 4),
                        run_of("lse", a->lse, 4 * a->N),
                        run_of("the workspace", a->ws, (int64_t)L.total),
                        rows_of("hidden", a->hidden, a->N, a->d, a->ld_hidden, a->dt),
                        rows_of("weight", a->weight, a->V, a->d, a->ld_weight, a->weight_dt),
                        run_of("targets", a->targets, 8 * a->N),
                        run_of("row_scale", a->row_scale, 4 * a->N)};
  const shampoo_status apart = check_apart(spans, 5);
  if (apart != SHAMPOO_OK) return apart;
  return a->dt == SHAMPOO_F32 ? run_xent<Elem::F32, float>(a, L, stream) : run_xent<Elem::BF16, uint16_t>(a, L, stream);
}

}  // extern "C"
