// Feed-forward layers (see include/shampoo.h): argument checks, workspace
// carving, launches.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "ffn_kernels.hpp"
#include "host_common.hpp"
#include "product_plan.hpp"
#include "shampoo.h"

using namespace shampoo;

namespace {

constexpr int64_t FFN_MAX_ROWS = INT32_MAX / 4, FFN_MAX_COLS = int64_t(1) << 18, FFN_MAX_LD = int64_t(1) << 20;

bool is_dt(int dt) { return dt == SHAMPOO_F32 || dt == SHAMPOO_BF16; }
bool one_of(int dt, int a, int b) { return dt == a || dt == b; }

shampoo_status check_types(int dt, int w_dt, int act) {
  if (!is_dt(dt)) return fail(SHAMPOO_E_UNSUPPORTED, "dtype %d (F32, BF16)", dt);
  if (!one_of(w_dt, dt, SHAMPOO_F32)) return fail(SHAMPOO_E_UNSUPPORTED, "weight dtype %d for dtype %d", w_dt, dt);
  if (act < SHAMPOO_ACT_NONE || act > SHAMPOO_ACT_SILU) return fail(SHAMPOO_E_INVALID, "activation %d", act);
  return SHAMPOO_OK;
}
shampoo_status check_sizes(int64_t rows, int64_t a, int64_t b) {
  if (rows < 0 || a < 1 || b < 1) return fail(SHAMPOO_E_INVALID, "sizes %lld, %lld, %lld", (long long)rows, (long long)a, (long long)b);
  if (rows > FFN_MAX_ROWS || a > FFN_MAX_COLS || b > FFN_MAX_COLS ||
      (rows / 128 + 1) * (std::max(a, b) / 64 + 2) > INT32_MAX / 4)
    return fail(SHAMPOO_E_UNSUPPORTED, "sizes %lld, %lld, %lld too large", (long long)rows, (long long)a, (long long)b);
  return SHAMPOO_OK;
}

// Rows of a call's argument.
struct Rows {
  const char* name;
  const void* p;
  int64_t rows, cols, ld;
  int dt;
};
// Each argument that is given: strides, alignment.
template <size_t COUNT> shampoo_status check_rows(const Rows (&all)[COUNT]) {
  for (const Rows& r : all) {
    if (!r.p) continue;
    if (r.ld < r.cols) return fail(SHAMPOO_E_INVALID, "%s: row stride %lld < %lld columns", r.name, (long long)r.ld, (long long)r.cols);
    if (r.ld > FFN_MAX_LD) return fail(SHAMPOO_E_UNSUPPORTED, "%s: row stride %lld too large", r.name, (long long)r.ld);
    if (!aligned(r.p, size_of(r.dt))) return fail(SHAMPOO_E_INVALID, "%s is misaligned", r.name);
  }
  return SHAMPOO_OK;
}
Span span_of(const Rows& r) { return rows_of(r.name, r.p, r.rows, r.cols, r.ld, r.dt); }
shampoo_status check_ws(const void* ws, size_t have, size_t need) {
  if (need && (!ws || have < need || !aligned(ws, 256)))
    return fail(SHAMPOO_E_WORKSPACE, "workspace %zu bytes < %zu needed (256-byte aligned)", ws ? have : 0, need);
  return SHAMPOO_OK;
}

struct Carve {
  size_t at = 0;
  size_t take(size_t bytes) {
    const size_t p = at;
    at += align_up(bytes);
    return p;
  }
};

// An operand of the products: as it is, or copied to rows that start on 16
// bytes, in the products' type, zeros behind the columns (float32 weights
// beside bfloat16, odd strides, 8 bits).
struct Operand {
  bool copy;
  int64_t ld;
  size_t at;
};
Operand operand(Carve& c, const void* p, int64_t rows, int64_t cols, int64_t ld, int from, int dt, bool wanted = true) {
  const int64_t ve = 16 / (int64_t)size_of(dt);
  Operand o{from != dt || cols % ve != 0 || ld % ve != 0 || !aligned(p, 16), ld, 0};
  if (!wanted) o.copy = false;
  if (o.copy) {
    o.ld = up(cols, 8);
    o.at = c.take((size_t)rows * o.ld * size_of(dt));
  }
  return o;
}
// Where the operand is, the copy made.
hipError_t place(const Operand& o, const void*& p, const void* scale, int64_t rows, int64_t cols, int64_t ld, int from, int dt, void* ws,
                 hipStream_t st) {
  if (!o.copy || rows == 0) return hipSuccess;
  void* to = (unsigned char*)ws + o.at;
  if (from == SHAMPOO_E4M3) {
    const int64_t per = (o.ld + 15) / 16;
    const int wgs = (int)std::min<int64_t>((rows * per + 255) / 256, 16384);
    if (dt == SHAMPOO_F32)
      hipLaunchKernelGGL(widen_rows_kernel<float>, dim3(wgs), dim3(256), 0, st, (const uint8_t*)p, (const uint8_t*)scale, up(cols, 128),
                         up(up(cols, 128) / 128, 4), rows, (int)cols, (float*)to, o.ld);
    else
      hipLaunchKernelGGL(widen_rows_kernel<uint16_t>, dim3(wgs), dim3(256), 0, st, (const uint8_t*)p, (const uint8_t*)scale, up(cols, 128),
                         up(up(cols, 128) / 128, 4), rows, (int)cols, (uint16_t*)to, o.ld);
  } else {
    const dim3 wgs((unsigned)std::min<int64_t>((rows + 3) / 4, 16384), (unsigned)((o.ld + 511) / 512));
    if (from == SHAMPOO_F32 && dt == SHAMPOO_BF16)
      hipLaunchKernelGGL((copy_rows_kernel<float, uint16_t>), wgs, dim3(256), 0, st, (const float*)p, ld, rows, (int)cols, (uint16_t*)to, o.ld);
    else if (dt == SHAMPOO_F32)
      hipLaunchKernelGGL((copy_rows_kernel<float, float>), wgs, dim3(256), 0, st, (const float*)p, ld, rows, (int)cols, (float*)to, o.ld);
    else
      hipLaunchKernelGGL((copy_rows_kernel<uint16_t, uint16_t>), wgs, dim3(256), 0, st, (const uint16_t*)p, ld, rows, (int)cols, (uint16_t*)to, o.ld);
  }
  p = to;
  return hipGetLastError();
}

int kept_code(int dt) { return dt == SHAMPOO_E4M3 ? 4 : out_code(dt); }
// A call of few rows takes no matrix cores, unless it keeps blocks of 8 bits,
// which reach over its workgroups.
bool few_rows(int64_t rows, const void* keep, int keep_dt) { return rows <= FFN_ROWS_MAX && !(keep && keep_dt == SHAMPOO_E4M3); }

// ---------------------------------------------------------------------------
// one layer
// ---------------------------------------------------------------------------
// y = act(x w^T + bias) + residual on operands that start on 16 bytes
struct Layer {
  const void *x, *w;
  int64_t ldx, ldw, M, N, K;
  void* y;
  int64_t ldy;
  int y_dt;
  FfnArgs ffn;
  Shape shape;
  float* part;
};

// Partial results in rows that start on 16 bytes.
size_t padded_bytes(const Shape& s, int64_t batch, int64_t M, int64_t N) { return partial_bytes(s, batch, M, up(N, 4)); }
void pad_partials(ProductArgs& g, const Shape& s, int64_t batch) {
  if (s.splits == 1) return;
  g.ldc = up(g.N, 4);
  g.strideC = g.M * g.ldc;
  g.split_stride = batch * g.strideC;
  g.vec = 1;
}
hipError_t finish_layer(const FinishArgs& f, hipStream_t st) {
  hipLaunchKernelGGL(ffn_finish_kernel<false>, dim3((unsigned)((up(f.N, 32) + 1023) / 1024), (unsigned)std::min(f.M, 65535)), dim3(256), 0, st, f);
  return hipGetLastError();
}

template <Elem E> hipError_t run_layer(const Layer& l, hipStream_t st) {
  ProductArgs g{};
  g.A = l.x; g.B = l.w;
  g.lda = l.ldx; g.ldb = l.ldw;
  g.M = (int)l.M; g.N = (int)l.N; g.K = (int)l.K;
  set_shape(g, l.shape);
  g.ffn = l.ffn;
  const Out o{l.y, l.ldy, 0, out_code(l.y_dt), 1, 0.f};
  point_output(g, l.shape, o, l.part, 1);
  if (l.shape.splits == 1) return launch_layer<E, false, false, Epi::LINEAR>(g, l.shape, 1, st);
  pad_partials(g, l.shape, 1);
  HIP_TRY_ERR((launch_layer<E, false, false, Epi::STORE>(g, l.shape, 1, st)));
  return finish_layer({l.part, g.split_stride, l.shape.splits, (int)l.M, (int)l.N, 0, l.y, l.ldy, out_code(l.y_dt), l.ffn}, st);
}

// Waves that share a row's k in ffn_rows_kernel: one for each 512 elements.
int row_waves(int64_t K) { return K > 1024 ? 4 : K > 512 ? 2 : 1; }

template <typename TX, typename TW, bool ROUND, bool GATED> hipError_t launch_rows(const RowsArgs& g, hipStream_t st) {
  const int cols = 16 / g.kw;  // of a workgroup
  const dim3 grid((unsigned)((g.N + cols - 1) / cols));
  if (g.M == 1) hipLaunchKernelGGL((ffn_rows_kernel<TX, TW, ROUND, 1, GATED>), grid, dim3(256), 0, st, g);
  else if (g.M == 2) hipLaunchKernelGGL((ffn_rows_kernel<TX, TW, ROUND, 2, GATED>), grid, dim3(256), 0, st, g);
  else hipLaunchKernelGGL((ffn_rows_kernel<TX, TW, ROUND, 4, GATED>), grid, dim3(256), 0, st, g);
  return hipGetLastError();
}
template <bool GATED> hipError_t launch_rows_of(const RowsArgs& g, int dt, int w_dt, hipStream_t st) {
  if (dt == SHAMPOO_F32) return launch_rows<float, float, false, GATED>(g, st);
  if (w_dt == SHAMPOO_F32) return launch_rows<uint16_t, float, true, GATED>(g, st);
  return launch_rows<uint16_t, uint16_t, false, GATED>(g, st);
}
int rows16(const void* p, int64_t ld, int dt) { return aligned(p, 16) && ld * (int64_t)size_of(dt) % 16 == 0; }

struct LinearLayout {
  bool few;
  Operand x, w;
  Shape shape;
  size_t part, total;
};

shampoo_status linear_layout(const shampoo_linear_args* a, LinearLayout* L) {
  if (!a) return fail(SHAMPOO_E_INVALID, "null arguments");
  shampoo_status r = check_types(a->dt, a->w_dt, a->activation);
  if (r != SHAMPOO_OK) return r;
  if (a->bias && !one_of(a->bias_dt, a->dt, SHAMPOO_F32)) return fail(SHAMPOO_E_UNSUPPORTED, "bias dtype %d for dtype %d", (int)a->bias_dt, (int)a->dt);
  if (!one_of(a->y_dt, a->dt, SHAMPOO_F32)) return fail(SHAMPOO_E_UNSUPPORTED, "result dtype %d for dtype %d", (int)a->y_dt, (int)a->dt);
  if (a->keep && !one_of(a->keep_dt, a->dt, SHAMPOO_E4M3)) return fail(SHAMPOO_E_UNSUPPORTED, "dtype %d to keep for dtype %d", (int)a->keep_dt, (int)a->dt);
  r = check_sizes(a->M, a->N, a->K);
  if (r != SHAMPOO_OK) return r;
  Carve c;
  L->few = few_rows(a->M, a->keep, a->keep_dt);
  L->part = 0;
  if (!L->few) {
    L->x = operand(c, a->x, a->M, a->K, a->ld_x, a->dt, a->dt);
    L->w = operand(c, a->w, a->N, a->K, a->ld_w, a->w_dt, a->dt);
    L->shape = plan_linear(a->M, a->N, a->K, (int)size_of(a->dt), a->bias || a->residual || a->keep || a->activation);
    L->part = c.take(padded_bytes(L->shape, 1, a->M, a->N));
  }
  L->total = c.at;
  return SHAMPOO_OK;
}

template <Elem E> hipError_t run_linear(const shampoo_linear_args* a, const LinearLayout& L, const FfnArgs& ffn, hipStream_t st) {
  const void *x = a->x, *w = a->w;
  HIP_TRY_ERR(place(L.x, x, nullptr, a->M, a->K, a->ld_x, a->dt, a->dt, a->ws, st));
  HIP_TRY_ERR(place(L.w, w, nullptr, a->N, a->K, a->ld_w, a->w_dt, a->dt, a->ws, st));
  return run_layer<E>({x, w, L.x.ld, L.w.ld, a->M, a->N, a->K, a->y, a->ld_y, a->y_dt, ffn, L.shape, (float*)((unsigned char*)a->ws + L.part)}, st);
}

// ---------------------------------------------------------------------------
// its gradients
// ---------------------------------------------------------------------------
struct LinearGradLayout {
  bool pass, store;  // act_grad_kernel runs; and leaves dz
  Operand x, w;
  int64_t ld_dz;
  Shape dx, dw;
  size_t dz, sums, part, total;
};

shampoo_status linear_grad_layout(const shampoo_linear_grad_args* a, LinearGradLayout* L) {
  if (!a) return fail(SHAMPOO_E_INVALID, "null arguments");
  shampoo_status r = check_types(a->dt, a->w_dt, a->activation);
  if (r != SHAMPOO_OK) return r;
  if (a->dw && !one_of(a->x_dt, a->dt, SHAMPOO_E4M3)) return fail(SHAMPOO_E_UNSUPPORTED, "x's dtype %d for dtype %d", (int)a->x_dt, (int)a->dt);
  if (a->activation && !one_of(a->kept_dt, a->dt, SHAMPOO_E4M3))
    return fail(SHAMPOO_E_UNSUPPORTED, "kept dtype %d for dtype %d", (int)a->kept_dt, (int)a->dt);
  if ((a->dw && !one_of(a->dw_dt, a->dt, SHAMPOO_F32)) || (a->dbias && !one_of(a->dbias_dt, a->dt, SHAMPOO_F32)))
    return fail(SHAMPOO_E_UNSUPPORTED, "gradient dtypes %d, %d for dtype %d", (int)a->dw_dt, (int)a->dbias_dt, (int)a->dt);
  r = check_sizes(a->M, a->N, a->K);
  if (r != SHAMPOO_OK) return r;
  const int es = (int)size_of(a->dt);
  const int64_t ve = 16 / es;
  Carve c;
  const bool products = a->dx || a->dw;
  L->store = products && (a->activation || a->N % ve || a->ld_dy % ve || !aligned(a->dy, 16));
  L->pass = L->store || a->dbias;
  L->ld_dz = L->store ? up(a->N, 8) : a->ld_dy;
  L->x = operand(c, a->x, a->M, a->K, a->ld_x, a->x_dt, a->dt, a->dw);
  L->w = operand(c, a->w, a->N, a->K, a->ld_w, a->w_dt, a->dt, a->dx);
  L->dx = plan_linear_dx(a->M, a->N, a->K, es);
  L->dw = plan_linear_dw(a->M, a->N, a->K, es);
  L->dz = c.take(L->store ? (size_t)a->M * L->ld_dz * es : 0);
  L->sums = c.take(a->dbias ? (size_t)((a->M + GRAD_ROWS - 1) / GRAD_ROWS) * a->N * 4 : 0);
  size_t part = 0;
  if (a->dx) part = std::max(part, padded_bytes(L->dx, 1, a->M, a->K));
  if (a->dw) part = std::max(part, padded_bytes(L->dw, 1, a->N, a->K));
  L->part = c.take(part);
  L->total = c.at;
  return SHAMPOO_OK;
}

// C (+)= A B of operands that start on 16 bytes; one launch, and, over ranges
// of k, one for each matrix that sums them (where C is added to, it is its own
// residual).
template <Elem E, bool AS, bool BS, Epi EPI = Epi::STORE>
hipError_t run_product(ProductArgs& g, const Shape& s, const Out& o, float* part, int64_t batch, hipStream_t st) {
  set_shape(g, s);
  point_output(g, s, o, part, batch);
  pad_partials(g, s, batch);
  HIP_TRY_ERR((launch_layer<E, AS, BS, EPI>(g, s, batch, st)));
  if (s.splits == 1) return hipSuccess;
  for (int64_t b = 0; b < batch; ++b) {
    void* C = (unsigned char*)o.C + b * o.strideC * (o.c_dt == 0 ? 4 : 2);
    FinishArgs f{part + b * g.strideC, g.split_stride, s.splits, g.M, g.N, 0, C, o.ldc, o.c_dt, {}};
    f.ffn.residual = o.beta != 0.f ? C : nullptr;
    f.ffn.ld_residual = o.ldc;
    HIP_TRY_ERR(finish_layer(f, st));
  }
  return hipSuccess;
}
// zeros, or the unchanged accumulated gradient, of an empty batch
hipError_t no_gradient(void* p, int64_t ld, int dt, int accumulate, int64_t rows, int64_t cols, hipStream_t st) {
  if (!p || accumulate) return hipSuccess;
  return sum_splits(nullptr, 0, 0, Out{p, ld, 0, out_code(dt), 0, 0.f}, 1, (int)rows, (int)cols, st);
}

template <Elem E, typename T> hipError_t run_linear_grad(const shampoo_linear_grad_args* a, const LinearGradLayout& L, hipStream_t st) {
  unsigned char* ws = (unsigned char*)a->ws;
  if (a->M == 0) {
    HIP_TRY_ERR(no_gradient(a->dw, a->ld_dw, a->dw_dt, a->accumulate, a->N, a->K, st));
    return no_gradient(a->dbias, a->N, a->dbias_dt, a->accumulate, 1, a->N, st);
  }
  const void *dz = a->dy, *x = a->x, *w = a->w;
  if (L.pass) {
    const int64_t chunks = (a->M + GRAD_ROWS - 1) / GRAD_ROWS;
    const bool f8 = a->kept_dt == SHAMPOO_E4M3;
    const ActGradArgs g{a->dy, a->activation ? a->kept : nullptr, (const uint8_t*)a->kept_scale, L.store ? ws + L.dz : nullptr,
                        a->dbias ? (float*)(ws + L.sums) : nullptr, a->ld_dy, f8 ? up(a->N, KEEP_BLOCK) : a->ld_kept, L.ld_dz, (int)a->M, (int)a->N,
                        a->activation, kept_code(a->kept_dt), rows16(a->dy, a->ld_dy, a->dt), rows16(a->kept, a->ld_kept, a->dt),
                        (int)((a->N + 127) / 128)};
    hipLaunchKernelGGL(act_grad_kernel<T>, dim3((unsigned)(chunks * g.blocks)), dim3(256), 0, st, g);
    HIP_TRY_ERR(hipGetLastError());
    if (a->dbias) {
      hipLaunchKernelGGL(bias_grad_kernel, dim3((unsigned)((a->N + 63) / 64)), dim3(1024), 0, st, g.sums, (int)chunks, (int)a->N, a->dbias,
                         out_code(a->dbias_dt), a->accumulate);
      HIP_TRY_ERR(hipGetLastError());
    }
    if (L.store) dz = ws + L.dz;
  }
  float* part = (float*)(ws + L.part);
  if (a->dx) {
    HIP_TRY_ERR(place(L.w, w, nullptr, a->N, a->K, a->ld_w, a->w_dt, a->dt, ws, st));
    ProductArgs g{};
    g.A = dz; g.B = w;
    g.lda = L.ld_dz; g.ldb = L.w.ld;
    g.M = (int)a->M; g.N = (int)a->K; g.K = (int)a->N;
    const Out o{a->dx, a->ld_dx, 0, out_code(a->dt), 1, 0.f};
    HIP_TRY_ERR((run_product<E, false, true>(g, L.dx, o, part, 1, st)));
  }
  if (a->dw) {
    HIP_TRY_ERR(place(L.x, x, a->x_scale, a->M, a->K, a->ld_x, a->x_dt, a->dt, ws, st));
    ProductArgs g{};
    g.A = dz; g.B = x;
    g.lda = L.ld_dz; g.ldb = L.x.ld;
    g.M = (int)a->N; g.N = (int)a->K; g.K = (int)a->M;
    const Out o{a->dw, a->ld_dw, 0, out_code(a->dw_dt), 1, a->accumulate ? 1.f : 0.f};
    HIP_TRY_ERR((run_product<E, true, true>(g, L.dw, o, part, 1, st)));
  }
  return hipSuccess;
}

// ---------------------------------------------------------------------------
// gated block
// ---------------------------------------------------------------------------
struct GatedLayout {
  bool few;
  Operand x, gate, up_, down;
  int64_t ldh;
  Shape in, out;
  size_t h, part, total;
};

// The gate's and the up projection's rows share a stride in the products.
void gated_operands(Carve& c, Operand& gate, Operand& other, const void* wg, const void* wu, int64_t f, int64_t d, int64_t ldg, int64_t ldu, int w_dt,
                    int dt, bool wanted = true) {
  const bool apart = ldg != ldu;
  Carve probe;
  const bool copy = apart || operand(probe, wg, f, d, ldg, w_dt, dt).copy || operand(probe, wu, f, d, ldu, w_dt, dt).copy;
  gate = Operand{copy && wanted, ldg, 0};
  other = Operand{copy && wanted, ldu, 0};
  if (!gate.copy) return;
  gate.ld = other.ld = up(d, 8);
  gate.at = c.take((size_t)f * gate.ld * size_of(dt));
  other.at = c.take((size_t)f * gate.ld * size_of(dt));
}

shampoo_status gated_layout(const shampoo_gated_ffn_args* a, GatedLayout* L) {
  if (!a) return fail(SHAMPOO_E_INVALID, "null arguments");
  shampoo_status r = check_types(a->dt, a->w_dt, a->activation);
  if (r != SHAMPOO_OK) return r;
  if (!one_of(a->y_dt, a->dt, SHAMPOO_F32)) return fail(SHAMPOO_E_UNSUPPORTED, "result dtype %d for dtype %d", (int)a->y_dt, (int)a->dt);
  if ((a->keep_gate == nullptr) != (a->keep_up == nullptr)) return fail(SHAMPOO_E_INVALID, "both projections are kept, or neither");
  if (a->keep_gate && !one_of(a->keep_dt, a->dt, SHAMPOO_E4M3))
    return fail(SHAMPOO_E_UNSUPPORTED, "dtype %d to keep for dtype %d", (int)a->keep_dt, (int)a->dt);
  r = check_sizes(a->T, a->f, a->d);
  if (r != SHAMPOO_OK) return r;
  const int es = (int)size_of(a->dt);
  Carve c;
  L->few = few_rows(a->T, a->keep_gate, a->keep_dt);
  if (L->few) {
    L->ldh = up(a->f, 8);
    L->h = c.take((size_t)FFN_ROWS_MAX * L->ldh * 4);
    L->total = c.at;
    return SHAMPOO_OK;
  }
  L->x = operand(c, a->x, a->T, a->d, a->ld_x, a->dt, a->dt);
  gated_operands(c, L->gate, L->up_, a->w_gate, a->w_up, a->f, a->d, a->ld_gate, a->ld_up, a->w_dt, a->dt);
  L->down = operand(c, a->w_down, a->d, a->f, a->ld_down, a->w_dt, a->dt);
  L->ldh = gated_width(a->f);
  L->in = plan_gated_in(a->T, a->d, a->f, es);
  L->out = plan_gated_out(a->T, a->d, a->f, es, a->residual);
  L->h = c.take((size_t)a->T * L->ldh * es);
  L->part = c.take(std::max(partial_bytes(L->in, 1, a->T, 2 * up(a->f, 4)), padded_bytes(L->out, 1, a->T, a->d)));
  L->total = c.at;
  return SHAMPOO_OK;
}

FfnArgs gated_kept(void* gate, void* gate_scale, void* up_, void* up_scale, int64_t ld, int dt, int64_t f, int act) {
  FfnArgs e{};
  e.keep[0] = gate;
  e.keep[1] = up_;
  e.keep_scale[0] = (uint8_t*)gate_scale;
  e.keep_scale[1] = (uint8_t*)up_scale;
  e.ld_keep = dt == SHAMPOO_E4M3 ? up(f, KEEP_BLOCK) : ld;
  e.keep_dt = kept_code(dt);
  e.scale_vec = up(f, KEEP_BLOCK) % (4 * KEEP_BLOCK) == 0 && aligned(gate_scale, 4) && aligned(up_scale, 4);
  e.act = act;
  return e;
}

template <Elem E> hipError_t run_gated(const shampoo_gated_ffn_args* a, const GatedLayout& L, hipStream_t st) {
  unsigned char* ws = (unsigned char*)a->ws;
  const void *x = a->x, *wg = a->w_gate, *wu = a->w_up, *wd = a->w_down;
  HIP_TRY_ERR(place(L.x, x, nullptr, a->T, a->d, a->ld_x, a->dt, a->dt, ws, st));
  HIP_TRY_ERR(place(L.gate, wg, nullptr, a->f, a->d, a->ld_gate, a->w_dt, a->dt, ws, st));
  HIP_TRY_ERR(place(L.up_, wu, nullptr, a->f, a->d, a->ld_up, a->w_dt, a->dt, ws, st));
  HIP_TRY_ERR(place(L.down, wd, nullptr, a->d, a->f, a->ld_down, a->w_dt, a->dt, ws, st));
  float* part = (float*)(ws + L.part);
  ProductArgs g{};
  g.A = x; g.B = wg; g.B2 = wu;
  g.lda = L.x.ld; g.ldb = L.gate.ld;
  g.M = (int)a->T; g.N = (int)a->f; g.K = (int)a->d;
  set_shape(g, L.in);
  g.C = ws + L.h;
  g.ldc = L.ldh;
  g.c_dt = out_code(a->dt);
  g.vec = 1;
  g.ffn = gated_kept(a->keep_gate, a->keep_gate_scale, a->keep_up, a->keep_up_scale, a->ld_keep, a->keep_dt, a->f, a->activation);
  g.ffn.part = part;
  HIP_TRY_ERR((launch_layer<E, false, false, Epi::GATED>(g, L.in, 1, st)));
  if (L.in.splits > 1) {
    const FinishArgs f{part, 2 * a->T * up(a->f, 4), L.in.splits, (int)a->T, (int)a->f, (int)L.ldh, g.C, L.ldh, g.c_dt, g.ffn};
    hipLaunchKernelGGL(ffn_finish_kernel<true>, dim3((unsigned)((L.ldh + 1023) / 1024), (unsigned)std::min<int64_t>(a->T, 65535)), dim3(256), 0, st, f);
    HIP_TRY_ERR(hipGetLastError());
  }
  FfnArgs e{};
  e.residual = a->residual;
  e.ld_residual = a->ld_residual;
  return run_layer<E>({g.C, wd, L.ldh, L.down.ld, a->T, a->d, a->f, a->y, a->ld_y, a->y_dt, e, L.out, part}, st);
}

hipError_t run_gated_rows(const shampoo_gated_ffn_args* a, const GatedLayout& L, hipStream_t st) {
  const int es = (int)size_of(a->w_dt);
  RowsArgs g{};
  g.x = a->x; g.w = a->w_gate; g.w2 = a->w_up;
  g.y = a->ws;
  g.keep[0] = a->keep_gate; g.keep[1] = a->keep_up;
  g.ldx = a->ld_x; g.ldw = a->ld_gate; g.ldw2 = a->ld_up; g.ldy = L.ldh; g.ld_keep = a->ld_keep;
  g.M = (int)a->T; g.N = (int)a->f; g.K = (int)a->d;
  g.act = a->activation; g.y_dt = 0; g.keep_dt = kept_code(a->keep_dt);
  g.kw = row_waves(a->d);
  g.vec = rows16(a->x, a->ld_x, a->dt) && aligned(a->w_gate, 16) && aligned(a->w_up, 16) && a->ld_gate * es % 16 == 0 && a->ld_up * es % 16 == 0;
  HIP_TRY_ERR(launch_rows_of<true>(g, a->dt, a->w_dt, st));
  RowsArgs o{};
  o.x = a->ws; o.w = a->w_down;
  o.residual = a->residual; o.ld_residual = a->ld_residual;
  o.y = a->y;
  o.ldx = L.ldh; o.ldw = a->ld_down; o.ldy = a->ld_y;
  o.M = (int)a->T; o.N = (int)a->d; o.K = (int)a->f;
  o.y_dt = out_code(a->y_dt);
  o.kw = row_waves(a->f);
  o.vec = rows16(a->w_down, a->ld_down, a->w_dt);
  if (a->dt == SHAMPOO_F32) return launch_rows<float, float, false, false>(o, st);
  if (a->w_dt == SHAMPOO_F32) return launch_rows<float, float, true, false>(o, st);
  return launch_rows<float, uint16_t, false, false>(o, st);
}

// ---------------------------------------------------------------------------
// its gradients
// ---------------------------------------------------------------------------
struct GatedGradLayout {
  Operand dy, x, gate, up_, down;
  int64_t fp;
  bool pair;  // both projections' gradients in one launch
  Shape dh, dx, dwd, dwp;
  size_t D, h, part, total;
};

shampoo_status gated_grad_layout(const shampoo_gated_ffn_grad_args* a, GatedGradLayout* L) {
  if (!a) return fail(SHAMPOO_E_INVALID, "null arguments");
  shampoo_status r = check_types(a->dt, a->w_dt, a->activation);
  if (r != SHAMPOO_OK) return r;
  if ((a->dw_gate || a->dw_up) && !one_of(a->x_dt, a->dt, SHAMPOO_E4M3))
    return fail(SHAMPOO_E_UNSUPPORTED, "x's dtype %d for dtype %d", (int)a->x_dt, (int)a->dt);
  if (!one_of(a->kept_dt, a->dt, SHAMPOO_E4M3)) return fail(SHAMPOO_E_UNSUPPORTED, "kept dtype %d for dtype %d", (int)a->kept_dt, (int)a->dt);
  if (!one_of(a->dw_dt, a->dt, SHAMPOO_F32)) return fail(SHAMPOO_E_UNSUPPORTED, "gradient dtype %d for dtype %d", (int)a->dw_dt, (int)a->dt);
  r = check_sizes(a->T, a->f, a->d);
  if (r != SHAMPOO_OK) return r;
  const int es = (int)size_of(a->dt);
  Carve c;
  L->dy = operand(c, a->dy, a->T, a->d, a->ld_dy, a->dt, a->dt);
  L->x = operand(c, a->x, a->T, a->d, a->ld_x, a->x_dt, a->dt, a->dw_gate || a->dw_up);
  gated_operands(c, L->gate, L->up_, a->w_gate, a->w_up, a->f, a->d, a->ld_gate, a->ld_up, a->w_dt, a->dt, a->dx);
  L->down = operand(c, a->w_down, a->d, a->f, a->ld_down, a->w_dt, a->dt);
  L->fp = gated_width(a->f);
  L->pair = a->dw_gate && a->dw_up && a->ld_dw_gate == a->ld_dw_up;
  L->dh = plan_gated_dh(a->T, a->d, a->f, es);
  L->dx = plan_gated_dx(a->T, a->d, a->f, es);
  L->dwd = plan_gated_dw_down(a->T, a->d, a->f, es);
  L->dwp = plan_gated_dw(a->T, a->d, a->f, es, L->pair);
  L->D = c.take((size_t)a->T * 2 * L->fp * es);
  L->h = c.take((size_t)a->T * L->fp * es);
  size_t part = 0;
  if (a->dx) part = std::max(part, padded_bytes(L->dx, 1, a->T, a->d));
  if (a->dw_down) part = std::max(part, padded_bytes(L->dwd, 1, a->d, a->f));
  if (a->dw_gate || a->dw_up) part = std::max(part, padded_bytes(L->dwp, L->pair ? 2 : 1, a->f, a->d));
  L->part = c.take(part);
  L->total = c.at;
  return SHAMPOO_OK;
}

template <Elem E> hipError_t run_gated_grad(const shampoo_gated_ffn_grad_args* a, const GatedGradLayout& L, hipStream_t st) {
  unsigned char* ws = (unsigned char*)a->ws;
  if (a->T == 0) {
    HIP_TRY_ERR(no_gradient(a->dw_gate, a->ld_dw_gate, a->dw_dt, a->accumulate, a->f, a->d, st));
    HIP_TRY_ERR(no_gradient(a->dw_up, a->ld_dw_up, a->dw_dt, a->accumulate, a->f, a->d, st));
    return no_gradient(a->dw_down, a->ld_dw_down, a->dw_dt, a->accumulate, a->d, a->f, st);
  }
  const int64_t es = (int64_t)size_of(a->dt);
  const void *dy = a->dy, *x = a->x, *wg = a->w_gate, *wu = a->w_up, *wd = a->w_down;
  HIP_TRY_ERR(place(L.dy, dy, nullptr, a->T, a->d, a->ld_dy, a->dt, a->dt, ws, st));
  HIP_TRY_ERR(place(L.down, wd, nullptr, a->d, a->f, a->ld_down, a->w_dt, a->dt, ws, st));
  float* part = (float*)(ws + L.part);
  unsigned char *dg = ws + L.D, *du = dg + L.fp * es, *h = ws + L.h;
  {
    ProductArgs g{};
    g.A = dy; g.B = wd;
    g.lda = L.dy.ld; g.ldb = L.down.ld;
    g.M = (int)a->T; g.N = (int)a->f; g.K = (int)a->d;
    set_shape(g, L.dh);
    g.C = dg;
    g.ldc = 2 * L.fp;
    g.ffn = gated_kept(const_cast<void*>(a->kept_gate), const_cast<void*>(a->kept_gate_scale), const_cast<void*>(a->kept_up),
                       const_cast<void*>(a->kept_up_scale), a->ld_kept, a->kept_dt, a->f, a->activation);
    g.ffn.du = du;
    g.ffn.h = h;
    HIP_TRY_ERR((launch_layer<E, false, true, Epi::GATED_GRAD>(g, L.dh, 1, st)));
  }
  if (a->dx) {
    HIP_TRY_ERR(place(L.gate, wg, nullptr, a->f, a->d, a->ld_gate, a->w_dt, a->dt, ws, st));
    HIP_TRY_ERR(place(L.up_, wu, nullptr, a->f, a->d, a->ld_up, a->w_dt, a->dt, ws, st));
    ProductArgs g{};
    g.A = dg; g.B = wg; g.B2 = wu;
    g.lda = 2 * L.fp; g.ldb = L.gate.ld;
    g.M = (int)a->T; g.N = (int)a->d; g.K = (int)(2 * L.fp);
    g.kswitch = (int)(L.fp * es / 128);
    g.kpart = (int)a->f;
    const Out o{a->dx, a->ld_dx, 0, out_code(a->dt), 1, 0.f};
    HIP_TRY_ERR((run_product<E, false, true, Epi::STORE2>(g, L.dx, o, part, 1, st)));
  }
  const float beta = a->accumulate ? 1.f : 0.f;
  const int c_dt = out_code(a->dw_dt);
  if (a->dw_gate || a->dw_up) {
    HIP_TRY_ERR(place(L.x, x, a->x_scale, a->T, a->d, a->ld_x, a->x_dt, a->dt, ws, st));
    for (int which = 0; which < (L.pair ? 1 : 2); ++which) {
      void* C = which ? a->dw_up : a->dw_gate;
      const int64_t ldc = which ? a->ld_dw_up : a->ld_dw_gate;
      if (!C) continue;
      ProductArgs g{};
      g.A = which ? du : dg; g.B = x;
      g.lda = 2 * L.fp; g.ldb = L.x.ld;
      g.strideA = L.fp;
      g.M = (int)a->f; g.N = (int)a->d; g.K = (int)a->T;
      const int64_t apart = L.pair ? ((const char*)a->dw_up - (const char*)a->dw_gate) / (int64_t)size_of(a->dw_dt) : 0;
      const Out o{C, ldc, apart, c_dt, 1, beta};
      HIP_TRY_ERR((run_product<E, true, true>(g, L.dwp, o, part, L.pair ? 2 : 1, st)));
    }
  }
  if (a->dw_down) {
    ProductArgs g{};
    g.A = dy; g.B = h;
    g.lda = L.dy.ld; g.ldb = L.fp;
    g.M = (int)a->d; g.N = (int)a->f; g.K = (int)a->T;
    const Out o{a->dw_down, a->ld_dw_down, 0, c_dt, 1, beta};
    HIP_TRY_ERR((run_product<E, true, true>(g, L.dwd, o, part, 1, st)));
  }
  return hipSuccess;
}

// Kept values: rows in dt, or blocks of 8 bits with their scales.
shampoo_status check_kept(const char* name, const void* p, const void* scale, int64_t ld, int64_t cols, int dt) {
  if (!p) return SHAMPOO_OK;
  if (dt == SHAMPOO_E4M3) {
    if (!scale) return fail(SHAMPOO_E_INVALID, "%s: values and scales are given together", name);
    if (!aligned(p, 16)) return fail(SHAMPOO_E_INVALID, "%s is misaligned", name);
    return SHAMPOO_OK;
  }
  const Rows r[] = {{name, p, 1, cols, ld, dt}};
  return check_rows(r);
}
Span kept_span(const char* name, const void* p, int64_t rows, int64_t cols, int64_t ld, int dt) {
  return dt == SHAMPOO_E4M3 ? run_of(name, p, rows * up(cols, KEEP_BLOCK)) : rows_of(name, p, rows, cols, ld, dt);
}
Span scale_span(const char* name, const void* p, int64_t rows, int64_t cols, int dt) {
  return run_of(name, dt == SHAMPOO_E4M3 ? p : nullptr, rows * (up(cols, KEEP_BLOCK) / KEEP_BLOCK));
}
// x of a weight's gradient
shampoo_status check_x(const void* x, const void* scale, int64_t ld, int64_t cols, int dt) {
  if (dt != SHAMPOO_E4M3) {
    const Rows r[] = {{"x", x, 1, cols, ld, dt}};
    return check_rows(r);
  }
  if (!scale) return fail(SHAMPOO_E_INVALID, "x: values and scales are given together");
  if (!aligned(x, 16)) return fail(SHAMPOO_E_INVALID, "x is misaligned");
  return SHAMPOO_OK;
}
Span x_span(const void* x, int64_t rows, int64_t cols, int64_t ld, int dt) {
  return dt == SHAMPOO_E4M3 ? run_of("x", x, rows * up(cols, 128)) : rows_of("x", x, rows, cols, ld, dt);
}
Span x_scale_span(const void* s, int64_t rows, int64_t cols, int dt) {
  return run_of("x_scale", dt == SHAMPOO_E4M3 ? s : nullptr, rows * up(up(cols, 128) / 128, 4));
}

template <typename A, typename L> shampoo_status workspace_of(const A* a, size_t* bytes, shampoo_status (*layout)(const A*, L*)) {
  if (!bytes) return fail(SHAMPOO_E_INVALID, "null pointer argument");
  L l{};
  const shampoo_status r = layout(a, &l);
  if (r != SHAMPOO_OK) return r;
  *bytes = l.total;
  return SHAMPOO_OK;
}

}  // namespace

extern "C" {

shampoo_status shampoo_linear_workspace(const shampoo_linear_args* args, size_t* bytes) { return workspace_of(args, bytes, linear_layout); }

shampoo_status shampoo_linear(const shampoo_linear_args* a, hipStream_t stream) {
  LinearLayout L{};
  shampoo_status r = linear_layout(a, &L);
  if (r != SHAMPOO_OK) return r;
  if (a->M == 0) return SHAMPOO_OK;
  if (!a->x || !a->w || !a->y) return fail(SHAMPOO_E_INVALID, "null pointer argument");
  const Rows rows[] = {{"y", a->y, a->M, a->N, a->ld_y, a->y_dt},
                       {"x", a->x, a->M, a->K, a->ld_x, a->dt},
                       {"w", a->w, a->N, a->K, a->ld_w, a->w_dt},
                       {"residual", a->residual, a->M, a->N, a->ld_residual, a->y_dt},
                       {"bias", a->bias, 1, a->N, a->N, a->bias_dt}};
  r = check_rows(rows);
  if (r == SHAMPOO_OK) r = check_kept("keep", a->keep, a->keep_scale, a->ld_keep, a->N, a->keep_dt);
  if (r == SHAMPOO_OK) r = check_ws(a->ws, a->ws_bytes, L.total);
  if (r != SHAMPOO_OK) return r;
  const bool in_place = a->residual == a->y && a->ld_residual == a->ld_y;
  const Span spans[] = {span_of(rows[0]),
                        kept_span("keep", a->keep, a->M, a->N, a->ld_keep, a->keep_dt),
                        scale_span("keep's scales", a->keep ? a->keep_scale : nullptr, a->M, a->N, a->keep_dt),
                        run_of("the workspace", a->ws, (int64_t)L.total),
                        span_of(rows[1]),
                        span_of(rows[2]),
                        in_place ? run_of("residual", nullptr, 0) : span_of(rows[3]),
                        span_of(rows[4])};
  r = check_apart(spans, 4);
  if (r != SHAMPOO_OK) return r;
  if (L.few) {
    RowsArgs g{};
    g.x = a->x; g.w = a->w; g.bias = a->bias; g.residual = a->residual; g.y = a->y;
    g.keep[0] = a->keep;
    g.ldx = a->ld_x; g.ldw = a->ld_w; g.ld_residual = a->ld_residual; g.ldy = a->ld_y; g.ld_keep = a->ld_keep;
    g.M = (int)a->M; g.N = (int)a->N; g.K = (int)a->K;
    g.act = a->activation; g.y_dt = out_code(a->y_dt); g.keep_dt = kept_code(a->keep_dt);
    g.bias_bf16 = a->bias_dt == SHAMPOO_BF16;
    g.kw = row_waves(a->K);
    g.vec = rows16(a->x, a->ld_x, a->dt) && rows16(a->w, a->ld_w, a->w_dt);
    HIP_TRY(launch_rows_of<false>(g, a->dt, a->w_dt, stream));
    return SHAMPOO_OK;
  }
  FfnArgs e{};
  e.bias = a->bias;
  e.bias_bf16 = a->bias_dt == SHAMPOO_BF16;
  e.residual = a->residual;
  e.ld_residual = a->ld_residual;
  e.keep[0] = a->keep;
  e.keep_scale[0] = (uint8_t*)a->keep_scale;
  e.ld_keep = a->keep_dt == SHAMPOO_E4M3 ? up(a->N, KEEP_BLOCK) : a->ld_keep;
  e.keep_dt = kept_code(a->keep_dt);
  e.scale_vec = up(a->N, KEEP_BLOCK) % (4 * KEEP_BLOCK) == 0 && aligned(a->keep_scale, 4);
  e.act = a->activation;
  HIP_TRY(a->dt == SHAMPOO_F32 ? run_linear<Elem::F32>(a, L, e, stream) : run_linear<Elem::BF16>(a, L, e, stream));
  return SHAMPOO_OK;
}

shampoo_status shampoo_linear_grad_workspace(const shampoo_linear_grad_args* args, size_t* bytes) {
  return workspace_of(args, bytes, linear_grad_layout);
}

shampoo_status shampoo_linear_grad(const shampoo_linear_grad_args* a, hipStream_t stream) {
  LinearGradLayout L{};
  shampoo_status r = linear_grad_layout(a, &L);
  if (r != SHAMPOO_OK) return r;
  if (!a->dx && !a->dw && !a->dbias) return fail(SHAMPOO_E_INVALID, "no output");
  if (a->M > 0 && (!a->dy || (a->dx && !a->w) || (a->dw && !a->x) || (a->activation && !a->kept)))
    return fail(SHAMPOO_E_INVALID, "null pointer argument");
  const bool x = a->dw && a->M > 0, kept = a->activation != 0 && a->M > 0;
  const Rows rows[] = {{"dx", a->M ? a->dx : nullptr, a->M, a->K, a->ld_dx, a->dt},
                       {"dw", a->dw, a->N, a->K, a->ld_dw, a->dw_dt},
                       {"dbias", a->dbias, 1, a->N, a->N, a->dbias_dt},
                       {"dy", a->M ? a->dy : nullptr, a->M, a->N, a->ld_dy, a->dt},
                       {"w", a->dx && a->M ? a->w : nullptr, a->N, a->K, a->ld_w, a->w_dt}};
  r = check_rows(rows);
  if (r == SHAMPOO_OK && kept) r = check_kept("kept", a->kept, a->kept_scale, a->ld_kept, a->N, a->kept_dt);
  if (r == SHAMPOO_OK && x) r = check_x(a->x, a->x_scale, a->ld_x, a->K, a->x_dt);
  if (r == SHAMPOO_OK) r = check_ws(a->ws, a->ws_bytes, L.total);
  if (r != SHAMPOO_OK) return r;
  const Span spans[] = {span_of(rows[0]), span_of(rows[1]), span_of(rows[2]), run_of("the workspace", a->ws, (int64_t)L.total), span_of(rows[3]),
                        span_of(rows[4]), kept_span("kept", kept ? a->kept : nullptr, a->M, a->N, a->ld_kept, a->kept_dt),
                        scale_span("kept's scales", kept ? a->kept_scale : nullptr, a->M, a->N, a->kept_dt),
                        x_span(x ? a->x : nullptr, a->M, a->K, a->ld_x, a->x_dt),
                        x_scale_span(x ? a->x_scale : nullptr, a->M, a->K, a->x_dt)};
  r = check_apart(spans, 4);
  if (r != SHAMPOO_OK) return r;
  HIP_TRY(a->dt == SHAMPOO_F32 ? (run_linear_grad<Elem::F32, float>(a, L, stream)) : (run_linear_grad<Elem::BF16, uint16_t>(a, L, stream)));
  return SHAMPOO_OK;
}

shampoo_status shampoo_gated_ffn_workspace(const shampoo_gated_ffn_args* args, size_t* bytes) { return workspace_of(args, bytes, gated_layout); }

shampoo_status shampoo_gated_ffn(const shampoo_gated_ffn_args* a, hipStream_t stream) {
  GatedLayout L{};
  shampoo_status r = gated_layout(a, &L);
  if (r != SHAMPOO_OK) return r;
  if (a->T == 0) return SHAMPOO_OK;
  if (!a->x || !a->w_gate || !a->w_up || !a->w_down || !a->y) return fail(SHAMPOO_E_INVALID, "null pointer argument");
  const Rows rows[] = {{"y", a->y, a->T, a->d, a->ld_y, a->y_dt},
                       {"x", a->x, a->T, a->d, a->ld_x, a->dt},
                       {"w_gate", a->w_gate, a->f, a->d, a->ld_gate, a->w_dt},
                       {"w_up", a->w_up, a->f, a->d, a->ld_up, a->w_dt},
                       {"w_down", a->w_down, a->d, a->f, a->ld_down, a->w_dt},
                       {"residual", a->residual, a->T, a->d, a->ld_residual, a->y_dt}};
  r = check_rows(rows);
  if (r == SHAMPOO_OK) r = check_kept("keep_gate", a->keep_gate, a->keep_gate_scale, a->ld_keep, a->f, a->keep_dt);
  if (r == SHAMPOO_OK) r = check_kept("keep_up", a->keep_up, a->keep_up_scale, a->ld_keep, a->f, a->keep_dt);
  if (r == SHAMPOO_OK) r = check_ws(a->ws, a->ws_bytes, L.total);
  if (r != SHAMPOO_OK) return r;
  const bool in_place = a->residual == a->y && a->ld_residual == a->ld_y;
  const Span spans[] = {span_of(rows[0]),
                        kept_span("keep_gate", a->keep_gate, a->T, a->f, a->ld_keep, a->keep_dt),
                        kept_span("keep_up", a->keep_up, a->T, a->f, a->ld_keep, a->keep_dt),
                        scale_span("keep_gate's scales", a->keep_gate ? a->keep_gate_scale : nullptr, a->T, a->f, a->keep_dt),
                        scale_span("keep_up's scales", a->keep_up ? a->keep_up_scale : nullptr, a->T, a->f, a->keep_dt),
                        run_of("the workspace", a->ws, (int64_t)L.total),
                        span_of(rows[1]),
                        span_of(rows[2]),
                        span_of(rows[3]),
                        span_of(rows[4]),
                        in_place ? run_of("residual", nullptr, 0) : span_of(rows[5])};
  r = check_apart(spans, 6);
  if (r != SHAMPOO_OK) return r;
  HIP_TRY(L.few ? run_gated_rows(a, L, stream)
                : a->dt == SHAMPOO_F32 ? run_gated<Elem::F32>(a, L, stream) : run_gated<Elem::BF16>(a, L, stream));
  return SHAMPOO_OK;
}

shampoo_status shampoo_gated_ffn_grad_workspace(const shampoo_gated_ffn_grad_args* args, size_t* bytes) {
  return workspace_of(args, bytes, gated_grad_layout);
}

shampoo_status shampoo_gated_ffn_grad(const shampoo_gated_ffn_grad_args* a, hipStream_t stream) {
  GatedGradLayout L{};
  shampoo_status r = gated_grad_layout(a, &L);
  if (r != SHAMPOO_OK) return r;
  if (!a->dx && !a->dw_gate && !a->dw_up && !a->dw_down) return fail(SHAMPOO_E_INVALID, "no output");
  const bool any = a->T > 0, x = any && (a->dw_gate || a->dw_up);
  if (any && (!a->dy || !a->w_down || !a->kept_gate || !a->kept_up || (a->dx && (!a->w_gate || !a->w_up)) || (x && !a->x)))
    return fail(SHAMPOO_E_INVALID, "null pointer argument");
  const bool w = any && a->dx;
  const Rows rows[] = {{"dx", any ? a->dx : nullptr, a->T, a->d, a->ld_dx, a->dt},
                       {"dw_gate", a->dw_gate, a->f, a->d, a->ld_dw_gate, a->dw_dt},
                       {"dw_up", a->dw_up, a->f, a->d, a->ld_dw_up, a->dw_dt},
                       {"dw_down", a->dw_down, a->d, a->f, a->ld_dw_down, a->dw_dt},
                       {"dy", any ? a->dy : nullptr, a->T, a->d, a->ld_dy, a->dt},
                       {"w_gate", w ? a->w_gate : nullptr, a->f, a->d, a->ld_gate, a->w_dt},
                       {"w_up", w ? a->w_up : nullptr, a->f, a->d, a->ld_up, a->w_dt},
                       {"w_down", any ? a->w_down : nullptr, a->d, a->f, a->ld_down, a->w_dt}};
  r = check_rows(rows);
  if (r == SHAMPOO_OK && any) r = check_kept("kept_gate", a->kept_gate, a->kept_gate_scale, a->ld_kept, a->f, a->kept_dt);
  if (r == SHAMPOO_OK && any) r = check_kept("kept_up", a->kept_up, a->kept_up_scale, a->ld_kept, a->f, a->kept_dt);
  if (r == SHAMPOO_OK && x) r = check_x(a->x, a->x_scale, a->ld_x, a->d, a->x_dt);
  if (r == SHAMPOO_OK) r = check_ws(a->ws, a->ws_bytes, L.total);
  if (r != SHAMPOO_OK) return r;
  const Span spans[] = {span_of(rows[0]), span_of(rows[1]), span_of(rows[2]), span_of(rows[3]), run_of("the workspace", a->ws, (int64_t)L.total),
                        span_of(rows[4]), span_of(rows[5]), span_of(rows[6]), span_of(rows[7]),
                        kept_span("kept_gate", any ? a->kept_gate : nullptr, a->T, a->f, a->ld_kept, a->kept_dt),
                        kept_span("kept_up", any ? a->kept_up : nullptr, a->T, a->f, a->ld_kept, a->kept_dt),
                        scale_span("kept_gate's scales", any ? a->kept_gate_scale : nullptr, a->T, a->f, a->kept_dt),
                        scale_span("kept_up's scales", any ? a->kept_up_scale : nullptr, a->T, a->f, a->kept_dt),
                        x_span(x ? a->x : nullptr, a->T, a->d, a->ld_x, a->x_dt),
                        x_scale_span(x ? a->x_scale : nullptr, a->T, a->d, a->x_dt)};
  r = check_apart(spans, 5);
  if (r != SHAMPOO_OK) return r;
  HIP_TRY(a->dt == SHAMPOO_F32 ? run_gated_grad<Elem::F32>(a, L, stream) : run_gated_grad<Elem::BF16>(a, L, stream));
  return SHAMPOO_OK;
}

}  // extern "C"
