// Row passes of the projection's softmax cross entropy (gfx950); the products
// are in product_core.hpp.
//
// With logits z = x W^T, the product's epilogue leaves for each row and each
// piece of 128 columns the maximum m_j and s_j = sum exp(z - m_j), for the row
// its target's logit z_t, and, for gradients, E = exp(z - m_j).  Then
//     M = max_j m_j,  s = sum_j s_j exp(m_j - M),  lse = M + log s,
//     loss = (M - z_t) + log s,
//     P = g (softmax - onehot) = E g exp(m_j - M) / s, and g (exp(-loss) - 1) at t.
// Nothing large is subtracted: M - z_t is a difference of two logits of the
// same sum (zero where the target leads), s at least 1, so a loss is never
// negative and keeps its digits where the target's probability is near one.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gemm_common.hpp"

namespace shampoo {

typedef float floatx2_t __attribute__((ext_vector_type(2)));

// 1 / max(number of rows whose target is kept, 1)
__global__ __launch_bounds__(1024) void xent_count_kernel(const int64_t* __restrict__ targets, int N, int64_t ignore,
                                                          float* __restrict__ inv_count) {
  __shared__ int red[16];
  int c = 0;
  for (int i = threadIdx.x; i < N; i += 1024) c += targets[i] != ignore;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) c += __shfl_xor(c, d);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = c;
  __syncthreads();
  if (threadIdx.x == 0) {
    int t = 0;
    for (int w = 0; w < 16; ++w) t += red[w];
    *inv_count = 1.0f / (float)max(t, 1);
  }
}

struct RowArgs {
  const floatx2_t* stats;      // [pieces][M]
  float* nll;                  // [M]: the target's logit; replaced by -log of its probability
  const int64_t* targets;      // [M]
  const float* row_scale;      // [M] or null
  floatx2_t* norm;             // [M]: (M, 1 / s)
  float* lse;                  // [M] or null
  float* loss;                 // [M] (times row_scale and scale)
  int64_t ignore;
  int M, V, pieces;
  float scale;
};

// R rows per workgroup of 1024 threads: thread t joins pieces t / R, + 1024 /
// R, ... of row t % R.  Bound by the latency of its reads: 8192 rows of 1024 pieces (67 MB) 25
// us; one row of 256 pieces 3.9 us.
template <int R>
__global__ __launch_bounds__(1024) void xent_rows_kernel(RowArgs g) {
  __shared__ floatx2_t red[1024];
  const int tid = threadIdx.x, lr = tid % R, grp = tid / R;
  constexpr int G = 1024 / R;
  const int m = blockIdx.x * R + lr;
  float mx = -INFINITY, s = 0.f;
  if (m < g.M) {
#pragma unroll 8
    for (int p = grp; p < g.pieces; p += G) {
      const floatx2_t v = g.stats[(int64_t)p * g.M + m];
      const float nm = fmaxf(mx, v[0]);
      const float ref = nm == -INFINITY ? 0.f : nm;
      s = s * __expf(mx - ref) + v[1] * __expf(v[0] - ref);
      mx = nm;
    }
  }
  red[tid] = floatx2_t{mx, s};
  __syncthreads();
  for (int d = G / 2; d > 0; d /= 2) {
    if (grp < d) {
      const floatx2_t o = red[tid + d * R];
      const float nm = fmaxf(mx, o[0]);
      const float ref = nm == -INFINITY ? 0.f : nm;
      s = s * __expf(mx - ref) + o[1] * __expf(o[0] - ref);
      mx = nm;
      red[tid] = floatx2_t{mx, s};
    }
    __syncthreads();
  }
  if (grp == 0 && m < g.M) {
    const float ls = logf(s);
    g.norm[m] = floatx2_t{mx, 1.f / s};
    if (g.lse) g.lse[m] = mx + ls;
    const int64_t t = g.targets[m];
    float l = 0.f;
    if (t != g.ignore) {
      const float nll = t >= 0 && t < g.V ? (mx - g.nll[m]) + ls : __builtin_nanf("");
      g.nll[m] = nll;
      l = nll * (g.scale * (g.row_scale ? g.row_scale[m] : 1.f));
    }
    g.loss[m] = l;
  }
}

// Sum of the row losses (float64, fixed order), times 1 / count for the mean
// (inv_count not null): read from there, or, with `targets` (for the mean
// only), counted here and left there, which saves a call of one panel the
// counting launch.
__global__ __launch_bounds__(1024) void xent_reduce_kernel(const float* __restrict__ rows, const int64_t* __restrict__ targets, int N,
                                                           int64_t ignore, float* __restrict__ inv_count, float* __restrict__ out) {
  __shared__ double red[16];
  __shared__ int kept[16];
  double a = 0.0;
  int c = 0;
  for (int i = threadIdx.x; i < N; i += 1024) {
    a += (double)rows[i];
    if (targets) c += targets[i] != ignore;
  }
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    a += __shfl_xor(a, d);
    c += __shfl_xor(c, d);
  }
  if ((threadIdx.x & 63) == 0) {
    red[threadIdx.x >> 6] = a;
    kept[threadIdx.x >> 6] = c;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    double t = 0.0;
    int k = 0;
    for (int w = 0; w < 16; ++w) {
      t += red[w];
      k += kept[w];
    }
    if (targets && inv_count) *inv_count = 1.0f / (float)max(k, 1);
    *out = (float)(inv_count ? t * (double)*inv_count : t);
  }
}

struct GradArgs {
  void* E;                    // [M][ld], in place
  int64_t ld;
  const floatx2_t* stats;     // [pieces][M]
  const float* nll;
  const floatx2_t* norm;
  const int64_t* targets;
  const float* row_scale;
  int64_t ignore;
  int M, V, pieces;
  const void* hidden;         // [M][ldh], 16-byte aligned rows
  int64_t ldh;
  void* kept;                 // [M][ldk]; may be hidden itself
  int64_t ldk;
  int d, first;               // d entries, by the workgroups from `first` on
};

// P from E, in place: a workgroup of 4 waves takes 4 rows x 2048 columns, 16
// bytes a lane at a time.  Bound by memory: 8192 x 131072 (2.1 GB read and
// written) 0.77-0.87 ms = 4.9-5.6 TB/s.  It cannot join the product that makes E: a
// row's lse is known only after all of its pieces.  T: float, or uint16_t for bfloat16.
// Workgroups from `first` on leave hidden's rows for the weight's gradient,
// zeros where the target is ignored: a zero of P times a NaN or an infinity in
// a padding row would be NaN in every row of that gradient.
template <typename T>
__global__ __launch_bounds__(256) void xent_grad_kernel(GradArgs g) {
  constexpr int VE = 16 / sizeof(T);
  const int m = blockIdx.y * 4 + (threadIdx.x >> 6), lane = threadIdx.x & 63;
  if (m >= g.M) return;
  const int64_t t = g.targets[m];
  const bool skip = t == g.ignore, bad = !skip && (t < 0 || t >= g.V);
  if ((int)blockIdx.x >= g.first) {
    const T* from = reinterpret_cast<const T*>(g.hidden) + (int64_t)m * g.ldh;
    T* to = reinterpret_cast<T*>(g.kept) + (int64_t)m * g.ldk;
    if (!skip && from == to) return;
#pragma unroll
    for (int u = 0; u < 2048 / (64 * VE); ++u) {
      const int c = ((int)blockIdx.x - g.first) * 2048 + (u * 64 + lane) * VE;
      if (c < g.d) *reinterpret_cast<u32x4*>(to + c) = skip ? u32x4{0, 0, 0, 0} : *reinterpret_cast<const u32x4*>(from + c);
    }
    return;
  }
  // 1 / count and the caller's scale wait for the products' float32 results:
  // here they would round every -1 of an unlikely target the same way.  The
  // rows' own scales do so in bfloat16: the gradients are 2.2e-3 from float64
  // instead of 2.0e-3 (their own rounding 1.7e-3).  Kept apart, in dhidden's float32
  // rows and hidden's copy, they would cost dweight a rounding of that copy:
  // emulated, dhidden 2.0e-3 and dweight 2.6e-3.
  float w = g.row_scale ? g.row_scale[m] : 1.f;
  if (bad) w = __builtin_nanf("");
  const floatx2_t norm = g.norm[m];
  T* row = reinterpret_cast<T*>(g.E) + (int64_t)m * g.ld;
#pragma unroll
  for (int u = 0; u < 2048 / (64 * VE); ++u) {
    const int c = blockIdx.x * 2048 + (u * 64 + lane) * VE;
    if (c >= g.ld || c >= g.pieces * 128) continue;
    u32x4 out = u32x4{0, 0, 0, 0};
    if (!skip) {
      const float f = w * (__expf(g.stats[(int64_t)(c >> 7) * g.M + m][0] - norm[0]) * norm[1]);
      const u32x4 in = *reinterpret_cast<const u32x4*>(row + c);
      struct Pack { T v[VE]; };
      Pack p = __builtin_bit_cast(Pack, in);
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        float y;
        if constexpr (sizeof(T) == 4) y = p.v[e];
        else y = __builtin_bit_cast(float, (uint32_t)p.v[e] << 16);
        // a piece of nothing (maximum -inf) holds zeros
        y = y == 0.f ? (f == f ? 0.f : f) : y * f;
        // p_t - 1 from the loss: the difference would lose it where p_t is near one
        if (c + e == t) y = w * expm1f(-g.nll[m]);
        if (c + e >= g.V) y = 0.f;
        if constexpr (sizeof(T) == 4) p.v[e] = y;
        else p.v[e] = __builtin_bit_cast(uint16_t, (__bf16)y);
      }
      out = __builtin_bit_cast(u32x4, p);
    }
    *reinterpret_cast<u32x4*>(row + c) = out;
  }
}

// C = alpha x the sum of `splits` float32 partial results (+ beta C), any output type
// (0 float32, 1 half, 2 bfloat16); rows of N elements, ldc apart, batches of M
// rows.  2^tx threads of a workgroup go along a row, 4 columns each (vec: N
// and the rows' starts allow 16-byte accesses); the others take further rows.
__global__ __launch_bounds__(256) void sum_splits_kernel(const float* __restrict__ part, int splits, int64_t split_stride,
                                                         void* __restrict__ C, int64_t ldc, int64_t strideC, int M, int N,
                                                         int c_dt, float alpha, const float* __restrict__ alpha_dev, float beta, int tx,
                                                         int vec) {
  if (alpha_dev) alpha *= *alpha_dev;
  const int64_t b = blockIdx.z;
  const int n = 4 * ((int)(threadIdx.x & ((1 << tx) - 1)) + ((int)blockIdx.x << tx));
  if (n >= N) return;
  for (int m = (blockIdx.y << (8 - tx)) + (threadIdx.x >> tx); m < M; m += gridDim.y << (8 - tx)) {
    const float* p = part + (b * M + m) * (int64_t)N + n;
    float a[4] = {0.f, 0.f, 0.f, 0.f};
    if (vec) {
#pragma unroll 4
      for (int s = 0; s < splits; ++s) {
        const floatx4 v = *reinterpret_cast<const floatx4*>(p + s * split_stride);
#pragma unroll
        for (int e = 0; e < 4; ++e) a[e] += v[e];
      }
    } else {
      for (int s = 0; s < splits; ++s)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (n + e < N) a[e] += p[s * split_stride + e];
    }
    const int64_t at = b * strideC + m * ldc + n;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (n + e >= N) break;
      if (c_dt == 0) {
        float* o = reinterpret_cast<float*>(C) + at + e;
        *o = alpha * a[e] + (beta != 0.f ? beta * *o : 0.f);
      } else if (c_dt == 1) {
        _Float16* o = reinterpret_cast<_Float16*>(C) + at + e;
        *o = (_Float16)(alpha * a[e] + (beta != 0.f ? beta * (float)*o : 0.f));
      } else {
        __bf16* o = reinterpret_cast<__bf16*>(C) + at + e;
        *o = (__bf16)(alpha * a[e] + (beta != 0.f ? beta * (float)*o : 0.f));
      }
    }
  }
}

// Rows of `cols` elements, ld apart, as rows of ldo elements (a multiple of
// 8) with zeros behind: an operand whose rows do not start on 16 bytes, or a
// float32 weight rounded to bfloat16.  TI, TO: float, or uint16_t for
// bfloat16.  A wave takes a row at a time, 4 elements a lane.
template <typename TI, typename TO>
__global__ __launch_bounds__(256) void pad_rows_kernel(const TI* __restrict__ x, int64_t ld, int64_t rows, int cols, TO* __restrict__ o,
                                                       int ldo, int vec) {
  struct Four { TI v[4]; };
  struct Out { TO v[4]; };
  auto turn = [](TI v) -> TO {
    if constexpr (sizeof(TI) == sizeof(TO)) return v;
    else return __builtin_bit_cast(uint16_t, (__bf16)v);
  };
  const int lane = threadIdx.x & 63;
  for (int64_t r = blockIdx.x * (int64_t)4 + (threadIdx.x >> 6); r < rows; r += (int64_t)gridDim.x * 4) {
    const TI* from = x + r * ld;
    TO* to = o + r * ldo;
    for (int c = 4 * lane; c < ldo; c += 256) {
      Out w;
      if (vec && c + 4 <= cols) {
        const Four f = *reinterpret_cast<const Four*>(from + c);
#pragma unroll
        for (int e = 0; e < 4; ++e) w.v[e] = turn(f.v[e]);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) w.v[e] = c + e < cols ? turn(from[c + e]) : TO(0);
      }
      *reinterpret_cast<Out*>(to + c) = w;
    }
  }
}

}  // namespace shampoo
