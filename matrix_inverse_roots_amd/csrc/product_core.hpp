// Rectangular matrix product on CDNA4 matrix cores (gfx950) for the 8-bit
// block-scaled product and the projection's softmax cross entropy.
//
//     C[m, n] = sum_k A(m, k) B(n, k)
//
// Element types: bfloat16 (v_mfma_f32_32x32x16_bf16), float32
// (v_mfma_f32_32x32x2_f32) and 8-bit floating point with a power-of-two
// scale for each block of 128 k (v_mfma_scale_f32_32x32x64_f8f6f4, which
// applies the scales to the operands' exponents inside the matrix core: no
// instruction is spent on them).  Accumulation is float32 throughout.
//
// Operand layouts.  "k-contiguous": row r at r * ld, k along the row.
// "k-strided" (template flags AS, BS; bfloat16 and float32): element (r, k)
// at k * ld + r, an operand read as its transpose.
//
// Structure.  One workgroup of WM x WN waves computes a tile of
// 32 FM WM x 32 FN WN outputs; workgroups are persistent and walk the tiles
// of their XCD's share, so that the loads of the next tile run through the
// end of the current one.  A stage is 64 bytes of k of every row of both
// operands; stages go straight to LDS (global_load_lds, 16 bytes a lane)
// into a ring of NS buffers.  Each wave reads the fragments of stage s + 1
// into registers while the matrix cores work on stage s, so that stage s's
// buffer is free by then and takes stage s + NS; one barrier per stage, which
// a wave enters with its LDS reads done.
//
// LDS layouts, conflict-free for the reads (16 lanes of a ds_read_b128 are
// served together: lanes 0-3, 12-15, 20-23, 24-27 of each 32):
//   k-contiguous: rows of 64 bytes, 16-byte chunk c of row r at
//     c ^ ((r >> 2) & 3); lane l reads row l % 32, chunks h and 2 + h of the
//     row, h = l / 32.  A fragment is 32 bytes a lane: the k a lane holds are
//     the same for both operands, which is all a dot product needs.
//   k-strided bfloat16: k-rows of the tile's width, chunk c of k-row k at
//     c ^ 4 (k & 3); fragments come from ds_read_b64_tr_b16, which gives lane
//     j of 16 column j of 4 k-rows.
//   k-strided float32: chunk c of k-row k at c ^ 8 ((k >> 2) & 1); fragments
//     come from 4-byte reads.
// The matrix-core operands are swapped (the B side feeds the first operand),
// so that lane l holds row l % 32 of a 32 x 32 block of C and, in value v,
// column 8 (v / 4) + 4 (l / 32) + v % 4: runs of 4 consecutive columns.
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

// What a chunk outside an operand reads (16 bytes of zeros).
__device__ __attribute__((aligned(16))) static const uint32_t product_zeros[4] = {0, 0, 0, 0};

enum class Elem { BF16, F32, F8 };
enum class Epi { STORE, SOFTMAX };

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
  int nst;                            // k-stages (even; F8: a multiple of 8 or the last range's rest)
  int splits, split_stages;           // ranges of k; stages of each but the last
  int c_dt;                           // 0 float32, 1 half, 2 bfloat16
  int vec;                            // rows of C allow 16-byte stores
  float beta;                         // C = acc + beta C (STORE)
  int64_t items;                      // batch * splits * mt * nt
  // SOFTMAX
  floatx2* stats;                     // [pieces][M]: (max, sum of exp(z - max)) of 128 columns
  float* target_logit;                // [M]
  const int64_t* targets;             // [M]
};

template <Elem E> struct ElemTraits;
template <> struct ElemTraits<Elem::BF16> { static constexpr int size = 2; };
template <> struct ElemTraits<Elem::F32> { static constexpr int size = 4; };
template <> struct ElemTraits<Elem::F8> { static constexpr int size = 1; };

// By value: __builtin_bit_cast of a vector's element reads element 0.
__device__ __forceinline__ float bits_float(uint32_t b) { return __builtin_bit_cast(float, b); }
__device__ __forceinline__ uint32_t float_bits(float f) { return __builtin_bit_cast(uint32_t, f); }

// acc += B fragment x A fragment over one stage (64 bytes of k)
template <Elem E, int FB, int FA>
__device__ __forceinline__ floatx16 stage_mma(intx8 b, intx8 a, floatx16 acc, int scb, int sca) {
  if constexpr (E == Elem::F8) {
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(b, a, acc, FB, FA, 0, scb, 0, sca);
  } else if constexpr (E == Elem::BF16) {
    struct Two { bf16x8 v[2]; };
    const Two bb = __builtin_bit_cast(Two, b), aa = __builtin_bit_cast(Two, a);
    acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(bb.v[0], aa.v[0], acc, 0, 0, 0);
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(bb.v[1], aa.v[1], acc, 0, 0, 0);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      acc = __builtin_amdgcn_mfma_f32_32x32x2f32(bits_float(b[j]), bits_float(a[j]), acc, 0, 0, 0);
    return acc;
  }
}

// wait until at most K vector memory operations of this wave are in flight,
// and none of its LDS reads
template <int K> __device__ __forceinline__ void wait_stage() {
  static_assert(K >= 0 && K < 64, "vmcnt has 6 bits");
  __builtin_amdgcn_s_waitcnt((K & 15) | (0x7 << 4) | ((K >> 4) << 14));
}

__device__ __forceinline__ uint32_t pack_bf16(float x, float y) {
  typedef __bf16 b2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, b2{(__bf16)x, (__bf16)y});
}
__device__ __forceinline__ uint32_t pack_f16(float x, float y) {
  typedef _Float16 h2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, h2{(_Float16)x, (_Float16)y});
}

template <Elem E, int FM, int FN, int WM, int WN, int NS, bool AS, bool BS, Epi EPI, int FA, int FB>
__global__ __launch_bounds__(64 * WM * WN, 2) void product_kernel(ProductArgs g) {
  constexpr int ES = ElemTraits<E>::size;
  constexpr int W = WM * WN, TM = 32 * FM * WM, TN = 32 * FN * WN;
  constexpr int OPA = TM * 64, STAGE = (TM + TN) * 64;
  constexpr int NIA = TM / 16 / W, NIB = TN / 16 / W, NI = NIA + NIB;
  constexpr int SK = 64 / ES;  // k of one stage
  static_assert(NIA * W * 16 == TM && NIB * W * 16 == TN, "loads divide among the waves");
  static_assert(E != Elem::F8 || (!AS && !BS), "8-bit operands are k-contiguous");
  static_assert(!(AS && TM < 64) && !(BS && TN < 64), "k-strided swizzles need 64 columns");
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];

  // this workgroup's items: the XCD's contiguous share, dealt round-robin
  const int per = gridDim.x >> 3;
  const int xcd = blockIdx.x & 7, slot = blockIdx.x >> 3;
  const int64_t q8 = g.items >> 3, r8 = g.items & 7;
  const int64_t mine = q8 + (xcd < r8 ? 1 : 0);
  if (mine <= slot) return;
  const int64_t first = xcd * q8 + (xcd < r8 ? xcd : r8) + slot;
  const int nitem = (int)((mine - slot + per - 1) / per);

  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int l32 = lane & 31, half = lane >> 5;

  struct Item { int64_t batch; int split, tm, tn, k0, stages; };
  // tiles in bands of 8 rows of tiles, column by column: the tiles that run
  // at the same time on an XCD share the operands' panels in its L2
  auto item_of = [&](int it) {
    Item r;
    int64_t w = first + (int64_t)it * per;
    const int tiles = g.mt * g.nt;
    const int64_t bs = w / tiles;
    int t = (int)(w - bs * tiles);
    r.batch = bs / g.splits;
    r.split = (int)(bs - r.batch * g.splits);
    const int band = t / (8 * g.nt), rows = min(8, g.mt - 8 * band);
    t -= band * 8 * g.nt;
    r.tm = 8 * band + t % rows;
    r.tn = t / rows;
    r.k0 = r.split * g.split_stages;
    r.stages = min(g.split_stages, g.nst - r.k0);
    return r;
  };

  // ---- loads -------------------------------------------------------------
  const unsigned char* LA;
  const unsigned char* LB;
  uint32_t offA[NIA], offB[NIB];
  const int Kb = g.K * ES;  // k-contiguous: bytes of a row
  int lit = 0, lk = 0, lend = 0, ls = 0;  // item, stage, its end, ring slot of the next load
  const int kchunk = 16 * ((lane & 3) ^ ((lane >> 4) & 3));  // k-contiguous: byte of the stage this lane loads
  auto k_of = [&](int I, int T) { return (I * 1024 + lane * 16) / (T * ES); };  // k-strided: k-row in the stage
  auto begin_loads = [&](const Item& t) {
    LA = reinterpret_cast<const unsigned char*>(g.A) + t.batch * g.strideA * ES;
    LB = reinterpret_cast<const unsigned char*>(g.B) + t.batch * g.strideB * ES;
    auto contiguous = [&](const unsigned char*& P, uint32_t* off, int n, int rows, int row0, int64_t ld) {
      P += (int64_t)row0 * ld * ES + (int64_t)t.k0 * 64;
      for (int q = 0; q < n; ++q) {
        const int r = min(16 * (wave * n + q) + (lane >> 2), rows - 1 - row0);
        off[q] = (uint32_t)(r * ld * ES) + kchunk;
      }
    };
    auto strided = [&](const unsigned char*& P, uint32_t* off, int n, int T, int rows, int row0, int64_t ld) {
      P += (int64_t)t.k0 * SK * ld * ES + (int64_t)row0 * ES;
      for (int q = 0; q < n; ++q) {
        const int I = wave * n + q, k = k_of(I, T);
        const int pos = (I * 1024 + lane * 16) % (T * ES) / 16;
        int c = pos ^ (ES == 2 ? 4 * (k & 3) : 8 * ((k >> 2) & 1));
        if (row0 + c * (16 / ES) >= rows) c = 0;
        off[q] = (uint32_t)(k * ld * ES) + 16 * c;
      }
    };
    if constexpr (AS) strided(LA, offA, NIA, TM, g.M, t.tm * TM, g.lda);
    else contiguous(LA, offA, NIA, g.M, t.tm * TM, g.lda);
    if constexpr (BS) strided(LB, offB, NIB, TN, g.N, t.tn * TN, g.ldb);
    else contiguous(LB, offB, NIB, g.N, t.tn * TN, g.ldb);
    lk = t.k0;
    lend = t.k0 + t.stages;
  };
  // one stage into the ring; false once every item's stages are issued
  auto issue = [&]() -> bool {
    if (lit >= nitem) return false;
    unsigned char* sa = smem + ls * STAGE;
    unsigned char* sb = sa + OPA;
    const unsigned char* zero = reinterpret_cast<const unsigned char*>(product_zeros);
    const bool whole = (lk + 1) * 64 <= Kb;  // (a k-row is ES bytes here)
    auto load = [&](const unsigned char* P, const uint32_t* off, int n, unsigned char* dst, bool strided, int T) {
#pragma unroll
      for (int q = 0; q < n; ++q) {
        const unsigned char* p = P + off[q];
        if (!whole) {
          const bool in = strided ? lk * SK + k_of(wave * n + q, T) < g.K : lk * 64 + kchunk < Kb;
          p = in ? p : zero;
        }
        __builtin_amdgcn_global_load_lds((const void*)p, (void*)(dst + (wave * n + q) * 1024), 16, 0, 0);
      }
    };
    load(LA, offA, NIA, sa, AS, TM);
    load(LB, offB, NIB, sb, BS, TN);
    LA += AS ? SK * g.lda * ES : 64;
    LB += BS ? SK * g.ldb * ES : 64;
    ls = ls + 1 == NS ? 0 : ls + 1;
    if (++lk == lend && ++lit < nitem) begin_loads(item_of(lit));
    return true;
  };

  // ---- fragments ---------------------------------------------------------
  const int kc0 = l32 * 64 + 16 * (half ^ ((l32 >> 2) & 3)), kc1 = kc0 ^ 32;
  auto frag = [&](const unsigned char* base, int row, bool strided, int T) -> intx8 {
    if (!strided) {
      const u32x4 x = *reinterpret_cast<const u32x4*>(base + row * 64 + kc0);
      const u32x4 y = *reinterpret_cast<const u32x4*>(base + row * 64 + kc1);
      return intx8{(int)x[0], (int)x[1], (int)x[2], (int)x[3], (int)y[0], (int)y[1], (int)y[2], (int)y[3]};
    }
    if constexpr (E == Elem::BF16) {
      // stage k 16 st + 8 half + 4 q + i of column row + 16 grp + 4 u
      const int i = (lane & 15) >> 2, u = lane & 3, grp = (lane >> 4) & 1;
      const int col = row + 16 * grp + 4 * u;
      const unsigned char* p = base + (8 * half + i) * (T * 2) + 16 * ((col >> 3) ^ (4 * i)) + 2 * (col & 7);
      typedef __attribute__((address_space(3))) shortx4_t lds_s4;
      struct Four { shortx4_t v[4]; } f;
#pragma unroll
      for (int st = 0; st < 2; ++st)
#pragma unroll
        for (int q = 0; q < 2; ++q)
          f.v[2 * st + q] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4*)(p + (16 * st + 4 * q) * (T * 2)));
      return __builtin_bit_cast(intx8, f);
    } else {
      const unsigned char* p = base + (4 * half) * (T * 4) + 4 * ((row + l32) ^ (32 * half));
      intx8 f;
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = *reinterpret_cast<const int*>(p + ((j < 4 ? j : 4 + j)) * (T * 4));
      return f;
    }
  };
  intx8 fa[2][FM], fb[2][FN];
  auto read_frags = [&](int slot_, int set) {
    const unsigned char* sa = smem + slot_ * STAGE;
    const unsigned char* sb = sa + OPA;
#pragma unroll
    for (int i = 0; i < FM; ++i) fa[set][i] = frag(sa, (wm * FM + i) * 32, AS, TM);
#pragma unroll
    for (int j = 0; j < FN; ++j) fb[set][j] = frag(sb, (wn * FN + j) * 32, BS, TN);
  };

  // ---- scales (F8): one dword = 4 blocks of 128 k of a row ----------------
  constexpr int NSC = E == Elem::F8 ? FM + FN : 1;
  uint32_t sc[NSC], sn[NSC];
  auto load_scales = [&](const Item& t, int kb4, uint32_t* to) {
    if constexpr (E == Elem::F8) {
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        const int r = min(t.tm * TM + (wm * FM + i) * 32 + l32, g.M - 1) >> g.sa_shift;
        to[i] = *reinterpret_cast<const uint32_t*>(g.sa + t.batch * g.strideSa + (int64_t)r * g.ldsa + 4 * kb4);
      }
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        const int r = min(t.tn * TN + (wn * FN + j) * 32 + l32, g.N - 1) >> g.sb_shift;
        to[FM + j] = *reinterpret_cast<const uint32_t*>(g.sb + t.batch * g.strideSb + (int64_t)r * g.ldsb + 4 * kb4);
      }
    }
  };

  floatx16 acc[FM][FN];
  Item cur = item_of(0);
  begin_loads(cur);
#pragma unroll
  for (int s = 0; s < NS; ++s) issue();  // a dry ring leaves its slots unread
  if constexpr (E == Elem::F8) load_scales(cur, cur.k0 >> 3, sc);
  wait_stage<0>();
  barrier_no_fence();
  int rs = 0;  // ring slot of the stage being multiplied
  read_frags(0, 0);
  wait_stage<0>();
  barrier_no_fence();

  for (int it = 0; it < nitem; ++it) {
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.f;
    const Item nxt = it + 1 < nitem ? item_of(it + 1) : cur;
    for (int s = 0; s < cur.stages; s += 2) {
      if constexpr (E == Elem::F8) {
        if ((s & 7) == 0) {
          if (s) {
#pragma unroll
            for (int i = 0; i < NSC; ++i) sc[i] = sn[i];
          }
          const bool more = s + 8 < cur.stages;
          load_scales(more ? cur : nxt, more ? (cur.k0 + s + 8) >> 3 : nxt.k0 >> 3, sn);
        }
      }
      const int shift = 4 * (s & 6);  // byte of the block of 128
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const bool dma = issue();  // into slot rs, read into registers before the last barrier
        const int nx = rs + 1 == NS ? 0 : rs + 1;
        read_frags(nx, 1 - u);  // (after the last stage: a stale slot, unused)
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
          for (int j = 0; j < FN; ++j)
            acc[i][j] = stage_mma<E, FB, FA>(fb[u][j], fa[u][i], acc[i][j],
                                             E == Elem::F8 ? (int)(sc[E == Elem::F8 ? FM + j : 0] >> shift) : 0,
                                             E == Elem::F8 ? (int)(sc[E == Elem::F8 ? i : 0] >> shift) : 0);
        // the stage after next has landed; NS - 2 younger ones may be in flight
        if (dma) wait_stage<(NS - 2) * NI>();
        else wait_stage<0>();
        barrier_no_fence();
        rs = nx;
      }
    }

    // ---- epilogue --------------------------------------------------------
    const int m0 = cur.tm * TM + wm * FM * 32, n0 = cur.tn * TN + wn * FN * 32;
    if constexpr (EPI == Epi::STORE) {
      const int64_t base = cur.batch * g.strideC + cur.split * g.split_stride;
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        const int m = m0 + 32 * i + l32;
        const int64_t row = base + (int64_t)m * g.ldc;
#pragma unroll
        for (int j = 0; j < FN; ++j) {
          const int nb = n0 + 32 * j;
          if (g.c_dt == 0) {
            float* C = reinterpret_cast<float*>(g.C) + row;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const int n = nb + 8 * q + 4 * half;
              floatx4 v = floatx4{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
              if (m >= g.M || n >= g.N) continue;
              if (g.vec && n + 4 <= g.N) {
                floatx4* P = reinterpret_cast<floatx4*>(C + n);
                if (g.beta != 0.f) v += g.beta * *P;
                *P = v;
              } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  if (n + e < g.N) C[n + e] = v[e] + (g.beta != 0.f ? g.beta * C[n + e] : 0.f);
              }
            }
          } else {
            // two 16-bit runs of 4 columns become one of 8: the halves of the
            // wave swap one run each
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              const int n = nb + 16 * q + 8 * half;
              float x[8];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const auto sw = __builtin_amdgcn_permlane32_swap(float_bits(acc[i][j][8 * q + e]),
                                                                 float_bits(acc[i][j][8 * q + 4 + e]), false, false);
                x[e] = bits_float(sw[0]);
                x[4 + e] = bits_float(sw[1]);
              }
              if (m >= g.M || n >= g.N) continue;
              uint16_t* C = reinterpret_cast<uint16_t*>(g.C) + row + n;
              auto widen = [&](uint16_t b) {
                return g.c_dt == 2 ? __builtin_bit_cast(float, (uint32_t)b << 16) : (float)__builtin_bit_cast(_Float16, b);
              };
              if (g.vec && n + 8 <= g.N) {
                if (g.beta != 0.f) {
                  const u32x4 old = *reinterpret_cast<const u32x4*>(C);
#pragma unroll
                  for (int e = 0; e < 8; ++e) x[e] += g.beta * widen((uint16_t)(old[e >> 1] >> (16 * (e & 1))));
                }
                u32x4 o;
#pragma unroll
                for (int e = 0; e < 4; ++e) o[e] = g.c_dt == 2 ? pack_bf16(x[2 * e], x[2 * e + 1]) : pack_f16(x[2 * e], x[2 * e + 1]);
                *reinterpret_cast<u32x4*>(C) = o;
              } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                  if (n + e < g.N) {
                    const float y = x[e] + (g.beta != 0.f ? g.beta * widen(C[e]) : 0.f);
                    C[e] = (uint16_t)((g.c_dt == 2 ? pack_bf16(y, y) : pack_f16(y, y)) & 0xffff);
                  }
              }
            }
          }
        }
      }
    } else {
      // 128 columns of the wave's rows: maximum, sum of exponentials, the
      // target's logit; the exponentials against that maximum, rounded to
      // the gradients' type, where the caller wants gradients
      static_assert(FN == 4 || EPI != Epi::SOFTMAX, "a piece is 128 columns");
      constexpr float L2E = 1.4426950408889634f;
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        const int m = m0 + 32 * i + l32;
        const int64_t tg = m < g.M ? g.targets[m] : -1;
        const int t = tg >= n0 && tg < g.N && tg < n0 + 128 ? (int)(tg - n0) : -1;
        float mx = -INFINITY, tl = 0.f;
        bool hit = false;
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
          for (int v = 0; v < 16; ++v) {
            const int c = 32 * j + 8 * (v >> 2) + 4 * half + (v & 3);
            if (n0 + c >= g.N) acc[i][j][v] = -INFINITY;
            mx = fmaxf(mx, acc[i][j][v]);
            if (t == c) { tl = acc[i][j][v]; hit = true; }
          }
        mx = fmaxf(mx, __shfl_xor(mx, 32));
        const float ref = mx == -INFINITY ? 0.f : mx;
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
          for (int v = 0; v < 16; ++v) {
            const float e = __builtin_amdgcn_exp2f((acc[i][j][v] - ref) * L2E);
            acc[i][j][v] = e;
            sum += e;
          }
        sum += __shfl_xor(sum, 32);
        if (m < g.M && n0 < g.N) {
          if (half == 0) g.stats[(int64_t)(n0 >> 7) * g.M + m] = floatx2{mx, sum};
          if (hit) g.target_logit[m] = tl;
        }
        if (g.C) {
          // rows of ldc elements, a multiple of 128: no edge within a piece
#pragma unroll
          for (int j = 0; j < FN; ++j) {
            if constexpr (E == Elem::F32) {
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                const floatx4 v = floatx4{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
                if (m < g.M && n0 < g.N)
                  *reinterpret_cast<floatx4*>(reinterpret_cast<float*>(g.C) + (int64_t)m * g.ldc + n0 + 32 * j + 8 * q + 4 * half) = v;
              }
            } else {
#pragma unroll
              for (int q = 0; q < 2; ++q) {
                uint32_t p0 = pack_bf16(acc[i][j][8 * q], acc[i][j][8 * q + 1]), p1 = pack_bf16(acc[i][j][8 * q + 2], acc[i][j][8 * q + 3]);
                uint32_t p2 = pack_bf16(acc[i][j][8 * q + 4], acc[i][j][8 * q + 5]), p3 = pack_bf16(acc[i][j][8 * q + 6], acc[i][j][8 * q + 7]);
                const auto a = __builtin_amdgcn_permlane32_swap(p0, p2, false, false);
                const auto b = __builtin_amdgcn_permlane32_swap(p1, p3, false, false);
                if (m < g.M && n0 < g.N)
                  *reinterpret_cast<u32x4*>(reinterpret_cast<uint16_t*>(g.C) + (int64_t)m * g.ldc + n0 + 32 * j + 16 * q + 8 * half) =
                      u32x4{a[0], b[0], a[1], b[1]};
              }
            }
          }
        }
      }
    }
    if constexpr (E == Elem::F8) {
#pragma unroll
      for (int i = 0; i < NSC; ++i) sc[i] = sn[i];
    }
    cur = nxt;
  }
}

}  // namespace shampoo
