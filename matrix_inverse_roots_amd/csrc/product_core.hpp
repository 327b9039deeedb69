// Rectangular matrix product on CDNA4 matrix cores (gfx950) for the 8-bit
// block-scaled product and the projection's softmax cross entropy.
//
//     C[m, n] = sum_k A(m, k) B(n, k)
//
// Element types: bfloat16 (v_mfma_f32_32x32x16_bf16), float32
// (v_mfma_f32_32x32x2_f32) and 8-bit floating point with a power-of-two
// scale for each block of 128 k (v_mfma_scale_f32_32x32x64_f8f6f4, which
// applies the scales to the operands' exponents inside the matrix core: no
// instruction is spent on them).  Accumulation is float32 throughout.  The
// 8-bit matrix instructions align the products of one instruction to the
// largest of them and drop what lies some 13 bits below (measured: 1.5e-5
// relative on random operands, at every K), which a 16-bit result does not
// show and a float32 result does.  F8W, for float32 results, widens the
// operands with their scales to bfloat16 in registers (exactly; blocks whose
// scales are at the ends of their range apart, see there) and multiplies
// those, at half the matrix-core rate (results 1.7e-7 from float64).
//
// Operand layouts.  "k-contiguous": row r at r * ld, k along the row.
// "k-strided" (template flags AS, BS; bfloat16 and float32): element (r, k)
// at k * ld + r, an operand read as its transpose.
//
// Structure.  One workgroup of WM x WN waves computes a tile of
// 32 FM WM x 32 FN WN outputs; workgroups are persistent and walk the tiles
// of their XCD's share, so that the loads of the next tile run through the
// end of the current one.  A stage is 128 bytes of k of every row of both
// operands; stages go straight to LDS (buffer_load ... lds, 16 bytes a lane)
// into NB buffers (two, or four where a compute unit holds one small
// workgroup).  Each wave reads one half of a stage's k into registers
// while the matrix cores work on the half before it, so a stage's buffer is
// free when its second half is multiplied, and takes the stage NB on: loads
// have the time of NB - 1 stages to land.  One barrier per stage.
//
// What it reaches (MI355X): 8-bit 16384 x 8192 x 8192 0.90-0.97 ms = 2.3-2.4
// PF/s; bfloat16 8192 x 131072 x 4096 with the softmax epilogue 6.9-7.3 ms =
// 1.2-1.3 PF/s, and 6.7-7.2 ms for either gradient, k-strided operands included.
// The matrix cores are busy 75-78% of the cycles there (61% in 8 bits) at 1.6
// GHz: power bounds it, more than loads (all from one cached address: 1-7%
// faster) or LDS (no conflicts).  Without any loads the 8-bit product would
// take 0.69 ms and the bfloat16 loss with gradients 18.1 of its 22.3 ms.
//
// LDS layouts, conflict-free for the reads (16 lanes of a ds_read_b128 are
// served together: lanes 0-3, 12-15, 20-23, 24-27 of each 32):
//   k-contiguous: rows of 128 bytes, 16-byte chunk c of row r at
//     c ^ ((r >> 1) & 7); lane l reads row l % 32, chunks h and 2 + h of each
//     half row, h = l / 32.  A fragment is 32 bytes a lane: the k a lane holds
//     are the same for both operands, which is all a dot product needs.
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

#include "ffn_epilogue.hpp"
#include "product_types.hpp"

namespace shampoo {

// matrix-core instructions that a fragment pair (32 bytes a lane) takes
template <Elem E> constexpr int MMA_STEPS = E == Elem::F8 ? 1 : E == Elem::BF16 ? 2 : E == Elem::F8W ? 4 : 8;

// 8 bytes of a fragment times 2^(byte - 127), as bfloat16
template <int F> __device__ __forceinline__ bf16x8 widen_f8(int lo, int hi, int byte) {
  const float scale = bits_float((uint32_t)byte << 23);
  struct Four { __bf16 v __attribute__((ext_vector_type(2))); };
  struct { decltype(Four::v) v[4]; } r;
  if constexpr (F == 0) {
    r.v[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, false);
    r.v[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, true);
    r.v[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, false);
    r.v[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, true);
  } else {
    r.v[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(lo, scale, false);
    r.v[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(lo, scale, true);
    r.v[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(hi, scale, false);
    r.v[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(hi, scale, true);
  }
  return __builtin_bit_cast(bf16x8, r);
}

// acc += step `st` of B fragment x A fragment
template <Elem E, int FB, int FA>
__device__ __forceinline__ floatx16 mma_step(int st, intx8 b, intx8 a, floatx16 acc, int scb, int sca) {
  if constexpr (E == Elem::F8) {
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(b, a, acc, FB, FA, 0, scb, 0, sca);
  } else if constexpr (E == Elem::BF16) {
    struct Two { bf16x8 v[2]; };
    const Two bb = __builtin_bit_cast(Two, b), aa = __builtin_bit_cast(Two, a);
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(bb.v[st], aa.v[st], acc, 0, 0, 0);
  } else {
    return __builtin_amdgcn_mfma_f32_32x32x2f32(bits_float(b[st]), bits_float(a[st]), acc, 0, 0, 0);
  }
}

// wait until at most K vector memory operations of this wave are in flight,
// and no LDS reads
template <int K> __device__ __forceinline__ void wait_stage() {
  static_assert(K >= 0 && K < 64, "vmcnt has 6 bits");
  __builtin_amdgcn_s_waitcnt((K & 15) | (0x7 << 4) | ((K >> 4) << 14));
}

// ds_read_b64_tr_b16.  The restrict-qualified parameter tells the compiler
// that nothing writes what the read sees while it runs: without it, it would
// wait for every load into LDS in flight before each such read (the waits
// and barriers that order them are the kernel's own).
typedef __attribute__((address_space(3))) shortx4_t lds_s4;
__device__ __forceinline__ shortx4_t read_transposed(const lds_s4* __restrict__ p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16(const_cast<lds_s4*>(p));
}

// A buffer descriptor: loads at offsets past `bytes` return zeros.
typedef __amdgpu_buffer_rsrc_t rsrc_t;
constexpr uint32_t RSRC_FLAGS = 0x00027000;       // raw 32-bit buffer
constexpr uint32_t RSRC_OUTSIDE = 0x80000000u;    // an offset outside every descriptor
__device__ __forceinline__ rsrc_t rsrc_of(const unsigned char* p, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<unsigned char*>(p), 0, bytes, RSRC_FLAGS);
}

// Groups of scales (or targets) in LDS: for the current stage and the NB (NB +
// 1) ahead, a power of two.
constexpr int scale_groups(int nb) { return nb > 2 ? 8 : 4; }

template <Elem E, int FM, int FN, int WM, int WN, int NB, bool AS, bool BS, Epi EPI, int FA, int FB>
__global__ __launch_bounds__(64 * WM * WN, 2) void product_kernel(ProductArgs g) {
  constexpr int ES = ElemTraits<E>::size;
  constexpr int W = WM * WN, TM = 32 * FM * WM, TN = 32 * FN * WN;
  constexpr int OPA = TM * 128, STAGE = (TM + TN) * 128;
  constexpr int NIA = TM / 8 / W, NIB = TN / 8 / W;
  constexpr int SK = 128 / ES;  // k of one stage
  constexpr bool SCALED = E == Elem::F8 || E == Elem::F8W;
  constexpr bool DUAL = EPI == Epi::GATED, TWO = EPI == Epi::STORE2;
  constexpr int TNO = DUAL ? TN / 2 : TN;  // columns of a tile's results
  constexpr int TURN = 16 * FN;            // DUAL: rows of B1 and B2 take turns
  // registers of the next tile's first fragments are given to these epilogues,
  // which read them again behind
  constexpr bool AGAIN = EPI == Epi::LINEAR || EPI == Epi::GATED || EPI == Epi::GATED_GRAD;
  // LDS: NB buffers, then groups of scales (a group each for NB stages ahead at
  // most, and the current one), then as many groups of targets
  constexpr int NI = NIA + NIB, NG = scale_groups(NB), SCALES = NB * STAGE, SGROUP = 4 * (TM + TN);
  constexpr int TARGETS = SCALES + (SCALED ? NG * SGROUP : 0);
  static_assert(NB >= 2 && NB <= 4, "groups of scales are counted with masks");
  static_assert(NIA * W * 8 == TM && NIB * W * 8 == TN, "loads divide among the waves");
  static_assert(!SCALED || (!AS && !BS), "8-bit operands are k-contiguous");
  static_assert(!SCALED || (TM + TN) % (64 * W) == 0, "each wave loads the scales of as many rows");
  static_assert(TM % 64 == 0 && TM <= 64 * W, "a wave loads the targets of 64 rows");
  static_assert(!(AS && TM < 64) && !(BS && TN < 64), "k-strided swizzles need 64 columns");
  static_assert(!DUAL || (FN % 2 == 0 && !BS && TURN % (NIB * 8) == 0), "a wave loads from one of the two matrices");
  static_assert(!TWO || BS, "two matrices follow each other along strided k");
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
  typedef __attribute__((address_space(3))) unsigned char lds_u8;
  lds_u8* const lds = (lds_u8*)smem;

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

  struct Item { int batch, split, tm, tn, k0, stages; };
  // Tiles in bands of 8 rows of tiles, column by column: the tiles that run
  // at the same time on an XCD share the operands' panels in its L2.  A place
  // (matrix and range of k, band, tile of the band) is found by division once
  // and then moved on by `per`: divisions at every tile would take as long as
  // several stages.
  struct Place { int bs, band, u; };
  auto band_size = [&](int band) { return min(8, g.mt - 8 * band) * g.nt; };
  auto place_of = [&](int64_t w) {
    Place p;
    const int tiles = g.mt * g.nt;
    p.bs = (int)(w / tiles);
    p.u = (int)(w - (int64_t)p.bs * tiles);
    p.band = p.u / (8 * g.nt);
    p.u -= p.band * 8 * g.nt;
    return p;
  };
  auto move_on = [&](Place& p) {
    p.u += per;
    for (int size = band_size(p.band); p.u >= size; size = band_size(p.band)) {
      p.u -= size;
      if (8 * ++p.band >= g.mt) {
        p.band = 0;
        ++p.bs;
      }
    }
  };
  auto item_at = [&](const Place& p) {
    Item r;
    r.batch = g.splits == 1 ? p.bs : p.bs / g.splits;
    r.split = p.bs - r.batch * g.splits;
    const int rows = min(8, g.mt - 8 * p.band);
    r.tn = rows == 8 ? p.u >> 3 : p.u / rows;
    r.tm = 8 * p.band + p.u - r.tn * rows;
    r.k0 = r.split * g.split_stages;
    r.stages = min(g.split_stages, g.nst - r.k0);
    return r;
  };

  // ---- loads -------------------------------------------------------------
  // offA, offB: this lane's bytes within a stage's part of the tile; tailA,
  // tailB: the same in the last stage, where what is past K lies outside.  PA,
  // PB: where that part starts (k-contiguous: at the item's first stage, with
  // the stage's distance in `ahead`); endA, endB: bytes from there to the end
  // of the operand's last row or k-row, past which a descriptor reads zeros.
  const int last = g.nst - 1, rest = g.K - last * SK;  // the last stage, and its k
  uint32_t offA[NIA], offB[NIB], tailA[NIA], tailB[NIB];
  // DUAL: half a wave's rows of B1, then as many of B2, so that the first half
  // of a wave's fragments and the second are the same columns of both
  const bool second = DUAL && (wave * NIB * 8 / TURN & 1);
  auto offsets = [&](uint32_t* off, uint32_t* tail, int n, bool strided, int T, int64_t ld, bool dual) {
#pragma unroll
    for (int q = 0; q < n; ++q) {
      const int at = (wave * n + q) * 1024 + lane * 16;
      if (strided) {
        const int k = at / (T * ES), pos = at % (T * ES) / 16;
        off[q] = (uint32_t)(k * ld * ES) + 16 * (pos ^ (ES == 2 ? 4 * (k & 3) : 8 * ((k >> 2) & 1)));
        tail[q] = k < rest ? off[q] : RSRC_OUTSIDE;
      } else {
        const int row = at >> 7, byte = 16 * ((lane & 7) ^ ((row >> 1) & 7));
        off[q] = (uint32_t)((dual ? row / (2 * TURN) * TURN + row % TURN : row) * ld * ES) + byte;
        tail[q] = byte < rest * ES ? off[q] : RSRC_OUTSIDE;
      }
    }
  };
  offsets(offA, tailA, NIA, AS, TM, g.lda, false);
  offsets(offB, tailB, NIB, BS, TN, g.ldb, DUAL);
  const int Kb = (g.K * ES + 15) & ~15;  // k-contiguous: bytes of a row, in whole chunks
  const unsigned char *PA, *PB;
  int64_t endA, endB;
  int ahead = 0;
  Place lp = place_of(first);
  // a descriptor's size: what is left, at most 2^31 - 1 and never below zero
  auto clip = [](int64_t bytes) {
    const int high = (int)(bytes >> 31);
    return high < 0 ? 0u : high > 0 ? 0x7fffffffu : (uint32_t)bytes;
  };
  int lit = 0, lk = 0, lend = 0, ls = 0, lg = 0;  // item, stage, its end, buffer, scale group of the next load
  Item li;
  // STORE2: B from the stage `lk` on
  auto begin_two = [&]() {
    const bool in2 = lk >= g.kswitch;
    const int64_t kb = (int64_t)(lk - (in2 ? g.kswitch : 0)) * SK * g.ldb * ES;
    const int rb = li.tn * TN;
    PB = reinterpret_cast<const unsigned char*>(in2 ? g.B2 : g.B) + kb + (int64_t)rb * ES;
    endB = (g.kpart - 1) * g.ldb * ES + (((g.N - rb) * ES + 15) & ~15) - kb;
  };
  auto begin_loads = [&]() {
    li = item_at(lp);
    lk = li.k0;
    ahead = 0;
    lend = li.k0 + li.stages;
    const int ra = li.tm * TM, rb = li.tn * TNO;
    const int64_t ka = AS ? (int64_t)lk * SK * g.lda * ES : (int64_t)lk * 128, kb = BS ? (int64_t)lk * SK * g.ldb * ES : (int64_t)lk * 128;
    PA = reinterpret_cast<const unsigned char*>(g.A) + li.batch * g.strideA * ES + ka + (AS ? (int64_t)ra * ES : ra * g.lda * ES);
    PB = reinterpret_cast<const unsigned char*>(second ? g.B2 : g.B) + li.batch * g.strideB * ES + kb + (BS ? (int64_t)rb * ES : rb * g.ldb * ES);
    // strided: the last k-row's columns, in whole chunks (rows start on 16
    // bytes); columns past the tile's read what follows, and nothing past that
    endA = AS ? (g.K - 1) * g.lda * ES + (((g.M - ra) * ES + 15) & ~15) - ka : (g.M - 1 - ra) * g.lda * ES + Kb - ka;
    endB = BS ? (g.K - 1) * g.ldb * ES + (((g.N - rb) * ES + 15) & ~15) - kb : (g.N - 1 - rb) * g.ldb * ES + Kb - kb;
    if constexpr (TWO) begin_two();
    if constexpr (EPI == Epi::SOFTMAX) {
      // the low halves of the rows' targets (a column fits; what else matches
      // one there, the row pass does not read), ahead of the item's first
      // stage and waited for with it: one item more than there are buffers
      if (wave * 64 < TM) {
        const int64_t* p = g.targets + min(ra + wave * 64 + lane, g.M - 1);
        __builtin_amdgcn_global_load_lds((const void*)p, (void*)(smem + TARGETS + ((lit & (NG - 1)) * TM + wave * 64) * 4), 4, 0, 0);
      }
    }
  };
  // one stage into its buffer (zeros once every item's stages are issued)
  auto issue = [&]() {
    const bool tail = lk == last;
    const rsrc_t ra = rsrc_of(PA, clip(endA)), rb = rsrc_of(PB, clip(endB));
    lds_u8* const sa = lds + ls * STAGE + wave * (NIA * 1024);
    lds_u8* const sb = lds + ls * STAGE + OPA + wave * (NIB * 1024);
    const int aheadA = AS ? 0 : ahead, aheadB = BS ? 0 : ahead;
#pragma unroll
    for (int q = 0; q < NIA; ++q) {
      uint32_t o = offA[q];
      if (!SCALED && tail) o = tailA[q];
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, sa + q * 1024, 16, o, aheadA, 0, 0);
    }
#pragma unroll
    for (int q = 0; q < NIB; ++q) {
      uint32_t o = offB[q];
      if (!SCALED && tail) o = tailB[q];
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, sb + q * 1024, 16, o, aheadB, 0, 0);
    }
  };
  auto issue_scales = [&]() {
    if constexpr (SCALED) {
      // with the first stage of 4: the 4 scales of each of the tile's rows
      // for the 512 k that follow
      if (((lk - li.k0) & 3) == 0 && lend >= 0) {
        constexpr int NSG = (TM + TN) / (64 * W);
#pragma unroll
        for (int q = 0; q < NSG; ++q) {
          const int first_row = (wave * NSG + q) * 64;  // wave-uniform: A's rows, then B's
          const bool isA = first_row < TM;
          const int row = isA ? min(li.tm * TM + first_row + lane, g.M - 1) >> g.sa_shift
                              : min(li.tn * TN + first_row - TM + lane, g.N - 1) >> g.sb_shift;
          const uint8_t* p = isA ? g.sa + li.batch * g.strideSa + (int64_t)row * g.ldsa
                                 : g.sb + li.batch * g.strideSb + (int64_t)row * g.ldsb;
          __builtin_amdgcn_global_load_lds((const void*)(p + lk), (void*)(smem + SCALES + lg * SGROUP + first_row * 4), 4, 0, 0);
        }
        lg = (lg + 1) & (NG - 1);
      }
    }
  };
  auto advance = [&]() {
    ls = NB == 2 ? ls ^ 1 : NB == 4 ? (ls + 1) & 3 : ls == NB - 1 ? 0 : ls + 1;
    if (lend < 0) return;  // nothing left: the descriptors stay empty
    if (AS) PA += SK * g.lda * ES, endA -= SK * g.lda * ES;
    if (BS) PB += SK * g.ldb * ES, endB -= SK * g.ldb * ES;
    ahead += 128;
    if (++lk == lend) {
      if (++lit < nitem) {
        move_on(lp);
        begin_loads();
      } else {
        endA = endB = 0;  // descriptors of nothing: zeros
        ahead = 0;
        lend = -1;
      }
    } else if (TWO && lk == g.kswitch) {
      begin_two();
    }
  };

  // ---- fragments ---------------------------------------------------------
  const int kc = l32 * 128 + 16 * (half ^ ((l32 >> 1) & 7));
  // k-strided bfloat16: k 16 st + 8 half + 4 q + i of column row + 16 grp + 4 u
  const int ti = (lane & 15) >> 2, tu = lane & 3, tgrp = (lane >> 4) & 1;
  auto frag = [&](const unsigned char* base, int row, int hh, bool strided, int T) -> intx8 {
    if (!strided) {
      const u32x4 x = *reinterpret_cast<const u32x4*>(base + row * 128 + (kc ^ (64 * hh)));
      const u32x4 y = *reinterpret_cast<const u32x4*>(base + row * 128 + (kc ^ (64 * hh + 32)));
      return intx8{(int)x[0], (int)x[1], (int)x[2], (int)x[3], (int)y[0], (int)y[1], (int)y[2], (int)y[3]};
    }
    if constexpr (E == Elem::BF16) {
      const int col = row + 16 * tgrp + 4 * tu;
      const unsigned char* p = base + (32 * hh + 8 * half + ti) * (T * 2) + 16 * ((col >> 3) ^ (4 * ti)) + 2 * (col & 7);
      struct Four { shortx4_t v[4]; } f;
#pragma unroll
      for (int st = 0; st < 2; ++st)
#pragma unroll
        for (int q = 0; q < 2; ++q)
          f.v[2 * st + q] = read_transposed((const lds_s4*)(p + (16 * st + 4 * q) * (T * 2)));
      return __builtin_bit_cast(intx8, f);
    } else {
      const unsigned char* p = base + (16 * hh + 4 * half) * (T * 4) + 4 * ((row + l32) ^ (32 * half));
      intx8 f;
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = *reinterpret_cast<const int*>(p + ((j < 4 ? j : 4 + j)) * (T * 4));
      return f;
    }
  };
  intx8 fa[2][FM], fb[2][FN];
  auto read_frags = [&](int buffer, int hh) {
    const unsigned char* sa = smem + buffer * STAGE;
    const unsigned char* sb = sa + OPA;
#pragma unroll
    for (int i = 0; i < FM; ++i) fa[hh][i] = frag(sa, (wm * FM + i) * 32, hh, AS, TM);
#pragma unroll
    for (int j = 0; j < FN; ++j) fb[hh][j] = frag(sb, (wn * FN + j) * 32, hh, BS, TN);
  };
  // the scale bytes of a stage, which is a block of 128 k
  int sc[2][FM + FN];
  auto read_scales = [&](int group, int stage, int* to) {
    if constexpr (SCALED) {
      const unsigned char* p = smem + SCALES + group * SGROUP + l32 * 4 + (stage & 3);
#pragma unroll
      for (int i = 0; i < FM; ++i) to[i] = p[(wm * FM + i) * 128];
#pragma unroll
      for (int j = 0; j < FN; ++j) to[FM + j] = p[(TM + (wn * FN + j) * 32) * 4];
    }
  };

  floatx16 acc[FM][FN];
  auto multiply = [&](int hh) {
    if constexpr (E == Elem::F8W) {
#pragma unroll
      for (int st = 0; st < 4; ++st) {
        bf16x8 a[FM], b[FN];
#pragma unroll
        for (int i = 0; i < FM; ++i) a[i] = widen_f8<FA>(fa[hh][i][2 * st], fa[hh][i][2 * st + 1], sc[0][i]);
#pragma unroll
        for (int j = 0; j < FN; ++j) b[j] = widen_f8<FB>(fb[hh][j][2 * st], fb[hh][j][2 * st + 1], sc[0][FM + j]);
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
          for (int j = 0; j < FN; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(b[j], a[i], acc[i][j], 0, 0, 0);
      }
      return;
    } else {
#pragma unroll
      for (int st = 0; st < MMA_STEPS<E>; ++st)  // outermost: consecutive instructions write different blocks
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
          for (int j = 0; j < FN; ++j)
            acc[i][j] = mma_step<E, FB, FA>(st, fb[hh][j], fa[hh][i], acc[i][j], SCALED ? sc[0][FM + j] : 0, SCALED ? sc[0][i] : 0);
    }
  };
  // F8W: scale bytes from 17 to 239 keep every value of either format times its
  // scale a normal bfloat16 number (2^-16 at byte 17, 1.75 2^15 at 239).  A
  // wave that meets another among the scales of an item notes the item, and
  // at the end makes its part of those tiles anew, from memory: values widened
  // alone, each block's sum times both scales at once, so that only the
  // results' own range is left.  Behind the loop because its registers are
  // full: the same inside it spilled 73 of them.  The noting costs 0.7% (144 x
  // 1024^3: 363 to 366 us).
  constexpr uint32_t FIRST_SAFE = 17, SAFE_SPAN = 239 - FIRST_SAFE;
  uint32_t extreme = 0;
  uint64_t again = 0;  // items to make anew; bit 63 stands for all from 63 on
  auto note_scales = [&]() {
    if constexpr (E == Elem::F8W) {
#pragma unroll
      for (int i = 0; i < FM + FN; ++i) extreme = max(extreme, (uint32_t)sc[0][i] - FIRST_SAFE);
    }
  };
  auto store_apart = [&](const Item& item) {
    const uint8_t* const A = reinterpret_cast<const uint8_t*>(g.A) + item.batch * g.strideA + (int64_t)item.k0 * SK;
    const uint8_t* const B = reinterpret_cast<const uint8_t*>(g.B) + item.batch * g.strideB + (int64_t)item.k0 * SK;
    const uint8_t* const SA = g.sa + item.batch * g.strideSa + item.k0;
    const uint8_t* const SB = g.sb + item.batch * g.strideSb + item.k0;
    float* const C = reinterpret_cast<float*>(g.C) + item.batch * g.strideC + item.split * g.split_stride;
#pragma nounroll
    for (int i = 0; i < FM; ++i) {
      const int m = item.tm * TM + (wm * FM + i) * 32 + l32, ma = min(m, g.M - 1);
      const uint8_t* const sa = SA + (int64_t)(ma >> g.sa_shift) * g.ldsa;
#pragma nounroll
      for (int j = 0; j < FN; ++j) {
        const int n0 = item.tn * TN + (wn * FN + j) * 32, nb = min(n0 + l32, g.N - 1);
        const uint8_t* const sb = SB + (int64_t)(nb >> g.sb_shift) * g.ldsb;
        const uint8_t* a = A + ma * g.lda + 8 * half;
        const uint8_t* b = B + nb * g.ldb + 8 * half;
        float sum[16];
#pragma unroll
        for (int v = 0; v < 16; ++v) sum[v] = 0.f;
#pragma nounroll
        for (int s = 0; s < item.stages; ++s, a += SK, b += SK) {
          floatx16 t;
#pragma unroll
          for (int v = 0; v < 16; ++v) t[v] = 0.f;
#pragma unroll
          for (int st = 0; st < SK / 16; ++st) {
            const u32x2 x = *reinterpret_cast<const u32x2*>(a + 16 * st), y = *reinterpret_cast<const u32x2*>(b + 16 * st);
            t = __builtin_amdgcn_mfma_f32_32x32x16_bf16(widen_f8<FB>((int)y[0], (int)y[1], 127), widen_f8<FA>((int)x[0], (int)x[1], 127), t, 0, 0, 0);
          }
          const int ea = (int)sa[s] - 254, eb = sb[s];
#pragma unroll
          for (int v = 0; v < 16; ++v) sum[v] += ldexpf(t[v], ea + __shfl(eb, 8 * (v >> 2) + 4 * half + (v & 3)));
        }
#pragma unroll
        for (int v = 0; v < 16; ++v) {
          const int n = n0 + 8 * (v >> 2) + 4 * half + (v & 3);
          if (m < g.M && n < g.N) C[m * g.ldc + n] = sum[v];  // by the lane that wrote it before
        }
      }
    }
  };
  // The reads (and loads) of a half go between its first matrix-core
  // instructions: left to itself the compiler puts them behind the last and
  // waits for them there.
  constexpr int NMMA = FM * FN * MMA_STEPS<E>;
  constexpr int NREAD = FM * (AS ? 4 : 2) + FN * (BS ? 4 : 2) + (SCALED ? FM + FN : 0);
  constexpr int STEPS = NMMA * 3 / 4 < 24 ? NMMA * 3 / 4 : 24, RPS = (NREAD + STEPS - 1) / STEPS;
  // loads over the whole half: a compute unit takes 16 cycles for each, and a
  // wave that meets a full queue stalls with its matrix-core instructions
  constexpr int LGAP = NMMA >= 2 * (NIA + NIB) ? NMMA / (NIA + NIB) : 1;
  auto interleave = [&](bool loads) {
#pragma unroll
    for (int k = 0; k < (NMMA < 64 ? NMMA : 64); ++k) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      if (k < STEPS) __builtin_amdgcn_sched_group_barrier(0x100, RPS, 0);
      if (loads && k % LGAP == 0 && k / LGAP < NIA + NIB) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
    }
  };
  begin_loads();
#pragma nounroll
  for (int s = 0; s < NB; ++s) {
    issue();
    issue_scales();
    advance();
  }
  wait_stage<(NB - 1) * NI>();
  barrier_no_fence();
  int rb = 0, rg = 0;  // buffer and scale group of the stage being multiplied
  read_frags(0, 0);
  read_scales(0, 0, sc[0]);

  Place cp = place_of(first);
#pragma nounroll
  for (int it = 0; it < nitem; ++it) {
    const Item cur = item_at(cp);
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.f;
#pragma nounroll
    for (int s = 0; s < cur.stages; ++s) {
      note_scales();
      // first half of the stage's k; its second half into registers
      read_frags(rb, 1);
      multiply(0);
      interleave(false);
      // this wave is done with the buffer, and its part of the next stage has
      // landed; NB - 2 younger stages may be in flight
      wait_stage<(NB - 2) * NI>();
      barrier_no_fence();
      // second half; the buffer takes the stage NB on (at the very end the
      // next buffer is stale, and what is read from it unused)
      issue_scales();
      const bool last = s + 1 == cur.stages;
      if (last || (s & 3) == 3) rg = (rg + 1) & (NG - 1);
      const int next = NB == 2 ? rb ^ 1 : NB == 4 ? (rb + 1) & 3 : rb == NB - 1 ? 0 : rb + 1;
      issue();
      read_frags(next, 0);
      read_scales(rg, last ? 0 : s + 1, sc[1]);
      multiply(1);
      interleave(true);
#pragma unroll
      for (int i = 0; i < FM + FN; ++i) sc[0][i] = sc[1][i];
      rb = next;
      advance();
    }

    if constexpr (E == Elem::F8W) {
      if (__any(extreme > SAFE_SPAN)) again |= uint64_t(1) << min(it, 63);
      extreme = 0;
    }

    // ---- epilogue --------------------------------------------------------
    int el32 = l32, ehalf = half;
    asm volatile("" : "+v"(el32), "+v"(ehalf));  // addresses made here, not kept through the loop
    const int m0 = cur.tm * TM + wm * FM * 32, n0 = cur.tn * TN + wn * FN * 32;
    if constexpr (EPI == Epi::LINEAR) {
      linear_epilogue<FM, FN>(g, acc, m0, n0, el32, ehalf);
    } else if constexpr (EPI == Epi::GATED) {
      gated_epilogue<FM, FN>(g, acc, m0, n0 / 2, el32, ehalf, cur.split);
    } else if constexpr (EPI == Epi::GATED_GRAD) {
      gated_grad_epilogue<FM, FN, ES>(g, acc, m0, n0, el32, ehalf);
    } else if constexpr (EPI == Epi::STORE || EPI == Epi::STORE2) {
      const int64_t base = cur.batch * g.strideC + cur.split * g.split_stride;
      const float alpha = g.alpha * (g.alpha_dev ? *g.alpha_dev : 1.f);
      if (alpha != 1.f) {
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
          for (int j = 0; j < FN; ++j) acc[i][j] *= alpha;
      }
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        const int m = m0 + 32 * i + el32;
        const int64_t row = base + (int64_t)m * g.ldc;
#pragma unroll
        for (int j = 0; j < FN; ++j) {
          const int nb = n0 + 32 * j;
          if (g.c_dt == 0) {
            float* C = reinterpret_cast<float*>(g.C) + row;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const int n = nb + 8 * q + 4 * ehalf;
              floatx4 v = floatx4{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
              if (m >= g.M || n >= g.N) continue;
              if (g.vec && n + 4 <= g.N) {
                floatx4_any* P = reinterpret_cast<floatx4_any*>(C + n);
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
              const int n = nb + 16 * q + 8 * ehalf;
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
                  const u32x4 old = *reinterpret_cast<const u32x4_any*>(C);
#pragma unroll
                  for (int e = 0; e < 8; ++e) x[e] += g.beta * widen((uint16_t)(old[e >> 1] >> (16 * (e & 1))));
                }
                u32x4 o;
#pragma unroll
                for (int e = 0; e < 4; ++e) o[e] = g.c_dt == 2 ? pack_bf16(x[2 * e], x[2 * e + 1]) : pack_f16(x[2 * e], x[2 * e + 1]);
                *reinterpret_cast<u32x4_any*>(C) = o;
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
      // 128 columns of the wave's rows: maximum and sum of exponentials; the
      // exponentials against that maximum, rounded to the gradients' type,
      // where the caller wants gradients
      static_assert(FN == 4 || EPI != Epi::SOFTMAX, "a piece is 128 columns");
      constexpr float L2E = 1.4426950408889634f;
      uint32_t target[FM];
#pragma unroll
      for (int i = 0; i < FM; ++i)
        target[i] = reinterpret_cast<const uint32_t*>(smem + TARGETS)[(it & (NG - 1)) * TM + (wm * FM + i) * 32 + el32];
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        const int m = m0 + 32 * i + el32;
        if (n0 + 128 > g.N) {
          const int edge = g.N - n0 - 4 * ehalf;  // columns past the vocabulary count for nothing
#pragma unroll
          for (int j = 0; j < FN; ++j)
#pragma unroll
            for (int v = 0; v < 16; ++v)
              if (32 * j + 8 * (v >> 2) + (v & 3) >= edge) acc[i][j][v] = -INFINITY;
        }
        // The target's logit: the very number that enters the row's sum, so
        // that its rounding drops out of the loss.  One piece of a row has it.
        const uint32_t col = target[i] - (uint32_t)n0;
        const bool here = col < 128u && (int)(col >> 2 & 1) == ehalf && m < g.M;
        if (__any(here)) {
          float zt = 0.f;
#pragma unroll
          for (int j = 0; j < FN; ++j)
#pragma unroll
            for (int v = 0; v < 16; ++v)
              if ((col & ~4u) == 32u * j + 8 * (v >> 2) + (v & 3)) zt = acc[i][j][v];
          if (here) g.target_logit[m] = zt;
        }
        float mx = -INFINITY;
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
          for (int v = 0; v < 16; ++v) mx = fmaxf(mx, acc[i][j][v]);
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
        if (m < g.M && n0 < g.N && ehalf == 0) g.stats[(int64_t)(n0 >> 7) * g.M + m] = floatx2{mx, sum};
        if (g.C) {
          // rows of ldc elements, a multiple of 128: no edge within a piece
#pragma unroll
          for (int j = 0; j < FN; ++j) {
            if constexpr (E == Elem::F32) {
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                const floatx4 v = floatx4{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
                if (m < g.M && n0 < g.N)
                  *reinterpret_cast<floatx4*>(reinterpret_cast<float*>(g.C) + (int64_t)m * g.ldc + n0 + 32 * j + 8 * q + 4 * ehalf) = v;
              }
            } else {
#pragma unroll
              for (int q = 0; q < 2; ++q) {
                uint32_t p0 = pack_bf16(acc[i][j][8 * q], acc[i][j][8 * q + 1]), p1 = pack_bf16(acc[i][j][8 * q + 2], acc[i][j][8 * q + 3]);
                uint32_t p2 = pack_bf16(acc[i][j][8 * q + 4], acc[i][j][8 * q + 5]), p3 = pack_bf16(acc[i][j][8 * q + 6], acc[i][j][8 * q + 7]);
                const auto a = __builtin_amdgcn_permlane32_swap(p0, p2, false, false);
                const auto b = __builtin_amdgcn_permlane32_swap(p1, p3, false, false);
                if (m < g.M && n0 < g.N)
                  *reinterpret_cast<u32x4*>(reinterpret_cast<uint16_t*>(g.C) + (int64_t)m * g.ldc + n0 + 32 * j + 16 * q + 8 * ehalf) =
                      u32x4{a[0], b[0], a[1], b[1]};
              }
            }
          }
        }
      }
    }
    if constexpr (AGAIN) read_frags(rb, 0);
    move_on(cp);
  }
  if constexpr (E == Elem::F8W) {
    if (again == 0) return;
    cp = place_of(first);
#pragma nounroll
    for (int it = 0; it < nitem; ++it, move_on(cp))
      if (again >> min(it, 63) & 1) store_apart(item_at(cp));
  }
}

}  // namespace shampoo
