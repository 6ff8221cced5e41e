// What the tcgen05 kernels of causal chunks share (prefill_umma.cu, window_umma.cu): tile shapes, scores read from
// tensor memory, weights written back to it.
#pragma once

#include <float.h>

#include <algorithm>

#include "pa_common.cuh"
#include "pa_internal.h"
#include "pa_ptx.cuh"

namespace pa {

constexpr int kUmThreads = 352;            // 8 softmax warps, K producer, V producer, MMA
constexpr int kUmTileRows = 128;            // rows per Q tile (MMA M)
constexpr int kUmRows = 2 * kUmTileRows;    // rows per CTA
constexpr int kUmKeys = 128;                // keys per K/V tile (N of S, K of PV)
constexpr int kUmSub = kUmKeys / 16;
constexpr int kUmTmemCols = 512;
constexpr int kUmSegSlots = 8;   // segment records in flight between the K producer and their readers
constexpr int kUmItemSlots = 4;  // item tile counts in flight between the K producer and the MMA warp
// Ring depths (build-time overridable): K 2 / V 3 measured 1 % faster than K 3 / V 2 (V tiles are
// needed later in a tile's chain, so their loads profit from the deeper ring)
#ifndef PA_UM_KSTAGES
#define PA_UM_KSTAGES 2
#endif
#ifndef PA_UM_VSTAGES
#define PA_UM_VSTAGES 3
#endif
constexpr int kUmKStages = PA_UM_KSTAGES;   // K ring depth
constexpr int kUmVStages = PA_UM_VSTAGES;   // V ring depth
constexpr float kUmRescaleThreshold = 8.f;  // log2 units: O is rescaled when the max grows by > 2^8

template <int D>
struct UmCfg {
  static constexpr int kHalves = D / 64;
  static constexpr int kQHalf = kUmTileRows * 128;   // one 64-column half of a Q tile
  static constexpr int kQBytes = kUmTileRows * D * 2;
  static constexpr int kKvHalf = kUmKeys * 128;      // one 64-column half of a K or V tile
  static constexpr int kKvBytes = kUmKeys * D * 2;
  static constexpr int kSmemBytes = 1024 + 1024 + 2 * kQBytes + (kUmKStages + kUmVStages) * kKvBytes;
  static_assert(kSmemBytes <= 227 * 1024, "shared memory per CTA");
};

// Byte offset of (row r, 8-element chunk c) in a [half][rows][128 B] swizzled operand.
__device__ __forceinline__ uint32_t sw_off(int r, int c, int half_bytes) {
  return (uint32_t)((c >> 3) * half_bytes + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}

// Softmax helpers: one thread owns one row of S (its TMEM lane); `taddr` is the row's first column.
//
// One code path serves every tile.  The exponentials are taken as 2^(sc * s - m) with sc > 0, so
// the row maximum can be taken over the raw scores and scaled once.  A tile that has masked keys
// (outside the causal bound, or in a sub-tile that was not loaded), or a non-positive scale, first
// rewrites the loaded scores in registers (ScoreFix): a masked key becomes -inf, whose probability
// is exactly 0.  The common case, keys [0, nv) valid (the causal bound and the end of the loaded
// keys both cut a prefix), costs one compare and select per key of the 64-key blocks that the cut
// falls in, and a block wholly past the cut for every row of the warp is skipped.  Anything else
// (a sub-tile skipped for an out-of-range block id, or a scale <= 0) takes the general rewrite: key c valid when bit c % 32 of mask[c / 32] is set, a negative scale flips
// the sign of every score and uses |scale| (the same products sc * s), a zero scale makes every
// score 0 with scale 1 (the same uniform weights).

__device__ __forceinline__ float fmax3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// v = -inf unless j < nv (one compare, one select)
__device__ __forceinline__ void keep_below(uint32_t& v, int j, int nv) {
  asm("{\n\t.reg .pred p;\n\tsetp.lt.s32 p, %1, %2;\n\tselp.b32 %0, %0, 0xff800000, p;\n\t}"
      : "+r"(v)
      : "r"(j), "r"(nv));
}

struct ScoreFix {
  int mode;       // 0: scores used as loaded; 1: keys >= nv masked; 2: general rewrite
  int nv;         // mode 1: keys [0, nv) of the tile are valid
  uint32_t flip;  // mode 2: sign bit flipped (negative scale)
  bool zero;      // mode 2: scores replaced by 0 (zero scale)
};

// The softmax code runs once per tile on every SM; it is kept compact (one 64-column block in a
// loop, not the whole row unrolled) so that it stays in the instruction cache: fully unrolled rows,
// with a separate masked variant, measured slower from instruction fetch alone.

// Columns [c0, c0 + 64) of the row of S into registers (two loads in flight, one wait), rewritten
// as `fix` says; m0 / m1 are the mask words of the block's two 32-key chunks.  One instantiation
// per masking mode (kMode = fix.mode): mode 0 runs no masking code at all, mode 1 applies the prefix
// cut only in a block that the cut falls in, mode 2 is the rare general rewrite.  (One copy of the
// code for modes 0 and 1, the cut behind a warp-uniform branch, measured slower.)
template <int kMode>
__device__ __forceinline__ void s_load64(uint32_t taddr, uint32_t (&sv)[64], const ScoreFix& fix, int c0,
                                         uint32_t m0, uint32_t m1) {
  tmem_ld32(taddr, *reinterpret_cast<uint32_t(*)[32]>(&sv[0]));
  tmem_ld32(taddr + 32u, *reinterpret_cast<uint32_t(*)[32]>(&sv[32]));
  tmem_wait_ld();
  tmem_pin32(*reinterpret_cast<uint32_t(*)[32]>(&sv[0]));
  tmem_pin32(*reinterpret_cast<uint32_t(*)[32]>(&sv[32]));
  if (kMode == 1) {
    const int nv = fix.nv - c0;
    if (nv < 64) {
#pragma unroll
      for (int j = 0; j < 64; ++j) keep_below(sv[j], j, nv);
    }
  } else if (kMode == 2) {
#pragma unroll
    for (int j = 0; j < 64; ++j) {
      const uint32_t v = fix.zero ? 0u : (sv[j] ^ fix.flip);
      sv[j] = (((j < 32 ? m0 : m1) >> (j & 31)) & 1u) ? v : 0xff800000u;  // -inf
    }
  }
}

// Maximum of the 64 scores held in sv, times sc (> 0).
__device__ __forceinline__ float s_max64(const uint32_t (&sv)[64], float sc) {
  float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
  for (int j = 0; j < 64; j += 8)
#pragma unroll
    for (int u = 0; u < 4; ++u) m[u] = fmax3(m[u], __uint_as_float(sv[j + 2 * u]), __uint_as_float(sv[j + 2 * u + 1]));
  return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])) * sc;
}

// Probabilities 2^(sc * s - m_sub) of the 64 keys held in sv, written as 16-bit pairs into the 32
// columns at taddr (keys 2c and 2c + 1 in column c); returns their sum.  Packed pairs: one f32x2 fma
// for the scaled, shifted arguments and one f32x2 add for the sum.
template <bool kBf16>
__device__ __forceinline__ float p_store64(uint32_t taddr, const uint32_t (&sv)[64], float sc, float m_sub) {
  const uint64_t sc2 = f2_pack(sc, sc), nm2 = f2_pack(-m_sub, -m_sub);
  uint64_t acc2[2] = {f2_pack(0.f, 0.f), f2_pack(0.f, 0.f)};
  uint32_t w[32];
#pragma unroll
  for (int c = 0; c < 32; ++c) {
    float x0, x1;
    f2_unpack(f2_fma(f2_pack(__uint_as_float(sv[2 * c]), __uint_as_float(sv[2 * c + 1])), sc2, nm2), x0, x1);
    const uint64_t e2 = f2_pack(fast_exp2(x0), fast_exp2(x1));
    acc2[c & 1] = f2_add(acc2[c & 1], e2);
    float e0, e1;
    f2_unpack(e2, e0, e1);
    w[c] = pack2<kBf16>(e0, e1);
  }
  tmem_st32(taddr, w);
  float a0, a1, b0, b1;
  f2_unpack(acc2[0], a0, a1);
  f2_unpack(acc2[1], b0, b1);
  return (a0 + b0) + (a1 + b1);
}

}  // namespace pa
