// tcgen05 tree attention (bf16/fp16 pools, block_size % 16 == 0).
//
// Persistent: one CTA per SM walks its equal share of the units (tree_common.cuh).  Per key tile: S = Q K^T
// into a TMEM buffer, the softmax threads (one TMEM lane each) turn it into P in place, O += P V in TMEM;
// one pass with a running stabiliser (a score, unscaled) that moves only when the maximum's weight grows by more than
// 2^8 (numerator and denominator use the same one, so the result is the softmax's in real arithmetic).  K and V
// pass through a ring each that runs on into the next unit while the last one is finished, so that the loads
// never pause at a border.
//
// Two groups of four softmax warps, each with an O of its own.
//   Narrow kernel (no sequence has more than 128 (node, head) rows): bound by HBM (618 MB of a serving batch
//     with up to 16 drafts in 102 us, 1.34 GB of four long documents in 210 us: 6.0 and 6.4 TB/s).  The groups
//     take the key tiles of a unit in turn and their states are joined at its end (both Os lie in the same TMEM
//     lanes, so only (maximum, sum) goes through shared memory, and each group writes half of the columns).  A
//     tile passes every 1,400 cycles at HBM's rate, the round S, softmax, P V through the barriers takes about
//     3,500, so four tiles (three at head_dim 64, which takes 128-key tiles to have the same bytes per round)
//     are in flight; and one thread would need 2,100 cycles for the waits, issues and commits of a tile, so four
//     warps share them (K, V, S, P V), each product's one commit telling the softmax, the producer and the other
//     issuer alike.
//   Wide kernel: bound by the softmax and the tensor core (the serving batch with 48 to 64 drafts, 134 GFLOP:
//     160 us, 0.84 PFLOP/s).  A unit of more than 128 rows has two Q tiles, one per group, that share every
//     128-key K and V tile; each group has one S buffer, and while one computes its softmax the tensor core has
//     the other's products.  (A barrier that is complete already costs its waiter 110-230 cycles, a commit 100:
//     one thread issuing both products took 4,600 cycles a tile without ever having to wait.)  Each group starts
//     on the next unit by itself, and the scores of the first 64 keys of a tile stay in registers between maximum
//     and weights (171 -> 163 us).  A tile takes a group 3,600 cycles: 1,650 of softmax, the rest the round P V, S
//     through the barriers.  All 128 scores of a row in registers, an S buffer for both groups and weights of
//     their own instead took 5,500 (2,700 of softmax).  In a unit of at most 128 rows the groups take tiles in
//     turn.
//
// Masks.  Only tiles that reach into the drafted region look at masks: a row's visibility bits are cut
// out of its mask words.  A masked score becomes -inf by selection, whatever it was.  A masked value cannot
// be deselected (0 * NaN), so in those tiles non-finite elements of V are zeroed in shared memory before
// the product, and added at the end, by themselves, to the rows that see them.
//
// Warps: 0-3 and 4-7 softmax, 8 K and 9 V producer (TMA), 10 Q and S, 11 P V.  Every wait is bounded
// (PA_DEVERR_TIMEOUT).  A wait tells a barrier's phase from the next one only, so each barrier below is
// waited for before its next phase but one can complete.
#include <cudaTypedefs.h>
#include <float.h>

#include <algorithm>

#include "pa_ptx.cuh"
#include "tree_common.cuh"

namespace pa {

// 12 warps: a thirteenth would leave 128 registers a thread
constexpr int kTuThreads = 384;
constexpr float kTuRescale = 8.f;
// fp16 weights are formed 2^7 higher: the largest, 2^(8 + 7), still fits, and what the type's smallest step rounds
// away of a weight is at most 2^-32 of the row's largest (unscaled 2^-25: 131,000 keys of that weight next to one
// strong key lost 0.4 % of the result).  Sums and accumulators carry the factor alike and lose it in the quotient.
constexpr float kTuLift = 7.f;

template <int D, bool kWide>
struct TuCfg {
  static constexpr int kUnitRows = kWide ? 256 : 128;
  static constexpr int kKeys = tree_tile_keys(D, kUnitRows);
  static constexpr int kSubs = kKeys / 16;
  static constexpr int kHalves = D / 64;
  static constexpr int kQHalf = 128 * 128;          // one 64-column half of a 128-row Q tile
  static constexpr int kQTile = kQHalf * kHalves;
  static constexpr int kQBytes = (kWide ? 2 : 1) * kQTile;
  static constexpr int kKvBytes = kKeys * D * 2;    // a stage: one K or V tile
  static constexpr int kGroup = 1024 * kHalves;     // 8 keys of it
  static constexpr int kHead = kWide ? 2048 : 4096;  // barriers, masks, row statistics
  static constexpr int kFit = (227 * 1024 - 1024 - kHead - kQBytes) / kKvBytes;
  static constexpr int kKStages = kFit / 2 < 12 ? kFit / 2 : 12;
  static constexpr int kVStages = kFit - kFit / 2 < 12 ? kFit - kFit / 2 : 12;
  static constexpr int kSmemBytes = 1024 + kHead + kQBytes + (kKStages + kVStages) * kKvBytes;
  // TMEM: S buffers (narrow: tiles in flight; wide: one per group), then the two Os
  static constexpr int kBufs = kWide ? 2 : (512 - 2 * D) / kKeys;
  static constexpr int kOColumn = kBufs * kKeys;
  static_assert(kOColumn + 2 * D <= 512, "tensor memory");
};

// Whether one of the two 16-bit floats in w is infinite or NaN.
template <bool kBf16>
__device__ __forceinline__ bool any_nonfinite(uint32_t w) {
  constexpr uint32_t e = kBf16 ? 0x7f80u : 0x7c00u;
  return (w & e) == e || ((w >> 16) & e) == e;
}

// The pair with its non-finite halves replaced by zero.
template <bool kBf16>
__device__ __forceinline__ uint32_t drop_nonfinite(uint32_t w) {
  constexpr uint32_t e = kBf16 ? 0x7f80u : 0x7c00u;
  if ((w & e) == e) w &= 0xffff0000u;
  if (((w >> 16) & e) == e) w &= 0x0000ffffu;
  return w;
}

__device__ __forceinline__ float fmax3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Scores this thread's row does not see (of 32 consecutive ones, by the bits of keep) become -inf.
__device__ __forceinline__ void tu_select(uint32_t (&sv)[32], uint32_t keep) {
#pragma unroll
  for (int c = 0; c < 32; ++c)
    if (!((keep >> c) & 1u)) sv[c] = 0xff800000u;
}

__device__ __forceinline__ float tu_max(const uint32_t (&sv)[32], float top) {
  float m[4] = {top, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
  for (int c = 0; c < 32; c += 8)
#pragma unroll
    for (int u = 0; u < 4; ++u)
      m[u] = fmax3(m[u], __uint_as_float(sv[c + 2 * u]), __uint_as_float(sv[c + 2 * u + 1]));
  return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}

// Weights 2^(s * sc - m) of 32 scores as 16-bit pairs into the 16 columns at taddr; their sum.  Weights are
// rounded to the pool's type for the product with V, as its tensor-core operand has to be (half a step each, so for
// random values the output's error grows from one rounding's to two's: bf16 1.7e-3 -> 2.3e-3 of the result as root
// mean squares); the sum keeps 32 bits.
template <bool kBf16>
__device__ __forceinline__ float tu_weights(uint32_t taddr, const uint32_t (&sv)[32], float sc, float m) {
  const uint64_t sc2 = f2_pack(sc, sc), nm2 = f2_pack(-m, -m);
  uint64_t sum2[2] = {f2_pack(0.f, 0.f), f2_pack(0.f, 0.f)};
  uint32_t p[16];
#pragma unroll
  for (int c = 0; c < 16; ++c) {
    float x0, x1;
    f2_unpack(f2_fma(f2_pack(__uint_as_float(sv[2 * c]), __uint_as_float(sv[2 * c + 1])), sc2, nm2), x0, x1);
    const float e0 = fast_exp2(x0), e1 = fast_exp2(x1);
    sum2[c & 1] = f2_add(sum2[c & 1], f2_pack(e0, e1));
    p[c] = pack2<kBf16>(e0, e1);
  }
  tmem_st16(taddr, p);
  float a0, a1, b0, b1;
  f2_unpack(sum2[0], a0, a1);
  f2_unpack(sum2[1], b0, b1);
  return (a0 + a1) + (b0 + b1);
}

// The scores of a warp's rows in `columns` columns from taddr on become (s - m) * sc.
__device__ __forceinline__ void tu_distances(uint32_t taddr, int columns, float sc, float m) {
#pragma unroll 1
  for (int c0 = 0; c0 < columns; c0 += 32) {
    uint32_t sv[32];
    tmem_ld32_sync(taddr + (uint32_t)c0, sv);
#pragma unroll
    for (int c = 0; c < 32; ++c) sv[c] = __float_as_uint((__uint_as_float(sv[c]) - m) * sc);
    tmem_st32(taddr + (uint32_t)c0, sv);
  }
  tmem_wait_st();
}

template <typename T, int D, bool kWide>
__global__ void __launch_bounds__(kTuThreads, 1)
    tree_umma_kernel(const TreeArgs a, const __grid_constant__ CUtensorMap kmap,
                     const __grid_constant__ CUtensorMap vmap, const __grid_constant__ CUtensorMap qmap) {
  using Cfg = TuCfg<D, kWide>;
  using Walk = TreeWalk<Cfg::kKeys>;
  constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
  constexpr int kHalves = Cfg::kHalves, kKeys = Cfg::kKeys, kSubs = Cfg::kSubs;
  constexpr int kKStages = Cfg::kKStages, kVStages = Cfg::kVStages, kBufs = Cfg::kBufs;
  constexpr int kUnitRows = Cfg::kUnitRows;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  // Tile t of the CTA (counted over its units): K stage t % kKStages, V stage t % kVStages, narrow: S buffer
  // t % kBufs and group t % 2.  "Item": a tile's scores of one group.
  uint64_t* bars = reinterpret_cast<uint64_t*>(base);
  uint64_t* kfull = bars;          // [kKStages] the tile's keys landed
  uint64_t* vfull = bars + 12;     // [kVStages] its values
  uint64_t* sdone = bars + 24;     // [kKStages] the S products of the tile are done (the K stage is free)
  uint64_t* vdone = bars + 36;     // [kVStages] the P V products of the tile are done (the V stage is free)
  uint64_t* p_full = bars + 48;    // [kBufs] the buffer's weights are written (and O rescaled)
  uint64_t* q_full = bars + 52;    // one phase per unit
  uint64_t* o_full = bars + 53;    // wide: one phase per unit of one Q tile: both Os complete
  uint64_t* ml_full = bars + 54;   // one phase per unit whose groups are joined: statistics written
  uint64_t* fin = bars + 55;       // [2] all products of an issuer are over
  uint64_t* s_full = bars + 61;    // [2] wide: the group's scores are written, one phase per item
  uint64_t* pv_done = bars + 57;   // [2] wide: O += P V of the group's item done, one phase per item
  uint64_t* o_free = bars + 59;    // [2] one phase per unit: the Os read (narrow: both, [0]; wide: each)
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(base + 504);
  volatile int* bad_v = reinterpret_cast<int*>(base + 508);  // V of a drafted region held non-finite elements
  volatile uint32_t* kmask = reinterpret_cast<uint32_t*>(base + 512);  // [32] 16-key sub-tiles loaded, per tile
  TreeSched* sched = reinterpret_cast<TreeSched*>(base + 640);
  // (maximum, sum) per row: narrow [2][128], of both groups; wide [128], of group 1
  float2* ml = reinterpret_cast<float2*>(base + (kWide ? 1024 : 2048));
  static_assert(640 + sizeof(TreeSched) <= (kWide ? 1024 : 2048) && kKStages <= 12 && kVStages <= 12, "head");
  // (S of tile t + kBufs waits for P V of tile t, and phases stay one apart only if the rings are not shorter)
  static_assert(kWide || (kKStages >= kBufs && kVStages >= kBufs && kBufs <= 4), "ring depths");
  static_assert(kKStages >= 2 && kVStages >= 2, "ring depths");
  uint8_t* qs = base + Cfg::kHead;
  uint8_t* ks = qs + Cfg::kQBytes;
  uint8_t* vs = ks + kKStages * Cfg::kKvBytes;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    prefetch_tensormap(&kmap);
    prefetch_tensormap(&vmap);
    prefetch_tensormap(&qmap);
    for (int k = 0; k < kKStages; ++k) {
      mbar_init(&kfull[k], 1);
      mbar_init(&sdone[k], 1);
    }
    for (int k = 0; k < kVStages; ++k) {
      mbar_init(&vfull[k], 1);
      mbar_init(&vdone[k], 1);
    }
    for (int k = 0; k < kBufs; ++k) mbar_init(&p_full[k], 4);
    mbar_init(q_full, 1);
    mbar_init(&o_free[0], kWide ? 4 : 8);
    mbar_init(&o_free[1], 4);
    mbar_init(ml_full, 8);
    mbar_init(&fin[0], 1);
    mbar_init(&fin[1], 1);
    mbar_init(&s_full[0], 1);
    mbar_init(&s_full[1], 1);
    mbar_init(&pv_done[0], 1);
    mbar_init(&pv_done[1], 1);
    mbar_init(o_full, 1);
    *bad_v = 0;
    tree_schedule_init(a, *sched);
    fence_barrier_init();
  }
  if (warp == 10) tmem_alloc(tmem_slot, 512);
  __syncthreads();
  // nothing of global memory is read or written before the preceding grid is over
  pdl_wait_primary();
  pdl_launch_dependents();
  const int nodes_unit = kUnitRows >> a.group_shift;
  tree_schedule<kTuThreads, kKeys, kTreeGap, kTreeMinShare>(a, nodes_unit, *sched);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const TreeSpan span = sched->span;
  auto tS = [&](int buf) { return tmem + (uint32_t)(kKeys * buf); };  // wide: buffer = group
  auto tO = [&](int g) { return tmem + (uint32_t)(Cfg::kOColumn + D * g); };

  // the Q tiles of a unit (one thread)
  auto load_q = [&](const TreeUnit& w) {
    const int tiles = kWide && w.rows > 128 ? 2 : 1;
    mbar_arrive_expect_tx(q_full, tiles * Cfg::kQTile);
    for (int k = 0; k < tiles; ++k)
#pragma unroll
      for (int h = 0; h < kHalves; ++h)
        tma_load_3d(qs + k * Cfg::kQTile + h * Cfg::kQHalf, &qmap, h * 64, w.kvh << a.group_shift,
                    (int)(w.sq.q0 + w.node0) + k * (128 >> a.group_shift), q_full);
  };

  if (warp == 8 || warp == 9) {
    // ------------------------------- producers: warp 8 K, warp 9 V --------------------------------
    // One box is 8 x (up to 8) keys x head_dim of one block: a tile takes kKeys / min(block_size, 64) of them,
    // one per lane, and lies in shared memory as [8-key group][64-column half][8][128 bytes, swizzled].
    const bool is_v = warp == 9;
    uint64_t* full = is_v ? vfull : kfull;
    uint64_t* freed = is_v ? vdone : sdone;
    uint8_t* ring = is_v ? vs : ks;
    const CUtensorMap* map = is_v ? &vmap : &kmap;
    const int depth = is_v ? kVStages : kKStages;
    const int box_keys = min(a.block_size, 64), boxes = kKeys / box_keys;
    const uint64_t once = l2_policy_evict_first();
    int t = 0, s = 0, round = 0;
    bool alive = true;
    Walk walk(a, span, nodes_unit);
    TreeUnit w;
    while (alive && walk.next(w)) {
      const int32_t* table = a.block_table + (int64_t)w.b * a.bt_stride;
      // table entry of this lane's box of tile x of the unit (-1: behind the context)
      auto entry = [&](int x) -> int {
        const int pos = x * kKeys + lane * box_keys;
        return lane < boxes && x < w.x1 && pos < w.sq.n ? ld_s32(table + (pos >> a.block_shift)) : -1;
      };
      int blk = entry(w.x0);
      for (int x = w.x0; x < w.x1; ++x, ++t) {
        const int blk_next = entry(x + 1);
        if (round > 0 && !__all_sync(0xffffffffu, mbar_wait(&freed[s], (unsigned)((round - 1) & 1), a.err, a.epoch))) {
          alive = false;
          break;
        }
        const int pos = x * kKeys + lane * box_keys;
        const bool in = lane < boxes && pos < w.sq.n;
        const bool ok = in && blk >= 0 && blk < a.num_blocks;
        if (in && !ok && !is_v) raise_error(a.err, PA_DEVERR_BLOCK_ID);
        const unsigned lanes = __ballot_sync(0xffffffffu, ok);
        if (lane == 0) {
          if (!is_v) {
            // 16-key sub-tiles that hold data.  Read after S of the tile, which waits for the arrival
            // below; tile t - 32, the slot's last, is more than a ring ago.
            uint32_t m = 0;
            const int per = box_keys / 16;
            for (int k = 0; k < boxes; ++k)
              if ((lanes >> k) & 1u) m |= ((1u << per) - 1u) << (k * per);
            kmask[t & 31] = m;
          }
          if (lanes != 0) mbar_arrive_expect_tx(&full[s], (unsigned)(__popc(lanes) * box_keys * D * 2));
          else mbar_arrive(&full[s]);
        }
        __syncwarp();
        if (ok) {
          // the last reader of the keys marks them first to be evicted
          uint8_t* dst = ring + s * Cfg::kKvBytes + lane * box_keys * D * 2;
          const int group = (pos & (a.block_size - 1)) >> 3;
          if (w.last_tile) tma_load_5d_hint(dst, map, 0, 0, w.kvh * kHalves, group, blk, &full[s], once);
          else tma_load_5d(dst, map, 0, 0, w.kvh * kHalves, group, blk, &full[s]);
        }
        blk = blk_next;
        if (++s == depth) {
          s = 0;
          ++round;
        }
      }
    }
    if (lane == 0) {
      if (!alive) raise_timeout(a.err, a.epoch);
      // leave no copy in flight, whatever the other warps have made of this launch: the last load of each
      // stage (the stage is not loaded again after it)
      for (int k = t > depth ? t - depth : 0; k < t; ++k) mbar_wait(&full[k % depth], (unsigned)((k / depth) & 1));
    }
    __syncwarp();
  } else if (warp == 10 || warp == 11) {
    // ------------------------- products: warp 10 Q and S, warp 11 P V ------------------------------
    if (lane == 0) {
      const uint32_t id_s = umma_idesc_f16(kBf16, 128, kKeys, false, false);
      const uint32_t id_pv = umma_idesc_f16(kBf16, 128, D, false, true);
      const uint64_t qd = umma_desc_sw128(smem_u32(qs), 16, 1024), kd = umma_desc_sw128(smem_u32(ks), 16, Cfg::kGroup);
      const uint64_t vd = umma_desc_sw128(smem_u32(vs), 1024, Cfg::kGroup);
      bool ok = true;
      auto wait = [&](uint64_t* bar, int phase) {
        ok = ok && mbar_wait(bar, (unsigned)(phase & 1), a.err, a.epoch);
        return ok;
      };
      auto s_product = [&](int buf, int q_tile, int stage) {
        const uint64_t q = qd + (uint64_t)(q_tile * (Cfg::kQTile >> 4)), k = kd + (uint64_t)(stage * (Cfg::kKvBytes >> 4));
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          umma_ss(tS(buf), q + (kk >> 2) * (Cfg::kQHalf >> 4) + (kk & 3) * 2, k + (kk >> 2) * 64 + (kk & 3) * 2, id_s,
                  kk > 0 ? 1u : 0u);
      };
      auto pv_product = [&](int g, int buf, int stage, bool first) {
        const uint64_t v = vd + (uint64_t)(stage * (Cfg::kKvBytes >> 4));
#pragma unroll
        for (int kk = 0; kk < kKeys / 16; ++kk)
          umma_ts(tO(g), tS(buf) + 8u * (uint32_t)kk, v + kk * (2 * Cfg::kGroup >> 4), id_pv, kk > 0 || !first ? 1u : 0u);
      };
      Walk walk(a, span, nodes_unit);
      TreeUnit w;
      int un = 0;
      int t = 0, s = 0, round = 0;  // tiles so far, ring stage and round
      int done0 = 0, done1 = 0;     // wide: items of each group so far
      if (warp == 10) {
        while (ok && walk.next(w)) {
          // Q is free once the S products of the unit before are done
          if (t > 0 && !wait(&sdone[(t - 1) % kKStages], (t - 1) / kKStages)) break;
          load_q(w);
          if (!wait(q_full, un)) {
            mbar_wait(q_full, (unsigned)(un & 1));  // no copy in flight
            break;
          }
          const bool pair = kWide && w.rows > 128;
          for (int x = w.x0; x < w.x1 && ok; ++x, ++t) {
            // an S overwrites weights: of the tile kBufs before (narrow), of the group's item before (wide)
            if (!kWide && t >= kBufs && !wait(&vdone[(t - kBufs) % kVStages], (t - kBufs) / kVStages)) break;
            if (!wait(&kfull[s], round)) break;
            for (int g = kWide && !pair ? (x - w.x0) & 1 : 0, last = pair ? 1 : g; g <= last; ++g) {
              if (kWide) {
                const int done = g ? done1++ : done0++;
                if (done > 0 && !wait(&pv_done[g], done - 1)) break;
              }
              tc_fence_after();
              s_product(kWide ? g : t % kBufs, pair ? g : 0, s);
              if (kWide) umma_commit(&s_full[g]);
            }
            if (!ok) break;
            umma_commit(&sdone[s]);
            if (++s == kKStages) {
              s = 0;
              ++round;
            }
          }
          ++un;
        }
      } else {
        while (ok && walk.next(w)) {
          const bool pair = kWide && w.rows > 128;
          // the unit's first products overwrite the Os that the unit before it left
          if (!kWide && un > 0 && !wait(o_free, un - 1)) break;
          for (int x = w.x0; x < w.x1 && ok; ++x, ++t) {
            const int i = x - w.x0;
            if (!wait(&vfull[s], round)) break;
            for (int g = kWide ? (pair ? 0 : i & 1) : t & 1, last = pair ? 1 : g; g <= last; ++g) {
              if (kWide && un > 0 && i < (pair ? 1 : 2) && !wait(&o_free[g], un - 1)) break;
              const int phase = kWide ? (g ? done1++ : done0++) : t / kBufs;
              if (!wait(&p_full[kWide ? g : t % kBufs], phase)) break;
              tc_fence_after();
              pv_product(g, kWide ? g : t % kBufs, s, pair ? i == 0 : i < 2);
              if (kWide) umma_commit(&pv_done[g]);
            }
            if (!ok) break;
            umma_commit(&vdone[s]);
            if (++s == kVStages) {
              s = 0;
              ++round;
            }
          }
          if (kWide && !pair) {
            if (w.x1 - w.x0 == 1 && un > 0 && !wait(&o_free[1], un - 1)) break;  // (no phase is left out)
            if (ok) umma_commit(o_full);
          }
          ++un;
        }
      }
      if (!ok) raise_timeout(a.err, a.epoch);
      umma_commit(&fin[warp - 10]);  // no product in flight when the tensor memory is given back
      mbar_wait(&fin[warp - 10], 0);
    }
    __syncwarp();
  } else {
    // ---------------------------------------- softmax --------------------------------------------
    const int grp = warp >> 2;
    const int r = threadIdx.x & 127;  // row of the group's tile = TMEM lane
    const uint32_t lane_base = (uint32_t)(32 * (warp & 3)) << 16;
    // rows are 16-byte aligned at least; whole 32-byte sectors per thread halve the store traffic
    const bool aligned = ((reinterpret_cast<uintptr_t>(a.out) | reinterpret_cast<uintptr_t>(a.ws_acc)) & 31u) == 0;
    int t = 0, un = 0, item = 0, solo = 0;  // tiles of earlier units, those, this group's items, joined units
    bool alive = true, cut = false;
    Walk walk(a, span, nodes_unit);
    TreeUnit w;
    while (alive && walk.next(w)) {
      const int n = w.x1 - w.x0;
      const int hist = w.sq.n - w.sq.m;
      const bool pair = kWide && w.rows > 128;                        // two Q tiles, one per group
      const int rows = pair ? min(128, w.rows - 128 * grp) : w.rows;  // of this group's tile
      const bool live = (r & ~31) < rows;                             // whole warps
      const int node = w.node0 + (pair ? grp * (128 >> a.group_shift) : 0) + (min(r, rows - 1) >> a.group_shift);
      const int64_t* words = a.tree_mask != nullptr ? a.tree_mask + (w.sq.q0 + node) * a.mask_words : nullptr;
      // (read before it is needed: most trees have one mask word, and no tile reaches it before the first)
      const uint64_t word0 = words != nullptr && live ? (uint64_t)ld_s64(words) : 0ull;
      float m_use = -INFINITY, l_run = 0.f;

      // Bits of the 64 keys from kb on that this row sees (bit c: key kb + c); `loaded`: their sub-tiles
      // that hold data.
      auto visible = [&](int kb, uint32_t loaded) -> uint64_t {
        const int nv = w.sq.n - kb;
        if (nv <= 0) return 0ull;
        const int s0 = kb - hist;  // node of the first key
        uint64_t keep;
        if (s0 + 64 <= 0) {
          keep = ~0ull;
        } else if (words == nullptr) {
          const int c = node + 1 - s0;  // chain: nodes up to its own
          keep = c <= 0 ? 0ull : (c >= 64 ? ~0ull : (1ull << c) - 1ull);
        } else if (s0 < 0) {
          keep = (word0 << -s0) | ((1ull << -s0) - 1ull);
        } else {
          const int i = s0 >> 6, sh = s0 & 63;
          keep = (i == 0 ? word0 : (i < a.mask_words ? (uint64_t)ld_s64(words + i) : 0ull)) >> sh;
          if (sh != 0 && i + 1 < a.mask_words) keep |= (uint64_t)ld_s64(words + i + 1) << (64 - sh);
        }
        if (nv < 64) keep &= (1ull << nv) - 1ull;
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (!((loaded >> u) & 1u)) keep &= ~(0xffffull << (16 * u));
        return keep;
      };

      // Scores of S buffer buf into weights; `before` >= 0: the group's previous tile of the unit.
      // kMasked: the tile may hold keys that the row does not see.
      auto tile = [&](auto masked, int buf, uint64_t keep0, uint64_t keep1, int before) {
        constexpr bool kMasked = decltype(masked)::value;
        const uint32_t srow = tS(buf) + lane_base;
        // Blocks of 64 keys.  128 are read twice but for the first block (maximum, weights), as a whole row does not
        // stay in registers, and the loops keep the code in the instruction cache.  Weights go to columns whose
        // scores have been read by then.
        int last = kKeys / 64 - 1;  // the last block that a row of the warp sees
        if (kMasked && kKeys == 128 && __all_sync(0xffffffffu, keep1 == 0ull)) last = 0;
        uint32_t lo[32], hi[32];
        auto load = [&](int h) {
          const uint64_t keep = h ? keep1 : keep0;
          tmem_ld32(srow + 64u * h, lo);
          tmem_ld32(srow + 64u * h + 32u, hi);
          tmem_wait_ld();
          tmem_pin32(lo);
          tmem_pin32(hi);
          if (kMasked) {
            tu_select(lo, (uint32_t)keep);
            tu_select(hi, (uint32_t)(keep >> 32));
          }
        };
        float top = -INFINITY, sum = 0.f;
#pragma unroll 1
        for (int h = last; h >= 0; --h) {
          load(h);
          top = tu_max(lo, top);
          top = tu_max(hi, top);
        }
        if (!kMasked || (keep0 | keep1) != 0) top = fmaxf(top, -FLT_MAX);  // keys were seen, whatever their scores
        float corr = 1.f;
        if ((top - m_use) * a.scale_log2 > kTuRescale) {
          corr = fast_exp2((m_use - top) * a.scale_log2);  // m_use = -inf: 0
          m_use = top;
        }
        // s * sc - m * sc in one rounding, but where m * sc of a row is itself rounded by more than an eighth: that
        // stays in the exponent, and scores of 2^31 had infinite weights.  There the warp's scores are replaced by
        // their scaled distances first (differences for every row: 1.5 % longer over 19 shapes, up to 11 % for one).
        constexpr float kLift = kBf16 ? 0.f : kTuLift;
        const float m_sub = m_use == -INFINITY ? 0.f : m_use;
        float w_scale = a.scale_log2, w_sub = m_sub * a.scale_log2 - kLift;
        const bool far = __any_sync(0xffffffffu, !(fabsf(w_sub) <= 1048576.f));
        if (far) {
          if (kKeys == 128) {
            tu_distances(srow, kKeys, a.scale_log2, m_sub);
          } else {  // (all 64 are in registers)
#pragma unroll
            for (int c = 0; c < 32; ++c) {
              lo[c] = __float_as_uint((__uint_as_float(lo[c]) - m_sub) * a.scale_log2);
              hi[c] = __float_as_uint((__uint_as_float(hi[c]) - m_sub) * a.scale_log2);
            }
          }
          w_scale = 1.f;
          w_sub = -kLift;
        }
#pragma unroll 1
        for (int h = 0; h <= last; ++h) {
          if (kKeys == 128 && (h > 0 || far)) load(h);
          sum += tu_weights<kBf16>(srow + 32u * h, lo, w_scale, w_sub);
          sum += tu_weights<kBf16>(srow + 32u * h + 16u, hi, w_scale, w_sub);
        }
        if (kMasked && kKeys == 128 && last == 0) {
          uint32_t z[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) z[i] = 0u;
          tmem_st32(srow + 32u, z);
        }
        l_run = l_run * corr + sum;
        if (before >= 0 && __any_sync(0xffffffffu, corr != 1.f)) {
          // O is stable once the product of the group's previous tile is done (wide: this tile's S waited for
          // it); this tile's waits for us
          if (!kWide && !__all_sync(0xffffffffu, mbar_wait(&vdone[before % kVStages],
                                                           (unsigned)((before / kVStages) & 1), a.err, a.epoch))) {
            alive = false;
            return;
          }
          tc_fence_after();
#pragma unroll 1
          for (int c0 = 0; c0 < D; c0 += 32) {
            uint32_t v[32];
            tmem_ld32_sync(tO(grp) + lane_base + c0, v);
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * corr);
            tmem_st32(tO(grp) + lane_base + c0, v);
          }
        }
      };

      const int step = pair ? 1 : 2;
      for (int i = pair ? 0 : (kWide ? grp : ((grp - t) & 1)); i < n; i += step, ++item) {
        const int ti = t + i, buf = kWide ? grp : ti % kBufs, before = i < step ? -1 : ti - step;
        const int kb = (w.x0 + i) * kKeys;
        uint64_t* scores = kWide ? &s_full[grp] : &sdone[ti % kKStages];
        if (!__all_sync(0xffffffffu, mbar_wait(scores, (unsigned)((kWide ? item : ti / kKStages) & 1), a.err, a.epoch))) {
          alive = false;
          break;
        }
        tc_fence_after();
        const uint32_t loaded = kmask[ti & 31];
        if (kb + kKeys <= hist && loaded == (1u << kSubs) - 1u) {
          if (live) tile(std::false_type{}, buf, ~0ull, ~0ull, before);
        } else {
          if (live)
            tile(std::true_type{}, buf, visible(kb, loaded & 15u), kKeys == 128 ? visible(kb + 64, loaded >> 4) : 0ull,
                 before);
          if (!pair || grp == 0) {
            // V of the tile: rows without a token zeroed, non-finite elements of drafted tokens taken out
            // (pair: the other group's product is issued after this one's)
            if (!__all_sync(0xffffffffu, mbar_wait(&vfull[ti % kVStages], (unsigned)((ti / kVStages) & 1), a.err,
                                                   a.epoch))) {
              alive = false;
              break;
            }
            // one thread: one 16-byte column of every 8th (16th) key
            uint8_t* col = vs + (ti % kVStages) * Cfg::kKvBytes;
            const int c = r % (8 * kHalves), key0 = r / (8 * kHalves);
            constexpr int kStep = 128 / (8 * kHalves);  // 8 or 16: the swizzle stays the same
            col += (c >> 3) * 1024 + (key0 & 7) * 128 + (((c & 7) ^ (key0 & 7)) << 4);
            const bool all = loaded == (1u << kSubs) - 1u;
            // (keys of the history that are loaded stay as they are)
            for (int key = key0 + (all ? max(0, hist - kb) / kStep * kStep : 0); key < kKeys; key += kStep) {
              uint4* p = reinterpret_cast<uint4*>(col + (key >> 3) * Cfg::kGroup);
              if (kb + key >= w.sq.n || !((loaded >> (key >> 4)) & 1u)) {
                *p = make_uint4(0, 0, 0, 0);
              } else if (kb + key >= hist) {
                uint4 x = *p;
                if (any_nonfinite<kBf16>(x.x) || any_nonfinite<kBf16>(x.y) || any_nonfinite<kBf16>(x.z) ||
                    any_nonfinite<kBf16>(x.w)) {
                  x.x = drop_nonfinite<kBf16>(x.x);
                  x.y = drop_nonfinite<kBf16>(x.y);
                  x.z = drop_nonfinite<kBf16>(x.z);
                  x.w = drop_nonfinite<kBf16>(x.w);
                  *p = x;
                  *bad_v = 1;
                }
              }
            }
            fence_proxy_async_smem();
          }
        }
        if (!alive) break;
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[buf]);
      }
      // the Os that this group reads: its own (pair), or both (products complete in the order in which their one
      // thread issued them)
      const int end = t + n - 1;
      uint64_t* complete = !kWide ? &vdone[end % kVStages] : pair ? &pv_done[grp] : o_full;
      const int phase = !kWide ? end / kVStages : pair ? item - 1 : solo;
      if (alive) alive = __all_sync(0xffffffffu, mbar_wait(complete, (unsigned)(phase & 1), a.err, a.epoch));
      if (!alive) break;
      tc_fence_after();

      // ---- the unit's rows: the output, or this CTA's piece of it ----------------------------------
      const bool whole = w.x0 == 0 && w.x1 == w.T;
      const int64_t row0 = (w.sq.q0 + w.node0) * a.n_q_heads + ((int64_t)w.kvh << a.group_shift);
      const int ur = pair ? 128 * grp + r : r;  // row of the unit
      const int64_t qh = row0 + (int64_t)(ur >> a.group_shift) * a.n_q_heads + (ur & (a.group - 1));
      const int64_t piece = ((int64_t)blockIdx.x * 2 + (w.x0 == 0 ? 1 : 0)) * kUnitRows + ur;
      // what this thread writes: columns [c_begin, c_end) of f0 O_0 + f1 O_1 (factors of absent Os unused)
      bool use0 = grp == 0, use1 = grp == 1;
      float M = m_use, L = l_run, f0 = 1.f, f1 = 1.f;
      int c_begin = 0, c_end = D;
      if (!pair) {
        if (!kWide || grp == 1) ml[kWide ? r : 128 * grp + r] = make_float2(m_use, l_run);
        __syncwarp();
        if (lane == 0) mbar_arrive(ml_full);
        if (kWide && grp == 1) {
          c_end = 0;  // group 0 writes the unit
        } else {
          if (!__all_sync(0xffffffffu, mbar_wait(ml_full, (unsigned)(solo & 1), a.err, a.epoch))) {
            alive = false;
            break;
          }
          const int first = kWide ? 0 : t & 1;  // the group of the unit's first tile
          use0 = n > 1 || first == 0;
          use1 = n > 1 || first == 1;
          const float2 s0 = kWide ? make_float2(m_use, l_run) : ml[r], s1 = ml[kWide ? r : 128 + r];
          M = fmaxf(s0.x, s1.x);
          const float M0 = M == -INFINITY ? 0.f : M;
          f0 = fast_exp2((s0.x - M0) * a.scale_log2);
          f1 = fast_exp2((s1.x - M0) * a.scale_log2);
          L = fmaf(s0.y, f0, s1.y * f1);
          if (!kWide) {
            c_begin = grp * (D / 2);
            c_end = c_begin + D / 2;
          }
        }
        ++solo;
      }
      const bool none = M == -INFINITY;  // the row sees none of these keys
      const float norm = whole ? (none ? 0.f : 1.f / L) : 1.f;
      if (live) {
#pragma unroll 1
        for (int c0 = c_begin; c0 < c_end; c0 += 32) {
          float acc[32];
          uint32_t v[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) acc[i] = 0.f;
          if (use0) {
            tmem_ld32_sync(tO(0) + lane_base + c0, v);
#pragma unroll
            for (int i = 0; i < 32; ++i) acc[i] = __uint_as_float(v[i]) * f0;
          }
          if (use1) {
            tmem_ld32_sync(tO(1) + lane_base + c0, v);
#pragma unroll
            for (int i = 0; i < 32; ++i) acc[i] = fmaf(__uint_as_float(v[i]), f1, acc[i]);
          }
          if (r < rows) {
            if (*bad_v != 0) {
              // the non-finite elements that were taken out of V, for the rows that see them
              const int32_t* table = a.block_table + (int64_t)w.b * a.bt_stride;
              const int last = min(w.x1 * kKeys, w.sq.n);
              for (int pos = max(w.x0 * kKeys, hist); pos < last; ++pos) {
                const int s = pos - hist;
                const int blk = ld_s32(table + (pos >> a.block_shift));
                if (!tree_sees(words, node, s) || blk < 0 || blk >= a.num_blocks) continue;
                const T* vr = static_cast<const T*>(a.v_pool) + (int64_t)blk * a.kv_block_stride +
                              ((int64_t)(pos & (a.block_size - 1)) * a.n_kv_heads + w.kvh) * D + c0;
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                  const float x = static_cast<float>(vr[i]);
                  if (!(fabsf(x) <= FLT_MAX)) acc[i] += x;
                }
              }
            }
            if (whole) {
              T* o = static_cast<T*>(a.out) + qh * D + c0;
#pragma unroll
              for (int i = 0; i < 32; i += 16) {
                uint32_t x[8];
#pragma unroll
                for (int e = 0; e < 8; ++e)
                  x[e] = none ? 0u : pack2<kBf16>(acc[i + 2 * e] * norm, acc[i + 2 * e + 1] * norm);
                st_global32(o + i, x, aligned);
              }
            } else {
              float* o = a.ws_acc + piece * D + c0;
#pragma unroll
              for (int i = 0; i < 32; i += 8) {
                uint32_t x[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = none ? 0u : __float_as_uint(acc[i + e]);
                st_global32(o + i, x, aligned);
              }
            }
          }
        }
        if (!whole && r < rows && (pair || grp == 0)) {
          a.ws_m[piece] = M;
          a.ws_l[piece] = none ? 0.f : L;
        }
      }
      // O has been read: the next unit's first products may overwrite it
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (!kWide) {
          mbar_arrive(o_free);
        } else if (pair) {
          mbar_arrive(&o_free[grp]);
        } else if (grp == 0) {  // (it has read both)
          mbar_arrive(&o_free[0]);
          mbar_arrive(&o_free[1]);
        }
      }
      if (!whole && w.x0 == 0) {
        cut = true;  // at most one unit of a CTA: the one that its span ends in
        if (threadIdx.x == 0) tree_record(a, *sched, w, row0, a.ws_rec + blockIdx.x);
      }
      t += n;
      ++un;
    }
    if (!alive && lane == 0) raise_timeout(a.err, a.epoch);
    if (threadIdx.x == 0 && !cut && a.split) a.ws_rec[blockIdx.x].rows = 0;
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 10) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (sched->refused) tree_zero_refused<T>(a);
}

// ------------------------------------------------------------------------------------------------
// Units cut between CTAs: CTA c's second piece (its first tiles), then the first pieces of the CTAs
// up to `last`, joined like any partitions.  One warp per row, eight to a block: bound by its three dependent
// reads and by the blocks' launches (blocks of four rows 4 % slower over batches of short contexts, of two 15 %; a
// few blocks that loop over the rows 3 to 10 %).
constexpr int kTjWarps = 8;

template <typename T, int D>
__global__ void __launch_bounds__(kTjWarps * 32) tree_join_kernel(const TreeArgs a, int unit_rows) {
  constexpr int kPer = D / 32;  // columns of a lane
  using Vec = typename std::conditional<kPer == 4, float4, float2>::type;
  const int lane = threadIdx.x & 31;
  const int c = blockIdx.y;
  pdl_launch_dependents();
  pdl_wait_primary();
  const TreeRec rec = a.ws_rec[c];
  const int r = blockIdx.x * kTjWarps + (threadIdx.x >> 5);
  if (r >= rec.rows) return;
  const int pieces = rec.last - c + 1;
  auto piece = [&](int i) -> int64_t { return ((int64_t)(c + i) * 2 + (i == 0 ? 1 : 0)) * unit_rows + r; };
  auto columns = [&](int64_t p) { return *reinterpret_cast<const Vec*>(a.ws_acc + p * D + lane * kPer); };
  // a unit has two pieces, or the rare long one more: the first two are read at once, before their maxima
  const int64_t p0 = piece(0), p1 = piece(1);
  const float m0 = a.ws_m[p0], m1 = a.ws_m[p1], l0 = a.ws_l[p0], l1 = a.ws_l[p1];
  const Vec v0 = columns(p0), v1 = columns(p1);
  float M = fmaxf(m0, m1);
  for (int i = 2 + lane; i < pieces; i += 32) M = fmaxf(M, a.ws_m[piece(i)]);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
  const float base = M == -INFINITY ? 0.f : M;
  float L = 0.f, acc[kPer];
#pragma unroll
  for (int k = 0; k < kPer; ++k) acc[k] = 0.f;
  auto add = [&](float m, float l, const Vec& v) {
    const float f = fast_exp2((m - base) * a.scale_log2);
    L = fmaf(l, f, L);
    const float* x = reinterpret_cast<const float*>(&v);
#pragma unroll
    for (int k = 0; k < kPer; ++k) acc[k] = fmaf(x[k], f, acc[k]);
  };
  add(m0, l0, v0);
  add(m1, l1, v1);
#pragma unroll 4
  for (int i = 2; i < pieces; ++i) {
    const int64_t p = piece(i);
    add(a.ws_m[p], a.ws_l[p], columns(p));
  }
  const int64_t qh = rec.row0 + (int64_t)(r >> a.group_shift) * a.n_q_heads + (r & (a.group - 1));
  T* o = static_cast<T*>(a.out) + qh * D + lane * kPer;
  alignas(16) T x[kPer];
#pragma unroll
  for (int k = 0; k < kPer; ++k) x[k] = Elt<T>::from_float(M == -INFINITY ? 0.f : acc[k] / L);
  if constexpr (sizeof(x) == 16) *reinterpret_cast<uint4*>(o) = *reinterpret_cast<const uint4*>(x);
  else if constexpr (sizeof(x) == 8) *reinterpret_cast<uint2*>(o) = *reinterpret_cast<const uint2*>(x);
  else *reinterpret_cast<uint32_t*>(o) = *reinterpret_cast<const uint32_t*>(x);
}

// ------------------------------------------------------------------------------------------------
template <typename T, int D, bool kWide>
static cudaError_t launch_tu(const TreeArgs& a, const CUtensorMap& km, const CUtensorMap& vm, cudaStream_t s) {
  CUtensorMap qm;
  if (!encode_q_map(&qm, a.q, std::is_same<T, __nv_bfloat16>::value ? PA_BF16 : PA_FP16, a.total_q, a.n_q_heads, D,
                    a.group, 128 / a.group))
    return cudaErrorInvalidValue;
  constexpr int smem = TuCfg<D, kWide>::kSmemBytes;
  static bool attr_set[64] = {};  // per instantiation and device; idempotent, so a race is harmless
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !attr_set[dev]) {
    e = cudaFuncSetAttribute(tree_umma_kernel<T, D, kWide>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) attr_set[dev] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.ctas);
  cfg.blockDim = dim3(kTuThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, tree_umma_kernel<T, D, kWide>, a, km, vm, qm);
}

template <typename T, int D>
static cudaError_t launch_tu_rows(const TreeArgs& a, const CUtensorMap& km, const CUtensorMap& vm, cudaStream_t s) {
  return tree_unit_rows(a.max_nodes, a.group) == 128 ? launch_tu<T, D, false>(a, km, vm, s)
                                                     : launch_tu<T, D, true>(a, km, vm, s);
}

cudaError_t launch_tree_umma(const TreeArgs& a, pa_dtype dt, cudaStream_t s, int* launches) {
  CUtensorMap km, vm;
  if (!encode_group_map(&km, a.k_pool, dt, a.num_blocks, a.block_size, a.n_kv_heads, a.head_dim, a.kv_block_stride) ||
      !encode_group_map(&vm, a.v_pool, dt, a.num_blocks, a.block_size, a.n_kv_heads, a.head_dim, a.kv_block_stride))
    return cudaErrorInvalidValue;
  cudaError_t e;
  if (dt == PA_BF16)
    e = a.head_dim == 64 ? launch_tu_rows<__nv_bfloat16, 64>(a, km, vm, s)
                         : launch_tu_rows<__nv_bfloat16, 128>(a, km, vm, s);
  else
    e = a.head_dim == 64 ? launch_tu_rows<__half, 64>(a, km, vm, s) : launch_tu_rows<__half, 128>(a, km, vm, s);
  ++*launches;
  return e;
}

template <typename T, int D>
static cudaError_t launch_join(const TreeArgs& a, int unit_rows, cudaStream_t s) {
  const int64_t rows = std::min((int64_t)a.max_nodes * a.group, (int64_t)unit_rows);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((rows + kTjWarps - 1) / kTjWarps), (unsigned)a.ctas);
  cfg.blockDim = dim3(kTjWarps * 32);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, tree_join_kernel<T, D>, a, unit_rows);
}

template <typename T>
static cudaError_t launch_join_t(const TreeArgs& a, int unit_rows, cudaStream_t s) {
  return a.head_dim == 64 ? launch_join<T, 64>(a, unit_rows, s) : launch_join<T, 128>(a, unit_rows, s);
}

cudaError_t launch_tree_join(const TreeArgs& a, pa_dtype dt, int unit_rows, cudaStream_t s, int* launches) {
  ++*launches;
  switch (dt) {
    case PA_BF16: return launch_join_t<__nv_bfloat16>(a, unit_rows, s);
    case PA_FP16: return launch_join_t<__half>(a, unit_rows, s);
    case PA_FP32: return launch_join_t<float>(a, unit_rows, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace pa
