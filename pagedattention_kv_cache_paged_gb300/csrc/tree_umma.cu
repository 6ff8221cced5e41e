// tcgen05 tree attention (bf16/fp16 pools, block_size % 16 == 0).
//
// Persistent: one CTA per SM walks its equal share of the units (tree_common.cuh).  Per 64-key tile:
// S = Q K^T into a TMEM buffer, the softmax threads (one TMEM lane each) turn it into P in place, O +=
// P V in TMEM; one pass with a running stabiliser that moves only when the maximum grows by more than
// 2^8 (numerator and denominator use the same one, so the result is the softmax's in real arithmetic).
// K and V pass through a ring each that runs on into the next unit while the last one is finished, so that
// the loads never pause at a border.
//
// One thread is too slow to keep an SM's share of HBM3e moving (a wait, an issue and a commit cost it a
// few hundred cycles, a 64-key tile passes every 1,400), so the control work is spread over five warps: K
// and V producers, S products, P V products, Q; and each tile has one commit per product, whose barrier
// tells the softmax, the producer and the other issuer alike.
//
// Two groups of four softmax warps, each with two S buffers and an O of its own (512 TMEM columns):
//   narrow (a sequence's rows fit one 128-row tile): the groups take the key tiles of the unit in
//     turn, which halves the serial work per tile; their states are joined at the unit's end (both
//     Os lie in the same TMEM lanes, so only (maximum, sum) goes through shared memory, and each
//     group writes half of the columns);
//   wide: the unit has two 128-row tiles, one per group, that share every K and V tile.
//
// Masks.  Only tiles that reach into the drafted region look at masks: a row's 64 visibility bits are
// cut out of its mask words.  A masked score becomes -inf by selection, whatever it was.  A masked
// value cannot be deselected (0 * NaN), so in those tiles non-finite elements of V are zeroed in
// shared memory before the product, and added at the end, by themselves, to the rows that see them.
//
// Warps: 0-3 and 4-7 softmax, 8 K and 9 V producer (TMA), 10 S, 11 P V, 12 Q.  Every wait is bounded
// (PA_DEVERR_TIMEOUT).  A wait tells a barrier's phase from the next one only, so each barrier below is
// waited for before its next phase but one can complete.
#include <cudaTypedefs.h>
#include <float.h>

#include "pa_ptx.cuh"
#include "tree_common.cuh"

namespace pa {

constexpr int kTuThreads = 416;
constexpr int kTuSubs = kTreeKeys / 16;
constexpr float kTuRescale = 8.f;

template <int D, bool kWide>
struct TuCfg {
  static constexpr int kHalves = D / 64;
  static constexpr int kQHalf = 128 * 128;          // one 64-column half of a 128-row Q tile
  static constexpr int kQTile = kQHalf * kHalves;
  static constexpr int kQBytes = (kWide ? 2 : 1) * kQTile;
  static constexpr int kKvBytes = kTreeKeys * D * 2;  // a stage: one K or V tile
  static constexpr int kGroup = 1024 * kHalves;     // 8 keys of it
  static constexpr int kHead = 4096;                // barriers, masks, row statistics
  static constexpr int kFit = (227 * 1024 - 1024 - kHead - kQBytes) / kKvBytes;
  static constexpr int kKStages = kFit / 2 < 12 ? kFit / 2 : 12;
  static constexpr int kVStages = kFit - kFit / 2 < 12 ? kFit - kFit / 2 : 12;
  static constexpr int kSmemBytes = 1024 + kHead + kQBytes + (kKStages + kVStages) * kKvBytes;
  static constexpr int kBufs = kWide ? 2 : 4;       // S buffers: tiles whose scores or weights are in TMEM
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


// The span of this CTA (all threads; sm: one word per warp twice, carry and result).
struct TuSched {
  int64_t sums[kTuThreads / 32];
  int64_t tops[kTuThreads / 32];
  int64_t carry;
  TreeSpan span;
  int64_t share;
  int64_t cut_start;  // where the unit that the span ends in begins on the line
  int snap;
  int refused;  // a sequence of the batch is refused, and its rows are this CTA's to zero
};

__device__ __forceinline__ void tu_schedule(const TreeArgs& a, int nodes_unit, TuSched& sm) {
  constexpr int kWarps = kTuThreads / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int gap = a.share > 0 ? 0 : kTreeGap;
  if (threadIdx.x == 0) {
    sm.span = TreeSpan{a.batch, 0, 0, a.batch, 0, 0};
    sm.carry = 0;
    sm.refused = 0;
  }
  int tiles = 0, units = 0;
  auto look = [&](int b) -> int64_t {  // this thread's sequence: its length on the line
    tiles = units = 0;
    if (b >= a.batch) return 0;
    const TreeSeq s = tree_seq(a, b);
    if (s.bad) {
      if (blockIdx.x == 0) raise_error(a.err, s.bad);
      if (s.m > 0 && b % gridDim.x == blockIdx.x) sm.refused = 1;
    }
    if (s.n == 0 || s.m == 0) return 0;
    tiles = tree_tiles(s.n);
    units = (s.m + nodes_unit - 1) / nodes_unit * a.n_kv_heads;
    return (int64_t)units * (tiles + gap);
  };
  __syncthreads();
  // the whole line and its longest unit
  int64_t mine = 0, total = 0, longest = 0;
  for (int b = threadIdx.x; b < a.batch; b += kTuThreads) {
    const int64_t c = look(b);
    total += c;
    longest = max(longest, (int64_t)(c > 0 ? tiles + gap : 0));
    mine = c;
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    total += __shfl_xor_sync(0xffffffffu, total, off);
    longest = max(longest, __shfl_xor_sync(0xffffffffu, longest, off));
  }
  if (lane == 0) {
    sm.sums[warp] = total;
    sm.tops[warp] = longest;
  }
  __syncthreads();
  total = longest = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    total += sm.sums[w];
    longest = max(longest, sm.tops[w]);
  }
  int64_t share = a.share;
  if (share <= 0) {
    // fewer CTAs than that would wait longer for their first keys than they save
    share = (total + gridDim.x - 1) / gridDim.x;
    share = max(share, min(longest, (int64_t)kTreeMinShare));
  }
  // contexts that are never cut: every border moves to the nearest unit's
  const int snap = !a.split || longest <= (a.share > 0 ? 0 : kTreeMinShare) ? INT32_MAX : (a.share > 0 ? 1 : kTreeSnap);
  const int64_t lo = (int64_t)blockIdx.x * share, hi = lo + share;
  if (threadIdx.x == 0) {
    sm.share = share;
    sm.snap = snap;
  }
  const bool one_chunk = a.batch <= kTuThreads;
  __syncthreads();
  for (int b0 = 0; b0 < a.batch; b0 += kTuThreads) {
    const int b = b0 + threadIdx.x;
    const int64_t c = one_chunk ? mine : look(b);
    int64_t v = c;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int64_t t = __shfl_up_sync(0xffffffffu, v, off);
      if (lane >= off) v += t;
    }
    if (lane == 31) sm.sums[warp] = v;
    __syncthreads();
    int64_t pre = sm.carry, chunk = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) pre += sm.sums[w];
      chunk += sm.sums[w];
    }
    pre += v - c;
    const int64_t len = tiles + gap;
    if (c > 0 && lo >= pre && lo < pre + c) {
      const int64_t off = lo - pre;
      sm.span.b0 = b;
      sm.span.u0 = (int)(off / len);
      sm.span.x0 = tree_cut(off % len, tiles, snap);
    }
    if (c > 0 && hi >= pre && hi < pre + c) {
      const int64_t off = hi - pre;
      sm.span.b1 = b;
      sm.span.u1 = (int)(off / len);
      sm.span.x1 = tree_cut(off % len, tiles, snap);
      sm.cut_start = hi - off % len;
    }
    __syncthreads();
    if (threadIdx.x == 0) sm.carry += chunk;
    __syncthreads();
  }
}

template <typename T, int D, bool kWide>
__global__ void __launch_bounds__(kTuThreads, 1)
    tree_umma_kernel(const TreeArgs a, const __grid_constant__ CUtensorMap kmap,
                     const __grid_constant__ CUtensorMap vmap, const __grid_constant__ CUtensorMap qmap) {
  using Cfg = TuCfg<D, kWide>;
  constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
  constexpr int kHalves = Cfg::kHalves;
  constexpr int kKStages = Cfg::kKStages, kVStages = Cfg::kVStages, kBufs = Cfg::kBufs;
  constexpr int kUnitRows = kWide ? 256 : 128;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  // Tile i of the CTA (counted over its units): K stage i % kKStages, V stage i % kVStages, S buffer i % kBufs.
  uint64_t* bars = reinterpret_cast<uint64_t*>(base);
  uint64_t* kfull = bars;          // [kKStages] the tile's keys landed
  uint64_t* vfull = bars + 12;     // [kVStages] its values
  uint64_t* sdone = bars + 24;     // [kKStages] its scores are in its S buffer (and the K stage is free)
  uint64_t* vdone = bars + 36;     // [kVStages] O += P V done (and the V stage and the S buffer are free)
  uint64_t* p_full = bars + 48;    // [kBufs] its weights are written (and O rescaled)
  uint64_t* q_full = bars + 52;    // one phase per unit
  uint64_t* o_free = bars + 53;    // one phase per unit: both Os read
  uint64_t* ml_full = bars + 54;   // one phase per unit (narrow): both groups' statistics written
  uint64_t* q_empty = bars + 55;   // one phase per unit: its S products are done (sdone would not do: the Q
                                   // producer may be more than one phase ahead of it)
  uint64_t* fin = bars + 56;       // [2] all products of an issuer are over
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(base + 480);
  volatile int* bad_v = reinterpret_cast<int*>(base + 484);  // V of a drafted region held non-finite elements
  volatile uint32_t* kmask = reinterpret_cast<uint32_t*>(base + 512);  // [32] 16-key sub-tiles loaded, per tile
  TuSched* sched = reinterpret_cast<TuSched*>(base + 640);
  float2* ml = reinterpret_cast<float2*>(base + 2048);  // [2][128] the groups' (maximum, sum) per row
  static_assert(sizeof(TuSched) <= 2048 - 640 && kKStages <= 12 && kVStages <= 12, "head of the shared memory");
  // (S of tile i + kBufs waits for P V of tile i, and phases stay one apart only if the rings are not shorter)
  static_assert(kKStages >= kBufs && kVStages >= kBufs, "ring depths");
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
    for (int k = 0; k < kBufs; ++k) mbar_init(&p_full[k], kWide ? 8 : 4);
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    mbar_init(o_free, 8);
    mbar_init(ml_full, 8);
    mbar_init(&fin[0], 1);
    mbar_init(&fin[1], 1);
    *bad_v = 0;
    fence_barrier_init();
  }
  if (warp == 10) tmem_alloc(tmem_slot, 512);
  // nothing of global memory is read or written before the preceding grid is over
  pdl_wait_primary();
  pdl_launch_dependents();
  const int nodes_unit = kUnitRows >> a.group_shift;
  tu_schedule(a, nodes_unit, *sched);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const TreeSpan span = sched->span;
  // S of group g in buffer i, and its O.  Narrow: tile i is group i % 2's and its four buffers are the four
  // 64-column ranges; wide: a buffer holds both groups' scores.
  auto tS = [&](int i, int g) { return tmem + 64u * (uint32_t)(kWide ? 2 * i + g : i); };
  auto tO = [&](int g) { return tmem + 256u + 128u * (uint32_t)g; };

  if (warp == 8 || warp == 9) {
    // ------------------------------- producers: warp 8 K, warp 9 V --------------------------------
    // One box is 8 x (up to 8) keys x head_dim of one block: a tile takes 64 / min(block_size, 64) of them,
    // one per lane, and lies in shared memory as [8-key group][64-column half][8][128 bytes, swizzled].
    const bool is_v = warp == 9;
    uint64_t* full = is_v ? vfull : kfull;
    uint64_t* freed = is_v ? vdone : sdone;
    uint8_t* ring = is_v ? vs : ks;
    const CUtensorMap* map = is_v ? &vmap : &kmap;
    const int depth = is_v ? kVStages : kKStages;
    const int box_keys = min(a.block_size, kTreeKeys), boxes = kTreeKeys / box_keys;
    const uint64_t once = l2_policy_evict_first();
    int t = 0, s = 0, round = 0;
    bool alive = true;
    TreeWalk walk(a, span, nodes_unit);
    TreeUnit w;
    while (alive && walk.next(w)) {
      const int32_t* table = a.block_table + (int64_t)w.b * a.bt_stride;
      // table entry of this lane's box of tile x of the unit (-1: behind the context)
      auto entry = [&](int x) -> int {
        const int pos = x * kTreeKeys + lane * box_keys;
        return lane < boxes && x < w.x1 && pos < w.sq.n ? ld_nc_s32(table + (pos >> a.block_shift)) : -1;
      };
      int blk = entry(w.x0);
      for (int x = w.x0; x < w.x1; ++x, ++t) {
        const int blk_next = entry(x + 1);
        if (round > 0 && !__all_sync(0xffffffffu, mbar_wait(&freed[s], (unsigned)((round - 1) & 1), a.err, a.epoch))) {
          alive = false;
          break;
        }
        const int pos = x * kTreeKeys + lane * box_keys;
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
  } else if (warp == 12) {
    // --------------------------------------- Q producer ------------------------------------------
    if (lane == 0) {
      int un = 0;
      bool alive = true;
      TreeWalk walk(a, span, nodes_unit);
      TreeUnit w;
      for (; walk.next(w); ++un) {
        if (un > 0 && !mbar_wait(q_empty, (unsigned)((un - 1) & 1), a.err, a.epoch)) {
          alive = false;
          break;
        }
        const int tiles = kWide && w.rows > 128 ? 2 : 1;
        mbar_arrive_expect_tx(q_full, tiles * Cfg::kQTile);
        for (int k = 0; k < tiles; ++k)
#pragma unroll
          for (int h = 0; h < kHalves; ++h)
            tma_load_3d(qs + k * Cfg::kQTile + h * Cfg::kQHalf, &qmap, h * 64, w.kvh << a.group_shift,
                        (int)(w.sq.q0 + w.node0) + k * (128 >> a.group_shift), q_full);
      }
      if (!alive) raise_timeout(a.err, a.epoch);
      if (un > 0) mbar_wait(q_full, (unsigned)((un - 1) & 1));  // no copy in flight
    }
    __syncwarp();
  } else if (warp == 10) {
    // -------------------------------------- S = Q K^T --------------------------------------------
    if (lane == 0) {
      const uint32_t id = umma_idesc_f16(kBf16, 128, kTreeKeys, false, false);
      const uint64_t qd = umma_desc_sw128(smem_u32(qs), 16, 1024), kd = umma_desc_sw128(smem_u32(ks), 16, Cfg::kGroup);
      int t = 0, s = 0, round = 0, un = 0;
      bool ok = true;
      auto wait = [&](uint64_t* bar, int phase) {
        ok = ok && mbar_wait(bar, (unsigned)(phase & 1), a.err, a.epoch);
        return ok;
      };
      TreeWalk walk(a, span, nodes_unit);
      TreeUnit w;
      while (ok && walk.next(w)) {
        const bool two = kWide && w.rows > 128;
        if (!wait(q_full, un)) break;
        for (int x = w.x0; x < w.x1; ++x, ++t) {
          // the buffer still holds the weights of tile t - kBufs until their product is done
          if (t >= kBufs && !wait(&vdone[(t - kBufs) % kVStages], (t - kBufs) / kVStages)) break;
          if (!wait(&kfull[s], round)) break;
          tc_fence_after();
          const uint64_t kt = kd + (uint64_t)(s * (Cfg::kKvBytes >> 4));
          const int buf = t % kBufs;
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            umma_ss(tS(buf, 0), qd + (kk >> 2) * (Cfg::kQHalf >> 4) + (kk & 3) * 2, kt + (kk >> 2) * 64 + (kk & 3) * 2, id,
                    kk > 0 ? 1u : 0u);
          if (two) {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              umma_ss(tS(buf, 1), qd + (Cfg::kQTile >> 4) + (kk >> 2) * (Cfg::kQHalf >> 4) + (kk & 3) * 2,
                      kt + (kk >> 2) * 64 + (kk & 3) * 2, id, kk > 0 ? 1u : 0u);
          }
          umma_commit(&sdone[s]);
          if (x == w.x1 - 1) umma_commit(q_empty);
          if (++s == kKStages) {
            s = 0;
            ++round;
          }
        }
        ++un;
      }
      if (!ok) raise_timeout(a.err, a.epoch);
      umma_commit(&fin[0]);  // no product in flight when the tensor memory is given back
      mbar_wait(&fin[0], 0);
    }
    __syncwarp();
  } else if (warp == 11) {
    // -------------------------------------- O += P V ---------------------------------------------
    if (lane == 0) {
      const uint32_t id = umma_idesc_f16(kBf16, 128, D, false, true);
      const uint64_t vd = umma_desc_sw128(smem_u32(vs), 1024, Cfg::kGroup);
      int t = 0, s = 0, round = 0, un = 0;
      bool ok = true;
      auto wait = [&](uint64_t* bar, int phase) {
        ok = ok && mbar_wait(bar, (unsigned)(phase & 1), a.err, a.epoch);
        return ok;
      };
      TreeWalk walk(a, span, nodes_unit);
      TreeUnit w;
      while (ok && walk.next(w)) {
        const bool two = kWide && w.rows > 128;
        // the unit's first products overwrite the Os that the unit before it left
        if (un > 0 && !wait(o_free, un - 1)) break;
        for (int x = w.x0; x < w.x1; ++x, ++t) {
          const int buf = t % kBufs;
          if (!wait(&vfull[s], round) || !wait(&p_full[buf], t / kBufs)) break;
          tc_fence_after();
          const uint64_t vt = vd + (uint64_t)(s * (Cfg::kKvBytes >> 4));
          const int g = kWide ? 0 : t & 1;
          const uint32_t more = x >= w.x0 + (kWide ? 1 : 2) ? 1u : 0u;
#pragma unroll
          for (int kk = 0; kk < kTreeKeys / 16; ++kk)
            umma_ts(tO(g), tS(buf, g) + 8u * (uint32_t)kk, vt + kk * (2 * Cfg::kGroup >> 4), id, kk > 0 ? 1u : more);
          if (two) {
#pragma unroll
            for (int kk = 0; kk < kTreeKeys / 16; ++kk)
              umma_ts(tO(1), tS(buf, 1) + 8u * (uint32_t)kk, vt + kk * (2 * Cfg::kGroup >> 4), id, kk > 0 ? 1u : more);
          }
          umma_commit(&vdone[s]);
          if (++s == kVStages) {
            s = 0;
            ++round;
          }
        }
        ++un;
      }
      if (!ok) raise_timeout(a.err, a.epoch);
      umma_commit(&fin[1]);  // no product in flight when the tensor memory is given back
      mbar_wait(&fin[1], 0);
    }
    __syncwarp();
  } else {
    // ---------------------------------------- softmax --------------------------------------------
    const int grp = warp >> 2;
    const int r = threadIdx.x & 127;  // row of the group's tile = TMEM lane
    const uint32_t lane_base = (uint32_t)(32 * (warp & 3)) << 16;
    int t = 0, un = 0;  // tiles of the CTA's earlier units, and those
    bool alive = true, cut = false;
    TreeWalk walk(a, span, nodes_unit);
    TreeUnit w;
    while (alive && walk.next(w)) {
      const int n = w.x1 - w.x0;
      const int hist = w.sq.n - w.sq.m;
      const int rows = kWide ? min(128, w.rows - 128 * grp) : w.rows;  // of this group's tile
      const bool live = (r & ~31) < rows;                               // whole warps
      const int node = w.node0 + (kWide ? grp * (128 >> a.group_shift) : 0) + (max(min(r, rows - 1), 0) >> a.group_shift);
      const int64_t* words = a.tree_mask != nullptr ? a.tree_mask + (w.sq.q0 + node) * a.mask_words : nullptr;
      float m_use = -INFINITY, l_run = 0.f;

      // Bits of the tile at key kb that this row sees (bit c: key kb + c), sub-tiles that are not
      // loaded and keys behind the context left out.
      auto visible = [&](int kb, uint32_t loaded) -> uint64_t {
        const int s0 = kb - hist;  // node of the tile's first key
        uint64_t keep;
        if (s0 + kTreeKeys <= 0) {
          keep = ~0ull;
        } else if (words == nullptr) {
          const int nv = node + 1 - s0;  // chain: nodes up to its own
          keep = nv <= 0 ? 0ull : (nv >= 64 ? ~0ull : (1ull << nv) - 1ull);
        } else if (s0 < 0) {
          keep = ((uint64_t)__ldg(words) << -s0) | ((1ull << -s0) - 1ull);
        } else {
          const int i = s0 >> 6, sh = s0 & 63;
          keep = (i < a.mask_words ? (uint64_t)__ldg(words + i) : 0ull) >> sh;
          if (sh != 0 && i + 1 < a.mask_words) keep |= (uint64_t)__ldg(words + i + 1) << (64 - sh);
        }
        const int nv = w.sq.n - kb;
        if (nv < 64) keep &= (1ull << nv) - 1ull;
#pragma unroll
        for (int u = 0; u < kTuSubs; ++u)
          if (!((loaded >> u) & 1u)) keep &= ~(0xffffull << (16 * u));
        return keep;
      };

      // Scores of S buffer buf into weights; `before` >= 0: the group's previous tile of the unit.
      // kMasked: the tile may hold keys that the row does not see.
      auto tile = [&](auto masked, int buf, uint64_t keep, int before) {
        constexpr bool kMasked = decltype(masked)::value;
        const uint32_t srow = tS(buf, grp) + lane_base;
        uint32_t sv[64];
        tmem_ld32(srow, *reinterpret_cast<uint32_t(*)[32]>(&sv[0]));
        tmem_ld32(srow + 32u, *reinterpret_cast<uint32_t(*)[32]>(&sv[32]));
        tmem_wait_ld();
        tmem_pin32(*reinterpret_cast<uint32_t(*)[32]>(&sv[0]));
        tmem_pin32(*reinterpret_cast<uint32_t(*)[32]>(&sv[32]));
        if (kMasked) {
#pragma unroll
          for (int c = 0; c < 64; ++c)
            if (!((keep >> c) & 1ull)) sv[c] = 0xff800000u;
        }
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int c = 0; c < 64; c += 8)
#pragma unroll
          for (int u = 0; u < 4; ++u)
            mx[u] = fmax3(mx[u], __uint_as_float(sv[c + 2 * u]), __uint_as_float(sv[c + 2 * u + 1]));
        float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * a.scale_log2;
        if (!kMasked || keep != 0) top = fmaxf(top, -FLT_MAX);  // keys were seen, whatever their scores
        float corr = 1.f;
        if (top > m_use + kTuRescale || (m_use == -INFINITY && top != -INFINITY)) {
          corr = fast_exp2(m_use - top);  // m_use = -inf: 0
          m_use = top;
        }
        const float m_sub = m_use == -INFINITY ? 0.f : m_use;
        const uint64_t sc2 = f2_pack(a.scale_log2, a.scale_log2), nm2 = f2_pack(-m_sub, -m_sub);
        uint64_t sum2[2] = {f2_pack(0.f, 0.f), f2_pack(0.f, 0.f)};
        uint32_t p[32];
#pragma unroll
        for (int c = 0; c < 32; ++c) {
          float x0, x1;
          f2_unpack(f2_fma(f2_pack(__uint_as_float(sv[2 * c]), __uint_as_float(sv[2 * c + 1])), sc2, nm2), x0, x1);
          const float e0 = fast_exp2(x0), e1 = fast_exp2(x1);
          sum2[c & 1] = f2_add(sum2[c & 1], f2_pack(e0, e1));
          // weights are rounded to the pool's type for the product with V (half a step each); their sum
          // keeps 32 bits
          p[c] = pack2<kBf16>(e0, e1);
        }
        tmem_st32(srow, p);
        float a0, a1, b0, b1;
        f2_unpack(sum2[0], a0, a1);
        f2_unpack(sum2[1], b0, b1);
        l_run = l_run * corr + ((a0 + a1) + (b0 + b1));
        if (before >= 0 && __any_sync(0xffffffffu, corr != 1.f)) {
          // O is stable once the product of the group's previous tile is done; this tile's waits for us
          if (!__all_sync(0xffffffffu, mbar_wait(&vdone[before % kVStages], (unsigned)((before / kVStages) & 1),
                                                           a.err, a.epoch))) {
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

      const int step = kWide ? 1 : 2;
      for (int i = kWide ? 0 : ((grp - t) & 1); i < n; i += step) {
        const int ti = t + i, buf = ti % kBufs, before = i < step ? -1 : ti - step;
        const int kb = (w.x0 + i) * kTreeKeys;
        const bool edge = kb + kTreeKeys > hist;
        if (!__all_sync(0xffffffffu, mbar_wait(&sdone[ti % kKStages], (unsigned)((ti / kKStages) & 1), a.err, a.epoch))) {
          alive = false;
          break;
        }
        tc_fence_after();
        const uint32_t loaded = kmask[ti & 31];
        if (!edge && loaded == (1u << kTuSubs) - 1u) {
          if (live) tile(std::false_type{}, buf, ~0ull, before);
        } else {
          if (live) tile(std::true_type{}, buf, visible(kb, loaded), before);
          if (!kWide || grp == 0) {
            // V of the tile: rows without a token zeroed, non-finite elements of drafted tokens taken out
            if (!__all_sync(0xffffffffu, mbar_wait(&vfull[ti % kVStages], (unsigned)((ti / kVStages) & 1), a.err,
                                                   a.epoch))) {
              alive = false;
              break;
            }
            uint8_t* vst = vs + (ti % kVStages) * Cfg::kKvBytes;
            for (int e = r; e < kTreeKeys * 8 * kHalves; e += 128) {
              const int key = e / (8 * kHalves), c = e % (8 * kHalves);
              uint4* p = reinterpret_cast<uint4*>(vst + (key >> 3) * Cfg::kGroup + (c >> 3) * 1024 + (key & 7) * 128 +
                                                   (((c & 7) ^ (key & 7)) << 4));
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
      // both Os: products complete in the order in which their one thread issued them
      const int end = t + n - 1;
      if (alive)
        alive = __all_sync(0xffffffffu, mbar_wait(&vdone[end % kVStages], (unsigned)((end / kVStages) & 1), a.err, a.epoch));
      if (!alive) break;
      tc_fence_after();

      // ---- the unit's rows: the output, or this CTA's piece of it ----------------------------------
      const bool whole = w.x0 == 0 && w.x1 == w.T;
      const int64_t row0 = (w.sq.q0 + w.node0) * a.n_q_heads + ((int64_t)w.kvh << a.group_shift);
      const int ur = kWide ? 128 * grp + r : r;  // row of the unit
      const int64_t qh = row0 + (int64_t)(ur >> a.group_shift) * a.n_q_heads + (ur & (a.group - 1));
      const int64_t piece = ((int64_t)blockIdx.x * 2 + (w.x0 == 0 ? 1 : 0)) * kUnitRows + ur;
      float M = m_use, L = l_run, f0 = 1.f, f1 = 0.f;
      bool has0 = true, has1 = false;
      if (!kWide) {
        ml[128 * grp + r] = make_float2(m_use, l_run);
        __syncwarp();
        if (lane == 0) mbar_arrive(ml_full);
        if (!__all_sync(0xffffffffu, mbar_wait(ml_full, (unsigned)(un & 1), a.err, a.epoch))) {
          alive = false;
          break;
        }
        has0 = n > 1 || (t & 1) == 0;
        has1 = n > 1 || (t & 1) == 1;
        const float2 s0 = ml[r], s1 = ml[128 + r];
        M = fmaxf(s0.x, s1.x);
        const float M0 = M == -INFINITY ? 0.f : M;
        f0 = fast_exp2(s0.x - M0);
        f1 = fast_exp2(s1.x - M0);
        L = fmaf(s0.y, f0, s1.y * f1);
      }
      const bool none = M == -INFINITY;  // the row sees none of these keys
      const float norm = whole ? (none ? 0.f : 1.f / L) : 1.f;
      constexpr int kCols = kWide ? D : D / 2;
      const int col0 = kWide ? 0 : grp * kCols;
      if (live) {
#pragma unroll 1
        for (int c0 = col0; c0 < col0 + kCols; c0 += 32) {
          float acc[32];
          uint32_t v[32];
          if (kWide) {
            tmem_ld32_sync(tO(grp) + lane_base + c0, v);
#pragma unroll
            for (int i = 0; i < 32; ++i) acc[i] = __uint_as_float(v[i]);
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) acc[i] = 0.f;
            if (has0) {
              tmem_ld32_sync(tO(0) + lane_base + c0, v);
#pragma unroll
              for (int i = 0; i < 32; ++i) acc[i] = __uint_as_float(v[i]) * f0;
            }
            if (has1) {
              tmem_ld32_sync(tO(1) + lane_base + c0, v);
#pragma unroll
              for (int i = 0; i < 32; ++i) acc[i] = fmaf(__uint_as_float(v[i]), f1, acc[i]);
            }
          }
          if (r < rows) {
            if (*bad_v != 0) {
              // the non-finite elements that were taken out of V, for the rows that see them
              const int32_t* table = a.block_table + (int64_t)w.b * a.bt_stride;
              const int end = min(w.x1 * kTreeKeys, w.sq.n);
              for (int pos = max(w.x0 * kTreeKeys, hist); pos < end; ++pos) {
                const int s = pos - hist;
                const bool see = words != nullptr ? ((__ldg(words + (s >> 6)) >> (s & 63)) & 1) != 0 : s <= node;
                const int blk = __ldg(table + (pos >> a.block_shift));
                if (!see || blk < 0 || blk >= a.num_blocks) continue;
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
              for (int i = 0; i < 32; i += 8) {
                float f[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) f[e] = none ? 0.f : acc[i + e] * norm;
                uint4 x;
                x.x = pack2<kBf16>(f[0], f[1]);
                x.y = pack2<kBf16>(f[2], f[3]);
                x.z = pack2<kBf16>(f[4], f[5]);
                x.w = pack2<kBf16>(f[6], f[7]);
                *reinterpret_cast<uint4*>(o + i) = x;
              }
            } else {
              float* o = a.ws_acc + piece * D + c0;
#pragma unroll
              for (int i = 0; i < 32; i += 4)
                *reinterpret_cast<float4*>(o + i) = none ? make_float4(0.f, 0.f, 0.f, 0.f)
                                                         : make_float4(acc[i], acc[i + 1], acc[i + 2], acc[i + 3]);
            }
          }
        }
        if (!whole && r < rows && (kWide || grp == 0)) {
          a.ws_m[piece] = M;
          a.ws_l[piece] = none ? 0.f : L;
        }
      }
      // O has been read: the next unit's first products may overwrite it
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(o_free);
      if (!whole && w.x0 == 0) {
        cut = true;  // at most one unit of a CTA: the one that its span ends in
        if (threadIdx.x == 0) {
          // the CTA that the unit's last tile went to
          const int64_t at = sched->cut_start, share = sched->share;
          int64_t last = (at + w.T - 1) / share;
          if (tree_cut(last * share - at, w.T, sched->snap) == w.T) --last;
          a.ws_rec[blockIdx.x] = TreeRec{row0, w.rows, (int32_t)last};
        }
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
  if (sched->refused) {
    // sequences whose lengths do not fit together: zeros
    for (int b = blockIdx.x; b < a.batch; b += gridDim.x) {
      const TreeSeq s = tree_seq(a, b);
      if (s.n != 0 || s.bad == 0) continue;
      uint4* o = reinterpret_cast<uint4*>(static_cast<T*>(a.out) + s.q0 * a.n_q_heads * D);
      for (int64_t i = threadIdx.x; i < (int64_t)s.m * a.n_q_heads * (D / 8); i += kTuThreads) o[i] = make_uint4(0, 0, 0, 0);
    }
  }
}

// ------------------------------------------------------------------------------------------------
// Units cut between CTAs: CTA c's second piece (its first tiles), then the first pieces of the CTAs
// up to `last`, joined like any partitions.  One warp per row.
constexpr int kTjWarps = 8;

template <typename T, int D>
__global__ void __launch_bounds__(kTjWarps * 32) tree_join_kernel(const TreeArgs a, int unit_rows) {
  constexpr int kPer = D / 32;
  const int lane = threadIdx.x & 31;
  const int c = blockIdx.y;
  pdl_launch_dependents();
  pdl_wait_primary();
  const TreeRec rec = a.ws_rec[c];
  const int r = blockIdx.x * kTjWarps + (threadIdx.x >> 5);
  if (r >= rec.rows) return;
  const int pieces = rec.last - c + 1;
  auto piece = [&](int i) -> int64_t { return ((int64_t)(c + i) * 2 + (i == 0 ? 1 : 0)) * unit_rows + r; };
  float M = -INFINITY;
  for (int i = lane; i < pieces; i += 32) M = fmaxf(M, a.ws_m[piece(i)]);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
  float L = 0.f, acc[kPer];
#pragma unroll
  for (int k = 0; k < kPer; ++k) acc[k] = 0.f;
  if (M != -INFINITY) {
#pragma unroll 4
    for (int i = 0; i < pieces; ++i) {
      const int64_t p = piece(i);
      const float f = fast_exp2(a.ws_m[p] - M);
      L = fmaf(a.ws_l[p], f, L);
      const float* src = a.ws_acc + p * D + lane * kPer;
#pragma unroll
      for (int k = 0; k < kPer; ++k) acc[k] = fmaf(src[k], f, acc[k]);
    }
  }
  const int64_t qh = rec.row0 + (int64_t)(r >> a.group_shift) * a.n_q_heads + (r & (a.group - 1));
  T* o = static_cast<T*>(a.out) + qh * D + lane * kPer;
#pragma unroll
  for (int k = 0; k < kPer; ++k) o[k] = Elt<T>::from_float(M == -INFINITY ? 0.f : acc[k] / L);
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
static cudaError_t launch_join(const TreeArgs& a, cudaStream_t s) {
  const int unit_rows = tree_unit_rows(a.max_nodes, a.group);
  const int64_t rows = min((int64_t)a.max_nodes * a.group, (int64_t)unit_rows);
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

cudaError_t launch_tree_join(const TreeArgs& a, pa_dtype dt, cudaStream_t s, int* launches) {
  ++*launches;
  if (dt == PA_BF16) return a.head_dim == 64 ? launch_join<__nv_bfloat16, 64>(a, s) : launch_join<__nv_bfloat16, 128>(a, s);
  return a.head_dim == 64 ? launch_join<__half, 64>(a, s) : launch_join<__half, 128>(a, s);
}

}  // namespace pa
