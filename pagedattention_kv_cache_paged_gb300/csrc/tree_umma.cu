// tcgen05 tree attention (bf16/fp16 pools, block_size % 16 == 0).
//
// One CTA = one tile of a sequence's (node, query head) rows of one KV head x one partition of the
// keys; two CTAs per SM.  Per 64-key tile j: S(j) = Q K(j)^T into one of two TMEM buffers, the softmax
// threads (one TMEM lane each) turn it into P(j) in place, O += P(j) V(j) in TMEM; one pass with a
// running stabiliser that moves only when the maximum grows by more than 2^8 (numerator and
// denominator use the same one, so the result is the softmax's in real arithmetic).  Issue order
// S(j+1), P(j) V(j): the tensor core works while the softmax does.
//
// Rows.  The MMA has 128 rows whether or not a tree fills them, and reading K and V once is what
// bounds the kernel, so idle rows cost nothing.  They are used all the same: with at most 64 (32) rows
// the Q tile is loaded kSplit = 2 (4) times, copy s in lanes s * 128 / kSplit on, and the threads of
// copy s take keys [s * 64 / kSplit, ...) of every tile (their P is zero elsewhere), so that the
// serial work per tile shrinks with the rows; the copies' states are joined at the end like partitions.
//
// Masks.  Only tiles that reach into the drafted region or past the partition's end look at masks: a
// row's 64 visibility bits are cut out of its mask words.  A masked score becomes -inf by selection,
// whatever it was.  A masked value cannot be deselected (0 * NaN), so in those tiles non-finite
// elements of V are zeroed in shared memory before the product, and added at the end, by themselves,
// to the rows that see them.
//
// Warps: 0-3 softmax, 4 producer (TMA: one box of 16 keys x 64 columns per lane), 5 MMA.  Every wait is
// bounded (PA_DEVERR_TIMEOUT).
#include <cudaTypedefs.h>
#include <float.h>

#include "pa_ptx.cuh"
#include "tree_common.cuh"

namespace pa {

constexpr int kTuThreads = 192;
constexpr int kTuKeys = 64;
constexpr int kTuSubs = kTuKeys / 16;
constexpr int kTuTmemCols = 256;  // S: 2 x 64, O: D
constexpr float kTuRescale = 8.f;

template <int D>
struct TuCfg {
  static constexpr int kHalves = D / 64;
  static constexpr int kStages = D == 128 ? 2 : 4;
  static constexpr int kQHalf = 128 * 128;
  static constexpr int kQBytes = 128 * D * 2;
  static constexpr int kKvHalf = kTuKeys * 128;
  static constexpr int kKvBytes = kTuKeys * D * 2;
  static constexpr int kSmemBytes = 1024 + 1024 + kQBytes + 2 * kStages * kKvBytes;
};

__device__ __forceinline__ void named_barrier(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

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

// kCols consecutive scores of this thread's row.
template <int kCols>
__device__ __forceinline__ void load_scores(uint32_t taddr, uint32_t (&sv)[kCols]) {
  if constexpr (kCols == 64) {
    tmem_ld32(taddr, *reinterpret_cast<uint32_t(*)[32]>(&sv[0]));
    tmem_ld32(taddr + 32u, *reinterpret_cast<uint32_t(*)[32]>(&sv[32]));
    tmem_wait_ld();
    tmem_pin32(*reinterpret_cast<uint32_t(*)[32]>(&sv[0]));
    tmem_pin32(*reinterpret_cast<uint32_t(*)[32]>(&sv[32]));
  } else if constexpr (kCols == 32) {
    tmem_ld32_sync(taddr, sv);
  } else {
    tmem_ld16(taddr, sv);
    tmem_wait_ld();
    tmem_pin16(sv);
  }
}

// The kCols weights (as kCols / 2 words) of copy `part`'s keys into the row's 32 P columns, zeros into
// the other copies' columns.
template <int kCols>
__device__ __forceinline__ void store_weights(uint32_t taddr, int part, const uint32_t (&w)[kCols / 2]) {
  if constexpr (kCols == 64) {
    tmem_st32(taddr, w);
  } else {
    uint32_t z[kCols / 2];
#pragma unroll
    for (int i = 0; i < kCols / 2; ++i) z[i] = 0u;
#pragma unroll
    for (int s = 0; s < 64 / kCols; ++s) {  // `part` is uniform over the warp
      if constexpr (kCols == 32) {
        if (s == part) tmem_st16(taddr + 16u * s, w);
        else tmem_st16(taddr + 16u * s, z);
      } else {
        if (s == part) tmem_st8(taddr + 8u * s, w);
        else tmem_st8(taddr + 8u * s, z);
      }
    }
  }
}

// kCols columns of O of this thread's row.
template <int kCols>
__device__ __forceinline__ void load_out(uint32_t taddr, float (&f)[kCols]) {
  uint32_t v[kCols];
  load_scores<kCols>(taddr, v);
#pragma unroll
  for (int i = 0; i < kCols; ++i) f[i] = __uint_as_float(v[i]);
}

template <typename T, int D, int kSplit>
__global__ void __launch_bounds__(kTuThreads, 2)
    tree_umma_kernel(const TreeArgs a, int q_tiles, const __grid_constant__ CUtensorMap kmap,
                     const __grid_constant__ CUtensorMap vmap, const __grid_constant__ CUtensorMap qmap) {
  using Cfg = TuCfg<D>;
  constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
  constexpr int kHalves = Cfg::kHalves;
  constexpr int kStages = Cfg::kStages;
  constexpr int kRows = 128 / kSplit;  // distinct (node, head) rows of a tile
  constexpr int kCols = kTuKeys / kSplit;  // keys of a tile per thread

  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(base);
  uint64_t* kfull = bars;         // [kStages]
  uint64_t* kempty = bars + 4;    // [kStages] S of the stage's tile done
  uint64_t* vfull = bars + 8;     // [kStages]
  uint64_t* vempty = bars + 12;   // [kStages] P V of the stage's tile done
  uint64_t* q_ready = bars + 16;
  uint64_t* s_full = bars + 17;   // [2] S(j) in buffer j % 2
  uint64_t* p_full = bars + 19;   // [2] P(j) written (and O rescaled)
  uint64_t* pv_done = bars + 21;  // [2] O += P(j) V(j) done, in barrier j % 2
  // (a wait tells a phase from the next one only: at the end the last two products may be outstanding or
  // both over, so the last one has a barrier of its own)
  uint64_t* o_full = bars + 23;   // O complete
  uint64_t* fin = bars + 24;      // a launch that gave up: its products are over
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(base + 512);
  int* bad_v = reinterpret_cast<int*>(base + 516);  // V of the drafted region holds non-finite elements
  volatile uint32_t* kmask = reinterpret_cast<uint32_t*>(base + 544);  // [8] sub-tiles loaded, per tile
  uint8_t* qs = base + 1024;
  uint8_t* ks = qs + Cfg::kQBytes;
  uint8_t* vs = ks + kStages * Cfg::kKvBytes;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  // KV heads innermost (they read the same physical blocks), then the tiles that read the same keys
  int rest = blockIdx.x;
  const int kvh = rest % a.n_kv_heads;
  rest /= a.n_kv_heads;
  const int qt = rest % q_tiles;
  rest /= q_tiles;
  const int part = rest % a.max_parts;
  const int b = rest / a.max_parts;

  pdl_wait_primary();
  pdl_launch_dependents();
  const TreeSeq sq = tree_seq(a, b);
  if (sq.bad && threadIdx.x == 0 && qt == 0 && part == 0 && kvh == 0) raise_error(a.err, sq.bad);
  const int nodes_tile = kRows >> a.group_shift;
  const int node0 = qt * nodes_tile;
  const int n_parts = sq.n == 0 ? 1 : (sq.n + a.part_tokens - 1) / a.part_tokens;
  if (node0 >= sq.m || part >= n_parts) return;
  const int rows = min(kRows, (sq.m - node0) << a.group_shift);  // rows of the tile that exist
  const int64_t row0 = (sq.q0 + node0) * a.n_q_heads + (int64_t)kvh * a.group;
  // row r of the tile: query row / head offset in out and the workspace
  auto out_row = [&](int r) -> int64_t {
    return row0 + (int64_t)(r >> a.group_shift) * a.n_q_heads + (r & (a.group - 1));
  };
  if (sq.n == 0) {  // nothing to see
    T* o = static_cast<T*>(a.out);
    for (int i = threadIdx.x; i < rows * (D / 8); i += kTuThreads)
      *reinterpret_cast<uint4*>(o + out_row(i / (D / 8)) * D + (i % (D / 8)) * 8) = make_uint4(0, 0, 0, 0);
    return;
  }
  const int hist = sq.n - sq.m;
  const int t_begin = part * a.part_tokens;
  const int t_end = min(t_begin + a.part_tokens, sq.n);
  const int n_tiles = (t_end - t_begin + kTuKeys - 1) / kTuKeys;
  const int warps_per_copy = 4 / kSplit;
  const int live_warps = min(warps_per_copy, (rows + 31) >> 5) * kSplit;

  if (threadIdx.x == 0) {
    prefetch_tensormap(&kmap);
    prefetch_tensormap(&vmap);
    prefetch_tensormap(&qmap);
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&kfull[s], 1);
      mbar_init(&kempty[s], 1);
      mbar_init(&vfull[s], 1);
      mbar_init(&vempty[s], 1);
    }
    for (int k = 0; k < 2; ++k) {
      mbar_init(&s_full[k], 1);
      mbar_init(&p_full[k], 32 * live_warps);
      mbar_init(&pv_done[k], 1);
    }
    mbar_init(q_ready, 1);
    mbar_init(o_full, 1);
    mbar_init(fin, 1);
    *bad_v = 0;
    fence_barrier_init();
  }
  if (warp == 5) tmem_alloc(tmem_slot, kTuTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  auto tS = [&](int k) { return tmem + 64u * (uint32_t)k; };
  const uint32_t tO = tmem + 128u;

  if (warp == 4) {
    // ---------------------------------------- producer -------------------------------------------
    constexpr int kBoxes = kTuSubs * kHalves;  // boxes of one operand's tile
    const int kind = lane / kBoxes;            // lanes of kind 0 load K boxes, of kind 1 V boxes
    const int sub = (lane % kBoxes) / kHalves;
    const int half = lane % kHalves;
    const int32_t* table = a.block_table + (int64_t)b * a.bt_stride;
    // table entry of this lane's sub-tile of tile j (-1: behind the partition's keys)
    auto entry = [&](int j) -> int {
      const int pos = t_begin + j * kTuKeys + sub * 16;
      return kind < 2 && pos < t_end ? ld_nc_s32(table + (pos >> a.block_shift)) : -1;
    };
    // K and V are read once by a lone tile of rows; several tiles read them from L2
    const uint64_t policy = l2_policy_evict_first();
    bool alive = true;
    auto issue = [&](int v, int j, int blk) {  // whole warp
      const int s = j % kStages;
      uint64_t* full = (v ? vfull : kfull) + s;
      if (j >= kStages &&
          !__all_sync(0xffffffffu, mbar_wait((v ? vempty : kempty) + s, (unsigned)((j / kStages - 1) & 1), a.err,
                                             a.epoch))) {
        alive = false;
        return;
      }
      const int pos = t_begin + j * kTuKeys + sub * 16;
      const bool in = kind == v && pos < t_end;
      const bool ok = in && blk >= 0 && blk < a.num_blocks;
      if (in && !ok && !v && half == 0) raise_error(a.err, PA_DEVERR_BLOCK_ID);
      const unsigned lanes = __ballot_sync(0xffffffffu, ok);
      if (lane == 0) {
        if (!v) {
          uint32_t m = 0;
#pragma unroll
          for (int u = 0; u < kTuSubs; ++u) m |= ((lanes >> (u * kHalves)) & 1u) << u;
          // read by the softmax threads after S(j), which waits for the arrival below; slot j % 8 is
          // free: K(j) waits for S(j - kStages), which came after the weights of tile j - 8
          kmask[j & 7] = m;
        }
        if (lanes != 0) mbar_arrive_expect_tx(full, (unsigned)__popc(lanes) * 2048u);
        else mbar_arrive(full);
      }
      __syncwarp();
      if (ok) {
        uint8_t* dst = (v ? vs : ks) + s * Cfg::kKvBytes + half * Cfg::kKvHalf + sub * 2048;
        const CUtensorMap* map = v ? &vmap : &kmap;
        const int x = kvh * D + half * 64, y = pos & (a.block_size - 1);
        if (q_tiles == 1) tma_load_3d_hint(dst, map, x, y, blk, full, policy);
        else tma_load_3d(dst, map, x, y, blk, full);
      }
    };
    int first[kStages];
#pragma unroll
    for (int j = 0; j < kStages; ++j) first[j] = entry(j);
    int next = entry(kStages);
    if (lane == 0) {
      mbar_arrive_expect_tx(q_ready, Cfg::kQBytes);
#pragma unroll
      for (int c = 0; c < kSplit; ++c)
#pragma unroll
        for (int h = 0; h < kHalves; ++h)
          tma_load_3d(qs + h * Cfg::kQHalf + c * kRows * 128, &qmap, h * 64, kvh << a.group_shift,
                      (int)(sq.q0 + node0), q_ready);
    }
    __syncwarp();
#pragma unroll
    for (int j = 0; j < kStages; ++j)
      if (j < n_tiles) {
        issue(0, j, first[j]);
        issue(1, j, first[j]);
      }
    // K(j) then V(j - 1): the order in which the products free their stages
    for (int j = kStages; j <= n_tiles && alive; ++j) {
      const bool is_k = kind == 0;
      if (j < n_tiles) {
        issue(0, j, next);
        if (is_k) next = entry(j + 1);
      }
      if (alive && j > kStages) {
        issue(1, j - 1, next);
        if (!is_k) next = entry(j);
      }
    }
    if (!alive && lane == 0) raise_timeout(a.err, a.epoch);
    if (!alive && lane == 0) {  // leave no copy in flight
      mbar_wait(q_ready, 0);
      for (int s = 0; s < kStages; ++s) {
        // whichever phase the stage is in, its last copies land within a bounded wait for either parity
        mbar_wait_for(&kfull[s], 0, nullptr, 0, 10000000ull);
        mbar_wait_for(&kfull[s], 1, nullptr, 0, 10000000ull);
        mbar_wait_for(&vfull[s], 0, nullptr, 0, 10000000ull);
        mbar_wait_for(&vfull[s], 1, nullptr, 0, 10000000ull);
      }
    }
  } else if (warp == 5) {
    // ------------------------------------------ MMA ----------------------------------------------
    if (lane == 0) {
      const uint32_t id_s = umma_idesc_f16(kBf16, 128, kTuKeys, false, false);
      const uint32_t id_pv = umma_idesc_f16(kBf16, 128, D, false, true);
      bool ok = mbar_wait(q_ready, 0, a.err, a.epoch);
      auto issue_s = [&](int j) {
        ok = ok && mbar_wait(&kfull[j % kStages], (unsigned)((j / kStages) & 1), a.err, a.epoch);
        if (!ok) return;
        tc_fence_after();
        const uint32_t qa = smem_u32(qs);
        const uint32_t ka = smem_u32(ks + (j % kStages) * Cfg::kKvBytes);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          umma_ss(tS(j & 1), umma_desc_sw128(qa + (kk >> 2) * Cfg::kQHalf + (kk & 3) * 32, 16, 1024),
                  umma_desc_sw128(ka + (kk >> 2) * Cfg::kKvHalf + (kk & 3) * 32, 16, 1024), id_s, kk > 0 ? 1u : 0u);
        umma_commit(&s_full[j & 1]);
        umma_commit(&kempty[j % kStages]);
      };
      issue_s(0);
      for (int j = 0; j < n_tiles && ok; ++j) {
        // S(j + 1) overwrites P(j - 1), whose product was issued before it and reads it first
        if (j + 1 < n_tiles) issue_s(j + 1);
        ok = ok && mbar_wait(&vfull[j % kStages], (unsigned)((j / kStages) & 1), a.err, a.epoch) &&
             mbar_wait(&p_full[j & 1], (unsigned)((j >> 1) & 1), a.err, a.epoch);
        if (!ok) break;
        tc_fence_after();
        const uint32_t va = smem_u32(vs + (j % kStages) * Cfg::kKvBytes);
#pragma unroll
        for (int kk = 0; kk < kTuKeys / 16; ++kk)
          umma_ts(tO, tS(j & 1) + 8u * (uint32_t)kk, umma_desc_sw128(va + kk * 2048, Cfg::kKvHalf, 1024), id_pv,
                  (j > 0 || kk > 0) ? 1u : 0u);
        umma_commit(&vempty[j % kStages]);
        umma_commit(j == n_tiles - 1 ? o_full : &pv_done[j & 1]);
      }
      if (!ok) {
        raise_timeout(a.err, a.epoch);
        umma_commit(fin);
        mbar_wait(fin, 0);
      }
    }
    __syncwarp();
  } else {
    // ---------------------------------------- softmax --------------------------------------------
    const int copy = warp / warps_per_copy;  // which of the kSplit copies of the rows
    const int r = threadIdx.x & (kRows - 1);
    const uint32_t lane_base = (uint32_t)(32 * warp) << 16;
    const bool live = (r & ~31) < rows;  // whole warps
    const int node = node0 + min(r, rows - 1) / a.group;
    const int64_t* words = a.tree_mask != nullptr ? a.tree_mask + (sq.q0 + node) * a.mask_words : nullptr;
    float m_use = -INFINITY, l_run = 0.f;
    bool alive = true;

    // Bits of the tile at key kb that this row sees (bit c: key kb + c), sub-tiles that are not loaded
    // and keys behind the partition left out.
    auto visible = [&](int kb, uint32_t loaded) -> uint64_t {
      const int s0 = kb - hist;  // node of the tile's first key
      uint64_t keep;
      if (s0 + kTuKeys <= 0) {
        keep = ~0ull;
      } else if (words == nullptr) {
        const int nv = node + 1 - s0;  // chain: nodes up to its own
        keep = nv <= 0 ? 0ull : (nv >= 64 ? ~0ull : (1ull << nv) - 1ull);
      } else if (s0 < 0) {
        keep = ((uint64_t)__ldg(words) << -s0) | ((1ull << -s0) - 1ull);
      } else {
        const int w = s0 >> 6, sh = s0 & 63;
        keep = (w < a.mask_words ? (uint64_t)__ldg(words + w) : 0ull) >> sh;
        if (sh != 0 && w + 1 < a.mask_words) keep |= (uint64_t)__ldg(words + w + 1) << (64 - sh);
      }
      const int nv = t_end - kb;
      if (nv < 64) keep &= (1ull << nv) - 1ull;
#pragma unroll
      for (int u = 0; u < kTuSubs; ++u)
        if (!((loaded >> u) & 1u)) keep &= ~(0xffffull << (16 * u));
      return keep;
    };

    // one tile; kMasked: it may hold keys that the row does not see
    auto tile = [&](auto masked, int j, uint64_t keep) {
      constexpr bool kMasked = decltype(masked)::value;
      const uint32_t srow = tS(j & 1) + lane_base;
      uint32_t sv[kCols];
      load_scores<kCols>(srow + (uint32_t)(copy * kCols), sv);
      bool any = true;
      if (kMasked) {
        keep >>= copy * kCols;
        if (kCols < 64) keep &= (1ull << (kCols & 63)) - 1ull;
        any = keep != 0;
#pragma unroll
        for (int c = 0; c < kCols; ++c)
          if (!((keep >> c) & 1ull)) sv[c] = 0xff800000u;
      }
      float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int c = 0; c < kCols; ++c) mx[c & 3] = fmaxf(mx[c & 3], __uint_as_float(sv[c]));
      float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * a.scale_log2;
      if (any) top = fmaxf(top, -FLT_MAX);  // keys were seen, whatever their scores
      float corr = 1.f;
      if (top > m_use + kTuRescale || (m_use == -INFINITY && top != -INFINITY)) {
        corr = fast_exp2(m_use - top);  // m_use = -inf: 0
        m_use = top;
      }
      const float m_sub = m_use == -INFINITY ? 0.f : m_use;
      const uint64_t sc2 = f2_pack(a.scale_log2, a.scale_log2), nm2 = f2_pack(-m_sub, -m_sub);
      uint64_t sum2[2] = {f2_pack(0.f, 0.f), f2_pack(0.f, 0.f)};
      uint32_t w[kCols / 2];
#pragma unroll
      for (int c = 0; c < kCols / 2; ++c) {
        float x0, x1;
        f2_unpack(f2_fma(f2_pack(__uint_as_float(sv[2 * c]), __uint_as_float(sv[2 * c + 1])), sc2, nm2), x0, x1);
        const float e0 = fast_exp2(x0), e1 = fast_exp2(x1);
        sum2[c & 1] = f2_add(sum2[c & 1], f2_pack(e0, e1));
        // weights are rounded to the pool's type for the product with V (half a step each); the sum
        // keeps them in 32 bits
        w[c] = pack2<kBf16>(e0, e1);
      }
      store_weights<kCols>(srow, copy, w);
      float a0, a1, b0, b1;
      f2_unpack(sum2[0], a0, a1);
      f2_unpack(sum2[1], b0, b1);
      l_run = l_run * corr + ((a0 + a1) + (b0 + b1));
      if (j > 0 && __any_sync(0xffffffffu, corr != 1.f)) {
        // O is stable once the product of tile j - 1 is done; that of tile j waits for this warp
        if (!__all_sync(0xffffffffu, mbar_wait(&pv_done[(j - 1) & 1], (unsigned)(((j - 1) >> 1) & 1), a.err, a.epoch))) {
          alive = false;
          return;
        }
        tc_fence_after();
#pragma unroll 1
        for (int c0 = 0; c0 < D; c0 += 32) {
          uint32_t v[32];
          tmem_ld32_sync(tO + lane_base + c0, v);
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * corr);
          tmem_st32(tO + lane_base + c0, v);
        }
      }
    };

    if (live) {
      for (int j = 0; j < n_tiles; ++j) {
        const int kb = t_begin + j * kTuKeys;
        const bool edge = kb + kTuKeys > t_end || kb + kTuKeys > hist;
        if (!__all_sync(0xffffffffu, mbar_wait(&s_full[j & 1], (unsigned)((j >> 1) & 1), a.err, a.epoch))) {
          alive = false;
          break;
        }
        tc_fence_after();
        const uint32_t loaded = kmask[j & 7];
        if (!edge && loaded == (1u << kTuSubs) - 1u) {
          tile(std::false_type{}, j, ~0ull);
        } else {
          tile(std::true_type{}, j, visible(kb, loaded));
          // V of the tile: rows without a token zeroed, non-finite elements of drafted tokens taken out
          if (!alive || !__all_sync(0xffffffffu, mbar_wait(&vfull[j % kStages], (unsigned)((j / kStages) & 1), a.err,
                                                           a.epoch))) {
            alive = false;
            break;
          }
          uint8_t* vst = vs + (j % kStages) * Cfg::kKvBytes;
          const int idx = (copy * min(warps_per_copy, (rows + 31) >> 5) + (r >> 5)) * 32 + lane;
          for (int e = idx; e < kTuKeys * 8 * kHalves; e += 32 * live_warps) {
            const int key = e / (8 * kHalves), c = e % (8 * kHalves);
            uint4* p = reinterpret_cast<uint4*>(vst + (c >> 3) * Cfg::kKvHalf + key * 128 + (((c & 7) ^ (key & 7)) << 4));
            if (kb + key >= t_end || !((loaded >> (key >> 4)) & 1u)) {
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
                *reinterpret_cast<volatile int*>(bad_v) = 1;
              }
            }
          }
          fence_proxy_async_smem();
        }
        if (!alive) break;
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&p_full[j & 1]);
      }
      if (alive) alive = __all_sync(0xffffffffu, mbar_wait(o_full, 0, a.err, a.epoch));
      tc_fence_after();
      if (!alive && lane == 0) raise_timeout(a.err, a.epoch);
    }
    // ---- join the copies and write: thread (r, copy) ends with columns [copy * kW, + kW) ----------
    // (every copy of the Q, K and V buffers is consumed by now: they hold the exchanged states)
    constexpr int kW = D / kSplit;
    constexpr int kChunk = kW < 32 ? kW : 32;
    constexpr int kPad = kW + 4;  // floats; keeps 16-byte accesses of neighbouring rows in other banks
    float acc[kW];
    float M = m_use, L = l_run;
    const bool done = alive && live;
    if constexpr (kSplit == 1) {
      if (done) {
#pragma unroll
        for (int c0 = 0; c0 < kW; c0 += kChunk)
          load_out<kChunk>(tO + lane_base + c0, *reinterpret_cast<float(*)[kChunk]>(&acc[c0]));
      }
    } else {
      float2* ml = reinterpret_cast<float2*>(qs);
      float* xs = reinterpret_cast<float*>(qs + 1024);
      named_barrier(1, 128);  // all four warps' products are done: the buffers are free
      ml[copy * kRows + r] = done ? make_float2(m_use, l_run) : make_float2(-INFINITY, 0.f);
      named_barrier(1, 128);
      M = -INFINITY;
#pragma unroll
      for (int s = 0; s < kSplit; ++s) M = fmaxf(M, ml[s * kRows + r].x);
      const float M0 = M == -INFINITY ? 0.f : M;
      L = 0.f;
#pragma unroll
      for (int s = 0; s < kSplit; ++s) L = fmaf(ml[s * kRows + r].y, fast_exp2(ml[s * kRows + r].x - M0), L);
      const float f = fast_exp2(m_use - M0);
      if (done) {
#pragma unroll
        for (int t = 0; t < kSplit; ++t) {
#pragma unroll
          for (int c0 = 0; c0 < kW; c0 += kChunk) {
            float v[kChunk];
            load_out<kChunk>(tO + lane_base + t * kW + c0, v);
            if (t == copy) {
#pragma unroll
              for (int i = 0; i < kChunk; ++i) acc[c0 + i] = v[i] * f;
            } else {
              float* dst = xs + ((r * kSplit + t) * kSplit + copy) * kPad + c0;
#pragma unroll
              for (int i = 0; i < kChunk; i += 4)
                *reinterpret_cast<float4*>(dst + i) = make_float4(v[i] * f, v[i + 1] * f, v[i + 2] * f, v[i + 3] * f);
            }
          }
        }
      }
      named_barrier(1, 128);
      if (done) {
#pragma unroll
        for (int s = 0; s < kSplit; ++s) {
          if (s == copy) continue;
          const float* src = xs + ((r * kSplit + copy) * kSplit + s) * kPad;
#pragma unroll
          for (int i = 0; i < kW; i += 4) {
            const float4 v = *reinterpret_cast<const float4*>(src + i);
            acc[i] += v.x;
            acc[i + 1] += v.y;
            acc[i + 2] += v.z;
            acc[i + 3] += v.w;
          }
        }
      }
    }
    const int col0 = kSplit == 1 ? 0 : copy * kW;
    if (done && *reinterpret_cast<volatile int*>(bad_v) != 0 && r < rows) {
      // the non-finite elements that were taken out of V, for the rows that see them
      const int32_t* table = a.block_table + (int64_t)b * a.bt_stride;
      for (int t = max(t_begin, hist); t < t_end; ++t) {
        const int s = t - hist;
        const bool see = words != nullptr ? ((__ldg(words + (s >> 6)) >> (s & 63)) & 1) != 0 : s <= node;
        const int blk = __ldg(table + (t >> a.block_shift));
        if (!see || blk < 0 || blk >= a.num_blocks) continue;
        const T* v = static_cast<const T*>(a.v_pool) + (int64_t)blk * a.kv_block_stride +
                     (int64_t)(t & (a.block_size - 1)) * a.n_kv_heads * D + (int64_t)kvh * D + col0;
#pragma unroll
        for (int i = 0; i < kW; ++i) {
          const float x = static_cast<float>(v[i]);
          if (!(fabsf(x) <= FLT_MAX)) acc[i] += x;
        }
      }
    }
    if (r < rows && live) {
      const bool none = !alive || M == -INFINITY;  // the row sees none of these keys
      const int64_t qh = out_row(r);
      if (n_parts == 1) {
        const float inv = none ? 0.f : 1.f / L;
        T* o = static_cast<T*>(a.out) + qh * D + col0;
#pragma unroll
        for (int i = 0; i < kW; i += 8) {
          float f[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) f[e] = none ? 0.f : acc[i + e] * inv;
          uint4 w;
          w.x = pack2<kBf16>(f[0], f[1]);
          w.y = pack2<kBf16>(f[2], f[3]);
          w.z = pack2<kBf16>(f[4], f[5]);
          w.w = pack2<kBf16>(f[6], f[7]);
          *reinterpret_cast<uint4*>(o + i) = w;
        }
      } else {
        const int64_t pi = qh * a.max_parts + part;
        float* o = a.ws_acc + pi * D + col0;
#pragma unroll
        for (int i = 0; i < kW; i += 4)
          *reinterpret_cast<float4*>(o + i) = none ? make_float4(0.f, 0.f, 0.f, 0.f)
                                                   : make_float4(acc[i], acc[i + 1], acc[i + 2], acc[i + 3]);
        if (copy == 0) {
          a.ws_m[pi] = none ? -INFINITY : M;
          a.ws_l[pi] = none ? 0.f : L;
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 5) {
    tc_fence_after();
    tmem_dealloc(tmem, kTuTmemCols);
  }
}

// ------------------------------------------------------------------------------------------------
template <typename T, int D, int kSplit>
static cudaError_t launch_tu(const TreeArgs& a, const CUtensorMap& km, const CUtensorMap& vm, cudaStream_t s) {
  constexpr int rows = 128 / kSplit;
  CUtensorMap qm;
  if (!encode_q_map(&qm, a.q, std::is_same<T, __nv_bfloat16>::value ? PA_BF16 : PA_FP16, a.total_q, a.n_q_heads, D,
                    a.group, rows / a.group))
    return cudaErrorInvalidValue;
  constexpr int smem = TuCfg<D>::kSmemBytes;
  static bool attr_set[64] = {};  // per instantiation and device; idempotent, so a race is harmless
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !attr_set[dev]) {
    e = cudaFuncSetAttribute(tree_umma_kernel<T, D, kSplit>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) attr_set[dev] = true;
  }
  const int nodes_tile = rows / a.group;
  const int q_tiles = (a.max_nodes + nodes_tile - 1) / nodes_tile;
  const int64_t grid = (int64_t)a.batch * a.max_parts * q_tiles * a.n_kv_heads;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kTuThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, tree_umma_kernel<T, D, kSplit>, a, q_tiles, km, vm, qm);
}

template <typename T, int D>
static cudaError_t launch_tu_rows(const TreeArgs& a, const CUtensorMap& km, const CUtensorMap& vm, cudaStream_t s) {
  const int64_t rows = (int64_t)a.max_nodes * a.group;
  if (rows <= 32) return launch_tu<T, D, 4>(a, km, vm, s);
  if (rows <= 64) return launch_tu<T, D, 2>(a, km, vm, s);
  return launch_tu<T, D, 1>(a, km, vm, s);
}

cudaError_t launch_tree_umma(const TreeArgs& a, pa_dtype dt, cudaStream_t s, int* launches) {
  CUtensorMap km, vm;
  if (!encode_pool_map(&km, a.k_pool, dt, a.num_blocks, a.block_size, a.n_kv_heads, a.head_dim, a.kv_block_stride) ||
      !encode_pool_map(&vm, a.v_pool, dt, a.num_blocks, a.block_size, a.n_kv_heads, a.head_dim, a.kv_block_stride))
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

}  // namespace pa
