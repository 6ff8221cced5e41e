// tcgen05 attention of causal chunks behind a sliding window (paged_attention_window; bf16/fp16, block_size % 16 == 0).
//
// The pipeline is that of prefill_umma.cu: one CTA per SM, two Q tiles of 128 (token, head) rows of one KV head that share
// every 128-key K and V tile, two softmax groups, a K producer, a V producer and an MMA warp, S_k and O_k in tensor
// memory.  What differs:
//
// * Items are blocks of 256 / G tokens of one sequence (times KV heads), counted over the batch, so that no tile is computed
//   for rows of another sequence and short chunks spread over the SMs.  The K producer alone finds them, walking the batch
//   once (the next item while the current one's tiles are on their way), and hands a record to every other role.
//   (Blocks of the packed rows, as the prefill kernel takes them: 24 chunks of 1 to 300 tokens, 12 heads, head_dim 64,
//   window 500: 130 us.)  An item of one Q tile leaves the second softmax group out.
// * Keys: a query at position p attends to j > p - window and j < sinks.  An item's keys are the 16-key sub-tiles that hold
//   sinks and those from its first row's window on, packed into tiles without a gap (a sub-tile is a box of its own
//   anyway); nothing else is loaded or looked up.  Tiles that every row sees whole take no mask, the others one bit a key.
//   Two instantiations of the softmax, no more: the code has to stay in the instruction cache (a third for causal cuts
//   alone cost 4 %, code for very large scores inside the loop 20 %).
// * The stabiliser is an unscaled score (see tree_umma.cu for why, and for the lift of fp16 weights).
// * A masked value cannot be deselected in a product (0 * NaN), and a tile that some rows of an item do not see whole may
//   hold a value that is not finite.  A warp of its own, the guard, looks through every such V tile before its products and
//   makes those values 0 that not every row sees; rows that do see one get their NaN when they are written (win_poison).
//   (That look by the softmax groups took a quarter of the call.  Looked for in the results instead, with such rows
//   computed again key by key, one NaN took 8 prompts from 344 us to 16 ms, and 2,048 rows over 8,192 tokens without a window
//   from 264 us to 236 ms; by the guard both take as long with it as without.)
//
// Bound by the round S, softmax, P V of a tile (4,000 cycles for two Q tiles).  8 prompts of 2,048 rows, 32 / 8 heads,
// head_dim 128, bf16, window 1,024 and 4: 330 us (810 TFLOP/s over the pairs that are seen; 449 with the prefill kernel's
// loaders and waits in line).  The 24 chunks above: 57 us, 2.2 items a CTA on the average and 3 at most.
//
// Every mbarrier wait is bounded (PA_DEVERR_TIMEOUT, with a cooperative abort); tensor memory is always released.
#include <cudaTypedefs.h>

#include "prefill_common.cuh"
#include "window_mask.h"

namespace pa {

// mbar_wait with everything but its first try out of line: the kernel has two dozen waits, and its code has to stay in the
// instruction cache.
static __device__ __noinline__ bool win_wait_on(uint64_t* bar, unsigned parity, const unsigned* err, unsigned epoch) {
  return mbar_wait(bar, parity, err, epoch);
}
__device__ __forceinline__ bool win_wait(uint64_t* bar, unsigned parity, const unsigned* err = nullptr,
                                         unsigned epoch = 0) {
  return mbar_try_wait(bar, parity) || win_wait_on(bar, parity, err, epoch);
}

constexpr int kWinThreads = kUmThreads + 32;  // the guard is the last warp
constexpr int kWinSlots = 8;  // item records in flight between the K producer and their readers

// Rows [T0, T1) of sequence b; first: position of row T0; n: the sequence's context (0 and !ok: refused).
struct WinItem {
  int b, T0, T1, first, n;
  bool ok;
  __device__ __forceinline__ int kv_end() const { return ok ? first + (T1 - T0) : 0; }
  // Whether the second Q tile has rows (tile_tokens: of a Q tile).
  __device__ __forceinline__ bool both(int tile_tokens) const { return T1 - T0 > tile_tokens; }
};

// Items of a call at most: every sequence may end inside a block.  (An unordered query_start_loc could claim rows again and
// again; items end here all the same.)
__host__ __device__ inline int64_t win_items(int batch, int64_t rows, int block_tokens, int n_kv_heads) {
  return ((batch < rows ? batch : rows) + rows / block_tokens) * n_kv_heads;
}

// The items' blocks in order.
struct WinWalk {
  const AttnArgs& a;
  const int block_tokens, max_len, items;
  int b, before, q0;  // sequence, blocks before it, its first row

  __device__ __forceinline__ WinWalk(const AttnArgs& args, int tokens, int longest)
      : a(args), block_tokens(tokens), max_len(longest),
        items((int)win_items(args.batch, args.rows, tokens, args.n_kv_heads)), b(0), before(0),
        q0(ld_nc_s32(args.query_start_loc)) {}
  // Item w (not before the last one asked for); false: there are no more.
  __device__ __forceinline__ bool find(int w, WinItem& it) {
    const int block = w / a.n_kv_heads;
    while (b < a.batch && w < items) {
      const int q1 = ld_nc_s32(a.query_start_loc + b + 1);
      const int r0 = max(q0, 0), r1 = (int)min((int64_t)q1, a.rows);
      const int blocks = r1 > r0 ? (r1 - r0 + block_tokens - 1) / block_tokens : 0;
      if (block < before + blocks) {
        const int n = ld_nc_s32(a.context_lens + b);
        it.b = b;
        it.T0 = r0 + (block - before) * block_tokens;
        it.T1 = min(it.T0 + block_tokens, r1);
        it.ok = q0 >= 0 && q1 <= a.rows && n >= q1 - q0 && n <= max_len;
        it.n = it.ok ? n : 0;
        it.first = it.ok ? n - (q1 - q0) + (it.T0 - q0) : 0;
        return true;
      }
      before += blocks;
      q0 = q1;
      ++b;
    }
    return false;
  }
};

// An item's keys as a line of 16-key sub-tiles: those that hold sinks (if these end before the window begins), then
// those from the window's first key on.
struct WinSubs {
  int sinks, skip, n;  // how many hold sinks, how many are left out behind them, how many in all
  __device__ __forceinline__ WinSubs(const AttnArgs& a, const WinItem& it) {
    const int low = it.ok ? max(it.first + 1 - a.window, 0) : 0;
    sinks = (min(a.sinks, low) + 15) >> 4;
    skip = max((low >> 4) - sinks, 0);
    n = ((it.kv_end() + 15) >> 4) - skip;
  }
  __device__ __forceinline__ int tiles() const { return (n + kUmSub - 1) / kUmSub; }
  __device__ __forceinline__ int key(int u) const { return 16 * (u >= sinks ? u + skip : u); }  // first key of sub-tile u
};

// A tile of an item.  It may begin with sub-tiles of sinks: columns below `split` are keys from `start` on, the others continue
// to kb + column.
struct WinTile {
  int start, split, kb;
  __device__ __forceinline__ WinTile(const WinSubs& sb, int tile) {
    start = tile * kUmKeys;
    split = 16 * max(sb.sinks - tile * kUmSub, 0);
    kb = start + (split < kUmKeys ? 16 * sb.skip : 0);
  }
  __device__ __forceinline__ bool mixed() const { return split > 0 && split < kUmKeys; }
  __device__ __forceinline__ int key(int column) const { return (column < split ? start : kb) + column; }
};

// What the rows of an item see of the keys: all of them, some, none.
struct WinSees {
  int first, last, low_first, low_last, sinks;  // positions of the first and the last row, and where their windows begin
  __device__ __forceinline__ WinSees(const AttnArgs& a, const WinItem& it)
      : first(it.first), last(it.kv_end() - 1), low_first(window_low(it.first, a.window)),
        low_last(window_low(it.kv_end() - 1, a.window)), sinks(a.sinks) {}
  __device__ __forceinline__ bool all(int key) const { return key <= first && (key >= low_last || key < sinks); }
  __device__ __forceinline__ bool some(int key) const { return key <= last && (key >= low_first || key < sinks); }
  // Whether every row sees every key of the tile.
  __device__ __forceinline__ bool whole(const WinTile& t, unsigned loaded) const {
    return loaded == (1u << kUmSub) - 1u && !t.mixed() && t.kb + kUmKeys - 1 <= first &&
           (t.kb >= low_last || t.kb + kUmKeys <= sinks);
  }
};

// The scores of a warp's rows in the 128 columns from taddr on become (s - m) * sc.  (Rare, and kept out of the loop's
// code.)
static __device__ __noinline__ void s_distances(uint32_t taddr, float sc, float m) {
#pragma unroll 1
  for (int c0 = 0; c0 < kUmKeys; c0 += 32) {
    uint32_t sv[32];
    tmem_ld32_sync(taddr + (uint32_t)c0, sv);
#pragma unroll
    for (int c = 0; c < 32; ++c) sv[c] = __float_as_uint((__uint_as_float(sv[c]) - m) * sc);
    tmem_st32(taddr + (uint32_t)c0, sv);
  }
  tmem_wait_st();
}

// The scores of a warp's rows in the 128 columns from taddr on that a row does not see (bits of mask) become -inf.
static __device__ __noinline__ void s_mask(uint32_t taddr, uint32_t m0, uint32_t m1, uint32_t m2, uint32_t m3) {
#pragma unroll 1
  for (int c0 = 0; c0 < kUmKeys; c0 += 32) {
    uint32_t sv[32];
    tmem_ld32_sync(taddr + (uint32_t)c0, sv);
#pragma unroll
    for (int c = 0; c < 32; ++c)
      if (!((m0 >> c) & 1u)) sv[c] = 0xff800000u;
    tmem_st32(taddr + (uint32_t)c0, sv);
    m0 = m1, m1 = m2, m2 = m3;
  }
  tmem_wait_st();
}

// Row maximum and weights of one S tile, as prefill_umma.cu's with an unscaled stabiliser (sc > 0); sees: whether the row
// sees a key of the tile.  Weights are 2^(s * sc - m * sc) in one rounding, but where m * sc of a row is itself rounded by
// more than an eighth (scores of 2^20): there they are 2^((s - m) * sc).
template <bool kBf16>
__device__ __forceinline__ float row_softmax_window(uint32_t srow, float sc, bool sees, float& m_use, float& l_run) {
  // (bf16: 2^8 lower, so that a weight is 1 at most and its product with the largest values stays finite)
  constexpr float kLift = kBf16 ? -8.f : 7.f;
  const ScoreFix fix{};
  // (keys that are seen count, whatever their scores: a row of scores of -inf is told from one that sees nothing)
  float mx = sees ? -FLT_MAX : -INFINITY;
#pragma unroll 1
  for (int h = 0; h < 2; ++h) {
    uint32_t sv[64];
    s_load64<0>(srow + 64u * h, sv, fix, 64 * h, 0u, 0u);
    mx = fmaxf(mx, s_max64(sv, 1.f));
  }
  float corr = 1.f;
  if ((mx - m_use) * sc > kUmRescaleThreshold) {
    corr = fast_exp2((m_use - mx) * sc);  // m_use = -inf -> 0
    m_use = mx;
  }
  const float m_sub = m_use == -INFINITY ? 0.f : m_use;
  const bool far = __any_sync(0xffffffffu, !(fabsf(m_sub * sc) <= 1048576.f));
  if (far) s_distances(srow, sc, m_sub);
  const float w_scale = far ? 1.f : sc, w_sub = (far ? 0.f : m_sub * sc) - kLift;
  float rs = 0.f;
#pragma unroll 1
  for (int h = 0; h < 2; ++h) {
    uint32_t sv[64];
    s_load64<0>(srow + 64u * h, sv, fix, 64 * h, 0u, 0u);
    rs += p_store64<kBf16>(srow + 32u * h, sv, w_scale, w_sub);
  }
  l_run = l_run * corr + rs;
  return corr;
}

// acc, NaN from then on if one of eight 16-bit floats is infinite or NaN (multiplied by 0 they give NaN).
template <bool kBf16>
__device__ __forceinline__ void note_nonfinite(const uint4& v, uint32_t& acc) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (kBf16)
      asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(acc) : "r"(w[i]), "r"(0u));
    else
      asm("fma.rn.f16x2 %0, %1, %2, %0;" : "+r"(acc) : "r"(w[i]), "r"(0u));
  }
}

// The guard's look through a V tile (one warp): false if all of it is finite.
template <bool kBf16, int kBytes>
__device__ __forceinline__ bool v_nonfinite(const uint8_t* tile, int lane) {
  uint32_t acc[2] = {0u, 0u};
#pragma unroll 1
  for (int e = lane; e < kBytes / 16; e += 8 * 32) {
    uint4 v[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) v[u] = *reinterpret_cast<const uint4*>(tile + 16 * (e + 32 * u));
#pragma unroll
    for (int u = 0; u < 8; ++u) note_nonfinite<kBf16>(v[u], acc[u & 1]);
  }
  return __any_sync(0xffffffffu, ((acc[0] | acc[1]) & 0x7fff7fffu) != 0u);
}

// Zeros for the rows of a V tile that hold no data or lie past the context, and for the values that are not finite and that
// not every row of the item sees.  Returns whether some row sees one of these.
template <bool kBf16, int kBytes>
__device__ __noinline__ bool v_clear(uint8_t* tile, int lane, const WinTile t, const WinSees sees, int n, unsigned loaded) {
  constexpr uint32_t kExp = kBf16 ? 0x7f80u : 0x7c00u;
  bool seen = false;
#pragma unroll 1
  for (int e = lane; e < kBytes / 16; e += 32) {
    const int row = (e >> 3) & (kUmKeys - 1), key = t.key(row);
    uint4* p = reinterpret_cast<uint4*>(tile + 16 * e);
    if (!((loaded >> (row >> 4)) & 1u) || key >= n) {
      *p = make_uint4(0, 0, 0, 0);
      continue;
    }
    if (sees.all(key)) continue;
    uint4 v = *p;
    uint32_t* w = reinterpret_cast<uint32_t*>(&v);
    bool found = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t keep = 0xffffffffu;
      if ((w[i] & kExp) == kExp) keep &= 0xffff0000u;
      if (((w[i] >> 16) & kExp) == kExp) keep &= 0x0000ffffu;
      found |= keep != 0xffffffffu;
      w[i] &= keep;
    }
    if (found) {
      *p = v;
      seen |= sees.some(key);
    }
  }
  return __any_sync(0xffffffffu, seen);
}

// NaN for the outputs of a warp's rows (`out` a lane's row, `bound` its position; -1: none) whose columns hold a value that is not finite
// and that the row sees, among the keys that only some rows of the item see: the guard made these 0.
template <typename T, int D>
__device__ __noinline__ void win_poison(const AttnArgs& a, const WinItem it, int kvh, int bound, T* out) {
  constexpr int kPer = D / 32, kUnroll = 8;
  const int lane = threadIdx.x & 31;
  const WinSees sees(a, it);
  const int low = window_low(bound, a.window);
  const int32_t* table = a.block_table + (int64_t)it.b * a.bt_stride;
  uint32_t cols[kPer] = {};  // column lane' * kPer + c: bit lane' of cols[c]
  // keys behind the first row's, then those before the last row's window
#pragma unroll 1
  for (int range = 0; range < 2; ++range) {
    const int end = range == 0 ? sees.last + 1 : min(sees.low_last, sees.first + 1);
#pragma unroll 1
    for (int j0 = range == 0 ? sees.first + 1 : sees.low_first; j0 < end; j0 += kUnroll) {
      T v[kUnroll][kPer];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int j = j0 + u;
        const int blk = j < end ? ld_nc_s32(table + (j >> a.block_shift)) : -1;
        const bool here = blk >= 0 && blk < a.num_blocks;
        const T* src = static_cast<const T*>(a.v_pool) + (here ? (int64_t)blk * a.kv_block_stride : 0) +
                       ((int64_t)(j & (a.block_size - 1)) * a.n_kv_heads + kvh) * D + lane * kPer;
#pragma unroll
        for (int c = 0; c < kPer; ++c) v[u][c] = here ? src[c] : Elt<T>::from_float(0.f);
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int j = j0 + u;
        const bool mine = j <= bound && (j >= low || j < a.sinks);
#pragma unroll
        for (int c = 0; c < kPer; ++c) {
          const unsigned bad = __ballot_sync(0xffffffffu, !(fabsf(static_cast<float>(v[u][c])) <= FLT_MAX));
          if (mine) cols[c] |= bad;
        }
      }
    }
  }
#pragma unroll
  for (int c = 0; c < kPer; ++c)
    for (uint32_t m = cols[c]; m != 0u; m &= m - 1u) out[(__ffs(m) - 1) * kPer + c] = Elt<T>::from_float(NAN);
}

// Record number idx of the K producer's ring; false: the wait gave up, or there are no more items (it.b < 0).
__device__ __forceinline__ bool win_read(const AttnArgs& a, uint64_t* rec_full, const int* recs, int idx, WinItem& it) {
  const int slot = idx % kWinSlots;
  it = WinItem{};
  if (!win_wait(&rec_full[slot], (unsigned)((idx / kWinSlots) & 1), a.err, a.epoch)) return false;
  const int* r = recs + 8 * slot;
  it.b = r[0];
  it.T0 = r[1];
  it.T1 = r[2];
  it.first = r[3];
  it.n = r[4];
  it.ok = r[5] != 0;
  return it.b >= 0;
}

template <typename T, int D, int G>
__global__ void __launch_bounds__(kWinThreads, 1)
    window_umma_kernel(const __grid_constant__ AttnArgs a, const __grid_constant__ CUtensorMap kmap,
                       const __grid_constant__ CUtensorMap vmap, const __grid_constant__ CUtensorMap qmap) {
  using Cfg = UmCfg<D>;
  constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
  constexpr int kHalves = Cfg::kHalves;
  constexpr int kQB = kUmRows / G;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(base);
  uint64_t* kfull = bars + 0;     // [kUmKStages]
  uint64_t* kempty = bars + 4;    // [kUmKStages] completes when both groups' S products have read the tile
  uint64_t* vfull = bars + 8;     // [kUmVStages]
  uint64_t* vempty = bars + 12;   // [kUmVStages] completes when both groups' P V products have read the tile
  uint64_t* q_ready = bars + 16;  // one phase per item: its Q tiles landed
  // per group k, one phase per tile
  uint64_t* s_full = bars + 17;   // [2] S_k computed (and, with it, every earlier product of the CTA)
  uint64_t* p_full = bars + 19;   // [2] P_k written to TMEM (and O_k rescaled)
  uint64_t* pv_done = bars + 21;  // [2] O_k += P_k V finished
  uint64_t* fin = bars + 23;
  uint64_t* mready = bars + 24;   // [8] per tile slot: the sub-tile mask below is written
  uint64_t* q_empty = bars + 32;  // one phase per item: its S products completed, Q may be reloaded
  uint64_t* o_free = bars + 33;   // [2] one phase per item with tiles of group k: it has read O_k
  uint64_t* rec_full = bars + 36;   // [kWinSlots] the record in the slot is written
  uint64_t* rec_empty = bars + 44;  // [kWinSlots] the V producer, the MMA warp, the guard and all 8 softmax warps have read it
  uint64_t* guarded = bars + 52;    // [kUmVStages] the V tile has landed and the guard is done with it
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(base + 512);
  volatile int* v_flag = reinterpret_cast<int*>(base + 520);   // [kUmVStages] some rows see a value that the guard made 0
  uint32_t* kmask = reinterpret_cast<uint32_t*>(base + 544);   // [8] sub-tiles holding data, per tile slot
  int* recs = reinterpret_cast<int*>(base + 576);              // [kWinSlots][8] item records; b < 0: no more
  uint8_t* qs = base + 1024;                       // [2][Q tile]
  uint8_t* ks = qs + 2 * Cfg::kQBytes;             // [kUmKStages][K tile]
  uint8_t* vs = ks + kUmKStages * Cfg::kKvBytes;   // [kUmVStages][V tile]
  static_assert(kUmKStages <= 4 && kUmVStages <= 4, "barrier slots");
  static_assert(576 + kWinSlots * 32 <= 1024 && 56 * 8 <= 512, "records and barriers fit their 1 KB slot");

  // Item w: block w / n_kv_heads of the batch, KV head w % n_kv_heads; this CTA takes blockIdx.x, blockIdx.x + gridDim.x, ...
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int max_len = (int)min(a.bt_stride << a.block_shift, (int64_t)kTreeMaxContext);
  const int bmask = a.block_size - 1;

  if (threadIdx.x == 0) {
    prefetch_tensormap(&kmap);
    prefetch_tensormap(&vmap);
    prefetch_tensormap(&qmap);
    // one commit per tile closes a K (V) stage: it follows both groups' S (P V) products of the tile
    for (int s = 0; s < kUmKStages; ++s) {
      mbar_init(&kfull[s], 1);
      mbar_init(&kempty[s], 1);
    }
    for (int s = 0; s < kUmVStages; ++s) {
      mbar_init(&vfull[s], 1);
      mbar_init(&vempty[s], 1);
      mbar_init(&guarded[s], 1);
    }
    for (int k = 0; k < 2; ++k) {
      mbar_init(&s_full[k], 1);
      mbar_init(&p_full[k], 128);
      mbar_init(&pv_done[k], 1);
      mbar_init(&o_free[k], 128);
    }
    mbar_init(q_ready, 1);
    mbar_init(q_empty, 1);
    for (int k = 0; k < kWinSlots; ++k) {
      mbar_init(&rec_full[k], 1);
      mbar_init(&rec_empty[k], 11);  // V producer, MMA, guard, 8 softmax warps
    }
    mbar_init(fin, 1);
    for (int s = 0; s < 8; ++s) mbar_init(&mready[s], 1);
    fence_barrier_init();
  }
  if (warp == 10) tmem_alloc(tmem_slot, kUmTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // S_k at columns [128k, +128) (P_k, two 16-bit values per column, in its first 64), O_k at
  // [256 + 128k, +D)
  auto tS = [&](int k) { return tmem + 128u * (uint32_t)k; };
  auto tO = [&](int k) { return tmem + 256u + 128u * (uint32_t)k; };

  if (warp == 8 || warp == 9) {
    // ------- producers, lane 0 alone (see prefill_umma.cu), in one code: warp 8 finds the items, writes their records and
    // streams K tiles; warp 9 loads each item's Q tiles, then its V tiles -------
    if (lane == 0) {
      const bool is_v = warp == 9;
      uint64_t* full = is_v ? vfull : kfull;
      uint64_t* empty = is_v ? vempty : kempty;
      uint8_t* ring = is_v ? vs : ks;
      const CUtensorMap* map = is_v ? &vmap : &kmap;
      const int depth = is_v ? kUmVStages : kUmKStages;
      int i = 0;    // tiles issued, counted over all items of the CTA
      int rec = 0;  // records written (K) or read (V), which is the Q loads issued
      bool alive = true;
      WinWalk walk(a, kQB, max_len);
      WinItem it{}, next{};
      bool more = !is_v && walk.find((int)blockIdx.x, next);
      for (int w = blockIdx.x; alive; w += gridDim.x) {
        const int kvh = w % a.n_kv_heads, slot = rec % kWinSlots;
        if (is_v) {
          if (!win_read(a, rec_full, recs, rec, it)) {
            alive = it.b < 0;
            break;
          }
          mbar_arrive(&rec_empty[slot]);
          // both Q tiles of the item, once every S product of the previous item has completed
          if (rec > 0 && !win_wait(q_empty, (unsigned)((rec - 1) & 1), a.err, a.epoch)) {
            alive = false;
            break;
          }
          const int q_tiles = it.both(kUmTileRows / G) ? 2 : 1;
          mbar_arrive_expect_tx(q_ready, (uint32_t)(q_tiles * Cfg::kQBytes));
          for (int k = 0; k < q_tiles; ++k)
#pragma unroll
            for (int h = 0; h < kHalves; ++h)
              tma_load_3d(qs + k * Cfg::kQBytes + h * Cfg::kQHalf, &qmap, h * 64, kvh * G, it.T0 + k * (kUmTileRows / G),
                          q_ready);
        } else {
          it = next;
          if (rec >= kWinSlots && !win_wait(&rec_empty[slot], (unsigned)((rec / kWinSlots - 1) & 1), a.err, a.epoch)) {
            alive = false;
            break;
          }
          int* r = recs + 8 * slot;
          r[0] = more ? it.b : -1;
          r[1] = it.T0;
          r[2] = it.T1;
          r[3] = it.first;
          r[4] = it.n;
          r[5] = it.ok ? 1 : 0;
          mbar_arrive(&rec_full[slot]);
          if (!more) break;
        }
        ++rec;
        const WinSubs sb(a, it);
        const int nt = sb.tiles();
        const int32_t* table = a.block_table + (int64_t)it.b * a.bt_stride;
        // the table entries of a tile's sub-tiles (-1: past the item's keys), read one tile ahead so that their latency
        // passes during the wait for the ring slot
        int ys[kUmSub];
        auto table_of = [&](int tile, int (&dst)[kUmSub]) {
#pragma unroll
          for (int sub = 0; sub < kUmSub; ++sub) {
            const int u = tile * kUmSub + sub;
            dst[sub] = u < sb.n ? ld_nc_s32(table + (sb.key(u) >> a.block_shift)) : -1;
          }
        };
        if (nt > 0) table_of(0, ys);
        // (K: the next item is looked up, and its Q tiles prefetched into L2, behind this one's second tile, or its last)
        for (int tile = 0; tile < nt || (!is_v && tile == 0); ++tile) {
          if (tile < nt) {
            int ys_next[kUmSub];
            if (tile + 1 < nt) table_of(tile + 1, ys_next);
            const int s = i % depth, round = i / depth;
            if (round > 0 && !win_wait(&empty[s], (unsigned)((round - 1) & 1), a.err, a.epoch)) {
              alive = false;
              break;
            }
            unsigned m = 0;
#pragma unroll
            for (int sub = 0; sub < kUmSub; ++sub) {
              if (tile * kUmSub + sub < sb.n) {
                if (ys[sub] < 0 || ys[sub] >= a.num_blocks) {
                  if (!is_v) raise_error(a.err, PA_DEVERR_BLOCK_ID);
                } else {
                  m |= 1u << sub;
                }
              }
            }
            if (!is_v) {
              // publish which sub-tiles hold data.  Slot i % 8 was last read for tile i - 8, which both groups finished
              // long ago: K tile i is loaded only after both S products of tile i - kUmKStages completed, which needed
              // each group's P of tile i - kUmKStages - 1.
              kmask[i & 7] = m;
              mbar_arrive(&mready[i & 7]);
            }
            uint8_t* st = ring + s * Cfg::kKvBytes;
            if (m == 0) {
              mbar_arrive(&full[s]);
            } else {
              mbar_arrive_expect_tx(&full[s], (uint32_t)__popc(m) * kHalves * 2048u);
#pragma unroll
              for (int sub = 0; sub < kUmSub; ++sub) {
                if (!((m >> sub) & 1u)) continue;
                const int yo = sb.key(tile * kUmSub + sub) & bmask;
#pragma unroll
                for (int h = 0; h < kHalves; ++h)
                  tma_load_3d(st + h * Cfg::kKvHalf + sub * 2048, map, kvh * D + h * 64, yo, ys[sub], &full[s]);
              }
            }
            ++i;
#pragma unroll
            for (int sub = 0; sub < kUmSub; ++sub) ys[sub] = ys_next[sub];
          }
          if (!is_v && tile == min(1, max(nt - 1, 0))) {
            const int wn = w + (int)gridDim.x;
            more = walk.find(wn, next);
            if (more) {
#pragma unroll
              for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int h = 0; h < kHalves; ++h)
                  tma_prefetch_3d(&qmap, h * 64, wn % a.n_kv_heads * G, next.T0 + k * (kUmTileRows / G));
            }
          }
        }
      }
      if (!alive) raise_timeout(a.err, a.epoch);
      // Leave no copy in flight: after a normal run every issued tile was consumed and these waits
      // return at once; after a timeout elsewhere they wait (bounded) for this ring's last tiles.
      for (int k = i > depth ? i - depth : 0; k < i; ++k) win_wait(&full[k % depth], (unsigned)((k / depth) & 1));
      if (is_v && rec > 0) win_wait(q_ready, (unsigned)((rec - 1) & 1));
    }
  } else if (warp == 10) {
    // ------------------------------------------ MMA ---------------------------------------------
    const uint32_t id_s = umma_idesc_f16(kBf16, 128, kUmKeys, false, false);
    const uint32_t id_pv = umma_idesc_f16(kBf16, 128, D, false, true);
    auto issue_s = [&](int k, int g) {
      const uint32_t qa = smem_u32(qs + k * Cfg::kQBytes);
      const uint32_t ka = smem_u32(ks + (g % kUmKStages) * Cfg::kKvBytes);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t qo = (kk >> 2) * Cfg::kQHalf + (kk & 3) * 32;
        const uint32_t ko = (kk >> 2) * Cfg::kKvHalf + (kk & 3) * 32;
        umma_ss(tS(k), umma_desc_sw128(qa + qo, 16, 1024), umma_desc_sw128(ka + ko, 16, 1024), id_s,
                kk > 0 ? 1u : 0u);
      }
      umma_commit(&s_full[k]);
    };
    auto issue_pv = [&](int k, int g, bool first) {
      const uint32_t va = smem_u32(vs + (g % kUmVStages) * Cfg::kKvBytes);
      // A = P_k from TMEM: 16 keys = 8 columns per instruction; an item's first tile starts O_k
#pragma unroll
      for (int kk = 0; kk < kUmKeys / 16; ++kk)
        umma_ts(tO(k), tS(k) + 8u * (uint32_t)kk, umma_desc_sw128(va + kk * 2048, Cfg::kKvHalf, 1024), id_pv,
                (!first || kk > 0) ? 1u : 0u);
      umma_commit(&pv_done[k]);
    };
    // lane 0 alone issues (no warp-collective step, as for the producers)
    int g = 0;   // tiles of earlier items
    int g1 = 0;  // those that group 1 took part in
    int turns = 0, turns1 = 0;  // earlier items with tiles, and with tiles of group 1
    int n = 0;   // items done
    bool alive = lane == 0;
    for (; alive; ++n) {
      WinItem it;
      if (!win_read(a, rec_full, recs, n, it)) {
        alive = it.b < 0;
        break;
      }
      mbar_arrive(&rec_empty[n % kWinSlots]);
      const int n_all = WinSubs(a, it).tiles();
      const bool both = it.both(kUmTileRows / G);
      bool ok = true;
      auto wait = [&](uint64_t* bar, unsigned parity) {
        ok = ok && win_wait(bar, parity, a.err, a.epoch);
        return ok;
      };
      // the item's first P V into O_k waits until group k has read O_k of its previous item.  (Of those with tiles: the
      // groups go through items without any on their own, and may be several ahead.)
      auto own_o = [&](int k, int j) {
        const int before = k == 0 ? turns : turns1;
        return j > 0 || before == 0 || wait(&o_free[k], (unsigned)((before - 1) & 1));
      };
      // O_k += P_k V of item tile j; group 1's product, if there is one, closes the V tile
      auto pv_of = [&](int k, int j) {
        const int gj = g + j;
        if (!own_o(k, j) || !wait(&p_full[k], (unsigned)((k == 0 ? gj : g1 + j) & 1)) ||
            !wait(&guarded[gj % kUmVStages], (unsigned)((gj / kUmVStages) & 1)))
          return false;
        tc_fence_after();
        issue_pv(k, gj, j == 0);
        if (k == 1 || !both) umma_commit(&vempty[gj % kUmVStages]);
        return true;
      };
      // Fixed issue order per tile: S_0(j), P_1(j-1) V, S_1(j), P_0(j) V (see prefill_umma.cu)
      wait(q_ready, (unsigned)(n & 1));
      for (int j = 0; j < n_all && ok; ++j) {
        const int gj = g + j;
        if (!wait(&kfull[gj % kUmKStages], (unsigned)((gj / kUmKStages) & 1))) break;
        tc_fence_after();
        issue_s(0, gj);
        if (both) {
          if (j > 0 && !pv_of(1, j - 1)) break;
          tc_fence_after();
          issue_s(1, gj);
        }
        umma_commit(&kempty[gj % kUmKStages]);
        if (j == n_all - 1) umma_commit(q_empty);  // after the item's last S products
        if (!pv_of(0, j)) break;
      }
      if (ok && both && n_all > 0) pv_of(1, n_all - 1);
      if (ok && n_all == 0) umma_commit(q_empty);
      alive = ok;
      g += n_all;
      if (n_all > 0) ++turns;
      if (both) {
        g1 += n_all;
        if (n_all > 0) ++turns1;
      }
    }
    if (lane == 0) {
      if (!alive) raise_timeout(a.err, a.epoch);
      if (g > 0) {
        umma_commit(fin);
        win_wait(fin, 0, a.err, a.epoch);
      }
    }
  } else if (warp == 11) {
    // ------------------------------------------ guard -------------------------------------------
    // (never more than the ring ahead of the products, which wait for it and not for vfull: another wait in the MMA warp's
    // code costs 2 %)
    int i = 0;  // tiles of earlier items
    bool alive = true;
    for (int rec = 0; alive; ++rec) {
      WinItem it;
      if (!__all_sync(0xffffffffu, win_read(a, rec_full, recs, rec, it))) {
        alive = __all_sync(0xffffffffu, it.b < 0);
        break;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&rec_empty[rec % kWinSlots]);
      const WinSubs sb(a, it);
      const WinSees sees(a, it);
      const int nt = sb.tiles();
      for (int tile = 0; tile < nt; ++tile, ++i) {
        const int s = i % kUmVStages;
        const unsigned parity = (unsigned)((i / kUmVStages) & 1);
        if (!__all_sync(0xffffffffu, win_wait(&mready[i & 7], (unsigned)((i >> 3) & 1), a.err, a.epoch)) ||
            !__all_sync(0xffffffffu, win_wait(&vfull[s], parity, a.err, a.epoch))) {
          alive = false;
          break;
        }
        const unsigned loaded = kmask[i & 7];
        const WinTile t(sb, tile);
        bool seen = false;
        if (!sees.whole(t, loaded) && v_nonfinite<kBf16, Cfg::kKvBytes>(vs + s * Cfg::kKvBytes, lane)) {
          seen = v_clear<kBf16, Cfg::kKvBytes>(vs + s * Cfg::kKvBytes, lane, t, sees, it.n, loaded);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          v_flag[s] = seen ? 1 : 0;
          mbar_arrive(&guarded[s]);
        }
      }
    }
    if (!alive && lane == 0) raise_timeout(a.err, a.epoch);
  } else {
    // --------------------------------------- softmax groups ---------------------------------------
    const int grp = warp >> 2;           // 0 or 1
    const int r = threadIdx.x & 127;     // row inside the Q tile = TMEM lane
    const int row = grp * kUmTileRows + r;
    const uint32_t lane_base = (uint32_t)(32 * (warp & 3)) << 16;
    const float sc = a.scale_log2;
    int i = 0;     // tiles of this CTA so far
    int mine = 0;  // those of this group
    bool alive = true;
    int rec = 0;
    for (int w = blockIdx.x; alive; w += gridDim.x, ++rec) {
      WinItem it;
      const bool got = __all_sync(0xffffffffu, win_read(a, rec_full, recs, rec, it));
      if (!got) {
        alive = __all_sync(0xffffffffu, it.b < 0);
        break;
      }
      if (lane == 0) mbar_arrive(&rec_empty[rec % kWinSlots]);
      if (!it.ok && threadIdx.x == 0) raise_error(a.err, PA_DEVERR_QUERY_LOC);
      const int tok = it.T0 + row / G;
      const int head = w % a.n_kv_heads * G + row % G;
      float m_use = -INFINITY;  // stabilising maximum (a score) the exponentials are taken against
      float l_run = 0.f;
      const int bound = it.ok && tok < it.T1 ? it.first + (tok - it.T0) : -1;  // the row's position
      const int low = window_low(bound, a.window);                             // first key of its window
      const WinSubs sb(a, it);
      const WinSees sees_all(a, it);
      bool poison = false;  // some rows see a value that the guard made 0
      const int all = sb.tiles();
      const int nt = grp == 0 || it.both(kUmTileRows / G) ? all : 0;
      for (int tile = 0; tile < nt; ++tile, ++i, ++mine) {
        const WinTile t(sb, tile);
        const int split = t.split, kb = t.kb;
        if (!__all_sync(0xffffffffu, win_wait(&mready[i & 7], (unsigned)((i >> 3) & 1), a.err, a.epoch))) {
          alive = false;
          break;
        }
        const unsigned loaded = kmask[i & 7];
        // S_k of this tile is complete, and with it O_k += P_k V of the previous tile (issued before)
        if (!__all_sync(0xffffffffu, win_wait(&s_full[grp], (unsigned)(mine & 1), a.err, a.epoch))) {
          alive = false;
          break;
        }
        tc_fence_after();
        // tiles that every row of the warp sees whole, with every sub-tile loaded, need no mask
        const unsigned all_sub = (1u << kUmSub) - 1u;
        const bool mixed = t.mixed();
        const bool whole = __all_sync(0xffffffffu, loaded == all_sub && kb + kUmKeys - 1 <= bound && !mixed &&
                                                       (kb >= low || kb + kUmKeys <= a.sinks));
        const uint32_t srow = tS(grp) + lane_base;
        bool sees = true;
        if (!whole) {
          uint32_t mask[kUmKeys / 32];
          auto seen = [&](int k0) { return window_seen32(bound, low, a.sinks, k0); };  // keys from k0 on, 32 columns
#pragma unroll
          for (int q = 0; q < kUmKeys / 32; ++q) {
            const uint32_t lm = (((loaded >> (2 * q)) & 1u) ? 0x0000FFFFu : 0u) |
                                (((loaded >> (2 * q + 1)) & 1u) ? 0xFFFF0000u : 0u);
            mask[q] = seen(kb + 32 * q);
            if (mixed) {
              const int h = split - 32 * q;
              const uint32_t first = h >= 32 ? 0xFFFFFFFFu : (h <= 0 ? 0u : (1u << h) - 1u);
              mask[q] = (mask[q] & ~first) | (seen(tile * kUmKeys + 32 * q) & first);
            }
            mask[q] &= lm;
          }
          sees = (mask[0] | mask[1] | mask[2] | mask[3]) != 0u;
          s_mask(srow, mask[0], mask[1], mask[2], mask[3]);
        }
        const float corr = row_softmax_window<kBf16>(srow, sc, sees, m_use, l_run);
        // O_k is stable here (its last product completed before this S_k was issued); the item's
        // first tile starts O_k afresh, so only later tiles rescale it
        if (tile > 0 && __any_sync(0xffffffffu, corr != 1.f)) {
#pragma unroll 1
          for (int c0 = 0; c0 < D; c0 += 32) {
            uint32_t v[32];
            tmem_ld32_sync(tO(grp) + lane_base + c0, v);
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = __float_as_uint(__uint_as_float(v[j]) * corr);
            tmem_st32(tO(grp) + lane_base + c0, v);
          }
        }
        if (!sees_all.whole(t, loaded)) {  // (the stage, and its flag, are not filled again before this P's product)
          if (!__all_sync(0xffffffffu,
                          win_wait(&guarded[i % kUmVStages], (unsigned)((i / kUmVStages) & 1), a.err, a.epoch))) {
            alive = false;
            break;
          }
          poison |= v_flag[i % kUmVStages] != 0;
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&p_full[grp]);
      }
      if (!alive && lane == 0) raise_timeout(a.err, a.epoch);
      if (alive && nt > 0) {
        alive = __all_sync(0xffffffffu, win_wait(&pv_done[grp], (unsigned)((mine - 1) & 1), a.err, a.epoch));
        tc_fence_after();
      }
      i += all - nt;
      const bool have = alive && nt > 0 && m_use != -INFINITY;
      const float inv = have ? 1.f / l_run : 0.f;
      T* orow = static_cast<T*>(a.out) + ((int64_t)tok * a.n_q_heads + head) * D;
      const bool wide = (reinterpret_cast<uintptr_t>(a.out) & 31u) == 0;
#pragma unroll 1
      for (int c0 = 0; c0 < D; c0 += 32) {
        uint32_t v[32];
        tmem_ld32_sync(tO(grp) + lane_base + c0, v);
        if (tok < it.T1) {
#pragma unroll
          for (int j = 0; j < 32; j += 16) {
            uint32_t x[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
              x[e] = pack2<kBf16>(have ? __uint_as_float(v[j + 2 * e]) * inv : 0.f,
                                  have ? __uint_as_float(v[j + 2 * e + 1]) * inv : 0.f);
            st_global32(orow + c0 + j, x, wide);
          }
        }
      }
      if (poison) win_poison<T, D>(a, it, w % a.n_kv_heads, bound, orow);
      // O_k has been read: the next item's first P V may overwrite it
      if (nt > 0) {
        tc_fence_before();
        mbar_arrive(&o_free[grp]);
      }
    }
    if (!alive && lane == 0) raise_timeout(a.err, a.epoch);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 10) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, kUmTmemCols);
  }
}

// ------------------------------------------------------------------------------------------------

template <typename T, int D, int G>
static cudaError_t launch_win_g(const AttnArgs& a, const CUtensorMap& km, const CUtensorMap& vm, cudaStream_t s) {
  CUtensorMap qm;
  if (!encode_q_map(&qm, a.q, std::is_same<T, __nv_bfloat16>::value ? PA_BF16 : PA_FP16, a.rows, a.n_q_heads, D, G,
                    kUmTileRows / G))
    return cudaErrorInvalidValue;
  constexpr int smem = UmCfg<D>::kSmemBytes;
  static bool attr_set[64] = {};  // per instantiation and device; idempotent, so a race is harmless
  static int sm_count[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const bool known = dev >= 0 && dev < 64;
  if (!known || !attr_set[dev]) {
    e = cudaFuncSetAttribute(window_umma_kernel<T, D, G>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    if (known) attr_set[dev] = true;
  }
  int sms = known ? sm_count[dev] : 0;
  if (sms == 0) {
    e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    if (known) sm_count[dev] = sms;
  }
  // (how many there are is known on the device alone)
  const int64_t items = win_items(a.batch, a.rows, kUmRows / G, a.n_kv_heads);
  if (items > 0x7fffffffLL - sms) return cudaErrorInvalidConfiguration;  // (item numbers are int32)
  window_umma_kernel<T, D, G><<<(unsigned)std::min<int64_t>(items, sms), kWinThreads, smem, s>>>(a, km, vm, qm);
  return cudaGetLastError();
}

template <typename T, int D>
static cudaError_t launch_win_d(const AttnArgs& a, const CUtensorMap& km, const CUtensorMap& vm, cudaStream_t s) {
  switch (a.group) {
    case 1: return launch_win_g<T, D, 1>(a, km, vm, s);
    case 2: return launch_win_g<T, D, 2>(a, km, vm, s);
    case 4: return launch_win_g<T, D, 4>(a, km, vm, s);
    case 8: return launch_win_g<T, D, 8>(a, km, vm, s);
    case 16: return launch_win_g<T, D, 16>(a, km, vm, s);
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t launch_window_umma(const AttnArgs& a, pa_dtype dt, cudaStream_t s, int* launches) {
  if (a.rows == 0) return cudaSuccess;
  CUtensorMap km, vm;
  if (!encode_pool_map(&km, a.k_pool, dt, a.num_blocks, a.block_size, a.n_kv_heads, a.head_dim, a.kv_block_stride) ||
      !encode_pool_map(&vm, a.v_pool, dt, a.num_blocks, a.block_size, a.n_kv_heads, a.head_dim, a.kv_block_stride))
    return cudaErrorInvalidValue;
  cudaError_t e;
  if (dt == PA_BF16)
    e = a.head_dim == 64 ? launch_win_d<__nv_bfloat16, 64>(a, km, vm, s) : launch_win_d<__nv_bfloat16, 128>(a, km, vm, s);
  else
    e = a.head_dim == 64 ? launch_win_d<__half, 64>(a, km, vm, s) : launch_win_d<__half, 128>(a, km, vm, s);
  ++*launches;
  return e;
}

}  // namespace pa
