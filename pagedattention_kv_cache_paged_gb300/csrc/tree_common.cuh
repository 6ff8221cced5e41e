// What the tree-attention kernels share: a sequence's rows and lengths.
#pragma once

#include "pa_common.cuh"
#include "pa_internal.h"

namespace pa {

// The rows and lengths of sequence b, or n = 0 and an error bit when they do not fit together.
struct TreeSeq {
  int64_t q0;  // first row (refused: the first among the call's)
  int m;       // nodes; of a refused sequence the rows that it has among the call's, all of which become zeros
  int n;       // context length; 0 when the sequence is refused
  unsigned bad;
};

__device__ __forceinline__ TreeSeq tree_seq(const TreeArgs& a, int b) {
  TreeSeq s{};
  const int q0 = ld_s32(a.query_start_loc + b), q1 = ld_s32(a.query_start_loc + b + 1);
  s.n = ld_s32(a.context_lens + b);
  s.q0 = q0;
  if (q0 < 0 || q1 < q0 || q1 > a.total_q) {
    s.bad = PA_DEVERR_QUERY_LOC;
  } else {
    s.m = q1 - q0;
    if (s.m > a.max_nodes || s.n < s.m) s.bad |= PA_DEVERR_QUERY_LOC;
    if (a.tree_mask != nullptr && s.m > 64 * a.mask_words) s.bad |= PA_DEVERR_TREE;
    if ((unsigned)s.n > (unsigned)a.max_context) s.bad |= PA_DEVERR_CONTEXT_LEN;
  }
  if (s.bad) {
    s.n = 0;
    s.q0 = max(q0, 0);
    s.m = (int)max(min((int64_t)q1, a.total_q) - s.q0, (int64_t)0);
  }
  return s;
}

// ------------------------------------------------------------------------------------------------
// Division of the tensor-core kernel's work among its CTAs.
//
// A unit is (sequence, KV head, tile of its nodes); its key tiles are read in order.  All units in a
// row (sequences, then KV heads, then node tiles) make one line of key tiles, each unit followed by a gap
// for what it costs besides its keys, and CTA c takes positions [c * share, (c + 1) * share) of the line:
// every CTA streams the same bytes whatever the lengths, and only the units that a cut falls into have to
// be joined afterwards.  A cut closer than `snap` tiles to a unit's border moves to it.
struct TreeSpan {
  int b0, u0, x0;  // first sequence, unit of it, tile of that
  int b1, u1, x1;  // end (exclusive); b1 = batch: the end of the line
};

// Tile of a unit of T tiles at which a cut at position x of the unit (its gap included) is made.
__device__ __forceinline__ int tree_cut(int64_t x, int T, int snap) {
  if (x >= T) return T;
  const int d = (int)x, e = T - (int)x;
  if (d <= e) return d < snap ? 0 : d;
  return e < snap ? T : (int)x;
}

// The units of a CTA's span one after the other.  Every role of the CTA walks on its own: the lengths
// come from L1, and nothing has to be handed over.
struct TreeUnit {
  TreeSeq sq;
  int b, kvh, node0, rows;  // rows: (node, head) rows that exist
  int T, x0, x1;            // key tiles of the unit, and those of this CTA
  bool last_tile;           // no later node tile reads the same keys
};

template <int kKeys>
struct TreeWalk {
  const TreeArgs& a;
  const TreeSpan span;
  const int nodes_unit;
  int b, u, x;
  TreeSeq sq;

  __device__ __forceinline__ TreeWalk(const TreeArgs& args, const TreeSpan& s, int nodes)
      : a(args), span(s), nodes_unit(nodes), b(s.b0), u(s.u0), x(s.x0) {
    if (b < a.batch) sq = tree_seq(a, b);
  }
  __device__ __forceinline__ bool next(TreeUnit& w) {
    for (;;) {
      if (b >= a.batch || b > span.b1 || (b == span.b1 && u > span.u1)) return false;
      const int q_tiles = sq.n == 0 ? 0 : (sq.m + nodes_unit - 1) / nodes_unit;
      if (u >= q_tiles * a.n_kv_heads) {
        ++b;
        u = x = 0;
        if (b < a.batch) sq = tree_seq(a, b);
        continue;
      }
      const int qt = u % q_tiles;
      w.sq = sq;
      w.b = b;
      w.kvh = u / q_tiles;
      w.node0 = qt * nodes_unit;
      w.rows = min(nodes_unit, sq.m - w.node0) << a.group_shift;
      w.T = (sq.n + kKeys - 1) / kKeys;
      w.x0 = x;
      w.x1 = b == span.b1 && u == span.u1 ? span.x1 : w.T;
      w.last_tile = qt == q_tiles - 1;
      ++u;
      x = 0;
      if (w.x0 < w.x1) return true;
    }
  }
};

// Where a CTA's span of the line begins and ends.
struct TreeSched {
  int32_t sums[16];  // per warp
  int32_t tops[16];
  int32_t share;
  int32_t cut_start;  // where the unit that the span ends in begins on the line
  int32_t snap;
  TreeSpan span;
  int32_t refused;    // a sequence of the batch is refused, and its rows are this CTA's to zero
};

__device__ __forceinline__ void tree_schedule_init(const TreeArgs& a, TreeSched& sm) {
  sm.span = TreeSpan{a.batch, 0, 0, a.batch, 0, 0};
  sm.refused = 0;
}

// All threads; sm initialised, and a barrier since.  The caller's next barrier publishes the result.  One
// thread looks after one sequence at a time; positions on the line fit 32 bits (the host sees to it).
template <int kThreads, int kKeys, int kGap, int kMinShare>
__device__ __forceinline__ void tree_schedule(const TreeArgs& a, int nodes_unit, TreeSched& sm) {
  constexpr int kWarps = kThreads / 32, kSnap = kGap - 1;
  static_assert(kWarps <= 16, "sums per warp");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int gap = a.share > 0 ? 0 : kGap;
  int tiles = 0;
  auto look = [&](int b) -> int {  // this thread's sequence: its length on the line
    tiles = 0;
    if (b >= a.batch) return 0;
    const TreeSeq s = tree_seq(a, b);
    if (s.bad) {
      if (blockIdx.x == 0) raise_error(a.err, s.bad);
      if (s.m > 0 && b % gridDim.x == blockIdx.x) sm.refused = 1;
    }
    if (s.n == 0 || s.m == 0) return 0;
    tiles = (s.n + kKeys - 1) / kKeys;
    return (s.m + nodes_unit - 1) / nodes_unit * a.n_kv_heads * (tiles + gap);
  };
  const bool one_chunk = a.batch <= kThreads;
  int c = look(threadIdx.x);
  int total = c, longest = c > 0 ? tiles + gap : 0;
  for (int b = threadIdx.x + kThreads; b < a.batch; b += kThreads) {
    const int more = look(b);
    total += more;
    longest = max(longest, more > 0 ? tiles + gap : 0);
  }
  auto scan = [&](int x) {  // inclusive, over the warp
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, x, off);
      if (lane >= off) x += u;
    }
    return x;
  };
  int v = one_chunk ? scan(c) : 0;
  const int warp_total = one_chunk ? v : __reduce_add_sync(0xffffffffu, total);  // (in lane 31)
  const int warp_top = __reduce_max_sync(0xffffffffu, longest);
  if (lane == 31) {
    sm.sums[warp] = warp_total;
    sm.tops[warp] = warp_top;
  }
  __syncthreads();
  int pre = 0;
  total = longest = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const int x = sm.sums[w];
    if (w < warp) pre += x;
    total += x;
    longest = max(longest, sm.tops[w]);
  }
  int share = a.share;
  if (share <= 0) {
    // fewer tiles than kMinShare would wait longer for their first keys than they save
    share = (int)(((unsigned)total + gridDim.x - 1) / gridDim.x);
    share = max(share, min(longest, kMinShare));
  }
  // contexts that are never cut: every border moves to the nearest unit's
  const int snap = !a.split || longest <= (a.share > 0 ? 0 : kMinShare) ? INT32_MAX : (a.share > 0 ? 1 : kSnap);
  const int64_t lo = (int64_t)blockIdx.x * share, hi = lo + share;
  if (threadIdx.x == 0) {
    sm.share = share;
    sm.snap = snap;
  }
  // this thread's sequence b lies at [first, first + c) of the line
  auto place = [&](int b, int64_t first) {
    const unsigned len = (unsigned)(tiles + gap);
    if (c > 0 && lo >= first && lo < first + c) {
      const unsigned off = (unsigned)(lo - first), u = off / len;
      sm.span.b0 = b;
      sm.span.u0 = (int)u;
      sm.span.x0 = tree_cut(off - u * len, tiles, snap);
      // the producers' first table entries
      const int pos = min(sm.span.x0, tiles - 1) * kKeys;
      asm volatile("prefetch.global.L1 [%0];" ::"l"(a.block_table + (int64_t)b * a.bt_stride + (pos >> a.block_shift)));
    }
    if (c > 0 && hi >= first && hi < first + c) {
      const unsigned off = (unsigned)(hi - first), u = off / len;
      sm.span.b1 = b;
      sm.span.u1 = (int)u;
      sm.span.x1 = tree_cut(off - u * len, tiles, snap);
      sm.cut_start = (int)(hi - (off - u * len));
    }
  };
  if (one_chunk) {
    place(threadIdx.x, (int64_t)pre + v - c);
    return;
  }
  int carry = 0;
  for (int b0 = 0; b0 < a.batch; b0 += kThreads) {
    c = look(b0 + threadIdx.x);
    v = scan(c);
    __syncthreads();  // the sums before have been read
    if (lane == 31) sm.sums[warp] = v;
    __syncthreads();
    pre = carry;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) pre += sm.sums[w];
      carry += sm.sums[w];
    }
    place(b0 + threadIdx.x, (int64_t)pre + v - c);
  }
}

// Zeros for the sequences whose lengths do not fit together (those that fall to this CTA).
template <typename T>
__device__ __forceinline__ void tree_zero_refused(const TreeArgs& a) {
  for (int b = blockIdx.x; b < a.batch; b += gridDim.x) {
    const TreeSeq s = tree_seq(a, b);
    if (s.n != 0 || s.bad == 0) continue;
    uint4* o = reinterpret_cast<uint4*>(static_cast<T*>(a.out) + s.q0 * a.n_q_heads * a.head_dim);
    const int64_t n = (int64_t)s.m * a.n_q_heads * a.head_dim * sizeof(T) / 16;
    for (int64_t i = threadIdx.x; i < n; i += blockDim.x) o[i] = make_uint4(0, 0, 0, 0);
  }
}

// The record of a unit that starts in this CTA and ends in a later one (one thread).
__device__ __forceinline__ void tree_record(const TreeArgs& a, const TreeSched& sm, const TreeUnit& w, int64_t row0,
                                            TreeRec* rec) {
  // the CTA that the unit's last tile went to
  int last = (sm.cut_start + w.T - 1) / sm.share;
  if (tree_cut((int64_t)last * sm.share - sm.cut_start, w.T, sm.snap) == w.T) --last;
  *rec = TreeRec{row0, w.rows, last};
}

// Whether a row (the mask words of its node, or nullptr and the node of a chain) sees node s.
__device__ __forceinline__ bool tree_sees(const int64_t* words, int node, int s) {
  return words != nullptr ? ((ld_s64(words + (s >> 6)) >> (s & 63)) & 1) != 0 : s <= node;
}

}  // namespace pa
