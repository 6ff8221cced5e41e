// What the tree-attention kernels share: a sequence's rows and lengths.
#pragma once

#include "pa_common.cuh"
#include "pa_internal.h"

namespace pa {

// The rows and lengths of sequence b, or n = 0 and an error bit when they do not fit together.
struct TreeSeq {
  int64_t q0;
  int m;      // nodes (0: no rows of this sequence are written)
  int n;      // context length; 0 when the sequence is refused
  unsigned bad;
};

__device__ __forceinline__ TreeSeq tree_seq(const TreeArgs& a, int b) {
  TreeSeq s{};
  const int64_t q0 = __ldg(a.query_start_loc + b), q1 = __ldg(a.query_start_loc + b + 1);
  s.n = __ldg(a.context_lens + b);
  s.q0 = q0;
  if (q0 < 0 || q1 < q0 || q1 > a.total_q) {
    s.bad = PA_DEVERR_QUERY_LOC;
    s.n = 0;
    return s;
  }
  s.m = (int)min(q1 - q0, (int64_t)a.max_nodes);
  if (q1 - q0 > a.max_nodes || s.n < q1 - q0) s.bad |= PA_DEVERR_QUERY_LOC;
  if (a.tree_mask != nullptr && q1 - q0 > (int64_t)64 * a.mask_words) s.bad |= PA_DEVERR_TREE;
  if (s.n < 0 || s.n > (a.bt_stride << a.block_shift)) s.bad |= PA_DEVERR_CONTEXT_LEN;
  if (s.bad) s.n = 0;
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

}  // namespace pa
