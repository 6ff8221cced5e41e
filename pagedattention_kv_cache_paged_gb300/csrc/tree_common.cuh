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

}  // namespace pa
