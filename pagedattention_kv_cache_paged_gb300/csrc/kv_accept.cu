// paged_kv_accept: the K/V rows of the accepted drafted tokens move to the end of the history, in
// every layer, one launch.
//
// Entry i of a sequence's list moves row h + idx[i] to row h + i with idx[i] >= i.  Both ends lie in
// the drafted region, and a row may be the source of one entry and the destination of a later one
// (idx[0] = 1, idx[1] = 2), never of an earlier one: a destination i is read by a later entry j > i
// only if idx[j] = i < j.  So one thread that owns a 16-byte column of the rows may load a batch of
// entries, then store it, and go on to the next batch: no other thread touches its column.  Memory
// bound: every row is read once and written once.
#include "pa_common.cuh"
#include "pa_internal.h"

namespace pa {

constexpr int kAccThreads = 256;
constexpr int kAccList = 64;   // entries whose rows are looked up at a time
constexpr int kAccBatch = 8;   // rows in flight per thread

__global__ void __launch_bounds__(kAccThreads) kv_accept_kernel(const AcceptArgs a) {
  __shared__ int64_t s_src[kAccList], s_dst[kAccList];
  const int b = blockIdx.x % a.batch;
  const int layer = blockIdx.x / a.batch;
  const int tid = threadIdx.x;
  int n = a.accepted_lens[b];
  if (n < 0 || n > a.max_accepted) {
    if (tid == 0) raise_error(a.err, PA_DEVERR_QUERY_LOC);
    n = n < 0 ? 0 : a.max_accepted;
  }
  const int64_t h = a.history_lens[b];
  const int64_t cap = a.bt_stride * a.block_size;
  const int32_t* table = a.block_table + (int64_t)b * a.bt_stride;
  uint4* const kp = static_cast<uint4*>(a.k_pool) + layer * a.layer_stride_vecs;
  uint4* const vp = static_cast<uint4*>(a.v_pool) + layer * a.layer_stride_vecs;
  for (int i0 = 0; i0 < n; i0 += kAccList) {
    const int cnt = min(kAccList, n - i0);
    __syncthreads();
    if (tid < cnt) {
      const int i = i0 + tid;
      const int32_t idx = a.accepted[(int64_t)b * a.accepted_stride + i];
      int64_t src = -1, dst = -1;
      unsigned bad = 0;
      if (idx < i) {
        bad = PA_DEVERR_TREE;
      } else if (h < 0 || h + idx >= cap) {
        bad = PA_DEVERR_CONTEXT_LEN;
      } else if (idx != i) {
        const int64_t ps = h + idx, pd = h + i;
        const int32_t bs = table[ps / a.block_size], bd = table[pd / a.block_size];
        if (bs < 0 || bs >= a.num_blocks || bd < 0 || bd >= a.num_blocks) {
          bad = PA_DEVERR_BLOCK_ID;
        } else {
          src = bs * a.block_stride_vecs + (ps % a.block_size) * a.row_vecs;
          dst = bd * a.block_stride_vecs + (pd % a.block_size) * a.row_vecs;
        }
      }
      if (bad) raise_error(a.err, bad);
      s_src[tid] = src;
      s_dst[tid] = dst;
    }
    __syncthreads();
    for (int c = tid; c < 2 * a.row_vecs; c += kAccThreads) {
      uint4* const pool = (c < a.row_vecs ? kp : vp) + (c < a.row_vecs ? c : c - a.row_vecs);
      for (int j0 = 0; j0 < cnt; j0 += kAccBatch) {
        uint4 r[kAccBatch];
#pragma unroll
        for (int u = 0; u < kAccBatch; ++u)
          if (j0 + u < cnt && s_src[j0 + u] >= 0) r[u] = pool[s_src[j0 + u]];
#pragma unroll
        for (int u = 0; u < kAccBatch; ++u)
          if (j0 + u < cnt && s_src[j0 + u] >= 0) pool[s_dst[j0 + u]] = r[u];
      }
    }
  }
}

cudaError_t launch_kv_accept(const AcceptArgs& a, cudaStream_t s, int* launches) {
  const int64_t grid = (int64_t)a.batch * a.num_layers;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  kv_accept_kernel<<<(unsigned)grid, kAccThreads, 0, s>>>(a);
  ++*launches;
  return cudaGetLastError();
}

}  // namespace pa
