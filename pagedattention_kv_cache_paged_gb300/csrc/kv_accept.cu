// paged_kv_accept: the K/V rows of the accepted drafted tokens move to the end of the history, in
// every layer, one launch.
//
// Entry i of a sequence's list moves row h + idx[i] to row h + i with idx[i] >= i.  Both ends lie in
// the drafted region, and a row may be the source of one entry and the destination of a later one
// (idx[0] = 1, idx[1] = 2), never of an earlier one: a destination i is read by a later entry j > i
// only if idx[j] = i < j.  So one thread that owns a 16-byte column of a layer's rows may load a batch
// of entries, then store it, and go on to the next batch: no other thread touches its column.  Every
// row that moves is read once and written once.  288 rows of 2 KB, K and V, in 32 layers, of which 261
// move (68 MB): 14.3 us in calls that take turns over eight batches' pools, so that the rows come from DRAM and go
// back there (4.8 TB/s, 0.71 of the copy rate), 9.7 us over one batch's, which stay in L2.  Bound by the chain of a CTA
// (list, table, row, store), one wave behind the other, and by DRAM on top of it; three rows in one layer take
// 2.4 us.  Eight rows in flight at four CTAs per SM: four at eight CTAs 15.8 us.
#include <algorithm>

#include "pa_common.cuh"
#include "pa_internal.h"

namespace pa {

constexpr int kAccThreads = 256;
constexpr int kAccCtas = 4;    // per SM
constexpr int kAccBatch = 8;   // rows in flight per thread

__global__ void __launch_bounds__(kAccThreads, kAccCtas) kv_accept_kernel(const AcceptArgs a, const int layers_cta) {
  __shared__ int64_t s_src[32], s_dst[32];
  __shared__ int s_count;
  const int b = blockIdx.x % a.batch;
  const int l0 = blockIdx.x / a.batch * layers_cta;
  const int layers = min(layers_cta, a.num_layers - l0);
  const int tid = threadIdx.x;
  const int cols = 2 * a.row_vecs;
  const int lanes = max(kAccThreads / cols, 1);  // narrow rows: several layers side by side
  const int lane = cols < kAccThreads ? tid / cols : 0;
  const int32_t* list = a.accepted + b * a.accepted_stride;
  const int64_t h = a.history_lens[b];
  // the first entries are read along with their number
  int32_t idx = tid < 32 && tid < a.max_accepted ? list[tid] : 0;
  int n = a.accepted_lens[b];
  if (n < 0 || n > a.max_accepted) {
    if (tid == 0) raise_error(a.err, PA_DEVERR_QUERY_LOC);
    n = n < 0 ? 0 : a.max_accepted;
  }
  const int64_t cap = a.bt_stride * a.block_size;
  const int32_t* table = a.block_table + b * a.bt_stride;
  for (int i0 = 0; i0 < n; i0 += 32) {
    if (i0) __syncthreads();
    if (tid < 32) {
      const int i = i0 + tid;
      if (i0) idx = i < n ? list[i] : 0;
      int64_t src = -1, dst = -1;
      if (i < n) {
        unsigned bad = 0;
        const int64_t ps = h + idx, pd = h + i;
        if (idx < i) {
          bad = PA_DEVERR_TREE;
        } else if (h < 0 || ps >= cap) {
          bad = PA_DEVERR_CONTEXT_LEN;
        } else if (idx != i) {
          const int32_t bs = table[ps / a.block_size], bd = table[pd / a.block_size];
          if (bs < 0 || bs >= a.num_blocks || bd < 0 || bd >= a.num_blocks) {
            bad = PA_DEVERR_BLOCK_ID;
          } else {
            src = bs * a.block_stride_vecs + (ps % a.block_size) * a.row_vecs;
            dst = bd * a.block_stride_vecs + (pd % a.block_size) * a.row_vecs;
          }
        }
        if (bad) raise_error(a.err, bad);
      }
      const unsigned moves = __ballot_sync(0xffffffffu, src >= 0);
      if (src >= 0) {
        const int at = __popc(moves & ((1u << tid) - 1));
        s_src[at] = src;
        s_dst[at] = dst;
      }
      if (tid == 0) s_count = __popc(moves);
    }
    __syncthreads();
    const int cnt = s_count;
    if (cnt == 0 || lane >= lanes) continue;
    for (int c = tid - lane * cols; c < cols; c += kAccThreads) {
      uint4* pool = static_cast<uint4*>(c < a.row_vecs ? a.k_pool : a.v_pool) + (c < a.row_vecs ? c : c - a.row_vecs) +
                    (l0 + lane) * a.layer_stride_vecs;
      const int64_t step = lanes * a.layer_stride_vecs;
      for (int l = lane; l < layers; l += lanes, pool += step) {
        for (int j0 = 0; j0 < cnt; j0 += kAccBatch) {
          uint4 r[kAccBatch];
#pragma unroll
          for (int u = 0; u < kAccBatch; ++u)
            if (j0 + u < cnt) r[u] = pool[s_src[j0 + u]];
#pragma unroll
          for (int u = 0; u < kAccBatch; ++u)
            if (j0 + u < cnt) pool[s_dst[j0 + u]] = r[u];
        }
      }
    }
  }
}

cudaError_t launch_kv_accept(const AcceptArgs& a, int sms, cudaStream_t s, int* launches) {
  // Layers of a sequence divided among its CTAs for two waves of CTAs: a CTA looks its rows up once, and the
  // second wave evens out lists of different lengths.  64 sequences x 32 layers: 14.3 us; one wave 14.8,
  // a CTA per layer 14.8.
  const int per_seq = std::max(1, std::min(a.num_layers, 2 * sms * kAccCtas / a.batch));
  const int layers_cta = (a.num_layers + per_seq - 1) / per_seq;
  const int64_t grid = (int64_t)a.batch * ((a.num_layers + layers_cta - 1) / layers_cta);
  if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  kv_accept_kernel<<<(unsigned)grid, kAccThreads, 0, s>>>(a, layers_cta);
  ++*launches;
  return cudaGetLastError();
}

}  // namespace pa
