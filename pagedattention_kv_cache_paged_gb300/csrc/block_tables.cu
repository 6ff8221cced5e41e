// build_block_tables: a step's index arrays from the requests' lengths, one launch.
//
// With exclusive sums over the batch, q_b of the new tokens and f_b of the blocks to take
// (need_b = max(0, ceil((h_b + m_b) / S) - c_b)), everything is a function of one token: token j of
// sequence b sits at position p = h_b + j, in table entry k = p / S, which is the row's own when
// k < c_b and else the free list's entry count - 1 - (f_b + k - c_b).  The token that opens a block
// (p % S == 0) also writes the table entry.  So the tokens are the parallel axis, whatever their
// split into sequences, and nothing waits for the table.
//
// Every CTA forms the sums itself, a chunk of kSeqs sequences at a time (two block scans), and
// serves the tokens of its own range that fall into the chunk: reading all lengths again in each CTA
// costs less than a second launch.  The counts and the free list's length are read by every CTA and
// updated in place, so the last CTA to finish (a ticket in free_state[1], which returns to 0) writes
// them; a grid of one CTA writes them as it goes.
#include "pa_common.cuh"
#include "pa_internal.h"

namespace pa {

constexpr int kBtThreads = 1024;
constexpr int kBtWarps = kBtThreads / 32;

struct BtChunk {
  int64_t tok[kBtThreads + 1];    // first token of each sequence of the chunk
  int32_t hist[kBtThreads];       // history; -1: the sequence does not fit
  int32_t count[kBtThreads];      // blocks held
  int64_t take[kBtThreads];       // blocks taken before it
  int64_t scan[2][kBtWarps];
  int64_t carry_tok, carry_take, served;
  int last;
};

// Inclusive sum of v over the CTA's threads in front of and including this one.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* warp_sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int64_t u = __shfl_up_sync(0xffffffffu, v, off);
    if (lane >= off) v += u;
  }
  if (lane == 31) warp_sums[warp] = v;
  __syncthreads();
  if (warp == 0) {
    int64_t w = warp_sums[lane];
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int64_t u = __shfl_up_sync(0xffffffffu, w, off);
      if (lane >= off) w += u;
    }
    warp_sums[lane] = w;
  }
  __syncthreads();
  return warp > 0 ? v + warp_sums[warp - 1] : v;
}

// One chunk of sequences from b0 on: their sums into sm (carried on in sm.carry_*).  `report` records
// what does not fit; `update` writes the counts back.
__device__ __forceinline__ void bt_chunk(const TablesArgs& a, BtChunk& sm, int b0, int64_t avail, bool report,
                                         bool update) {
  const int i = threadIdx.x, b = b0 + i;
  const bool have = b < a.batch;
  int32_t h = have ? a.history_lens[b] : 0;
  int32_t m = have ? a.new_lens[b] : 0;
  const int32_t c = have ? a.block_counts[b] : 0;
  unsigned bad = 0;
  if (h < 0 || m < 0) bad |= PA_DEVERR_CONTEXT_LEN;
  const int64_t n = (int64_t)h + m;
  const int64_t cap = (int64_t)a.max_blocks << a.block_shift;
  if (n > cap) bad |= PA_DEVERR_CONTEXT_LEN;
  m = m < 0 ? 0 : m;
  const int64_t held_min = ((int64_t)(h < 0 ? 0 : h) + a.block_size - 1) >> a.block_shift;
  if (c < held_min || c > a.max_blocks) bad |= PA_DEVERR_BLOCK_ID;
  if (a.parents != nullptr && m > 64 * a.mask_words) bad |= PA_DEVERR_TREE;
  const int64_t tok0 = sm.carry_tok, take0 = sm.carry_take;
  const int64_t tok_end = tok0 + block_scan(m, sm.scan[0]);
  if (tok_end > a.token_capacity && m > 0) bad |= PA_DEVERR_QUERY_LOC;
  const int64_t blocks = (n + a.block_size - 1) >> a.block_shift;
  const int64_t need = bad == 0 && blocks > c ? blocks - c : 0;
  const int64_t take_end = take0 + block_scan(need, sm.scan[1]);
  if (need > 0 && take_end > avail) bad |= PA_DEVERR_NO_BLOCKS;
  if (have) {
    sm.tok[i] = tok_end - m;
    sm.hist[i] = bad ? -1 : h;
    sm.count[i] = c;
    sm.take[i] = take_end - need;
    if (report) {
      if (bad) raise_error(a.err, bad);
      a.query_start_loc[b + 1] = (int32_t)(tok_end < INT32_MAX ? tok_end : INT32_MAX);
      a.context_lens[b] = bad ? 0 : (int32_t)n;
    }
    if (update && need > 0 && bad == 0) {
      a.block_counts[b] = (int32_t)blocks;
      atomicMax(reinterpret_cast<unsigned long long*>(&sm.served), (unsigned long long)take_end);
    }
  }
  const int last = min(kBtThreads, a.batch - b0) - 1;
  __syncthreads();  // everyone has read the carries
  if (i == last) {
    sm.tok[last + 1] = tok_end;
    sm.carry_tok = tok_end;
    sm.carry_take = take_end;
  }
  __syncthreads();
}

__global__ void __launch_bounds__(kBtThreads) block_tables_kernel(const TablesArgs a, int64_t per_cta) {
  __shared__ BtChunk sm;
  const int tid = threadIdx.x;
  const bool alone = gridDim.x == 1;
  const int64_t count = a.free_state[0];
  const int64_t avail = count < 0 ? 0 : (count > a.free_capacity ? a.free_capacity : count);
  if (tid == 0) {
    sm.carry_tok = sm.carry_take = sm.served = 0;
    if (blockIdx.x == 0) {
      a.query_start_loc[0] = 0;
      if (count != avail) raise_error(a.err, PA_DEVERR_NO_BLOCKS);
    }
  }
  __syncthreads();
  const int64_t lo = (int64_t)blockIdx.x * per_cta;
  const int64_t hi = min(lo + per_cta, a.token_capacity);
  for (int b0 = 0; b0 < a.batch; b0 += kBtThreads) {
    bt_chunk(a, sm, b0, avail, blockIdx.x == 0, alone);
    const int n_seq = min(kBtThreads, a.batch - b0);
    const int64_t t0 = max(lo, sm.tok[0]), t1 = min(hi, sm.tok[n_seq]);
    for (int64_t t = t0 + tid; t < t1; t += kBtThreads) {
      int s = 0, e = n_seq - 1;  // the last sequence of the chunk that begins at or before t and has tokens
      while (s < e) {
        const int mid = (s + e + 1) >> 1;
        if (sm.tok[mid] <= t) s = mid; else e = mid - 1;
      }
      const int b = b0 + s;
      const int j = (int)(t - sm.tok[s]);
      const int32_t h = sm.hist[s];
      int64_t slot = -1;
      int32_t pos = 0;
      if (h >= 0) {
        const int32_t p = h + j;
        const int32_t k = p >> a.block_shift;
        const int32_t c = sm.count[s];
        int32_t* entry = a.block_table + (int64_t)b * a.bt_stride + k;
        int32_t id;
        if (k < c) {
          id = *entry;
        } else {
          id = a.free_blocks[avail - 1 - (sm.take[s] + k - c)];
          if (id < 0 || id >= a.num_blocks) id = -1;
          if ((p & (a.block_size - 1)) == 0) *entry = id;
        }
        if (id >= 0 && id < a.num_blocks)
          slot = ((int64_t)id << a.block_shift) + (p & (a.block_size - 1));
        else
          raise_error(a.err, PA_DEVERR_BLOCK_ID);
        pos = p;
      }
      if (a.parents != nullptr) {
        int64_t* row = a.tree_mask + t * a.mask_words;
        const int32_t* par = a.parents + (t - j);
        int word = a.mask_words - 1, depth = 0;
        uint64_t bits = 0;
        // the chain of ancestors runs downward, so each mask word is finished before the next
        for (int up = h >= 0 ? j : -1; up >= 0; ++depth) {
          for (; word > (up >> 6); --word, bits = 0) row[word] = (int64_t)bits;
          bits |= 1ull << (up & 63);
          const int32_t next = par[up];
          if (next < -1 || next >= up) {
            if (up == j) raise_error(a.err, PA_DEVERR_TREE);
            break;
          }
          up = next;
          if (up < 0) break;
        }
        for (; word >= 0; --word, bits = 0) row[word] = (int64_t)bits;
        if (h >= 0) pos = h + depth;
      }
      a.slot_mapping[t] = slot;
      a.positions[t] = pos;
    }
    if (blockIdx.x != 0 && sm.carry_tok >= hi && b0 + kBtThreads < a.batch) {
      // nothing of this CTA's range lies in the later chunks
      break;
    }
    __syncthreads();
  }
  // behind the last sequence's tokens (a CTA that left the loop early has none there)
  for (int64_t t = max(lo, sm.carry_tok) + tid; t < hi; t += kBtThreads) {
    a.slot_mapping[t] = -1;
    a.positions[t] = 0;
    if (a.parents != nullptr)
      for (int w = 0; w < a.mask_words; ++w) a.tree_mask[t * a.mask_words + w] = 0;
  }
  if (!alone) {
    __syncthreads();
    if (tid == 0) {
      __threadfence();
      const int ticket = atomicAdd(a.free_state + 1, 1);
      sm.last = ticket == (int)gridDim.x - 1;
      __threadfence();
      sm.carry_tok = sm.carry_take = sm.served = 0;
    }
    __syncthreads();
    if (!sm.last) return;
    for (int b0 = 0; b0 < a.batch; b0 += kBtThreads) bt_chunk(a, sm, b0, avail, false, true);
  }
  __syncthreads();
  if (tid == 0) {
    a.free_state[0] = (int32_t)(avail - sm.served);
    if (!alone) a.free_state[1] = 0;
  }
}

cudaError_t launch_block_tables(const TablesArgs& a, cudaStream_t s, int* launches) {
  // one CTA up to 4096 tokens, else enough of them for 4 tokens a thread, one per SM at most
  int64_t ctas = (a.token_capacity + 4 * kBtThreads - 1) / (4 * kBtThreads);
  ctas = ctas < 1 ? 1 : (ctas > 148 ? 148 : ctas);
  const int64_t per_cta = (a.token_capacity + ctas - 1) / ctas;
  block_tables_kernel<<<(unsigned)ctas, kBtThreads, 0, s>>>(a, per_cta);
  ++*launches;
  return cudaGetLastError();
}

}  // namespace pa
