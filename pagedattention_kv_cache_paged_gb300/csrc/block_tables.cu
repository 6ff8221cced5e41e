// build_block_tables: a step's index arrays from the requests' lengths, one launch.
//
// With exclusive sums over the batch, q_b of the new tokens and f_b of the blocks to take
// (need_b = max(0, ceil((h_b + m_b) / S) - c_b)), everything is a function of one token: token j of
// sequence b sits at position p = h_b + j, in table entry k = p / S, which is the row's own when
// k < c_b and else the free list's entry count - 1 - (f_b + k - c_b).  The token that opens a block
// (p % S == 0) also writes the table entry.  So the tokens are the parallel axis, whatever their
// split into sequences, and nothing waits for the table.
//
// Every CTA forms the sums itself, kBtSeqs sequences at a time, and serves the tokens of its own range
// that fall among them: reading all lengths again in each CTA costs less than a second launch.  Without
// trees a thread takes four tokens in a row: one search for their sequence, one table entry for a block's
// worth of them, 16-byte stores.  With trees it takes one: a node's mask is a walk up its ancestors, one
// dependent read each, from the range's parents in shared memory.
//
// The counts and the free list's length are read by every CTA and updated in place, so the last CTA to
// finish (a ticket in free_state[1], which returns to 0) writes them: a sequence took what its
// context_lens entry (0 if it did not fit) needs beyond its count.  A grid of one CTA does without.
//
// Bound by latency: two dependent rounds to memory (lengths, then ids), the scan between them, and the ticket.
// 64 trees of up to 16 tokens: 6.4 us.  256 trees of 60 to 128: 10.4 us, half of it the walks up the ancestors.
// 2,048 prompts, 1.1 M tokens, 13.8 MB written: 12.0 us, 1.1 TB/s; of 16,000 cycles the lengths and their sums
// take 4,700, the two rounds of search, id and stores of each thread 8,900, the ticket 2,700.
#include "pa_common.cuh"
#include "pa_internal.h"

namespace pa {

constexpr int kBtThreads = 512;
constexpr int kBtWarps = kBtThreads / 32;
constexpr int kBtPer = 4;                       // sequences a thread sums up per chunk
constexpr int kBtSeqs = kBtPer * kBtThreads;
constexpr int kBtStage = 2048;                  // parents of a CTA's range that are staged

struct BtShared {
  int32_t tok[kBtSeqs + 1];   // first token of each sequence of the chunk (saturated at the capacity + 1)
  int32_t hist[kBtSeqs];      // history; -1: the sequence does not fit
  int32_t count[kBtSeqs];     // blocks held
  int32_t take[kBtSeqs];      // blocks taken before it (of a sequence that fits)
  int64_t sums[2][kBtWarps];
  int64_t carry_tok, carry_take;
  unsigned long long served;
  int last;
};

// Inclusive sums of (a, b) over the CTA's threads, both at once (two barriers).
__device__ __forceinline__ void bt_scan(int64_t& a, int64_t& b, BtShared& sm) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int64_t u = __shfl_up_sync(0xffffffffu, a, off), v = __shfl_up_sync(0xffffffffu, b, off);
    if (lane >= off) {
      a += u;
      b += v;
    }
  }
  if (lane == 31) {
    sm.sums[0][warp] = a;
    sm.sums[1][warp] = b;
  }
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kBtWarps; ++w) {
    if (w < warp) {
      a += sm.sums[0][w];
      b += sm.sums[1][w];
    }
  }
}

struct BtSeq {
  int32_t h, m, c;
  int32_t blocks;  // of the context
  unsigned bad;
};

// What sequence b asks for, as far as that can be told from it alone.
__device__ __forceinline__ BtSeq bt_seq(const TablesArgs& a, int b) {
  BtSeq s{};
  if (b >= a.batch) return s;
  s.h = a.history_lens[b];
  s.m = a.new_lens[b];
  s.c = a.block_counts[b];
  const int64_t n = (int64_t)s.h + s.m;
  if (s.h < 0 || s.m < 0 || n > ((int64_t)a.max_blocks << a.block_shift)) s.bad |= PA_DEVERR_CONTEXT_LEN;
  const int64_t held_min = ((int64_t)(s.h < 0 ? 0 : s.h) + a.block_size - 1) >> a.block_shift;
  if (s.c < held_min || s.c > a.max_blocks) s.bad |= PA_DEVERR_BLOCK_ID;
  if (a.parents != nullptr && s.m > 64 * a.mask_words) s.bad |= PA_DEVERR_TREE;
  s.m = s.m < 0 ? 0 : s.m;
  s.blocks = s.bad ? 0 : (int32_t)((n + a.block_size - 1) >> a.block_shift);
  return s;
}

// Sequences [b0, b0 + kBtSeqs): their places into sm (carried on in sm.carry_*).  `report`: what is written
// per sequence; `update`: the counts too.
__device__ __forceinline__ void bt_chunk(const TablesArgs& a, BtShared& sm, int b0, int64_t avail, bool report,
                                         bool update) {
  const int i0 = threadIdx.x * kBtPer;
  BtSeq s[kBtPer];
  int64_t tok = 0, take = 0;
#pragma unroll
  for (int k = 0; k < kBtPer; ++k) s[k] = bt_seq(a, b0 + i0 + k);
  // a sequence whose tokens pass the capacity has no blocks to take either; those behind it have none that do
  // not, so the sums may be formed before that is known
#pragma unroll
  for (int k = 0; k < kBtPer; ++k) {
    tok += s[k].m;
    take += max(0, s[k].blocks - s[k].c);
  }
  int64_t tok_end = tok, take_end = take;
  const int64_t tok0 = sm.carry_tok, take0 = sm.carry_take;
  bt_scan(tok_end, take_end, sm);
  int64_t t = tok0 + tok_end - tok, f = take0 + take_end - take;
  const int64_t most = min(a.token_capacity + 1, (int64_t)INT32_MAX);
#pragma unroll
  for (int k = 0; k < kBtPer; ++k) {
    const int i = i0 + k, b = b0 + i;
    const int64_t need = max(0, s[k].blocks - s[k].c), end = t + s[k].m;
    unsigned bad = s[k].bad;
    if (end > a.token_capacity && s[k].m > 0) bad |= PA_DEVERR_QUERY_LOC;
    if (bad == 0 && need > 0 && f + need > avail) bad |= PA_DEVERR_NO_BLOCKS;
    sm.tok[i] = (int32_t)min(t, most);
    sm.hist[i] = bad ? -1 : s[k].h;
    sm.count[i] = s[k].c;
    sm.take[i] = (int32_t)min(f, (int64_t)INT32_MAX);
    if (report && b < a.batch) {
      if (bad) raise_error(a.err, bad);
      a.query_start_loc[b + 1] = (int32_t)min(end, (int64_t)INT32_MAX);
      a.context_lens[b] = bad ? 0 : s[k].h + s[k].m;
    }
    if (update && bad == 0 && need > 0) {
      a.block_counts[b] = s[k].blocks;
      atomicAdd(&sm.served, (unsigned long long)need);
    }
    t = end;
    f += need;
  }
  __syncthreads();  // everyone has read the carries
  if (threadIdx.x == kBtThreads - 1) {
    sm.tok[kBtSeqs] = (int32_t)min(t, most);
    sm.carry_tok = t;
    sm.carry_take = f;
  }
  __syncthreads();
}

template <bool kTree>
__global__ void __launch_bounds__(kBtThreads) block_tables_kernel(const TablesArgs a, int per_cta, bool vec) {
  constexpr int kTok = kTree ? 1 : 4;  // tokens in a row per thread
  __shared__ BtShared sm;
  __shared__ int32_t stage[kTree ? kBtStage : 1];
  const int tid = threadIdx.x;
  const bool alone = gridDim.x == 1;
  const int64_t lo = (int64_t)blockIdx.x * per_cta;
  const int64_t hi = min(lo + per_cta, a.token_capacity);
  pdl_wait_primary();
  pdl_launch_dependents();
  const int64_t count = a.free_state[0];
  if (kTree)
    for (int i = tid; i < kBtStage && lo + i < hi; i += kBtThreads) stage[i] = ld_s32(a.parents + lo + i);
  if (tid == 0) {
    sm.carry_tok = sm.carry_take = 0;
    sm.served = 0;
  }
  __syncthreads();
  const int64_t avail = count < 0 ? 0 : (count > a.free_capacity ? a.free_capacity : count);
  if (blockIdx.x == 0 && tid == 0) {
    a.query_start_loc[0] = 0;
    if (count != avail) raise_error(a.err, PA_DEVERR_NO_BLOCKS);
  }
  // parent of the node at token t
  auto parent = [&](int64_t t) -> int32_t {
    const int64_t i = t - lo;
    return i >= 0 && i < kBtStage ? stage[i] : ld_s32(a.parents + t);
  };
  for (int b0 = 0; b0 < a.batch; b0 += kBtSeqs) {
    bt_chunk(a, sm, b0, avail, blockIdx.x == 0, alone);
    const int n_seq = min(kBtSeqs, a.batch - b0);
    // (both bounds at most the capacity: tokens past it belong to sequences that do not fit)
    const int64_t t0 = max(lo, (int64_t)sm.tok[0]), t1 = min(hi, (int64_t)sm.tok[n_seq]);
    // groups of four tokens, aligned to the range's start
    for (int64_t g = t0 - (t0 - lo) % kTok + (int64_t)tid * kTok; g < t1; g += (int64_t)kBtThreads * kTok) {
      const int64_t first = max(g, t0);
      int s = 0, e = n_seq - 1;  // the last sequence of the chunk that begins at or before `first`
      while (s < e) {
        const int mid = (s + e + 1) >> 1;
        if (sm.tok[mid] <= first) s = mid; else e = mid - 1;
      }
      int64_t slots[kTok];
      int32_t pos[kTok];
      int32_t last_k = -1, id = -1, last_s = -1;
#pragma unroll
      for (int u = 0; u < kTok; ++u) {
        const int64_t t = g + u;
        slots[u] = -1;
        pos[u] = 0;
        if (t < first || t >= t1) continue;
        while (sm.tok[s + 1] <= t) ++s;  // (ends: t < t1 <= tok[n_seq])
        const int j = (int)(t - sm.tok[s]);
        const int32_t h = sm.hist[s];
        if (h >= 0) {
          const int32_t p = h + j, k = p >> a.block_shift;
          if (s != last_s || k != last_k) {
            const int32_t c = sm.count[s];
            int32_t* entry = a.block_table + (int64_t)(b0 + s) * a.bt_stride + k;
            if (k < c) {
              id = *entry;
              if (id < 0 || id >= a.num_blocks) id = -1;
            } else {
              id = a.free_blocks[avail - 1 - (sm.take[s] + k - c)];
              if (id < 0 || id >= a.num_blocks) id = -1;
              if ((p & (a.block_size - 1)) == 0) *entry = id;
            }
            if (id < 0) raise_error(a.err, PA_DEVERR_BLOCK_ID);
            last_s = s;
            last_k = k;
          }
          if (id >= 0) slots[u] = ((int64_t)id << a.block_shift) + (p & (a.block_size - 1));
          pos[u] = p;
        }
        if (kTree) {
          int64_t* row = a.tree_mask + t * a.mask_words;
          int word = a.mask_words - 1, depth = 0;
          uint64_t bits = 0;
          // the chain of ancestors runs downward, so each mask word is finished before the next
          for (int up = h >= 0 ? j : -1; up >= 0;) {
            for (; word > (up >> 6); --word, bits = 0) row[word] = (int64_t)bits;
            bits |= 1ull << (up & 63);
            const int32_t next = parent(t - j + up);
            if (next < -1 || next >= up) {
              if (up == j) raise_error(a.err, PA_DEVERR_TREE);
              break;
            }
            if (next < 0) break;
            up = next;
            ++depth;
          }
          for (; word >= 0; --word, bits = 0) row[word] = (int64_t)bits;
          if (h >= 0) pos[u] = h + depth;
        }
      }
      if (!kTree && vec && g >= t0 && g + kTok <= t1) {
        *reinterpret_cast<int4*>(a.positions + g) = make_int4(pos[0], pos[1 % kTok], pos[2 % kTok], pos[3 % kTok]);
        *reinterpret_cast<longlong2*>(a.slot_mapping + g) = make_longlong2(slots[0], slots[1 % kTok]);
        *reinterpret_cast<longlong2*>(a.slot_mapping + g + 2) = make_longlong2(slots[2 % kTok], slots[3 % kTok]);
      } else {
#pragma unroll
        for (int u = 0; u < kTok; ++u) {
          if (g + u < first || g + u >= t1) continue;
          a.slot_mapping[g + u] = slots[u];
          a.positions[g + u] = pos[u];
        }
      }
    }
    // nothing of this CTA's range lies in the later chunks (the first CTA goes on: it reports them)
    if (blockIdx.x != 0 && sm.carry_tok >= hi && b0 + kBtSeqs < a.batch) break;
    __syncthreads();
  }
  // behind the last sequence's tokens (a CTA that left the loop early has none there)
  for (int64_t t = max(lo, min(sm.carry_tok, hi)) + tid; t < hi; t += kBtThreads) {
    a.slot_mapping[t] = -1;
    a.positions[t] = 0;
    if (kTree)
      for (int w = 0; w < a.mask_words; ++w) a.tree_mask[t * a.mask_words + w] = 0;
  }
  if (!alone) {
    __syncthreads();
    if (tid == 0) {
      __threadfence();
      sm.last = atomicAdd(a.free_state + 1, 1) == (int)gridDim.x - 1;
      __threadfence();
    }
    __syncthreads();
    if (!sm.last) return;
    int64_t took = 0;
    const bool here = a.batch <= kBtSeqs;  // all sequences are still in shared memory
    for (int b = tid; b < a.batch; b += kBtThreads) {
      const int32_t n = here ? (sm.hist[b] < 0 ? 0 : sm.hist[b] + sm.tok[b + 1] - sm.tok[b]) : __ldcg(a.context_lens + b);
      const int32_t c = here ? sm.count[b] : a.block_counts[b];
      const int32_t blocks = (int32_t)(((int64_t)n + a.block_size - 1) >> a.block_shift);
      if (n > 0 && blocks > c) {
        a.block_counts[b] = blocks;
        took += blocks - c;
      }
    }
    if (took > 0) atomicAdd(&sm.served, (unsigned long long)took);
  }
  __syncthreads();
  if (tid == 0) {
    a.free_state[0] = (int32_t)(avail - (int64_t)sm.served);
    if (!alone) a.free_state[1] = 0;
  }
}

cudaError_t launch_block_tables(const TablesArgs& a, int sms, cudaStream_t s, int* launches) {
  // One CTA while its threads have a group of four tokens each (with trees one); then as many CTAs as keep
  // that up, two per SM at most, in whole groups.
  const bool tree = a.parents != nullptr;
  const int64_t share = tree ? kBtThreads : 4 * kBtThreads;
  int64_t ctas = (a.token_capacity + share - 1) / share;
  ctas = ctas < 1 ? 1 : (ctas > 2 * sms ? 2 * sms : ctas);
  const int64_t per_cta = ((a.token_capacity + ctas - 1) / ctas + 3) / 4 * 4;
  const bool vec = ((reinterpret_cast<uintptr_t>(a.slot_mapping) | reinterpret_cast<uintptr_t>(a.positions)) & 15u) == 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(kBtThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  ++*launches;
  return tree ? cudaLaunchKernelEx(&cfg, block_tables_kernel<true>, a, (int)per_cta, vec)
              : cudaLaunchKernelEx(&cfg, block_tables_kernel<false>, a, (int)per_cta, vec);
}

}  // namespace pa
