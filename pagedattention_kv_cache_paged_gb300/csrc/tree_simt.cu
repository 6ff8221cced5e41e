// Tree attention on CUDA cores (every dtype and shape), and the merge of split contexts.
//
// Node r of sequence b sees keys t < h_b (its history) and the nodes s = t - h_b whose bit is set in
// its mask row (a chain: s <= r).  One pass over the keys with a running maximum, sum and
// accumulator.  One CTA per (sequence, node, KV head, partition of the keys) serves the query group
// of the KV head: each warp takes kChunk keys at a time, 16-byte vectors of a K or V row per lane.
// A key that a node does not see is not loaded, so that nothing it holds can reach the sums.
//
// A partition that saw keys has a finite maximum (at least -FLT_MAX), one that saw none has -inf:
// a row whose every score is -inf is then told from a row that sees nothing (NaN, and zeros).
#include <float.h>

#include "pa_common.cuh"
#include "pa_internal.h"
#include "tree_common.cuh"

namespace pa {

constexpr int kTsWarps = 4;
constexpr int kTsUnroll = 4;

template <typename T, int D, int G>
__global__ void __launch_bounds__(kTsWarps * 32) tree_simt_kernel(const TreeArgs a) {
  constexpr int kVec = Elt<T>::kVec;
  constexpr int kLanesPerRow = D / kVec;
  constexpr int kRowsPerLoad = 32 / kLanesPerRow;
  constexpr int kChunk = kRowsPerLoad * kTsUnroll;

  __shared__ float sm_m[kTsWarps][G];
  __shared__ float sm_l[kTsWarps][G];
  __shared__ float sm_acc[kTsWarps][G][D];

  const int kvh = blockIdx.x % a.n_kv_heads;
  int64_t rest = blockIdx.x / a.n_kv_heads;
  const int part = (int)(rest % a.max_parts);
  rest /= a.max_parts;
  const int node = (int)(rest % a.max_nodes);
  const int b = (int)(rest / a.max_nodes);
  const int lane = threadIdx.x & 31;
  const int warp = threadIdx.x >> 5;
  const int dsub = lane % kLanesPerRow;
  const int rsub = lane / kLanesPerRow;

  const TreeSeq sq = tree_seq(a, b);
  if (sq.bad && threadIdx.x == 0 && node == 0 && part == 0) raise_error(a.err, sq.bad);
  if (node >= sq.m) return;
  const int n_parts = sq.n == 0 ? 1 : (sq.n + a.part_tokens - 1) / a.part_tokens;
  if (part >= n_parts) return;
  const int64_t row = sq.q0 + node;
  const int hist = sq.n - sq.m;  // a refused sequence: below 0, and no key is visited
  const int64_t t_begin = (int64_t)part * a.part_tokens;
  const int64_t t_end = min(t_begin + a.part_tokens, (int64_t)sq.n);

  const T* qrow = static_cast<const T*>(a.q) + (row * a.n_q_heads + (int64_t)kvh * G) * D;
  float qf[G][kVec];
#pragma unroll
  for (int h = 0; h < G; ++h) {
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(qrow + h * D + dsub * kVec));
    Elt<T>::unpack(v, qf[h]);
#pragma unroll
    for (int e = 0; e < kVec; ++e) qf[h][e] *= a.scale_log2;
  }
  float m[G], l[G], acc[G][kVec];
#pragma unroll
  for (int h = 0; h < G; ++h) {
    m[h] = -INFINITY;
    l[h] = 0.f;
#pragma unroll
    for (int e = 0; e < kVec; ++e) acc[h][e] = 0.f;
  }

  const int32_t* table = a.block_table + (int64_t)b * a.bt_stride;
  const int64_t* words = a.tree_mask != nullptr ? a.tree_mask + row * a.mask_words : nullptr;
  const int64_t row_elems = (int64_t)a.n_kv_heads * D;
  const T* kbase = static_cast<const T*>(a.k_pool) + (int64_t)kvh * D + dsub * kVec;
  const T* vbase = static_cast<const T*>(a.v_pool) + (int64_t)kvh * D + dsub * kVec;
  const int bmask = a.block_size - 1;

  for (int64_t c0 = t_begin + (int64_t)warp * kChunk; c0 < t_end; c0 += (int64_t)kTsWarps * kChunk) {
    uint4 kr[kTsUnroll], vr[kTsUnroll];
    bool valid[kTsUnroll];
#pragma unroll
    for (int u = 0; u < kTsUnroll; ++u) {
      const int64_t t = c0 + u * kRowsPerLoad + rsub;
      valid[u] = t < t_end;
      if (valid[u] && t >= hist) {
        const int s = (int)(t - hist);
        valid[u] = words != nullptr ? ((__ldg(words + (s >> 6)) >> (s & 63)) & 1) != 0 : s <= node;
      }
      kr[u] = make_uint4(0, 0, 0, 0);
      vr[u] = make_uint4(0, 0, 0, 0);
      if (valid[u]) {
        const int blk = __ldg(table + (t >> a.block_shift));
        if (blk < 0 || blk >= a.num_blocks) {
          raise_error(a.err, PA_DEVERR_BLOCK_ID);
          valid[u] = false;
        } else {
          const int64_t off = (int64_t)blk * a.kv_block_stride + (t & bmask) * row_elems;
          kr[u] = __ldg(reinterpret_cast<const uint4*>(kbase + off));
          vr[u] = __ldg(reinterpret_cast<const uint4*>(vbase + off));
        }
      }
    }
    float s[kTsUnroll][G];
#pragma unroll
    for (int u = 0; u < kTsUnroll; ++u) {
      float kf[kVec];
      Elt<T>::unpack(kr[u], kf);
#pragma unroll
      for (int h = 0; h < G; ++h) {
        float d = 0.f;
#pragma unroll
        for (int e = 0; e < kVec; ++e) d = fmaf(qf[h][e], kf[e], d);
#pragma unroll
        for (int off = kLanesPerRow / 2; off > 0; off >>= 1) d += __shfl_xor_sync(0xffffffffu, d, off);
        s[u][h] = valid[u] ? d : -INFINITY;
      }
    }
    bool any = valid[0];
#pragma unroll
    for (int u = 1; u < kTsUnroll; ++u) any |= valid[u];
    if (!__any_sync(0xffffffffu, any)) continue;
#pragma unroll
    for (int h = 0; h < G; ++h) {
      float mx = s[0][h];
#pragma unroll
      for (int u = 1; u < kTsUnroll; ++u) mx = fmaxf(mx, s[u][h]);
#pragma unroll
      for (int off = kLanesPerRow; off < 32; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
      const float m_new = fmaxf(fmaxf(m[h], mx), -FLT_MAX);
      const float corr = fast_exp2(m[h] - m_new);  // m = -inf -> 0
      l[h] *= corr;
#pragma unroll
      for (int e = 0; e < kVec; ++e) acc[h][e] *= corr;
      m[h] = m_new;
    }
#pragma unroll
    for (int u = 0; u < kTsUnroll; ++u) {
      float vf[kVec];
      Elt<T>::unpack(vr[u], vf);
#pragma unroll
      for (int h = 0; h < G; ++h) {
        const float p = valid[u] ? fast_exp2(s[u][h] - m[h]) : 0.f;
        l[h] += p;
#pragma unroll
        for (int e = 0; e < kVec; ++e) acc[h][e] = fmaf(p, vf[e], acc[h][e]);
      }
    }
  }

#pragma unroll
  for (int h = 0; h < G; ++h) {
#pragma unroll
    for (int off = kLanesPerRow; off < 32; off <<= 1) {
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], off);
#pragma unroll
      for (int e = 0; e < kVec; ++e) acc[h][e] += __shfl_xor_sync(0xffffffffu, acc[h][e], off);
    }
  }
  if (rsub == 0) {
#pragma unroll
    for (int h = 0; h < G; ++h) {
#pragma unroll
      for (int e = 0; e < kVec; ++e) sm_acc[warp][h][dsub * kVec + e] = acc[h][e];
    }
  }
  if (lane == 0) {
#pragma unroll
    for (int h = 0; h < G; ++h) {
      sm_m[warp][h] = m[h];
      sm_l[warp][h] = l[h];
    }
  }
  __syncthreads();

  for (int i = threadIdx.x; i < G * D; i += kTsWarps * 32) {
    const int h = i / D;
    const int d = i - h * D;
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < kTsWarps; ++w) M = fmaxf(M, sm_m[w][h]);
    float L = 0.f, A = 0.f;
    if (M != -INFINITY) {
#pragma unroll
      for (int w = 0; w < kTsWarps; ++w) {
        const float f = fast_exp2(sm_m[w][h] - M);  // a warp without keys: 0, and its sums are 0
        L = fmaf(sm_l[w][h], f, L);
        A = fmaf(sm_acc[w][h][d], f, A);
      }
    }
    const int64_t qh = row * a.n_q_heads + (int64_t)kvh * G + h;
    if (n_parts == 1) {
      static_cast<T*>(a.out)[qh * D + d] = Elt<T>::from_float(M == -INFINITY ? 0.f : A / L);
    } else {
      const int64_t pi = qh * a.max_parts + part;
      a.ws_acc[pi * D + d] = A;
      if (d == 0) {
        a.ws_m[pi] = M;
        a.ws_l[pi] = L;
      }
    }
  }
}

// Partial states of a row into its output: sum_p acc_p 2^(m_p - M) / sum_p l_p 2^(m_p - M).  One warp
// per (node, query head); a sequence with one partition was written directly.
constexpr int kTmWarps = 4;

template <typename T, int D>
__global__ void __launch_bounds__(kTmWarps * 32) tree_merge_kernel(const TreeArgs a, int ctas_per_seq) {
  constexpr int kPer = D / 32;
  const int lane = threadIdx.x & 31;
  pdl_wait_primary();
  const int b = blockIdx.x / ctas_per_seq;
  const int64_t r = (int64_t)(blockIdx.x % ctas_per_seq) * kTmWarps + (threadIdx.x >> 5);
  const TreeSeq sq = tree_seq(a, b);
  const int parts = sq.n == 0 ? 1 : (sq.n + a.part_tokens - 1) / a.part_tokens;
  if (parts <= 1 || r >= (int64_t)sq.m * a.n_q_heads) return;
  const int64_t row = sq.q0 * a.n_q_heads + r;
  const float* pm = a.ws_m + row * a.max_parts;
  const float* pl = a.ws_l + row * a.max_parts;
  const float* pacc = a.ws_acc + row * a.max_parts * (int64_t)D + lane * kPer;
  float M = -INFINITY;
  for (int p = lane; p < parts; p += 32) M = fmaxf(M, pm[p]);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
  float L = 0.f, acc[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) acc[i] = 0.f;
  if (M != -INFINITY) {
#pragma unroll 4
    for (int p = 0; p < parts; ++p) {
      const float w = fast_exp2(pm[p] - M);
      L = fmaf(pl[p], w, L);
#pragma unroll
      for (int i = 0; i < kPer; ++i) acc[i] = fmaf(pacc[(int64_t)p * D + i], w, acc[i]);
    }
  }
  T* o = static_cast<T*>(a.out) + row * D + lane * kPer;
#pragma unroll
  for (int i = 0; i < kPer; ++i) o[i] = Elt<T>::from_float(M == -INFINITY ? 0.f : acc[i] / L);
}

template <typename T, int D>
static cudaError_t launch_simt_g(const TreeArgs& a, cudaStream_t s) {
  const int64_t grid = (int64_t)a.batch * a.max_nodes * a.max_parts * a.n_kv_heads;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  const dim3 blk(kTsWarps * 32);
  switch (a.group) {
    case 1: tree_simt_kernel<T, D, 1><<<(unsigned)grid, blk, 0, s>>>(a); break;
    case 2: tree_simt_kernel<T, D, 2><<<(unsigned)grid, blk, 0, s>>>(a); break;
    case 4: tree_simt_kernel<T, D, 4><<<(unsigned)grid, blk, 0, s>>>(a); break;
    case 8: tree_simt_kernel<T, D, 8><<<(unsigned)grid, blk, 0, s>>>(a); break;
    case 16: tree_simt_kernel<T, D, 16><<<(unsigned)grid, blk, 0, s>>>(a); break;
    default: return cudaErrorInvalidValue;
  }
  return cudaGetLastError();
}

template <typename T>
static cudaError_t launch_simt_t(const TreeArgs& a, cudaStream_t s) {
  switch (a.head_dim) {
    case 64: return launch_simt_g<T, 64>(a, s);
    case 128: return launch_simt_g<T, 128>(a, s);
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t launch_tree_simt(const TreeArgs& a, pa_dtype dt, cudaStream_t s, int* launches) {
  cudaError_t e;
  switch (dt) {
    case PA_BF16: e = launch_simt_t<__nv_bfloat16>(a, s); break;
    case PA_FP16: e = launch_simt_t<__half>(a, s); break;
    case PA_FP32: e = launch_simt_t<float>(a, s); break;
    default: return cudaErrorInvalidValue;
  }
  ++*launches;
  return e;
}

template <typename T>
static cudaError_t launch_merge_t(const TreeArgs& a, cudaStream_t s) {
  const int64_t rows = (int64_t)a.max_nodes * a.n_q_heads;
  const int64_t per_seq = (rows + kTmWarps - 1) / kTmWarps;
  if (per_seq * a.batch > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(per_seq * a.batch));
  cfg.blockDim = dim3(kTmWarps * 32);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return a.head_dim == 64 ? cudaLaunchKernelEx(&cfg, tree_merge_kernel<T, 64>, a, (int)per_seq)
                          : cudaLaunchKernelEx(&cfg, tree_merge_kernel<T, 128>, a, (int)per_seq);
}

cudaError_t launch_tree_merge(const TreeArgs& a, pa_dtype dt, cudaStream_t s, int* launches) {
  cudaError_t e;
  switch (dt) {
    case PA_BF16: e = launch_merge_t<__nv_bfloat16>(a, s); break;
    case PA_FP16: e = launch_merge_t<__half>(a, s); break;
    case PA_FP32: e = launch_merge_t<float>(a, s); break;
    default: return cudaErrorInvalidValue;
  }
  ++*launches;
  return e;
}

}  // namespace pa
