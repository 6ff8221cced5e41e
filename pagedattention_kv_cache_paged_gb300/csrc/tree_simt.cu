// Tree attention on CUDA cores (every dtype and shape; the kernel of fp32 pools).
//
// Two CTAs of four warps per SM walk their equal share of the units (tree_common.cuh).  A unit's rows (up to
// 32 (node, head) rows, 16 at head_dim 128) stay in shared memory.  Each warp takes its own 32 (16) keys of
// every key tile, staged in fp32 with cp.async through a ring of three buffers of its own (K, V, the next
// K), and keeps its own softmax state (running maximum, sum and rescaled accumulator) for all rows, so that
// nothing is read from shared memory twice and the warps meet at the end of the unit only, where their
// states are joined.  Lane (rg, cg) of 4 x 8 holds kRT rows x every 8th key of S, and the same rows x head_dim
// / 8 columns of O; P takes K's buffer on its way from one layout to the other.  Per four dimensions (keys) a
// warp reads kRT + 4 (kRT + 8) conflict-free 128-byte wavefronts for 16 (32) kRT fma's per lane: with 8 rows
// or more a lane's work is bound by the fma units (37 T fma/s), with few rows in all by HBM.
//
// Masks are looked at in tiles that reach into the drafted region only: a masked score becomes -inf by
// selection.  A masked value cannot be deselected in a product (0 * NaN), so there non-finite elements of V
// are zeroed in shared memory, and added at the end, by themselves, to the rows that see them.
//
// A row that saw keys has a finite maximum at the end (at least -FLT_MAX), one that saw none has -inf: a row
// whose every score is -inf is told from a row that sees nothing (NaN, and zeros).
#include <float.h>

#include "pa_ptx.cuh"
#include "tree_common.cuh"

namespace pa {

constexpr int kTsWarps = 4;
constexpr int kTsThreads = 32 * kTsWarps;

template <int D, int kRT>
struct TsCfg {
  static constexpr int kRows = 4 * kRT;
  static constexpr int kKeys = tree_simt_keys(D);    // of a tile
  static constexpr int kWarpKeys = kKeys / kTsWarps;
  static constexpr int kRow = D + 4;                 // floats per staged row of Q, K and V: spreads rows over banks
  static constexpr int kPRow = kWarpKeys + 4;
  static constexpr int kSlot = kWarpKeys * kRow;     // one K or V buffer
  static constexpr int kSmemBytes = (kRows * kRow + kTsWarps * 3 * kSlot) * 4;
  static_assert(kRows * kPRow <= kSlot && kRows * D <= 3 * kSlot, "P in a K buffer, O in a ring");
};

__device__ __forceinline__ void cp_async16(void* dst, const void* src, bool ok) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(ok ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}

__device__ __forceinline__ void fma4(float& acc, const float4& a, const float4& b) {
  acc = fmaf(a.x, b.x, acc);
  acc = fmaf(a.y, b.y, acc);
  acc = fmaf(a.z, b.z, acc);
  acc = fmaf(a.w, b.w, acc);
}

template <typename T, int D, int kRT>
__global__ void __launch_bounds__(kTsThreads, 2) tree_simt_kernel(const TreeArgs a) {
  using Cfg = TsCfg<D, kRT>;
  constexpr int kKeys = Cfg::kKeys, kWK = Cfg::kWarpKeys, kRow = Cfg::kRow, kPRow = Cfg::kPRow, kRows = Cfg::kRows;
  constexpr int kSlot = Cfg::kSlot;
  constexpr int kKJ = kWK / 8;           // keys per lane
  constexpr int kOC = D / 32;            // 4-column groups per lane
  constexpr int kVec = Elt<T>::kVec;     // elements per 16 bytes of a pool row
  constexpr int kRowVecs = D / kVec;     // lanes per pool row
  constexpr int kPass = 32 / kRowVecs;   // pool rows per pass of the warp

  extern __shared__ __align__(16) float smem[];
  float* const qs = smem;                               // [kRows][kRow]
  float* const rings = qs + kRows * kRow;               // [warps][3][kWK][kRow]
  __shared__ TreeSched sched;
  __shared__ float s_m[kTsWarps][kRows], s_l[kTsWarps][kRows];
  __shared__ int s_bad_v;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rg = lane >> 3, cg = lane & 7;
  float* const ring = rings + warp * 3 * kSlot;
  if (tid == 0) {
    tree_schedule_init(a, sched);
    s_bad_v = 0;
  }
  __syncthreads();
  pdl_wait_primary();
  pdl_launch_dependents();
  const int nodes_unit = kRows >> a.group_shift;
  tree_schedule<kTsThreads, kKeys, kTreeSimtGap, kTreeSimtMinShare>(a, nodes_unit, sched);
  __syncthreads();

  const int64_t row_elems = (int64_t)a.n_kv_heads * D;
  const int bmask = a.block_size - 1;
  bool cut = false;
  TreeWalk<kKeys> walk(a, sched.span, nodes_unit);
  TreeUnit w;
  while (walk.next(w)) {
    const int hist = w.sq.n - w.sq.m;
    const int32_t* table = a.block_table + (int64_t)w.b * a.bt_stride;
    const int64_t row0 = (w.sq.q0 + w.node0) * a.n_q_heads + ((int64_t)w.kvh << a.group_shift);
    auto out_row = [&](int r) -> int64_t {
      return row0 + (int64_t)(r >> a.group_shift) * a.n_q_heads + (r & (a.group - 1));
    };
    auto words_of = [&](int node) -> const int64_t* {
      return a.tree_mask != nullptr ? a.tree_mask + (w.sq.q0 + node) * a.mask_words : nullptr;
    };
    // element offset of the pool row (KV head 0) of this lane's key of the warp's part of tile x; -1: no key
    auto locate = [&](int x) -> int64_t {
      const int pos = x * kKeys + warp * kWK + lane;
      if (lane >= kWK || x >= w.x1 || pos >= w.sq.n) return -1;
      const int blk = __ldg(table + (pos >> a.block_shift));
      if (blk < 0 || blk >= a.num_blocks) {
        raise_error(a.err, PA_DEVERR_BLOCK_ID);
        return -1;
      }
      return (int64_t)blk * a.kv_block_stride + (pos & bmask) * row_elems;
    };
    // the warp's keys (or values) at the lanes' offsets `off` into a buffer, zeros where there is no key
    auto load = [&](float* dst, const void* pool, int64_t off) {
      const T* src = static_cast<const T*>(pool) + (int64_t)w.kvh * D + (lane % kRowVecs) * kVec;
#pragma unroll
      for (int k = 0; k < kWK; k += kPass) {
        const int key = k + lane / kRowVecs;
        const int64_t o = __shfl_sync(0xffffffffu, off, key);
        float* at = dst + key * kRow + (lane % kRowVecs) * kVec;
        if constexpr (kVec == 4) {
          cp_async16(at, src + (o < 0 ? 0 : o), o >= 0);
        } else {
          float f[8];
          Elt<T>::unpack(o >= 0 ? __ldg(reinterpret_cast<const uint4*>(src + o)) : make_uint4(0, 0, 0, 0), f);
          *reinterpret_cast<float4*>(at) = make_float4(f[0], f[1], f[2], f[3]);
          *reinterpret_cast<float4*>(at + 4) = make_float4(f[4], f[5], f[6], f[7]);
        }
      }
      cp_async_commit();
    };

    __syncthreads();  // the unit before is done with the shared memory
    // loads in the order K, V, K, V, ..: load number i goes to buffer i % 3, each a group of its own
    int64_t off = locate(w.x0), off_next = locate(w.x0 + 1);
    load(ring, a.k_pool, off);
    load(ring + kSlot, a.v_pool, off);
    load(ring + 2 * kSlot, a.k_pool, off_next);
    // the rows, scaled into the log2 domain; rows behind the last are zeros
    for (int i = tid; i < kRows * (D / 4); i += kTsThreads) {
      const int r = i / (D / 4), c = i % (D / 4) * 4;
      float f[4] = {0.f, 0.f, 0.f, 0.f};
      if (r < w.rows) {
        const T* q = static_cast<const T*>(a.q) + out_row(r) * D + c;
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = static_cast<float>(q[e]) * a.scale_log2;
      }
      *reinterpret_cast<float4*>(qs + r * kRow + c) = make_float4(f[0], f[1], f[2], f[3]);
    }
    __syncthreads();

    // row i of this lane: 4 i + rg
    float m[kRT], l[kRT], o[kRT][kOC * 4];
    unsigned seen = 0;
#pragma unroll
    for (int i = 0; i < kRT; ++i) {
      m[i] = -INFINITY;
      l[i] = 0.f;
#pragma unroll
      for (int e = 0; e < kOC * 4; ++e) o[i][e] = 0.f;
    }
    int slot = 0;  // of K of the tile
    for (int x = w.x0; x < w.x1; ++x) {
      float* const kt = ring + slot * kSlot;
      float* const vt = ring + (slot == 2 ? 0 : slot + 1) * kSlot;
      const int kb = x * kKeys + warp * kWK;
      const unsigned have = __ballot_sync(0xffffffffu, off >= 0);  // keys of the tile with data
      const unsigned full = kWK == 32 ? 0xffffffffu : (1u << (kWK & 31)) - 1u;
      const bool edge = kb + kWK > hist || have != full;
      const int64_t off_after = locate(x + 2);
      cp_async_wait<2>();
      __syncwarp();

      // ---- S = Q K^T: keys cg + 8 j ----
      float s[kRT][kKJ];
#pragma unroll
      for (int i = 0; i < kRT; ++i)
#pragma unroll
        for (int j = 0; j < kKJ; ++j) s[i][j] = 0.f;
#pragma unroll 4
      for (int d = 0; d < D; d += 4) {
        float4 q[kRT], k[kKJ];
#pragma unroll
        for (int i = 0; i < kRT; ++i) q[i] = *reinterpret_cast<const float4*>(qs + (4 * i + rg) * kRow + d);
#pragma unroll
        for (int j = 0; j < kKJ; ++j) k[j] = *reinterpret_cast<const float4*>(kt + (cg + 8 * j) * kRow + d);
#pragma unroll
        for (int i = 0; i < kRT; ++i)
#pragma unroll
          for (int j = 0; j < kKJ; ++j) fma4(s[i][j], q[i], k[j]);
      }
      if (edge) {
#pragma unroll
        for (int i = 0; i < kRT; ++i) {
          const int node = w.node0 + (min(4 * i + rg, w.rows - 1) >> a.group_shift);
          const int64_t* words = words_of(node);
          bool any = false;
#pragma unroll
          for (int j = 0; j < kKJ; ++j) {
            const int pos = kb + cg + 8 * j;
            const bool see = ((have >> (cg + 8 * j)) & 1u) != 0 && (pos < hist || tree_sees(words, node, pos - hist));
            if (!see) s[i][j] = -INFINITY;
            any |= see;
          }
          if ((__ballot_sync(0xffffffffu, any) >> (8 * rg)) & 0xffu) seen |= 1u << i;
        }
      } else {
        seen = 0xffffffffu;
      }
      // ---- softmax step; the eight lanes of a row group hold its rows ----
      __syncwarp();  // K has been read: its buffer takes P
#pragma unroll
      for (int i = 0; i < kRT; ++i) {
        float mx = s[i][0];
#pragma unroll
        for (int j = 1; j < kKJ; ++j) mx = fmaxf(mx, s[i][j]);
#pragma unroll
        for (int b = 1; b < 8; b <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, b));
        const float m_new = fmaxf(m[i], mx);
        const float m_sub = m_new == -INFINITY ? 0.f : m_new;
        const float corr = fast_exp2(m[i] - m_sub);  // m = -inf: 0
        m[i] = m_new;
        l[i] *= corr;
#pragma unroll
        for (int e = 0; e < kOC * 4; ++e) o[i][e] *= corr;
#pragma unroll
        for (int j = 0; j < kKJ; ++j) {
          const float p = fast_exp2(s[i][j] - m_sub);
          l[i] += p;
          kt[(4 * i + rg) * kPRow + cg + 8 * j] = p;
        }
      }
      cp_async_wait<1>();
      __syncwarp();
      if (edge) {
        // non-finite values of drafted tokens (keys without data are zeros)
        for (int i = lane; i < kWK * (D / 4); i += 32) {
          const int key = i / (D / 4);
          if (kb + key < hist) continue;
          float4* p = reinterpret_cast<float4*>(vt + key * kRow + i % (D / 4) * 4);
          float4 v = *p;
          if (!(fabsf(v.x) <= FLT_MAX && fabsf(v.y) <= FLT_MAX && fabsf(v.z) <= FLT_MAX && fabsf(v.w) <= FLT_MAX)) {
            v.x = fabsf(v.x) <= FLT_MAX ? v.x : 0.f;
            v.y = fabsf(v.y) <= FLT_MAX ? v.y : 0.f;
            v.z = fabsf(v.z) <= FLT_MAX ? v.z : 0.f;
            v.w = fabsf(v.w) <= FLT_MAX ? v.w : 0.f;
            *p = v;
            s_bad_v = 1;
          }
        }
        __syncwarp();
      }
      // ---- O += P V: columns 4 cg + 32 e ----
#pragma unroll 2
      for (int k = 0; k < kWK; k += 4) {
        float4 p[kRT];
#pragma unroll
        for (int i = 0; i < kRT; ++i) p[i] = *reinterpret_cast<const float4*>(kt + (4 * i + rg) * kPRow + k);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
#pragma unroll
          for (int e = 0; e < kOC; ++e) {
            const float4 v = *reinterpret_cast<const float4*>(vt + (k + u) * kRow + 4 * cg + 32 * e);
#pragma unroll
            for (int i = 0; i < kRT; ++i) {
              const float pu = u == 0 ? p[i].x : u == 1 ? p[i].y : u == 2 ? p[i].z : p[i].w;
              o[i][4 * e] = fmaf(pu, v.x, o[i][4 * e]);
              o[i][4 * e + 1] = fmaf(pu, v.y, o[i][4 * e + 1]);
              o[i][4 * e + 2] = fmaf(pu, v.z, o[i][4 * e + 2]);
              o[i][4 * e + 3] = fmaf(pu, v.w, o[i][4 * e + 3]);
            }
          }
        }
      }
      __syncwarp();  // P and V have been read: V of the next tile and K of the one after it
      load(kt, a.v_pool, off_next);
      load(vt, a.k_pool, off_after);
      slot = slot == 0 ? 2 : slot - 1;
      off = off_next;
      off_next = off_after;
    }

    // ---- join the warps' states and write the unit's rows, or this CTA's piece of them ----
    cp_async_wait<0>();
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kRT; ++i) {
#pragma unroll
      for (int b = 1; b < 8; b <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], b);
      const int r = 4 * i + rg;
      if (cg == 0) {
        s_m[warp][r] = (seen >> i) & 1u ? fmaxf(m[i], -FLT_MAX) : -INFINITY;
        s_l[warp][r] = l[i];
      }
#pragma unroll
      for (int e = 0; e < kOC; ++e)
        *reinterpret_cast<float4*>(ring + r * D + 4 * cg + 32 * e) =
            make_float4(o[i][4 * e], o[i][4 * e + 1], o[i][4 * e + 2], o[i][4 * e + 3]);
    }
    __syncthreads();
    const bool whole = w.x0 == 0 && w.x1 == w.T;
    for (int i = tid; i < w.rows * (D / 4); i += kTsThreads) {
      const int r = i / (D / 4), c = i % (D / 4) * 4;
      float M = -INFINITY;
#pragma unroll
      for (int k = 0; k < kTsWarps; ++k) M = fmaxf(M, s_m[k][r]);
      float L = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
      if (M != -INFINITY) {
#pragma unroll
        for (int k = 0; k < kTsWarps; ++k) {
          const float f = fast_exp2(s_m[k][r] - M);  // a warp without keys: 0, and its sums are 0
          const float4 v = *reinterpret_cast<const float4*>(rings + k * 3 * kSlot + r * D + c);
          L = fmaf(s_l[k][r], f, L);
          acc[0] = fmaf(v.x, f, acc[0]);
          acc[1] = fmaf(v.y, f, acc[1]);
          acc[2] = fmaf(v.z, f, acc[2]);
          acc[3] = fmaf(v.w, f, acc[3]);
        }
      }
      if (s_bad_v != 0) {
        // the non-finite elements that were taken out of V, for the rows that see them
        const int node = w.node0 + (r >> a.group_shift);
        const int last = min(w.x1 * kKeys, w.sq.n);
        for (int pos = max(w.x0 * kKeys, hist); pos < last; ++pos) {
          const int blk = __ldg(table + (pos >> a.block_shift));
          if (!tree_sees(words_of(node), node, pos - hist) || blk < 0 || blk >= a.num_blocks) continue;
          const T* v = static_cast<const T*>(a.v_pool) + (int64_t)blk * a.kv_block_stride + (pos & bmask) * row_elems +
                       (int64_t)w.kvh * D + c;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float f = static_cast<float>(v[e]);
            if (!(fabsf(f) <= FLT_MAX)) acc[e] += f;
          }
        }
      }
      if (whole) {
        T* out = static_cast<T*>(a.out) + out_row(r) * D + c;
#pragma unroll
        for (int e = 0; e < 4; ++e) out[e] = Elt<T>::from_float(M == -INFINITY ? 0.f : acc[e] / L);
      } else {
        const int64_t piece = ((int64_t)blockIdx.x * 2 + (w.x0 == 0 ? 1 : 0)) * kRows + r;
        *reinterpret_cast<float4*>(a.ws_acc + piece * D + c) = make_float4(acc[0], acc[1], acc[2], acc[3]);
        if (c == 0) {
          a.ws_m[piece] = M;
          a.ws_l[piece] = L;
        }
      }
    }
    if (!whole && w.x0 == 0) {
      cut = true;  // at most one unit of a CTA: the one that its span ends in
      if (tid == 0) tree_record(a, sched, w, row0, a.ws_rec + blockIdx.x);
    }
  }
  if (tid == 0 && !cut && a.split) a.ws_rec[blockIdx.x].rows = 0;
  if (sched.refused) tree_zero_refused<T>(a);
}

template <typename T, int D, int kRT>
static cudaError_t launch_ts(const TreeArgs& a, cudaStream_t s) {
  constexpr int smem = TsCfg<D, kRT>::kSmemBytes;
  static bool attr_set[64] = {};  // per instantiation and device; idempotent, so a race is harmless
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !attr_set[dev]) {
    e = cudaFuncSetAttribute(tree_simt_kernel<T, D, kRT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) attr_set[dev] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.ctas);
  cfg.blockDim = dim3(kTsThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, tree_simt_kernel<T, D, kRT>, a);
}

template <typename T, int D>
static cudaError_t launch_ts_rows(const TreeArgs& a, cudaStream_t s) {
  switch (tree_simt_rows(a.max_nodes, a.group, D)) {
    case 8: return launch_ts<T, D, 2>(a, s);
    case 16: return launch_ts<T, D, 4>(a, s);
    default:
      if constexpr (D == 64) return launch_ts<T, D, 8>(a, s);
      return cudaErrorInvalidValue;
  }
}

template <typename T>
static cudaError_t launch_ts_t(const TreeArgs& a, cudaStream_t s) {
  return a.head_dim == 64 ? launch_ts_rows<T, 64>(a, s) : launch_ts_rows<T, 128>(a, s);
}

cudaError_t launch_tree_simt(const TreeArgs& a, pa_dtype dt, cudaStream_t s, int* launches) {
  ++*launches;
  switch (dt) {
    case PA_BF16: return launch_ts_t<__nv_bfloat16>(a, s);
    case PA_FP16: return launch_ts_t<__half>(a, s);
    case PA_FP32: return launch_ts_t<float>(a, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace pa
