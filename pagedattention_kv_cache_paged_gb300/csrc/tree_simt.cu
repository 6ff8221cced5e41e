// Tree attention on CUDA cores (every dtype and shape; the kernel of fp32 pools).
//
// Two CTAs of 128 threads per SM walk their equal share of the units (tree_common.cuh).  A unit's rows
// (up to 64 (node, head) rows) stay in shared memory; its key tiles (64 keys, 32 at head_dim 128) are
// staged there in fp32 with cp.async, two deep.  Per tile: S = Q K^T, one online-softmax step (running
// maximum and sum, accumulator rescaled), O += P V, all in fp32 registers: thread (ty, tx) of 8 x 16 holds
// kRT rows x every 16th key of S, and the same rows x head_dim / 16 columns of O; P goes through shared memory
// within the warp.  Per four dimensions it reads kRT + 4 vectors for 16 kRT fma's, so with 4 rows or more the
// fma units bound it (37 T fma/s), with fewer the reads do, and below 16 rows HBM.  Rows are padded by 16
// bytes, which spreads the 16 keys that a half-warp reads over the banks.
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

constexpr int kTsThreads = 128;

template <int D, int kRT>
struct TsCfg {
  static constexpr int kRows = 8 * kRT;
  static constexpr int kKeys = tree_simt_keys(D);
  static constexpr int kRow = D + 4;        // floats per staged row of Q, K and V
  static constexpr int kPRow = kKeys + 4;   // of P
  static constexpr int kKV = kKeys * kRow;
  static constexpr int kFloats = kRows * kRow + 4 * kKV + kRows * kPRow;
  static constexpr int kSmemBytes = kFloats * 4;
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
  constexpr int kKeys = Cfg::kKeys, kRow = Cfg::kRow, kPRow = Cfg::kPRow, kRows = Cfg::kRows;
  constexpr int kCK = kKeys / 16;        // keys per thread
  constexpr int kOC = D / 64;            // 4-column groups per thread
  constexpr int kVec = Elt<T>::kVec;     // elements per 16 bytes of a pool row
  constexpr int kRowVecs = D / kVec;
  constexpr int kRowsPass = kTsThreads / kRowVecs;

  extern __shared__ __align__(16) float smem[];
  float* const qs = smem;                     // [kRows][kRow]
  float* const ks = qs + kRows * kRow;        // [2][kKeys][kRow]
  float* const vs = ks + 2 * Cfg::kKV;        // [2][kKeys][kRow]
  float* const ps = vs + 2 * Cfg::kKV;        // [kRows][kPRow]
  __shared__ TreeSched sched;
  __shared__ int64_t s_off[2][kKeys];         // element offset of each key's pool row of KV head 0; -1: none
  __shared__ int s_gap[2];                    // x + 1: a key inside the context has no data in tile x
  __shared__ int s_bad_v;

  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
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
    // where the keys of tile x lie, into s_off[buf] (one thread per key)
    auto locate = [&](int x, int buf) {
      if (tid < kKeys) {
        const int pos = x * kKeys + tid;
        int64_t off = -1;
        if (x < w.x1 && pos < w.sq.n) {
          const int blk = __ldg(table + (pos >> a.block_shift));
          if (blk < 0 || blk >= a.num_blocks) {
            raise_error(a.err, PA_DEVERR_BLOCK_ID);
            s_gap[buf] = x + 1;
          } else {
            off = (int64_t)blk * a.kv_block_stride + (pos & bmask) * row_elems;
          }
        }
        s_off[buf][tid] = off;
      }
    };
    // tile in s_off[buf] into K and V buffer buf, zeros where there is no key
    auto load = [&](int buf) {
      const T* kp = static_cast<const T*>(a.k_pool) + (int64_t)w.kvh * D + (tid % kRowVecs) * kVec;
      const T* vp = static_cast<const T*>(a.v_pool) + (int64_t)w.kvh * D + (tid % kRowVecs) * kVec;
#pragma unroll
      for (int r = 0; r < kKeys; r += kRowsPass) {
        const int key = r + tid / kRowVecs;
        const int64_t off = s_off[buf][key];
        const int at = (buf * kKeys + key) * kRow + (tid % kRowVecs) * kVec;
        if constexpr (kVec == 4) {
          cp_async16(ks + at, kp + (off < 0 ? 0 : off), off >= 0);
          cp_async16(vs + at, vp + (off < 0 ? 0 : off), off >= 0);
        } else {
          uint4 kv = make_uint4(0, 0, 0, 0), vv = kv;
          if (off >= 0) {
            kv = __ldg(reinterpret_cast<const uint4*>(kp + off));
            vv = __ldg(reinterpret_cast<const uint4*>(vp + off));
          }
          float f[8];
          Elt<T>::unpack(kv, f);
          *reinterpret_cast<float4*>(ks + at) = make_float4(f[0], f[1], f[2], f[3]);
          *reinterpret_cast<float4*>(ks + at + 4) = make_float4(f[4], f[5], f[6], f[7]);
          Elt<T>::unpack(vv, f);
          *reinterpret_cast<float4*>(vs + at) = make_float4(f[0], f[1], f[2], f[3]);
          *reinterpret_cast<float4*>(vs + at + 4) = make_float4(f[4], f[5], f[6], f[7]);
        }
      }
      cp_async_commit();
    };

    if (tid < 2) s_gap[tid] = 0;
    __syncthreads();  // the unit before is done with the shared memory
    locate(w.x0, 0);
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
    load(0);
    locate(w.x0 + 1, 1);

    float m[kRT], l[kRT], o[kRT][kOC * 4];
    bool seen[kRT];
#pragma unroll
    for (int i = 0; i < kRT; ++i) {
      m[i] = -INFINITY;
      l[i] = 0.f;
      seen[i] = false;
#pragma unroll
      for (int e = 0; e < kOC * 4; ++e) o[i][e] = 0.f;
    }
    for (int x = w.x0; x < w.x1; ++x) {
      const int buf = (x - w.x0) & 1;
      cp_async_wait<0>();
      __syncthreads();  // tile x is here, s_off of tile x + 1 is, and everyone is done with tile x - 1
      const int kb = x * kKeys;
      const bool edge = kb + kKeys > hist || s_gap[buf] == x + 1;
      bool ok[kCK];
      if (edge) {
#pragma unroll
        for (int j = 0; j < kCK; ++j) ok[j] = s_off[buf][tx + 16 * j] >= 0;
        // non-finite values of drafted tokens (keys without data are zeros)
        for (int i = tid; i < kKeys * (D / 4); i += kTsThreads) {
          const int key = i / (D / 4);
          if (kb + key < hist) continue;
          float4* p = reinterpret_cast<float4*>(vs + (buf * kKeys + key) * kRow + i % (D / 4) * 4);
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
        __syncthreads();
      }
      if (x + 1 < w.x1) load(buf ^ 1);

      // ---- S = Q K^T: rows ty * kRT + i, keys tx + 16 j ----
      float s[kRT][kCK];
#pragma unroll
      for (int i = 0; i < kRT; ++i)
#pragma unroll
        for (int j = 0; j < kCK; ++j) s[i][j] = 0.f;
      const float* kt = ks + buf * Cfg::kKV + tx * kRow;
      const float* qt = qs + ty * kRT * kRow;
#pragma unroll 4
      for (int d = 0; d < D; d += 4) {
        float4 q[kRT], k[kCK];
#pragma unroll
        for (int i = 0; i < kRT; ++i) q[i] = *reinterpret_cast<const float4*>(qt + i * kRow + d);
#pragma unroll
        for (int j = 0; j < kCK; ++j) k[j] = *reinterpret_cast<const float4*>(kt + 16 * j * kRow + d);
#pragma unroll
        for (int i = 0; i < kRT; ++i)
#pragma unroll
          for (int j = 0; j < kCK; ++j) fma4(s[i][j], q[i], k[j]);
      }
      if (edge) {
#pragma unroll
        for (int i = 0; i < kRT; ++i) {
          const int r = min(ty * kRT + i, w.rows - 1), node = w.node0 + (r >> a.group_shift);
          const int64_t* words = a.tree_mask != nullptr ? a.tree_mask + (w.sq.q0 + node) * a.mask_words : nullptr;
          bool any = false;
#pragma unroll
          for (int j = 0; j < kCK; ++j) {
            const int pos = kb + tx + 16 * j;
            const bool see = ok[j] && (pos < hist || tree_sees(words, node, pos - hist));
            if (!see) s[i][j] = -INFINITY;
            any |= see;
          }
          // (a half-warp holds the row)
          seen[i] |= ((__ballot_sync(0xffffffffu, any) >> (tid & 16)) & 0xffffu) != 0;
        }
      } else {
#pragma unroll
        for (int i = 0; i < kRT; ++i) seen[i] = true;
      }
      // ---- softmax step ----
#pragma unroll
      for (int i = 0; i < kRT; ++i) {
        float mx = s[i][0];
#pragma unroll
        for (int j = 1; j < kCK; ++j) mx = fmaxf(mx, s[i][j]);
#pragma unroll
        for (int off = 1; off < 16; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
        const float m_new = fmaxf(m[i], mx);
        const float m_sub = m_new == -INFINITY ? 0.f : m_new;
        const float corr = fast_exp2(m[i] - m_sub);  // m = -inf: 0
        m[i] = m_new;
        l[i] *= corr;
#pragma unroll
        for (int e = 0; e < kOC * 4; ++e) o[i][e] *= corr;
#pragma unroll
        for (int j = 0; j < kCK; ++j) {
          const float p = fast_exp2(s[i][j] - m_sub);
          l[i] += p;
          ps[(ty * kRT + i) * kPRow + tx + 16 * j] = p;
        }
      }
      __syncwarp();  // the rows of P that a warp reads are its own
      // ---- O += P V: columns 4 tx + 64 e ----
      const float* vt = vs + buf * Cfg::kKV + tx * 4;
      const float* pt = ps + ty * kRT * kPRow;
#pragma unroll 2
      for (int k = 0; k < kKeys; k += 4) {
        float4 p[kRT];
#pragma unroll
        for (int i = 0; i < kRT; ++i) p[i] = *reinterpret_cast<const float4*>(pt + i * kPRow + k);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
#pragma unroll
          for (int e = 0; e < kOC; ++e) {
            const float4 v = *reinterpret_cast<const float4*>(vt + (k + u) * kRow + 64 * e);
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
      __syncthreads();  // s_off[buf] has been read
      locate(x + 2, buf);
    }

    // ---- the unit's rows: the output, or this CTA's piece of it ----
    const bool whole = w.x0 == 0 && w.x1 == w.T;
#pragma unroll
    for (int i = 0; i < kRT; ++i) {
      const int r = ty * kRT + i;
#pragma unroll
      for (int off = 1; off < 16; off <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], off);
      if (r >= w.rows) continue;
      const int node = w.node0 + (r >> a.group_shift);
      if (s_bad_v != 0) {
        // the non-finite elements that were taken out of V, for the rows that see them
        const int64_t* words = a.tree_mask != nullptr ? a.tree_mask + (w.sq.q0 + node) * a.mask_words : nullptr;
        const int last = min(w.x1 * kKeys, w.sq.n);
        for (int pos = max(w.x0 * kKeys, hist); pos < last; ++pos) {
          const int blk = __ldg(table + (pos >> a.block_shift));
          if (!tree_sees(words, node, pos - hist) || blk < 0 || blk >= a.num_blocks) continue;
          const T* v = static_cast<const T*>(a.v_pool) + (int64_t)blk * a.kv_block_stride + (pos & bmask) * row_elems +
                       (int64_t)w.kvh * D + tx * 4;
#pragma unroll
          for (int e = 0; e < kOC * 4; ++e) {
            const float f = static_cast<float>(v[(e >> 2) * 64 + (e & 3)]);
            if (!(fabsf(f) <= FLT_MAX)) o[i][e] += f;
          }
        }
      }
      const float M = seen[i] ? fmaxf(m[i], -FLT_MAX) : -INFINITY;
      if (whole) {
        T* out = static_cast<T*>(a.out) + out_row(r) * D + tx * 4;
#pragma unroll
        for (int e = 0; e < kOC * 4; ++e)
          out[(e >> 2) * 64 + (e & 3)] = Elt<T>::from_float(seen[i] ? o[i][e] / l[i] : 0.f);
      } else {
        const int64_t piece = ((int64_t)blockIdx.x * 2 + (w.x0 == 0 ? 1 : 0)) * kRows + r;
#pragma unroll
        for (int e = 0; e < kOC; ++e)
          *reinterpret_cast<float4*>(a.ws_acc + piece * D + tx * 4 + 64 * e) =
              make_float4(o[i][4 * e], o[i][4 * e + 1], o[i][4 * e + 2], o[i][4 * e + 3]);
        if (tx == 0) {
          a.ws_m[piece] = M;
          a.ws_l[piece] = l[i];
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
  switch (tree_simt_rows(a.max_nodes, a.group)) {
    case 8: return launch_ts<T, D, 1>(a, s);
    case 16: return launch_ts<T, D, 2>(a, s);
    case 32: return launch_ts<T, D, 4>(a, s);
    default: return launch_ts<T, D, 8>(a, s);
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
