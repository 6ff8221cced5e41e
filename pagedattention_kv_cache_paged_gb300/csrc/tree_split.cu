// Tree attention with mma.sync (every dtype and block size; the kernel of fp32 pools).
//
// fp32 on bf16 tensor cores: x = x0 + x1 + x2, each part the bf16 rounding of what the ones before leave, holds
// the 24 bits of x, and of the nine products of two split values the six with i + j <= 2 are formed (the others
// come to at most 2^-23 of the product, of either sign).  16-bit queries and keys are operands as they are (so that
// the score of an infinite key is what it should be: a second part of infinity, or a product with it, would be NaN);
// fp16 values of V split into two parts and bf16 ones are their own first part, both exactly, and weights are split
// like fp32 values whatever the pool's type.  The tensor core adds
// in fp32 but cuts off where it should round, so that one accumulator for a whole context loses its last bits one
// after the other (28,000 keys: 5e-6 of the result).  For fp32 pools the products of 16 dimensions (S) or 16 keys
// (P V) are therefore summed by themselves, small ones first, and added up by rounded additions (2e-7, for 4-6 %
// of the time).
//
// On CUDA cores the same work is bound by shared memory, which hands every lane its operands (27 sequences of up to
// 1,941 tokens, 12 drafts, 12 heads, head_dim 64, fp32: 64 us where this takes 54, 3.1 TB/s): in fragments each
// value is read once per warp.  Bound by the products (six for one, in tiles of 16 rows) where a unit has many rows,
// by HBM where it has few (21 sequences of up to 8,984 tokens, head_dim 128, 4 rows: 4.2 TB/s), and by the latency
// of a unit's start and end where contexts are short.  16-bit pools with blocks of 8 (16 requests of up to 1,941
// tokens, 12 drafts, 32 / 8 heads, head_dim 128, 67.5 MB): bf16 89.6 us, fp16 85.1, 0.8 TB/s, bound like fp32 ones by
// tiles of 16 rows that each read their keys again (three of them a KV head) and by the split of weights and values.
//
// Three (at head_dim 128 two) CTAs of four warps per SM walk their equal share of the units (tree_common.cuh); a
// unit has up to 32 (node, head) rows (16 at head_dim 128).  Each warp takes its own 16 keys of every key tile,
// staged in fp32 with cp.async through a ring of three buffers of its own, and keeps its own softmax state (running
// maximum, sum and rescaled accumulator) for all rows; the warps meet at the end of the unit, where their states
// are joined.  The order of the contracted index is free, so a lane's four dimensions (S) and four keys (P V)
// are consecutive: K and V fragments are 16-byte reads, and column c of the two score tiles of 16 keys is key
// 4 (c / 2) + c % 2 and that + 2, so that P is an operand as it stands.  16-byte chunks of a staged row are
// permuted (by the row's bit 0 in K, bits 2 and 3 in V) so that eight lanes meet all banks.  32 keys a warp with
// two CTAs per SM took 20 % longer.
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

template <typename T>
struct Parts;  // 16-bit parts of a query's or key's element, and the bf16 parts that hold one of V
template <> struct Parts<__nv_bfloat16> { static constexpr int kScore = 1, kN = 1; };
template <> struct Parts<__half> { static constexpr int kScore = 1, kN = 2; };
template <> struct Parts<float> { static constexpr int kScore = 3, kN = 3; };

template <typename T, int D, int kMT>
struct TsCfg {
  static constexpr int kRows = 16 * kMT;
  static constexpr int kKeys = kTreeSplitKeys;    // of a tile
  static constexpr int kWarpKeys = kKeys / kTsWarps;
  static constexpr int kSlot = kWarpKeys * D;         // floats of one K or V buffer
  static constexpr int kQFrags = kMT * (D / 16) * Parts<T>::kScore * 32;  // 16 bytes each
  static constexpr int kSmemBytes = kQFrags * 16 + kTsWarps * 3 * kSlot * 4;
  static_assert(kRows * D <= 3 * kSlot && kWarpKeys == 16, "O in a ring, one step of 16 keys");
};

__device__ __forceinline__ void cp_async16(void* dst, const void* src, bool ok) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(ok ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}

// Two bf16 values; what rounds past the largest becomes that.
__device__ __forceinline__ uint32_t pack2_finite(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.satfinite.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Four consecutive elements (of a row that starts on 16 bytes).
__device__ __forceinline__ void read4(const float* p, float (&f)[4]) {
  const float4 v = *reinterpret_cast<const float4*>(p);
  f[0] = v.x, f[1] = v.y, f[2] = v.z, f[3] = v.w;
}
__device__ __forceinline__ void write4(float* p, const float (&f)[4]) {
  *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
}
template <typename T>
__device__ __forceinline__ void read4(const T* p, float (&f)[4]) {
  const uint2 v = *reinterpret_cast<const uint2*>(p);
  const T* e = reinterpret_cast<const T*>(&v);
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = static_cast<float>(e[i]);
}
template <typename T>
__device__ __forceinline__ void write4(T* p, const float (&f)[4]) {
  constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
  *reinterpret_cast<uint2*>(p) = make_uint2(pack2<kBf16>(f[0], f[1]), pack2<kBf16>(f[2], f[3]));
}

// The first kN bf16 parts of two values, packed in pairs (a in the low halves).
template <int kN>
__device__ __forceinline__ void split2(float a, float b, uint32_t (&part)[kN]) {
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    // (the largest numbers of fp32 round to infinity otherwise; infinities still come out as NaN)
    part[i] = kN == 3 && i == 0 ? pack2_finite(a, b) : pack2<true>(a, b);
    if (i + 1 < kN) {
      a -= __uint_as_float(part[i] << 16);
      b -= __uint_as_float(part[i] & 0xffff0000u);
    }
  }
}

// Two elements of a query or key as operands of their own type (fp16) or in bf16 parts.
template <typename T, int kN>
__device__ __forceinline__ void split_score(float a, float b, uint32_t (&part)[kN]) {
  if constexpr (std::is_same<T, __half>::value) part[0] = pack2<false>(a, b);
  else split2<kN>(a, b, part);
}

template <typename T, int D, int kMT>
__global__ void __launch_bounds__(kTsThreads, tree_split_ctas(D)) tree_split_kernel(const TreeArgs a) {
  using Cfg = TsCfg<T, D, kMT>;
  constexpr int kKeys = Cfg::kKeys, kWK = Cfg::kWarpKeys, kRows = Cfg::kRows, kSlot = Cfg::kSlot;
  constexpr int kS = Parts<T>::kScore;   // parts of q and k
  constexpr int kN = Parts<T>::kN;       // parts of v
  constexpr bool kScoreBf16 = !std::is_same<T, __half>::value;
  constexpr bool kFresh = kN == 3;       // sums of a step's products on their own first
  constexpr int kNT = kWK / 8;           // score tiles of 8 keys
  constexpr int kKD = D / 16;            // steps of 16 dimensions
  constexpr int kOT = D / 8;             // output tiles of 8 columns
  constexpr int kVec = Elt<T>::kVec;     // elements per 16 bytes of a pool row
  constexpr int kRowVecs = D / kVec;     // lanes per pool row
  constexpr int kPass = 32 / kRowVecs;   // pool rows per pass of the warp

  extern __shared__ __align__(16) uint8_t smem[];
  uint4* const qf = reinterpret_cast<uint4*>(smem);     // [m tile][16-dim step][part][lane]: A fragments
  float* const rings = reinterpret_cast<float*>(smem + Cfg::kQFrags * 16);  // [warps][3][kWK][D]
  __shared__ TreeSched sched;
  __shared__ float s_m[kTsWarps][kRows], s_l[kTsWarps][kRows];
  __shared__ int s_bad_v;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t = lane & 3;  // row (column) group and thread of the mma layouts
  float* const ring = rings + warp * 3 * kSlot;
  if (tid == 0) {
    tree_schedule_init(a, sched);
    s_bad_v = 0;
  }
  __syncthreads();
  pdl_wait_primary();
  pdl_launch_dependents();
  const int nodes_unit = kRows >> a.group_shift;
  tree_schedule<kTsThreads, kKeys, kTreeSplitGap, kTreeSplitMinShare>(a, nodes_unit, sched);
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
    // element offset of the pool row (KV head 0) of this lane's key of the warp's part of tile x; -1: no key,
    // -2: a key whose block is out of range
    auto locate = [&](int x) -> int64_t {
      const int pos = x * kKeys + warp * kWK + lane;
      if (lane >= kWK || x >= w.x1 || pos >= w.sq.n) return -1;
      const int blk = ld_s32(table + (pos >> a.block_shift));
      if (blk < 0 || blk >= a.num_blocks) {
        raise_error(a.err, PA_DEVERR_BLOCK_ID);
        return -2;
      }
      return (int64_t)blk * a.kv_block_stride + (pos & bmask) * row_elems;
    };
    // place of 16-byte chunk c of a key's staged row
    auto k_chunk = [](int key, int c) { return key * (D / 4) + (c ^ ((key & 1) << 2)); };
    auto v_chunk = [](int key, int c) { return key * (D / 4) + (c ^ ((key >> 1) & 6)); };
    // the warp's keys (or values) at the lanes' offsets `off` into a buffer, zeros where there is no key
    auto load = [&](auto is_v, float* dst, int64_t off) {
      constexpr bool kV = decltype(is_v)::value;
      if (!__any_sync(0xffffffffu, off != -1)) {  // (behind the last tile)
        cp_async_commit();
        return;
      }
      const T* src = static_cast<const T*>(kV ? a.v_pool : a.k_pool) + (int64_t)w.kvh * D + (lane % kRowVecs) * kVec;
#pragma unroll
      for (int k = 0; k < kWK; k += kPass) {
        const int key = k + lane / kRowVecs;
        const int64_t o = __shfl_sync(0xffffffffu, off, key);
        float4* const at = reinterpret_cast<float4*>(dst);
        const int c = lane % kRowVecs * (kVec / 4);
        if constexpr (kVec == 4) {
          cp_async16(at + (kV ? v_chunk(key, c) : k_chunk(key, c)), src + (o < 0 ? 0 : o), o >= 0);
        } else {
          float f[8];
          Elt<T>::unpack(o >= 0 ? *reinterpret_cast<const uint4*>(src + o) : make_uint4(0, 0, 0, 0), f);
          at[kV ? v_chunk(key, c) : k_chunk(key, c)] = make_float4(f[0], f[1], f[2], f[3]);
          at[kV ? v_chunk(key, c + 1) : k_chunk(key, c + 1)] = make_float4(f[4], f[5], f[6], f[7]);
        }
      }
      cp_async_commit();
    };

    __syncthreads();  // the unit before is done with the shared memory
    // loads in the order K, V, K, V, ..: load number i goes to buffer i % 3, each a group of its own
    int64_t off = locate(w.x0), off_next = locate(w.x0 + 1);
    load(std::false_type{}, ring, off);
    load(std::true_type{}, ring + kSlot, off);
    load(std::false_type{}, ring + 2 * kSlot, off_next);
    // the rows' fragments: lane (g, t) holds dimensions 4 t .. 4 t + 3 of rows g and g + 8; rows behind the last
    // are zeros
    for (int i = tid; i < kMT * kKD * 32; i += kTsThreads) {
      const int l = i & 31, step = (i >> 5) % kKD, mt = (i >> 5) / kKD;
      float f[2][4] = {};
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = 16 * mt + 8 * h + (l >> 2);
        if (r < w.rows) read4(static_cast<const T*>(a.q) + out_row(r) * D + 16 * step + 4 * (l & 3), f[h]);
      }
      uint32_t p0[kS], p1[kS], p2[kS], p3[kS];
      split_score<T>(f[0][0], f[0][1], p0);
      split_score<T>(f[1][0], f[1][1], p1);
      split_score<T>(f[0][2], f[0][3], p2);
      split_score<T>(f[1][2], f[1][3], p3);
#pragma unroll
      for (int p = 0; p < kS; ++p) qf[((mt * kKD + step) * kS + p) * 32 + l] = make_uint4(p0[p], p1[p], p2[p], p3[p]);
    }
    __syncthreads();

    // rows of this lane: 16 mt + 8 h + g
    float m[kMT][2], l[kMT][2], o[kMT][kOT][4];
    unsigned seen = 0;
#pragma unroll
    for (int mt = 0; mt < kMT; ++mt) {
      m[mt][0] = m[mt][1] = -INFINITY;
      l[mt][0] = l[mt][1] = 0.f;
#pragma unroll
      for (int i = 0; i < kOT; ++i) o[mt][i][0] = o[mt][i][1] = o[mt][i][2] = o[mt][i][3] = 0.f;
    }
    int slot = 0;  // of K of the tile
    const int x_end = min(w.x1, (w.sq.n - warp * kWK + kKeys - 1) / kKeys);  // (in the last tile a warp may have no keys)
    for (int x = w.x0; x < x_end; ++x) {
      float* const kt = ring + slot * kSlot;
      float* const vt = ring + (slot == 2 ? 0 : slot + 1) * kSlot;
      const int kb = x * kKeys + warp * kWK;
      const unsigned have = __ballot_sync(0xffffffffu, off >= 0);  // keys of the tile with data
      const bool edge = kb + kWK > hist || have != (1u << kWK) - 1u;
      const int64_t off_after = locate(x + 2);
      cp_async_wait<2>();
      __syncwarp();

      // ---- S = Q K^T ----
      float s[kMT][kNT][4];
#pragma unroll
      for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
        for (int n = 0; n < kNT; ++n) s[mt][n][0] = s[mt][n][1] = s[mt][n][2] = s[mt][n][3] = 0.f;
      const float4* const kc = reinterpret_cast<const float4*>(kt);
#pragma unroll
      for (int step = 0; step < kKD; ++step) {
        uint4 q[kMT][kS];
#pragma unroll
        for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
          for (int p = 0; p < kS; ++p) q[mt][p] = qf[((mt * kKD + step) * kS + p) * 32 + lane];
#pragma unroll
        for (int n = 0; n < kNT; ++n) {
          // column g of score tile n is key 16 (n / 2) + 4 (g / 2) + g % 2 + 2 (n % 2)
          const int key = 16 * (n >> 1) + 4 * (g >> 1) + (g & 1) + 2 * (n & 1);
          const float4 k = kc[k_chunk(key, 4 * step + t)];
          uint32_t b0[kS], b1[kS];
          split_score<T>(k.x, k.y, b0);
          split_score<T>(k.z, k.w, b1);
#pragma unroll
          for (int mt = 0; mt < kMT; ++mt) {
            float part[4] = {0.f, 0.f, 0.f, 0.f};
            float(&f)[4] = kFresh ? part : s[mt][n];
#pragma unroll
            for (int d = 2; d >= 0; --d)  // small products first
#pragma unroll
              for (int i = 0; i < kS; ++i)
                if (i <= d && d - i < kS)
                  mma_16816<kScoreBf16>(f, q[mt][i].x, q[mt][i].y, q[mt][i].z, q[mt][i].w, b0[d - i], b1[d - i]);
#pragma unroll
            for (int e = 0; kFresh && e < 4; ++e) s[mt][n][e] += part[e];
          }
        }
      }
      __syncwarp();  // K has been read: V of the next tile
      load(std::true_type{}, kt, off_next);
      if (edge) {
#pragma unroll
        for (int mt = 0; mt < kMT; ++mt) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int node = w.node0 + (min(16 * mt + 8 * h + g, w.rows - 1) >> a.group_shift);
            const int64_t* words = words_of(node);
            bool any = false;
#pragma unroll
            for (int n = 0; n < kNT; ++n) {
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int key = 16 * (n >> 1) + 4 * t + e + 2 * (n & 1), pos = kb + key;
                const bool see = ((have >> key) & 1u) != 0 && (pos < hist || tree_sees(words, node, pos - hist));
                if (!see) s[mt][n][2 * h + e] = -INFINITY;
                any |= see;
              }
            }
            if ((__ballot_sync(0xffffffffu, any) >> (4 * g)) & 0xfu) seen |= 1u << (2 * mt + h);
          }
        }
      } else {
        seen = 0xffffffffu;
      }
      // ---- softmax step; the four lanes of a row group hold its rows ----
      float corr[kMT][2];
#pragma unroll
      for (int mt = 0; mt < kMT; ++mt) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float mx = -INFINITY;
#pragma unroll
          for (int n = 0; n < kNT; ++n) mx = fmaxf(mx, fmaxf(s[mt][n][2 * h], s[mt][n][2 * h + 1]));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
          const float m_new = fmaxf(m[mt][h], mx);
          const float m_sub = m_new == -INFINITY ? 0.f : m_new;
          corr[mt][h] = fast_exp2((m[mt][h] - m_sub) * a.scale_log2);  // m = -inf: 0
          m[mt][h] = m_new;
          float sum = 0.f;
#pragma unroll
          for (int n = 0; n < kNT; ++n) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              // (the difference first: of s * scale - m in one rounding the rounding of m is left, which passes 2^7
              // for scores of 2^31)
              const float p = fast_exp2((s[mt][n][2 * h + e] - m_sub) * a.scale_log2);
              s[mt][n][2 * h + e] = p;
              sum += p;
            }
          }
          l[mt][h] = l[mt][h] * corr[mt][h] + sum;
          if (!kFresh && __any_sync(0xffffffffu, corr[mt][h] != 1.f)) {
#pragma unroll
            for (int i = 0; i < kOT; ++i) {
              o[mt][i][2 * h] *= corr[mt][h];
              o[mt][i][2 * h + 1] *= corr[mt][h];
            }
          }
        }
      }
      cp_async_wait<2>();
      __syncwarp();
      float4* const vc = reinterpret_cast<float4*>(vt);
      if (edge) {
        // non-finite values of drafted tokens (keys without data are zeros)
        for (int i = lane; i < kWK * (D / 4); i += 32) {
          if (kb + i / (D / 4) < hist) continue;
          float4 v = vc[i];
          if (!(fabsf(v.x) <= FLT_MAX && fabsf(v.y) <= FLT_MAX && fabsf(v.z) <= FLT_MAX && fabsf(v.w) <= FLT_MAX)) {
            v.x = fabsf(v.x) <= FLT_MAX ? v.x : 0.f;
            v.y = fabsf(v.y) <= FLT_MAX ? v.y : 0.f;
            v.z = fabsf(v.z) <= FLT_MAX ? v.z : 0.f;
            v.w = fabsf(v.w) <= FLT_MAX ? v.w : 0.f;
            vc[i] = v;
            s_bad_v = 1;
          }
        }
        __syncwarp();
      }
      // ---- O += P V; columns 32 b + 4 c + q make up output tile 4 b + q ----
      {
        static_assert(kNT == 2, "one step of 16 keys");
        uint32_t p[kMT][4][3];
#pragma unroll
        for (int mt = 0; mt < kMT; ++mt) {
          split2<3>(s[mt][0][0], s[mt][0][1], p[mt][0]);
          split2<3>(s[mt][0][2], s[mt][0][3], p[mt][1]);
          split2<3>(s[mt][1][0], s[mt][1][1], p[mt][2]);
          split2<3>(s[mt][1][2], s[mt][1][3], p[mt][3]);
        }
#pragma unroll
        for (int b = 0; b < D / 32; ++b) {
          float4 v[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) v[u] = vc[v_chunk(4 * t + u, 8 * b + g)];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            auto pick = [&](const float4& f) { return c == 0 ? f.x : c == 1 ? f.y : c == 2 ? f.z : f.w; };
            uint32_t b0[kN], b1[kN];
            split2<kN>(pick(v[0]), pick(v[1]), b0);
            split2<kN>(pick(v[2]), pick(v[3]), b1);
#pragma unroll
            for (int mt = 0; mt < kMT; ++mt) {
              float part[4] = {0.f, 0.f, 0.f, 0.f};
              float(&at)[4] = o[mt][4 * b + c];
              float(&f)[4] = kFresh ? part : at;
#pragma unroll
              for (int d = 2; d >= 0; --d)
#pragma unroll
                for (int i = 0; i < 3; ++i)
                  if (i <= d && d - i < kN)
                    mma_16816<true>(f, p[mt][0][i], p[mt][1][i], p[mt][2][i], p[mt][3][i], b0[d - i], b1[d - i]);
#pragma unroll
              for (int e = 0; kFresh && e < 4; ++e) at[e] = fmaf(at[e], corr[mt][e >> 1], part[e]);
            }
          }
        }
      }
      __syncwarp();  // V has been read: K of the tile after the next
      load(std::false_type{}, vt, off_after);
      slot = slot == 0 ? 2 : slot - 1;
      off = off_next;
      off_next = off_after;
    }

    // ---- join the warps' states and write the unit's rows, or this CTA's piece of them ----
    cp_async_wait<0>();
    __syncwarp();
    // (positions ascend over the warps and the tiles: these had keys in the first tile, the others nowhere)
    const int busy = min(kTsWarps, (min(w.x1 * kKeys, w.sq.n) - w.x0 * kKeys + kWK - 1) / kWK);
    if (warp < busy)
#pragma unroll
    for (int mt = 0; mt < kMT; ++mt) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float sum = l[mt][h];
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        const int r = 16 * mt + 8 * h + g;
        if (t == 0) {
          s_m[warp][r] = (seen >> (2 * mt + h)) & 1u ? fmaxf(m[mt][h], -FLT_MAX) : -INFINITY;
          s_l[warp][r] = sum;
        }
        // output tile 4 b + q, columns 2 t and 2 t + 1: columns 32 b + 4 (2 t) + q and 32 b + 4 (2 t + 1) + q
#pragma unroll
        for (int b = 0; b < D / 32; ++b) {
          float4* const at = reinterpret_cast<float4*>(ring + r * D + 32 * b + 8 * t);
          at[0] = make_float4(o[mt][4 * b][2 * h], o[mt][4 * b + 1][2 * h], o[mt][4 * b + 2][2 * h], o[mt][4 * b + 3][2 * h]);
          at[1] = make_float4(o[mt][4 * b][2 * h + 1], o[mt][4 * b + 1][2 * h + 1], o[mt][4 * b + 2][2 * h + 1],
                              o[mt][4 * b + 3][2 * h + 1]);
        }
      }
    }
    __syncthreads();
    const bool whole = w.x0 == 0 && w.x1 == w.T;
    for (int i = tid; i < w.rows * (D / 4); i += kTsThreads) {
      const int r = i / (D / 4), c = i % (D / 4) * 4;
      float M = -INFINITY;
#pragma unroll
      for (int k = 0; k < kTsWarps; ++k) M = k < busy ? fmaxf(M, s_m[k][r]) : M;
      float L = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
      if (M != -INFINITY) {
#pragma unroll
        for (int k = 0; k < kTsWarps; ++k) {
          if (k >= busy) break;
          const float f = fast_exp2((s_m[k][r] - M) * a.scale_log2);  // a warp without keys: 0, and its sums are 0
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
          const int blk = ld_s32(table + (pos >> a.block_shift));
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
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[e] = M == -INFINITY ? 0.f : acc[e] / L;
        write4(static_cast<T*>(a.out) + out_row(r) * D + c, acc);
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

template <typename T, int D, int kMT>
static cudaError_t launch_ts(const TreeArgs& a, cudaStream_t s) {
  constexpr int smem = TsCfg<T, D, kMT>::kSmemBytes;
  static bool attr_set[64] = {};  // per instantiation and device; idempotent, so a race is harmless
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !attr_set[dev]) {
    e = cudaFuncSetAttribute(tree_split_kernel<T, D, kMT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
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
  return cudaLaunchKernelEx(&cfg, tree_split_kernel<T, D, kMT>, a);
}

template <typename T, int D>
static cudaError_t launch_ts_rows(const TreeArgs& a, cudaStream_t s) {
  if constexpr (D == 64) {
    if (tree_split_rows(a.max_nodes, a.group, D) == 32) return launch_ts<T, D, 2>(a, s);
  }
  return launch_ts<T, D, 1>(a, s);
}

template <typename T>
static cudaError_t launch_ts_t(const TreeArgs& a, cudaStream_t s) {
  return a.head_dim == 64 ? launch_ts_rows<T, 64>(a, s) : launch_ts_rows<T, 128>(a, s);
}

cudaError_t launch_tree_split(const TreeArgs& a, pa_dtype dt, cudaStream_t s, int* launches) {
  ++*launches;
  switch (dt) {
    case PA_BF16: return launch_ts_t<__nv_bfloat16>(a, s);
    case PA_FP16: return launch_ts_t<__half>(a, s);
    case PA_FP32: return launch_ts_t<float>(a, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace pa
