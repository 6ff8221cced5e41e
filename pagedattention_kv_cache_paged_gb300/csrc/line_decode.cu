// Decode attention over the visible part of a context: a sliding window and the first tokens ("sinks"), or all of
// it.  Pools of 16-bit values (paged_attention_window) and the 4-bit cache (paged_attention_decode_q4), every block
// size.
//
// out = softmax(scale * q K^T) V over the positions j < sinks and j >= n - window.  The visible positions, packed to
// the left, make a unit's line of tokens: nothing else is read, neither rows nor table entries.
//
// Division of the work.  A unit is (sequence, `heads` KV heads next to one another).  All units in a row make one line
// of steps, a step being 16 tokens for every warp of the CTA; each CTA takes an equal share of it, whatever the
// lengths, and units that a cut falls into are joined by a second launch (as in tree attention, tree_common.cuh).
//
// A warp works by itself.  It takes 16 tokens of one KV head a step, copied into a ring of its own in shared memory a few
// steps ahead (also across units, so that the loads never pause; table entries are read one step earlier still), by
// TMA boxes or by cp.async, and forms both products with mma.sync m16n8k16 in the transposed form: S^T = K Q^T with the tokens
// as rows and the query heads as columns, O^T = V^T P^T with the dimensions as rows.  So a query group of up to 8
// heads costs 8 columns instead of 16 rows, K and V are the wide operand, and a head's stabiliser and accumulator
// lie in the same lanes.  One pass with a running stabiliser (a score, unscaled) that moves only when a weight
// would grow by more than 2^8: a vote per step, no shuffles.  The warps of a head are joined in shared memory at the
// end of a unit.
//
// 16-bit pools: K and V^T fragments by ldmatrix, weights rounded to the pool's type for the product with V (as the
// framework's other tensor-core kernels do; in fp16 formed 2^7 higher, see tree_umma.cu).
//
// 4-bit cache: codes become 16-bit operands with a logical instruction or two for two values and without any conversion,
// since the order of a contraction is free: the dimensions (tokens) of an operand register are those whose codes lie 16
// bits apart.  See PackedRows (bf16 and fp16 queries) and PackedWideRows (fp32).
#include <float.h>

#include <algorithm>

#include "pa_ptx.cuh"
#include "q4_common.cuh"
#include "tree_common.cuh"

namespace pa {

// TMA views of the pools (16-bit pools in blocks of a multiple of 16 tokens).
struct LineMaps {
  CUtensorMap k, v;
};

// ------------------------------------------------------------------------------------------------
// Sequences and the line
// ------------------------------------------------------------------------------------------------

// What is visible of a sequence: its first tokens and its last ones, `seen` in all; position of visible token v is v, or
// v + skip from `first` on.
// With a.aligned both parts are whole 16-key sub-tiles, whose ends a row's mask cuts off: positions below a.sinks and from
// `low` up to n.
struct LineSeq {
  int first, skip, seen;
  int low, n;
  bool bad;
};

__device__ __forceinline__ LineSeq line_seq(const LineArgs& a, int b) {
  LineSeq s{};
  const int n = ld_s32(a.context_lens + b);
  if (n < 0 || n > a.max_context) {
    s.bad = true;
    return s;
  }
  const int low = n > a.window ? n - a.window : 0;
  s.low = low;
  s.n = n;
  s.first = min(a.sinks, low);
  s.skip = low - s.first;
  s.seen = n - s.skip;
  if (a.aligned) {
    s.first = (s.first + 15) & ~15;
    s.skip = max((low & ~15) - s.first, 0);
    s.seen = ((n + 15) & ~15) - s.skip;
  }
  return s;
}

struct LineUnit {
  LineSeq sq;
  int b, hg;       // sequence, group of KV heads
  int T, x0, x1;   // steps of the unit, and those of this CTA
};

// The units of a CTA's span one after the other (loads and products walk on their own).
struct LineWalk {
  const LineArgs& a;
  const TreeSpan span;
  const int step_tokens;
  int b, u, x;
  LineSeq sq;

  __device__ __forceinline__ LineWalk(const LineArgs& args, const TreeSpan& s, int tokens)
      : a(args), span(s), step_tokens(tokens), b(s.b0), u(s.u0), x(s.x0) {
    sq = LineSeq{};
    if (b < a.batch) sq = line_seq(a, b);
  }
  __device__ __forceinline__ bool next(LineUnit& w) {
    for (;;) {
      if (b >= a.batch || b > span.b1 || (b == span.b1 && u > span.u1)) return false;
      if (sq.seen == 0 || u >= a.units) {
        ++b;
        u = x = 0;
        if (b < a.batch) sq = line_seq(a, b);
        continue;
      }
      w.sq = sq;
      w.b = b;
      w.hg = u;
      w.T = (sq.seen + step_tokens - 1) / step_tokens;
      w.x0 = x;
      w.x1 = b == span.b1 && u == span.u1 ? span.x1 : w.T;
      ++u;
      x = 0;
      if (w.x0 < w.x1) return true;
    }
  }
};

// All threads; sm initialised (span empty, refused 0), and a barrier since.  The caller's next barrier publishes it.
template <int kThreads>
__device__ __forceinline__ void line_schedule(const LineArgs& a, int step_tokens, TreeSched& sm) {
  constexpr int kWarps = kThreads / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int gap = a.share > 0 ? 0 : kLineGap;
  int tiles = 0;
  auto look = [&](int b) -> int {  // length of sequence b on the line
    tiles = 0;
    if (b >= a.batch) return 0;
    const LineSeq s = line_seq(a, b);
    if (s.bad && blockIdx.x == 0) raise_error(a.err, PA_DEVERR_CONTEXT_LEN);
    if (s.seen == 0) {
      if (b % gridDim.x == blockIdx.x) sm.refused = 1;
      return 0;
    }
    tiles = (s.seen + step_tokens - 1) / step_tokens;
    return a.units * (tiles + gap);
  };
  auto scan = [&](int x) {  // inclusive, over the warp
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, x, off);
      if (lane >= off) x += u;
    }
    return x;
  };
  // (a batch of up to kThreads sequences: one look and one scan for both passes)
  const bool one_chunk = a.batch <= kThreads;
  int c = look(threadIdx.x);
  int total = c;
  for (int b = threadIdx.x + kThreads; b < a.batch; b += kThreads) total += look(b);
  int v = one_chunk ? scan(c) : 0;
  const int warp_total = one_chunk ? v : __reduce_add_sync(0xffffffffu, total);  // (in lane 31)
  if (lane == 31) sm.sums[warp] = warp_total;
  __syncthreads();
  int pre = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const int x = sm.sums[w];
    if (w < warp) pre += x;
    total += x;
  }
  const int share = a.share > 0 ? a.share : max((int)(((unsigned)total + gridDim.x - 1) / gridDim.x), 1);
  const int snap = !a.split ? INT32_MAX : (a.share > 0 ? 1 : kLineGap - 1);
  const int64_t lo = (int64_t)blockIdx.x * share, hi = lo + share;
  if (threadIdx.x == 0) {
    sm.share = share;
    sm.snap = snap;
  }
  // this thread's sequence b lies at [at, at + c) of the line
  auto place = [&](int b, int64_t at) {
    if (c <= 0) return;
    const unsigned len = (unsigned)(tiles + gap);
    if (lo >= at && lo < at + c) {
      const unsigned off = (unsigned)(lo - at), u = off / len;
      sm.span.b0 = b;
      sm.span.u0 = (int)u;
      sm.span.x0 = tree_cut(off - u * len, tiles, snap);
    }
    if (hi >= at && hi < at + c) {
      const unsigned off = (unsigned)(hi - at), u = off / len;
      sm.span.b1 = b;
      sm.span.u1 = (int)u;
      sm.span.x1 = tree_cut(off - u * len, tiles, snap);
      sm.cut_start = (int)(hi - (off - u * len));
    }
  };
  if (one_chunk) {
    place(threadIdx.x, (int64_t)pre + v - c);
    return;
  }
  int carry = 0;
  for (int b0 = 0; b0 < a.batch; b0 += kThreads) {
    c = look(b0 + threadIdx.x);
    v = scan(c);
    __syncthreads();  // the sums before have been read
    if (lane == 31) sm.sums[warp] = v;
    __syncthreads();
    pre = carry;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) pre += sm.sums[w];
      carry += sm.sums[w];
    }
    place(b0 + threadIdx.x, (int64_t)pre + v - c);
  }
}

// ------------------------------------------------------------------------------------------------
// Copies and fragments
// ------------------------------------------------------------------------------------------------

// kBytes (4, 8 or 16) to shared memory, zeros when !ok; asynchronous.
template <int kBytes>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src, bool ok) {
  const int n = ok ? kBytes : 0;
  if constexpr (kBytes == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %3, %2;" ::"r"(dst), "l"(src), "r"(n), "n"(kBytes) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}

// An 8 x 8 tile of 16-bit values, two a lane, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ uint32_t lds32(uint32_t p) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(p) : "memory");
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t p) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(p) : "memory");
  return v;
}

__device__ __forceinline__ float4 lds128(uint32_t p) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(p) : "memory");
  return v;
}
__device__ __forceinline__ uint4 lds128u(uint32_t p) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(p) : "memory");
  return v;
}
__device__ __forceinline__ void sts128(uint32_t p, const float4& v) {
  asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(p), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w) : "memory");
}
__device__ __forceinline__ void sts64(uint32_t p, float x, float y) {
  asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(p), "f"(x), "f"(y) : "memory");
}
__device__ __forceinline__ float dot4(const float4& a, const float4& b, float c) {
  return fmaf(a.w, b.w, fmaf(a.z, b.z, fmaf(a.y, b.y, fmaf(a.x, b.x, c))));
}

// (x & a) | b
__device__ __forceinline__ uint32_t and_or(uint32_t x, uint32_t a, uint32_t b) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(r) : "r"(x), "r"(a), "r"(b));
  return r;
}

// a - b of two bf16 pairs.
__device__ __forceinline__ uint32_t sub_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

__device__ __forceinline__ uint32_t add_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// D = A * B of fp16 values.
__device__ __forceinline__ void mma_16816_of(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                             uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// Nibble k (0 .. 3) of both halves of w as bf16: 128 + code.
__device__ __forceinline__ uint32_t code_bf16(uint32_t w, int k) {
  return and_or(k == 0 ? w : w >> (4 * k), 0x000f000fu, 0x43004300u);
}
constexpr float kCodeBias = 128.f;  // of code_bf16

// Weights are formed 2^8 lower (sums and accumulators alike; the quotient is the same), so that the largest is 1 and its
// product with the largest values stays finite.
constexpr float kLineLift = -8.f;

// A softmax row's state: a lane has heads 2 tig and 2 tig + 1 of every 8 (columns of the transposed products).
template <int NT>
struct LineState {
  float sc[NT][2];  // exponent (base 2) of a weight per unit of score
  float m[NT][2];   // stabiliser (a score), the same in the lanes of a column
  float l[NT][2];   // this lane's share of the sum
};

// Weights of a step: s[nt][0..1] token g, [2..3] token g + 8 (rows), heads 2 tig, 2 tig + 1 (columns); ok0, ok1: whether
// the two tokens exist.  Scores become weights; where a stabiliser moved (a weight would pass 2^kGrow), or `more` of a lane
// asked for it, `rescale(nt, f0, f1, x)` is called with the factors of the columns' accumulators and the logarithms (base 2)
// of the column's weights.
template <int NT, int kGrow, typename Rescale>
__device__ __forceinline__ void line_softmax(float (&s)[NT][4], bool ok0, bool ok1, float lift, LineState<NT>& st,
                                             bool more, Rescale rescale) {
  float x[NT][4];
  bool move = more;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (!(i < 2 ? ok0 : ok1)) s[nt][i] = -INFINITY;
      x[nt][i] = (s[nt][i] - st.m[nt][i & 1]) * st.sc[nt][i & 1];
      move |= !(x[nt][i] <= (float)kGrow);  // (also at the start, and for NaN)
    }
  if (__any_sync(0xffffffffu, move)) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float f[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        // (at least the lowest number where there is a token: what saw only scores of -inf is told from what saw none)
        float mx = fmaxf(ok0 ? fmaxf(s[nt][e], -FLT_MAX) : -INFINITY, ok1 ? fmaxf(s[nt][2 + e], -FLT_MAX) : -INFINITY);
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
        const float old = st.m[nt][e], m = fmaxf(old, mx);
        f[e] = old == m ? 1.f : fast_exp2((old - m) * st.sc[nt][e]);
        st.m[nt][e] = m;
        st.l[nt][e] *= f[e];
        const float base = m == -INFINITY ? 0.f : m;
        x[nt][e] = (s[nt][e] - base) * st.sc[nt][e];
        x[nt][2 + e] = (s[nt][2 + e] - base) * st.sc[nt][e];
      }
      rescale(nt, f[0], f[1], x[nt]);
    }
  }
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float p = fast_exp2(lift == 0.f ? x[nt][i] : x[nt][i] + lift);
      s[nt][i] = p;
      st.l[nt][i & 1] += p;
    }
}

// ------------------------------------------------------------------------------------------------
// 16-bit pools
// ------------------------------------------------------------------------------------------------
// Bound by HBM (and, in short calls, by what does not shrink with the bytes: start, schedule, first loads, join).  kTma
// (block sizes that are multiples of 16): a warp's step is a sub-tile of 16 keys of one block, loaded by lane 0 in TMA boxes
// of 16 keys by 64 columns; otherwise its 16 tokens lie anywhere, and every lane copies parts of two of them.  32 / 8 heads,
// head_dim 128, bf16: 64 requests behind a window of 1,024 and 4 (260 MB) take 54 us by TMA, 59 by cp.async; 16 behind
// 8,192 and 64 (541 MB) 91 us (6.0 TB/s) and 117.
template <typename T, int D, int NT, bool kTmaBoxes>
struct FullRows {
  using Out = T;
  static constexpr bool kTma = kTmaBoxes;
  using Row = int64_t;  // offset of a row
  static constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
  static constexpr int kWarps = 4, kCtas = 3;
  static constexpr int kStages = D == 128 ? 2 : 4;
  static constexpr int kRow = 2 * D;             // bytes of a token
  static constexpr int kStage = 2 * 16 * kRow;   // K, then V
  static constexpr int kExtra = 0;               // shared memory of a warp besides its ring
  static constexpr float kLift = kBf16 ? kLineLift : 7.f;
  static constexpr bool kQuads = false;  // whether accumulators i .. i + 3 hold neighbouring dimensions
  static constexpr int kAcc = D / 16;

  const T* k;
  const T* v;
  uint32_t q[NT][D / 16][2];

  __device__ __forceinline__ FullRows(const LineArgs& a, uint32_t, int)
      : k(static_cast<const T*>(a.k)), v(static_cast<const T*>(a.v)) {}

  // 8-element chunk c of token t of an operand, in its place (ldmatrix reads eight rows of a chunk without conflicts)
  // (a TMA box puts 64 columns of the 16 tokens together, with the 128-byte swizzle)
  static __device__ __forceinline__ uint32_t at(int t, int c) {
    return kTma ? (uint32_t)((c >> 3) * 2048 + t * 128 + (((c & 7) ^ (t & 7)) << 4))
                : (uint32_t)(t * kRow + ((c ^ (t & 7)) << 4));
  }

  // kTma: the boxes of KV head h, block `block`, from token `token` of it on (one lane).
  static __device__ __forceinline__ void load_boxes(uint8_t* st, const LineMaps& maps, int block, int token,
                                                    int h, uint64_t* bar, uint64_t policy) {
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
      tma_load_3d_hint(st + i * 2048, &maps.k, h * D + i * 64, token, block, bar, policy);
      tma_load_3d_hint(st + 16 * kRow + i * 2048, &maps.v, h * D + i * 64, token, block, bar, policy);
    }
  }
  // kTma: zeros in the V rows of tokens that do not exist (whatever lies there times a weight of 0 has to be 0).
  static __device__ __forceinline__ void clear_rows(uint8_t* st, int lane, unsigned exist) {
    for (int i = lane; i < 16 * (D / 8); i += 32) {
      const int t = i / (D / 8);
      if (!((exist >> t) & 1u)) *reinterpret_cast<uint4*>(st + 16 * kRow + at(t, i % (D / 8))) = make_uint4(0, 0, 0, 0);
    }
    __syncwarp();
  }

  // tokens r and r + 8 of the step (r = lane / 4), rows `row` of the pools (element offsets)
  __device__ __forceinline__ void load(const LineArgs& a, uint32_t st, int lane, const int64_t (&row)[2],
                                       const bool (&ok)[2]) const {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int t = (lane >> 2) + 8 * h;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const int c = (lane & 3) + 4 * i;
        copy_async<16>(st + at(t, c), k + row[h] + 8 * c, ok[h]);
        copy_async<16>(st + 16 * kRow + at(t, c), v + row[h] + 8 * c, ok[h]);
      }
    }
  }
  // (block, token in it) of KV head h as an offset
  static __device__ __forceinline__ int64_t row_of(const LineArgs& a, int block, int token, int h) {
    return block * a.block_stride + (int64_t)(token * a.n_kv_heads + h) * D;
  }

  __device__ __forceinline__ void query(const LineArgs& a, int64_t head0, int lane, LineState<NT>& ls) {
    const int g = lane >> 2, tig = lane & 3;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const bool have = nt * 8 + g < a.group;
      const T* p = static_cast<const T*>(a.q) + (head0 + nt * 8 + g) * D + 2 * tig;
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          q[nt][ks][h] = have ? (uint32_t)ld_s32(reinterpret_cast<const int32_t*>(p + ks * 16 + 8 * h)) : 0u;
    }
  }

  __device__ __forceinline__ void step(uint32_t st, int lane, bool ok0, bool ok1, LineState<NT>& ls,
                                       float (&o)[NT][kAcc][4]) {
    float s[NT][4], s2[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) s[nt][i] = s2[nt][i] = 0.f;
    const int mi = lane >> 3, r = lane & 7;
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
      uint32_t x[4];
      ldsm_x4(st + at(r + 8 * (mi & 1), 2 * ks + (mi >> 1)), x[0], x[1], x[2], x[3]);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
        mma_16816<kBf16>(ks & 1 ? s2[nt] : s[nt], x[0], x[1], x[2], x[3], q[nt][ks][0], q[nt][ks][1]);
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) s[nt][i] += s2[nt][i];
    line_softmax<NT, 8>(s, ok0, ok1, kLift, ls, false, [&](int nt, float f0, float f1, const float (&)[4]) {
#pragma unroll
      for (int i = 0; i < kAcc; ++i) {
        o[nt][i][0] *= f0, o[nt][i][2] *= f0;
        o[nt][i][1] *= f1, o[nt][i][3] *= f1;
      }
    });
    uint32_t p[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int h = 0; h < 2; ++h) p[nt][h] = transpose8(pack2<kBf16>(s[nt][2 * h], s[nt][2 * h + 1]));
#pragma unroll
    for (int mt = 0; mt < kAcc; ++mt) {
      uint32_t x[4];
      ldsm_x4_t(st + 16 * kRow + at(r + 8 * (mi >> 1), 2 * mt + (mi & 1)), x[0], x[1], x[2], x[3]);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) mma_16816<kBf16>(o[nt][mt], x[0], x[1], x[2], x[3], p[nt][0], p[nt][1]);
    }
  }
  __device__ __forceinline__ void finish(LineState<NT>&, float (&)[NT][kAcc][4]) const {}
  // dimension of accumulator i, element pair h (rows g and g + 8)
  static __device__ __forceinline__ int dim_of(int i, int h, int g) { return 16 * i + g + 8 * h; }
};

// ------------------------------------------------------------------------------------------------
// fp32 pools: products on CUDA cores, in 32 bits throughout.  A lane has the scores of its two tokens and two heads
// (16 products for four 16-byte reads), and of its two heads D / 8 dimensions of the output; weights pass through
// shared memory.  Bound by latency, one warp a scheduler (issue 34 %, DRAM 41 % busy): a third of its time goes into waits for
// rows and shared memory, a tenth into issuing the copies; five or eight warps with two stages each take as long.  64
// requests behind a window of 1,024 and 4, 32 / 8 heads, head_dim 128 take 160 us (3.3 TB/s).
// ------------------------------------------------------------------------------------------------
template <int D, int NT>
struct FloatRows {
  static constexpr bool kTma = false;
  using Out = float;
  using Row = int64_t;
  static constexpr int kWarps = 4, kCtas = 1;
  static constexpr int kStages = D == 128 ? (NT == 2 ? 2 : 3) : 4;
  static constexpr int kRow = 4 * D;
  static constexpr int kStage = 2 * 16 * kRow;
  static constexpr int kQuery = NT * 8 * kRow;               // a warp's queries
  static constexpr int kExtra = kQuery + NT * 16 * 8 * 4;    // and the weights of a step, [nt][token][head]
  static constexpr float kLift = kLineLift;
  static constexpr bool kQuads = false;
  static constexpr int kAcc = D / 16;

  const float* k;
  const float* v;
  uint32_t own;

  __device__ __forceinline__ FloatRows(const LineArgs& a, uint32_t extra, int)
      : k(static_cast<const float*>(a.k)), v(static_cast<const float*>(a.v)), own(extra) {}

  // 4-element chunk c of token (or head) t: rows of a chunk read together lie in different banks
  static __device__ __forceinline__ uint32_t at(int t, int c) { return (uint32_t)(t * kRow + ((c ^ (t & 7)) << 4)); }

  __device__ __forceinline__ void load(const LineArgs&, uint32_t st, int lane, const int64_t (&row)[2],
                                       const bool (&ok)[2]) const {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int t = (lane >> 2) + 8 * h;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        const int c = (lane & 3) + 4 * i;
        copy_async<16>(st + at(t, c), k + row[h] + 4 * c, ok[h]);
        copy_async<16>(st + 16 * kRow + at(t, c), v + row[h] + 4 * c, ok[h]);
      }
    }
  }
  static __device__ __forceinline__ int64_t row_of(const LineArgs& a, int block, int token, int h) {
    return block * a.block_stride + (int64_t)(token * a.n_kv_heads + h) * D;
  }

  __device__ __forceinline__ void query(const LineArgs& a, int64_t head0, int lane, LineState<NT>& ls) {
    __syncwarp();
    for (int i = lane; i < NT * 8 * (D / 4); i += 32) {
      const int h = i / (D / 4), c = i % (D / 4);
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      if (h < a.group) x = *reinterpret_cast<const float4*>(static_cast<const float*>(a.q) + (head0 + h) * D + 4 * c);
      sts128(own + at(h, c), x);
    }
    __syncwarp();
  }

  __device__ __forceinline__ void step(uint32_t st, int lane, bool ok0, bool ok1, LineState<NT>& ls,
                                       float (&o)[NT][kAcc][4]) {
    const int g = lane >> 2, tig = lane & 3;
    float s[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) s[nt][i] = 0.f;
#pragma unroll 4
    for (int c = 0; c < D / 4; ++c) {
      const float4 k0 = lds128(st + at(g, c)), k1 = lds128(st + at(g + 8, c));
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float4 x = lds128(own + at(nt * 8 + 2 * tig + e, c));
          s[nt][e] = dot4(x, k0, s[nt][e]);
          s[nt][2 + e] = dot4(x, k1, s[nt][2 + e]);
        }
    }
    line_softmax<NT, 8>(s, ok0, ok1, kLift, ls, false, [&](int nt, float f0, float f1, const float (&)[4]) {
#pragma unroll
      for (int i = 0; i < kAcc; ++i) {
        o[nt][i][0] *= f0, o[nt][i][2] *= f0;
        o[nt][i][1] *= f1, o[nt][i][3] *= f1;
      }
    });
    const uint32_t ps = own + kQuery;
    __syncwarp();
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int h = 0; h < 2; ++h) sts64(ps + (nt * 16 + g + 8 * h) * 32 + 8 * tig, s[nt][2 * h], s[nt][2 * h + 1]);
    __syncwarp();
#pragma unroll 4
    for (int t = 0; t < 16; ++t) {
      float4 x[D / 32];
#pragma unroll
      for (int i = 0; i < D / 32; ++i) x[i] = lds128(st + 16 * kRow + at(t, g + 8 * i));
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const uint2 w = lds64(ps + (nt * 16 + t) * 32 + 8 * tig);
        const float p0 = __uint_as_float(w.x), p1 = __uint_as_float(w.y);
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {  // dimensions 32 i + 4 g .. + 3: accumulators 2 i and 2 i + 1
          float(&u)[4] = o[nt][2 * i];
          float(&y)[4] = o[nt][2 * i + 1];
          u[0] = fmaf(p0, x[i].x, u[0]), u[1] = fmaf(p1, x[i].x, u[1]);
          u[2] = fmaf(p0, x[i].y, u[2]), u[3] = fmaf(p1, x[i].y, u[3]);
          y[0] = fmaf(p0, x[i].z, y[0]), y[1] = fmaf(p1, x[i].z, y[1]);
          y[2] = fmaf(p0, x[i].w, y[2]), y[3] = fmaf(p1, x[i].w, y[3]);
        }
      }
    }
  }
  __device__ __forceinline__ void finish(LineState<NT>&, float (&)[NT][kAcc][4]) const {}
  static __device__ __forceinline__ int dim_of(int i, int h, int g) { return 32 * (i >> 1) + 4 * g + 2 * (i & 1) + h; }
};

// ------------------------------------------------------------------------------------------------
// The 4-bit cache
// ------------------------------------------------------------------------------------------------

// What both forms share: a step's codes, scales and zeros in shared memory.
template <int D>
struct PackedStage {
  static constexpr int kGroups = D / kQ4Group;
  static constexpr int kRow = D / 2;                // bytes of a token's codes
  static constexpr int kPair = 4 * kGroups;         // and of its scales and zeros
  static constexpr int kParams = 2 * 16 * kRow;     // K codes, V codes, K pairs, V pairs
  static constexpr int kVParams = kParams + 16 * kPair;
  static constexpr int kStage = kParams + 2 * 16 * kPair;
  static constexpr int kPiece = kRow / 4;           // a lane copies a quarter of a token's codes
  using Row = uint32_t;  // number of a row; more than 2^32 rows do not fit the memory, and the host refuses them

  const uint8_t *kc, *vc, *pairs;  // this lane's piece of row 0
  uint32_t dk, dv, dp;             // and where pieces of its first token go

  // Byte x of the codes of the token in place t: halves of 32 bytes trade places in every second pair of rows, so that
  // four rows' halves lie in different banks.
  static __device__ __forceinline__ uint32_t at(int t, int x) {
    return (uint32_t)(t * kRow + (kGroups == 2 ? x ^ ((t & 2) << 4) : x));
  }
  // Place of token t's V codes: even tokens first, because a lane's tokens of a product are two apart.
  static __device__ __forceinline__ int v_place(int t) { return (t & 8) | ((t & 1) << 2) | ((t >> 1) & 3); }

  __device__ __forceinline__ PackedStage(const LineArgs& a, int lane) {
    const int c = lane & 3, t = lane >> 2;
    kc = static_cast<const uint8_t*>(a.k) + c * kPiece;
    vc = static_cast<const uint8_t*>(a.v) + c * kPiece;
    pairs = static_cast<const uint8_t*>(c & 2 ? a.v_params : a.k_params);
    dk = at(t, c * kPiece);
    dv = 16 * kRow + at(v_place(t), c * kPiece);
    dp = (c & 2 ? kVParams : kParams) + (t + 8 * (c & 1)) * kPair;
  }
  __device__ __forceinline__ void load(uint32_t st, int lane, const Row (&row)[2], const bool (&ok)[2]) const {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      copy_async<kPiece>(st + dk + 8 * h * kRow, kc + (uint64_t)row[h] * kRow, ok[h]);
      copy_async<kPiece>(st + dv + 8 * h * kRow, vc + (uint64_t)row[h] * kRow, ok[h]);
    }
    // K's and V's pairs of the two tokens, one of the four a lane
    copy_async<kPair>(st + dp, pairs + (uint64_t)(lane & 1 ? row[1] : row[0]) * kPair, lane & 1 ? ok[1] : ok[0]);
  }
  static __device__ __forceinline__ Row row_of(const LineArgs& a, int block, int token, int h) {
    return ((Row)block * (Row)a.block_size + (Row)token) * (Row)a.n_kv_heads + (Row)h;
  }
};

// bf16 and fp16 queries: every operand is fp16, and the codes of two values become one by a single AND: bits 0-3 of a
// half are the number code * 2^-24, bits 4-7 code * 2^-20 (what the words hold above them comes down by one shift).
//
// Queries.  A head's values are multiplied by the power of two that takes their largest to 2^14 .. 2^15, and become fp16; those
// that meet codes in bits 4-7 are taken 16 times smaller, the largest to 2^10 or more.  fp16's smallest step, 2^-24, holds
// the 8 bits of bf16 from 2^-17 on and the 11 of fp16 from 2^-14 on: smaller values than 2^-27 and 2^-24 of the largest are
// rounded, by 2^-25 or 2^-35 of it.  With c, z, s a group's codes, zero and scale: score = sum over groups of
// s * (sum q c - z * sum q).
//
// Values.  weight * scale is rounded to fp16 after a factor of the head's and the group's own, chosen so that the largest
// product so far lies at 2 or more: fp16's smallest step is 2^-25 of it or less, and rounds by half of that.  The factor is
// looked at again, with the stabiliser's vote, where a scale passes 2^11 over it (a weight may be 2^kGrow, and the product
// has to fit): it is taken down to products of 2 .. 4 if need be, accumulators with it.  It grows as a stabiliser
// that moves takes the products down.  So a large scale of a small weight costs the others nothing.
// O = C (w s) - z (w s): the second product once for all dimensions of a group.
//
// A sum's summands are aligned with the largest exponent of their operands and cut off 24 bits below it, and a code of bits 0-3
// lies 2^10 below what its operand's exponent stands for: of 16 products and a sum each may lose 2^-14 of the largest weight
// times scale, per code's unit (measured 2^-12.4 of a scale where all values are 0; fp16's own half step is 2^-11).
//
// Bound by instructions: 443 for 16 tokens of a KV head at head_dim 128, half of them on the integer pipe, issued at 0.6 a
// clock by the 16 warps that the registers allow (more warps at fewer registers, and the next step's scores next to this
// one's values, spill and are slower).  32 / 8 heads: 64 requests of 512 to 4,096 tokens (171 MB) take 57 us, 4 of 32,768 to
// 131,000 (378 MB) 110 us.
template <typename T, int D, int NT>
struct PackedRows : PackedStage<D> {
  static constexpr bool kTma = false;
  using Out = T;
  using Stage = PackedStage<D>;
  using typename Stage::Row;
  using Stage::kGroups, Stage::kRow, Stage::kPair, Stage::kParams, Stage::kVParams, Stage::at;
  static constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
  static constexpr int kWarps = 8, kCtas = NT == 2 ? 1 : 2;
  static constexpr int kStages = 4;
  static constexpr int kExtra = 0;
  static constexpr float kLift = 0.f;
  static constexpr bool kQuads = true;
  static constexpr int kAcc = D / 16;
  static constexpr int kGrow = 4;
  static constexpr float kMostVk = 8.50705917302346159e37f;     // 2^126
  static constexpr float kMostScale = 1.06338239662793269e37f;  // 2^123: times a weight of 2^kGrow it is finite

  uint32_t q[NT][kGroups][4][2];
  float sum_q[NT][kGroups][2];  // sums of a group's query values, heads 2 tig, 2 tig + 1, times 2^-24
  float unit[NT][2];            // score of a head per unit of the above
  float vk[NT][kGroups][2];     // the factor of a head's products of weights and scales
  float most;                   // the largest scale that all of these allow
  float oz[NT][kGroups][4];     // sums of weights times scales times zeros (rows alike) times 2^-24
  uint32_t kb, vb, pb, zb;      // this lane's reads: codes of K and V, pairs, zeros

  __device__ __forceinline__ PackedRows(const LineArgs& a, uint32_t, int lane) : Stage(a, lane) {
    const int g = lane >> 2, tig = lane & 3;
    kb = at(g, 8 * tig);
    vb = 16 * kRow + at(tig, 4 * g);  // (place of token 2 tig)
    pb = kParams + g * kPair;
    zb = kVParams + 2 * tig * kPair;
  }
  __device__ __forceinline__ void load(const LineArgs&, uint32_t st, int lane, const Row (&row)[2],
                                       const bool (&ok)[2]) const {
    Stage::load(st, lane, row, ok);
  }
  // the other half of 32 bytes (group 1) of a row of codes
  static __device__ __forceinline__ uint32_t half(uint32_t at0, int gr) { return gr ? at0 ^ 32u : at0; }

  // Lane (g, tig) has the values of dimensions 16 tig .. + 15 of each group of head g; product j of a group takes those
  // at j and j + 4 (the low and the high half of a word of codes), and at j + 8 and j + 12.
  __device__ __forceinline__ void query(const LineArgs& a, int64_t head0, int lane, LineState<NT>& ls) {
    const int g = lane >> 2, tig = lane & 3;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const bool have = nt * 8 + g < a.group;
      const T* p = static_cast<const T*>(a.q) + (head0 + nt * 8 + g) * D + 16 * tig;
      float x[kGroups][16];
      float top = 0.f;
#pragma unroll
      for (int gr = 0; gr < kGroups; ++gr) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint4 v = have ? *reinterpret_cast<const uint4*>(p + gr * kQ4Group + 8 * i) : make_uint4(0, 0, 0, 0);
          Elt<T>::unpack(v, *reinterpret_cast<float(*)[8]>(&x[gr][8 * i]));
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) top = fmaxf(top, fabsf(x[gr][i]));
      }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // 2^(14 - exponent); an infinite query has scores that are not finite whatever the factor
      const int e = min(max((int)(__float_as_uint(top) >> 23), 27), 254);
      const float f = __uint_as_float((uint32_t)(127 + 14 + 127 - e) << 23);
      const float unit_g = __uint_as_float((uint32_t)min(e + 10, 254) << 23);  // 2^24 / f
#pragma unroll
      for (int gr = 0; gr < kGroups; ++gr) {
        float part = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float step = j & 1 ? 0.0625f : 1.f;
            const uint32_t both = pack2<false>(x[gr][8 * h + j] * f * step, x[gr][8 * h + j + 4] * f * step);
            q[nt][gr][j][h] = both;
            const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&both));
            part = fmaf(v.x + v.y, 1.f / step, part);
          }
        part += __shfl_xor_sync(0xffffffffu, part, 1);
        part += __shfl_xor_sync(0xffffffffu, part, 2);
        part *= 1.f / 16777216.f;
#pragma unroll
        for (int i = 0; i < 2; ++i) sum_q[nt][gr][i] = __shfl_sync(0xffffffffu, part, (2 * tig + i) * 4);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        unit[nt][i] = __shfl_sync(0xffffffffu, unit_g, (2 * tig + i) * 4);
        ls.sc[nt][i] = fminf(ls.sc[nt][i] * unit[nt][i], FLT_MAX);
      }
    }
    most = 0.f;
#pragma unroll
    for (int gr = 0; gr < kGroups; ++gr) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        vk[nt][gr][0] = vk[nt][gr][1] = kMostVk;
#pragma unroll
        for (int k = 0; k < 4; ++k) oz[nt][gr][k] = 0.f;
      }
    }
  }

  __device__ __forceinline__ void step(uint32_t st, int, bool ok0, bool ok1, LineState<NT>& ls,
                                       float (&o)[NT][kAcc][4]) {
    // ---- scores ----
    uint32_t pair[2][kGroups];  // (scale, zero) of tokens g and g + 8
    auto read_pairs = [&](uint32_t p) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if constexpr (kGroups == 2) {
          const uint2 v = lds64(p + 8 * h * kPair);
          pair[h][0] = v.x, pair[h][1] = v.y;
        } else {
          pair[h][0] = lds32(p + 8 * h * kPair);
        }
      }
    };
    read_pairs(st + pb);
    float s[NT][4];
#pragma unroll
    for (int gr = 0; gr < kGroups; ++gr) {
      uint2 w[2];  // 16 codes of tokens g and g + 8
#pragma unroll
      for (int h = 0; h < 2; ++h) w[h] = lds64(st + half(kb, gr) + 8 * h * kRow);
      float dot[NT][4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t mask = j & 1 ? 0x00f000f0u : 0x000f000fu;
        if (j == 2) {
#pragma unroll
          for (int h = 0; h < 2; ++h) w[h].x >>= 8, w[h].y >>= 8;
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          if (j == 0)
            mma_16816_of(dot[nt], w[0].x & mask, w[1].x & mask, w[0].y & mask, w[1].y & mask, q[nt][gr][j][0],
                         q[nt][gr][j][1]);
          else
            mma_16816<false>(dot[nt], w[0].x & mask, w[1].x & mask, w[0].y & mask, w[1].y & mask, q[nt][gr][j][0],
                             q[nt][gr][j][1]);
        }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t pr = pair[i >> 1][gr];
          const float d = fmaf(-q4_zero(pr), sum_q[nt][gr][i & 1], dot[nt][i]);
          s[nt][i] = gr == 0 ? q4_scale(pr) * d : fmaf(q4_scale(pr), d, s[nt][i]);
        }
    }
    // ---- weights ----
    read_pairs(st + pb + 16 * kPair);
    bool large = false;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int gr = 0; gr < kGroups; ++gr) large |= q4_scale(pair[h][gr]) > most;
    line_softmax<NT, kGrow>(s, ok0, ok1, kLift, ls, large, [&](int nt, float f0, float f1, const float (&x)[4]) {
#pragma unroll
      for (int gr = 0; gr < kGroups; ++gr) {
        float g[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          // (no weight of this step is above 1, and the products so far shrank by f; approximate quotients, since exact ones
          // cost a unit 1 to 5 us in code that runs once)
          const float f = e ? f1 : f0, old = vk[nt][gr][e];
          float top = fmaxf(fast_exp2(x[e]) * q4_scale(pair[0][gr]), fast_exp2(x[2 + e]) * q4_scale(pair[1][gr]));
#pragma unroll
          for (int off = 4; off < 32; off <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
          float now = fminf(__fdividef(old, f), kMostVk);
          if (top * now >= 4.f) now = __uint_as_float((uint32_t)(255 - (int)(__float_as_uint(top) >> 23)) << 23);
          vk[nt][gr][e] = now;
          g[e] = f == 0.f ? 0.f : f * __fdividef(now, old);
        }
#pragma unroll
        for (int i = 4 * gr; i < 4 * gr + 4; ++i) {
          o[nt][i][0] *= g[0], o[nt][i][2] *= g[0];
          o[nt][i][1] *= g[1], o[nt][i][3] *= g[1];
        }
        oz[nt][gr][0] *= g[0], oz[nt][gr][2] *= g[0];
        oz[nt][gr][1] *= g[1], oz[nt][gr][3] *= g[1];
        most = fminf(nt == 0 && gr == 0 ? kMostScale : most, 2048.f / fmaxf(vk[nt][gr][0], vk[nt][gr][1]));
      }
    });
    // ---- values ----
    // tokens 2 tig and 2 tig + 1, then those 8 further on: the zeros of both as halves of a word, whole numbers
    uint32_t zero[2][kGroups];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t za[kGroups], zc[kGroups];
      if constexpr (kGroups == 2) {
        const uint4 v = lds128u(st + zb + 8 * h * kPair);
        za[0] = v.x, za[1] = v.y, zc[0] = v.z, zc[1] = v.w;
      } else {
        const uint2 v = lds64(st + zb + 8 * h * kPair);
        za[0] = v.x, zc[0] = v.y;
      }
#pragma unroll
      for (int gr = 0; gr < kGroups; ++gr)  // (128 + zero in bf16 has it in its low bits)
        zero[h][gr] = add_bf16x2(__byte_perm(za[gr], zc[gr], 0x7632), 0x43004300u) & 0x000f000fu;
    }
#pragma unroll
    for (int gr = 0; gr < kGroups; ++gr) {
      uint32_t p[NT][2];  // weights times scales, transposed: rows heads, columns tokens
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          p[nt][h] = transpose8(pack2<false>(s[nt][2 * h] * q4_scale(pair[h][gr]) * vk[nt][gr][0],
                                             s[nt][2 * h + 1] * q4_scale(pair[h][gr]) * vk[nt][gr][1]));
      uint32_t m[2][2];  // codes, the tokens of a pair in the halves of a word
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t ca = lds32(st + half(vb, gr) + 8 * h * kRow), cb = lds32(st + half(vb, gr) + (8 * h + 4) * kRow);
        m[h][0] = __byte_perm(ca, cb, 0x5410);
        m[h][1] = __byte_perm(ca, cb, 0x7632);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t mask = j & 1 ? 0x00f000f0u : 0x000f000fu;
        if (j == 2) {
#pragma unroll
          for (int h = 0; h < 2; ++h) m[h][0] >>= 8, m[h][1] >>= 8;
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          mma_16816<false>(o[nt][4 * gr + j], m[0][0] & mask, m[0][1] & mask, m[1][0] & mask, m[1][1] & mask, p[nt][0],
                           p[nt][1]);
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
        mma_16816<false>(oz[nt][gr], zero[0][gr], zero[0][gr], zero[1][gr], zero[1][gr], p[nt][0], p[nt][1]);
    }
  }
  // Scores and values in their own units.
  __device__ __forceinline__ void finish(LineState<NT>& ls, float (&o)[NT][kAcc][4]) const {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int e = 0; e < 2; ++e)
        if (ls.m[nt][e] != -INFINITY) ls.m[nt][e] = fmaxf(ls.m[nt][e] * unit[nt][e], -FLT_MAX);
#pragma unroll
      for (int i = 0; i < kAcc; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k)
          o[nt][i][k] = fmaf(o[nt][i][k], i & 1 ? 1048576.f : 16777216.f, -16777216.f * oz[nt][i / 4][k]) *
                        (1.f / vk[nt][i / 4][k & 1]);
    }
  }
  static __device__ __forceinline__ int dim_of(int i, int h, int g) {
    return kQ4Group * (i / 4) + 8 * g + (i & 3) + 4 * h;
  }
};

// fp32 queries: three bf16 parts of 8 bits each that make the value, times (128 + code) - (128 + zero) in bf16, which are
// exact; weight * scale in three parts too.  A step's sums are formed by themselves and added up by rounded additions (the
// tensor core truncates its sums).  The serving batch above takes 79 us.
template <int D, int NT>
struct PackedWideRows : PackedStage<D> {
  static constexpr bool kTma = false;
  using Out = float;
  using Stage = PackedStage<D>;
  using typename Stage::Row;
  using Stage::kGroups, Stage::kRow, Stage::kPair, Stage::kParams, Stage::kVParams, Stage::at, Stage::v_place;
  static constexpr int kParts = 3;
  static constexpr int kWarps = 8, kCtas = 1;
  static constexpr int kStages = 4;
  static constexpr int kExtra = 0;
  static constexpr float kLift = kLineLift;
  static constexpr bool kQuads = true;
  static constexpr int kAcc = D / 16;

  uint32_t q[NT][kParts][kGroups][4][2];

  __device__ __forceinline__ PackedWideRows(const LineArgs& a, uint32_t, int lane) : Stage(a, lane) {}
  __device__ __forceinline__ void load(const LineArgs&, uint32_t st, int lane, const Row (&row)[2],
                                       const bool (&ok)[2]) const {
    Stage::load(st, lane, row, ok);
  }

  // (dimensions as above)
  __device__ __forceinline__ void query(const LineArgs& a, int64_t head0, int lane, LineState<NT>&) {
    const int g = lane >> 2, tig = lane & 3;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const bool have = nt * 8 + g < a.group;
      const float* p = static_cast<const float*>(a.q) + (head0 + nt * 8 + g) * D + 16 * tig;
#pragma unroll
      for (int gr = 0; gr < kGroups; ++gr) {
        float x[16];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4 v = have ? *reinterpret_cast<const float4*>(p + gr * kQ4Group + 4 * i) : make_float4(0, 0, 0, 0);
          x[4 * i] = v.x, x[4 * i + 1] = v.y, x[4 * i + 2] = v.z, x[4 * i + 3] = v.w;
        }
#pragma unroll
        for (int w = 0; w < kParts; ++w)
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h)
              q[nt][w][gr][j][h] = split(x[8 * h + j], x[8 * h + j + 4]);
      }
    }
  }
  // Two numbers as bf16; they become what is left of them, exactly.
  static __device__ __forceinline__ uint32_t split(float& u, float& v) {
    const uint32_t both = pack2<true>(u, v);
    u -= __uint_as_float(both << 16);
    v -= __uint_as_float(both & 0xffff0000u);
    return both;
  }

  __device__ __forceinline__ void step(uint32_t st, int lane, bool ok0, bool ok1, LineState<NT>& ls,
                                       float (&o)[NT][kAcc][4]) const {
    const int g = lane >> 2, tig = lane & 3;
    // ---- scores ----
    float s[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) s[nt][i] = 0.f;
#pragma unroll
    for (int gr = 0; gr < kGroups; ++gr) {
      uint2 w[2];  // 16 codes of tokens g and g + 8
      uint32_t pair[2], bias[2];  // their (scale, zero); 128 + zero, twice
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        w[h] = lds64(st + at(g + 8 * h, 32 * gr + 8 * tig));
        pair[h] = lds32(st + kParams + (g + 8 * h) * kPair + 4 * gr);
        const float b = q4_zero(pair[h]) + kCodeBias;
        bias[h] = (__float_as_uint(b) >> 16) | __float_as_uint(b);
      }
      float dot[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) dot[nt][i] = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t x[4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          x[h] = sub_bf16x2(code_bf16(w[h].x, j), bias[h]);
          x[2 + h] = sub_bf16x2(code_bf16(w[h].y, j), bias[h]);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int p = kParts - 1; p >= 0; --p)
            mma_16816<true>(d, x[0], x[1], x[2], x[3], q[nt][p][gr][j][0], q[nt][p][gr][j][1]);
#pragma unroll
          for (int i = 0; i < 4; ++i) dot[nt][i] += d[i];
        }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[nt][i] = fmaf(q4_scale(pair[i >> 1]), dot[nt][i], s[nt][i]);
    }
    line_softmax<NT, 8>(s, ok0, ok1, kLift, ls, false, [&](int nt, float f0, float f1, const float (&)[4]) {
#pragma unroll
      for (int i = 0; i < kAcc; ++i) {
        o[nt][i][0] *= f0, o[nt][i][2] *= f0;
        o[nt][i][1] *= f1, o[nt][i][3] *= f1;
      }
    });
    // ---- values ----
    const uint32_t vst = st + 16 * kRow, vps = st + kVParams;
#pragma unroll
    for (int gr = 0; gr < kGroups; ++gr) {
      // weights times scales, transposed: rows heads, columns tokens
      const float sv[2] = {q4_scale(lds32(vps + g * kPair + 4 * gr)), q4_scale(lds32(vps + (g + 8) * kPair + 4 * gr))};
      uint32_t p[NT][kParts][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float u = s[nt][2 * h] * sv[h], v = s[nt][2 * h + 1] * sv[h];
#pragma unroll
          for (int w = 0; w < kParts; ++w) p[nt][w][h] = transpose8(split(u, v));
        }
      // tokens 2 tig and 2 tig + 1, then those 8 further on: 128 + zero of both, and the codes with the tokens of a pair
      // in the halves of a word
      uint32_t bias[2], m[2][2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int t = 2 * tig + 8 * h;
        const uint32_t za = lds32(vps + t * kPair + 4 * gr), zc = lds32(vps + (t + 1) * kPair + 4 * gr);
        bias[h] = add_bf16x2(__byte_perm(za, zc, 0x7632), 0x43004300u);
        const uint32_t ca = lds32(vst + at(v_place(t), 32 * gr + 4 * g));
        const uint32_t cb = lds32(vst + at(v_place(t + 1), 32 * gr + 4 * g));
        m[h][0] = __byte_perm(ca, cb, 0x5410);
        m[h][1] = __byte_perm(ca, cb, 0x7632);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t x[4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          x[2 * h] = sub_bf16x2(code_bf16(m[h][0], j), bias[h]);
          x[2 * h + 1] = sub_bf16x2(code_bf16(m[h][1], j), bias[h]);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int w = kParts - 1; w >= 0; --w) mma_16816<true>(d, x[0], x[1], x[2], x[3], p[nt][w][0], p[nt][w][1]);
#pragma unroll
          for (int i = 0; i < 4; ++i) o[nt][4 * gr + j][i] += d[i];
        }
      }
    }
  }
  __device__ __forceinline__ void finish(LineState<NT>&, float (&)[NT][kAcc][4]) const {}
  static __device__ __forceinline__ int dim_of(int i, int h, int g) {
    return kQ4Group * (i / 4) + 8 * g + (i & 3) + 4 * h;
  }
};

// ------------------------------------------------------------------------------------------------
// The kernel
// ------------------------------------------------------------------------------------------------
template <typename Rows>
struct LineCfg {
  static constexpr int kThreads = Rows::kWarps * 32;
  static constexpr int kPad = 4;
  static constexpr int kRing = Rows::kWarps * (Rows::kStages * Rows::kStage + Rows::kExtra);
};

// Shared memory: the warps' rings (and what else a warp needs), then their states at the end of a unit, [warp][row]
// [head_dim + kPad], [warp][row] twice.
template <typename Rows, int D>
constexpr int line_smem(int group) {
  return (Rows::kTma ? 1024 : 0) + LineCfg<Rows>::kRing + Rows::kWarps * group * (D + LineCfg<Rows>::kPad + 2) * 4;
}
constexpr int kLineStatic = 512;  // the schedule, the rings' barriers


// kRuns: a warp's sums of kLineRun steps at most are formed in registers, and runs added up in shared memory.  The tensor core
// cuts its sums off where it should round: a step takes up to 2^-23 of what a sum holds from it, always in the same
// direction (131,072 tokens by one warp lost 8e-4 of the result over the 4-bit cache, whose codes are not centred, and two
// million 1.3 %); now 3e-5 at most, and sums of rounded additions have fewer summands as well.  Calls in which no CTA can
// have that many steps of a unit take the form without (4-bit serving
// batch: 57.0 us, and 58.4 by this form, which it takes with a table as wide as for 131,072 tokens).
template <typename Rows, int D, int NT, bool kRuns>
__global__ void __launch_bounds__(LineCfg<Rows>::kThreads, Rows::kCtas)
    line_decode_kernel(const LineArgs a, const __grid_constant__ LineMaps maps) {
  using T = typename Rows::Out;
  constexpr int kWarps = Rows::kWarps, kStages = Rows::kStages, kThreads = LineCfg<Rows>::kThreads;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* const smem =
      Rows::kTma ? reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023)) : smem_raw;
  __shared__ TreeSched sched;
  // kTma: a warp's ring, when its steps have landed and the position of their first key (-1: no keys)
  __shared__ uint64_t landed[Rows::kTma ? kWarps : 1][kStages];
  __shared__ int32_t step_key[Rows::kTma ? kWarps : 1][kStages];
  constexpr int kOutRow = LineCfg<Rows>::kPad + D;  // (the pad keeps the rows that a store writes in different banks)
  float* const out_o = reinterpret_cast<float*>(smem + LineCfg<Rows>::kRing);
  float* const out_m = out_o + kWarps * a.group * kOutRow;
  float* const out_l = out_m + kWarps * a.group;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int lanes_head = kWarps / a.heads;  // warps of a KV head
  const int head = warp / lanes_head, part = warp - head * lanes_head;
  const int step_tokens = 16 * lanes_head;
  if (threadIdx.x == 0) {
    sched.span = TreeSpan{a.batch, 0, 0, a.batch, 0, 0};
    sched.refused = 0;
  }
  if (Rows::kTma && lane == 0) {
    prefetch_tensormap(&maps.k);
    prefetch_tensormap(&maps.v);
    for (int s = 0; s < kStages; ++s) mbar_init(&landed[warp][s], 1);
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  __syncthreads();
  pdl_wait_primary();
  line_schedule<kThreads>(a, step_tokens, sched);
  __syncthreads();
  pdl_launch_dependents();
  const TreeSpan span = sched.span;
  if (a.split && threadIdx.x == 0) a.ws_rec[blockIdx.x] = TreeRec{0, 0, 0};

  const uint32_t ring = smem_u32(smem) + (uint32_t)(warp * (kStages * Rows::kStage + Rows::kExtra));
  Rows rows(a, ring + kStages * Rows::kStage, lane);

  // ---- the loads, kStages - 1 steps ahead (kTma: kStages, a stage is filled again as soon as it has been read) ----
  LineWalk ahead(a, span, step_tokens);
  LineUnit lu;
  lu.b = 0;
  bool more = ahead.next(lu);
  int lx = more ? lu.x0 : 0;
  const int32_t* table = a.block_table + lu.b * a.bt_stride;
  int block[2], at[2];  // block and token in it of this lane's two tokens of the next step
  bool have[2];
  unsigned oks = 0;  // two bits a step in flight: whether this lane's two tokens exist
  const uint64_t policy = Rows::kTma ? l2_policy_evict_first() : 0;  // (keys and values are read once)
  auto prefetch_queries = [&]() {  // of the unit that the loads have come to
    const int64_t head0 = (int64_t)lu.b * a.n_q_heads + (int64_t)(lu.hg * a.heads + head) * a.group;
    const int bytes = a.group * D * (int)sizeof(T);
    for (int i = lane * 128; i < bytes; i += 32 * 128)
      asm volatile("prefetch.global.L1 [%0];" ::"l"(static_cast<const char*>(a.q) + head0 * D * (int)sizeof(T) + i));
  };
  auto look = [&]() {  // table entries of the next step
#pragma unroll
    for (int h = 0; h < (Rows::kTma ? 1 : 2); ++h) {
      const int v = (lx * lanes_head + part) * 16 + (Rows::kTma ? 0 : (lane >> 2) + 8 * h);
      const int pos = v < lu.sq.first ? v : v + lu.sq.skip;
      have[h] = more && v < lu.sq.seen && (!Rows::kTma || lane == 0);
      at[h] = Rows::kTma ? pos : pos & (a.block_size - 1);
      block[h] = have[h] ? ld_s32(table + (pos >> a.block_shift)) : 0;
    }
  };
  auto load = [&](int stage) {
    if constexpr (Rows::kTma) {
      if (!more) return;
      if (lane == 0) {
        bool ok = have[0];
        if (ok && (unsigned)block[0] >= a.block_limit) {
          raise_error(a.err, PA_DEVERR_BLOCK_ID);
          ok = false;
        }
        step_key[warp][stage] = ok ? at[0] : -1;
        if (ok) {
          mbar_arrive_expect_tx(&landed[warp][stage], Rows::kStage);
          Rows::load_boxes(smem + (warp * kStages + stage) * Rows::kStage, maps, block[0], at[0] & (a.block_size - 1),
                           lu.hg * a.heads + head, &landed[warp][stage], policy);
        } else {
          mbar_arrive(&landed[warp][stage]);
        }
      }
      if (++lx == lu.x1) {
        more = ahead.next(lu);
        lx = more ? lu.x0 : 0;
        table = a.block_table + lu.b * a.bt_stride;
        if (more) prefetch_queries();
      }
      look();
      return;
    }
    if (more) {
      typename Rows::Row row[2];
      bool ok[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        ok[h] = have[h];
        if (have[h] && (unsigned)block[h] >= a.block_limit) {
          raise_error(a.err, PA_DEVERR_BLOCK_ID);
          ok[h] = false;
        }
        row[h] = ok[h] ? Rows::row_of(a, block[h], at[h], lu.hg * a.heads + head) : 0;
      }
      if constexpr (!Rows::kTma) rows.load(a, ring + stage * Rows::kStage, lane, row, ok);
      oks = oks << 2 | (ok[1] ? 2u : 0u) | (ok[0] ? 1u : 0u);
      if (++lx == lu.x1) {
        more = ahead.next(lu);
        lx = more ? lu.x0 : 0;
        table = a.block_table + lu.b * a.bt_stride;
        if (more) prefetch_queries();
      }
      look();
    } else {
      oks <<= 2;
    }
    copy_commit();
  };
  look();
#pragma unroll
  for (int s = 0; s < (Rows::kTma ? kStages : kStages - 1); ++s) load(s);

  // ---- the products ----
  LineWalk walk(a, span, step_tokens);
  LineUnit w;
  int stage = 0;
  unsigned phase = 0;  // kTma: of the ring's barriers
  bool alive = true;   // kTma: no wait has given up (if one has, the units are walked through without their keys)
  while (walk.next(w)) {
    const int64_t head0 = (int64_t)w.b * a.n_q_heads + (int64_t)(w.hg * a.heads + head) * a.group;
    const int g = lane >> 2, tig = lane & 3;
    LineState<NT> ls;
    float o[NT][Rows::kAcc][4];
    // this warp's sums to its rows in shared memory, or added to what is there (every lane has the same elements each time)
    auto store = [&](bool add) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = (warp << a.group_shift) + nt * 8 + 2 * tig + e;
          const bool here = nt * 8 + 2 * tig + e < a.group;
          float* p = out_o + r * kOutRow;
          float f_old = 0.f, f_new = 1.f, m = ls.m[nt][e], l = ls.l[nt][e];
          if (add) {
            __syncwarp();
            if (here) {
              const float before = out_m[r], most = fmaxf(before, m), base = most == -INFINITY ? 0.f : most;
              f_old = fast_exp2((before - base) * a.scale_log2);
              f_new = fast_exp2((m - base) * a.scale_log2);
              l = fmaf(out_l[r], f_old, l * f_new);
              m = most;
            }
            __syncwarp();
          }
          if (here) {
            if constexpr (Rows::kQuads) {
#pragma unroll
              for (int i = 0; i < Rows::kAcc; i += 4)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  float4* at = reinterpret_cast<float4*>(p + Rows::dim_of(i, h, g));
                  float4 v = make_float4(o[nt][i][2 * h + e], o[nt][i + 1][2 * h + e], o[nt][i + 2][2 * h + e],
                                         o[nt][i + 3][2 * h + e]);
                  if (add) {
                    const float4 y = *at;
                    v = make_float4(fmaf(y.x, f_old, v.x * f_new), fmaf(y.y, f_old, v.y * f_new),
                                    fmaf(y.z, f_old, v.z * f_new), fmaf(y.w, f_old, v.w * f_new));
                  }
                  *at = v;
                }
            } else {
#pragma unroll
              for (int i = 0; i < Rows::kAcc; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  float* at = p + Rows::dim_of(i, h, g);
                  const float v = o[nt][i][2 * h + e];
                  *at = add ? fmaf(*at, f_old, v * f_new) : v;
                }
            }
            if (g == 0) {
              out_m[r] = m;
              out_l[r] = l;
            }
          }
        }
    };
    // whether a warp has all of its head, and four neighbouring dimensions in four accumulators
    auto direct = [&]() { return Rows::kQuads && lanes_head == 1 && (!kRuns || w.x1 - w.x0 <= kLineRun); };
    int x = w.x0;
    do {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          ls.sc[nt][e] = a.scale_log2;
          ls.m[nt][e] = -INFINITY;
          ls.l[nt][e] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < Rows::kAcc; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) o[nt][i][j] = 0.f;
      }
      rows.query(a, head0, lane, ls);
      do {
        if constexpr (Rows::kTma) {
          if (alive && !__all_sync(0xffffffffu, mbar_wait(&landed[warp][stage], phase, a.err, a.epoch))) {
            alive = false;
            if (lane == 0) raise_timeout(a.err, a.epoch);
          }
          if (!alive) continue;
          const int key = step_key[warp][stage], t = lane >> 2;
          if (key >= 0) {
            auto exists = [&](int p) { return p < w.sq.n && (p >= w.sq.low || p < a.sinks); };
            bool ok0 = true, ok1 = true;
            if (key + 16 > w.sq.n || key < w.sq.low) {  // (whole steps below the sinks' end take this way too)
              ok0 = exists(key + t);
              ok1 = exists(key + t + 8);
              Rows::clear_rows(smem + (warp * kStages + stage) * Rows::kStage, lane,
                               __ballot_sync(0xffffffffu, exists(key + (lane & 15))));
            }
            rows.step(ring + stage * Rows::kStage, lane, ok0, ok1, ls, o);
          }
          fence_proxy_async_smem();
          __syncwarp();
          load(stage);
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1u;
          }
          continue;
        }
        copy_wait<kStages - 2>();
        __syncwarp();  // every lane's copies of this step are there, and the stage before has been read by all
        const unsigned ok = oks >> (2 * (kStages - 2));
        load(stage == 0 ? kStages - 1 : stage - 1);
        if constexpr (!Rows::kTma) rows.step(ring + stage * Rows::kStage, lane, ok & 1, (ok & 2) != 0, ls, o);
        stage = stage + 1 == kStages ? 0 : stage + 1;
      } while (++x < w.x1 && (!kRuns || (unsigned)(x - w.x0) % kLineRun != 0));
      // the sums in their own units, and l of all lanes
      rows.finish(ls, o);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int off = 4; off < 32; off <<= 1) ls.l[nt][e] += __shfl_xor_sync(0xffffffffu, ls.l[nt][e], off);
      if (!direct()) store(kRuns && x - w.x0 > kLineRun);
    } while (kRuns && x < w.x1);
    // ---- the unit's end ----
    const bool whole = w.x0 == 0 && w.x1 == w.T;
    const int unit_rows = a.heads << a.group_shift;
    const int64_t row0 = (int64_t)w.b * a.n_q_heads + (int64_t)w.hg * unit_rows;
    const int64_t slot0 = ((int64_t)blockIdx.x * 2 + (w.x0 == 0 ? 1 : 0)) * unit_rows;
    // four neighbouring dimensions of a row: its output, or this CTA's part of it
    auto put = [&](int r, int d, const float4& v, float M, float L) {
      if (whole) {
        const float norm = M == -INFINITY ? 0.f : 1.f / L;
        T* out = static_cast<T*>(a.out) + (row0 + r) * D + d;
        if constexpr (sizeof(T) == 4)
          *reinterpret_cast<float4*>(out) = make_float4(v.x * norm, v.y * norm, v.z * norm, v.w * norm);
        else
          *reinterpret_cast<uint2*>(out) = make_uint2(pack2<std::is_same<T, __nv_bfloat16>::value>(v.x * norm, v.y * norm),
                                                      pack2<std::is_same<T, __nv_bfloat16>::value>(v.z * norm, v.w * norm));
      } else {
        *reinterpret_cast<float4*>(a.ws_acc + (slot0 + r) * D + d) = v;
        if (d == 0) {
          a.ws_m[slot0 + r] = M;
          a.ws_l[slot0 + r] = L;
        }
      }
    };
    if (direct()) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = nt * 8 + 2 * tig + e;
          if (r < a.group) {
#pragma unroll
            for (int i = 0; i < Rows::kAcc; i += 4)
#pragma unroll
              for (int h = 0; h < 2; ++h)
                put((head << a.group_shift) + r, Rows::dim_of(i, h, g),
                    make_float4(o[nt][i][2 * h + e], o[nt][i + 1][2 * h + e], o[nt][i + 2][2 * h + e],
                                o[nt][i + 3][2 * h + e]),
                    ls.m[nt][e], ls.l[nt][e]);
          }
        }
    } else {
      // the warps of a head joined in shared memory
      __syncthreads();
      for (int i = threadIdx.x; i < unit_rows * (D / 4); i += kThreads) {
        const int r = i / (D / 4), d = i % (D / 4) * 4;
        // row r of warp 0 of its head, and how far apart the head's warps are
        const int at0 = ((r >> a.group_shift) * lanes_head << a.group_shift) + (r & (a.group - 1));
        float M = -INFINITY, L = 0.f;
        for (int k = 0; k < lanes_head; ++k) M = fmaxf(M, out_m[at0 + (k << a.group_shift)]);
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (M != -INFINITY) {
          for (int k = 0; k < lanes_head; ++k) {
            const int at = at0 + (k << a.group_shift);
            const float f = fast_exp2((out_m[at] - M) * a.scale_log2);
            const float4 x = *reinterpret_cast<const float4*>(out_o + at * kOutRow + d);
            L = fmaf(out_l[at], f, L);
            v = make_float4(fmaf(x.x, f, v.x), fmaf(x.y, f, v.y), fmaf(x.z, f, v.z), fmaf(x.w, f, v.w));
          }
        }
        put(r, d, v, M, L);
      }
      __syncthreads();
    }
    if (!whole && w.x0 == 0 && threadIdx.x == 0) {
      // the CTA that the unit's last step went to
      int last = (sched.cut_start + w.T - 1) / sched.share;
      if (tree_cut((int64_t)last * sched.share - sched.cut_start, w.T, sched.snap) == w.T) --last;
      a.ws_rec[blockIdx.x] = TreeRec{row0, unit_rows, last};
    }
  }
  copy_wait<0>();
  if constexpr (Rows::kTma) {
    // after a wait gave up: leave no copy in flight (bounded again; every stage was filled once more than it was read)
    if (!alive && lane == 0)
      for (int s = 0; s < kStages; ++s) mbar_wait(&landed[warp][s], s < stage ? phase ^ 1u : phase);
  }
  // sequences that see nothing
  if (sched.refused) {
    for (int b = blockIdx.x; b < a.batch; b += gridDim.x) {
      if (line_seq(a, b).seen != 0) continue;
      uint4* p = reinterpret_cast<uint4*>(static_cast<T*>(a.out) + (int64_t)b * a.n_q_heads * D);
      const int64_t n = (int64_t)a.n_q_heads * D * (int)sizeof(T) / 16;
      for (int64_t i = threadIdx.x; i < n; i += kThreads) p[i] = make_uint4(0, 0, 0, 0);
    }
  }
}

// ------------------------------------------------------------------------------------------------
// Units cut between CTAs, all pieces of a row (the first in the second slot of the CTA that the unit begins in, the
// others in the first slots of the CTAs after it).  A warp per row; where units are expected in many pieces (kWide: few
// sequences with long contexts), a CTA per row, whose warps take pieces in turn.
constexpr int kLjWarps = 4, kLjWideWarps = 8;
constexpr int kLjWidePieces = 12;  // (geometric means over the shapes of kLineGap: 4 to 12 alike, 24 3 % more, never 5 and 21 %)

template <typename T, int D, bool kWide>
__global__ void __launch_bounds__(32 * (kWide ? kLjWideWarps : kLjWarps)) line_join_kernel(const LineArgs a) {
  constexpr int kPer = D / 32, kWarps = kWide ? kLjWideWarps : 1;
  using Vec = typename std::conditional<kPer == 4, float4, float2>::type;
  __shared__ float s_acc[kWarps][D], s_l[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int unit_rows = a.heads << a.group_shift;
  int c = blockIdx.y;
  pdl_launch_dependents();
  pdl_wait_primary();
  if constexpr (kWide) {  // blockIdx.y: a unit; its record, if it was cut
    __shared__ int s_cta;
    if (threadIdx.x == 0) s_cta = -1;
    __syncthreads();
    for (int i = threadIdx.x; i < a.ctas; i += 32 * kWarps)
      if (a.ws_rec[i].rows > 0 && a.ws_rec[i].row0 == (int64_t)c * unit_rows) s_cta = i;
    __syncthreads();
    c = s_cta;
    if (c < 0) return;
  }
  const TreeRec rec = a.ws_rec[c];
  const int r = kWide ? blockIdx.x : blockIdx.x * kLjWarps + warp;
  if (r >= rec.rows) return;
  const int pieces = rec.last - c + 1, first = kWide ? warp : 0;
  auto piece = [&](int i) -> int64_t { return ((int64_t)(c + i) * 2 + (i == 0 ? 1 : 0)) * unit_rows + r; };
  float M = -INFINITY;
  for (int i = lane; i < pieces; i += 32) M = fmaxf(M, a.ws_m[piece(i)]);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
  const float base = M == -INFINITY ? 0.f : M;
  float L = 0.f, acc[kPer];
#pragma unroll
  for (int k = 0; k < kPer; ++k) acc[k] = 0.f;
#pragma unroll 8
  for (int i = first; i < pieces; i += kWarps) {
    const int64_t p = piece(i);
    const Vec v = *reinterpret_cast<const Vec*>(a.ws_acc + p * D + lane * kPer);
    const float f = fast_exp2((a.ws_m[p] - base) * a.scale_log2);
    L = fmaf(a.ws_l[p], f, L);
#pragma unroll
    for (int k = 0; k < kPer; ++k) acc[k] = fmaf(reinterpret_cast<const float*>(&v)[k], f, acc[k]);
  }
  T* o = static_cast<T*>(a.out) + (rec.row0 + r) * D;
  if constexpr (kWide) {
#pragma unroll
    for (int k = 0; k < kPer; ++k) s_acc[warp][lane * kPer + k] = acc[k];
    if (lane == 0) s_l[warp] = L;
    __syncthreads();
    for (int d = threadIdx.x; d < D; d += 32 * kWarps) {
      float sum = 0.f, total = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        sum += s_acc[w][d];
        total += s_l[w];
      }
      o[d] = Elt<T>::from_float(M == -INFINITY ? 0.f : sum / total);
    }
  } else {
#pragma unroll
    for (int k = 0; k < kPer; ++k) o[lane * kPer + k] = Elt<T>::from_float(M == -INFINITY ? 0.f : acc[k] / L);
  }
}

// ------------------------------------------------------------------------------------------------
namespace {

cudaLaunchConfig_t overlapped(dim3 grid, int threads, int smem, cudaStream_t s, cudaLaunchAttribute* attr) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = s;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

template <typename Rows, int D, int NT, bool kRuns>
cudaError_t launch_form(const LineArgs& a, cudaStream_t s, const LineMaps& maps) {
  constexpr int most = line_smem<Rows, D>(8 * NT);
  static_assert(most + (Rows::kTma ? kLineStatic : 256) <= 227 * 1024, "shared memory of a CTA");
  static bool attr_set[64] = {};  // per instantiation and device; idempotent, so a race is harmless
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !attr_set[dev]) {
    e = cudaFuncSetAttribute(line_decode_kernel<Rows, D, NT, kRuns>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) attr_set[dev] = true;
  }
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg =
      overlapped(dim3((unsigned)a.ctas), LineCfg<Rows>::kThreads, line_smem<Rows, D>(a.group), s, attr);
  return cudaLaunchKernelEx(&cfg, line_decode_kernel<Rows, D, NT, kRuns>, a, maps);
}
template <typename Rows, int D, int NT>
cudaError_t launch_rows(const LineArgs& a, cudaStream_t s, const LineMaps& maps = LineMaps{}) {
  return a.runs ? launch_form<Rows, D, NT, true>(a, s, maps) : launch_form<Rows, D, NT, false>(a, s, maps);
}

template <typename T, int D>
cudaError_t launch_packed(const LineArgs& a, cudaStream_t s) {
  return a.group > 8 ? launch_rows<PackedRows<T, D, 2>, D, 2>(a, s) : launch_rows<PackedRows<T, D, 1>, D, 1>(a, s);
}
template <int D>
cudaError_t launch_wide(const LineArgs& a, cudaStream_t s) {
  return a.group > 8 ? launch_rows<PackedWideRows<D, 2>, D, 2>(a, s) : launch_rows<PackedWideRows<D, 1>, D, 1>(a, s);
}
template <typename T, int D>
cudaError_t launch_full(const LineArgs& a, pa_dtype dt, cudaStream_t s) {
  if (a.aligned) {
    LineMaps maps;
    if (!encode_pool_map(&maps.k, a.k, dt, a.block_limit, a.block_size, a.n_kv_heads, D, a.block_stride) ||
        !encode_pool_map(&maps.v, a.v, dt, a.block_limit, a.block_size, a.n_kv_heads, D, a.block_stride))
      return cudaErrorInvalidValue;
    return a.group > 8 ? launch_rows<FullRows<T, D, 2, true>, D, 2>(a, s, maps)
                       : launch_rows<FullRows<T, D, 1, true>, D, 1>(a, s, maps);
  }
  return a.group > 8 ? launch_rows<FullRows<T, D, 2, false>, D, 2>(a, s) : launch_rows<FullRows<T, D, 1, false>, D, 1>(a, s);
}

template <int D>
cudaError_t launch_float(const LineArgs& a, cudaStream_t s) {
  return a.group > 8 ? launch_rows<FloatRows<D, 2>, D, 2>(a, s) : launch_rows<FloatRows<D, 1>, D, 1>(a, s);
}

template <typename Rows, int D>
int resident(int group) {
  const int fit = 228 * 1024 / (line_smem<Rows, D>(group) + kLineStatic + 1024);
  return std::max(1, std::min(fit, Rows::kCtas));
}
template <int D, int NT>
int resident_of(bool packed, pa_dtype dt, int group) {
  if (packed)
    return dt == PA_BF16   ? resident<PackedRows<__nv_bfloat16, D, NT>, D>(group)
           : dt == PA_FP16 ? resident<PackedRows<__half, D, NT>, D>(group)
                           : resident<PackedWideRows<D, NT>, D>(group);
  return dt == PA_FP32 ? resident<FloatRows<D, NT>, D>(group) : resident<FullRows<__half, D, NT, true>, D>(group);
}

template <typename T, int D, bool kWide>
cudaError_t launch_join_as(const LineArgs& a, cudaStream_t s) {
  const int rows = a.heads * a.group, warps = kWide ? kLjWideWarps : kLjWarps;
  cudaLaunchAttribute attr[1];
  const dim3 grid((unsigned)(kWide ? rows : (rows + warps - 1) / warps), (unsigned)(kWide ? a.batch * a.units : a.ctas));
  const cudaLaunchConfig_t cfg = overlapped(grid, 32 * warps, 0, s, attr);
  return cudaLaunchKernelEx(&cfg, line_join_kernel<T, D, kWide>, a);
}
template <typename T>
cudaError_t launch_join(const LineArgs& a, cudaStream_t s) {
  const bool wide = a.ctas >= (int64_t)kLjWidePieces * a.batch * a.units;
  if (a.head_dim == 64) return wide ? launch_join_as<T, 64, true>(a, s) : launch_join_as<T, 64, false>(a, s);
  return wide ? launch_join_as<T, 128, true>(a, s) : launch_join_as<T, 128, false>(a, s);
}

}  // namespace

int line_ctas(bool packed, pa_dtype dt, int head_dim, int group) {
  if (head_dim == 64) return group > 8 ? resident_of<64, 2>(packed, dt, group) : resident_of<64, 1>(packed, dt, group);
  return group > 8 ? resident_of<128, 2>(packed, dt, group) : resident_of<128, 1>(packed, dt, group);
}

cudaError_t launch_line_decode(const LineArgs& a, pa_dtype dt, bool packed, cudaStream_t s, int* launches) {
  cudaError_t e = cudaErrorInvalidValue;
  const bool d64 = a.head_dim == 64;
  if (packed) {
    if (dt == PA_BF16) e = d64 ? launch_packed<__nv_bfloat16, 64>(a, s) : launch_packed<__nv_bfloat16, 128>(a, s);
    if (dt == PA_FP16) e = d64 ? launch_packed<__half, 64>(a, s) : launch_packed<__half, 128>(a, s);
    if (dt == PA_FP32) e = d64 ? launch_wide<64>(a, s) : launch_wide<128>(a, s);
  } else {
    if (dt == PA_BF16) e = d64 ? launch_full<__nv_bfloat16, 64>(a, dt, s) : launch_full<__nv_bfloat16, 128>(a, dt, s);
    if (dt == PA_FP16) e = d64 ? launch_full<__half, 64>(a, dt, s) : launch_full<__half, 128>(a, dt, s);
    if (dt == PA_FP32) e = d64 ? launch_float<64>(a, s) : launch_float<128>(a, s);
  }
  if (e != cudaSuccess) return e;
  ++*launches;
  if (!a.split) return e;
  ++*launches;
  switch (dt) {
    case PA_BF16: return launch_join<__nv_bfloat16>(a, s);
    case PA_FP16: return launch_join<__half>(a, s);
    case PA_FP32: return launch_join<float>(a, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace pa
