// Softmax of one key tile of the tree attention's tensor-core kernels: key
// masks, row extremes and exponentials.
//
// Softcap: tanh(t) of t = s * scale / softcap comes from the first three terms of
// its series, t - t^3/3 + 2t^5/15, on the FMA pipe, whenever every score of the
// warp's tile is small enough for that; otherwise element by element.  What is cut
// off is below the next term, 17/315 |t|^7, and reaches the score times softcap;
// tiles of one row may take different forms, so it counts in full.  The series is
// taken up to |t| = 1/4 and only where softcap times that term stays below 2^-14, an
// eighth of the half step that a weight is rounded by in f16 (softcap 30: |t| <=
// 0.233; 1000: 0.142).
#pragma once

#include <math.h>

#include "pva_device.cuh"
#include "pva_tree.h"

namespace pva {
namespace tile {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kRescaleThreshold = 8.0f;  // log2 units: O is rescaled when the max grows > 2^8

// Kernels without a softcap, with one, and with one above kCapOfExp, where 3e-7 of
// it passes 2^-14.  Taking tanh_of for all of them: softcap 5 on 500-token chunks 281
// against 387 us, on long contexts 772 against 1175; and its code beside the other
// form in one kernel: drafts with a softcap of 50 83 against 85 us.
constexpr int kNoCap = 0, kCap = 1, kLargeCap = 2;
constexpr float kCapOfExp = 200.0f;
inline int cap_form(float softcap) {
  return softcap == 0.0f ? kNoCap : softcap <= kCapOfExp ? kCap : kLargeCap;
}

// tanh(t), off by at most 2^-19 of its size: up to 1/4 by four terms of the series
// (the next, 62/2835 t^9, is 2^-21.5 of t there), else 1 - 2 / (exp(2t) + 1), whose
// error of 3e-7 is more than that of smaller values.
__device__ __forceinline__ float tanh_of(float t) {
  const float w = t * t;
  const float p = fmaf(w, fmaf(w, -17.0f / 315.0f, 2.0f / 15.0f), -1.0f / 3.0f);
  return fabsf(t) <= 0.25f ? fmaf(t * w, p, t) : tanh_via_exp2(t);
}

// Whether a row sees key c of 32, from its mask (one bit per key).
template <bool MASKED>
__device__ __forceinline__ bool seen(uint32_t mask, int c) {
  return !MASKED || ((mask >> c) & 1u);
}

// Bits [lo, hi) of 32.
__device__ __forceinline__ uint32_t bit_range(int lo, int hi) {
  lo = max(lo, 0);
  hi = min(hi, 32);
  if (hi <= lo) return 0u;
  return (0xffffffffu >> (32 - (hi - lo))) << lo;
}

// What a query row sees: cache rows [lo, hi), and the nodes of its mask.
struct RowView {
  int lo, hi;
  const uint32_t* anc;  // nullptr: a chain (hi covers the row's own node)
};
__device__ __forceinline__ RowView row_view(const TreeParams& p, const TreeSegment& s, int node) {
  RowView v;
  const int depth = p.parents ? p.depth[(size_t)s.b * p.T + node] : node;
  const long long lo = p.window > 0 ? (long long)s.past + depth + 1 - p.window : 0;
  v.lo = lo > 0 ? (int)lo : 0;
  v.hi = p.parents ? s.past : s.past + node + 1;
  v.anc = p.parents ? p.mask + ((size_t)s.b * p.T + node) * p.W32 : nullptr;
  return v;
}
// The mask of the keys [k0, k0 + 32).
__device__ __forceinline__ uint32_t row_mask(const TreeParams& p, const RowView& v, int past,
                                             int k0) {
  uint32_t m = bit_range(v.lo - k0, v.hi - k0);
  const int first = k0 - past;  // the node that the first key stands for
  if (v.anc && first > -32 && first < 32 * p.W32) {
    const int word = first >> 5;
    const uint32_t a = word >= 0 ? v.anc[word] : 0u;
    const uint32_t b = word + 1 < p.W32 ? v.anc[word + 1] : 0u;
    m |= __funnelshift_r(a, b, first & 31);
  }
  return m;
}

// Largest of 32 scores, and with a softcap the smallest, for the series' range.
template <bool MASKED, int CAP>
__device__ __forceinline__ void extremes(const uint32_t (&v)[32], uint32_t m, float& mx,
                                         float& mn) {
  const float ninf = __int_as_float(0xff800000), pinf = __int_as_float(0x7f800000);
  float a[4] = {mx, ninf, ninf, ninf}, b[2] = {mn, pinf};
#pragma unroll
  for (int e = 0; e < 32; e += 2) {
    const float x0 = __uint_as_float(v[e]), x1 = __uint_as_float(v[e + 1]);
    const bool s0 = seen<MASKED>(m, e), s1 = seen<MASKED>(m, e + 1);
    float& t = a[(e >> 1) & 3];
    t = fmax3f(t, s0 ? x0 : ninf, s1 ? x1 : ninf);
    if (CAP) {
      float& u = b[(e >> 1) & 1];
      u = fmin3f(u, s0 ? x0 : pinf, s1 ? x1 : pinf);
    }
  }
  mx = fmaxf(fmax3f(a[0], a[1], a[2]), a[3]);
  if (CAP) mn = fminf(b[0], b[1]);
}

// 2^(x - m) of 32 scores, added to the two partial sums, and P as 16-bit pairs.
// MODE 0: x = s * s_mul; with a softcap x = cap_mul * tanh(s * s_mul), by the
// series' three terms (1), by exp (2) or by tanh_of (3).  P is rounded to the
// storage type for the tensor-core product: at most half a step of each weight, as
// V's own elements carry; the row sum adds the fp32 values.
template <typename T, int MODE, bool MASKED>
__device__ __forceinline__ void exponentials(const uint32_t (&v)[32], uint32_t m, float s_mul,
                                             float cap_mul, float m_eff, float2 (&acc)[2],
                                             uint32_t (&pw)[16]) {
  const float ninf = __int_as_float(0xff800000);
  const float2 z = make_float2(0.0f, 0.0f);
  const float2 mul2 = make_float2(s_mul, s_mul), neg_m = make_float2(-m_eff, -m_eff);
  // cap_mul * tanh(u) with u = s * s_mul, as a polynomial in s
  const float q1 = cap_mul * s_mul, q3 = q1 * s_mul * s_mul * (-1.0f / 3.0f);
  const float q5 = q1 * (s_mul * s_mul) * (s_mul * s_mul) * (2.0f / 15.0f);
  const float2 c1 = make_float2(q1, q1), c3 = make_float2(q3, q3), c5 = make_float2(q5, q5);
#pragma unroll
  for (int g = 0; g < 16; g += 8) {
    float2 x[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int e = 2 * (g + k);
      const float2 s = make_float2(__uint_as_float(v[e]), __uint_as_float(v[e + 1]));
      if (MODE == 0) {
        x[k] = ffma2(s, mul2, neg_m);
      } else if (MODE == 1) {
        const float2 w = ffma2(s, s, z);
        x[k] = ffma2(s, ffma2(w, ffma2(w, c5, c3), c1), neg_m);
      } else if (MODE == 2) {
        x[k].x = fmaf(cap_mul, tanh_via_exp2(s.x * s_mul), -m_eff);
        x[k].y = fmaf(cap_mul, tanh_via_exp2(s.y * s_mul), -m_eff);
      } else {
        x[k].x = fmaf(cap_mul, tanh_of(s.x * s_mul), -m_eff);
        x[k].y = fmaf(cap_mul, tanh_of(s.y * s_mul), -m_eff);
      }
      x[k].x = seen<MASKED>(m, e) ? x[k].x : ninf;
      x[k].y = seen<MASKED>(m, e + 1) ? x[k].y : ninf;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] = make_float2(ex2_approx(x[k].x), ex2_approx(x[k].y));
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      acc[k & 1] = fadd2(acc[k & 1], x[k]);
      pw[g + k] = pack2<T>(x[k].x, x[k].y);
    }
  }
}

// The running state of a query row, or of half of one.
struct RowState {
  float m = -INFINITY;  // reference of the exponentials, base-2 units (the row's)
  float l = 0.0f;       // sum of 2^(x - m) over this thread's columns
};

// One arrival for the whole warp, after what all of its lanes did.
__device__ __forceinline__ void warp_arrive(uint64_t* bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// A row that one thread has to itself.
struct RowAlone {
  __device__ __forceinline__ bool exchange(float mine, float& other) {
    other = mine;
    return true;
  }
};

// A row whose columns two threads share: warps of the same rows, one half each.
// A value's place alternates between two, since a warp may be at the next tile's
// scores while the other has yet to read this tile's value.
struct RowPair {
  float* place;   // [turn][row][half] in shared memory, at this thread's row
  uint64_t* bar;  // of the two warps; an arrival each
  int half;
  volatile int* abort;
  uint32_t* status;
  uint32_t met = 0, turn = 0;
  __device__ __forceinline__ bool meet() {
    warp_arrive(bar);
    return __all_sync(0xffffffffu, mbar_wait<false>(bar, met++ & 1, abort, status));
  }
  // The other thread's value; false: the wait for it was given up.
  __device__ __forceinline__ bool exchange(float mine, float& other) {
    float* at = place + (turn & 1) * (2 * kTcRows);
    ++turn;
    at[half] = mine;
    if (!meet()) return false;
    other = at[half ^ 1];
    return true;
  }
};

// The kernels' shared memory: barriers, segments and the rows' meeting places
// first, then the tiles, which have to lie on 1024-byte boundaries.  The first
// part fills the 3 KB that the largest rings leave, so there is no room to round
// addresses up: the kernels use no other shared memory, whose start then is such
// a boundary, and refuse to run if it is not.
constexpr int kHeadBytes = 3 * 1024;
__device__ __forceinline__ bool misplaced(const void* smem, const TreeParams& p) {
  if ((smem_u32(smem) & 1023) == 0) return false;
  if (threadIdx.x == 0) {
    wait_prior_grid();
    atomicOr(p.status, PVA_DEV_WAIT_TIMEOUT);
    tree_note_cut(p, blockIdx.x, nullptr);
  }
  return true;
}

// Softmax of N score columns of this thread's row (TMEM address t_s, keys [k0, k0
// + N)): P over the first N / 2 of them.  The reference moves where the row's
// maximum passes it by more than 2^8; alpha is the factor that O then has to be
// scaled by.  All warps of the rows call; false: a wait was given up.
//
// Tiles without a mask are read once and worked on in registers (2048-token
// chunks of 8 sequences, d = 128, queries rotated before: 1.13 ms, in a loop 1.26
// ms; long contexts with a softcap, while its series holds: 401 us, in a loop 453
// us).  The others go over the columns twice, 32 at a time in a loop: reading
// tensor memory again is about 18 cycles, while unrolled code for every kind of
// mask and softcap spills and does not stay in the instruction cache (a window and
// a softcap at d = 64, 500-token chunks: 214 us, in loops 185 us).  What bounds
// those chunks is the chain scores, softmax, P V, next scores of each warpgroup:
// issue slots are 40% full, the tensor pipe 31%, memory 6%.  Any instruction more
// lengthens the chain: a quarter of the exponentials by a polynomial on the FMA pipe
// made them 203 us.
template <typename T, int N, int CAP, typename Row>
__device__ __forceinline__ bool softmax_columns(const TreeParams& p, const RowView& view, int past,
                                                int k0, uint32_t t_s, float s_mul, float cap_mul,
                                                Row& others, RowState& st, float& alpha) {
  const float NEG_INF = __int_as_float(0xff800000);
  const bool all = __all_sync(0xffffffffu, view.lo <= k0 && view.hi >= k0 + N);
  float mx = NEG_INF, mn = __int_as_float(0x7f800000), m_eff;
  // mx: this thread's largest score; the transforms rise, so the row's largest
  // score is its maximum
  auto new_maximum = [&]() -> bool {
    float other;
    if (!others.exchange(mx, other)) return false;
    mx = fmaxf(mx, other);
    float mt = NEG_INF;
    if (mx != NEG_INF) {
      const float t = mx * s_mul;
      mt = CAP == kLargeCap ? cap_mul * tanh_of(t) : CAP ? cap_mul * tanh_via_exp2(t) : t;
    }
    alpha = 1.0f;
    if (mt > st.m + kRescaleThreshold) {
      alpha = ex2_approx(st.m - mt);  // 0 when m is -inf
      st.m = mt;
    }
    m_eff = st.m == NEG_INF ? 0.0f : st.m;
    return true;
  };
  // a softcap's series has to hold for the warp's own columns
  auto small_scores = [&]() {
    return CAP && __all_sync(0xffffffffu, mx == NEG_INF || fmaxf(fabsf(mx), fabsf(mn)) <= p.series_to);
  };
  float2 acc[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
  bool series, done = false;
  if (all) {
    uint32_t v[N / 32][32];
#pragma unroll
    for (int c = 0; c < N / 32; ++c) tmem_ld32(t_s + c * 32, v[c]);
#pragma unroll
    for (int c = 0; c < N / 32; ++c) {
      tmem_wait_ld_of(v[c]);
      extremes<false, CAP>(v[c], 0u, mx, mn);
    }
    series = small_scores();
    if (!new_maximum()) return false;
    if (!CAP || series) {
      done = true;
#pragma unroll
      for (int c = 0; c < N / 32; ++c) {
        uint32_t pw[16];
        exponentials<T, CAP ? 1 : 0, false>(v[c], 0u, s_mul, cap_mul, m_eff, acc, pw);
        tmem_st16(t_s + c * 16, pw);
      }
    }
  } else {
    uint32_t v[32];
#pragma unroll 1
    for (int c = 0; c < N; c += 32) {
      tmem_ld32(t_s + c, v);
      const uint32_t mask = row_mask(p, view, past, k0 + c);
      tmem_wait_ld_of(v);
      extremes<true, CAP>(v, mask, mx, mn);
    }
    series = small_scores();
    if (!new_maximum()) return false;
  }
  if (!done) {
    uint32_t v[32];
#pragma unroll 1
    for (int c = 0; c < N; c += 32) {
      tmem_ld32(t_s + c, v);
      const uint32_t mask = all ? 0xffffffffu : row_mask(p, view, past, k0 + c);
      tmem_wait_ld_of(v);
      uint32_t pw[16];
      if (!CAP)
        exponentials<T, 0, true>(v, mask, s_mul, cap_mul, m_eff, acc, pw);
      else if (series)
        exponentials<T, 1, true>(v, mask, s_mul, cap_mul, m_eff, acc, pw);
      else
        exponentials<T, CAP == kLargeCap ? 3 : 2, true>(v, mask, s_mul, cap_mul, m_eff, acc, pw);
      // over columns whose scores have been read in this pass
      tmem_st16(t_s + c / 2, pw);
    }
  }
  const float2 r = fadd2(acc[0], acc[1]);
  st.l = st.l * alpha + r.x + r.y;
  return true;
}

// Score column where the 16 weights of MMA step kk lie: each half's weights over
// its own columns, so that no thread writes over scores another still reads.
template <int BN>
__device__ __forceinline__ int p_column(int kk) {
  constexpr int steps = BN / 32;  // of one half
  return kk < steps ? kk * 8 : BN / 2 + (kk - steps) * 8;
}

// Columns [begin, end) of O that a thread of the row scales and stores.
struct Columns {
  int begin, end;
};
template <int D>
__device__ __forceinline__ Columns half_columns(int half) {
  constexpr int split = (D / 2 + 31) / 32 * 32;
  return half ? Columns{split, D} : Columns{0, split};
}

// Columns of O (TMEM address t_o) times f.
__device__ __forceinline__ void scale_o(uint32_t t_o, Columns cols, float f) {
#pragma unroll 1
  for (int c = cols.begin; c < cols.end; c += 32) {
    uint32_t o[32];
    tmem_ld32(t_o + c, o);
    tmem_wait_ld_of(o);
#pragma unroll
    for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
    tmem_st32(t_o + c, o);
  }
}

// Zeros in the V rows of a tile (keys [k0, k0 + BN)) outside [lo, hi): cache rows
// there may hold anything, and 0 * NaN is NaN.  r: 0 .. 127, a thread per row.
template <int BN, int CH>
__device__ __forceinline__ void zero_v_rows(uint8_t* v_tile, int r, int k0, int lo, int hi) {
  if (r < BN && (k0 + r < lo || k0 + r >= hi)) {
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int u = 0; u < 8; ++u)
        *reinterpret_cast<uint4*>(v_tile + c * (BN * 128) + r * 128 + u * 16) =
            make_uint4(0, 0, 0, 0);
  }
  fence_proxy_async_smem();
}

// Columns of a row's result: O / l to the output, or the unnormalised sums to its
// slot.
template <typename T, int D>
__device__ __forceinline__ void store_row(const TreeParams& p, const TreeSegment& s, uint32_t t_o,
                                          bool own, int row, int node, Columns cols, float m, float l) {
  const bool whole = s.slot < 0;
  const float inv = !whole ? 1.0f : l != 0.0f ? 1.0f / l : 0.0f;
  T* out = static_cast<T*>(p.out) + (((size_t)s.b * p.T + node) * p.H + (size_t)s.h * p.G +
                                     (row - node * p.G)) * D;
  const size_t at = whole ? 0 : (size_t)s.slot * p.rows + (row - s.t * p.rows);
  float* part = p.part_o + at * D;
  if (own && !whole && cols.begin == 0) p.part_ml[at] = make_float2(m, l);
#pragma unroll 1
  for (int c = cols.begin; c < cols.end; c += 32) {
    uint32_t v[32];
    tmem_ld32(t_o + c, v);
    tmem_wait_ld_of(v);
    if (own && whole) {
#pragma unroll
      for (int e = 0; e < 32; e += 8) {
        uint4 w;
        w.x = pack2<T>(__uint_as_float(v[e + 0]) * inv, __uint_as_float(v[e + 1]) * inv);
        w.y = pack2<T>(__uint_as_float(v[e + 2]) * inv, __uint_as_float(v[e + 3]) * inv);
        w.z = pack2<T>(__uint_as_float(v[e + 4]) * inv, __uint_as_float(v[e + 5]) * inv);
        w.w = pack2<T>(__uint_as_float(v[e + 6]) * inv, __uint_as_float(v[e + 7]) * inv);
        *reinterpret_cast<uint4*>(out + c + e) = w;
      }
    } else if (own) {
#pragma unroll
      for (int e = 0; e < 32; e += 4)
        *reinterpret_cast<uint4*>(part + c + e) = make_uint4(v[e], v[e + 1], v[e + 2], v[e + 3]);
    }
  }
}

// A lane's share of the copies of a key tile: one lane per page, or one for the
// whole tile.
struct TileCopy {
  bool mine;
  int block, y;  // cache block and first row in it
  __device__ __forceinline__ int plane(const TreeParams& p, const TreeSegment& s) const {
    return block * p.Hkv + s.h;
  }
};
struct TileCopies {
  int box, copies;  // rows of one copy, copies side by side
  __device__ __forceinline__ TileCopies(const TreeParams& p, int bn)
      : box(p.table && p.page < bn ? p.page : bn), copies(bn / box) {}
  __device__ __forceinline__ TileCopy locate(const TreeParams& p, const TreeSegment& s, int bn,
                                             int j, int lane) const {
    TileCopy c{false, 0, 0};
    const long long r0 = (long long)j * bn + lane * box;
    if (lane >= copies || r0 >= s.past + s.n || r0 + box <= s.lo) return c;
    const int in = (int)r0 / p.page;
    c.mine = true;
    c.block = p.table ? p.table[(size_t)s.b * p.max_blocks + in] : s.b;
    c.y = (int)r0 - in * p.page;
    return c;
  }
};

}  // namespace tile
}  // namespace pva
