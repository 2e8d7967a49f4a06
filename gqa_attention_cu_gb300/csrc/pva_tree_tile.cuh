// Softmax of one key tile of the tree attention's tensor-core kernels: key
// masks, row extremes and exponentials of one row per thread.
//
// Softcap: tanh(t) of t = s * scale / softcap comes from the first three terms
// of its series, t - t^3/3 + 2t^5/15 (error below the next term, 17/315 |t|^7 <
// 3.3e-6 for |t| <= 1/4), on the FMA pipe, whenever every score of the warp's
// tile is that small; otherwise from 1 - 2 / (exp(2t) + 1).
#pragma once

#include <math.h>

#include "pva_device.cuh"
#include "pva_tree.h"

namespace pva {
namespace tile {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kRescaleThreshold = 8.0f;  // log2 units: O is rescaled when the max grows > 2^8
constexpr float kSeriesLimit = 0.25f;      // |t| up to which tanh is summed

// One bit per key of a tile, for one query row.
template <int BN>
struct Mask {
  uint32_t w[BN / 32];
};

template <int BN, bool MASKED>
__device__ __forceinline__ bool seen(const Mask<BN>& m, int c) {
  return !MASKED || ((m.w[c >> 5] >> (c & 31)) & 1u);
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
// The mask of the keys [k0, k0 + BN).
template <int BN>
__device__ __forceinline__ Mask<BN> row_mask(const TreeParams& p, const RowView& v, int past,
                                             int k0) {
  Mask<BN> m;
#pragma unroll
  for (int w = 0; w < BN / 32; ++w) {
    const int key = k0 + 32 * w, first = key - past;
    m.w[w] = bit_range(v.lo - key, v.hi - key);
    // `first` is the node that the word's first key stands for
    if (v.anc && first > -32 && first < 32 * p.W32) {
      const int word = first >> 5;
      const uint32_t a = word >= 0 ? v.anc[word] : 0u;
      const uint32_t b = word + 1 < p.W32 ? v.anc[word + 1] : 0u;
      m.w[w] |= __funnelshift_r(a, b, first & 31);
    }
  }
  return m;
}

// Largest score of 32 columns of a tile (c0: the first), and with a softcap the
// smallest, for the series' range.
template <int BN, bool MASKED, bool CAP>
__device__ __forceinline__ void extremes(const uint32_t (&v)[32], int c0, const Mask<BN>& m,
                                         float& mx, float& mn) {
  const float ninf = __int_as_float(0xff800000), pinf = __int_as_float(0x7f800000);
  float a[2] = {mx, ninf}, b[2] = {mn, pinf};
#pragma unroll
  for (int e = 0; e < 32; e += 2) {
    const float x0 = __uint_as_float(v[e]), x1 = __uint_as_float(v[e + 1]);
    const bool s0 = seen<BN, MASKED>(m, c0 + e), s1 = seen<BN, MASKED>(m, c0 + e + 1);
    float& t = a[(e >> 1) & 1];
    t = fmax3f(t, s0 ? x0 : ninf, s1 ? x1 : ninf);
    if (CAP) {
      float& u = b[(e >> 1) & 1];
      u = fmin3f(u, s0 ? x0 : pinf, s1 ? x1 : pinf);
    }
  }
  mx = fmaxf(a[0], a[1]);
  if (CAP) mn = fminf(b[0], b[1]);
}

// 2^(x - m) over 32 columns, added to the two partial sums, and P as 16-bit
// pairs.  MODE 0: x = s * s_mul; with a softcap x = cap_mul * tanh(s * s_mul), by
// its series (1) or by exp (2).  P is rounded to the storage type for the
// tensor-core product: at most half a step of each weight, as V's own elements
// carry; the row sum adds the fp32 values.
template <typename T, int BN, int MODE, bool MASKED>
__device__ __forceinline__ void exponentials(const uint32_t (&v)[32], int c0, const Mask<BN>& m,
                                             float s_mul, float cap_mul, float m_eff,
                                             float2 (&acc)[2], uint32_t* pw) {
  const float ninf = __int_as_float(0xff800000);
  const float2 z = make_float2(0.0f, 0.0f);
  const float2 mul2 = make_float2(s_mul, s_mul), neg_m = make_float2(-m_eff, -m_eff);
  const float2 a2 = make_float2(cap_mul, cap_mul);
  const float2 c1 = make_float2(cap_mul * (-1.0f / 3.0f), cap_mul * (-1.0f / 3.0f));
  const float2 c2 = make_float2(cap_mul * (2.0f / 15.0f), cap_mul * (2.0f / 15.0f));
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
        const float2 u = ffma2(s, mul2, z), w = ffma2(u, u, z);
        x[k] = ffma2(u, ffma2(w, ffma2(w, c2, c1), a2), neg_m);
      } else {
        x[k].x = fmaf(cap_mul, tanh_via_exp2(s.x * s_mul), -m_eff);
        x[k].y = fmaf(cap_mul, tanh_via_exp2(s.y * s_mul), -m_eff);
      }
      x[k].x = seen<BN, MASKED>(m, c0 + e) ? x[k].x : ninf;
      x[k].y = seen<BN, MASKED>(m, c0 + e + 1) ? x[k].y : ninf;
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

// The running state of one query row.
struct RowState {
  float m;            // reference of the exponentials, base-2 units; -inf: no key seen yet
  float l = 0.0f;     // sum of 2^(x - m)
  bool wide = false;  // the warp has met scores beyond the series' range
  // Lanes without a row have a reference from the start: they ask for nothing.
  __device__ __forceinline__ explicit RowState(bool own) : m(own ? -INFINITY : 0.0f) {}
};

// The reference of rows that see their first keys in this tile: its maximum.
// (Their O and l are zero, so nothing has to be scaled.)
template <int BN, bool CAP, bool MASKED>
__device__ __forceinline__ void first_reference(uint32_t t_s, const Mask<BN>& mk, float s_mul,
                                                float cap_mul, RowState& st) {
  const float ninf = __int_as_float(0xff800000);
  float mx = ninf, mn = 0.0f;
  uint32_t v[2][32];
  tmem_ld32(t_s, v[0]);
#pragma unroll
  for (int c = 0; c < BN / 32; ++c) {
    tmem_wait_ld_of(v[c & 1]);
    if (c + 1 < BN / 32) tmem_ld32(t_s + (c + 1) * 32, v[(c + 1) & 1]);
    extremes<BN, MASKED, false>(v[c & 1], c * 32, mk, mx, mn);
  }
  if (st.m == ninf && mx != ninf) st.m = CAP ? cap_mul * tanh_via_exp2(mx * s_mul) : mx * s_mul;
}

// Exponentials of a tile against the reference as it is, in one pass over the
// scores: the next 32 columns are on their way from tensor memory while 32 are
// worked on.  Returns false, with nothing changed, where a row's maximum passes
// the reference by more than 2^8 (or a score the series' range).
template <typename T, int BN, int MODE, bool MASKED>
__device__ __forceinline__ bool softmax_fast(uint32_t t_s, const Mask<BN>& mk, float s_mul,
                                             float cap_mul, RowState& st) {
  constexpr bool CAP = MODE != 0;
  float mx = __int_as_float(0xff800000), mn = __int_as_float(0x7f800000);
  float2 acc[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
  uint32_t v[2][32], pw[BN / 2];
  tmem_ld32(t_s, v[0]);
#pragma unroll
  for (int c = 0; c < BN / 32; ++c) {
    tmem_wait_ld_of(v[c & 1]);
    if (c + 1 < BN / 32) tmem_ld32(t_s + (c + 1) * 32, v[(c + 1) & 1]);
    extremes<BN, MASKED, MODE == 1>(v[c & 1], c * 32, mk, mx, mn);
    exponentials<T, BN, MODE, MASKED>(v[c & 1], c * 32, mk, s_mul, cap_mul, st.m, acc, pw + c * 16);
  }
  // the transforms rise, so the largest score is the row's maximum
  // (a row that has seen no key yet has none here: every weight is 0)
  const float top = CAP ? cap_mul * tanh_via_exp2(mx * s_mul) : mx * s_mul;
  bool again = mx != __int_as_float(0xff800000) && top > st.m + kRescaleThreshold;
  if (MODE == 1)
    again = again || (mx != __int_as_float(0xff800000) &&
                      fmaxf(fabsf(mx * s_mul), fabsf(mn * s_mul)) > kSeriesLimit);
  if (__any_sync(0xffffffffu, again)) return false;
#pragma unroll
  for (int c = 0; c < BN / 64; ++c) {
    uint32_t w[32];
#pragma unroll
    for (int e = 0; e < 32; ++e) w[e] = pw[c * 32 + e];
    tmem_st32(t_s + c * 32, w);
  }
  const float2 r = fadd2(acc[0], acc[1]);
  st.l += r.x + r.y;
  return true;
}

// The same in two passes, maximum first; moves the reference where the maximum
// passes it by more than 2^8, and returns the factor O then has to be scaled by.
template <typename T, int BN, bool CAP>
__device__ __forceinline__ float softmax_full(uint32_t t_s, const Mask<BN>& mk, float s_mul,
                                              float cap_mul, RowState& st) {
  const float NEG_INF = __int_as_float(0xff800000);
  float mx = NEG_INF, mn = __int_as_float(0x7f800000);
  uint32_t v[32];
#pragma unroll
  for (int c = 0; c < BN / 32; ++c) {
    tmem_ld32(t_s + c * 32, v);
    tmem_wait_ld_of(v);
    extremes<BN, true, CAP>(v, c * 32, mk, mx, mn);
  }
  float mt = NEG_INF;
  if (mx != NEG_INF) mt = CAP ? cap_mul * tanh_via_exp2(mx * s_mul) : mx * s_mul;
  float alpha = 1.0f;
  if (mt > st.m + kRescaleThreshold) {
    alpha = ex2_approx(st.m - mt);  // 0 when m is -inf
    st.m = mt;
  }
  const float m_eff = st.m == NEG_INF ? 0.0f : st.m;
  if (CAP)
    st.wide = __any_sync(0xffffffffu, mx != NEG_INF && fmaxf(fabsf(mx * s_mul), fabsf(mn * s_mul)) >
                                                           kSeriesLimit);
  float2 acc[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
  // P of 64 columns lies over the first 32 of them: columns already read
#pragma unroll
  for (int half = 0; half < BN / 64; ++half) {
    uint32_t pw[32];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      tmem_ld32(t_s + half * 64 + c * 32, v);
      tmem_wait_ld_of(v);
      const int c0 = half * 64 + c * 32;
      if (!CAP)
        exponentials<T, BN, 0, true>(v, c0, mk, s_mul, cap_mul, m_eff, acc, pw + c * 16);
      else if (!st.wide)
        exponentials<T, BN, 1, true>(v, c0, mk, s_mul, cap_mul, m_eff, acc, pw + c * 16);
      else
        exponentials<T, BN, 2, true>(v, c0, mk, s_mul, cap_mul, m_eff, acc, pw + c * 16);
    }
    tmem_st32(t_s + half * 32, pw);
  }
  const float2 r = fadd2(acc[0], acc[1]);
  st.l = st.l * alpha + r.x + r.y;
  return alpha;
}

// Softmax of the tile at TMEM address t_s (BN score columns of this thread's
// row, keys [k0, k0 + BN)): P over its first BN / 2 columns.  Returns the factor
// O has to be scaled by.  A whole warp calls.
template <typename T, int BN, bool CAP>
__device__ __forceinline__ float softmax_tile(const TreeParams& p, const RowView& view, int past,
                                              int k0, uint32_t t_s, float s_mul, float cap_mul,
                                              RowState& st) {
  const bool all = __all_sync(0xffffffffu, view.lo <= k0 && view.hi >= k0 + BN);
  Mask<BN> mk;
  if (!all) {
    mk = row_mask<BN>(p, view, past, k0);
  } else {
#pragma unroll
    for (int w = 0; w < BN / 32; ++w) mk.w[w] = 0xffffffffu;
  }
  if (__any_sync(0xffffffffu, st.m == __int_as_float(0xff800000))) {
    if (all)
      first_reference<BN, CAP, false>(t_s, mk, s_mul, cap_mul, st);
    else
      first_reference<BN, CAP, true>(t_s, mk, s_mul, cap_mul, st);
  }
  bool done;
  if (!CAP)
    done = all ? softmax_fast<T, BN, 0, false>(t_s, mk, s_mul, cap_mul, st)
               : softmax_fast<T, BN, 0, true>(t_s, mk, s_mul, cap_mul, st);
  else if (!st.wide)
    done = all ? softmax_fast<T, BN, 1, false>(t_s, mk, s_mul, cap_mul, st)
               : softmax_fast<T, BN, 1, true>(t_s, mk, s_mul, cap_mul, st);
  else
    done = softmax_fast<T, BN, 2, true>(t_s, mk, s_mul, cap_mul, st);
  return done ? 1.0f : softmax_full<T, BN, CAP>(t_s, mk, s_mul, cap_mul, st);
}

// O columns [0, D) at TMEM address t_o times f.
template <int D>
__device__ __forceinline__ void scale_o(uint32_t t_o, float f) {
#pragma unroll 1
  for (int c = 0; c < D; c += 32) {
    uint32_t o[32];
    tmem_ld32(t_o + c, o);
    tmem_wait_ld();
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

// A row's result: O / l to the output, or the unnormalised sums to its slot.
template <typename T, int D>
__device__ __forceinline__ void store_row(const TreeParams& p, const TreeSegment& s, uint32_t t_o,
                                          bool own, int row, int node, float m, float l) {
  const bool whole = s.slot < 0;
  const float inv = !whole ? 1.0f : l != 0.0f ? 1.0f / l : 0.0f;
  T* out = static_cast<T*>(p.out) + (((size_t)s.b * p.T + node) * p.H + (size_t)s.h * p.G +
                                     (row - node * p.G)) * D;
  const size_t at = whole ? 0 : (size_t)s.slot * p.rows + (row - s.t * p.rows);
  float* part = p.part_o + at * D;
  if (own && !whole) p.part_ml[at] = make_float2(m, l);
#pragma unroll 1
  for (int c = 0; c < D; c += 32) {
    uint32_t v[32];
    tmem_ld32(t_o + c, v);
    tmem_wait_ld();
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
