// Rotary embedding of packed token rows with positions on several axes, and
// the write of key and value rows to a cache of blocks: what pva_rope_axes and
// the front end of pva_gqa_tree share.
//
// Pair k of a head row (dims (2k, 2k+1) when interleaved, else (k, k + rot/2))
// is turned by the table row of the position on its axis:
//   axes in sections     axis a owns sections[a] consecutive pairs, in order;
//   axes interleaved     axis k mod n where k < n * sections[k mod n], else 0.
#pragma once

#include "pva_device.cuh"

namespace pva {

constexpr int kMaxAxes = 4;

struct RopeTable {
  const void* cos;  // [rows, rot / 2]
  const void* sin;
  int is_f16;
  int rot;          // rotated dims of a head row (0: none)
  int rows;
  int interleaved;  // pairs of neighbouring dims
  int n_axes;
  int axes_interleaved;
  int sections[kMaxAxes];
  int inverse;      // turn by the negative angle (the gradient of the rotation)
};

__device__ __forceinline__ int axis_of_pair(const RopeTable& r, int k) {
  if (r.n_axes == 1) return 0;
  int a = 0;
  if (r.axes_interleaved) {
    a = k % r.n_axes;
    int sec = r.sections[0];
#pragma unroll
    for (int x = 1; x < kMaxAxes; ++x) sec = a == x ? r.sections[x] : sec;
    return k < r.n_axes * sec ? a : 0;
  }
  int end = 0;
#pragma unroll
  for (int x = 0; x < kMaxAxes - 1; ++x) {
    end += r.sections[x];
    a += (x + 1 < r.n_axes && k >= end) ? 1 : 0;
  }
  return a;
}

// One pass over token rows: rotated queries and keys, and key and value rows
// into the cache.
struct RopeStep {
  RopeTable rt;
  const void* q;  // [tokens, H, d] with a token stride; nullptr: none
  const void* k;  // [tokens, Hkv, d]
  const void* v;  // [tokens, Hkv, d]; only copied to the cache
  void* q_out;
  void* k_out;    // nullptr: keys go to the cache only
  void* k_cache;  // [blocks, Hkv, page, d]; nullptr: no cache
  void* v_cache;
  long long q_stride, k_stride, v_stride, q_out_stride, k_out_stride;  // elements
  int tokens, H, Hkv, d;
  const int64_t* pos;       // [n_axes, tokens]; tree form: may be nullptr
  const int64_t* slots;     // [tokens], -1: not cached
  int page;                 // rows of a cache block
  long long n_slots;        // blocks * page (both forms)
  // Tree form (TREE): token b * T + i is node i of sequence b; it goes to
  // cache row past[b] + i, and its query rows to [B][Hkv][T * G][d].
  const int32_t* hdr;       // hdr[0] == 0: the step was rejected, nothing is written
  const int32_t* past;
  const int32_t* lens;      // nodes in use per sequence; nullptr: T
  const int32_t* depth;     // [B, T], or nullptr: i
  const int32_t* table;     // [B, max_blocks]; nullptr: block b
  int T, max_blocks;
  int negate_q;             // a negative scale, moved into the queries
  void* out;                // attention output: rows of unused nodes are zeroed
  uint32_t* status;
};

constexpr int kRopeThreads = 128;
constexpr int kRopeRows = 4;  // head rows a thread has in flight

template <typename T>
__device__ __forceinline__ float load_f(T x) { return static_cast<float>(x); }
template <typename T>
__device__ __forceinline__ T round_to(float x);
template <>
__device__ __forceinline__ float round_to<float>(float x) { return x; }
template <>
__device__ __forceinline__ __half round_to<__half>(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 round_to<__nv_bfloat16>(float x) {
  return __float2bfloat16_rn(x);
}

template <typename T, int VEC>
struct alignas(sizeof(T) * VEC) Pack {
  T v[VEC];
};

__device__ __forceinline__ float table_at(const void* t, long long i, int is_f16) {
  return is_f16 ? __half2float(static_cast<const __half*>(t)[i])
                : static_cast<const float*>(t)[i];
}

// Neighbouring pairs across two packs <-> first and second members.
template <typename T, int VEC>
__device__ __forceinline__ void split_pairs(Pack<T, VEC>& x, Pack<T, VEC>& y) {
  Pack<T, VEC> a, b;
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    a.v[e] = 2 * e < VEC ? x.v[2 * e % VEC] : y.v[2 * e % VEC];
    b.v[e] = 2 * e + 1 < VEC ? x.v[(2 * e + 1) % VEC] : y.v[(2 * e + 1) % VEC];
  }
  x = a;
  y = b;
}
template <typename T, int VEC>
__device__ __forceinline__ void join_pairs(Pack<T, VEC>& x, Pack<T, VEC>& y) {
  Pack<T, VEC> a, b;
#pragma unroll
  for (int e = 0; e < 2 * VEC; ++e) {
    const T v = e % 2 ? y.v[e / 2] : x.v[e / 2];
    if (e < VEC) a.v[e % VEC] = v; else b.v[e % VEC] = v;
  }
  x = a;
  y = b;
}

// Axes of the VEC pairs that thread tid turns, two bits each.
template <int VEC>
__device__ __forceinline__ uint32_t rope_axes(const RopeStep& s, int tid) {
  uint32_t axes = 0;
  if (s.rt.n_axes == 1) return 0;
  const int u = tid % (s.d / (2 * VEC));
#pragma unroll
  for (int e = 0; e < VEC; ++e) axes |= (uint32_t)axis_of_pair(s.rt, u * VEC + e) << (2 * e);
  return axes;
}

// Does token tok (tid: one of kRopeThreads threads).  VEC pairs of a head row
// per thread: 16-byte accesses where sizes and alignment allow (VEC = 16 /
// sizeof(T)), single elements otherwise.
template <typename T, int VEC, bool TREE>
__device__ __forceinline__ void rope_token(const RopeStep& s, int tok, int tid, uint32_t axes,
                                           int depth) {
  using P = Pack<T, VEC>;
  const RopeTable& rt = s.rt;
  const int half = rt.rot / 2;
  const int units = s.d / (2 * VEC);  // of 2 * VEC dims
  const int u = tid % units, r0 = tid / units, step = kRopeThreads / units;
  const bool idle = r0 >= step;
  const bool turned = u * VEC < half;
  // the unit's two packs of dims: d0 .. d0 + VEC and d1 .. d1 + VEC
  int d0, d1;
  if (!turned) {
    d0 = rt.rot + (u - half / VEC) * 2 * VEC;
    d1 = d0 + VEC;
  } else if (rt.interleaved) {
    d0 = u * 2 * VEC;
    d1 = d0 + VEC;
  } else {
    d0 = u * VEC;
    d1 = d0 + half;
  }
  const int nq = s.q ? s.H : 0, nk = s.k ? s.Hkv : 0, nv = s.v ? s.Hkv : 0;
  const int n_rows = nq + nk + nv;
  const T* q = static_cast<const T*>(s.q);
  const T* k = static_cast<const T*>(s.k);
  const T* v = static_cast<const T*>(s.v);
  T* q_out = static_cast<T*>(s.q_out);
  T* k_out = static_cast<T*>(s.k_out);
  T* k_cache = static_cast<T*>(s.k_cache);
  T* v_cache = static_cast<T*>(s.v_cache);
  const int G = TREE ? s.H / s.Hkv : 1;

  // The first rows are on their way while the position, the tables' entries
  // and the slot are looked up, one after the other.
  P x0[kRopeRows], x1[kRopeRows];
  auto load_rows = [&](int r) {
#pragma unroll
    for (int y = 0; y < kRopeRows; ++y) {
      const int row = r + y * step;
      if (row >= n_rows) continue;
      const T* src = row < nq ? q + (size_t)tok * s.q_stride + (size_t)row * s.d
                     : row < nq + nk ? k + (size_t)tok * s.k_stride + (size_t)(row - nq) * s.d
                                     : v + (size_t)tok * s.v_stride + (size_t)(row - nq - nk) * s.d;
      x0[y] = *reinterpret_cast<const P*>(src + d0);
      x1[y] = *reinterpret_cast<const P*>(src + d1);
    }
  };
  if (!idle) load_rows(r0);
  int b = 0, node = tok;
  long long slot = -1;
  long long at[kMaxAxes];
  if (TREE) {
    b = tok / s.T;
    node = tok - b * s.T;
    if (node >= (s.lens ? s.lens[b] : s.T)) {  // an unused node: zeros out
      P z;
#pragma unroll
      for (int e = 0; e < VEC; ++e) z.v[e] = round_to<T>(0.0f);
      P* o = reinterpret_cast<P*>(static_cast<T*>(s.out) + (size_t)tok * s.H * s.d);
      for (int e = tid; e < s.H * s.d / VEC; e += kRopeThreads) o[e] = z;
      return;
    }
    const int row = s.past[b] + node;
    const int in_table = row / s.page;
    const int block = s.table ? s.table[(size_t)b * s.max_blocks + in_table] : b;
    slot = (long long)block * s.page + (row - in_table * s.page);
#pragma unroll
    for (int a = 0; a < kMaxAxes; ++a)
      at[a] = !s.pos ? (long long)s.past[b] + depth
                     : a < rt.n_axes ? s.pos[(size_t)a * s.tokens + tok] : 0;
  } else {
    bool bad = false;
#pragma unroll
    for (int a = 0; a < kMaxAxes; ++a) {
      at[a] = a < rt.n_axes ? s.pos[(size_t)a * s.tokens + tok] : 0;
      bad = bad || at[a] < 0 || at[a] >= rt.rows;
    }
    if (k_cache) {
      slot = s.slots[tok];
      bad = bad || slot < -1 || slot >= s.n_slots;
    }
    if (bad) {  // the token is left out, and the caller told
      if (tid == 0) atomicOr(s.status, PVA_DEV_ROPE);
      return;
    }
  }
  float c[VEC], n[VEC];
  if (turned) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const int p = u * VEC + e, a = (axes >> (2 * e)) & 3;
      long long x = at[0];
#pragma unroll
      for (int y = 1; y < kMaxAxes; ++y) x = a == y ? at[y] : x;
      const long long i = x * half + p;
      c[e] = table_at(rt.cos, i, rt.is_f16);
      n[e] = table_at(rt.sin, i, rt.is_f16);
      if (rt.inverse) n[e] = -n[e];
    }
  }
  long long cached = -1;
  size_t cache_row = 0;
  if (slot >= 0) {
    cached = s.n_slots >> 32 ? slot / s.page : (uint32_t)slot / (uint32_t)s.page;
    cache_row = (size_t)(slot - cached * s.page);
  }
  if (idle) return;
  for (int r = r0; r < n_rows; r += step * kRopeRows) {
    if (r != r0) load_rows(r);
#pragma unroll
    for (int y = 0; y < kRopeRows; ++y) {
      const int row = r + y * step;
      if (row >= n_rows) continue;
      const bool is_q = row < nq, is_v = row >= nq + nk;
      if (turned && !is_v) {
        if (rt.interleaved) split_pairs(x0[y], x1[y]);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float a = load_f(x0[y].v[e]), f = load_f(x1[y].v[e]);
          x0[y].v[e] = round_to<T>(__fsub_rn(__fmul_rn(c[e], a), __fmul_rn(n[e], f)));
          x1[y].v[e] = round_to<T>(__fadd_rn(__fmul_rn(n[e], a), __fmul_rn(c[e], f)));
        }
        if (rt.interleaved) join_pairs(x0[y], x1[y]);
      }
      if (is_q) {
        if (TREE && s.negate_q) {
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            x0[y].v[e] = -x0[y].v[e];
            x1[y].v[e] = -x1[y].v[e];
          }
        }
        T* dst = TREE ? q_out + ((((size_t)b * s.Hkv + row / G) * s.T + node) * G + row % G) * s.d
                      : q_out + (size_t)tok * s.q_out_stride + (size_t)row * s.d;
        *reinterpret_cast<P*>(dst + d0) = x0[y];
        *reinterpret_cast<P*>(dst + d1) = x1[y];
        continue;
      }
      const int h = is_v ? row - nq - nk : row - nq;
      if (k_out && !is_v) {
        T* dst = k_out + (size_t)tok * s.k_out_stride + (size_t)h * s.d;
        *reinterpret_cast<P*>(dst + d0) = x0[y];
        *reinterpret_cast<P*>(dst + d1) = x1[y];
      }
      if (cached >= 0) {
        T* dst = (is_v ? v_cache : k_cache) +
                 (((size_t)cached * s.Hkv + h) * s.page + cache_row) * s.d;
        *reinterpret_cast<P*>(dst + d0) = x0[y];
        *reinterpret_cast<P*>(dst + d1) = x1[y];
      }
    }
  }
}

// 16-byte accesses: whole packs in the rotated and in the copied dims, and
// every row on a 16-byte boundary.
inline bool rope_wide(const RopeStep& s, int vec) {
  const uintptr_t ptrs = (uintptr_t)s.q | (uintptr_t)s.k | (uintptr_t)s.v | (uintptr_t)s.q_out |
                         (uintptr_t)s.k_out | (uintptr_t)s.k_cache | (uintptr_t)s.v_cache |
                         (uintptr_t)s.out;
  const long long strides = s.q_stride | s.k_stride | s.v_stride | s.q_out_stride | s.k_out_stride;
  return (ptrs & 15) == 0 && strides % vec == 0 && s.rt.rot / 2 % vec == 0 &&
         (s.d - s.rt.rot) % (2 * vec) == 0;
}

namespace host {
// Checks the rotary arguments and fills the table block (inverse left at 0).
int check_rope(const void* cos_cache, const void* sin_cache, int rot, int rows, int interleaved,
               int n_axes, const int32_t* sections, int axes_interleaved, int rotary_dtype,
               int dtype, int d, RopeTable* t);
}  // namespace host

cudaError_t launch_rope(const RopeStep& s, int dtype, bool tree, int num_sms, cudaStream_t st);

}  // namespace pva
