// Rotary embedding of packed token rows with positions on several axes, and
// the write of key and value rows to a cache of blocks: what pva_rope_axes and
// the front end of pva_gqa_tree share.
//
// Pair k of a head row (dims (2k, 2k+1) when interleaved, else (k, k + rot/2))
// is turned by the table row of the position on its axis:
//   axes in sections     axis a owns sections[a] consecutive pairs, in order;
//   axes interleaved     axis k mod n where k < n * sections[k mod n], else 0.
#pragma once

#include <stddef.h>

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
  const int32_t* parents;   // [B, T], or nullptr: a chain
  const int32_t* table;     // [B, max_blocks]; nullptr: block b
  int T, max_blocks;
  uint32_t group_inv;       // ceil(2^32 / G): row / G is the high word of row * this while
                            // row * G < 2^32; 0: divide
  int negate_q;             // a negative scale, moved into the queries
  void* q_rest;             // nullptr, or what rounding took off the queries, laid out like them
  void* out;                // attention output: rows of unused nodes are zeroed
  uint32_t* status;
};

constexpr int kRopeThreads = 128;
constexpr int kRopeCtas = 8;  // CTAs an SM holds (64 registers: the 16-byte fp32 form spills 4 bytes)
constexpr int kRopeRows = 2;  // head rows a thread has in flight

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

// The first of a query's two parts: finite for any finite x, or there would be no
// rest of it (only f16 overflows within f32's range).  An infinity's rest is one.
template <typename T>
__device__ __forceinline__ T round_finite(float x) {
  return round_to<T>(x);
}
template <>
__device__ __forceinline__ __half round_finite<__half>(float x) {
  unsigned short h;
  asm("cvt.rn.satfinite.f16.f32 %0, %1;" : "=h"(h) : "f"(x));
  return __ushort_as_half(h);
}

template <typename T, int VEC>
struct alignas(sizeof(T) * VEC) Pack {
  T v[VEC];
};


template <bool PAST_L1, typename T>
__device__ __forceinline__ T load(const T* p) {
  if constexpr (!PAST_L1) {
    return *p;
  } else if constexpr (sizeof(T) == 16) {
    const uint4 v = __ldcg(reinterpret_cast<const uint4*>(p));
    return *reinterpret_cast<const T*>(&v);
  } else if constexpr (sizeof(T) == 8) {
    const uint2 v = __ldcg(reinterpret_cast<const uint2*>(p));
    return *reinterpret_cast<const T*>(&v);
  } else if constexpr (sizeof(T) == 4) {
    const uint32_t v = __ldcg(reinterpret_cast<const uint32_t*>(p));
    return *reinterpret_cast<const T*>(&v);
  } else {
    const unsigned short v = __ldcg(reinterpret_cast<const unsigned short*>(p));
    return *reinterpret_cast<const T*>(&v);
  }
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

template <bool PAST_L1>
__device__ __forceinline__ float table_at(const void* t, long long i, int is_f16) {
  return is_f16 ? __half2float(load<PAST_L1>(static_cast<const __half*>(t) + i))
                : load<PAST_L1>(static_cast<const float*>(t) + i);
}

// cos and sin of a token's pairs, and whether a position is off the tables.
struct alignas(16) RopeToken {
  float2 cs[128];
  int bad[kMaxAxes];  // read as one int4
};
static_assert(kMaxAxes == 4 && offsetof(RopeToken, bad) % 16 == 0 && sizeof(RopeToken) % 16 == 0,
              "16-byte reads of `bad`");

// Does the tokens first, first + stride, ... (tid: one of kRopeThreads threads,
// which share `sh` and the named barrier `bar`).  VEC pairs of a head row per
// thread: 16-byte accesses where sizes and alignment allow (VEC = 16 /
// sizeof(T)), single elements otherwise.  depth_of(tok): a tree node's depth.
//
// A token's table entries are fetched once, a pair per thread, into shared
// memory, and one token ahead: while the rows of token i are turned, the
// positions of token i + 2 and the entries of token i + 1 are on their way.
// go(): asked once, before the first write, whether rows may be written.  TREE
// reads past L1: its inputs may be older than this kernel's launch, but not than
// whatever the SM still holds of the last step's.
template <typename T, int VEC, bool TREE, typename Depth, typename Go>
__device__ __forceinline__ void rope_tokens(const RopeStep& s, int first, int stride, int tid,
                                            int bar, RopeToken (&sh)[2], Depth depth_of, Go go) {
  using P = Pack<T, VEC>;
  const RopeTable& rt = s.rt;
  const int half = rt.rot / 2;
  const int units = s.d / (2 * VEC);  // of 2 * VEC dims
  const int u = tid % units, r0 = tid / units, step = kRopeThreads / units;
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
  const int n_rows = r0 < step ? nq + nk + nv : 0;
  const T* q = static_cast<const T*>(s.q);
  const T* k = static_cast<const T*>(s.k);
  const T* v = static_cast<const T*>(s.v);
  T* q_out = static_cast<T*>(s.q_out);
  T* k_out = static_cast<T*>(s.k_out);
  T* k_cache = static_cast<T*>(s.k_cache);
  T* v_cache = static_cast<T*>(s.v_cache);
  const int G = TREE ? s.H / s.Hkv : 1;
  const int axis = tid < half ? axis_of_pair(rt, tid) : 0;  // of the pair this thread fetches

  struct Info {
    int64_t at, check;  // position on this thread's axis, and of axis tid
    int64_t slot;
  };
  auto fetch_info = [&](int tok) {
    Info f{0, 0, -1};
    if (tok >= s.tokens) return f;
    if (TREE) {
      const int b = tok / s.T, node = tok - b * s.T;
      // also called for steps that will be refused: nothing is taken for granted
      const int past = load<TREE>(s.past + b);
      const int in = past >= 0 ? (int)(((uint32_t)past + node) / (uint32_t)s.page) : -1;
      if (node < (s.lens ? load<TREE>(s.lens + b) : s.T) && (unsigned)in < (unsigned)s.max_blocks) {
        const int row = past + node;
        const int block = s.table ? load<TREE>(s.table + (size_t)b * s.max_blocks + in) : b;
        f.slot = (int64_t)block * s.page + (row - in * s.page);
        if (half) f.at = s.pos ? load<TREE>(s.pos + (size_t)axis * s.tokens + tok) : (int64_t)past + depth_of(tok);
      }
    } else {
      f.at = s.pos[(size_t)axis * s.tokens + tok];
      if (tid < rt.n_axes) f.check = s.pos[(size_t)tid * s.tokens + tok];
      if (k_cache) f.slot = s.slots[tok];
    }
    return f;
  };
  // a pair per thread: half <= 128 = kRopeThreads
  auto fetch_entry = [&](const Info& f) {
    float2 e = make_float2(1.0f, 0.0f);
    if (tid < half && f.at >= 0 && f.at < rt.rows) {
      const int64_t i = f.at * half + tid;
      e.x = table_at<TREE>(rt.cos, i, rt.is_f16);
      e.y = table_at<TREE>(rt.sin, i, rt.is_f16);
      if (rt.inverse) e.y = -e.y;
    }
    return e;
  };
  auto share = [&](RopeToken& t, float2 e, const Info& f) {
    if (tid < half) t.cs[tid] = e;
    if (!TREE && tid < kMaxAxes) t.bad[tid] = f.check < 0 || f.check >= rt.rows;
    asm volatile("bar.sync %0, %1;" ::"r"(bar), "n"(kRopeThreads) : "memory");
  };

  P x0[kRopeRows], x1[kRopeRows];
  auto load_rows = [&](int tok, int r) {
#pragma unroll
    for (int y = 0; y < kRopeRows; ++y) {
      const int row = r + y * step;
      if (row >= n_rows) continue;
      const T* src = row < nq ? q + (size_t)tok * s.q_stride + (size_t)row * s.d
                     : row < nq + nk ? k + (size_t)tok * s.k_stride + (size_t)(row - nq) * s.d
                                     : v + (size_t)tok * s.v_stride + (size_t)(row - nq - nk) * s.d;
      x0[y] = load<TREE>(reinterpret_cast<const P*>(src + d0));
      x1[y] = load<TREE>(reinterpret_cast<const P*>(src + d1));
    }
  };

  if (first >= s.tokens) return;
  load_rows(first, r0);
  Info now = fetch_info(first), next = fetch_info(first + stride);
  const float2 first_entry = fetch_entry(now);
  if (!go()) return;
  share(sh[0], first_entry, now);
  int buf = 0;
  for (int tok = first; tok < s.tokens; tok += stride, buf ^= 1) {
    if (tok != first) load_rows(tok, r0);
    const Info after = fetch_info(tok + 2 * stride);
    const float2 entry = fetch_entry(next);
    bool write = true;
    int b = 0, node = tok;
    if (TREE) {
      b = tok / s.T;
      node = tok - b * s.T;
      if (now.slot < 0) {
        // an unused node: zeros out
        write = false;
        P z;
#pragma unroll
        for (int e = 0; e < VEC; ++e) z.v[e] = round_to<T>(0.0f);
        P* o = reinterpret_cast<P*>(static_cast<T*>(s.out) + (size_t)tok * s.H * s.d);
        for (int e = tid; e < s.H * s.d / VEC; e += kRopeThreads) o[e] = z;
        // Its queries are zeros where the attention has them in one warp (32 rows) with
        // used ones: a warp's rows are rounded alike, and what the workspace held must
        // not decide how.
        const int used = s.lens ? load<TREE>(s.lens + b) : s.T;
        const int group = (long long)node * G < ((long long)used * G + 31) / 32 * 32 ? G * s.d / VEC : 0;
        for (int e = tid; e < s.Hkv * group; e += kRopeThreads) {
          const int h = e / group;
          const size_t at = (((size_t)b * s.Hkv + h) * s.T + node) * group + (e - h * group);
          reinterpret_cast<P*>(q_out)[at] = z;
          if (s.q_rest) reinterpret_cast<P*>(s.q_rest)[at] = z;
        }
      }
    } else {
      const int4 bad = *reinterpret_cast<const int4*>(sh[buf].bad);
      if (bad.x | bad.y | bad.z | bad.w || now.slot < -1 || now.slot >= (k_cache ? s.n_slots : 0)) {
        // the token is left out, and the caller told
        write = false;
        if (tid == 0) atomicOr(s.status, PVA_DEV_ROPE);
      }
    }
    if (write) {
      int64_t cached = -1;
      size_t cache_row = 0;
      if (now.slot >= 0) {
        cached = s.n_slots >> 32 ? now.slot / s.page : (uint32_t)now.slot / (uint32_t)s.page;
        cache_row = (size_t)(now.slot - cached * s.page);
      }
      // where the token's query rows go: kv head h's group at h * group_stride
      const size_t group_stride = TREE ? (size_t)s.T * G * s.d : 0;
      const size_t to = TREE ? ((size_t)b * s.Hkv * s.T + node) * G * s.d : (size_t)tok * s.q_out_stride;
      for (int r = r0; r < n_rows; r += step * kRopeRows) {
        if (r != r0) load_rows(tok, r);
#pragma unroll
        for (int y = 0; y < kRopeRows; ++y) {
          const int row = r + y * step;
          if (row >= n_rows) continue;
          const bool is_q = row < nq, is_v = row >= nq + nk;
          const int head = !TREE ? 0 : s.group_inv ? (int)__umulhi(row, s.group_inv) : row / G;
          const size_t q_to = to + head * group_stride + (size_t)(row - head * G) * s.d;
          if (turned && !is_v) {
            if (rt.interleaved) split_pairs(x0[y], x1[y]);
            P rest0, rest1;
            const bool parted = TREE && std::is_same<T, __half>::value && is_q && s.q_rest;
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
              const float2 cs = sh[buf].cs[u * VEC + e];
              const float a = load_f(x0[y].v[e]), f = load_f(x1[y].v[e]);
              const float g0 = __fsub_rn(__fmul_rn(cs.x, a), __fmul_rn(cs.y, f));
              const float g1 = __fadd_rn(__fmul_rn(cs.y, a), __fmul_rn(cs.x, f));
              x0[y].v[e] = parted ? round_finite<T>(g0) : round_to<T>(g0);
              x1[y].v[e] = parted ? round_finite<T>(g1) : round_to<T>(g1);
              if (TREE) {
                rest0.v[e] = round_to<T>(g0 - load_f(x0[y].v[e]));
                rest1.v[e] = round_to<T>(g1 - load_f(x1[y].v[e]));
              }
            }
            if (rt.interleaved) join_pairs(x0[y], x1[y]);
            if (TREE && is_q && s.q_rest) {
              if (rt.interleaved) join_pairs(rest0, rest1);
              T* dst = static_cast<T*>(s.q_rest) + q_to;
              if (s.negate_q) {
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                  rest0.v[e] = -rest0.v[e];
                  rest1.v[e] = -rest1.v[e];
                }
              }
              *reinterpret_cast<P*>(dst + d0) = rest0;
              *reinterpret_cast<P*>(dst + d1) = rest1;
            }
          } else if (TREE && is_q && s.q_rest) {  // dims that are only copied are exact
            P z;
#pragma unroll
            for (int e = 0; e < VEC; ++e) z.v[e] = round_to<T>(0.0f);
            T* dst = static_cast<T*>(s.q_rest) + q_to;
            *reinterpret_cast<P*>(dst + d0) = z;
            *reinterpret_cast<P*>(dst + d1) = z;
          }
          if (is_q) {
            if (TREE && s.negate_q) {
#pragma unroll
              for (int e = 0; e < VEC; ++e) {
                x0[y].v[e] = -x0[y].v[e];
                x1[y].v[e] = -x1[y].v[e];
              }
            }
            T* dst = q_out + q_to;
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
    if (tok + stride < s.tokens) share(sh[buf ^ 1], entry, next);
    now = next;
    next = after;
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

// Rows of a [tokens, heads, d] tensor with a token stride: `width` elements of each.
struct RowRange {
  const void* p;
  long long tokens, stride, width;
};
bool rows_meet(const RowRange& a, const RowRange& b, size_t size);

// The token rows of a call and where they go, and what every such call checks: an
// output may be its own input (the same address and stride); otherwise no output may
// overlap an input or the other output.
struct RowsIn {
  const void *q, *k, *v;
  const void *q_out, *k_out;
  long long q_stride, k_stride, v_stride, q_out_stride, k_out_stride;
  int tokens, H, Hkv, d;
  const void *k_cache, *v_cache;
  const int64_t* slot_map;
  int n_blocks, page_size, dtype;
};
int check_token_rows(const RowsIn& r);
}  // namespace host

cudaError_t launch_rope(const RopeStep& s, int dtype, bool tree, int num_sms, cudaStream_t st);

}  // namespace pva
