// Rotary embedding with positions on several axes (pva_rope_axes), and the
// same pass as the front end of pva_gqa_tree.
//
// (x0, x1) -> (c x0 - s x1, s x0 + c x1) with (c, s) the tables' entry
// [position on the pair's axis][pair], in f32, every product and sum rounded on
// its own, then rounded once to the storage type; dims at or past rot are
// copied.  The inverse turns by the negative angle: the rotation is orthogonal
// for cos^2 + sin^2 = 1, and its transpose, the gradient, is this one for any
// table.
//
// Bound by memory: every q, k and v row is read once and written once (twice
// where a key goes to k_out and the cache).  A CTA takes one token at a time: a
// thread keeps the cos and sin of its VEC pairs in registers and walks over
// the token's head rows with them, so the tables and the axis of each pair
// are looked up once a token and not once a head, and four rows' loads of 16
// bytes are in flight per thread.
#include <limits.h>

#include "pva_rope.cuh"

using namespace pva;
using namespace pva::host;

namespace pva {
namespace {

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

// VEC pairs of a head row per thread: 16-byte accesses where sizes and
// alignment allow (VEC = 16 / sizeof(T)), single elements otherwise.
template <typename T, int VEC, bool TREE>
__global__ void __launch_bounds__(kRopeThreads) pva_rope_kernel(RopeStep s) {
  using P = Pack<T, VEC>;
  allow_next_grid();
  wait_prior_grid();
  if (TREE && s.hdr[0] == 0) return;
  const RopeTable& rt = s.rt;
  const int half = rt.rot / 2;
  const int units = s.d / (2 * VEC);  // of 2 * VEC dims
  const int u = threadIdx.x % units, r0 = threadIdx.x / units, step = kRopeThreads / units;
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

  for (int tok = blockIdx.x; tok < s.tokens; tok += gridDim.x) {
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
        for (int e = threadIdx.x; e < s.H * s.d / VEC; e += kRopeThreads) o[e] = z;
        continue;
      }
      const int row = s.past[b] + node;
      const int in_table = row / s.page;
      const int block = s.table ? s.table[(size_t)b * s.max_blocks + in_table] : b;
      slot = (long long)block * s.page + (row - in_table * s.page);
      const int depth = s.depth ? s.depth[tok] : node;
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
        if (threadIdx.x == 0) atomicOr(s.status, PVA_DEV_ROPE);
        continue;
      }
    }
    float c[VEC], n[VEC];
    if (turned) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const int p = u * VEC + e, a = axis_of_pair(rt, p);
        long long x = at[0];
#pragma unroll
        for (int y = 1; y < kMaxAxes; ++y) x = a == y ? at[y] : x;
        const long long i = x * half + p;
        c[e] = table_at(rt.cos, i, rt.is_f16);
        n[e] = table_at(rt.sin, i, rt.is_f16);
        if (rt.inverse) n[e] = -n[e];
      }
    }
    const long long cached = slot < 0 ? -1 : slot / s.page;
    const size_t cache_row = slot < 0 ? 0 : (size_t)(slot - cached * s.page);
    if (idle) continue;
    for (int r = r0; r < n_rows; r += step * kRopeRows) {
      P x0[kRopeRows], x1[kRopeRows];
#pragma unroll
      for (int y = 0; y < kRopeRows; ++y) {
        const int row = r + y * step;
        if (row >= n_rows) continue;
        const T* src = row < nq ? q + (size_t)tok * s.q_stride + (size_t)row * s.d
                       : row < nq + nk
                           ? k + (size_t)tok * s.k_stride + (size_t)(row - nq) * s.d
                           : v + (size_t)tok * s.v_stride + (size_t)(row - nq - nk) * s.d;
        x0[y] = *reinterpret_cast<const P*>(src + d0);
        x1[y] = *reinterpret_cast<const P*>(src + d1);
      }
#pragma unroll
      for (int y = 0; y < kRopeRows; ++y) {
        const int row = r + y * step;
        if (row >= n_rows) continue;
        const bool is_q = row < nq, is_v = row >= nq + nk;
        if (turned && !is_v) {
          P y0, y1;
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            // pair e of the unit: interleaved pairs lie side by side across the packs
            const bool il = rt.interleaved;
            const float a = il ? load_f(2 * e < VEC ? x0[y].v[(2 * e) % VEC] : x1[y].v[(2 * e) % VEC])
                               : load_f(x0[y].v[e]);
            const float f = il ? load_f(2 * e + 1 < VEC ? x0[y].v[(2 * e + 1) % VEC]
                                                        : x1[y].v[(2 * e + 1) % VEC])
                               : load_f(x1[y].v[e]);
            const T g0 = round_to<T>(__fsub_rn(__fmul_rn(c[e], a), __fmul_rn(n[e], f)));
            const T g1 = round_to<T>(__fadd_rn(__fmul_rn(n[e], a), __fmul_rn(c[e], f)));
            if (il) {
              if (2 * e < VEC) y0.v[(2 * e) % VEC] = g0; else y1.v[(2 * e) % VEC] = g0;
              if (2 * e + 1 < VEC) y0.v[(2 * e + 1) % VEC] = g1; else y1.v[(2 * e + 1) % VEC] = g1;
            } else {
              y0.v[e] = g0;
              y1.v[e] = g1;
            }
          }
          x0[y] = y0;
          x1[y] = y1;
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
}

template <typename T>
cudaError_t launch_rope_type(const RopeStep& s, bool tree, int num_sms, cudaStream_t st) {
  constexpr int VEC = 16 / sizeof(T);
  const uintptr_t ptrs = (uintptr_t)s.q | (uintptr_t)s.k | (uintptr_t)s.v | (uintptr_t)s.q_out |
                         (uintptr_t)s.k_out | (uintptr_t)s.k_cache | (uintptr_t)s.v_cache |
                         (uintptr_t)s.out;
  const long long strides = s.q_stride | s.k_stride | s.v_stride | s.q_out_stride | s.k_out_stride;
  // 16-byte accesses: whole packs in the rotated and in the copied dims, and
  // every row on a 16-byte boundary
  const bool wide = (ptrs & 15) == 0 && strides % VEC == 0 && s.rt.rot / 2 % VEC == 0 &&
                    (s.d - s.rt.rot) % (2 * VEC) == 0;
  const int most = num_sms * 16;  // CTAs of 128 threads an SM holds
  const dim3 grid(s.tokens < most ? s.tokens : most);
  if (wide)
    return tree ? launch_dependent(pva_rope_kernel<T, VEC, true>, grid, dim3(kRopeThreads), 0, st, s)
                : launch_dependent(pva_rope_kernel<T, VEC, false>, grid, dim3(kRopeThreads), 0, st, s);
  return tree ? launch_dependent(pva_rope_kernel<T, 1, true>, grid, dim3(kRopeThreads), 0, st, s)
              : launch_dependent(pva_rope_kernel<T, 1, false>, grid, dim3(kRopeThreads), 0, st, s);
}

}  // namespace

cudaError_t launch_rope(const RopeStep& s, int dtype, bool tree, int num_sms, cudaStream_t st) {
  if (s.tokens == 0) return cudaSuccess;
  switch (dtype) {
    case PVA_F32: return launch_rope_type<float>(s, tree, num_sms, st);
    case PVA_F16: return launch_rope_type<__half>(s, tree, num_sms, st);
    default: return launch_rope_type<__nv_bfloat16>(s, tree, num_sms, st);
  }
}

namespace host {

int check_rope(const void* cos_cache, const void* sin_cache, int rot, int rows, int interleaved,
               int n_axes, const int32_t* sections, int axes_interleaved, int rotary_dtype,
               int dtype, int d, RopeTable* t) {
  if (rot < 2 || rot % 2 != 0 || rot > d)
    return fail(PVA_ERR_INVALID_ARG, "rotary_dim must be even with 2 <= rotary_dim <= head_size");
  if (!cos_cache || !sin_cache || rows < 1)
    return fail(PVA_ERR_INVALID_ARG, "rotary embedding needs cos/sin tables with rows >= 1");
  if (rotary_dtype != PVA_F32 && !(rotary_dtype == PVA_F16 && dtype != PVA_F32))
    return fail(PVA_ERR_INVALID_ARG, "cos/sin tables must be f32, or f16 with f16/bf16 rows");
  if (n_axes < 1 || n_axes > kMaxAxes)
    return fail(PVA_ERR_INVALID_ARG, "the number of position axes must be 1 to 4");
  if (n_axes > 1 && !sections)
    return fail(PVA_ERR_INVALID_ARG, "several position axes need their sections");
  const int half = rot / 2;
  t->cos = cos_cache;
  t->sin = sin_cache;
  t->is_f16 = rotary_dtype == PVA_F16 ? 1 : 0;
  t->rot = rot;
  t->rows = rows;
  t->interleaved = interleaved ? 1 : 0;
  t->n_axes = n_axes;
  t->axes_interleaved = axes_interleaved ? 1 : 0;
  t->inverse = 0;
  long long sum = 0;
  for (int a = 0; a < kMaxAxes; ++a) {
    t->sections[a] = a >= n_axes ? 0 : sections ? sections[a] : half;
    if (t->sections[a] < 0) return fail(PVA_ERR_INVALID_ARG, "a section is negative");
    sum += t->sections[a];
    // interleaved: axis a > 0 has the pairs a, a + n, ..., a + n (section - 1)
    if (axes_interleaved && a > 0 && a < n_axes && t->sections[a] > 0 &&
        a + (long long)n_axes * (t->sections[a] - 1) >= half)
      return fail(PVA_ERR_INVALID_ARG, "an interleaved section reaches past the last pair");
  }
  if (sum != half) return fail(PVA_ERR_INVALID_ARG, "the sections must add up to rotary_dim / 2");
  return PVA_OK;
}

}  // namespace host
}  // namespace pva

namespace {

// Element ranges [base, base + extent) of strided [tokens, heads, d] tensors.
bool apart(const void* a, long long na, const void* b, long long nb, size_t size) {
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return x + (size_t)na * size <= y || y + (size_t)nb * size <= x;
}

}  // namespace

extern "C" int pva_rope_axes(const void* q, const void* k, void* q_out, void* k_out,
                             const void* cos_cache, const void* sin_cache,
                             const int64_t* position_ids, int tokens, int num_heads,
                             int kv_num_heads, int head_size, int64_t q_stride, int64_t k_stride,
                             int64_t q_out_stride, int64_t k_out_stride, int rotary_dim,
                             int cache_rows, int rotary_interleaved, int n_axes,
                             const int32_t* sections, int axes_interleaved, int inverse,
                             int rotary_dtype, const void* v, int64_t v_stride, void* k_cache,
                             void* v_cache, const int64_t* slot_map, int n_blocks, int page_size,
                             int dtype, void* stream_) {
  return guarded([&]() -> int {
    if (dtype != PVA_F32 && dtype != PVA_F16 && dtype != PVA_BF16)
      return fail(PVA_ERR_INVALID_ARG, "dtype must be 0 (f32), 1 (f16) or 2 (bf16)");
    if (tokens < 0) return fail(PVA_ERR_INVALID_ARG, "tokens must be >= 0");
    if (tokens == 0) return PVA_OK;
    if (!q && !k) return fail(PVA_ERR_INVALID_ARG, "q or k is needed");
    if ((q && num_heads < 1) || (k && kv_num_heads < 1))
      return fail(PVA_ERR_INVALID_ARG, "head counts must be positive");
    if (head_size < 2 || head_size > 256 || head_size % 2 != 0)
      return fail(PVA_ERR_UNSUPPORTED, "head_size must be even, 2 to 256");
    if ((q != nullptr) != (q_out != nullptr))
      return fail(PVA_ERR_INVALID_ARG, "q and q_out come together");
    if (!position_ids) return fail(PVA_ERR_INVALID_ARG, "null position_ids pointer");
    const bool cache = k_cache || v_cache || slot_map || v;
    if (cache && !(k && v && k_cache && v_cache && slot_map))
      return fail(PVA_ERR_INVALID_ARG, "the cache write needs k, v, both caches and slot_map");
    if (cache && inverse)
      return fail(PVA_ERR_INVALID_ARG, "the inverse rotation does not write the cache");
    if (k && !k_out && !cache) return fail(PVA_ERR_INVALID_ARG, "k needs k_out or the cache");
    if (k_out && !k) return fail(PVA_ERR_INVALID_ARG, "k_out without k");
    if (cache && (n_blocks < 1 || page_size < 1))
      return fail(PVA_ERR_INVALID_ARG, "need n_blocks >= 1 and page_size >= 1");
    const long long qw = (long long)num_heads * head_size, kw = (long long)kv_num_heads * head_size;
    if ((q && (q_stride < qw || q_out_stride < qw)) || (k && k_stride < kw) ||
        (k_out && k_out_stride < kw) || (cache && v_stride < kw))
      return fail(PVA_ERR_INVALID_ARG, "a token stride is smaller than the token's heads");
    RopeStep s{};
    int rc = check_rope(cos_cache, sin_cache, rotary_dim, cache_rows, rotary_interleaved, n_axes,
                        sections, axes_interleaved, rotary_dtype, dtype, head_size, &s.rt);
    if (rc != PVA_OK) return rc;
    const size_t size = dtype == PVA_F32 ? 4 : 2;
    const uintptr_t mis = (uintptr_t)q | (uintptr_t)k | (uintptr_t)v | (uintptr_t)q_out |
                          (uintptr_t)k_out | (uintptr_t)k_cache | (uintptr_t)v_cache;
    if (mis % size) return fail(PVA_ERR_INVALID_ARG, "a tensor is not aligned to its elements");
    // An output may be its own input (the same address and stride); otherwise
    // no output may overlap an input or the other output.
    struct Range { const void* p; long long n, stride; };
    auto range = [&](const void* p, long long stride, long long w) {
      return Range{p, p ? (tokens - 1) * stride + w : 0, stride};
    };
    const Range in[3] = {range(q, q_stride, qw), range(k, k_stride, kw),
                         range(cache ? v : nullptr, v_stride, kw)};
    const Range out[2] = {range(q_out, q_out_stride, qw), range(k_out, k_out_stride, kw)};
    // rows of one projection interleave: two slices of it do not meet
    auto meet = [&](const Range& a, long long wa, const Range& b, long long wb) {
      if (!a.p || !b.p || apart(a.p, a.n, b.p, b.n, size)) return false;
      if (a.stride != b.stride) return true;
      const long long st = a.stride * (long long)size;
      long long off = ((long long)((intptr_t)b.p - (intptr_t)a.p)) % st;
      if (off < 0) off += st;
      return !(off >= wa * (long long)size && off + wb * (long long)size <= st);
    };
    const long long w_in[3] = {qw, kw, kw}, w_out[2] = {qw, kw};
    for (int o = 0; o < 2; ++o) {
      for (int i = 0; i < 3; ++i) {
        if (o == i && out[o].p == in[i].p && out[o].stride == in[i].stride) continue;
        if (meet(out[o], w_out[o], in[i], w_in[i]))
          return fail(PVA_ERR_INVALID_ARG, "an output overlaps an input it is not in place of");
      }
    }
    if (meet(out[0], qw, out[1], kw))
      return fail(PVA_ERR_INVALID_ARG, "q_out and k_out overlap");
    s.q = q;
    s.k = k;
    s.v = cache ? v : nullptr;
    s.q_out = q_out;
    s.k_out = k_out;
    s.k_cache = k_cache;
    s.v_cache = v_cache;
    s.q_stride = q ? q_stride : 0;
    s.k_stride = k ? k_stride : 0;
    s.v_stride = cache ? v_stride : 0;
    s.q_out_stride = q ? q_out_stride : 0;
    s.k_out_stride = k_out ? k_out_stride : 0;
    s.tokens = tokens;
    s.H = num_heads;
    s.Hkv = kv_num_heads;
    s.d = head_size;
    s.pos = position_ids;
    s.slots = slot_map;
    s.page = cache ? page_size : 1;
    s.n_slots = cache ? (long long)n_blocks * page_size : 0;
    s.rt.inverse = inverse ? 1 : 0;
    const cudaStream_t stream = static_cast<cudaStream_t>(stream_);
    std::lock_guard<std::mutex> lock(api_mutex());
    CallContext c;
    if ((rc = acquire(stream, 0, &c)) != PVA_OK) return rc;
    s.status = c.status;
    const cudaError_t e = launch_rope(s, dtype, false, c.num_sms, stream);
    return e == cudaSuccess ? PVA_OK : cuda_fail(e, "rotary launch");
  });
}
