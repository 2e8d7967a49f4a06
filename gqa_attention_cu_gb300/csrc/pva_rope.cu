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
// Every q, k and v row is read once and written once (twice where a key goes to
// k_out and the cache), so memory is the floor; what bounds it now is how many loads
// are under way (DRAM 57% busy, issue slots 56%).  A CTA takes one token at a time:
// the cos and sin of its pairs lie in shared memory, fetched while the token before
// is turned, and its threads walk over the token's head rows with them, so the
// tables and the axis of each pair are looked up once a token and not once a head;
// two rows' four loads of 16 bytes are in flight per thread.  16,001 tokens with 32
// + 8 + 8 head rows of 128 bf16 and the cache written as well: 85 us, 5.0 TB/s of
// 426 MB (63 us at the copy rate).  In the tree step (two parts of q, depths from
// the parents): 3000 tokens of 64 + 8 + 8 rows of 64 f16 in 24 us, 500 tokens of 32
// + 8 + 8 rows of 128 in 12 us with its launch.
#include <limits.h>

#include "pva_rope.cuh"

using namespace pva;
using namespace pva::host;

namespace pva {
namespace {

// Depth of a node by the way up, for kernels that do not wait for the front end's:
// whatever the parents are, at most T steps.
__device__ __forceinline__ int walk_up(const RopeStep& s, int tok) {
  const int node = tok % s.T;
  const int32_t* parents = s.parents + (tok - node);
  int depth = 0;
  for (int a = node, up; (up = load<true>(parents + a)) >= 0 && up < a; a = up) ++depth;
  return depth;
}

// The tree form looks everything up before the front end has finished, which it
// follows on the stream: the front end lets it start only when all work before
// the step is complete.  What it waits for is the permission to write -- and
// the depths of large trees, whose way up is too long to walk here.
constexpr int kWalkT = 64;
// CTAs an SM holds of the tree form, and as many are launched (500-token chunks of 6
// sequences in bf16, the whole step: 6 an SM 186.4, 7 184.0, 8 with a few registers
// spilled 189.6 us).
constexpr int kTreeCtas = 7;

template <typename T, int VEC, bool TREE>
__global__ void __launch_bounds__(kRopeThreads, TREE ? kTreeCtas : kRopeCtas) pva_rope_kernel(RopeStep s) {
  __shared__ RopeToken sh[2];
  allow_next_grid();
  const bool walk = TREE && s.parents && !s.pos && s.rt.rot > 0 && s.T <= kWalkT;
  const bool wait_first = !TREE || (s.parents && !s.pos && s.rt.rot > 0 && !walk);
  if (wait_first) wait_prior_grid();
  rope_tokens<T, VEC, TREE>(
      s, blockIdx.x, gridDim.x, threadIdx.x, 0, sh,
      [&](int tok) { return !s.parents ? tok % s.T : walk ? walk_up(s, tok) : s.depth[tok]; },
      [&]() {
        if (!wait_first) wait_prior_grid();
        return !TREE || s.hdr[0] != 0;
      });
}

template <typename T>
cudaError_t launch_rope_type(const RopeStep& s, bool tree, int num_sms, cudaStream_t st) {
  constexpr int VEC = 16 / sizeof(T);
  const bool wide = rope_wide(s, VEC);
  const int most = num_sms * (tree ? kTreeCtas : kRopeCtas);
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
    if (tokens < 0 || tokens > INT_MAX - 65536)
      return fail(PVA_ERR_INVALID_ARG, "tokens must be >= 0 and fit in int32");
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
