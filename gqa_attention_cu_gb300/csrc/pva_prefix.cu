// Attention of sequences that share prefixes (pva_gqa_prefix): host side, front end,
// fp32 attention and the join.
//
//   front end (pva_line.cuh)  bounds and block table of every entry (prefix or
//       sequence), and the line of places (pva_prefix.cuh).
//   attention                one piece of the line per CTA.
//   pva_prefix_join_kernel   out and lse of every query row from its parts; it looks up
//       where they lie while the attention runs (26.5 to 20.4 us for two requests).
//
// 64 sequences with 100 to 2000 own rows behind 32,768 shared ones, 32 query and 8 kv
// heads of 128 bf16: 86 us, 4.8 TB/s (floor 61); the attention is 75, half of it the
// prefix, whose tiles the tensor cores and the softmax take 1.3 us each for (0.98
// PFLOP/s), half own rows at 1.3 us a tile, which is memory.  Prefixes in the paired
// kernel in a launch of their own: 38 us and 50 for own rows, but the sums that 152
// pieces of 256 rows leave are 21 MB, and the whole 125 us.
#include <limits.h>
#include <math.h>

#include "pva_line.cuh"
#include "pva_prefix.cuh"
#include "pva_tree_f32.cuh"

using namespace pva;
using namespace pva::host;

namespace pva {
namespace {

// The entries on the line (pva_line.cuh): prefixes, then sequences.
struct PrefixFront {
  PrefixParams p;
  __device__ __forceinline__ int entries() const { return p.P + p.B; }
  __device__ __forceinline__ int32_t* start() const { return p.tile_start; }
  // Entries whose rows no token in use sees are idle: nothing of them is read, nor has
  // their table (or a prefix's length) to be sound.  (What depends on nothing is loaded
  // first.)
  __device__ __forceinline__ uint32_t check(int e, int i0, int n, bool& off, bool& idle) const {
    const bool is_prefix = e < p.P;
    const int b = is_prefix ? e : e - p.P;
    const int keys = is_prefix ? p.prefix_keys[b] : p.keys[b];
    const int32_t* table = is_prefix ? p.prefix_table : p.table;
    const int width = is_prefix ? p.prefix_blocks : p.max_blocks;
    const int first = !is_prefix ? b : p.prefix_start ? p.prefix_start[e] : 0;
    const int end = !is_prefix ? b + 1 : p.prefix_start ? p.prefix_start[e + 1] : p.B;
    int tokens = tree_nodes(p, min(max(first, 0), p.B - 1));
    const long long room = (long long)width * p.page;
    const bool some_off = table && line::off_pool(table + (size_t)b * width, (int)min((long long)keys, room), p.page,
                                                  p.n_blocks, i0, n);
    if (is_prefix) {
      if (first < 0 || end < first || end > p.B || (b == 0 && first != 0) || (b == p.P - 1 && end != p.B))
        return PVA_DEV_PREFIX;
      for (int i = first + 1 + (int)(threadIdx.x & 31); tokens == 0 && i - (int)(threadIdx.x & 31) < end; i += 32)
        tokens = __any_sync(0xffffffffu, i < end && tree_nodes(p, i) != 0);
      idle = first == end || tokens == 0;
      if (idle) return 0u;
      if (keys < 0 || keys > room) return PVA_DEV_KV_LEN;
      off = some_off;
    } else {
      if (tokens < 0 || tokens > p.T || tokens > keys || keys < 0 || keys > room) return PVA_DEV_KV_LEN;
      idle = tokens == 0;
      off = some_off && !idle;
    }
    return 0u;
  }
  __device__ __forceinline__ long long places(int e) const {
    PrefixEntry x = prefix_entry(p, e);
    x.keys = min(x.keys, INT_MAX - 65536);  // (an idle prefix's may be anything)
    return x.per_head(p) * p.Hkv;
  }
  __device__ __forceinline__ void publish(long long sum, uint32_t found, bool latched) const {
    if (!found && sum > INT_MAX - 4ll * p.pieces) found = PVA_DEV_TOO_MANY;
    if (found) atomicOr(p.status, found);
    const bool ok = !found && !latched;
    const int all = ok ? (int)sum : 0, even = (all + p.pieces - 1) / p.pieces;
    int chunk = even > p.min_chunk ? even : p.min_chunk;
    // One prefix of several query tiles: where it costs little, its items are all cut
    // alike, so that the CTAs of the same keys read them at the same time, from L2 (64
    // sequences behind 32,768 rows, with item costs that cut them otherwise: 113 to 101 us).
    if (all > 0 && p.P == 1) {
      const PrefixEntry head = prefix_entry(p, 0);
      const int per = head.places(p);
      if (head.q_tiles(p) > 1 && per > chunk) {
        const int alike = (per + per / chunk - 1) / (per / chunk);
        if (alike <= chunk + chunk / 8) chunk = alike;
      }
    }
    p.tile_start[entries()] = all;
    p.hdr[0] = ok;
    p.hdr[1] = all;
    p.hdr[2] = chunk;
  }
};

// out = sum_c 2^(m_c - M) O_c / sum_c 2^(m_c - M) l_c over a row's parts c, the prefix's
// and then its own, M = max m_c; lse = ln 2 (M + log2 of the lower sum).  One warp per
// query row: the lanes hold the places and weights of 32 parts at a time, and V
// channels, V * 32 at once.
template <typename T, int V>
__global__ void __launch_bounds__(256) pva_prefix_join_kernel(PrefixParams p) {
  struct alignas(4 * V) Part { float v[V]; };
  struct alignas(sizeof(T) * V) Out { T v[V]; };
  allow_next_grid();
  // The attention let this kernel start when all work before it was done: only its sums
  // have to be waited for.
  const int lane = threadIdx.x & 31;
  const long long at_row = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);  // (token of the batch, head)
  if (at_row >= (long long)p.B * p.T * p.H) return;
  const int tok = (int)(at_row / p.H), head = (int)(at_row - (long long)tok * p.H), b = tok / p.T, t = tok - b * p.T;
  const int h = head / p.G, g = head - h * p.G;
  const float NEG_INF = __int_as_float(0xff800000);
  // parts of kind 0 (the prefix) and 1 (own rows): the item's places and pieces
  int first[2] = {0, 0}, parts[2] = {0, 0}, in_tile[2], per[2], seen[2], x0[2];
  const int chunk = p.hdr[2];
  if (p.hdr[0] && t < tree_nodes(p, b)) {
#pragma unroll
    for (int kind = 0; kind < 2; ++kind) {
      const int e = kind ? p.P + b : p.prefix_start ? tree_find(p.prefix_start, p.P, b) : 0;
      const PrefixEntry entry = prefix_entry(p, e);
      per[kind] = entry.places(p);
      if (per[kind] == 0) continue;
      const int row = (tok - entry.tok0) * p.G + g, qt = row / p.rows;
      in_tile[kind] = row - qt * p.rows;
      seen[kind] = entry.seen(p, qt);
      x0[kind] = p.tile_start[e] + (h * entry.q_tiles(p) + qt) * per[kind];
      first[kind] = x0[kind] / chunk;
      parts[kind] = (x0[kind] + per[kind] - 1) / chunk - first[kind] + 1;
    }
  }
  // the place of part i, or -1 where a piece holds none of the item's tiles
  auto place = [&](int i) -> long long {
    const int kind = i >= parts[0];
    const int c = kind ? i - parts[0] : i;
    if (parts[kind] == 1) return p.row_at + (kind ? (long long)p.B * p.T * p.H : 0ll) + at_row;
    const int piece = first[kind] + c;
    const int begin = piece * chunk - x0[kind];  // places of the item before the piece
    const int into = max(begin, 0), take = min(per[kind], begin + chunk) - into;
    int from, to;
    prefix_tiles(p, !kind, into, take, seen[kind], from, to);
    return from < to ? (long long)tree_slot(piece, into == 0) * p.rows + in_tile[kind] : -1ll;
  };
  const int n = parts[0] + parts[1];
  long long at = lane < n ? place(lane) : -1;  // of parts 0 .. 31
  wait_prior_grid();
  if (!*(volatile int32_t*)p.hdr) return;  // rejected, or given up
  float2 ml = at >= 0 ? p.part_ml[at] : make_float2(NEG_INF, 0.0f);
  float m = ml.x;
  for (int i = 32 + lane; i < n; i += 32) {
    const long long x = place(i);
    if (x >= 0) m = fmaxf(m, p.part_ml[x].x);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  const float top = m == NEG_INF ? 0.0f : m;
  T* out = static_cast<T*>(p.out) + at_row * p.d;
  float l = 0.0f;
  for (int d0 = 0; d0 < p.d; d0 += 32 * V) {
    const int ch = d0 + lane * V;
    const bool in = ch < p.d;
    float acc[V];
    l = 0.0f;
#pragma unroll
    for (int e = 0; e < V; ++e) acc[e] = 0.0f;
    for (int i0 = 0; i0 < n; i0 += 32) {
      if (n > 32) {
        at = i0 + lane < n ? place(i0 + lane) : -1;
        ml = at >= 0 ? p.part_ml[at] : make_float2(NEG_INF, 0.0f);
      }
      const float w = exp2f(ml.x - top), wl = w * ml.y;  // 0 where there is no part
      const int k = min(32, n - i0);
#pragma unroll 8
      for (int i = 0; i < k; ++i) {
        const long long from = __shfl_sync(0xffffffffu, at, i);
        const float wi = __shfl_sync(0xffffffffu, w, i);
        l += __shfl_sync(0xffffffffu, wl, i);
        if (in && from >= 0) {
          const Part o = *reinterpret_cast<const Part*>(p.part_o + from * p.d + ch);
#pragma unroll
          for (int e = 0; e < V; ++e) acc[e] = fmaf(wi, o.v[e], acc[e]);
        }
      }
    }
    const float inv = l != 0.0f ? 1.0f / l : 0.0f;
    if (in) {
      Out o;
#pragma unroll
      for (int e = 0; e < V; ++e) o.v[e] = static_cast<T>(acc[e] * inv);
      *reinterpret_cast<Out*>(out + ch) = o;
    }
  }
  if (p.lse && lane == 0) p.lse[at_row] = m == NEG_INF ? NEG_INF : (m + log2f(l)) * 0.6931471805599453f;
}

template <typename T, int V>
cudaError_t launch_join(const PrefixParams& p, cudaStream_t s) {
  const long long rows = (long long)p.B * p.T * p.H;
  return launch_dependent(pva_prefix_join_kernel<T, V>, dim3((unsigned)((rows + 7) / 8)), dim3(256), 0, s, p);
}

int gqa_prefix(const void* q, const void* k_cache, const void* v_cache, const int32_t* lens, const int32_t* q_lens,
               const int32_t* block_table, const int32_t* prefix_lens, const int32_t* prefix_start,
               const int32_t* prefix_table, void* out, float* lse, int B, int T, int P, int n_blocks, int page_size,
               int max_blocks, int prefix_blocks, int H, int Hkv, int d, float scale, float softcap, int dtype,
               cudaStream_t stream) {
  if (!q || !k_cache || !v_cache || !lens || !prefix_lens || !out)
    return fail(PVA_ERR_INVALID_ARG, "null q, cache, lens, prefix_lens or out pointer");
  if (B < 1 || T < 1 || P < 1 || n_blocks < 1 || page_size < 1)
    return fail(PVA_ERR_INVALID_ARG, "need B >= 1, tokens >= 1, prefixes >= 1, n_blocks >= 1, page_size >= 1");
  if (!prefix_start && P != 1)
    return fail(PVA_ERR_INVALID_ARG, "several prefixes need prefix_start");
  if (H < 1 || Hkv < 1 || H % Hkv != 0)
    return fail(PVA_ERR_INVALID_ARG, "num_heads must be a positive multiple of a positive kv_num_heads");
  if (dtype != PVA_F32 && dtype != PVA_F16 && dtype != PVA_BF16)
    return fail(PVA_ERR_INVALID_ARG, "dtype must be 0 (f32), 1 (f16) or 2 (bf16)");
  if (!isfinite(scale) || !isfinite(softcap))
    return fail(PVA_ERR_INVALID_ARG, "scale and softcap must be finite");
  const bool tc = dtype != PVA_F32;
  if (tc ? d != 64 && d != 96 && d != 128 && d != 192 && d != 256 : d < 2 || d > 256 || d % 2 != 0)
    return fail(PVA_ERR_UNSUPPORTED,
                "head_size must be 64, 96, 128, 192 or 256 (f16/bf16), or even and at most 256 (f32)");
  const int G = H / Hkv;
  if (G > 128) return fail(PVA_ERR_UNSUPPORTED, "num_heads / kv_num_heads must be at most 128");
  if ((block_table != nullptr) != (prefix_table != nullptr))
    return fail(PVA_ERR_INVALID_ARG, "block_table and prefix_table come together");
  if (block_table) {
    if (max_blocks < 1 || prefix_blocks < 1) return fail(PVA_ERR_INVALID_ARG, "a table's width must be >= 1");
    if (page_size < 16 || (page_size & (page_size - 1)) != 0)
      return fail(PVA_ERR_UNSUPPORTED, "page_size must be a power of two of at least 16");
  } else {
    if ((long long)n_blocks != (long long)B + P)
      return fail(PVA_ERR_INVALID_ARG, "without tables the cache has one block a sequence and then one a prefix");
    max_blocks = prefix_blocks = 1;
  }
  if ((long long)B * T > INT_MAX - 65536 || (long long)B * T * G > INT_MAX / 2 || (long long)B * T * H / 8 > INT_MAX - 8 ||
      (long long)max_blocks * page_size > INT_MAX - 65536 || (long long)prefix_blocks * page_size > INT_MAX - 65536 ||
      (long long)n_blocks * Hkv > INT_MAX || (long long)B + P > INT_MAX - 65536)
    return fail(PVA_ERR_INVALID_ARG, "cache or token extents do not fit in int32");
  const size_t size = tc ? 2 : 4;
  const uintptr_t mis = (uintptr_t)q | (uintptr_t)k_cache | (uintptr_t)v_cache | (uintptr_t)out;
  if (tc && (mis & 15)) return fail(PVA_ERR_INVALID_ARG, "q, caches and out must be 16-byte aligned");
  if (mis % size || (uintptr_t)lse & 3) return fail(PVA_ERR_INVALID_ARG, "a tensor is not aligned to its elements");

  PrefixParams p{};
  p.keys = lens;
  p.lens = q_lens;
  p.table = block_table;
  p.prefix_keys = prefix_lens;
  p.prefix_start = prefix_start;
  p.prefix_table = prefix_table;
  p.P = P;
  p.prefix_blocks = prefix_blocks;
  p.B = B;
  p.T = T;
  p.H = H;
  p.Hkv = Hkv;
  p.G = G;
  p.d = d;
  p.page = page_size;
  p.max_blocks = max_blocks;
  p.n_blocks = n_blocks;
  const float s = scale != 0.0f ? scale : 1.0f / sqrtf((float)d);
  p.negated = tc && s < 0.0f;
  p.scale = tc ? fabsf(s) : s;
  p.softcap = softcap_size(softcap, p.scale);
  if (p.softcap != 0.0f) {
    // Nearest polynomials up to kNearTanh and kMidTanh (pva_tree_tile.cuh); above
    // kCapOfExp the series as in pva_gqa_tree, but while softcap times the term that it
    // leaves out is below 2^-18, for the sums that are given out as f32.
    const double cap = p.softcap;
    const double t = tile::cap_form(p.softcap) == tile::kCap
                         ? tile::kNearTanh
                         : fmin(0.25, pow(ldexp(1.0, -18) * 315.0 / 17.0 / cap, 1.0 / 7.0));
    p.series_to = (float)fmin(t * cap / fabs(p.scale), 1e9);
    if (fabs(p.scale) > 1e7 * cap) p.series_to = -1.0f;  // its coefficients would not be finite
    p.mid_to = (float)fmin(tile::kMidTanh * cap / fabs(p.scale), 1e9);
  }
  p.q_parts = 1;
  const long long R = (long long)B * T * G;
  p.tile_rows = tc ? G * (kTcRows / G) : R <= 8 ? 8 : R <= 16 ? 16 : 24;  // f32: R of the whole batch
  p.own_rows = tc && (long long)T * G < p.tile_rows ? T * G : p.tile_rows;
  // The paired kernel takes batches of more than two tiles of rows: its tile pair costs
  // 1.7 us where two tiles are 2.6, but a sequence's few own rows have its two score
  // buffers' place alone (d = 128, 32,768 shared rows, us, one-tile and paired kernel: 64
  // sequences of 100 to 2000 own rows x 4 heads 97 and 104, 128 of 100 to 1000 156 and
  // 134, 256 of 10 to 100 211 and 173).  So have prefixes with few rows, which the rule
  // does not tell apart: 128 sequences of 200 own rows behind 2 prefixes of 16,000 rows
  // 101 and 89, behind 4 or 8 of 8000 79 and 81, 101 and 102, behind 64 of 1000 99 and 113.
  // With a softcap two threads a row share the special functions in the one-tile kernel
  // (d = 64, 64 sequences: 115 and 126).
  const bool pair = tc && d <= 192 && R > 2 * p.tile_rows && p.softcap == 0.0f;
  p.rows = pair ? 2 * p.tile_rows : p.tile_rows;
  p.bn = tc ? tree_keys(d) : kTreeKeysF32;
  // Places: a key tile 4, an item's queries, pipeline and sums 8 (a prefix's fill a tile:
  // 16), a prefix's tile in the paired kernel 5 (6: 154 instead of 134 us above).  Own
  // items at 4 or 16 instead of 8: 114 and 116 instead of 96 us.
  p.tile_cost[0] = 4;
  p.tile_cost[1] = pair ? 5 : 4;
  p.item_cost[0] = 8;
  p.item_cost[1] = 16;
  p.min_chunk = 2 * p.tile_cost[0];  // two key tiles, as in pva_gqa_tree
  p.q = const_cast<void*>(q);
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.out = out;
  p.lse = lse;

  std::lock_guard<std::mutex> lock(api_mutex());
  int sms = 0;
  int rc = sm_count(&sms);
  if (rc != PVA_OK) return rc;
  p.pieces = tc ? sms : f32::ctas(p.rows, d) * sms;
  size_t used = 0;
  auto take = [&](size_t bytes) {
    const size_t at = used;
    used += (bytes + 255) / 256 * 256;
    return at;
  };
  p.row_at = 2ll * p.pieces * p.rows;
  const size_t places = (size_t)p.row_at + 2 * (size_t)B * T * H;
  const size_t at_hdr = take(32), at_start = take(4 * ((size_t)B + P + 1));
  const size_t at_o = take(sizeof(float) * places * d), at_ml = take(sizeof(float2) * places);
  CallContext c;
  if ((rc = acquire(stream, used, &c)) != PVA_OK) return rc;
  p.status = c.status;
  p.hold_ns = selftest_hold_ns();
  p.hdr = reinterpret_cast<int32_t*>(c.buf + at_hdr);
  p.tile_start = reinterpret_cast<int32_t*>(c.buf + at_start);
  p.part_o = reinterpret_cast<float*>(c.buf + at_o);
  p.part_ml = reinterpret_cast<float2*>(c.buf + at_ml);
  PrefixQueries tq;
  CUtensorMap tk, tv;
  if (tc) {
    const int box = block_table && page_size < p.bn ? page_size : p.bn;
    const long long planes = (long long)n_blocks * Hkv;
    if ((rc = get_encoder()) != PVA_OK ||
        (rc = encode_rows_map(&tq.tile, q, dtype, d, H, (long long)B * T, G, p.tile_rows / G)) != PVA_OK ||
        (rc = encode_rows_map(&tq.own, q, dtype, d, H, (long long)B * T, G, p.own_rows / G)) != PVA_OK ||
        (rc = encode_plane_map(&tk, k_cache, dtype, d, page_size, planes, 64, box, true)) != PVA_OK ||
        (rc = encode_plane_map(&tv, v_cache, dtype, d, page_size, planes, 64, box, true)) != PVA_OK)
      return rc;
  }
  cudaError_t e = line::launch_front(PrefixFront{p}, P + B, max_blocks > prefix_blocks ? max_blocks : prefix_blocks, c.status,
                                     stream);
  if (e != cudaSuccess) return cuda_fail(e, "prefix front-end launch");
  e = pair ? launch_prefix_pair(p, dtype, tq, tk, tv, stream)
      : tc ? launch_prefix_tc(p, dtype, tq, tk, tv, stream)
           : f32::launch<PrefixWork>(p, stream);
  if (e != cudaSuccess) return cuda_fail(e, "prefix attention launch");
  e = dtype == PVA_BF16 ? launch_join<__nv_bfloat16, 4>(p, stream)
      : dtype == PVA_F16 ? launch_join<__half, 4>(p, stream)
      // four channels a lane; one where rows of fp32 do not lie on 16-byte boundaries
      : d % 4 == 0 && ((uintptr_t)out & 15) == 0 ? launch_join<float, 4>(p, stream)
                                                 : launch_join<float, 1>(p, stream);
  return e == cudaSuccess ? PVA_OK : cuda_fail(e, "prefix join launch");
}

}  // namespace
}  // namespace pva

extern "C" int pva_gqa_prefix(const void* q, const void* k_cache, const void* v_cache, const int32_t* lens,
                              const int32_t* q_lens, const int32_t* block_table, const int32_t* prefix_lens,
                              const int32_t* prefix_start, const int32_t* prefix_table, void* out, float* lse, int B,
                              int tokens, int prefixes, int n_blocks, int page_size, int max_blocks, int prefix_blocks,
                              int num_heads, int kv_num_heads, int head_size, float scale, float softcap, int dtype,
                              void* stream) {
  return guarded([&]() -> int {
    return gqa_prefix(q, k_cache, v_cache, lens, q_lens, block_table, prefix_lens, prefix_start, prefix_table, out, lse,
                      B, tokens, prefixes, n_blocks, page_size, max_blocks, prefix_blocks, num_heads, kv_num_heads,
                      head_size, scale, softcap, dtype, static_cast<cudaStream_t>(stream));
  });
}
