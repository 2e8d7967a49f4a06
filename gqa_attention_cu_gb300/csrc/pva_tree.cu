// One step of a tree of drafted tokens over a KV cache (pva_gqa_tree): host
// side, front end, fp32 attention and the join of split items.  The f16/bf16
// attention kernel is in pva_tree_tc.cu, rotation and append in pva_rope.cu.
//
//   pva_tree_front_kernel  one CTA per sequence: bounds, the block table,
//       positions and parents; each node's ancestors as a bit mask and its
//       depth; the key tiles of each q tile.  The last CTA to finish adds the
//       tiles up and cuts the line of tiles (pva_tree.h) -- or rejects the
//       step, all of it, when any CTA found something wrong.
//   pva_rope_kernel        rotated queries to scratch, new rows to the cache,
//       zeros for unused nodes.
//   pva_tree_warp_front_kernel   the first of these for up to 32 sequences.
//   pva_tree_small_front_kernel  both of these for small steps.
//   attention              one piece of the line per CTA.
//   pva_tree_join_kernel   adds up the parts of items that lie across a cut.
//
// The front end is bound by the latency of its dependent reads (past, block
// table, parents up the tree), so it is as few launches as the step's size
// allows: one request of 8 nodes is ready for the attention after 8 us in one
// launch; 16 sequences of 32 nodes after 16 us, 10 of them the one-CTA front end,
// which the rotation's table lookups and queries run beside.
#include <limits.h>
#include <math.h>

#include "pva_rope.cuh"
#include "pva_tree_f32.cuh"

using namespace pva;
using namespace pva::host;

namespace pva {
namespace {

constexpr int kFrontThreads = 256;
constexpr int kMaxTreeNodes = 1024;
static_assert(kMaxTreeNodes <= 4 * kFrontThreads, "a thread of the front end reads four parents");
// Words of the status block (zero between calls).
constexpr int kWordArrived = 16, kWordBad = 17;

// Steps up to these sizes are checked by every CTA that rotates rows.
constexpr int kSmallB = 16, kSmallT = 64, kSmallNodes = 256, kSmallBlocks = 1024;

// And these by one CTA, a warp per sequence (up to 32 of them).
constexpr int kWarpFrontT = 128,  // four nodes a lane
              kWarpFrontBlocks = 512;

// Checks sequence b and finds its masks, depths and tiles.  N threads (32: a
// warp, else the CTA) work on one sequence; i0 is the caller's place among
// them.  Returns the PVA_DEV_* bits this thread has found; `tiles` is set in the
// group's first warp.  write: store masks, depths and tile starts.
template <int N>
__device__ __forceinline__ uint32_t front_sequence(const TreeParams& p, int b, int past, int n,
                                                   int i0, bool write, int* s_parent,
                                                   int* s_depth, long long& tiles) {
  // Parents and positions of all T nodes are read beside the lengths, whether
  // they are in use or not, and all before any is looked at; the table has to
  // wait for the lengths.  (A tree has at most 4 N nodes.)
  uint32_t bad = 0;
  int up[4];
  if (p.parents) {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (i0 + k * N < p.T) up[k] = p.parents[(size_t)b * p.T + i0 + k * N];
  }
  int off_table = p.T;  // the first node with a position outside the tables
  if (p.rot > 0 && p.pos) {
    for (int a = 0; a < p.n_axes; ++a)
#pragma unroll 4
      for (int i = i0; i < p.T; i += N) {
        const int64_t at = p.pos[((size_t)a * p.B + b) * p.T + i];
        if (at < 0 || at >= p.cache_rows) off_table = min(off_table, i);
      }
  }
  if (n < 0 || n > p.T) bad |= PVA_DEV_TREE;
  if (past < 0 || (long long)past + n > (long long)p.max_blocks * p.page) bad |= PVA_DEV_KV_CACHE;
  const bool sane = bad == 0;
  if (sane && n > 0) {
    // the blocks that hold the rows this step reads and writes
    if (p.table) {
      const long long from = p.window > 0 ? (long long)past + 1 - p.window : 0;
      const int first = from > 0 ? (int)(from / p.page) : 0, end = (past + n - 1) / p.page + 1;
      const int32_t* table = p.table + (size_t)b * p.max_blocks;
#pragma unroll 8
      for (int i = first + i0; i < end; i += N)
        if ((unsigned)table[i] >= (unsigned)p.n_blocks) bad |= PVA_DEV_BLOCKS;
    }
    if (p.parents) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int i = i0 + k * N;
        if (i >= n) continue;
        s_parent[i] = up[k];
        if (up[k] < -1 || up[k] >= i) bad |= PVA_DEV_TREE;
      }
    }
    if (off_table < n) bad |= PVA_DEV_ROPE;
    bool walk;
    if (N == 32) {
      walk = !__any_sync(0xffffffffu, bad);
      __syncwarp();
    } else {
      walk = !__syncthreads_or(bad);
    }
    for (int i = i0; i < n && walk; i += N) {
      int depth = i;
      if (p.parents) {
        // The way up visits falling node indices, so the words of the mask
        // are completed from the node's own word downwards.
        uint32_t* row = p.mask + ((size_t)b * p.T + i) * p.W32;
        if (write)
          for (int w = p.W32 - 1; w > i >> 5; --w) row[w] = 0;
        int w = i >> 5;
        uint32_t bits = 0;
        depth = 0;
        for (int a = i; a >= 0; a = s_parent[a], ++depth) {
          for (; w > a >> 5; --w, bits = 0)
            if (write) row[w] = bits;
          if (p.window <= 0 || depth < p.window) bits |= 1u << (a & 31);
        }
        --depth;
        if (write) {
          for (; w >= 0; --w, bits = 0) row[w] = bits;
          p.depth[(size_t)b * p.T + i] = depth;
        }
        if (s_depth) s_depth[i] = depth;
      }
      if (p.rot > 0 && !p.pos && (long long)past + depth >= p.cache_rows) bad |= PVA_DEV_ROPE;
    }
  }
  // tiles of each q tile, and where it starts within a kv head
  tiles = 0;
  if (i0 < 32) {
    int32_t* qs = p.q_start + (size_t)b * (p.QT + 1);
    long long carry = 0;
    const int qt = sane ? (int)(((long long)n * p.G + p.rows - 1) / p.rows) : 0;
    for (int t0 = 0; t0 <= p.QT; t0 += 32) {
      const int t = t0 + i0;
      int x = 0;
      if (t < qt) {
        int lo, first;
        x = tree_item_tiles(p, past, n, t, lo, first) + p.item_places;
      }
      int upto = x;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, upto, o);
        if (i0 >= o) upto += y;
      }
      if (t <= p.QT && write) qs[t] = (int)(carry + upto - x);
      carry += __shfl_sync(0xffffffffu, upto, 31);
    }
    tiles = carry * p.Hkv;
  }
  return bad;
}

// What the step comes to: `tiles` in all, `bad` found, `latched` before.
__device__ __forceinline__ void front_publish(const TreeParams& p, long long tiles,
                                              long long items, uint32_t bad, bool latched) {
  if (bad) atomicOr(p.status, bad | PVA_DEV_KV_CACHE);
  const bool ok = bad == 0 && !latched;
  const int all = ok ? (int)tiles : 0;
  const int even = (all + p.pieces - 1) / p.pieces;
  p.tile_start[p.B] = all;
  p.hdr[0] = ok ? 1 : 0;
  p.hdr[1] = all;
  const bool whole = ok && p.may_take_items && items >= 6LL * p.pieces && items <= INT_MAX / 2;
  p.hdr[2] = even > p.min_chunk ? even : p.min_chunk;
  p.hdr[3] = whole ? (int)items : 0;
  p.hdr[4] = 0;
}

__device__ __forceinline__ bool too_many(const TreeParams& p, long long tiles) {
  return tiles > INT_MAX - 4 * (long long)p.pieces;
}

__global__ void __launch_bounds__(kFrontThreads) pva_tree_front_kernel(TreeParams p) {
  wait_prior_grid();
  allow_next_grid();  // not before: the next kernel reads the step's inputs at once
  __shared__ int s_parent[kMaxTreeNodes];
  __shared__ uint32_t s_bad;
  __shared__ int s_last;
  __shared__ long long s_sum[kFrontThreads / 32];
  const int b = blockIdx.x, tid = threadIdx.x;
  // what the CTA that finishes last needs besides the others' results
  const bool latched = (*(volatile uint32_t*)p.status & PVA_DEV_KV_CACHE) != 0;
  if (tid == 0) s_bad = 0;
  long long tiles;
  const uint32_t bad = front_sequence<kFrontThreads>(p, b, p.past[b], tree_nodes(p, b), tid, true,
                                                     s_parent, nullptr, tiles);
  __syncthreads();
  if (bad) atomicOr(&s_bad, bad);
  if (tid == 0) {
    if (too_many(p, tiles)) atomicOr(&s_bad, PVA_DEV_TOO_MANY);
    p.tile_start[b] = too_many(p, tiles) ? 0 : (int)tiles;
  }
  __syncthreads();
  if (tid == 0) {
    if (s_bad) atomicOr(p.status + kWordBad, s_bad);
    __threadfence();
    s_last = atomicAdd(p.status + kWordArrived, 1u) == gridDim.x - 1;
  }
  __syncthreads();
  if (!s_last) return;
  // The last CTA: sums of the sequences' tiles, in place.
  __threadfence();
  auto sum_up = [&](auto value, int32_t* start) {
    long long carry = 0;
    for (int b0 = 0; b0 < p.B; b0 += kFrontThreads) {
      const int i = b0 + tid;
      const long long x = i < p.B ? value(i) : 0;
      long long upto = x;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, upto, o);
        if ((tid & 31) >= o) upto += y;
      }
      if ((tid & 31) == 31) s_sum[tid >> 5] = upto;
      __syncthreads();
      long long before = carry, all = carry;
      for (int w = 0; w < kFrontThreads / 32; ++w) {
        if (w < tid >> 5) before += s_sum[w];
        all += s_sum[w];
      }
      if (i < p.B) start[i] = (int)(before + upto - x);
      carry = all;
      __syncthreads();
    }
    return carry;
  };
  const long long carry = sum_up([&](int i) { return (long long)__ldcg(p.tile_start + i); }, p.tile_start);
  long long items = 0;
  if (p.may_take_items)
    items = sum_up(
        [&](int i) {
          const int n = min(max(tree_nodes(p, i), 0), p.T);
          return (long long)((n * p.G + p.rows - 1) / p.rows) * p.Hkv;
        },
        p.item_start);
  if (tid == 0) {
    const uint32_t all_bad = __ldcg(p.status + kWordBad) | (too_many(p, carry) ? PVA_DEV_TOO_MANY : 0u);
    p.status[kWordBad] = 0;  // for the next step
    p.status[kWordArrived] = 0;
    // a step after a rejected one would append after rows that are missing
    front_publish(p, carry, items, all_bad, latched);
  }
}

// The same for up to 32 sequences of short trees, a warp each: one CTA, which
// adds up in shared memory and waits for no other.
__global__ void __launch_bounds__(1024) pva_tree_warp_front_kernel(TreeParams p) {
  wait_prior_grid();
  allow_next_grid();
  __shared__ int s_parent[32][kWarpFrontT];
  __shared__ long long s_tiles[32];
  __shared__ uint32_t s_bad;
  const int tid = threadIdx.x, b = tid >> 5, lane = tid & 31;
  const bool latched = (*(volatile uint32_t*)p.status & PVA_DEV_KV_CACHE) != 0;
  if (tid == 0) s_bad = 0;
  __syncthreads();
  long long tiles;
  const uint32_t bad = front_sequence<32>(p, b, p.past[b], tree_nodes(p, b), lane, true, s_parent[b],
                                          nullptr, tiles);
  if (bad) atomicOr(&s_bad, bad);
  if (lane == 0) s_tiles[b] = tiles;
  __syncthreads();
  if (b > 0) return;
  const int B = blockDim.x >> 5;
  const long long x = lane < B ? s_tiles[lane] : 0;
  long long upto = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += y;
  }
  const long long all = __shfl_sync(0xffffffffu, upto, 31);
  if (lane < B) p.tile_start[lane] = too_many(p, all) ? 0 : (int)(upto - x);
  // few items: by pieces
  if (lane == 0) front_publish(p, all, 0, s_bad | (too_many(p, all) ? PVA_DEV_TOO_MANY : 0u), latched);
}

// A small step's front end and append in one launch.  Every CTA checks the
// whole step, so that none has to wait for another before it writes rows: a
// warp per sequence, a few loads deep.  The first CTA writes the results.
template <typename T, int VEC>
__global__ void __launch_bounds__(kFrontThreads) pva_tree_small_front_kernel(TreeParams p,
                                                                             RopeStep r) {
  allow_next_grid();  // the attention waits for all of this kernel
  wait_prior_grid();
  constexpr int kWarps = kFrontThreads / 32, kAtOnce = kFrontThreads / kRopeThreads;
  __shared__ RopeToken s_rope[kAtOnce][2];
  __shared__ int s_parent[kWarps][kSmallT];
  __shared__ int s_depth[kSmallNodes];
  __shared__ long long s_tiles[kSmallB];
  __shared__ uint32_t s_bad;
  __shared__ int s_past[kSmallB], s_n[kSmallB];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const bool first = blockIdx.x == 0;
  // read before the first CTA may latch this step's own errors, or after: the
  // step is refused either way
  const bool latched = (*(volatile uint32_t*)p.status & PVA_DEV_KV_CACHE) != 0;
  if (tid == 0) s_bad = 0;
  if (tid < p.B) {
    s_past[tid] = p.past[tid];
    s_n[tid] = tree_nodes(p, tid);
  }
  __syncthreads();
  for (int b = warp; b < p.B; b += kWarps) {
    long long tiles;
    const uint32_t bad = front_sequence<32>(p, b, s_past[b], s_n[b], lane, first, s_parent[warp],
                                            s_depth + b * p.T, tiles);
    if (bad) atomicOr(&s_bad, bad);
    if (lane == 0) s_tiles[b] = tiles;
    __syncwarp();
  }
  __syncthreads();
  long long before = 0, all = 0;
  for (int b = 0; b < p.B; ++b) {
    before += b < tid ? s_tiles[b] : 0;
    all += s_tiles[b];
  }
  const uint32_t bad = s_bad | (too_many(p, all) ? PVA_DEV_TOO_MANY : 0u);
  if (first) {
    if (tid < p.B) p.tile_start[tid] = too_many(p, before) ? 0 : (int)before;
    if (tid == 0) front_publish(p, all, 0, bad, latched);  // few items: by pieces
  }
  if (bad || latched) return;
  const int group = tid / kRopeThreads;
  rope_tokens<T, VEC, true>(r, blockIdx.x * kAtOnce + group, gridDim.x * kAtOnce,
                            tid % kRopeThreads, 1 + group, s_rope[group],
                            [&](int tok) { return p.parents ? s_depth[tok] : tok % p.T; },
                            []() { return true; });
}

// out = sum_c 2^(m_c - M) O_c / sum_c 2^(m_c - M) l_c over an item's parts c, in
// the order of the line; M = max m_c.  CTAs (c, y) take the item that piece c
// began and did not finish (the attention kernel names it), one warp per row.
// Lanes hold the weights of 32 parts at a time and V channels of the row, V *
// 32 at once.  So the work is that of the cut items, however many there are:
// 15 MB of parts (500-token chunks of 6 sequences) in 12 us after the attention's
// last CTA, those of 16 sequences of 32 nodes in 7 us.  (32 registers,
// 12 bytes spilled.)
template <typename T, int V>
__global__ void __launch_bounds__(256) pva_tree_join_kernel(TreeParams p) {
  struct alignas(4 * V) Part { float v[V]; };
  struct alignas(sizeof(T) * V) Out { T v[V]; };
  allow_next_grid();
  wait_prior_grid();
  const int lane = threadIdx.x & 31, r = blockIdx.y * 8 + (threadIdx.x >> 5);
  const int c0 = blockIdx.x;
  if (!p.hdr[0]) return;  // rejected, or given up
  const TreeCut it = p.cuts[c0];
  if (r < it.rows) {
    const int row = it.t * p.rows + r, node = row / p.G, n = it.parts;
    // part i: slots of consecutive pieces lie two apart, but for the first
    const float2* ml = p.part_ml + r;
    const float* po = p.part_o + (size_t)r * p.d;
    auto slot = [&](int i) { return (size_t)tree_slot(c0 + i, i == 0) * p.rows; };
    float m = __int_as_float(0xff800000);
    for (int i = lane; i < n; i += 32) m = fmaxf(m, ml[slot(i)].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float top = m == __int_as_float(0xff800000) ? 0.0f : m;
    T* out = static_cast<T*>(p.out) +
             (((size_t)it.b * p.T + node) * p.H + it.h * p.G + row - node * p.G) * p.d;
    for (int d0 = 0; d0 < p.d; d0 += 32 * V) {
      const int at = d0 + lane * V;
      const bool in = at < p.d;
      float acc[V], l = 0.0f;
#pragma unroll
      for (int e = 0; e < V; ++e) acc[e] = 0.0f;
      for (int i0 = 0; i0 < n; i0 += 32) {
        float w = 0.0f, wl = 0.0f;
        if (i0 + lane < n) {
          const float2 v = ml[slot(i0 + lane)];
          w = exp2f(v.x - top);
          wl = w * v.y;
        }
        const int k = min(32, n - i0);
#pragma unroll 8
        for (int i = 0; i < k; ++i) {
          Part o;
          if (in) o = *reinterpret_cast<const Part*>(po + slot(i0 + i) * p.d + at);
          const float wi = __shfl_sync(0xffffffffu, w, i);
          l += __shfl_sync(0xffffffffu, wl, i);
          if (in) {
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
        *reinterpret_cast<Out*>(out + at) = o;
      }
    }
  }
}

template <typename T>
cudaError_t launch_small_front(const TreeParams& p, const RopeStep& r, int num_sms,
                               cudaStream_t s) {
  constexpr int VEC = 16 / sizeof(T);
  constexpr int at_once = kFrontThreads / kRopeThreads;
  const int want = (r.tokens + at_once - 1) / at_once, most = 2 * num_sms;
  const dim3 grid(want < most ? want : most);
  return rope_wide(r, VEC)
             ? launch_dependent(pva_tree_small_front_kernel<T, VEC>, grid, dim3(kFrontThreads), 0, s, p, r)
             : launch_dependent(pva_tree_small_front_kernel<T, 1>, grid, dim3(kFrontThreads), 0, s, p, r);
}

cudaError_t launch_front(const TreeParams& p, const RopeStep& r, int dtype, int num_sms,
                         cudaStream_t s) {
  if (p.B <= kSmallB && p.T <= kSmallT && p.B * p.T <= kSmallNodes &&
      (long long)p.B * p.max_blocks <= kSmallBlocks) {
    switch (dtype) {
      case PVA_F32: return launch_small_front<float>(p, r, num_sms, s);
      case PVA_F16: return launch_small_front<__half>(p, r, num_sms, s);
      default: return launch_small_front<__nv_bfloat16>(p, r, num_sms, s);
    }
  }
  const cudaError_t e =
      p.B <= 32 && p.T <= kWarpFrontT && p.max_blocks <= kWarpFrontBlocks
          ? launch_dependent(pva_tree_warp_front_kernel, dim3(1), dim3(32 * p.B), 0, s, p)
          : launch_dependent(pva_tree_front_kernel, dim3(p.B), dim3(kFrontThreads), 0, s, p);
  if (e != cudaSuccess) return e;
  return launch_rope(r, dtype, true, num_sms, s);
}

cudaError_t launch_join(const TreeParams& p, int dtype, cudaStream_t s) {
  const long long rows = (long long)p.T * p.G;
  const dim3 grid(p.pieces, (unsigned)((rows < p.rows ? rows : p.rows) + 7) / 8);
  // four channels a lane; one where rows of fp32 do not lie on 16-byte boundaries
  switch (dtype) {
    case PVA_F32:
      return p.d % 4 == 0 && ((uintptr_t)p.out & 15) == 0
                 ? launch_dependent(pva_tree_join_kernel<float, 4>, grid, dim3(256), 0, s, p)
                 : launch_dependent(pva_tree_join_kernel<float, 1>, grid, dim3(256), 0, s, p);
    case PVA_F16:
      return launch_dependent(pva_tree_join_kernel<__half, 4>, grid, dim3(256), 0, s, p);
    default:
      return launch_dependent(pva_tree_join_kernel<__nv_bfloat16, 4>, grid, dim3(256), 0, s, p);
  }
}

}  // namespace

cudaError_t launch_tree_f32(const TreeParams& p, cudaStream_t s) {
  return f32::launch<tile::TreeWork>(p, s);
}

}  // namespace pva

namespace {

int gqa_tree(const void* q, const void* k_new, const void* v_new, void* k_cache, void* v_cache,
             const int32_t* past_lens, const int32_t* tree_lens, const int32_t* parents,
             const int32_t* block_table, const void* cos_cache, const void* sin_cache,
             const int64_t* position_ids, void* out, int B, int T, int n_blocks, int page_size,
             int max_blocks, int H, int Hkv, int d, int rot, int cache_rows,
             int rotary_interleaved, int n_axes, const int32_t* sections, int axes_interleaved,
             int rotary_dtype, float scale, float softcap, int window, int dtype,
             cudaStream_t stream) {
  if (!q || !k_new || !v_new || !k_cache || !v_cache || !past_lens || !out)
    return fail(PVA_ERR_INVALID_ARG, "null q, k_new, v_new, cache, past_lens or out pointer");
  if (B < 1 || T < 1 || n_blocks < 1 || page_size < 1)
    return fail(PVA_ERR_INVALID_ARG, "need B >= 1, tokens >= 1, n_blocks >= 1, page_size >= 1");
  if (H < 1 || Hkv < 1 || H % Hkv != 0)
    return fail(PVA_ERR_INVALID_ARG,
                "num_heads must be a positive multiple of a positive kv_num_heads");
  if (dtype != PVA_F32 && dtype != PVA_F16 && dtype != PVA_BF16)
    return fail(PVA_ERR_INVALID_ARG, "dtype must be 0 (f32), 1 (f16) or 2 (bf16)");
  if (!isfinite(scale) || !isfinite(softcap))
    return fail(PVA_ERR_INVALID_ARG, "scale and softcap must be finite");
  const bool tc = dtype != PVA_F32;
  if (tc ? d != 64 && d != 96 && d != 128 && d != 192 && d != 256
         : d < 2 || d > 256 || d % 2 != 0)
    return fail(PVA_ERR_UNSUPPORTED,
                "head_size must be 64, 96, 128, 192 or 256 (f16/bf16), or even and at most 256 (f32)");
  const int G = H / Hkv;
  if (parents && T > kMaxTreeNodes)
    return fail(PVA_ERR_UNSUPPORTED, "a tree has at most 1024 nodes");
  if (block_table) {
    if (max_blocks < 1) return fail(PVA_ERR_INVALID_ARG, "max_blocks must be >= 1");
    if (page_size < 16 || (page_size & (page_size - 1)) != 0)
      return fail(PVA_ERR_UNSUPPORTED, "page_size must be a power of two of at least 16");
  } else {
    if (n_blocks != B)
      return fail(PVA_ERR_INVALID_ARG, "without a block table the cache has one block a sequence");
    max_blocks = 1;
  }
  if ((long long)B * T > INT_MAX - 65536 || (long long)T * G > INT_MAX / 2 ||
      (long long)max_blocks * page_size > INT_MAX - 65536 ||
      (long long)n_blocks * Hkv > INT_MAX)
    return fail(PVA_ERR_INVALID_ARG, "cache or token extents do not fit in int32");
  RopeStep r{};
  int rc;
  if (rot != 0) {
    rc = check_rope(cos_cache, sin_cache, rot, cache_rows, rotary_interleaved, n_axes, sections,
                    axes_interleaved, rotary_dtype, dtype, d, &r.rt);
    if (rc != PVA_OK) return rc;
  }
  const size_t size = tc ? 2 : 4;
  const uintptr_t mis = (uintptr_t)q | (uintptr_t)k_new | (uintptr_t)v_new | (uintptr_t)k_cache |
                        (uintptr_t)v_cache | (uintptr_t)out;
  if (tc && (mis & 15))
    return fail(PVA_ERR_INVALID_ARG, "q, k_new, v_new, caches and out must be 16-byte aligned");
  if (mis % size) return fail(PVA_ERR_INVALID_ARG, "a tensor is not aligned to its elements");

  TreeParams p{};
  p.past = past_lens;
  p.lens = tree_lens;
  p.parents = parents;
  p.table = block_table;
  p.pos = rot ? position_ids : nullptr;
  p.B = B;
  p.T = T;
  p.H = H;
  p.Hkv = Hkv;
  p.G = G;
  p.d = d;
  p.page = page_size;
  p.max_blocks = max_blocks;
  p.n_blocks = n_blocks;
  p.window = window > 0 ? window : 0;
  const float s = scale != 0.0f ? scale : 1.0f / sqrtf((float)d);
  p.scale = fabsf(s);
  p.softcap = softcap_size(softcap, p.scale);
  if (p.softcap != 0.0f) {  // pva_tree_tile.cuh; and the products' squares have to be finite
    const double cap = p.softcap, t = fmin(0.25, pow(ldexp(1.0, -14) * 315.0 / 17.0 / cap, 1.0 / 7.0));
    p.series_to = (float)fmin(t * cap / p.scale, 1e9);
    if (p.scale > 1e7 * cap) p.series_to = -1.0f;  // nor would its coefficients be
  }
  p.rot = rot;
  p.n_axes = rot ? n_axes : 1;
  p.cache_rows = cache_rows;
  // two query tiles an item where a sequence can have more rows than one holds
  p.q_parts = tc && rot ? 2 : 1;  // without a rotation the queries are exact as they are
  const bool pair = tc && tree_takes_pair((long long)T * G, d, p.q_parts);
  const int rows_f32 = T * G <= 8 ? 8 : T * G <= 16 ? 16 : 24;
  p.rows = pair ? 2 * kTcRows : tc ? kTcRows : rows_f32;
  p.item_places = 2;
  p.bn = tc ? tree_keys(d) : kTreeKeysF32;
  p.QT = (int)(((long long)T * G + p.rows - 1) / p.rows);
  p.W32 = parents ? (T + 31) / 32 : 0;
  // Two tiles at least: half the parts to join for one more tile's time (one
  // request, 8 nodes on 2000 rows: 26.0 against 23.9 us), but not where a tile
  // is the paired kernel's (60 nodes on 500 rows: 30.3 against 31.6 us).
  p.min_chunk = pair ? 1 : 2;
  p.may_take_items = tc && p.QT > 1;
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.out = out;

  std::lock_guard<std::mutex> lock(api_mutex());
  int sms = 0;
  if ((rc = sm_count(&sms)) != PVA_OK) return rc;
  p.pieces = tc ? sms : f32::ctas(p.rows, d) * sms;
  // workspace, in 256-byte steps
  size_t used = 0;
  auto take = [&](size_t bytes) {
    const size_t at = used;
    used += (bytes + 255) / 256 * 256;
    return at;
  };
  const size_t at_cuts = take(sizeof(TreeCut) * p.pieces);
  const size_t at_hdr = take(32), at_tiles = take(4 * ((size_t)B + 1)), at_items = take(4 * ((size_t)B + 1));
  const size_t at_q_start = take(4 * (size_t)B * (p.QT + 1));
  const size_t at_depth = take(parents ? 4 * (size_t)B * T : 0);
  const size_t at_mask = take(4 * (size_t)B * T * p.W32);
  const size_t at_q = take((size_t)p.q_parts * B * T * H * d * size);
  const size_t at_o = take(sizeof(float) * 2 * p.pieces * p.rows * (size_t)d);
  const size_t at_ml = take(sizeof(float2) * 2 * p.pieces * (size_t)p.rows);
  CallContext c;
  if ((rc = acquire(stream, used, &c)) != PVA_OK) return rc;
  p.status = c.status;
  p.cuts = reinterpret_cast<TreeCut*>(c.buf + at_cuts);
  p.hold_ns = selftest_hold_ns();
  p.hdr = reinterpret_cast<int32_t*>(c.buf + at_hdr);
  p.tile_start = reinterpret_cast<int32_t*>(c.buf + at_tiles);
  p.item_start = reinterpret_cast<int32_t*>(c.buf + at_items);
  p.q_start = reinterpret_cast<int32_t*>(c.buf + at_q_start);
  p.depth = reinterpret_cast<int32_t*>(c.buf + at_depth);
  p.mask = reinterpret_cast<uint32_t*>(c.buf + at_mask);
  p.q = c.buf + at_q;
  p.part_o = reinterpret_cast<float*>(c.buf + at_o);
  p.part_ml = reinterpret_cast<float2*>(c.buf + at_ml);

  CUtensorMap tq, tk, tv;
  if (tc) {
    // boxes of one page's rows (a page shorter than a key tile), or of a tile
    const int box = block_table && page_size < p.bn ? page_size : p.bn;
    const long long planes = (long long)n_blocks * Hkv;
    if ((rc = get_encoder()) != PVA_OK ||
        (rc = encode_plane_map(&tq, p.q, dtype, d, T * G, (long long)p.q_parts * B * Hkv, 64, kTcRows,
                               true)) !=
            PVA_OK ||
        (rc = encode_plane_map(&tk, k_cache, dtype, d, page_size, planes, 64, box, true)) != PVA_OK ||
        (rc = encode_plane_map(&tv, v_cache, dtype, d, page_size, planes, 64, box, true)) != PVA_OK)
      return rc;
  }

  r.q = q;
  r.k = k_new;
  r.v = v_new;
  r.q_out = p.q;
  r.q_rest = p.q_parts == 2 ? c.buf + at_q + (size_t)B * T * H * d * size : nullptr;
  r.k_cache = k_cache;
  r.v_cache = v_cache;
  r.q_stride = (long long)H * d;
  r.k_stride = r.v_stride = (long long)Hkv * d;
  r.tokens = B * T;
  r.H = H;
  r.Hkv = Hkv;
  r.d = d;
  r.pos = p.pos;
  r.page = page_size;
  r.n_slots = (long long)n_blocks * page_size;
  r.hdr = p.hdr;
  r.past = past_lens;
  r.lens = tree_lens;
  r.depth = parents ? p.depth : nullptr;
  r.parents = parents;
  r.table = block_table;
  r.T = T;
  r.max_blocks = max_blocks;
  r.negate_q = s < 0.0f;
  r.group_inv = G > 1 && (long long)H * G < (1ll << 32) ? (uint32_t)(((1ull << 32) + G - 1) / G) : 0;
  r.out = out;
  r.status = c.status;

  cudaError_t e = launch_front(p, r, dtype, c.num_sms, stream);
  if (e != cudaSuccess) return cuda_fail(e, "tree front-end launch");
  e = pair ? launch_tree_pair(p, dtype, tq, tk, tv, stream)
      : tc ? launch_tree_tc(p, dtype, tq, tk, tv, stream)
           : launch_tree_f32(p, stream);
  if (e != cudaSuccess) return cuda_fail(e, "tree attention launch");
  e = launch_join(p, dtype, stream);
  return e == cudaSuccess ? PVA_OK : cuda_fail(e, "tree join launch");
}

}  // namespace

extern "C" int pva_gqa_tree(const void* q, const void* k_new, const void* v_new, void* k_cache,
                            void* v_cache, const int32_t* past_lens, const int32_t* tree_lens,
                            const int32_t* parents, const int32_t* block_table,
                            const void* cos_cache, const void* sin_cache,
                            const int64_t* position_ids, void* out, int B, int tokens,
                            int n_blocks, int page_size, int max_blocks, int num_heads,
                            int kv_num_heads, int head_size, int rotary_dim, int cache_rows,
                            int rotary_interleaved, int n_axes, const int32_t* sections,
                            int axes_interleaved, int rotary_dtype, float scale, float softcap,
                            int local_window, int dtype, void* stream) {
  return guarded([&]() -> int {
    return gqa_tree(q, k_new, v_new, k_cache, v_cache, past_lens, tree_lens, parents, block_table,
                    cos_cache, sin_cache, position_ids, out, B, tokens, n_blocks, page_size,
                    max_blocks, num_heads, kv_num_heads, head_size, rotary_dim, cache_rows,
                    rotary_interleaved, n_axes, sections, axes_interleaved, rotary_dtype, scale,
                    softcap, local_window, dtype, static_cast<cudaStream_t>(stream));
  });
}
