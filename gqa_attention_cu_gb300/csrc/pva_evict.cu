// Eviction of cache rows by their weight (pva_kvcache_evict): of each (layer,
// sequence, kv head) the first and last rows and the heaviest others stay, in their
// order, and close up.
//
//   pva_evict_select_kernel  one CTA per (layer, sequence, kv head): the weight of
//       the last row that stays is found by its bits, from the top (up to three counts,
//       of 11, 11 and 10 bits), then one pass in the rows' order lists those that stay and
//       writes their weights.
//   pva_evict_move_kernel    copies the listed rows to other blocks, or
//   pva_evict_close_kernel   closes them up in place: a CTA owns some columns of all
//       rows of one (layer, sequence, kv head, K or V), so rows are moved in order
//       with no other CTA to wait for.
//
// Weights are compared by a 32-bit key that rises with them; equal keys are taken
// from the lowest row on, so the choice does not depend on timing.
//
// 16 prompts of 4000 to 16,000 rows cut to 2048, 8 kv heads of 128 bf16, copied: 66 to 70
// us (floor 42).  The move is 44 of them, 268 MB at 6.1 TB/s; the choice 20, bound by the
// latency of votes and counts with one CTA an SM; of 16,000 rows, in cycles: lengths and
// table 8000, first count 10,000, second 6000, list 10,000.  In place: 87 us.  One prompt
// of 100,000 rows cut to 33,333: copied 138 us (floor 41), in place 353, where 16 CTAs a kv
// head walk its rows, a barrier every 256 of them.  One request of 700 rows: 13 us, of
// which 8 are launches.  (Clusters of four CTAs an item, counts through distributed shared
// memory: 60 us for the choice.  Four copies of the first count's bins: no less.  Each CTA
// copying its own rows: 67 against 69 us for 128 items, but 113 against 91 for 160.  Four
// rows in flight a thread and half as many CTAs in the move: 51 us.)
#include <limits.h>

#include "pva_device.cuh"

using namespace pva;
using namespace pva::host;

namespace pva {
namespace {

// A pool of blocks [layers][blocks][kv heads][page][row], and a table of it.
struct Pool {
  uint8_t* k;
  uint8_t* v;
  const int32_t* table;  // [B, max_blocks], or nullptr: block b
  long long layer_bytes;
  int blocks, page, max_blocks;
};

struct EvictParams {
  Pool from, to;
  int in_place;
  const float* weights;  // [layers][B][Hkv][width]
  float* weights_out;    // nullptr: not written
  int32_t* rows;         // [items][width] the rows that stay (the caller's `kept`, or workspace)
  const int32_t* lens;
  const int32_t* keep;
  int32_t* new_lens;
  int32_t* count;        // [items] rows that stay; workspace
  int32_t* length;       // [items] rows there were; -1: the sequence is left as it is
  int B, layers, Hkv, width, first, last, row_bytes;
  int held;              // weights that the first kernel's shared memory has room for
  uint32_t* status;
};

constexpr int kSelectThreads = 1024;  // at most; fewer for short rows of weights
constexpr int kSelectWarps = kSelectThreads / 32;
constexpr int kPerThread = 8;
constexpr int kBins = 2048;  // half of them in the last count
static_assert(kBins / 2 % kSelectThreads == 0, "whole bins a thread");
constexpr int kHeld = 48 * 1024;  // weights that lie in shared memory after the first count

// Rises with the weight; NaN is below every number, and -0 is 0.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0u;
  const uint32_t b = w == 0.0f ? 0u : __float_as_uint(w);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

constexpr uint32_t kLowestKey = 0x00800000u;  // of the finite weights

// What is wrong with sequence b (PVA_DEV_* bits); the whole CTA calls.
__device__ __forceinline__ uint32_t check_sequence(const EvictParams& p, int b, int n, int keep) {
  const int stay = min(n, keep);
  if (n < 0 || keep < 0 || n > p.width || (long long)n > (long long)p.from.max_blocks * p.from.page ||
      (long long)stay > (long long)p.to.max_blocks * p.to.page)
    return PVA_DEV_KV_LEN;
  bool off = false;
  for (int side = 0; side < (p.in_place ? 1 : 2); ++side) {
    const Pool& pool = side ? p.to : p.from;
    const int rows = side ? stay : n;
    if (!pool.table || rows == 0) continue;
    const int blocks = (rows - 1) / pool.page + 1;
    for (int i = threadIdx.x; i < blocks; i += blockDim.x)
      off |= (unsigned)pool.table[(size_t)b * pool.max_blocks + i] >= (unsigned)pool.blocks;
  }
  return __syncthreads_or(off) ? PVA_DEV_BLOCKS : 0u;
}

// Sum of the counts of the warps before this one, and of all: every warp adds up by itself.
__device__ __forceinline__ int warps_before(const int* counts, int warps, int& all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int mine = lane < warps ? counts[lane] : 0;
  int upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += y;
  }
  all = __shfl_sync(0xffffffffu, upto, 31);
  return __shfl_sync(0xffffffffu, upto - mine, warp);
}

__global__ void __launch_bounds__(kSelectThreads) pva_evict_select_kernel(EvictParams p) {
  allow_next_grid();
  wait_prior_grid();
  extern __shared__ float s_held[];
  __shared__ int s_bins[kBins];
  __shared__ int s_warp[kSelectWarps];
  __shared__ int s_bin, s_above, s_upto;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, threads = blockDim.x, warps = threads / 32;
  const int item = blockIdx.x, b = item / p.Hkv % p.B;
  const int n = p.lens[b], keep = p.keep[b];
  const bool latched = (*(volatile uint32_t*)p.status & PVA_DEV_KV_CACHE) != 0;
  const float* w = p.weights + (size_t)item * p.width;
  // The next tile's weights are on their way while the table is checked, or a tile counted.
  const int there = min(n, p.width);
  float next[kPerThread];
  auto fetch = [&](int j0) {
#pragma unroll
    for (int k = 0; k < kPerThread; ++k) {
      const int j = j0 + k * threads + tid;
      next[k] = j < there ? w[j] : 0.0f;
    }
  };
  fetch(0);
  const uint32_t bad = latched ? 0u : check_sequence(p, b, n, keep);
  if (latched || bad) {
    if (tid == 0) {
      p.length[item] = -1;
      p.count[item] = p.in_place ? n : 0;
      if (bad) atomicOr(p.status, bad);
    }
    return;
  }
  const int stay = min(n, keep);
  // rows [0, head) and [n - tail, n) stay in any case
  const int head = stay == n ? n : min(p.first, stay), tail = stay == n ? 0 : min(stay - head, p.last);
  if (tid == 0) {
    p.length[item] = n;
    p.count[item] = stay;
  }
  const int lo = head, hi = n - tail;
  const int want = stay - head - tail;  // of the rows [lo, hi)
  // The key of the lightest row that stays, bit by bit from the top: `above` of the
  // rows are heavier than all that share the bits found so far.  The first count is
  // made while the weights come in, the others go over shared memory, four a thread.
  uint32_t prefix = 0;
  int above = 0, upto_bin = 0;  // rows of the bits found and above
  const int held = min(n, p.held);
  auto bin_of = [&](uint32_t key, int shift, int bins) { return (key >> shift) & (bins - 1); };
  for (int i = tid; i < kBins; i += threads) s_bins[i] = 0;
  __syncthreads();
  for (int j0 = 0; j0 < n; j0 += threads * kPerThread) {
    float x[kPerThread];
#pragma unroll
    for (int k = 0; k < kPerThread; ++k) x[k] = next[k];
    if (j0 + threads * kPerThread < n) fetch(j0 + threads * kPerThread);
#pragma unroll
    for (int k = 0; k < kPerThread; ++k) {
      const int j = j0 + k * threads + tid;
      if (j < held) s_held[j] = x[k];
      // zeros are often many: one lane adds a warp's
      const bool counts = j >= lo && j < hi;
      const uint32_t zeros = __ballot_sync(0xffffffffu, counts && x[k] == 0.0f);
      if (counts && x[k] != 0.0f) atomicAdd(&s_bins[bin_of(weight_key(x[k]), 21, kBins)], 1);
      if (lane == 0 && zeros) atomicAdd(&s_bins[bin_of(weight_key(0.0f), 21, kBins)], __popc(zeros));
    }
  }
  __syncthreads();  // the list below reads other threads' weights, also without a further count
  auto weight = [&](int j) { return j < held ? s_held[j] : w[j]; };
  if (want > 0) {
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
      const int top = pass == 0 ? 32 : pass == 1 ? 21 : 10;  // bits above are found
      const int bins = 1 << (top - shift);
      if (pass > 0) {
        for (int i = tid; i < bins; i += threads) s_bins[i] = 0;
        __syncthreads();
        auto count = [&](float x, int j) {
          const uint32_t key = weight_key(x);
          if (key >> top == prefix >> top && j >= lo && j < hi) atomicAdd(&s_bins[bin_of(key, shift, bins)], 1);
        };
#pragma unroll 2
        for (int i = tid; 4 * i < held; i += threads) {
          const float4 x = reinterpret_cast<const float4*>(s_held)[i];
          count(x.x, 4 * i);
          if (4 * i + 1 < held) count(x.y, 4 * i + 1);
          if (4 * i + 2 < held) count(x.z, 4 * i + 2);
          if (4 * i + 3 < held) count(x.w, 4 * i + 3);
        }
        for (int j = held + tid; j < n; j += threads) count(w[j], j);
        __syncthreads();
      }
      // the bin where the count from the top passes `want`: thread t has bins
      // [per t, per (t + 1)) from the top
      const int per = bins / threads;
      int mine = 0;
      for (int i = 0; i < per; ++i) mine += s_bins[bins - 1 - (tid * per + i)];
      int upto = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += y;
      }
      if (lane == 31) s_warp[warp] = upto;
      __syncthreads();
      int all;
      int before = above + upto - mine + warps_before(s_warp, warps, all);
      if (before < want && before + mine >= want) {
        int i = 0;
        for (; before + s_bins[bins - 1 - (tid * per + i)] < want; ++i)
          before += s_bins[bins - 1 - (tid * per + i)];
        s_bin = bins - 1 - (tid * per + i);
        s_above = before;
        s_upto = before + s_bins[s_bin];
      }
      __syncthreads();
      prefix |= (uint32_t)s_bin << shift;
      above = s_above;
      upto_bin = s_upto;
      // All of the bin stay: its lower end will do as the limit (not below -inf, where
      // that is no number).  Mostly after the second count.
      if (upto_bin == want && prefix >= kLowestKey) break;
    }
  }
  // As weights: heavier than `limit`, or as heavy (a limit that is NaN is below all
  // numbers; without a limit nothing is either).
  const bool none = want == 0, nan_limit = prefix == 0;
  const float limit = __uint_as_float(prefix & 0x80000000u ? prefix & 0x7fffffffu : ~prefix);
  const bool ties = upto_bin != want;  // of the rows with this key the first ones alone
  const int equal = want - above;
  // In the rows' order: rows that stay because they are heavier (or first, or last),
  // and those with the key, counted side by side in 16 bits each within a tile.
  int32_t* rows = p.rows ? p.rows + (size_t)item * p.width : nullptr;
  float* out = p.weights_out ? p.weights_out + (size_t)item * p.width : nullptr;
  int done_over = 0, done_equal = 0;
#pragma unroll 1
  for (int t0 = 0; t0 < n; t0 += threads * kPerThread) {
    float x[kPerThread];
    uint32_t over[kPerThread], same[kPerThread];  // of the warp: bit i is row j0 + 32 k + i - lane
    int in_warp = 0;
    const int j0 = t0 + warp * (32 * kPerThread) + lane;
    const bool any = j0 - lane < n;
    if (any) {
#pragma unroll
      for (int k = 0; k < kPerThread; ++k) {
        const int j = j0 + 32 * k;
        x[k] = j < n ? weight(j) : 0.0f;
        const bool open = j >= lo && j < hi;
        if (ties) {
          const bool heavier = nan_limit ? x[k] == x[k] : x[k] > limit;
          const bool alike = nan_limit ? x[k] != x[k] : x[k] == limit;
          over[k] = __ballot_sync(0xffffffffu, j < n && (!open || heavier));
          same[k] = __ballot_sync(0xffffffffu, open && alike);
          in_warp += __popc(over[k]) | __popc(same[k]) << 16;
        } else {
          over[k] = __ballot_sync(0xffffffffu, j < n && (!open || (!none && x[k] >= limit)));
          in_warp += __popc(over[k]);
        }
      }
    }
    if (lane == 0) s_warp[warp] = in_warp;
    __syncthreads();  // all of the tile's weights have been read
    int all;
    const int before = warps_before(s_warp, warps, all);
    if (any) {
      int n_over = done_over + (before & 0xffff), n_equal = done_equal + (before >> 16);
      const uint32_t below = (1u << lane) - 1u;
#pragma unroll
      for (int k = 0; k < kPerThread; ++k) {
        int to = n_over + __popc(over[k] & below);
        bool stays = over[k] >> lane & 1u;
        if (ties) {
          const int my_equal = n_equal + __popc(same[k] & below);
          stays |= (same[k] >> lane & 1u) && my_equal < equal;
          to += min(my_equal, equal);
          n_equal += __popc(same[k]);
        }
        if (stays) {
          if (rows) rows[to] = j0 + 32 * k;
          if (out) out[to] = x[k];  // to <= the row itself: behind all that is still read
        }
        n_over += __popc(over[k]);
      }
    }
    done_over += all & 0xffff;
    done_equal += all >> 16;
    __syncthreads();  // before the next tile's counts
  }
  if (out)
    for (int j = stay + tid; j < n; j += threads) out[j] = 0.0f;
}

// Where row `row` of a sequence's kv head lies, from the start of its layer.
__device__ __forceinline__ long long row_at(const EvictParams& p, const Pool& pool, int b, int h,
                                            int row) {
  const int in = row / pool.page;
  const int block = pool.table ? pool.table[(size_t)b * pool.max_blocks + in] : b;
  return (((long long)block * p.Hkv + h) * pool.page + (row - in * pool.page)) * p.row_bytes;
}

constexpr int kMoveThreads = 256;
constexpr int kMoveAhead = 2;  // rows a thread has in flight

// lanes: threads side by side on a row (a power of two)
template <typename U>
__global__ void __launch_bounds__(kMoveThreads) pva_evict_move_kernel(EvictParams p, int lanes) {
  allow_next_grid();
  wait_prior_grid();
  const int item = blockIdx.y, b = item / p.Hkv % p.B, h = item % p.Hkv;
  const long long layer = item / p.Hkv / p.B;
  const int stay = p.count[item];
  if (blockIdx.x == 0 && threadIdx.x == 0 && h == 0 && layer == 0) p.new_lens[b] = stay;
  if (p.length[item] < 0) return;
  const unsigned n = stay;
  const int32_t* rows = p.rows + (size_t)item * p.width;
  const int units = p.row_bytes / (int)sizeof(U), u0 = threadIdx.x % lanes;
  const int per = kMoveThreads / lanes;  // rows of a CTA at once
  const long long from = layer * p.from.layer_bytes, to = layer * p.to.layer_bytes;
  // (a step of all CTAs may lead past 2^31)
  for (unsigned i0 = blockIdx.x * per * kMoveAhead + threadIdx.x / lanes; i0 < n;
       i0 += gridDim.x * per * kMoveAhead) {
    long long src[kMoveAhead], dst[kMoveAhead];
#pragma unroll
    for (int a = 0; a < kMoveAhead; ++a) {
      const unsigned i = i0 + a * per;
      if (i >= n) continue;
      src[a] = from + row_at(p, p.from, b, h, rows[i]);
      dst[a] = to + row_at(p, p.to, b, h, (int)i);
    }
    for (int u = u0; u < units; u += lanes) {
      U x[kMoveAhead], y[kMoveAhead];
#pragma unroll
      for (int a = 0; a < kMoveAhead; ++a) {
        if (i0 + a * per >= n) continue;
        x[a] = *reinterpret_cast<const U*>(p.from.k + src[a] + (long long)u * sizeof(U));
        y[a] = *reinterpret_cast<const U*>(p.from.v + src[a] + (long long)u * sizeof(U));
      }
#pragma unroll
      for (int a = 0; a < kMoveAhead; ++a) {
        if (i0 + a * per >= n) continue;
        *reinterpret_cast<U*>(p.to.k + dst[a] + (long long)u * sizeof(U)) = x[a];
        *reinterpret_cast<U*>(p.to.v + dst[a] + (long long)u * sizeof(U)) = y[a];
      }
    }
  }
}

// In place.  The i-th row that stays is row src(i) >= i, and src rises, so what
// chunk c of the rows is written over is read by no later chunk: it is enough that
// a chunk is read before it is written.  CTA (slice, item, K or V) has the units
// [slice * lanes, (slice + 1) * lanes) of every row.
template <typename U>
__global__ void __launch_bounds__(kMoveThreads) pva_evict_close_kernel(EvictParams p, int lanes) {
  allow_next_grid();
  wait_prior_grid();
  const int item = blockIdx.y, b = item / p.Hkv % p.B, h = item % p.Hkv;
  const long long layer = item / p.Hkv / p.B;
  const int n = p.count[item];
  if (blockIdx.x == 0 && blockIdx.z == 0 && threadIdx.x == 0 && h == 0 && layer == 0) p.new_lens[b] = n;
  if (p.length[item] < 0 || p.length[item] == n) return;
  const int32_t* rows = p.rows + (size_t)item * p.width;
  const int units = p.row_bytes / (int)sizeof(U), u = blockIdx.x * lanes + threadIdx.x % lanes;
  const int per = kMoveThreads / lanes;
  uint8_t* base = (blockIdx.z ? p.from.v : p.from.k) + layer * p.from.layer_bytes + (long long)u * sizeof(U);
  const bool in = u < units;
  for (int c = 0; c < n; c += per * kMoveAhead) {
    U x[kMoveAhead];
    int from[kMoveAhead];
#pragma unroll
    for (int a = 0; a < kMoveAhead; ++a) {
      const int i = c + a * per + threadIdx.x / lanes;
      from[a] = i < n ? rows[i] : i;
      if (in && from[a] != i) x[a] = *reinterpret_cast<const U*>(base + row_at(p, p.from, b, h, from[a]));
    }
    __syncthreads();
#pragma unroll
    for (int a = 0; a < kMoveAhead; ++a) {
      const int i = c + a * per + threadIdx.x / lanes;
      if (in && from[a] != i) *reinterpret_cast<U*>(base + row_at(p, p.from, b, h, i)) = x[a];
    }
  }
}

template <typename U>
cudaError_t launch_move(const EvictParams& p, int items, int num_sms, cudaStream_t s) {
  const int units = p.row_bytes / (int)sizeof(U);
  if (p.in_place) {
    const int lanes = 32 / (int)sizeof(U);  // 32 bytes of a row: whole sectors
    return launch_dependent(pva_evict_close_kernel<U>, dim3((units + lanes - 1) / lanes, items, 2),
                            dim3(kMoveThreads), 0, s, p, lanes);
  }
  int lanes = 1;
  while (lanes < units && lanes < 32) lanes *= 2;
  const int chunk = kMoveThreads / lanes * kMoveAhead;
  const int want = (p.width + chunk - 1) / chunk;
  const int most = (16 * num_sms + items - 1) / items;
  return launch_dependent(pva_evict_move_kernel<U>, dim3(want < most ? want : most, items),
                          dim3(kMoveThreads), 0, s, p, lanes);
}

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return a && b && x < y + nb && y < x + na;
}

}  // namespace
}  // namespace pva

extern "C" int pva_kvcache_evict(void* k_cache, void* v_cache, const float* weights,
                                 const int32_t* lens, const int32_t* keep, int32_t* new_lens,
                                 const int32_t* block_table, void* k_out, void* v_out,
                                 const int32_t* out_table, float* weights_out, int32_t* kept, int B,
                                 int layers, int64_t layer_stride, int n_blocks, int page_size,
                                 int max_blocks, int64_t out_layer_stride, int out_blocks,
                                 int out_page_size, int out_max_blocks, int kv_num_heads,
                                 int head_size, int width, int first, int last, int dtype,
                                 void* stream_) {
  return guarded([&]() -> int {
    if (!k_cache || !v_cache || !weights || !lens || !keep || !new_lens)
      return fail(PVA_ERR_INVALID_ARG, "null cache, weights, lens, keep or new_lens pointer");
    if ((k_out != nullptr) != (v_out != nullptr))
      return fail(PVA_ERR_INVALID_ARG, "k_out and v_out come together");
    if (B < 1 || layers < 1 || n_blocks < 1 || kv_num_heads < 1 || page_size < 1 || head_size < 1 || width < 1)
      return fail(PVA_ERR_INVALID_ARG, "counts and sizes must be positive");
    if (first < 0 || last < 0) return fail(PVA_ERR_INVALID_ARG, "first and last must not be negative");
    if (dtype != PVA_F32 && dtype != PVA_F16 && dtype != PVA_BF16)
      return fail(PVA_ERR_INVALID_ARG, "dtype must be 0 (f32), 1 (f16) or 2 (bf16)");
    if (block_table ? max_blocks < 1 : n_blocks != B)
      return fail(PVA_ERR_INVALID_ARG, block_table ? "max_blocks must be >= 1"
                                                   : "without a block table the cache has one block a sequence");
    const bool in_place = !k_out && !out_table;
    if (!k_out && out_table) {  // other blocks of the same pool
      k_out = k_cache;
      v_out = v_cache;
      out_layer_stride = layer_stride;
      out_blocks = n_blocks;
      out_page_size = page_size;
    }
    if (!in_place && (out_blocks < 1 || out_page_size < 1))
      return fail(PVA_ERR_INVALID_ARG, "counts and sizes must be positive");
    if (!in_place && (out_table ? out_max_blocks < 1 : out_blocks != B))
      return fail(PVA_ERR_INVALID_ARG, out_table ? "out_max_blocks must be >= 1"
                                                 : "without a block table the cache has one block a sequence");
    if (!block_table) max_blocks = 1;
    if (!out_table) out_max_blocks = 1;
    const long long items = (long long)layers * B * kv_num_heads;
    if (items > 65535) return fail(PVA_ERR_UNSUPPORTED, "at most 65535 layers x sequences x kv heads");
    auto fits = [&](long long blocks, long long page, long long table) {
      return table * page <= INT_MAX && blocks * kv_num_heads <= INT_MAX;
    };
    if ((long long)head_size * 4 > INT_MAX || !fits(n_blocks, page_size, max_blocks) ||
        (!in_place && !fits(out_blocks, out_page_size, out_max_blocks)) || width > INT_MAX - 65536)
      return fail(PVA_ERR_INVALID_ARG, "cache extents do not fit in int32");
    const long long size = dtype == PVA_F32 ? 4 : 2;
    const long long one = (long long)n_blocks * kv_num_heads * page_size * head_size;
    const long long out_one = (long long)out_blocks * kv_num_heads * out_page_size * head_size;
    if (layers > 1 && (layer_stride < one || (!in_place && out_layer_stride < out_one)))
      return fail(PVA_ERR_INVALID_ARG, "layer_stride is smaller than a layer's cache");
    EvictParams p{};
    p.in_place = in_place;
    p.from = {static_cast<uint8_t*>(k_cache), static_cast<uint8_t*>(v_cache), block_table,
              layers > 1 ? layer_stride * size : 0, n_blocks, page_size, max_blocks};
    p.to = in_place ? p.from
                    : Pool{static_cast<uint8_t*>(k_out), static_cast<uint8_t*>(v_out), out_table,
                           layers > 1 ? out_layer_stride * size : 0, out_blocks, out_page_size, out_max_blocks};
    p.row_bytes = (int)(head_size * size);
    const uintptr_t mis = (uintptr_t)k_cache | (uintptr_t)v_cache | (uintptr_t)p.from.layer_bytes |
                          (uintptr_t)p.to.k | (uintptr_t)p.to.v | (uintptr_t)p.to.layer_bytes |
                          (uintptr_t)p.row_bytes;
    if (mis % size || ((uintptr_t)weights | (uintptr_t)weights_out) % 4)
      return fail(PVA_ERR_INVALID_ARG, "a cache or the weights are not aligned to their elements");
    const size_t all = (size_t)items * width * 4, tables = 4 * (size_t)B * max_blocks,
                 out_tables = 4 * (size_t)B * out_max_blocks;
    struct Span { const void* p; size_t n; };
    const Span written[] = {{new_lens, 4 * (size_t)B}, {weights_out, all}, {kept, all}};
    const Span read[] = {{block_table, tables}, {out_table, out_tables}, {weights, all}};
    for (int i = 0; i < 3; ++i) {
      for (const Span& r : read) {
        if (i == 1 && weights_out == weights && r.p == weights) continue;
        if (overlap(written[i].p, written[i].n, r.p, r.n))
          return fail(PVA_ERR_INVALID_ARG, "an output overlaps an input (weights_out may be weights)");
      }
      for (int j = 0; j < i; ++j)
        if (overlap(written[i].p, written[i].n, written[j].p, written[j].n))
          return fail(PVA_ERR_INVALID_ARG, "new_lens, weights_out and kept overlap");
      if (i > 0 && (overlap(written[i].p, written[i].n, lens, 4 * (size_t)B) ||
                    overlap(written[i].p, written[i].n, keep, 4 * (size_t)B)))
        return fail(PVA_ERR_INVALID_ARG, "weights_out or kept overlaps lens or keep");
    }
    // the caches, layer by layer (what lies between their layers may be anything)
    const Span beside[] = {{new_lens, 4 * (size_t)B}, {weights_out, all}, {kept, all}, {weights, all}, {lens, 4 * (size_t)B},
                           {keep, 4 * (size_t)B}, {block_table, tables}, {out_table, out_tables}};
    for (const Pool& pool : {p.from, p.to}) {
      const size_t layer = (size_t)pool.blocks * kv_num_heads * pool.page * p.row_bytes;
      for (const uint8_t* cache : {pool.k, pool.v})
        for (const Span& s : beside) {
          if (!overlap(cache, (layers - 1) * (size_t)pool.layer_bytes + layer, s.p, s.n)) continue;
          for (int l = 0; l < layers; ++l)
            if (overlap(cache + l * pool.layer_bytes, layer, s.p, s.n))
              return fail(PVA_ERR_INVALID_ARG, "a cache overlaps the weights, lengths or tables");
        }
    }
    p.weights = weights;
    p.weights_out = weights_out;
    p.lens = lens;
    p.keep = keep;
    p.new_lens = new_lens;
    p.B = B;
    p.layers = layers;
    p.Hkv = kv_num_heads;
    p.width = width;
    p.first = first;
    p.last = last;
    const cudaStream_t stream = static_cast<cudaStream_t>(stream_);
    std::lock_guard<std::mutex> lock(api_mutex());
    const size_t head = ((size_t)items * 8 + 255) / 256 * 256;
    CallContext c;
    const int rc = acquire(stream, head + (kept ? 0 : all), &c);
    if (rc != PVA_OK) return rc;
    p.status = c.status;
    p.count = reinterpret_cast<int32_t*>(c.buf);
    p.length = p.count + items;
    p.rows = kept ? kept : reinterpret_cast<int32_t*>(c.buf + head);
    const long long rows = (long long)max_blocks * page_size < width ? (long long)max_blocks * page_size : width;
    p.held = (int)(rows < kHeld ? rows : kHeld);
    const size_t smem = sizeof(float) * (((size_t)p.held + 3) / 4 * 4);
    // 64 registers a thread: an SM holds one CTA of 1024 threads, two of 512, four of 256
    // (us, 1024, 512 and 256: 160 items of 12,000 rows 91, 84, 98; 512 of 9000 151, 134,
    // 131; 160 of 30,000 141, 151, 187; 2048 of 2000 287, 231, 211).
    // The rows are those that the tables and weights have room for, lengths being the
    // device's: with room for 131,072 rows 2048 items of 2000 take 308 us instead of 210, 128
    // of up to 16,000 77 instead of 70.
    const bool more = items > c.num_sms;  // up to that 1024 (128 items of up to 16,000: 70 of 71.5)
    const int threads = rows <= 2048 ? 256 : rows <= 8192 || (more && rows <= 16384) ? 512 : kSelectThreads;
    cudaError_t e = cudaFuncSetAttribute(pva_evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)(sizeof(float) * kHeld));
    if (e == cudaSuccess)
      e = launch_dependent(pva_evict_select_kernel, dim3((unsigned)items), dim3(threads), smem, stream, p);
    if (e != cudaSuccess) return cuda_fail(e, "eviction launch");
    e = mis % 16 == 0  ? launch_move<uint4>(p, (int)items, c.num_sms, stream)
        : mis % 4 == 0 ? launch_move<uint32_t>(p, (int)items, c.num_sms, stream)
                       : launch_move<uint16_t>(p, (int)items, c.num_sms, stream);
    return e == cudaSuccess ? PVA_OK : cuda_fail(e, "row move launch");
  });
}
