// Block tables and slot maps of a paged KV cache (pva_block_tables), and the
// move of an accepted path's rows (pva_kvcache_accept).
//
// pva_block_tables is all latency: a few words per sequence and eight bytes per
// new token.  One CTA does the allocation (the stack is shared by all
// sequences): a thread per sequence adds up what is given back and taken, then a
// warp per sequence moves its blocks, four sequences at a time; runs of more
// than 64 blocks are moved by all threads together.  700 sequences that take or
// give back 15,700 blocks: 10.3 us; a thread per block that finds its
// sequence by bisection 15.7 us, bound by the one SM's instructions; a thread
// per sequence 21 and 13 us, bound by its scattered words.  16 sequences with 8 new
// tokens each: 3 us, a launch and four dependent reads.  Slots are written by the
// same CTA while they are few, and by a grid of their own where they are many
// (250,000: 6 us after the allocation).
//
// pva_kvcache_accept moves rows in place.  A path rises, path[i] >= i, so row i
// is read (as some path[j], j <= i) before or when it is written if each thread
// keeps to one 16-byte column and goes through i in order: no copy is needed.
// A sequence's path and blocks are looked up once per CTA, which then moves the
// columns of many heads and layers with eight rows in flight per thread.  64
// sequences x 32 layers x 8 heads of 128 bf16, paths of up to 8 nodes (75 MB read
// and written): 11 us where they are in L2, 6.8 TB/s; 15 us where they are not.
#include <limits.h>

#include "pva_device.cuh"
#include "pva_path.h"

using namespace pva;
using namespace pva::host;

namespace pva {
namespace {

constexpr int kBlockThreads = 1024;
constexpr int kWordRefused = 18;  // status block: 1 where the last allocation was refused
// New tokens up to which the allocating CTA writes the slot map itself.
constexpr long long kSlotsInOne = 4096;
constexpr int kAhead = 8;          // loads a thread has under way
constexpr int kRunOfOne = 64;      // blocks of a sequence that one warp moves
constexpr int kRuns = 4;           // sequences that a warp has under way
constexpr int kOffsetsMax = 4096;  // sequences whose offsets a slot CTA keeps in shared memory

struct BlockParams {
  const int32_t* lens;
  int32_t* table;
  int32_t* held;
  int32_t* free_blocks;
  int32_t* free_count;
  const int32_t* cu_new;
  int64_t* slots;
  int B, max_blocks, page, pool;
  long long n_slots;
  int in_one;  // slots are written by the allocating CTA
  uint32_t* status;
};

__device__ __forceinline__ int blocks_for(int rows, int page) {
  return (int)(((long long)rows + page - 1) / page);
}

// The last index of start[0 .. n) that is <= x (entries ascend, start[0] <= x).
template <typename I>
__device__ __forceinline__ int last_at(const I* start, int n, I x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (start[mid] <= x) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// Sums over the CTA of two values, and over the threads before this one.
__device__ __forceinline__ void block_scan(long long& x, long long& y, long long* sums,
                                           long long& all_x, long long& all_y) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  long long ux = x, uy = y;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long a = __shfl_up_sync(0xffffffffu, ux, o), b = __shfl_up_sync(0xffffffffu, uy, o);
    if (lane >= o) {
      ux += a;
      uy += b;
    }
  }
  if (lane == 31) {
    sums[warp] = ux;
    sums[32 + warp] = uy;
  }
  __syncthreads();
  // every warp sums the warps' sums, a lane per warp
  long long sx = lane < warps ? sums[lane] : 0, sy = lane < warps ? sums[32 + lane] : 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long a = __shfl_up_sync(0xffffffffu, sx, o), b = __shfl_up_sync(0xffffffffu, sy, o);
    if (lane >= o) {
      sx += a;
      sy += b;
    }
  }
  all_x = __shfl_sync(0xffffffffu, sx, 31);
  all_y = __shfl_sync(0xffffffffu, sy, 31);
  const int w = warp > 0 ? warp - 1 : 0;
  const long long bx = __shfl_sync(0xffffffffu, sx, w), by = __shfl_sync(0xffffffffu, sy, w);
  x = ux - x + (warp > 0 ? bx : 0);
  y = uy - y + (warp > 0 ? by : 0);
  __syncthreads();
}

// Slot of token t of sequence b, whose new tokens end at `end`.
__device__ __forceinline__ int64_t slot_of(const BlockParams& p, int b, int t, int end) {
  const int row = p.lens[b] - (end - t), in = row / p.page;
  return (int64_t)p.table[(size_t)b * p.max_blocks + in] * p.page + (row - in * p.page);
}

// Blocks that one sequence gives back or takes: table entry i and stack place -i.
struct Run {
  int32_t* entries;
  int32_t* places;
  int n;
};
// Moves numbers i, i + step, ... (K of them) of a run of n; pass 0: back.
template <int K>
__device__ __forceinline__ void move_blocks(int32_t* entries, int32_t* places, int i, int step,
                                            int n, int pass) {
  int32_t id[K];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const long long x = i + (long long)k * step;
    if (x < n) id[k] = pass == 0 ? entries[x] : places[-x];
  }
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const long long x = i + (long long)k * step;
    if (x >= n) continue;
    if (pass == 0) {
      places[-x] = id[k];
      entries[x] = -1;
    } else {
      entries[x] = id[k];
    }
  }
}

__global__ void __launch_bounds__(kBlockThreads) pva_block_alloc_kernel(BlockParams p) {
  __shared__ long long s_sums[64];
  __shared__ int s_bad;
  __shared__ Run s_run[kBlockThreads];  // long runs of one round
  __shared__ int s_long;
  __shared__ int s_cu[kBlockThreads];   // offsets of the new tokens
  allow_next_grid();
  const int tid = threadIdx.x, threads = blockDim.x, lane = tid & 31;
  if (tid == 0) s_bad = 0;
  __syncthreads();
  wait_prior_grid();
  const int count = *p.free_count;
  const int rounds = (p.B + threads - 1) / threads;
  // Totals first: the step is refused as a whole.
  long long all_given = 0, all_taken = 0;
  long long given = 0, taken = 0;  // of this thread's sequence, in the last round
  int held = 0, need = 0;
  bool bad = count < 0 || count > p.pool;
  for (int r = 0; r < rounds; ++r) {
    const int b = r * threads + tid;
    given = taken = 0;
    held = need = 0;
    if (b < p.B) {
      const int len = p.lens[b];
      held = p.held[b];
      if (p.cu_new) {
        const int c0 = p.cu_new[b], c1 = p.cu_new[b + 1];
        bad = bad || (b == 0 && c0 != 0) || c1 < c0 || (long long)c1 - c0 > len ||
              (b == p.B - 1 && c1 > p.n_slots);
      }
      need = blocks_for(len, p.page);
      if (len < 0 || held < 0 || held > p.max_blocks || need > p.max_blocks) {
        bad = true;
        held = need = 0;
      }
      given = max(0, held - need);
      taken = max(0, need - held);
    }
    long long x = given, y = taken, all_x, all_y;
    if (bad) s_bad = 1;
    block_scan(x, y, s_sums, all_x, all_y);
    all_given += all_x;
    all_taken += all_y;
    given = x;
    taken = y;
  }
  const bool refuse = s_bad || count + all_given > p.pool || all_taken > count + all_given;
  if (tid == 0 && !p.in_one) p.status[kWordRefused] = refuse ? 1u : 0u;
  if (refuse) {
    if (tid == 0) atomicOr(p.status, PVA_DEV_BLOCKS);
    return;
  }
  const long long top = count + all_given - 1;
  for (int pass = 0; pass < 2; ++pass) {  // all is given back before any is taken
    if ((pass == 0 ? all_given : all_taken) == 0) continue;
    long long before = 0;
    for (int r = 0; r < rounds; ++r) {
      long long moved;
      if (rounds == 1) {
        moved = pass == 0 ? all_given : all_taken;
      } else {
        const int b = r * threads + tid;
        held = b < p.B ? p.held[b] : 0;
        need = b < p.B ? blocks_for(p.lens[b], p.page) : 0;
        given = max(0, held - need);
        taken = max(0, need - held);
        long long x, y;
        block_scan(given, taken, s_sums, x, y);
        moved = pass == 0 ? x : y;
      }
      // This thread's sequence.  Long runs are left to the whole CTA.
      const int count_b = pass == 0 ? max(0, held - need) : max(0, need - held);
      const long long at = pass == 0 ? given : taken;
      int32_t* entries = p.table + (size_t)(r * threads + tid) * p.max_blocks + min(held, need);
      int32_t* places = p.free_blocks + (top - before - at);
      if (tid == 0) s_long = 0;
      __syncthreads();
      if (count_b > kRunOfOne) {
        const int k = atomicAdd(&s_long, 1);
        s_run[k] = Run{entries, places, count_b};
      }
      // short runs: a warp per run, a lane per block, four runs under way
      unsigned todo = __ballot_sync(0xffffffffu, count_b > 0 && count_b <= kRunOfOne);
      while (todo) {
        int32_t *from[kRuns], *to[kRuns];
        int32_t id[kRuns][kRunOfOne / 32];
        int n[kRuns];
#pragma unroll
        for (int k = 0; k < kRuns; ++k) {
          const int src = todo ? __ffs(todo) - 1 : 0;
          n[k] = __shfl_sync(0xffffffffu, todo ? count_b : 0, src);
          todo &= todo - 1;
          from[k] = reinterpret_cast<int32_t*>(__shfl_sync(0xffffffffu, (unsigned long long)entries, src));
          to[k] = reinterpret_cast<int32_t*>(__shfl_sync(0xffffffffu, (unsigned long long)places, src));
#pragma unroll
          for (int x = 0; x < kRunOfOne / 32; ++x) {
            const int i = lane + 32 * x;
            if (i < n[k]) id[k][x] = pass == 0 ? from[k][i] : to[k][-i];
          }
        }
#pragma unroll
        for (int k = 0; k < kRuns; ++k)
#pragma unroll
          for (int x = 0; x < kRunOfOne / 32; ++x) {
            const int i = lane + 32 * x;
            if (i >= n[k]) continue;
            if (pass == 0) {
              to[k][-i] = id[k][x];
              from[k][i] = -1;
            } else {
              from[k][i] = id[k][x];
            }
          }
      }
      __syncthreads();
      for (int k = 0; k < s_long; ++k) {
        const Run run = s_run[k];
        for (int i = tid; i < run.n; i += kAhead * threads)
          move_blocks<kAhead>(run.entries, run.places, i, threads, run.n, pass);
      }
      __syncthreads();
      before += moved;
    }
  }
  if (rounds == 1) {
    if (tid < p.B) p.held[tid] = need;
  } else {
    for (int b = tid; b < p.B; b += threads) p.held[b] = blocks_for(p.lens[b], p.page);
  }
  if (tid == 0) *p.free_count = (int)(count + all_given - all_taken);
  if (!p.in_one || !p.cu_new) return;
  if (rounds == 1) {
    // offsets to shared memory; sequences behind the last start at the end
    const int end = p.cu_new[p.B];
    s_cu[tid] = tid < p.B ? p.cu_new[tid] : end + 1;
    __syncthreads();
    for (int t = tid; t < p.n_slots; t += threads) {
      const int b = last_at(s_cu, threads, t);
      p.slots[t] = t >= end ? -1 : slot_of(p, b, t, b + 1 < p.B ? s_cu[b + 1] : end);
    }
  } else {
    const int end = p.cu_new[p.B];
    for (int t = tid; t < p.n_slots; t += threads) {
      const int b = t < end ? last_at(p.cu_new, p.B, t) : 0;
      p.slots[t] = t >= end ? -1 : slot_of(p, b, t, p.cu_new[b + 1]);
    }
  }
}

// A thread per token; the sequence by bisection of the offsets, from shared
// memory where they fit.
__global__ void __launch_bounds__(256) pva_block_slots_kernel(BlockParams p) {
  __shared__ int s_cu[kOffsetsMax + 1];
  allow_next_grid();
  wait_prior_grid();
  if (p.status[kWordRefused]) return;
  const bool fits = p.B <= kOffsetsMax;
  if (fits) {
    for (int b = threadIdx.x; b <= p.B; b += blockDim.x) s_cu[b] = p.cu_new[b];
    __syncthreads();
  }
  const int* cu = fits ? s_cu : p.cu_new;
  const int end = cu[p.B];
  const long long step = (long long)gridDim.x * blockDim.x;
  for (long long t0 = (long long)blockIdx.x * blockDim.x + threadIdx.x; t0 < p.n_slots;
       t0 += kAhead * step) {
    int64_t slot[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const long long t = t0 + k * step;
      slot[k] = -1;
      if (t >= end) continue;
      const int b = last_at(cu, p.B, (int)t);
      slot[k] = slot_of(p, b, (int)t, cu[b + 1]);
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (t0 + k * step < p.n_slots) p.slots[t0 + k * step] = slot[k];
  }
}

struct AcceptParams {
  uint8_t* k;
  uint8_t* v;
  const int32_t* past;
  const int32_t* path;
  const int32_t* path_lens;
  const int32_t* table;
  int32_t* new_lens;
  int B, width, layers, n_blocks, Hkv, page, max_blocks;
  long long layer_bytes;
  int row_bytes;
  uint32_t* status;
};

constexpr int kAcceptThreads = 128, kPathRows = 128, kAcceptAhead = 8;

// CTA (c, b): a share of the columns (layer, K or V, kv head, unit U of a row) of
// sequence b.  The path is taken kPathRows nodes at a time; a column's thread is
// the same throughout, which is what makes the move in place safe.
template <typename U>
__global__ void __launch_bounds__(kAcceptThreads) pva_accept_kernel(AcceptParams p) {
  __shared__ long long s_from[kPathRows], s_to[kPathRows];  // rows of head 0; from -1: stays
  allow_next_grid();
  wait_prior_grid();
  const int b = blockIdx.y, tid = threadIdx.x;
  const int past = p.past[b], n = p.path_lens[b];
  const int32_t* path = p.path + (size_t)b * p.width;
  const int32_t* table = p.table ? p.table + (size_t)b * p.max_blocks : nullptr;
  // every CTA of a sequence checks it, and finds the same
  const bool latched = (*(volatile uint32_t*)p.status & PVA_DEV_KV_CACHE) != 0;
  const long long rows = (long long)p.max_blocks * p.page;
  bool bad_path = past < 0 || past > rows || n < 0 || n > p.width, bad_block = false;
  auto place = [&](int row, bool& bad) {
    const int in = row / p.page;
    const int block = table ? table[in] : b;
    bad = bad || block < 0 || block >= p.n_blocks;
    return (long long)block * p.Hkv * p.page + (row - in * p.page);
  };
  auto look_up = [&](int i0) {
    const int i = i0 + tid;
    if (i < n && !bad_path) {
      if (!path_node_ok(path, i, past, rows)) {
        bad_path = true;
      } else {
        const int x = path[i];
        s_to[tid] = place(past + i, bad_block);
        const long long from = place(past + x, bad_block);
        s_from[tid] = x == i ? -1 : from;
      }
    }
  };
  for (int i0 = 0; i0 < n && !bad_path; i0 += kPathRows) look_up(i0);
  const bool wrong_path = __syncthreads_or(bad_path);
  const bool wrong = __syncthreads_or(bad_block) || wrong_path;
  const bool first = blockIdx.x == 0 && tid == 0;
  if (latched || wrong) {
    if (first) {
      p.new_lens[b] = past;
      if (wrong) atomicOr(p.status, wrong_path ? PVA_DEV_TREE : PVA_DEV_BLOCKS);
    }
    return;
  }
  if (first) p.new_lens[b] = past + n;
  const int units = p.row_bytes / (int)sizeof(U);
  const long long columns = 2LL * p.layers * p.Hkv * units;
  for (int i0 = 0; i0 < n; i0 += kPathRows) {
    if (n > kPathRows) {
      __syncthreads();
      look_up(i0);
      __syncthreads();
    }
    const int m = min(n - i0, kPathRows);
    for (long long c = (long long)blockIdx.x * kAcceptThreads + tid; c < columns;
         c += (long long)gridDim.x * kAcceptThreads) {
      const int unit = (int)(c % units);
      const long long rest = c / units;
      const int h = (int)(rest % p.Hkv);
      const long long layer = rest / p.Hkv >> 1;
      uint8_t* base = ((rest / p.Hkv) & 1 ? p.v : p.k) + layer * p.layer_bytes +
                      (long long)h * p.page * p.row_bytes + (long long)unit * sizeof(U);
      for (int j = 0; j < m; j += kAcceptAhead) {
        U x[kAcceptAhead];
#pragma unroll
        for (int i = 0; i < kAcceptAhead; ++i)
          if (j + i < m && s_from[j + i] >= 0)
            x[i] = *reinterpret_cast<const U*>(base + s_from[j + i] * p.row_bytes);
#pragma unroll
        for (int i = 0; i < kAcceptAhead; ++i)
          if (j + i < m && s_from[j + i] >= 0)
            *reinterpret_cast<U*>(base + s_to[j + i] * p.row_bytes) = x[i];
      }
    }
  }
}

}  // namespace
}  // namespace pva

extern "C" int pva_block_tables(const int32_t* lens, int32_t* block_table, int32_t* held,
                                int32_t* free_blocks, int32_t* free_count, const int32_t* cu_new,
                                int64_t* slot_map, int B, int max_blocks, int page_size, int pool,
                                int64_t n_slots, void* stream_) {
  return guarded([&]() -> int {
    if (!lens || !block_table || !held || !free_blocks || !free_count)
      return fail(PVA_ERR_INVALID_ARG, "null lens, block_table, held or free list pointer");
    if (B < 1 || max_blocks < 1 || page_size < 1 || pool < 1 || n_slots < 0)
      return fail(PVA_ERR_INVALID_ARG,
                  "need B >= 1, max_blocks >= 1, page_size >= 1, pool >= 1, n_slots >= 0");
    if ((cu_new != nullptr) != (slot_map != nullptr) && !(cu_new && n_slots == 0))
      return fail(PVA_ERR_INVALID_ARG, "cu_new and slot_map come together");
    const cudaStream_t stream = static_cast<cudaStream_t>(stream_);
    std::lock_guard<std::mutex> lock(api_mutex());
    CallContext c;
    const int rc = acquire(stream, 0, &c);
    if (rc != PVA_OK) return rc;
    BlockParams p{lens, block_table, held, free_blocks, free_count, cu_new, slot_map, B,
                  max_blocks, page_size, pool, n_slots, n_slots <= kSlotsInOne ? 1 : 0, c.status};
    // few sequences: fewer warps to wait for
    const int threads = B <= 128 ? 256 : kBlockThreads;
    cudaError_t e = launch_dependent(pva_block_alloc_kernel, dim3(1), dim3(threads), 0, stream, p);
    if (e == cudaSuccess && cu_new && !p.in_one) {
      const long long want = (n_slots + 255) / 256, most = (long long)c.num_sms * 8;
      e = launch_dependent(pva_block_slots_kernel, dim3((unsigned)(want < most ? want : most)),
                           dim3(256), 0, stream, p);
    }
    return e == cudaSuccess ? PVA_OK : cuda_fail(e, "block table launch");
  });
}

extern "C" int pva_kvcache_accept(void* k_cache, void* v_cache, const int32_t* past_lens,
                                  const int32_t* path, const int32_t* path_lens,
                                  const int32_t* block_table, int32_t* new_lens, int B,
                                  int path_width, int layers, int64_t layer_stride, int n_blocks,
                                  int kv_num_heads, int page_size, int head_size, int max_blocks,
                                  int dtype, void* stream_) {
  return guarded([&]() -> int {
    if (!k_cache || !v_cache || !past_lens || !path || !path_lens || !new_lens)
      return fail(PVA_ERR_INVALID_ARG, "null cache, past_lens, path or new_lens pointer");
    if (B < 1 || path_width < 1 || layers < 1 || n_blocks < 1 || kv_num_heads < 1 ||
        page_size < 1 || head_size < 1)
      return fail(PVA_ERR_INVALID_ARG, "counts and sizes must be positive");
    if (dtype != PVA_F32 && dtype != PVA_F16 && dtype != PVA_BF16)
      return fail(PVA_ERR_INVALID_ARG, "dtype must be 0 (f32), 1 (f16) or 2 (bf16)");
    if (block_table ? max_blocks < 1 : n_blocks != B)
      return fail(PVA_ERR_INVALID_ARG,
                  block_table ? "max_blocks must be >= 1"
                              : "without a block table the cache has one block a sequence");
    if (!block_table) max_blocks = 1;
    if (B > 65535) return fail(PVA_ERR_UNSUPPORTED, "at most 65535 sequences");
    if ((long long)max_blocks * page_size > INT_MAX || (long long)head_size * 4 > INT_MAX ||
        (long long)n_blocks * kv_num_heads > INT_MAX)
      return fail(PVA_ERR_INVALID_ARG, "cache extents do not fit in int32");
    const long long size = dtype == PVA_F32 ? 4 : 2;
    const long long one = (long long)n_blocks * kv_num_heads * page_size * head_size;
    if (layers > 1 && layer_stride < one)
      return fail(PVA_ERR_INVALID_ARG, "layer_stride is smaller than a layer's cache");
    // one CTA of a sequence writes its new length while the others read these
    auto on_new_lens = [&](const int32_t* a, long long n) {
      const uintptr_t x = (uintptr_t)a, y = (uintptr_t)new_lens;
      return a && x < y + 4 * (uintptr_t)B && y < x + 4 * (uintptr_t)n;
    };
    if (on_new_lens(past_lens, B) || on_new_lens(path_lens, B) ||
        on_new_lens(path, (long long)B * path_width) ||
        on_new_lens(block_table, (long long)B * max_blocks))
      return fail(PVA_ERR_INVALID_ARG, "new_lens must not overlap an input");
    AcceptParams p{};
    p.k = static_cast<uint8_t*>(k_cache);
    p.v = static_cast<uint8_t*>(v_cache);
    p.past = past_lens;
    p.path = path;
    p.path_lens = path_lens;
    p.table = block_table;
    p.new_lens = new_lens;
    p.B = B;
    p.width = path_width;
    p.layers = layers;
    p.n_blocks = n_blocks;
    p.Hkv = kv_num_heads;
    p.page = page_size;
    p.max_blocks = max_blocks;
    p.layer_bytes = layers > 1 ? layer_stride * size : 0;
    p.row_bytes = (int)(head_size * size);
    const uintptr_t mis = (uintptr_t)k_cache | (uintptr_t)v_cache | (uintptr_t)p.layer_bytes |
                          (uintptr_t)p.row_bytes;
    if (mis % size) return fail(PVA_ERR_INVALID_ARG, "a cache is not aligned to its elements");
    const cudaStream_t stream = static_cast<cudaStream_t>(stream_);
    std::lock_guard<std::mutex> lock(api_mutex());
    CallContext c;
    const int rc = acquire(stream, 0, &c);
    if (rc != PVA_OK) return rc;
    p.status = c.status;
    // as many CTAs a sequence as it has columns for, up to about 16 per SM in all
    const int unit = mis % 16 == 0 ? 16 : mis % 4 == 0 ? 4 : 2;
    const long long columns = 2LL * layers * kv_num_heads * (p.row_bytes / unit);
    const long long want = (columns + kAcceptThreads - 1) / kAcceptThreads;
    const long long most = (16LL * c.num_sms + B - 1) / B;
    const dim3 grid((unsigned)(want < most ? want : most), B), block(kAcceptThreads);
    const cudaError_t e =
        unit == 16  ? launch_dependent(pva_accept_kernel<uint4>, grid, block, 0, stream, p)
        : unit == 4 ? launch_dependent(pva_accept_kernel<uint32_t>, grid, block, 0, stream, p)
                    : launch_dependent(pva_accept_kernel<uint16_t>, grid, block, 0, stream, p);
    return e == cudaSuccess ? PVA_OK : cuda_fail(e, "accept launch");
  });
}
