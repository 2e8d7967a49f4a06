// Block tables and slot maps of a paged KV cache (pva_block_tables), and the
// move of an accepted path's rows (pva_kvcache_accept).
//
// pva_block_tables is all latency: a few words per sequence and eight bytes per
// new token.  One CTA does the allocation (the stack is shared by all
// sequences): checks, prefix sums of what is given back and taken, then the
// blocks, a warp per sequence.  Slots are written by the same CTA while they
// are few, and by a grid of their own where they are many.
//
// pva_kvcache_accept moves rows in place.  A path rises, path[i] >= i, so row i
// is read (as some path[j], j <= i) before or when it is written if each thread
// keeps to one 16-byte column and goes through i in order: no copy is needed.
#include <limits.h>

#include "pva_device.cuh"

using namespace pva;
using namespace pva::host;

namespace pva {
namespace {

constexpr int kBlockThreads = 1024;
constexpr int kWordRefused = 18;  // status block: 1 while the last allocation was refused
// New tokens up to which the allocating CTA writes the slot map itself.
constexpr long long kSlotsInOne = 4096;

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

// Sum over the CTA of x, and of the threads before this one (exclusive).
__device__ __forceinline__ long long block_scan(long long x, long long* sums, long long& all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long upto = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += y;
  }
  if (lane == 31) sums[warp] = upto;
  __syncthreads();
  long long before = 0;
  all = 0;
  for (int w = 0; w < (int)blockDim.x / 32; ++w) {
    const long long s = sums[w];
    before += w < warp ? s : 0;
    all += s;
  }
  __syncthreads();
  return before + upto - x;
}

// Slot of token t of sequence b.
__device__ __forceinline__ int64_t slot_of(const BlockParams& p, int b, int t) {
  const int row = p.lens[b] - (p.cu_new[b + 1] - t);
  return (int64_t)p.table[(size_t)b * p.max_blocks + row / p.page] * p.page + row % p.page;
}

__global__ void __launch_bounds__(kBlockThreads) pva_block_alloc_kernel(BlockParams p) {
  allow_next_grid();
  wait_prior_grid();
  __shared__ long long s_sums[32];
  __shared__ int s_bad;
  const int tid = threadIdx.x;
  if (tid == 0) s_bad = 0;
  __syncthreads();
  const int count = *p.free_count;
  bool bad = count < 0 || count > p.pool;
  long long given = 0, taken = 0;
  for (int b = tid; b < p.B; b += kBlockThreads) {
    const int len = p.lens[b], held = p.held[b];
    if (len < 0 || held < 0 || held > p.max_blocks || blocks_for(len, p.page) > p.max_blocks) {
      bad = true;
      continue;
    }
    const int more = blocks_for(len, p.page) - held;
    if (more > 0) taken += more; else given -= more;
    if (p.cu_new) {
      const int c0 = p.cu_new[b], c1 = p.cu_new[b + 1];
      bad = bad || (b == 0 && c0 != 0) || c1 < c0 || (long long)c1 - c0 > len ||
            (b == p.B - 1 && c1 > p.n_slots);
    }
  }
  if (bad) s_bad = 1;
  long long all_given, all_taken;
  block_scan(given, s_sums, all_given);
  block_scan(taken, s_sums, all_taken);
  const bool refuse = s_bad || count + all_given > p.pool || all_taken > count + all_given;
  if (tid == 0 && !p.in_one) p.status[kWordRefused] = refuse ? 1u : 0u;
  if (refuse) {
    if (tid == 0) atomicOr(p.status, PVA_DEV_BLOCKS);
    return;
  }
  const int lane = tid & 31, warp = tid >> 5;
  const long long top = count + all_given - 1;
  // Two passes, given back first: both need the sequences' places on the
  // stack, found a thread per sequence, and move blocks, a warp per sequence.
  for (int pass = 0; pass < 2; ++pass) {
    if ((pass == 0 ? all_given : all_taken) == 0) continue;
    long long carry = 0;
    for (int b0 = 0; b0 < p.B; b0 += kBlockThreads) {
      const int b = b0 + tid;
      int held = 0, need = 0;
      if (b < p.B) {
        held = p.held[b];
        need = blocks_for(p.lens[b], p.page);
      }
      const int n = pass == 0 ? max(0, held - need) : max(0, need - held);
      long long all;
      long long at = carry + block_scan(n, s_sums, all);
      carry += all;
      // the warp goes through its 32 sequences together
      for (unsigned todo = __ballot_sync(0xffffffffu, n > 0); todo; todo &= todo - 1) {
        const int src = __ffs(todo) - 1;
        const int nn = __shfl_sync(0xffffffffu, n, src);
        const int from = __shfl_sync(0xffffffffu, min(held, need), src);
        const long long first = top - __shfl_sync(0xffffffffu, at, src);
        int32_t* row = p.table + (size_t)(b0 + warp * 32 + src) * p.max_blocks + from;
        for (int i = lane; i < nn; i += 32) {
          if (pass == 0) {
            p.free_blocks[first - i] = row[i];
            row[i] = -1;
          } else {
            row[i] = p.free_blocks[first - i];
          }
        }
      }
    }
    __syncthreads();
  }
  for (int b = tid; b < p.B; b += kBlockThreads) p.held[b] = blocks_for(p.lens[b], p.page);
  if (tid == 0) *p.free_count = (int)(count + all_given - all_taken);
  if (!p.in_one || !p.cu_new) return;
  __syncthreads();
  for (int b = warp; b < p.B; b += kBlockThreads / 32)
    for (int t = p.cu_new[b] + lane; t < p.cu_new[b + 1]; t += 32) p.slots[t] = slot_of(p, b, t);
  for (long long t = p.cu_new[p.B] + tid; t < p.n_slots; t += kBlockThreads) p.slots[t] = -1;
}

// A thread per token; the sequence by bisection of the offsets.
__global__ void __launch_bounds__(256) pva_block_slots_kernel(BlockParams p) {
  allow_next_grid();
  wait_prior_grid();
  if (p.status[kWordRefused]) return;
  const int end = p.cu_new[p.B];
  for (long long t = (long long)blockIdx.x * blockDim.x + threadIdx.x; t < p.n_slots;
       t += (long long)gridDim.x * blockDim.x) {
    if (t >= end) {
      p.slots[t] = -1;
      continue;
    }
    int lo = 0, hi = p.B - 1;  // the last b with cu_new[b] <= t
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (p.cu_new[mid] <= t) lo = mid; else hi = mid - 1;
    }
    p.slots[t] = slot_of(p, lo, (int)t);
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

// One CTA per (kv head, layer, sequence): threads are (K or V, column of 16,
// 4 or 2 bytes), each walking down the path.
template <typename U>
__global__ void __launch_bounds__(128) pva_accept_kernel(AcceptParams p) {
  allow_next_grid();
  wait_prior_grid();
  constexpr int kAhead = 8;
  const int b = blockIdx.z, layer = blockIdx.y, h = blockIdx.x;
  const int past = p.past[b], n = p.path_lens[b];
  const int32_t* path = p.path + (size_t)b * p.width;
  const int32_t* table = p.table ? p.table + (size_t)b * p.max_blocks : nullptr;
  // every CTA of a sequence checks it, and finds the same
  const bool latched = (*(volatile uint32_t*)p.status & PVA_DEV_KV_CACHE) != 0;
  bool bad_path = past < 0 || n < 0 || n > p.width, bad_block = false;
  const long long rows = (long long)p.max_blocks * p.page;
  for (int i = threadIdx.x; i < n && !bad_path; i += blockDim.x) {
    const int x = path[i];
    if (x < 0 || (i > 0 && path[i - 1] >= x) || past + (long long)x >= rows) {
      bad_path = true;
    } else if (table) {
      const int to = table[(past + i) / p.page], from = table[(past + x) / p.page];
      bad_block = bad_block || to < 0 || to >= p.n_blocks || from < 0 || from >= p.n_blocks;
    }
  }
  const bool wrong_path = __syncthreads_or(bad_path);
  const bool wrong = __syncthreads_or(bad_block) || wrong_path;
  const bool first = layer == 0 && h == 0 && threadIdx.x == 0;
  if (latched || wrong) {
    if (first) {
      p.new_lens[b] = past;
      if (wrong) atomicOr(p.status, wrong_path ? PVA_DEV_TREE : PVA_DEV_BLOCKS);
    }
    return;
  }
  if (first) p.new_lens[b] = past + n;
  const int columns = p.row_bytes / (int)sizeof(U);
  auto at = [&](uint8_t* base, int row) {
    const int in = row / p.page;
    const long long block = table ? table[in] : b;
    return reinterpret_cast<U*>(base + ((block * p.Hkv + h) * p.page + (row - in * p.page)) *
                                           (long long)p.row_bytes);
  };
  for (int c = threadIdx.x; c < 2 * columns; c += blockDim.x) {
    uint8_t* base = (c < columns ? p.k : p.v) + layer * p.layer_bytes;
    const int col = c < columns ? c : c - columns;
    for (int i0 = 0; i0 < n; i0 += kAhead) {
      U x[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (i0 + i < n) x[i] = at(base, past + path[i0 + i])[col];
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (i0 + i < n && path[i0 + i] != i0 + i) at(base, past + i0 + i)[col] = x[i];
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
    cudaError_t e = launch_dependent(pva_block_alloc_kernel, dim3(1), dim3(kBlockThreads), 0,
                                     stream, p);
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
    if (B > 65535 || layers > 65535)
      return fail(PVA_ERR_UNSUPPORTED, "at most 65535 sequences and layers");
    if ((long long)max_blocks * page_size > INT_MAX)
      return fail(PVA_ERR_INVALID_ARG, "cache extents do not fit in int32");
    const long long size = dtype == PVA_F32 ? 4 : 2;
    const long long one = (long long)n_blocks * kv_num_heads * page_size * head_size;
    if (layers > 1 && layer_stride < one)
      return fail(PVA_ERR_INVALID_ARG, "layer_stride is smaller than a layer's cache");
    const uintptr_t old0 = (uintptr_t)past_lens, new0 = (uintptr_t)new_lens;
    if (old0 < new0 + 4 * (uintptr_t)B && new0 < old0 + 4 * (uintptr_t)B)
      return fail(PVA_ERR_INVALID_ARG, "new_lens must not overlap past_lens");
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
    const dim3 grid(kv_num_heads, layers, B);
    const cudaError_t e =
        mis % 16 == 0 ? launch_dependent(pva_accept_kernel<uint4>, grid, dim3(128), 0, stream, p)
        : mis % 4 == 0
            ? launch_dependent(pva_accept_kernel<uint32_t>, grid, dim3(128), 0, stream, p)
            : launch_dependent(pva_accept_kernel<uint16_t>, grid, dim3(128), 0, stream, p);
    return e == cudaSuccess ? PVA_OK : cuda_fail(e, "accept launch");
  });
}
