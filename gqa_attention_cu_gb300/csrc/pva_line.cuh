// Front ends that check the entries of a call (sequences, prefixes), add their places
// up to a line and have it cut: what pva_gqa_prefix and pva_kvcache_weights share.
//
// An operation `Op` says how many entries there are, what is wrong with one, how many
// places it has, where the sums go, and what comes of the total:
//   int entries() const;
//   uint32_t check(int e, int i0, int n, bool& off, bool& idle) const;   PVA_DEV_* bits,
//       the same in all n threads (whole warps) that work on entry e; off: a block table entry that
//       thread i0 has looked at is outside the pool; idle (in all of them): the entry has
//       no places, and may be anything
//   long long places(int e) const;   of an entry that is sound and not idle
//   int32_t* start() const;          [entries + 1]
//   void publish(long long all, uint32_t found, bool latched) const;   one thread
#pragma once

#include <limits.h>

#include "pva_device.cuh"

namespace pva {
namespace line {

constexpr int kThreads = 128;                        // of an entry's CTA
constexpr int kSmallEntries = 32, kSmallThreads = 1024;
constexpr int kWordArrived = 16, kWordBad = 17;      // of the status block, zero between calls

__device__ __forceinline__ long long sum_upto(long long x) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, o);
    if ((threadIdx.x & 31) >= o) x += y;
  }
  return x;
}

// One CTA per entry; the last one to finish adds up.
template <typename Op>
__global__ void __launch_bounds__(kThreads) pva_line_front_kernel(Op op, uint32_t* status) {
  wait_prior_grid();
  allow_next_grid();
  __shared__ int s_last;
  __shared__ long long s_sum[kThreads / 32];
  const int tid = threadIdx.x, E = op.entries();
  const bool latched = (*(volatile uint32_t*)status & PVA_DEV_KV_CACHE) != 0;
  bool off = false, idle = false;
  uint32_t bad = op.check(blockIdx.x, tid, kThreads, off, idle);
  if (__syncthreads_or(off)) bad |= PVA_DEV_BLOCKS;
  if (tid == 0) {
    op.start()[blockIdx.x] = idle;  // until the sum takes its place
    if (bad) atomicOr(status + kWordBad, bad);
    __threadfence();
    s_last = atomicAdd(status + kWordArrived, 1u) == gridDim.x - 1;
  }
  __syncthreads();
  if (!s_last) return;
  __threadfence();
  const uint32_t found = __ldcg(status + kWordBad);
  long long carry = 0;
  for (int e0 = 0; e0 < E && !found; e0 += kThreads) {
    const int e = e0 + tid;
    const bool none = e >= E || __ldcg(op.start() + e);
    const long long all = e < E ? op.places(e) : 0;  // (looked up beside that)
    const long long x = none ? 0 : all, upto = sum_upto(x);
    if ((tid & 31) == 31) s_sum[tid >> 5] = upto;
    __syncthreads();
    long long before = carry;
    for (int w = 0; w < kThreads / 32; ++w) {
      before += w < tid >> 5 ? s_sum[w] : 0;
      carry += s_sum[w];
    }
    if (e < E) op.start()[e] = (int)min(before + upto - x, (long long)INT_MAX);
    __syncthreads();
  }
  if (tid == 0) {
    status[kWordBad] = 0;  // for the next call
    status[kWordArrived] = 0;
    op.publish(carry, found, latched);
  }
}

// The same for up to 32 entries: one CTA, `group` threads an entry, that waits for no
// other.
template <typename Op>
__global__ void __launch_bounds__(kSmallThreads) pva_line_small_front_kernel(Op op, uint32_t* status, int group) {
  wait_prior_grid();
  allow_next_grid();
  __shared__ long long s_places[kSmallEntries];
  __shared__ uint32_t s_bad;
  const int tid = threadIdx.x, E = op.entries(), e = tid / group;
  const bool latched = (*(volatile uint32_t*)status & PVA_DEV_KV_CACHE) != 0;
  if (tid == 0) s_bad = 0;
  __syncthreads();
  if (e < E) {
    bool off = false, idle = false;
    uint32_t bad = op.check(e, tid - e * group, group, off, idle);
    if (tid == e * group) s_places[e] = bad || idle ? 0 : op.places(e);
    if (off) bad |= PVA_DEV_BLOCKS;
    if (bad) atomicOr(&s_bad, bad);
  }
  __syncthreads();
  if (tid >= 32) return;
  const long long x = tid < E ? s_places[tid] : 0, upto = sum_upto(x);
  if (tid < E) op.start()[tid] = (int)min(upto - x, (long long)INT_MAX);
  const long long all = __shfl_sync(0xffffffffu, upto, 31);
  if (tid == 0) op.publish(all, s_bad, latched);
}

// blocks: the width of the widest table.  One CTA where its threads look at a few table
// entries each (2 sequences behind a prefix 20.4 to 18.5 us; 27 entries with 563 blocks by
// a warp each 78 to 87 us).
template <typename Op>
cudaError_t launch_front(const Op& op, int entries, int blocks, uint32_t* status, cudaStream_t s) {
  int group = kSmallThreads;  // whole warps an entry
  while (group > 32 && (long long)group * entries > kSmallThreads) group /= 2;
  if (entries > kSmallEntries || blocks > 8 * group)
    return launch_dependent(pva_line_front_kernel<Op>, dim3(entries), dim3(kThreads), 0, s, op, status);
  return launch_dependent(pva_line_small_front_kernel<Op>, dim3(1), dim3(group * entries), 0, s, op, status, group);
}

// Whether some of the table entries that hold `rows` rows are outside [0, blocks).
__device__ __forceinline__ bool off_pool(const int32_t* table, int rows, int page, int blocks, int i0, int n) {
  bool off = false;
  const int used = rows > 0 ? (rows - 1) / page + 1 : 0;
#pragma unroll 4
  for (int i = i0; i < used; i += n) off |= (unsigned)table[i] >= (unsigned)blocks;
  return off;
}

}  // namespace line
}  // namespace pva
