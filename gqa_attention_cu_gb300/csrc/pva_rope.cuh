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
  long long n_slots;        // blocks * page
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

namespace host {
// Checks the rotary arguments and fills the table block (inverse left at 0).
int check_rope(const void* cos_cache, const void* sin_cache, int rot, int rows, int interleaved,
               int n_axes, const int32_t* sections, int axes_interleaved, int rotary_dtype,
               int dtype, int d, RopeTable* t);
}  // namespace host

cudaError_t launch_rope(const RopeStep& s, int dtype, bool tree, int num_sms, cudaStream_t st);

}  // namespace pva
