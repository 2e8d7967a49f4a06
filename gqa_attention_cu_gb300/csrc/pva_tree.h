// Parameters of the tree step (pva_gqa_tree) shared by its kernels: the front
// end, the attention kernels (tensor cores, fp32) and the join of split items.
//
// Work is counted in key tiles.  Item (b, kv head, q tile t) covers the query
// rows [t * rows, (t + 1) * rows) of the n * G rows (row = node * G + head of
// the group) that sequence b has on one kv head, against the key tiles
// [item_lo / bn, ceil(item_hi / bn)).  All items' tiles form one line
// 0 .. n_tiles-1 (sequence, kv head, q tile, key tile), which is cut into
// pieces of `chunk` tiles, one piece per CTA: every CTA gets the same amount of
// keys whatever the lengths are.  An item that lies across a cut is computed
// by several CTAs, each of which leaves its unnormalised sums (O, the running
// maximum m and the sum l, all fp32) in a slot; the join kernel adds them in
// the order of the line, so results do not depend on timing.
#pragma once

#include "pva_internal.h"

namespace pva {

// Keys per key tile of the tensor-core kernel (TMEM holds two score tiles, O and Q).
__host__ __device__ constexpr int tree_keys(int d) { return d <= 128 ? 128 : 64; }

struct TreeParams {
  const int32_t* past;     // [B] cache rows before the step
  const int32_t* lens;     // [B] nodes in use, or nullptr: T
  const int32_t* parents;  // [B, T], or nullptr: a chain
  const int32_t* table;    // [B, max_blocks], or nullptr: sequence b owns block b
  const int64_t* pos;      // [n_axes, B, T], or nullptr
  int B, T, H, Hkv, G, d;
  int page, max_blocks, n_blocks;
  int window;
  float scale, softcap;
  int rot, n_axes, cache_rows;  // rotary positions checked by the front end
  int rows, bn;            // query rows and keys of a tile
  int QT;                  // q tiles of T nodes
  int W32;                 // mask words per node (0: chain)
  int pieces;              // CTAs of the attention kernel
  int min_chunk;           // key tiles a piece has at least
  // workspace
  int32_t* hdr;            // [0] accepted, [1] n_tiles, [2] chunk
  int32_t* tile_start;     // [B + 1] first tile of each sequence on the line
  int32_t* q_start;        // [B][QT + 1] tiles before each q tile, within one kv head
  int32_t* depth;          // [B, T]
  uint32_t* mask;          // [B, T, W32] bit j: node j is seen
  void* q;                 // [B][Hkv][T * G][d] rotated queries
  float* part_o;           // [2 * pieces][rows][d]
  float2* part_ml;         // [2 * pieces][rows]
  const void* k_cache;
  const void* v_cache;
  void* out;
  uint32_t* status;
};

// Keys [lo, hi) that some row of q tile t of a sequence (past, n nodes) sees:
// nodes follow their parents, so no row sees a node after its own.
__host__ __device__ inline void tree_item_range(const TreeParams& p, int past, int n, int t,
                                                int& lo, int& hi) {
  const int last_row = (t + 1) * p.rows < n * p.G ? (t + 1) * p.rows : n * p.G;
  hi = past + (last_row - 1) / p.G + 1;
  const int first = p.parents ? 0 : t * p.rows / p.G;  // least depth of the tile's nodes
  const long long from = p.window > 0 ? (long long)past + first + 1 - p.window : 0;
  lo = from > 0 ? (int)from : 0;
}

// Slot of a piece's part of an item: a piece holds at most one item that began
// before it and one that goes on after it.
__host__ __device__ inline int tree_slot(int piece, bool from_start) {
  return 2 * piece + (from_start ? 1 : 0);
}

// A piece's walk along the line of tiles.
struct TreeSegment {
  int b, h, t;      // sequence, kv head, q tile
  int past, n;      // rows before the step, nodes
  int j0, count;    // first key tile (index within the sequence) and how many
  int slot;         // slot of the partial sums, or -1: the whole item
  int lo;           // first key the item's rows see
};

#ifdef __CUDACC__
__device__ __forceinline__ int tree_nodes(const TreeParams& p, int b) {
  return p.lens ? p.lens[b] : p.T;
}

// Index of the last entry of start[0 .. n) that is <= x (entries ascend, the
// first one is <= x).  Called by a whole warp: 32 entries are compared at once,
// so few dependent loads stand between a piece and its first copy.
__device__ __forceinline__ int tree_find(const int32_t* start, int n, int x) {
  const int lane = threadIdx.x & 31;
  int lo = 0;
  while (n > 32) {  // 32 probes a step
    const int stride = (n + 31) / 32;
    const int i = lo + min(lane * stride, n - 1);
    const int hits = __popc(__ballot_sync(0xffffffffu, lane * stride < n && start[i] <= x));
    lo += (hits - 1) * stride;
    n = min(stride, n - (hits - 1) * stride);
  }
  return lo + __popc(__ballot_sync(0xffffffffu, lane < n && start[lo + min(lane, n - 1)] <= x)) - 1;
}

// The item at tile x of the line (a whole warp calls).
struct TreeItem {
  int b, h, t;
  int start, end;  // its tiles on the line
};
__device__ __forceinline__ TreeItem tree_item(const TreeParams& p, int x) {
  TreeItem i;
  i.b = tree_find(p.tile_start, p.B, x);
  const int32_t* qs = p.q_start + (size_t)i.b * (p.QT + 1);
  const int per_head = qs[p.QT], first = p.tile_start[i.b];
  i.h = (x - first) / per_head;
  const int base = first + i.h * per_head;
  i.t = tree_find(qs, p.QT, x - base);
  i.start = base + qs[i.t];
  i.end = base + qs[i.t + 1];
  return i;
}

// The segment at tile x of the line, for a piece that ends at `end` (a whole
// warp calls).
__device__ __forceinline__ TreeSegment tree_segment(const TreeParams& p, int piece, int x,
                                                    int end) {
  const TreeItem i = tree_item(p, x);
  TreeSegment s;
  s.b = i.b;
  s.h = i.h;
  s.t = i.t;
  const int in = x - i.start, all = i.end - i.start;
  s.past = p.past[s.b];
  s.n = tree_nodes(p, s.b);
  int hi;
  tree_item_range(p, s.past, s.n, s.t, s.lo, hi);
  s.j0 = s.lo / p.bn + in;
  s.count = all - in < end - x ? all - in : end - x;
  s.slot = in == 0 && s.count == all ? -1 : tree_slot(piece, in == 0);
  return s;
}
#endif

cudaError_t launch_tree_tc(const TreeParams& p, int dtype, const CUtensorMap& tq,
                           const CUtensorMap& tk, const CUtensorMap& tv, cudaStream_t s);
// Two query tiles per item (p.rows = 256), head sizes up to 192.
cudaError_t launch_tree_pair(const TreeParams& p, int dtype, const CUtensorMap& tq,
                             const CUtensorMap& tk, const CUtensorMap& tv, cudaStream_t s);
cudaError_t launch_tree_f32(const TreeParams& p, cudaStream_t s);

}  // namespace pva
