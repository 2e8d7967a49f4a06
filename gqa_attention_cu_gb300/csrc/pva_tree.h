// Parameters of the tree step (pva_gqa_tree) shared by its kernels: the front
// end, the attention kernels (tensor cores, fp32) and the join of split items.
//
// Work is counted in places.  Item (b, kv head, q tile t) covers the query
// rows [t * rows, (t + 1) * rows) of the n * G rows (row = node * G + head of
// the group) that sequence b has on one kv head, against the key tiles
// [item_lo / bn, ceil(item_hi / bn)): a place for each key tile, after
// `item_places` for what an item costs whatever its length (queries, pipeline,
// output).  All items' places form one line (sequence, kv head, q tile, key
// tile), which is cut into pieces of `chunk` places, one piece per CTA: every
// CTA gets the same amount of work whatever the lengths are.  An item that lies
// across a cut is computed by several CTAs, each of which leaves its unnormalised
// sums (O, the running maximum m and the sum l, all fp32) in a slot; the join
// kernel adds them in the order of the line, so results do not depend on timing.
//
// Where q tiles share keys and there are many items, CTAs instead take whole
// items in turn from a counter: then the q tiles of one kv head run side by
// side and find each other's keys in L2, where pieces of the line would be at
// far-apart places of the cache at any time.  (2048-token chunks of 8 sequences
// on 4.6k rows, d = 128, queries rotated before: 1.31 ms by pieces, bound by copies
// at 5.3 TB/s, against 1.10 ms.)  With fewer than 6 items per CTA the last ones would
// leave too many CTAs idle.
#pragma once

#include "pva_internal.h"

namespace pva {

// The item that a piece began and later pieces go on with.
struct alignas(16) TreeCut {
  int b, h, t;
  int parts;  // pieces that hold a part of it
  int rows;   // its query rows; 0: the piece finished all it began
  int pad[3];
};

// Keys per key tile of the tensor-core kernel (TMEM holds two score tiles, O and Q).
__host__ __device__ constexpr int tree_keys(int d) { return d <= 128 ? 128 : 64; }

// Whether the paired kernel takes a step of `rows` query rows per kv head.  Both
// parts of the queries of two tiles fit shared memory beside the ring up to d =
// 128, and then leave it three slots and the tensor cores half as much work again,
// so a pair has to be 7/8 full (4 query heads per kv head, d = 128, the paired
// kernel against the one-tile kernel, us: 8 sequences of 500 to 8000 rows, 40
// nodes 117 and 98, 64 nodes 129 and 130, 128 nodes 218 and 215; 4 sequences of
// 100,000 rows and more, 61 nodes 490 and 560).  Queries in one part: 87 and 92 us
// at 40 nodes already.
constexpr bool tree_takes_pair(long long rows, int d, int q_parts) {
  if (rows <= 128) return false;
  if (q_parts == 1) return d <= 192;
  return d <= 128 && 8 * rows >= 7 * ((rows + 255) / 256 * 256);
}

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
  float mid_to;            // and by the polynomial of mid_tanh, where that form is there
  float series_to;         // largest |q . k| whose softcap the tensor-core kernels take by series
  int rot, n_axes, cache_rows;  // rotary positions checked by the front end
  int rows, bn;            // query rows and keys of a tile
  int item_places;         // an item's fixed cost, in key tiles
  int QT;                  // q tiles of T nodes
  int W32;                 // mask words per node (0: chain)
  int pieces;              // CTAs of the attention kernel
  int may_take_items;      // the kernel can work by whole items
  int min_chunk;           // key tiles a piece has at least
  uint64_t hold_ns;        // > 0: the matrix warp waits as long for nothing and gives up
                           // (pva_selftest_give_up)
  // workspace
  int32_t* hdr;            // [0] accepted (until a wait is given up), [1] n_tiles, [2] chunk,
                           // [3] items to take (0: by pieces), [4] items taken
  int32_t* item_start;     // [B + 1] first item of each sequence
  int32_t* tile_start;     // [B + 1] first tile of each sequence on the line
  int32_t* q_start;        // [B][QT + 1] tiles before each q tile, within one kv head
  int32_t* depth;          // [B, T]
  uint32_t* mask;          // [B, T, W32] bit j: node j is seen
  void* q;                 // [q_parts][B][Hkv][T * G][d] rotated queries: the rounded values,
                           // and what rounding took off them
  int q_parts;
  float* part_o;           // [2 * pieces][rows][d]
  float2* part_ml;         // [2 * pieces][rows]
  TreeCut* cuts;           // [pieces]
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
  int parts;        // of the item, where this segment is its first part
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

// Key tiles of an item: how many, and the first one's index in the sequence.
__host__ __device__ inline int tree_item_tiles(const TreeParams& p, int past, int n, int t,
                                               int& lo, int& first) {
  int hi;
  tree_item_range(p, past, n, t, lo, hi);
  first = lo / p.bn;
  return (hi + p.bn - 1) / p.bn - first;
}

// Tells the join what a piece has left open: `s`, its last segment, or nothing.
__device__ __forceinline__ void tree_note_cut(const TreeParams& p, int piece, const TreeSegment* s) {
  TreeCut c{};
  if (s && s->parts > 1) {
    c.b = s->b;
    c.h = s->h;
    c.t = s->t;
    c.parts = s->parts;
    const int left = s->n * p.G - s->t * p.rows;
    c.rows = left < p.rows ? left : p.rows;
  }
  p.cuts[piece] = c;
}

// A CTA's segments, one after another: those of its piece of the line, or whole
// items.  One warp walks (all of its lanes hold the same state); only the first
// segment of a piece is looked up, the others follow from the one before by
// arithmetic, but for a new sequence's lengths.
struct TreeWalk {
  int piece, chunk, items, end;
  long long x;    // the place on the line where the next segment begins
  int b, h, t;    // its item
  int past, n;
  int into;       // places of the item that lie before x
  int next_item;  // whole items: the next one's number
  __device__ __forceinline__ TreeWalk(const TreeParams& p, int piece_) : piece(piece_) {
    const int places = p.hdr[1];
    chunk = p.hdr[2];
    items = p.hdr[3];
    x = (long long)piece * chunk;
    end = (int)(x + chunk < places ? x + chunk : places);
    if (items) {
      next_item = draw(p);
    } else if (x < end) {
      b = tree_find(p.tile_start, p.B, (int)x);
      const int first = p.tile_start[b], rel = (int)x - first;
      const int per_head = (p.tile_start[b + 1] - first) / p.Hkv;
      past = p.past[b];
      n = tree_nodes(p, b);
      h = rel / per_head;
      t = 0;
      into = rel - h * per_head;
      if (p.QT > 1) {
        const int32_t* qs = p.q_start + (size_t)b * (p.QT + 1);
        t = tree_find(qs, p.QT, into);
        into -= qs[t];
      }
    }
    if ((items || x >= end) && (threadIdx.x & 31) == 0) tree_note_cut(p, piece, nullptr);
  }
  __device__ __forceinline__ int draw(const TreeParams& p) {
    int i = 0;
    if ((threadIdx.x & 31) == 0) i = atomicAdd(p.hdr + 4, 1);
    return __shfl_sync(0xffffffffu, i, 0);
  }
  __device__ __forceinline__ int q_tiles(const TreeParams& p) const {
    return (n * p.G + p.rows - 1) / p.rows;
  }
  __device__ __forceinline__ bool next(const TreeParams& p, TreeSegment& s) {
    if (items) {
      if (next_item >= items) return false;
      s.b = tree_find(p.item_start, p.B, next_item);
      const int rel = next_item - p.item_start[s.b];
      s.past = past = p.past[s.b];
      s.n = n = tree_nodes(p, s.b);
      next_item = draw(p);
      s.h = rel / q_tiles(p);
      s.t = q_tiles(p) - 1 - (rel - s.h * q_tiles(p));  // the longest of a chain first
      s.count = tree_item_tiles(p, past, n, s.t, s.lo, s.j0);
      s.slot = -1;
      s.parts = 0;
      return true;
    }
    while (x < end) {
      s.b = b;
      s.h = h;
      s.t = t;
      s.past = past;
      s.n = n;
      int first;
      const int tiles = tree_item_tiles(p, past, n, t, s.lo, first), places = tiles + p.item_places;
      const int take = places - into < end - (int)x ? places - into : end - (int)x;
      // the item's first p.item_places places stand for its fixed cost
      const int from = into > p.item_places ? into - p.item_places : 0;
      const int to = into + take > p.item_places ? into + take - p.item_places : 0;
      s.j0 = first + from;
      s.count = to - from;
      s.slot = from == 0 && to == tiles ? -1 : tree_slot(piece, from == 0);
      const long long last = x - into + places - 1;
      s.parts = s.slot >= 0 && from == 0 ? (int)(last / chunk) - piece + 1 : 0;
      x += take;
      into += take;
      if (into == places) {  // on to the next item
        into = 0;
        if (++t == q_tiles(p)) {
          t = 0;
          if (++h == p.Hkv) {
            h = 0;
            if (x < end) {
              do {
                n = tree_nodes(p, ++b);
              } while (n == 0);
              past = p.past[b];
            }
          }
        }
      }
      const bool cut = x >= end && s.count > 0;
      if (x >= end && (threadIdx.x & 31) == 0) tree_note_cut(p, piece, cut ? &s : nullptr);
      if (s.count > 0) return true;
    }
    return false;
  }
};
#endif

cudaError_t launch_tree_tc(const TreeParams& p, int dtype, const CUtensorMap& tq,
                           const CUtensorMap& tk, const CUtensorMap& tv, cudaStream_t s);
// Two query tiles per item (p.rows = 256), head sizes up to 192.
cudaError_t launch_tree_pair(const TreeParams& p, int dtype, const CUtensorMap& tq,
                             const CUtensorMap& tk, const CUtensorMap& tv, cudaStream_t s);
cudaError_t launch_tree_f32(const TreeParams& p, cudaStream_t s);

}  // namespace pva
