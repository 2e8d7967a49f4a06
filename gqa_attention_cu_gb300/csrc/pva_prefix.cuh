// The work of attention behind shared prefixes (pva_gqa_prefix) for the kernels of
// the paged caches, which it runs with segments of its own.
//
// Two kinds of entries share one line of places (pva_tree.h): entry e < P is prefix e
// with the query rows of all its sequences, which see all of its keys; entry P + b is
// sequence b with its own rows, a chain.  So a prefix's keys and values are read once
// for as many query rows as a tile holds, and CTAs that are bound by the tensor cores
// (prefixes) run beside others that are bound by memory (own rows).  Every query row
// has one item of each kind.  An item that lies inside one piece leaves its row's
// unnormalised sums (O, the maximum and the weight) in the row's place of that kind,
// one across a cut in the pieces' slots; the join adds them up, prefix first, in the
// order of the line.
//
// Query rows come straight from q: a tile is tile_rows / G tokens x the G heads of a
// kv head.
#pragma once

#include "pva_tree_tile.cuh"

namespace pva {

struct PrefixParams : TreeParams {
  const int32_t* keys;          // [B] own cache rows (lens: tokens in use, or nullptr)
  const int32_t* prefix_keys;   // [P]
  const int32_t* prefix_start;  // [P + 1] first sequence of each, or nullptr: one prefix for all
  const int32_t* prefix_table;  // [P, prefix_blocks], or nullptr: block B + p
  int P, prefix_blocks;
  int tile_rows;                // query rows of an MMA tile: G times tokens
  int own_rows;                 // of them, those that a sequence of T tokens can have
  int tile_cost[2], item_cost[2];  // places of a key tile and of an item besides: own rows, prefix
  int negated;                  // a negative scale (tensor cores: as the sign of q)
  long long row_at;             // part_o's and part_ml's first row place, behind the slots
  float* lse;                   // [B, T, H], or nullptr
};

// Boxes of q: a tile's tokens, and no more than a sequence has (decoding: 1 of 32).
struct alignas(64) PrefixQueries {
  CUtensorMap tile, own;
};

// What an entry comes to.
struct PrefixEntry {
  int tok0, n, keys, all;  // first token, tokens, keys; all: every row sees all keys
  __host__ __device__ int q_tiles(const PrefixParams& p) const {
    return (int)(((long long)n * p.G + p.rows - 1) / p.rows);
  }
  __host__ __device__ int tiles(const PrefixParams& p) const { return (keys + p.bn - 1) / p.bn; }
  // places of one of its items
  __host__ __device__ int places(const PrefixParams& p) const {
    return n > 0 && keys > 0 ? tiles(p) * p.tile_cost[all] + p.item_cost[all] : 0;
  }
  __host__ __device__ long long per_head(const PrefixParams& p) const {
    return (long long)q_tiles(p) * places(p);
  }
  // key tiles that q tile t sees something of
  __host__ __device__ int seen(const PrefixParams& p, int t) const {
    if (all) return tiles(p);
    const long long last = (long long)(t + 1) * p.rows < (long long)n * p.G ? (long long)(t + 1) * p.rows : (long long)n * p.G;
    return (keys - n + (int)((last - 1) / p.G) + 1 + p.bn - 1) / p.bn;
  }
};

// The key tiles [from, to) that begin in the places [into, into + take) of an item:
// first its fixed cost, then tile after tile.
__host__ __device__ inline void prefix_tiles(const PrefixParams& p, int all, int into, int take, int seen, int& from,
                                             int& to) {
  const int item = p.item_cost[all], tile = p.tile_cost[all];
  from = into > item ? (into - item + tile - 1) / tile : 0;
  to = into + take > item ? (into + take - item + tile - 1) / tile : 0;
  if (to > seen) to = seen;
}

struct PrefixSegment : TreeSegment {  // b: the entry; past + n keys of a sequence, past of a prefix
  int tok0, all;
};

#ifdef __CUDACC__
__device__ __forceinline__ PrefixEntry prefix_entry(const PrefixParams& p, int e) {
  PrefixEntry x;
  if (e < p.P) {
    const int first = p.prefix_start ? p.prefix_start[e] : 0, end = p.prefix_start ? p.prefix_start[e + 1] : p.B;
    x = {first * p.T, (end - first) * p.T, p.prefix_keys[e], 1};
  } else {
    const int b = e - p.P;
    x = {b * p.T, tree_nodes(p, b), p.keys[b], 0};
  }
  return x;
}

// A CTA's segments: those of its piece of the line.  An entry is looked up once for
// all of its kv heads.
struct PrefixWalk {
  int piece, x, end;
  int e, start, stop;  // the entry at x and its places [start, stop)
  PrefixEntry entry;
  int per, qt, h, t, into;  // places of an item, q tiles; the item at x, places of it before x
  __device__ __forceinline__ PrefixWalk(const PrefixParams& p, int piece_) : piece(piece_), e(-1), stop(0) {
    const int places = p.hdr[1], chunk = p.hdr[2];
    const long long from = (long long)piece * chunk;
    x = (int)(from < places ? from : places);
    end = from + chunk < places ? (int)(from + chunk) : places;
  }
  __device__ __forceinline__ bool next(const PrefixParams& p, PrefixSegment& s) {
    while (x < end) {
      if (x >= stop) {
        if (e < 0) e = tree_find(p.tile_start, p.P + p.B, x);
        else ++e;
        while ((stop = p.tile_start[e + 1]) <= x) ++e;
        start = p.tile_start[e];
        entry = prefix_entry(p, e);
        per = entry.places(p);
        qt = entry.q_tiles(p);
        const int item = (x - start) / per;
        into = x - start - item * per;
        h = item / qt;
        t = item - h * qt;
      }
      const int take = end - x < per - into ? end - x : per - into;
      s.b = e;
      s.h = h;
      s.t = t;
      s.all = entry.all;
      s.tok0 = entry.tok0;
      s.n = entry.n;
      s.past = entry.all ? entry.keys : entry.keys - entry.n;
      s.lo = 0;
      int to;
      prefix_tiles(p, entry.all, into, take, entry.seen(p, t), s.j0, to);
      s.count = to - s.j0;
      s.slot = take == per ? -1 : tree_slot(piece, into == 0);
      s.parts = 0;
      x += take;
      into = 0;  // (after the last piece of an item, or at the end)
      if (++t == qt) {
        t = 0;
        ++h;
      }
      if (s.count > 0) return true;
    }
    return false;
  }
};

struct PrefixWork {
  using Params = PrefixParams;
  using Segment = PrefixSegment;
  using Walk = PrefixWalk;
  static __device__ __forceinline__ int total(const Segment& s) { return s.past + (s.all ? 0 : s.n); }
  static __device__ __forceinline__ int block(const Params& p, const Segment& s, int in) {
    if (s.all) return p.prefix_table ? p.prefix_table[(size_t)s.b * p.prefix_blocks + in] : p.B + s.b;
    const int b = s.b - p.P;
    return p.table ? p.table[(size_t)b * p.max_blocks + in] : b;
  }
  using Queries = PrefixQueries;
  static __device__ __forceinline__ void prefetch(const Queries& maps) {
    prefetch_tensor_map(&maps.tile);
    prefetch_tensor_map(&maps.own);
  }
  static __device__ __forceinline__ uint32_t q_bytes(const Params& p, const Segment& s) {
    return (uint32_t)(s.all ? p.tile_rows : p.own_rows) * 128u;
  }
  static __device__ __forceinline__ void load_q(const Params& p, const Segment& s, int y, int, void* dst,
                                                const Queries& maps, uint64_t* bar, int c) {
    tma_load_3d(dst, s.all ? &maps.tile : &maps.own, bar, c * 64, s.h * p.G, s.tok0 + (s.t * p.rows + y * p.tile_rows) / p.G);
  }
  static __device__ __forceinline__ uint32_t negate(const Params& p) { return p.negated ? 1u << 13 : 0u; }
  static __device__ __forceinline__ int row(const Params& p, const Segment& s, int y, int r) {
    return s.t * p.rows + y * p.tile_rows + r;
  }
  // a row of a token that is used; what the tile's other rows hold is not known
  static __device__ __forceinline__ bool owns(const Params& p, const Segment& s, int r, int row) {
    if (r >= p.tile_rows || row >= s.n * p.G) return false;
    if (!s.all || !p.lens) return true;
    const int tok = s.tok0 + row / p.G;
    return tok % p.T < p.lens[tok / p.T];
  }
  static __device__ __forceinline__ bool counts(bool own) { return own; }
  static constexpr bool kMid = true;
  // the join looks up at once what the front end has written
  static __device__ __forceinline__ void start() {
    wait_prior_grid();
    allow_next_grid();
  }
  static __device__ __forceinline__ tile::RowView view(const Params& p, const Segment& s, int node) {
    return {0, s.all ? s.past : s.past + node + 1, nullptr};
  }
  // where a row's sums go
  static __device__ __forceinline__ size_t place(const Params& p, const Segment& s, int row) {
    if (s.slot >= 0) return (size_t)s.slot * p.rows + (row - s.t * p.rows);
    const int node = row / p.G;
    return (size_t)p.row_at + ((size_t)(s.all ? 0 : p.B) * p.T + s.tok0 + node) * p.H + s.h * p.G + (row - node * p.G);
  }
  template <typename T, int D>
  static __device__ __forceinline__ void store(const Params& p, const Segment& s, uint32_t t_o, bool own, int row, int,
                                               tile::Columns cols, float m, float l) {
    const size_t at = own ? place(p, s, row) : 0;
    float* part = p.part_o + at * D;
    if (own && cols.begin == 0) p.part_ml[at] = make_float2(m, l);
#pragma unroll 1
    for (int c = cols.begin; c < cols.end; c += 32) {
      uint32_t v[32];
      tmem_ld32(t_o + c, v);
      tmem_wait_ld_of(v);
      if (own) {
#pragma unroll
        for (int e = 0; e < 32; e += 4)
          *reinterpret_cast<uint4*>(part + c + e) = make_uint4(v[e], v[e + 1], v[e + 2], v[e + 3]);
      }
    }
  }
  static __device__ __forceinline__ const float* q_row(const Params& p, const Segment& s, int row) {
    const int node = row / p.G;
    return static_cast<const float*>(p.q) + (((size_t)s.tok0 + node) * p.H + s.h * p.G + (row - node * p.G)) * p.d;
  }
  static __device__ __forceinline__ tile::RowOut row_out(const Params& p, const Segment& s, int row, int) {
    const size_t at = place(p, s, row);
    return {p.part_o + at * p.d, p.part_ml + at};
  }
  // a wait was given up: nothing is joined
  static __device__ __forceinline__ void give_up(const Params& p) { atomicExch(p.hdr, 0); }
};
#endif

cudaError_t launch_prefix_tc(const PrefixParams& p, int dtype, const PrefixQueries& tq, const CUtensorMap& tk,
                             const CUtensorMap& tv, cudaStream_t s);
// Two query tiles per item (p.rows = 2 p.tile_rows), head sizes up to 192, no softcap.
cudaError_t launch_prefix_pair(const PrefixParams& p, int dtype, const PrefixQueries& tq, const CUtensorMap& tk,
                               const CUtensorMap& tv, cudaStream_t s);

}  // namespace pva
