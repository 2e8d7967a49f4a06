// The weight that attention gives to each cache row (pva_kvcache_weights):
//   w[b, h, j] = decay * previous + sum over tokens t and heads g of the group of
//                exp(score(q[b, t, h G + g], k[j]) - lse[b, t, h G + g]).
//
// With lse given, one pass over the keys.  Without, either the scores of the first
// pass are kept (few query rows: 4 bytes a row and key, against 2 d bytes of the key
// itself) and a second kernel turns them into weights, or the keys are read twice.
//
//   front end (pva_line.cuh)  bounds and block tables, and the line of key tiles, which
//       is cut into a piece per SM.
//   pva_weights_tc_kernel     f16/bf16 on tensor cores: Store, Apply, Stats (below).
//   pva_weights_f32_kernel    f32 on the CUDA cores: Apply and Stats.
//   pva_weights_rows_kernel   joins the pieces' maxima and sums of each query row.
//   pva_weights_scores_kernel weights from kept scores.
//
// The line: (sequence, kv head, key tile of 128 keys), each tile counted once for
// every chunk of query rows that it is multiplied with.  A key's weight is written by
// one thread, chunk after chunk, so results do not depend on timing.
//
// Memory is the floor: 2 d bytes of a key, 4 or 8 of its weight.  Measured:
//   a decoding step of 32 sequences of 2000 to 16,000 rows, 32 query and 8 kv heads of
//     128 bf16, own sums: 120 us, of which the keys are 97 at 6.1 TB/s (91 us is the
//     floor), the kept scores 13 and the front end 6.  Keys leave L2 first, so that the
//     37 MB of scores are still there (without: 128 us).
//   32 tokens on 100,000 rows of one sequence, sums given: 40 us, the kernel 5.4 TB/s
//     (floor 31).  Of its steps: masks as a bound on the columns instead of a comparison
//     each 66 to 44 us (the last tile of a head was its CTA's longest), unmasked columns
//     in pairs without a test 147 to 67.
//   3 sequences of 300 to 900 rows, f32: 40 us, four launches of a few latencies each; one
//     token of 8 sequences of 8000 rows, f32: 298 us, with sums given 151 (floor 39).
//   32 tokens on 100,000 rows, own sums (keys read twice): 95 us (two reads 61).
#include <limits.h>
#include <math.h>

#include "pva_line.cuh"
#include "pva_tree.h"

using namespace pva;
using namespace pva::host;

namespace pva {
namespace {

constexpr int kKeys = 128;  // of a key tile
constexpr float kLog2e = 1.4426950408889634f;

struct WeightsParams {
  const void* q;           // [B, T, H, d]
  const void* k_cache;
  const int32_t* lens;     // [B] cache rows
  const int32_t* q_lens;   // [B] tokens in use, or nullptr: T
  const int32_t* table;    // [B, max_blocks], or nullptr: block b
  const float* previous;   // [B, Hkv, width], or nullptr
  const float* lse;        // [B, T, H], or nullptr
  float* weights;          // [B, Hkv, width]
  float decay, scale, softcap;
  int B, T, H, Hkv, G, d, width;
  int page, max_blocks, n_blocks;
  int tokens_at_once;      // of a chunk
  int pieces;
  uint64_t hold_ns;        // > 0: the matrix warp waits as long for nothing and gives up (pva_selftest_give_up)
  // workspace
  int32_t* hdr;            // [0] accepted (until a wait is given up), [1] places, [2] places of a piece
  int32_t* start;          // [B + 1] first place of each sequence
  float2* part;            // [B * Hkv + pieces][parts][T * G] (m, l) of a piece's keys
  int parts;               // that a piece leaves for a row
  float2* row;             // [B][Hkv][T * G] (m, 1 / l); with lse: not used
  float* scores;           // [places][rows][128]
  uint32_t* status;
};

// A sequence on the line.
struct Sequence {
  int n, q;       // cache rows, tokens
  int chunks;     // of query rows (one at least: the old weights fade in any case)
  int tiles;      // of keys
  __device__ __forceinline__ Sequence(const WeightsParams& p, int b)
      : n(p.lens[b]), q(p.q_lens ? p.q_lens[b] : p.T) {
    chunks = max(1, (q + p.tokens_at_once - 1) / p.tokens_at_once);
    tiles = (n + kKeys - 1) / kKeys;
  }
  __device__ __forceinline__ long long per_head() const { return (long long)tiles * chunks; }
};

// A piece's part of one (sequence, kv head): key tiles [j0, j1).
struct Segment {
  int b, h, n, q, chunks, j0, j1, slot;
};
// Tiles that begin in the places [from, to) of a head.
__host__ __device__ constexpr int first_tile(int place, int chunks) {
  return (int)(((unsigned)place + (unsigned)chunks - 1u) / (unsigned)chunks);
}
// The line may be as long as int32 allows, with more chunks to a tile than are left to its end.
static_assert(first_tile(INT_MAX - 608, 500000) == 4295 && first_tile(INT_MAX, 1 << 30) == 2 && first_tile(0, 7) == 0 &&
              first_tile(7, 7) == 1 && first_tile(8, 7) == 2, "tiles that begin before a place");

// Walks the segments of places [x, end); one warp, the same state in all lanes.
struct Walk {
  int piece;
  long long x, end;
  int b = -1;
  __device__ __forceinline__ Walk(const WeightsParams& p, int piece_, long long places, long long chunk)
      : piece(piece_) {
    x = piece * chunk;
    end = x + chunk < places ? x + chunk : places;
  }
  __device__ __forceinline__ bool next(const WeightsParams& p, Segment& s) {
    while (x < end) {
      if (b < 0) b = tree_find(p.start, p.B, (int)x);
      while (p.start[b + 1] <= x) ++b;
      const Sequence seq(p, b);
      const int rel = (int)x - p.start[b], per = (int)seq.per_head();
      s.b = b;
      s.h = rel / per;
      const int within = rel - s.h * per;
      const int take = (int)(end - x < per - within ? end - x : per - within);
      s.n = seq.n;
      s.q = seq.q;
      s.chunks = seq.chunks;
      s.j0 = first_tile(within, seq.chunks);
      s.j1 = first_tile(within + take, seq.chunks);
      s.slot = b * p.Hkv + s.h + piece;
      x += take;
      if (s.j0 < s.j1) return true;
    }
    return false;
  }
};

// Keys that token t of a sequence sees.
__device__ __forceinline__ int keys_of(const Segment& s, int t) { return s.n - s.q + t + 1; }

// Key tiles [j0, end) of chunk c: the first chunk visits all of a segment's.
__device__ __forceinline__ int chunk_end(const WeightsParams& p, const Segment& s, int c, bool stats) {
  if (c == 0 && !stats) return s.j1;
  const int last = min(s.q, (c + 1) * p.tokens_at_once);  // tokens up to here
  const int tiles = last > 0 ? (keys_of(s, last - 1) + kKeys - 1) / kKeys : 0;
  return max(s.j0, min(s.j1, tiles));
}

// The sequences on the line (pva_line.cuh).
struct WeightsFront {
  WeightsParams p;
  __device__ __forceinline__ int entries() const { return p.B; }
  __device__ __forceinline__ int32_t* start() const { return p.start; }
  __device__ __forceinline__ uint32_t check(int b, int i0, int n, bool& off, bool&) const {
    const int rows = p.lens[b], tokens = p.q_lens ? p.q_lens[b] : p.T;
    if (rows < 0 || rows > p.width || (long long)rows > (long long)p.max_blocks * p.page || tokens < 0 ||
        tokens > p.T || tokens > rows)
      return PVA_DEV_KV_LEN;
    off = p.table && line::off_pool(p.table + (size_t)b * p.max_blocks, rows, p.page, p.n_blocks, i0, n);
    return 0u;
  }
  __device__ __forceinline__ long long places(int b) const { return Sequence(p, b).per_head() * p.Hkv; }
  __device__ __forceinline__ void publish(long long sum, uint32_t found, bool latched) const {
    if (!found && sum > INT_MAX - 4ll * p.pieces) found = PVA_DEV_TOO_MANY;
    if (found) atomicOr(p.status, found);
    const int all = found || latched ? 0 : (int)sum;
    p.start[p.B] = all;
    p.hdr[0] = all > 0;
    p.hdr[1] = all;
    p.hdr[2] = max(1, (all + p.pieces - 1) / p.pieces);
  }
};

// score -> natural units, with the softcap.
template <bool CAP>
__device__ __forceinline__ float natural(float s, float scale, float softcap, float inv_cap) {
  const float x = s * scale;
  return CAP ? softcap * tanhf(x * inv_cap) : x;
}

// ---------------------------------------------------------------------------
// Tensor cores.  One CTA per piece, 576 threads:
//   warp 0      TMA producer: publishes the segments' chunks, loads the chunk's
//               query rows and then the key tiles through a ring.
//   warp 1      MMA issuer and TMEM owner; four score buffers.
//   warps 2..5, 6..9, ...   take the tiles of score buffer 0, 1, ...
// Store and Apply form S^T = K Q^T, 128 keys by N query rows: a thread has a key and
// adds up over its columns without meeting another.  Stats forms S = Q K^T, 128
// query rows by 128 keys: a thread has a row and keeps its running maximum and sum.
// ---------------------------------------------------------------------------
enum Mode { kStore, kApply, kStats };
constexpr int kGroups = 4;  // of four warps, with a score buffer each
constexpr int kTcThreads = 64 + 128 * kGroups;
constexpr int kItemSlots = 4;

struct ItemSlot {
  Segment s;
  int c, end, last;  // chunk, its last key tile + 1; no more work
};

struct Bars {
  uint64_t q_full[2], q_empty[2], drain, never;
  uint64_t s_full[kGroups], s_free[kGroups];
  uint64_t ring_full[12], ring_empty[12];
  uint64_t item_full[kItemSlots], item_empty[kItemSlots];
  ItemSlot items[kItemSlots];
  uint32_t tmem_base;
  int abort;
};
constexpr int kBarBytes = 1024;
static_assert(sizeof(Bars) <= kBarBytes, "barriers and segments");

template <int D, int N, int MODE>
struct WCfg {
  static constexpr int CH = (D + 63) / 64;
  static constexpr int Q_CHUNK = N * 128;       // bytes of 64 columns of the query rows
  static constexpr int Q_TILE = CH * Q_CHUNK;
  static constexpr int K_CHUNK = kKeys * 128;
  static constexpr int K_TILE = CH * K_CHUNK;
  static constexpr int Q_BUFS = 2 * Q_TILE <= 64 * 1024 ? 2 : 1;
  // barriers, then (Apply) each score warp's copy of the chunk's row values
  static constexpr int HEAD = kBarBytes + (MODE == kApply ? (4 * kGroups * N * 8 + 1023) / 1024 * 1024 : 0);
  static constexpr int OFF_RING = Q_BUFS * Q_TILE;
  static constexpr int SLOTS_FIT = (232448 - HEAD - OFF_RING) / K_TILE;
  static constexpr int SLOTS = SLOTS_FIT < 12 ? SLOTS_FIT : 12;
  static_assert(SLOTS >= 2, "ring depth");
  static constexpr int SMEM = HEAD + OFF_RING + SLOTS * K_TILE;
  static constexpr int COLS = MODE == kStats ? kKeys : N;  // of a score buffer
  static constexpr int TMEM_COLS = kGroups * COLS;
  static_assert(TMEM_COLS <= 512, "TMEM budget");
};

template <int W>
__device__ __forceinline__ void tmem_wait(uint32_t (&r)[W]) {
  if constexpr (W == 32) {
    tmem_wait_ld_of(r);
  } else {
    static_assert(W == 16, "one load");
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]),
                   "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]),
                   "+r"(r[13]), "+r"(r[14]), "+r"(r[15])::"memory");
  }
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

// l = sum of exp(x - m), m = max x: one more x.
__device__ __forceinline__ void add_score(float& m, float& l, float x) {
  const float NEG_INF = __int_as_float(0xff800000);
  if (x == NEG_INF) return;
  const float d = m - x, e = ex2_approx(-fabsf(d) * kLog2e);  // m = -inf: e = 0
  l = d >= 0.0f ? l + e : fmaf(l, e, 1.0f);
  m = fmaxf(m, x);
}
__device__ __forceinline__ void join_scores(float& m, float& l, float m2, float l2) {
  const float NEG_INF = __int_as_float(0xff800000);
  const float top = fmaxf(m, m2), base = top == NEG_INF ? 0.0f : top;
  l = l * exp2f((m - base) * kLog2e) + l2 * exp2f((m2 - base) * kLog2e);
  m = top;
}

template <typename T, int D, int N, int MODE, bool CAP>
__global__ void __launch_bounds__(kTcThreads, 1)
    pva_weights_tc_kernel(WeightsParams p, const __grid_constant__ CUtensorMap tmap_q,
                          const __grid_constant__ CUtensorMap tmap_k) {
  using C = WCfg<D, N, MODE>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  Bars* bars = reinterpret_cast<Bars*>(smem_raw);
  uint8_t* smem = smem_raw + C::HEAD;
  uint8_t* ring = smem + C::OFF_RING;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t* status = p.status;
  volatile int* abort = &bars->abort;
  if ((smem_u32(smem_raw) & 1023) != 0) {  // the tiles' layout rests on it
    if (threadIdx.x == 0) {
      wait_prior_grid();
      atomicOr(p.status, PVA_DEV_WAIT_TIMEOUT);
      atomicExch(p.hdr, 0);
    }
    return;
  }
  if (threadIdx.x == 0) {
    bars->abort = 0;
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars->q_full[i], 1);
      mbar_init(&bars->q_empty[i], 1);
    }
    for (int i = 0; i < kGroups; ++i) {
      mbar_init(&bars->s_full[i], 1);
      mbar_init(&bars->s_free[i], 4);
    }
    mbar_init(&bars->drain, 1);
    mbar_init(&bars->never, 1);
    for (int i = 0; i < C::SLOTS; ++i) {
      mbar_init(&bars->ring_full[i], 1);
      mbar_init(&bars->ring_empty[i], 1);
    }
    for (int i = 0; i < kItemSlots; ++i) {
      mbar_init(&bars->item_full[i], 1);
      mbar_init(&bars->item_empty[i], 1 + 4 * kGroups);
    }
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc<C::TMEM_COLS>(&bars->tmem_base);
  if (warp == 0 && lane == 0) {
    prefetch_tensor_map(&tmap_q);
    prefetch_tensor_map(&tmap_k);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  wait_prior_grid();
  allow_next_grid();  // the next kernel looks up at once what the front end has written
  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    return __all_sync(0xffffffffu, mbar_wait<false>(bar, parity, abort, status));
  };

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    Walk walk(p, blockIdx.x, p.hdr[0] ? p.hdr[1] : 0, p.hdr[2]);
    const int box = p.table && p.page < kKeys ? p.page : kKeys, copies = kKeys / box;
    const uint64_t once = read_once_policy();  // keys leave L2 first: scores and weights stay there
    uint32_t loads = 0, published = 0, q_loads = 0;
    bool ok = true;
    auto publish = [&](const ItemSlot& v) -> bool {
      const int sl = published % kItemSlots;
      if (!wait(&bars->item_empty[sl], ((published / kItemSlots) & 1) ^ 1)) return false;
      if (lane == 0) {
        bars->items[sl] = v;
        mbar_arrive(&bars->item_full[sl]);
      }
      __syncwarp();
      ++published;
      return true;
    };
    ItemSlot v;
    v.last = 0;
    while (ok && walk.next(p, v.s)) {
      const Segment& s = v.s;
      for (int c = 0; ok && c < s.chunks; ++c) {
        v.c = c;
        v.end = chunk_end(p, s, c, MODE == kStats);
        if (!(ok = publish(v))) break;
        if (v.end == s.j0) continue;
        const int qb = q_loads % C::Q_BUFS;
        if (!(ok = wait(&bars->q_empty[qb], ((q_loads / C::Q_BUFS) & 1) ^ 1))) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(&bars->q_full[qb], C::CH * (uint32_t)(p.tokens_at_once * p.G) * 128u);
          for (int x = 0; x < C::CH; ++x)
            tma_load_3d(smem + qb * C::Q_TILE + x * C::Q_CHUNK, &tmap_q, &bars->q_full[qb], x * 64,
                        s.h * p.G, s.b * p.T + c * p.tokens_at_once);
        }
        __syncwarp();
        ++q_loads;
        // a page a lane, or the whole tile; the next tile's block is looked up while this
        // one's slot is waited for
        struct Place {
          bool mine;
          int block, y;
        };
        auto locate = [&](int j) {
          const long long r0 = (long long)j * kKeys + lane * box;
          Place x{lane < copies && r0 < s.n, 0, 0};
          if (x.mine) {
            const int in = (int)r0 / p.page;
            x.block = p.table ? p.table[(size_t)s.b * p.max_blocks + in] : s.b;
            x.y = (int)r0 - in * p.page;
          }
          return x;
        };
        Place place = locate(s.j0);
        for (int j = s.j0; j < v.end; ++j, ++loads) {
          const int sl = loads % C::SLOTS;
          const Place next = locate(j + 1);
          const bool mine = place.mine;
          const uint32_t n_copies = __popc(__ballot_sync(0xffffffffu, mine));
          if (!(ok = wait(&bars->ring_empty[sl], ((loads / C::SLOTS) & 1) ^ 1))) break;
          if (lane == 0)
            mbar_arrive_expect_tx(&bars->ring_full[sl], n_copies * C::CH * (uint32_t)box * 128u);
          __syncwarp();
          if (mine) {
            uint8_t* dst = ring + sl * C::K_TILE + lane * box * 128;
#pragma unroll
            for (int x = 0; x < C::CH; ++x)
              tma_load_3d_once(dst + x * C::K_CHUNK, &tmap_k, &bars->ring_full[sl], x * 64, place.y,
                               place.block * p.Hkv + s.h, once);
          }
          __syncwarp();
          place = next;
        }
      }
    }
    if (ok) {
      v.last = 1;
      publish(v);
    }
    // Drain: every copy this warp issued must land before the CTA exits.
    for (int i = 0; i < C::Q_BUFS; ++i) {
      const uint32_t fills = q_loads > (uint32_t)i ? (q_loads - 1 - i) / C::Q_BUFS + 1 : 0;
      if (fills) mbar_drain<false>(&bars->q_full[i], (fills - 1) & 1, status);
    }
    for (int i = 0; i < C::SLOTS; ++i) {
      const uint32_t fills = loads > (uint32_t)i ? (loads - 1 - i) / C::SLOTS + 1 : 0;
      if (fills) mbar_drain<false>(&bars->ring_full[i], (fills - 1) & 1, status);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    const bool leader = elect_sync();
    constexpr uint32_t idesc = MODE == kStats ? idesc_f16<T>(kTcRows, kKeys, false, false)
                                              : idesc_f16<T>(kKeys, N, false, false);
    const uint64_t qdesc = sdesc_sw128(smem_u32(smem), 16, 1024);
    const uint64_t kdesc = sdesc_sw128(smem_u32(ring), 16, 1024);
    uint32_t loads = 0, taken = 0, q_cnt = 0;
    uint32_t turns = 0;  // a byte a score buffer: the parity of its next tile
    bool ok = true;
    while (ok) {
      const int isl = taken % kItemSlots;
      if (!(ok = wait(&bars->item_full[isl], (taken / kItemSlots) & 1))) break;
      const int j0 = bars->items[isl].s.j0, end = bars->items[isl].end, last = bars->items[isl].last;
      __syncwarp();
      if (leader) mbar_arrive(&bars->item_empty[isl]);
      ++taken;
      if (last) break;
      if (p.hold_ns && !(ok = __all_sync(0xffffffffu, mbar_wait<false>(&bars->never, 0, abort, status, p.hold_ns))))
        break;
      if (j0 == end) continue;
      const int qb = q_cnt % C::Q_BUFS;
      if (!(ok = wait(&bars->q_full[qb], (q_cnt / C::Q_BUFS) & 1))) break;
      ++q_cnt;
      const uint64_t qa = sdesc_advance(qdesc, qb * C::Q_TILE);
      for (int j = j0; j < end; ++j, ++loads) {
        const int sl = loads % C::SLOTS, buf = j % kGroups;
        if (!(ok = wait(&bars->ring_full[sl], (loads / C::SLOTS) & 1))) break;
        if (!(ok = wait(&bars->s_free[buf], (turns >> (8 * buf) & 1) ^ 1))) break;
        turns ^= 1u << (8 * buf);
        tc_fence_after();
        const uint64_t ka = sdesc_advance(kdesc, sl * C::K_TILE);
        if (leader) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint64_t x = sdesc_advance(qa, (kk >> 2) * C::Q_CHUNK + (kk & 3) * 32);
            const uint64_t y = sdesc_advance(ka, (kk >> 2) * C::K_CHUNK + (kk & 3) * 32);
            mma_ss(tmem + buf * C::COLS, MODE == kStats ? x : y, MODE == kStats ? y : x, idesc,
                   kk > 0 ? 1u : 0u);
          }
          mma_commit(&bars->s_full[buf]);
          mma_commit(&bars->ring_empty[sl]);
          if (j + 1 == end) mma_commit(&bars->q_empty[qb]);
        }
      }
    }
    // Drain: all issued MMAs complete before TMEM is released.
    if (leader) mma_commit(&bars->drain);
    mbar_drain<false>(&bars->drain, 0, status);
    __syncwarp();
  } else {
    // ------------------------------------------------------------ scores
    const int group = (warp - 2) >> 2, quarter = warp & 3, r = quarter * 32 + lane;
    const uint32_t t_s = tmem + ((uint32_t)(quarter * 32) << 16) + group * C::COLS;
    const float scale = p.scale, cap = p.softcap, inv_cap = CAP ? 1.0f / p.softcap : 0.0f;
    const float NEG_INF = __int_as_float(0xff800000);
    float* rows = reinterpret_cast<float*>(smem_raw + kBarBytes) + (warp - 2) * N * 2;
    const float to_base2 = scale * kLog2e;
    uint32_t tiles = 0, taken = 0;
    bool ok = true;
    while (ok) {
      const int isl = taken % kItemSlots;
      if (!(ok = wait(&bars->item_full[isl], (taken / kItemSlots) & 1))) break;
      const ItemSlot it = bars->items[isl];
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->item_empty[isl]);
      ++taken;
      if (it.last) break;
      const Segment& s = it.s;
      const int t0 = it.c * p.tokens_at_once;
      const int used = max(0, min(p.tokens_at_once, s.q - t0)) * p.G;  // query rows of the chunk
      const int row0 = t0 * p.G;
      if constexpr (MODE == kApply) {
        __syncwarp();
        for (int i = lane; i < used; i += 32) {
          const int t = t0 + i / p.G, g = i % p.G;
          float2 v;
          if (p.lse) {
            // a row that saw nothing (-inf) weighs nothing
            const float x = p.lse[((size_t)s.b * p.T + t) * p.H + s.h * p.G + g];
            v = make_float2(x == NEG_INF ? -NEG_INF : x, 1.0f);
          } else {
            v = p.row[((size_t)s.b * p.Hkv + s.h) * p.T * p.G + row0 + i];
          }
          // two columns beside each other: -m log2 e, -m' log2 e, 1 / l, 1 / l'
          float* to = rows + (i >> 1) * 4 + (i & 1);
          to[0] = -v.x * kLog2e;
          to[2] = v.y;
        }
        __syncwarp();
      }
      const int free_of_masks = used ? keys_of(s, t0) : 0;  // keys that all rows see
      // Store: running (m, l) of this key lane's scores, by column; Stats: of this row
      constexpr int ACC = MODE == kStore ? N : 1;
      float m[ACC], l[ACC];
#pragma unroll
      for (int c = 0; c < ACC; ++c) {
        m[c] = NEG_INF;
        l[c] = 0.0f;
      }
      const int my_row = t0 + r / p.G;  // Stats: the row's token
      // Each buffer's tiles are every kGroups-th of the keys: a key is always this thread's.
      for (int j = s.j0 + (group + kGroups - s.j0 % kGroups) % kGroups; j < it.end; j += kGroups, ++tiles) {
        const int k0 = j * kKeys, key = k0 + r;
        const bool all = k0 + kKeys <= free_of_masks;
        float base = 0.0f;
        const size_t at = ((size_t)s.b * p.Hkv + s.h) * p.width + key;
        if (MODE == kApply && key < s.n) {
          if (it.c > 0) base = p.weights[at];
          else if (p.previous) base = p.decay * p.previous[at];
        }
        if (!(ok = wait(&bars->s_full[group], tiles & 1))) break;
        tc_fence_after();
        if (MODE == kStats) {
          const int hi = r < used ? keys_of(s, my_row) : 0;
#pragma unroll 1
          for (int c = 0; c < kKeys; c += 32) {
            uint32_t v[32];
            tmem_ld32(t_s + c, v);
            tmem_wait_ld_of(v);
            if (r < used) {
              float x[32], top = NEG_INF;
#pragma unroll
              for (int e = 0; e < 32; ++e) {
                x[e] = natural<CAP>(__uint_as_float(v[e]), scale, cap, inv_cap);
                if (!all && k0 + c + e >= hi) x[e] = NEG_INF;
                top = fmaxf(top, x[e]);
              }
              if (top > m[0]) {
                l[0] *= ex2_approx((m[0] - top) * kLog2e);
                m[0] = top;
              }
              if (m[0] > NEG_INF) {
                float sum = 0.0f;
#pragma unroll
                for (int e = 0; e < 32; ++e) sum += ex2_approx((x[e] - m[0]) * kLog2e);
                l[0] += sum;
              }
            }
          }
        } else {
          // The rows that see this key are those from `from` on: tokens follow each other.
          const int behind = key - keys_of(s, t0);
          const int from = key >= s.n ? INT_MAX : behind < 0 ? 0 : (behind + 1) * p.G;
          // columns [c, c + W) of this thread's key, W at once
          constexpr int W = N < 32 ? 16 : 32;
          float2 acc[2] = {make_float2(base, 0.0f), make_float2(0.0f, 0.0f)};
          float* score = nullptr;
          if constexpr (MODE == kStore)
            score = p.scores + ((long long)p.start[s.b] + (long long)s.h * ((s.n + kKeys - 1) / kKeys) + j) *
                                   p.T * p.G * kKeys + r;
#pragma unroll 1
          for (int c = 0; c < used; c += W) {
            uint32_t v[W];
            if constexpr (W == 16) tmem_ld16(t_s + c, v); else tmem_ld32(t_s + c, v);
            tmem_wait(v);
            if (c + W >= used) {  // the last columns are read: the next product may go over them
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(&bars->s_free[group]);
            }
            if constexpr (MODE == kApply) {
              if (all && c + W <= used) {
#pragma unroll
                for (int e = 0; e < W; e += 2) {
                  const float4 w = *reinterpret_cast<const float4*>(rows + (c + e) * 2);
                  float2 x = make_float2(__uint_as_float(v[e]), __uint_as_float(v[e + 1]));
                  if (CAP) x = make_float2(natural<true>(x.x, scale, cap, inv_cap), natural<true>(x.y, scale, cap, inv_cap));
                  const float mul = CAP ? kLog2e : to_base2;
                  x = ffma2(x, make_float2(mul, mul), make_float2(w.x, w.y));
                  acc[(e >> 1) & 1] = ffma2(make_float2(ex2_approx(x.x), ex2_approx(x.y)), make_float2(w.z, w.w), acc[(e >> 1) & 1]);
                }
              } else {
#pragma unroll
                for (int e = 0; e < W; e += 2) {
                  const int i = c + e;
                  if (i >= used) break;
                  const float4 w = *reinterpret_cast<const float4*>(rows + i * 2);
                  float2 x = make_float2(__uint_as_float(v[e]), __uint_as_float(v[e + 1]));
                  if (CAP) x = make_float2(natural<true>(x.x, scale, cap, inv_cap), natural<true>(x.y, scale, cap, inv_cap));
                  const float mul = CAP ? kLog2e : to_base2;
                  x = ffma2(x, make_float2(mul, mul), make_float2(w.x, w.y));
                  x.x = i >= from ? ex2_approx(x.x) * w.z : 0.0f;
                  x.y = i + 1 >= from && i + 1 < used ? ex2_approx(x.y) * w.w : 0.0f;
                  acc[(e >> 1) & 1] = fadd2(acc[(e >> 1) & 1], x);
                }
              }
            } else {
#pragma unroll
              for (int e = 0; e < W; ++e) {
                if (c + e >= used) break;
                const float x = natural<CAP>(__uint_as_float(v[e]), scale, cap, inv_cap);
                const float y = c + e >= from ? x : NEG_INF;
                score[(c + e) * kKeys] = y;
                add_score(m[e], l[e], y);
              }
            }
          }
          if (MODE == kApply && key < s.n) p.weights[at] = (acc[0].x + acc[0].y) + (acc[1].x + acc[1].y);
          if (used > 0) continue;  // (the buffer is given back above)
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->s_free[group]);
      }
      if (!ok) break;
      // what this group (Stats) or warp (Store) has of each row
      float2* part = p.part + (size_t)s.slot * p.parts * p.T * p.G + row0;
      if constexpr (MODE == kStats)
        if (r < used) part[(size_t)group * p.T * p.G + r] = make_float2(m[0], l[0]);
      if constexpr (MODE == kStore) {
#pragma unroll
        for (int c = 0; c < N; ++c) {
          if (c >= used) break;
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) {
            const float m2 = __shfl_xor_sync(0xffffffffu, m[c], o), l2 = __shfl_xor_sync(0xffffffffu, l[c], o);
            join_scores(m[c], l[c], m2, l2);
          }
          if (lane == 0) part[(size_t)(warp - 2) * p.T * p.G + c] = make_float2(m[c], l[c]);
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc<C::TMEM_COLS>(tmem);
  // Whoever gave up: what the later kernels would work with is not there.
  if (threadIdx.x == 0 && *abort) atomicExch(p.hdr, 0);
}

// ---------------------------------------------------------------------------
// f32: a tile of 128 keys lies in shared memory, and 16 query rows at a time; two warps
// take the first 8 of them and two the others, a thread two keys (64 products for each
// 10 reads of 16 bytes of shared memory).  Exact f32 products.
// ---------------------------------------------------------------------------
constexpr int kRowsF32 = 16, kThreadsF32 = 128;
__host__ __device__ constexpr int f32_row(int d) { return (d + 3) / 4 * 4 + 4; }
size_t f32_smem(int d) { return sizeof(float) * (size_t)(kKeys + kRowsF32) * f32_row(d); }

// WIDE: rows lie on 16-byte boundaries.
template <int MODE, bool WIDE>
__global__ void __launch_bounds__(kThreadsF32) pva_weights_f32_kernel(WeightsParams p) {
  extern __shared__ float smem[];
  __shared__ Segment s_segment;
  __shared__ int s_more;
  __shared__ float2 s_rows[kRowsF32];
  __shared__ int s_hi[kRowsF32];
  __shared__ float2 s_half[2][kRowsF32 / 2][2];  // Stats: a row's (m, l) of its two warps
  __shared__ float s_sum[2][64];                 // Apply: the upper rows' part of the keys' weights
  allow_next_grid();
  wait_prior_grid();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, d = p.d, row = f32_row(d);
  const int group = tid >> 6, key0 = tid & 63;  // of the rows; keys key0 and key0 + 64
  const float NEG_INF = __int_as_float(0xff800000);
  float* sk = smem;
  float* sq = smem + (size_t)kKeys * row;
  const float* kc = static_cast<const float*>(p.k_cache);
  const float* q = static_cast<const float*>(p.q);
  for (int i = tid; i < (kKeys + kRowsF32) * (row - d); i += kThreadsF32)
    smem[(size_t)(i / (row - d)) * row + d + i % (row - d)] = 0.0f;
  Walk walk(p, blockIdx.x, p.hdr[0] ? p.hdr[1] : 0, p.hdr[2]);  // the first warp's counts
  while (true) {
    __syncthreads();
    if (warp == 0) {
      Segment s;
      const bool more = walk.next(p, s);
      if (lane == 0) {
        s_more = more;
        s_segment = s;
      }
    }
    __syncthreads();
    if (!s_more) break;
    const Segment s = s_segment;
    const int all_rows = s.q * p.G;
    auto copy_row = [&](float* dst, const float* src, bool there) {  // a warp
      if (WIDE) {
        for (int c = 4 * lane; c < d; c += 128)
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst + c)), "l"(src + (there ? c : 0)),
                       "r"(there ? 16 : 0)
                       : "memory");
      } else {
        for (int c = lane; c < d; c += 32) dst[c] = there ? src[c] : 0.0f;
      }
    };
    auto load_keys = [&](int j) {  // a warp 32 of them, whose places its lanes look up side by side
      static_assert(kKeys == kThreadsF32, "a key a lane");
      const int key = j * kKeys + tid;
      long long at = -1;
      if (key < s.n) {
        const int in = key / p.page;
        const int block = p.table ? p.table[(size_t)s.b * p.max_blocks + in] : s.b;
        at = (((long long)block * p.Hkv + s.h) * p.page + (key - in * p.page)) * d;
      }
      for (int i = 0; i < 32; ++i) {
        const long long from = __shfl_sync(0xffffffffu, at, i);
        copy_row(sk + (size_t)(warp * 32 + i) * row, kc + (from < 0 ? 0 : from), from >= 0);
      }
    };
    auto load_rows = [&](int r0) {
      for (int i = warp; i < kRowsF32; i += kThreadsF32 / 32) {
        const int r = r0 + i, t = r / p.G, g = r - t * p.G;
        const bool there = r < all_rows;
        copy_row(sq + (size_t)i * row, there ? q + (((size_t)s.b * p.T + t) * p.H + s.h * p.G + g) * d : q, there);
      }
      if (tid < kRowsF32) {
        const int r = r0 + tid, t = r / p.G, g = r - t * p.G;
        const bool there = r < all_rows;
        s_hi[tid] = there ? keys_of(s, t) : 0;
        if (MODE == kApply && there) {
          if (p.lse) {
            const float x = p.lse[((size_t)s.b * p.T + t) * p.H + s.h * p.G + g];
            s_rows[tid] = make_float2(x == NEG_INF ? -NEG_INF : x, 1.0f);
          } else {
            s_rows[tid] = p.row[((size_t)s.b * p.Hkv + s.h) * p.T * p.G + r];
          }
        }
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
    };
    auto scores = [&](float (&x)[2][8]) {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[0][e] = x[1][e] = 0.0f;
      const float* qa = sq + (size_t)group * 8 * row;
#pragma unroll 2
      for (int c = 0; c < d; c += 4) {
        const float4 k0 = *reinterpret_cast<const float4*>(sk + (size_t)key0 * row + c);
        const float4 k1 = *reinterpret_cast<const float4*>(sk + (size_t)(key0 + 64) * row + c);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float4 v = *reinterpret_cast<const float4*>(qa + (size_t)e * row + c);
          x[0][e] = fmaf(k0.w, v.w, fmaf(k0.z, v.z, fmaf(k0.y, v.y, fmaf(k0.x, v.x, x[0][e]))));
          x[1][e] = fmaf(k1.w, v.w, fmaf(k1.z, v.z, fmaf(k1.y, v.y, fmaf(k1.x, v.x, x[1][e]))));
        }
      }
#pragma unroll
      for (int y = 0; y < 2; ++y)
#pragma unroll
        for (int e = 0; e < 8; ++e)
          x[y][e] = p.softcap != 0.0f ? natural<true>(x[y][e], p.scale, p.softcap, 1.0f / p.softcap)
                                      : natural<false>(x[y][e], p.scale, 0.0f, 0.0f);
    };
    for (int j = s.j0; j < s.j1; ++j) {
      __syncthreads();
      load_keys(j);
      const int key = j * kKeys + key0;
      const size_t at = ((size_t)s.b * p.Hkv + s.h) * p.width + key;
      float sum[2] = {0.0f, 0.0f};
      if (MODE == kApply && p.previous && group == 0)
#pragma unroll
        for (int y = 0; y < 2; ++y)
          if (key + 64 * y < s.n) sum[y] = p.decay * p.previous[at + 64 * y];
      if (all_rows == 0) asm volatile("cp.async.wait_all;" ::: "memory");
      for (int r0 = 0; r0 < all_rows; r0 += kRowsF32) {
        if (r0) __syncthreads();
        load_rows(r0);
        __syncthreads();
        const bool mine = r0 + group * 8 < all_rows;  // uniform in a warp
        float x[2][8];
        if (mine) scores(x);
        if (MODE == kApply) {
          if (!mine) continue;
#pragma unroll
          for (int e = 0; e < 8; ++e)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const float2 w = s_rows[group * 8 + e];
              if (key + 64 * y < s_hi[group * 8 + e]) sum[y] = fmaf(exp2f((x[y][e] - w.x) * kLog2e), w.y, sum[y]);
            }
          continue;
        }
        if (mine) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int hi = s_hi[group * 8 + e];
            const float a = key < hi ? x[0][e] : NEG_INF, b = key + 64 < hi ? x[1][e] : NEG_INF;
            float m = fmaxf(a, b);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            const float top = m == NEG_INF ? 0.0f : m;
            float l = exp2f((a - top) * kLog2e) + exp2f((b - top) * kLog2e);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
            if (lane == 0) s_half[group][e][warp & 1] = make_float2(m, l);
          }
        }
        __syncthreads();
        if (tid < kRowsF32 && r0 + tid < all_rows) {  // a row's sums are this thread's throughout
          float2* part = p.part + (size_t)s.slot * p.T * p.G + r0 + tid;
          float2 v = s_half[tid >> 3][tid & 7][0];
          const float2 o = s_half[tid >> 3][tid & 7][1];
          join_scores(v.x, v.y, o.x, o.y);
          if (j > s.j0) join_scores(v.x, v.y, part->x, part->y);
          *part = v;
        }
      }
      if (MODE == kApply) {
        if (group == 1) {
          s_sum[0][key0] = sum[0];
          s_sum[1][key0] = sum[1];
        }
        __syncthreads();
        if (group == 0)
#pragma unroll
          for (int y = 0; y < 2; ++y)
            if (key + 64 * y < s.n) p.weights[at + 64 * y] = sum[y] + s_sum[y][key0];
      }
    }
  }
}

// (m, 1 / l) of every query row from its pieces', in the order of the line: a warp a row.
__global__ void __launch_bounds__(256) pva_weights_rows_kernel(WeightsParams p) {
  allow_next_grid();
  wait_prior_grid();
  if (!p.hdr[0]) return;
  const int lane = threadIdx.x & 31, R = p.T * p.G;
  const long long chunk = p.hdr[2], rows = (long long)p.B * p.Hkv * R;
  const float NEG_INF = __int_as_float(0xff800000);
  for (long long i = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); i < rows; i += (long long)gridDim.x * 8) {
    const int item = (int)(i / R), r = (int)(i - (long long)item * R), b = item / p.Hkv, h = item - b * p.Hkv;
    const Sequence s(p, b);
    if (r >= s.q * p.G) continue;
    const long long x0 = p.start[b] + h * s.per_head(), x1 = x0 + s.per_head();
    float m = NEG_INF, l = 0.0f;
    for (long long pc = x0 / chunk + lane; pc * chunk < x1; pc += 32) {
      // a piece that holds no tile's first place has no part
      const long long from = pc * chunk > x0 ? pc * chunk - x0 : 0, to = (pc + 1) * chunk < x1 ? (pc + 1) * chunk - x0 : x1 - x0;
      if (first_tile((int)from, s.chunks) >= first_tile((int)to, s.chunks)) continue;
      for (int i = 0; i < p.parts; ++i) {
        const float2 v = p.part[((size_t)(item + pc) * p.parts + i) * R + r];
        join_scores(m, l, v.x, v.y);
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float m2 = __shfl_xor_sync(0xffffffffu, m, o), l2 = __shfl_xor_sync(0xffffffffu, l, o);
      join_scores(m, l, m2, l2);
    }
    // a row that saw nothing weighs nothing
    if (lane == 0) p.row[i] = l == 0.0f ? make_float2(-NEG_INF, 0.0f) : make_float2(m, 1.0f / l);
  }
}

// Weights from kept scores: a warp a run of key tiles, a lane every 32nd key of a tile.
// The rows' maxima and sums are joined from the pieces' by the warp itself, anew for
// each (sequence, kv head) of its run, eight lanes a row at a time.
constexpr int kScoreWarps = 4, kStoreRows = 16;
__global__ void __launch_bounds__(32 * kScoreWarps) pva_weights_scores_kernel(WeightsParams p) {
  allow_next_grid();
  __shared__ float2 s_rows[kScoreWarps][kStoreRows];
  // The kernel before this one let it start when all work before the scores was done:
  // only the scores and the rows' sums have to be waited for.
  const int places = p.hdr[1], lane = threadIdx.x & 31, warp = threadIdx.x >> 5, R = p.T * p.G;
  const int warps = gridDim.x * kScoreWarps, run = (places + warps - 1) / warps, chunk = p.hdr[2];
  int x = (blockIdx.x * kScoreWarps + warp) * run;
  const int end = min(x + run, places);
  const float NEG_INF = __int_as_float(0xff800000);
  float2* rows = s_rows[warp];
  int last_item = -1, b = x < end ? tree_find(p.start, p.B, x) : 0, h = 0, k0 = 0, n = 0, used = 0, tiles = 0;
  float sum[4];
  auto look_up = [&](int tile) {
    while (p.start[b + 1] <= tile) ++b;
    const Sequence s(p, b);
    const int rel = tile - p.start[b];
    tiles = s.tiles;
    h = rel / tiles;
    k0 = (rel - h * tiles) * kKeys;
    n = s.n;
    used = s.q * p.G;
    const float* old = p.previous + (size_t)(b * p.Hkv + h) * p.width + k0 + lane;
#pragma unroll
    for (int k = 0; k < 4; ++k) sum[k] = p.previous && k0 + lane + 32 * k < n ? p.decay * old[32 * k] : 0.0f;
  };
  if (x < end) look_up(x);
  wait_prior_grid();
  if (!*(volatile int32_t*)p.hdr) return;  // (or given up)
  for (; x < end; ++x) {
    const int item = b * p.Hkv + h;
    const float* score = p.scores + (long long)x * R * kKeys + lane;
    if (item != last_item) {
      const int first = (p.start[b] + h * tiles) / chunk, pieces = (p.start[b] + (h + 1) * tiles - 1) / chunk - first + 1;
      __syncwarp();
      for (int r0 = 0; r0 < used; r0 += 4) {
        const int r = r0 + lane / 8;
        float m = NEG_INF, l = 0.0f;
        if (r < used)
          for (int i = lane % 8; i < pieces * p.parts; i += 8) {
            const float2 v = p.part[((size_t)(item + first) * p.parts + i) * R + r];
            join_scores(m, l, v.x, v.y);
          }
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) {
          const float m2 = __shfl_xor_sync(0xffffffffu, m, o), l2 = __shfl_xor_sync(0xffffffffu, l, o);
          join_scores(m, l, m2, l2);
        }
        // a row that saw nothing weighs nothing
        if (r < used && lane % 8 == 0) rows[r] = l == 0.0f ? make_float2(-NEG_INF, 0.0f) : make_float2(m, 1.0f / l);
      }
      __syncwarp();
      last_item = item;
    }
#pragma unroll 4
    for (int r = 0; r < used; ++r) {
      const float2 w = rows[r];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        sum[k] = fmaf(ex2_approx((score[r * kKeys + 32 * k] - w.x) * kLog2e), w.y, sum[k]);
    }
    float* to = p.weights + (size_t)item * p.width + k0 + lane;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (k0 + lane + 32 * k < n) to[32 * k] = sum[k];
    if (x + 1 < end) look_up(x + 1);
  }
}

template <typename T, int D, int N, int MODE>
cudaError_t launch_mode(const WeightsParams& p, const CUtensorMap& tq, const CUtensorMap& tk, cudaStream_t s) {
  constexpr int smem = WCfg<D, N, MODE>::SMEM;
  auto kern = p.softcap != 0.0f ? pva_weights_tc_kernel<T, D, N, MODE, true> : pva_weights_tc_kernel<T, D, N, MODE, false>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  return launch_dependent(kern, dim3(p.pieces), dim3(kTcThreads), smem, s, p, tq, tk);
}

template <typename T, int D>
cudaError_t launch_d(const WeightsParams& p, int mode, int n, const CUtensorMap& tq, const CUtensorMap& tk, cudaStream_t s) {
  if (mode == kStore) return launch_mode<T, D, 16, kStore>(p, tq, tk, s);
  if (mode == kStats) return launch_mode<T, D, kTcRows, kStats>(p, tq, tk, s);
  return n == 16   ? launch_mode<T, D, 16, kApply>(p, tq, tk, s)
         : n == 32 ? launch_mode<T, D, 32, kApply>(p, tq, tk, s)
         : n == 64 ? launch_mode<T, D, 64, kApply>(p, tq, tk, s)
                   : launch_mode<T, D, 128, kApply>(p, tq, tk, s);
}

template <typename T>
cudaError_t launch_type(const WeightsParams& p, int mode, int n, const CUtensorMap& tq, const CUtensorMap& tk, cudaStream_t s) {
  switch (p.d) {
    case 64: return launch_d<T, 64>(p, mode, n, tq, tk, s);
    case 96: return launch_d<T, 96>(p, mode, n, tq, tk, s);
    case 128: return launch_d<T, 128>(p, mode, n, tq, tk, s);
    case 192: return launch_d<T, 192>(p, mode, n, tq, tk, s);
    case 256: return launch_d<T, 256>(p, mode, n, tq, tk, s);
    default: return cudaErrorInvalidValue;
  }
}

template <int MODE>
cudaError_t launch_f32(const WeightsParams& p, cudaStream_t s) {
  const size_t smem = f32_smem(p.d);
  const bool wide = p.d % 4 == 0 && (((uintptr_t)p.q | (uintptr_t)p.k_cache) & 15) == 0;
  auto kern = wide ? pva_weights_f32_kernel<MODE, true> : pva_weights_f32_kernel<MODE, false>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  return launch_dependent(kern, dim3(p.pieces), dim3(kThreadsF32), smem, s, p);
}

int weights(const void* q, const void* k_cache, const int32_t* lens, const int32_t* q_lens, const int32_t* table,
            const float* previous, const float* lse, float* out, int B, int T, int n_blocks, int page, int max_blocks, int H,
            int Hkv, int d, int width, float decay, float scale, float softcap, int dtype, cudaStream_t stream) {
  if (!q || !k_cache || !lens || !out) return fail(PVA_ERR_INVALID_ARG, "null q, k_cache, lens or weights pointer");
  if (B < 1 || T < 1 || n_blocks < 1 || page < 1 || width < 1)
    return fail(PVA_ERR_INVALID_ARG, "need B >= 1, tokens >= 1, n_blocks >= 1, page_size >= 1, width >= 1");
  if (H < 1 || Hkv < 1 || H % Hkv != 0)
    return fail(PVA_ERR_INVALID_ARG, "num_heads must be a positive multiple of a positive kv_num_heads");
  if (dtype != PVA_F32 && dtype != PVA_F16 && dtype != PVA_BF16)
    return fail(PVA_ERR_INVALID_ARG, "dtype must be 0 (f32), 1 (f16) or 2 (bf16)");
  if (!isfinite(scale) || !isfinite(softcap) || !isfinite(decay))
    return fail(PVA_ERR_INVALID_ARG, "scale, softcap and decay must be finite");
  const bool tc = dtype != PVA_F32;
  if (tc ? d != 64 && d != 96 && d != 128 && d != 192 && d != 256 : d < 2 || d > 256 || d % 2 != 0)
    return fail(PVA_ERR_UNSUPPORTED,
                "head_size must be 64, 96, 128, 192 or 256 (f16/bf16), or even and at most 256 (f32)");
  const int G = H / Hkv;
  if (G > 128) return fail(PVA_ERR_UNSUPPORTED, "num_heads / kv_num_heads must be at most 128");
  if (table) {
    if (max_blocks < 1) return fail(PVA_ERR_INVALID_ARG, "max_blocks must be >= 1");
    if (page < 16 || (page & (page - 1)) != 0)
      return fail(PVA_ERR_UNSUPPORTED, "page_size must be a power of two of at least 16");
  } else {
    if (n_blocks != B)
      return fail(PVA_ERR_INVALID_ARG, "without a block table the cache has one block a sequence");
    max_blocks = 1;
  }
  if ((long long)B * T > INT_MAX - 65536 || (long long)T * G > INT_MAX / 2 ||
      (long long)max_blocks * page > INT_MAX - 65536 || (long long)n_blocks * Hkv > INT_MAX ||
      (long long)B * Hkv > INT_MAX - 65536 || width > INT_MAX - 65536)
    return fail(PVA_ERR_INVALID_ARG, "cache or token extents do not fit in int32");
  const size_t size = tc ? 2 : 4;
  const uintptr_t mis = (uintptr_t)q | (uintptr_t)k_cache;
  if (tc && (mis & 15)) return fail(PVA_ERR_INVALID_ARG, "q and k_cache must be 16-byte aligned");
  if (mis % size || ((uintptr_t)out | (uintptr_t)previous | (uintptr_t)lse) & 3)
    return fail(PVA_ERR_INVALID_ARG, "a tensor is not aligned to its elements");
  auto meets = [](const void* a, size_t na, const void* b, size_t nb) {
    const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
    return a && b && x < y + nb && y < x + na;
  };
  const size_t all = 4 * (size_t)B * Hkv * width;
  if ((previous != out && meets(out, all, previous, all)) || meets(out, all, lse, 4 * (size_t)B * T * H) ||
      meets(out, all, lens, 4 * (size_t)B) || meets(out, all, q_lens, 4 * (size_t)B) ||
      meets(out, all, table, 4 * (size_t)B * max_blocks) || meets(out, all, q, size * B * T * H * d) ||
      meets(out, all, k_cache, size * n_blocks * Hkv * page * d))
    return fail(PVA_ERR_INVALID_ARG, "weights overlap an input (previous may be weights)");

  WeightsParams p{};
  p.q = q;
  p.k_cache = k_cache;
  p.lens = lens;
  p.q_lens = q_lens;
  p.table = table;
  p.previous = previous;
  p.lse = lse;
  p.weights = out;
  p.decay = decay;
  p.scale = scale != 0.0f ? scale : 1.0f / sqrtf((float)d);
  p.softcap = softcap_size(softcap, p.scale);
  p.B = B;
  p.T = T;
  p.H = H;
  p.Hkv = Hkv;
  p.G = G;
  p.d = d;
  p.width = width;
  p.page = page;
  p.max_blocks = max_blocks;
  p.n_blocks = n_blocks;
  const long long R = (long long)T * G;
  // query rows of a chunk, and the score columns they take
  const int n = R <= 16 ? 16 : R <= 32 ? 32 : R <= 64 ? 64 : 128;
  p.tokens_at_once = tc ? (R <= 128 ? T : 128 / G) : T;
  // Scores are kept where there are few rows, and in no more memory than the keys have
  // or 256 MB (tables may be far wider than the pool), if there is as much.  Kept and read
  // twice, us, for 4, 8 and 16 query rows of 8 kv heads of 128 bf16: 32 sequences of 2000
  // to 16,000 rows 131, 147, 191 and 231; one of 100,000 rows 68, 83, 139 and 95; two of
  // 300 and 700 rows 21, -, 35 and 21.
  const size_t tiles = ((size_t)(width < (long long)max_blocks * page ? width : (long long)max_blocks * page) + kKeys - 1) / kKeys;
  const size_t kept = 4 * (size_t)B * Hkv * tiles * R * kKeys, pool = 2 * (size_t)n_blocks * Hkv * page * d;
  bool store = tc && !lse && R <= 16 && kept <= (pool > (256u << 20) ? pool : 256u << 20);

  std::lock_guard<std::mutex> lock(api_mutex());
  int rc = sm_count(&p.pieces);
  if (rc != PVA_OK) return rc;
  if (!tc) p.pieces *= (int)((228 * 1024) / (f32_smem(d) + 3 * 1024));  // CTAs an SM holds
  size_t at_hdr, at_start, at_part, at_row, at_scores;
  auto lay_out = [&]() {
    size_t used = 0;
    auto take = [&](size_t bytes) {
      const size_t at = used;
      used += (bytes + 255) / 256 * 256;
      return at;
    };
    at_hdr = take(32), at_start = take(4 * ((size_t)B + 1));
    p.parts = !tc ? 1 : store ? 4 * kGroups : kGroups;
    at_part = take(lse ? 0 : 8 * ((size_t)B * Hkv + p.pieces) * p.parts * R);
    at_row = take(lse ? 0 : 8 * (size_t)B * Hkv * R);
    at_scores = take(store ? kept : 0);
    return used;
  };
  const size_t most = lay_out();
  CallContext c;
  if (store) {
    store = false;
    const size_t least = lay_out();
    if ((rc = acquire_most(stream, most, least, &c, &store)) != PVA_OK) return rc;
    lay_out();
  } else if ((rc = acquire(stream, most, &c)) != PVA_OK) {
    return rc;
  }
  p.status = c.status;
  p.hdr = reinterpret_cast<int32_t*>(c.buf + at_hdr);
  p.start = reinterpret_cast<int32_t*>(c.buf + at_start);
  p.part = reinterpret_cast<float2*>(c.buf + at_part);
  p.row = reinterpret_cast<float2*>(c.buf + at_row);
  p.scores = reinterpret_cast<float*>(c.buf + at_scores);
  CUtensorMap tq, tk;
  if (tc) {
    const int box = table && page < kKeys ? page : kKeys;
    if ((rc = get_encoder()) != PVA_OK ||
        (rc = encode_rows_map(&tq, q, dtype, d, H, (long long)B * T, G, p.tokens_at_once)) != PVA_OK ||
        (rc = encode_plane_map(&tk, k_cache, dtype, d, page, (long long)n_blocks * Hkv, 64, box, true)) != PVA_OK)
      return rc;
  }
  cudaError_t e = line::launch_front(WeightsFront{p}, B, max_blocks, c.status, stream);
  if (e != cudaSuccess) return cuda_fail(e, "weights front-end launch");
  p.hold_ns = selftest_hold_ns();
  auto pass = [&](int mode) {
    if (!tc) return mode == kApply ? launch_f32<kApply>(p, stream) : launch_f32<kStats>(p, stream);
    return dtype == PVA_BF16 ? launch_type<__nv_bfloat16>(p, mode, n, tq, tk, stream)
                             : launch_type<__half>(p, mode, n, tq, tk, stream);
  };
  if (!lse) {
    if ((e = pass(store ? kStore : kStats)) != cudaSuccess) return cuda_fail(e, "row sums launch");
    p.hold_ns = 0;
  }
  if (!lse && !store) {
    const long long want = ((long long)B * Hkv * R + 7) / 8;
    e = launch_dependent(pva_weights_rows_kernel, dim3((unsigned)(want < 4096 ? want : 4096)), dim3(256), 0, stream, p);
    if (e != cudaSuccess) return cuda_fail(e, "row sums launch");
  }
  e = store ? launch_dependent(pva_weights_scores_kernel, dim3(c.num_sms * 16), dim3(32 * kScoreWarps), 0, stream, p) : pass(kApply);
  return e == cudaSuccess ? PVA_OK : cuda_fail(e, "weights launch");
}

}  // namespace
}  // namespace pva

extern "C" int pva_kvcache_weights(const void* q, const void* k_cache, const int32_t* lens, const int32_t* q_lens,
                                   const int32_t* block_table, const float* previous, const float* lse, float* weights_out,
                                   int B, int tokens, int n_blocks, int page_size, int max_blocks, int num_heads,
                                   int kv_num_heads, int head_size, int width, float decay, float scale, float softcap,
                                   int dtype, void* stream) {
  return guarded([&]() -> int {
    return weights(q, k_cache, lens, q_lens, block_table, previous, lse, weights_out, B, tokens, n_blocks, page_size, max_blocks,
                   num_heads, kv_num_heads, head_size, width, decay, scale, softcap, dtype,
                   static_cast<cudaStream_t>(stream));
  });
}
