// Tree attention over a KV cache on the tensor cores for steps with more than
// 128 query rows per kv head (drafts of many nodes, prompt chunks): two 128-row
// query tiles per CTA share every key tile, f16/bf16, head sizes up to 192 (128
// where the step rotates its queries).
//
// Two tiles halve the cache traffic per row, and give the tensor cores and the
// softmax something to do at the same time: while one warpgroup exponentiates
// its tile's scores, the MMAs of the other run.  Items are 256 rows; the line
// of key tiles, its pieces, slots and the join are those of pva_tree.h.
//
// Per CTA (320 threads):
//   warp 0      TMA producer: the two Q tiles of a segment (shared memory, held
//               for the segment), then K_j and V_j through a ring of slots.
//   warp 1      MMA issuer and TMEM owner.  Per key tile and query tile x:
//               PV_x(j) as soon as P_x(j) is there, then S_x(j+1), which reuses
//               the score columns that P_x(j) was read from (MMAs of one thread
//               run in issue order).
//   warps 2..5, 6..9   softmax and epilogue of tile 0 and 1, a thread per row.
// TMEM: S_x at [x BN, (x+1) BN), O_x at 2 BN + x D: all 512 columns at D = 128
// and D = 192.
//
// Rotated queries come in two parts, as in the one-tile kernel.  Here the second
// part costs more: at d = 128 half as many MMA steps again in a kernel that they
// bound, and a ring slot (2048-token chunks of 8 sequences: 1.51 against 1.13 ms;
// 61 nodes on 4 sequences of 100,000 rows and more: 0.49 against 0.36 ms), for
// one rounding less of three equal ones (bf16 results off by 0.0023 of their size in
// the mean square against 0.0029, 0.0017 being their own rounding).
// Queries that the caller rotated are taken as they are, at the smaller figures.
//
// The compiler gives 320 threads 168 registers each.  Up to D = 128, where a thread
// has the 128 scores of its row in registers, it spills 60 bytes (with a softcap 88 to
// 100); two threads a row are slower all the same (1.35 against 1.10 ms on the chunks
// above, queries rotated before).
#include "pva_tree_tile.cuh"

namespace pva {
namespace {

using namespace tile;

constexpr int kThreads = 320;
constexpr int kItemSlots = 4;
constexpr int kGroupWarps = 4;

template <int D, int PARTS>
struct PairCfg {
  static constexpr int BN = tree_keys(D);
  static constexpr int CH = (D + 63) / 64;
  static constexpr int Q_CHUNK = kTcRows * 128;
  static constexpr int Q_TILE = CH * Q_CHUNK;     // one query tile
  static constexpr int KV_CHUNK = BN * 128;
  static constexpr int KV_TILE = CH * KV_CHUNK;
  static constexpr int OFF_RING = 2 * PARTS * Q_TILE;
  static constexpr int SLOTS_FIT = (232448 - kHeadBytes - OFF_RING) / KV_TILE;
  static constexpr int SLOTS = SLOTS_FIT < 16 ? SLOTS_FIT : 16;
  static_assert(SLOTS >= 3, "V_j, K_j+1 and a slot on its way");
  static constexpr int SMEM = kHeadBytes + OFF_RING + SLOTS * KV_TILE;
  static constexpr int TMEM_COLS = 512;
  static constexpr int COL_S = 0;
  static constexpr int COL_O = 2 * BN;
  static_assert(COL_O + 2 * D <= TMEM_COLS, "TMEM budget");
  static_assert(SMEM <= 232448, "shared memory budget");
};

struct ItemSlot {
  TreeSegment s;
  int last;
};

struct Bars {
  uint64_t q_full, q_empty, drain;
  uint64_t s_full[2], p_full[2], o_ready[2], o_done[2], o_free[2];
  uint64_t ring_full[16], ring_empty[16];
  uint64_t item_full[kItemSlots], item_empty[kItemSlots];
  ItemSlot items[kItemSlots];
  uint32_t tmem_base;
  int abort;
};
static_assert(sizeof(Bars) <= kHeadBytes, "barriers and segments");

// Whether the item's second tile has rows.
__device__ __forceinline__ bool has_second(const TreeParams& p, const TreeSegment& s) {
  return s.n * p.G - s.t * p.rows > kTcRows;
}

template <typename T, int D, int PARTS, int CAP>
__global__ void __launch_bounds__(kThreads, 1)
    pva_tree_pair_kernel(TreeParams p, const __grid_constant__ CUtensorMap tmap_q,
                         const __grid_constant__ CUtensorMap tmap_k,
                         const __grid_constant__ CUtensorMap tmap_v) {
  using C = PairCfg<D, PARTS>;
  constexpr int BN = C::BN;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  if (misplaced(smem_raw, p)) return;
  Bars* bars = reinterpret_cast<Bars*>(smem_raw);
  uint8_t* smem = smem_raw + kHeadBytes;
  uint8_t* ring = smem + C::OFF_RING;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t* status = p.status;
  volatile int* abort = &bars->abort;

  if (threadIdx.x == 0) {
    bars->abort = 0;
    mbar_init(&bars->q_full, 1);
    mbar_init(&bars->q_empty, 1);
    mbar_init(&bars->drain, 1);
    for (int x = 0; x < 2; ++x) {
      mbar_init(&bars->s_full[x], 1);
      mbar_init(&bars->p_full[x], kGroupWarps);
      mbar_init(&bars->o_ready[x], 1);
      mbar_init(&bars->o_done[x], 1);
      mbar_init(&bars->o_free[x], kGroupWarps);
    }
    for (int s = 0; s < C::SLOTS; ++s) {
      mbar_init(&bars->ring_full[s], 1);
      mbar_init(&bars->ring_empty[s], 1);
    }
    for (int s = 0; s < kItemSlots; ++s) {
      mbar_init(&bars->item_full[s], 1);
      mbar_init(&bars->item_empty[s], 1 + 2 * kGroupWarps);
    }
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc<C::TMEM_COLS>(&bars->tmem_base);
  if (warp == 0 && lane == 0) {
    prefetch_tensor_map(&tmap_q);
    prefetch_tensor_map(&tmap_k);
    prefetch_tensor_map(&tmap_v);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  allow_next_grid();
  wait_prior_grid();

  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    return __all_sync(0xffffffffu, mbar_wait<false>(bar, parity, abort, status));
  };

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    TreeWalk walk(p, blockIdx.x);
    const TileCopies tc(p, BN);
    uint32_t loads = 0, published = 0;
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
    uint32_t q_loads = 0;
    ItemSlot v;
    v.last = 0;
    while (ok && walk.next(p, v.s)) {
      if (!(ok = publish(v))) break;
      const TreeSegment& s = v.s;
      // the Q tiles, once the S MMAs of the segment before are done with them
      if (!(ok = wait(&bars->q_empty, (q_loads & 1) ^ 1))) break;
      if (lane == 0) {
        const int n_q = has_second(p, s) ? 2 : 1;
        mbar_arrive_expect_tx(&bars->q_full, (uint32_t)(n_q * PARTS * C::Q_TILE));
        for (int part = 0; part < PARTS; ++part)
          for (int y = 0; y < n_q; ++y)
            for (int c = 0; c < C::CH; ++c)
              tma_load_3d(smem + (2 * part + y) * C::Q_TILE + c * C::Q_CHUNK, &tmap_q, &bars->q_full,
                          c * 64, s.t * p.rows + y * kTcRows, (part * p.B + s.b) * p.Hkv + s.h);
      }
      __syncwarp();
      ++q_loads;
      // the block of the next tile's copy is looked up while this tile's slots
      // are waited for
      TileCopy copy = tc.locate(p, s, BN, s.j0, lane);
      for (int j = s.j0; ok && j < s.j0 + s.count; ++j) {
        const TileCopy next = tc.locate(p, s, BN, j + 1, lane);
        const uint32_t n_copies = __popc(__ballot_sync(0xffffffffu, copy.mine));
#pragma unroll
        for (int kv = 0; kv < 2; ++kv, ++loads) {
          const int sl = loads % C::SLOTS;
          if (!(ok = wait(&bars->ring_empty[sl], ((loads / C::SLOTS) & 1) ^ 1))) break;
          if (lane == 0)
            mbar_arrive_expect_tx(&bars->ring_full[sl], n_copies * C::CH * (uint32_t)tc.box * 128u);
          __syncwarp();
          if (copy.mine) {
            uint8_t* dst = ring + sl * C::KV_TILE + lane * tc.box * 128;
#pragma unroll
            for (int c = 0; c < C::CH; ++c)
              tma_load_3d(dst + c * C::KV_CHUNK, kv ? &tmap_v : &tmap_k, &bars->ring_full[sl],
                          c * 64, copy.y, copy.plane(p, s));
          }
          __syncwarp();
        }
        copy = next;
      }
    }
    if (ok) {
      v.last = 1;
      publish(v);
    } else if (lane == 0) {
      tree_note_cut(p, blockIdx.x, nullptr);  // nothing to join
    }
    // Drain: every copy this warp issued must land before the CTA exits.
    if (q_loads) mbar_wait<false>(&bars->q_full, (q_loads - 1) & 1, abort, status);
    for (int s = 0; s < C::SLOTS; ++s) {
      const uint32_t fills = loads > (uint32_t)s ? (loads - 1 - s) / C::SLOTS + 1 : 0;
      if (fills) mbar_wait<false>(&bars->ring_full[s], (fills - 1) & 1, abort, status);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    const bool leader = elect_sync();
    constexpr uint32_t idesc_s = idesc_f16<T>(kTcRows, BN, false, false);
    constexpr uint32_t idesc_o = idesc_f16<T>(kTcRows, D, false, true);
    const uint64_t qdesc = sdesc_sw128(smem_u32(smem), 16, 1024);
    const uint64_t kdesc = sdesc_sw128(smem_u32(ring), 16, 1024);
    const uint64_t vdesc = sdesc_sw128(smem_u32(ring), C::KV_CHUNK, 1024);
    uint32_t loads = 0, items = 0;
    uint32_t done[2] = {0, 0};     // key tiles issued per query tile
    uint32_t o_items[2] = {0, 0};  // segments per query tile
    bool ok = true;
    auto wait_slot = [&](uint32_t L) -> bool {
      const bool r = wait(&bars->ring_full[L % C::SLOTS], (L / C::SLOTS) & 1);
      tc_fence_after();
      return r;
    };
    auto issue_s = [&](int x, uint32_t L) {
      const uint64_t qa = sdesc_advance(qdesc, x * C::Q_TILE);
      const uint64_t ka = sdesc_advance(kdesc, (L % C::SLOTS) * C::KV_TILE);
      if (leader) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          mma_ss(tmem + C::COL_S + x * BN, sdesc_advance(qa, (kk >> 2) * C::Q_CHUNK + (kk & 3) * 32),
                 sdesc_advance(ka, (kk >> 2) * C::KV_CHUNK + (kk & 3) * 32), idesc_s,
                 kk > 0 ? 1u : 0u);
        if (PARTS == 2) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            mma_ss(tmem + C::COL_S + x * BN,
                   sdesc_advance(qa, 2 * C::Q_TILE + (kk >> 2) * C::Q_CHUNK + (kk & 3) * 32),
                   sdesc_advance(ka, (kk >> 2) * C::KV_CHUNK + (kk & 3) * 32), idesc_s, 1u);
        }
        mma_commit(&bars->s_full[x]);
      }
    };
    while (ok) {
      const int isl = items % kItemSlots;
      if (!(ok = wait(&bars->item_full[isl], (items / kItemSlots) & 1))) break;
      const TreeSegment s = bars->items[isl].s;
      const int last = bars->items[isl].last;
      __syncwarp();
      if (leader) mbar_arrive(&bars->item_empty[isl]);
      if (last) break;
      const int n = s.count, n_q = has_second(p, s) ? 2 : 1;
      if (!(ok = wait(&bars->q_full, items & 1))) break;
      ++items;
      if (!(ok = wait_slot(loads))) break;
      for (int x = 0; x < n_q; ++x) issue_s(x, loads);
      if (leader) {
        mma_commit(&bars->ring_empty[loads % C::SLOTS]);
        if (n == 1) mma_commit(&bars->q_empty);
      }
      for (int j = 0; ok && j < n; ++j) {
        const uint32_t Lv = loads + 2 * j + 1, Lk = Lv + 1;
        if (!(ok = wait_slot(Lv))) break;
        const uint64_t va = sdesc_advance(vdesc, (Lv % C::SLOTS) * C::KV_TILE);
        for (int x = 0; ok && x < n_q; ++x) {
          if (j == 0 && !(ok = wait(&bars->o_free[x], (o_items[x] & 1) ^ 1))) break;
          if (!(ok = wait(&bars->p_full[x], done[x] & 1))) break;
          tc_fence_after();
          if (leader) {
#pragma unroll
            for (int kk = 0; kk < BN / 16; ++kk)
              mma_ts(tmem + C::COL_O + x * D, tmem + C::COL_S + x * BN + kk * 8,
                     sdesc_advance(va, kk * 16 * 128), idesc_o, (j > 0 || kk > 0) ? 1u : 0u);
            mma_commit(&bars->o_ready[x]);
            if (j + 1 == n) mma_commit(&bars->o_done[x]);
          }
          ++done[x];
          if (j + 1 < n) {
            if (x == 0 && !(ok = wait_slot(Lk))) break;
            issue_s(x, Lk);
          }
        }
        if (!ok) break;
        if (leader) {
          mma_commit(&bars->ring_empty[Lv % C::SLOTS]);
          if (j + 1 < n) {
            mma_commit(&bars->ring_empty[Lk % C::SLOTS]);
            if (j + 2 == n) mma_commit(&bars->q_empty);
          }
        }
      }
      for (int x = 0; x < n_q; ++x) ++o_items[x];
      loads += 2 * n;
    }
    // Drain: all issued MMAs complete before TMEM is released.
    if (leader) mma_commit(&bars->drain);
    wait(&bars->drain, 0);
  } else {
    // ------------------------------------------------- softmax + epilogue
    const int x = (warp - 2) >> 2;  // query tile
    const int quarter = warp & 3;   // TMEM lanes this warp may access
    const int r = quarter * 32 + lane;
    const uint32_t t_lane = tmem + ((uint32_t)(quarter * 32) << 16);
    const uint32_t t_s = t_lane + C::COL_S + x * BN, t_o = t_lane + C::COL_O + x * D;
    const float s_mul = CAP ? p.scale / p.softcap : p.scale * kLog2e;
    const float cap_mul = p.softcap * kLog2e;
    uint32_t taken = 0, loads = 0, tiles = 0, done = 0;
    bool ok = true;
    while (ok) {
      const int isl = taken % kItemSlots;
      if (!(ok = wait(&bars->item_full[isl], (taken / kItemSlots) & 1))) break;
      const ItemSlot it = bars->items[isl];
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->item_empty[isl]);
      ++taken;
      if (it.last) break;
      const TreeSegment& s = it.s;
      const int n = s.count;
      const uint32_t l0 = loads;
      loads += 2 * n;
      if (x == 1 && !has_second(p, s)) continue;
      const int row = s.t * p.rows + x * kTcRows + r;
      const bool own = row < s.n * p.G;
      const int node = own ? row / p.G : 0;
      const bool any_own = __any_sync(0xffffffffu, own);
      const int total = s.past + s.n;
      const RowView view = row_view(p, s, node);
      RowState st;
      RowAlone alone;
      for (int j = 0; j < n; ++j, ++tiles) {
        const int k0 = (s.j0 + j) * BN;
        // the first tile's warps clean V for both: its product is issued first
        if (x == 0 && (k0 < s.lo || k0 + BN > total)) {
          const uint32_t L = l0 + 2 * j + 1;
          if (!(ok = wait(&bars->ring_full[L % C::SLOTS], (L / C::SLOTS) & 1))) break;
          zero_v_rows<BN, C::CH>(ring + (L % C::SLOTS) * C::KV_TILE, r, k0, s.lo, total);
        }
        if (!(ok = wait(&bars->s_full[x], tiles & 1))) break;
        if (any_own) {
          tc_fence_after();
          float alpha;
          softmax_columns<T, BN, CAP>(p, view, s.past, k0, t_s, s_mul, cap_mul, alone, st, alpha);
          if (j > 0 && __any_sync(0xffffffffu, alpha != 1.0f)) {
            // O must hold PV(j-1); every earlier phase has passed, since S(j)
            // was issued after it, in order
            if (!(ok = wait(&bars->o_ready[x], (tiles - 1) & 1))) break;
            tc_fence_after();
            scale_o(t_o, Columns{0, D}, alpha);
          }
          tmem_wait_st();
        }
        tc_fence_before();
        warp_arrive(&bars->p_full[x]);
      }
      if (!ok) break;
      if (!(ok = wait(&bars->o_done[x], done & 1))) break;
      ++done;
      tc_fence_after();
      if (any_own) store_row<T, D>(p, s, t_o, own, row, node, Columns{0, D}, st.m, st.l);
      tc_fence_before();
      warp_arrive(&bars->o_free[x]);
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc<C::TMEM_COLS>(tmem);
}

template <typename T, int D, int PARTS>
cudaError_t launch_parts(const TreeParams& p, const CUtensorMap& tq, const CUtensorMap& tk,
                         const CUtensorMap& tv, cudaStream_t s) {
  constexpr int smem = PairCfg<D, PARTS>::SMEM;
  const int cap = cap_form(p.softcap);
  auto kern = cap == kNoCap ? pva_tree_pair_kernel<T, D, PARTS, kNoCap>
              : cap == kCap ? pva_tree_pair_kernel<T, D, PARTS, kCap>
                            : pva_tree_pair_kernel<T, D, PARTS, kLargeCap>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  return launch_dependent(kern, dim3(p.pieces), dim3(kThreads), smem, s, p, tq, tk, tv);
}

template <typename T, int D>
cudaError_t launch_d(const TreeParams& p, const CUtensorMap& tq, const CUtensorMap& tk,
                     const CUtensorMap& tv, cudaStream_t s) {
  if constexpr (tree_takes_pair(256, D, 2))
    if (p.q_parts == 2) return launch_parts<T, D, 2>(p, tq, tk, tv, s);
  if (p.q_parts != 1) return cudaErrorInvalidValue;
  return launch_parts<T, D, 1>(p, tq, tk, tv, s);
}

template <typename T>
cudaError_t launch_type(const TreeParams& p, const CUtensorMap& tq, const CUtensorMap& tk,
                        const CUtensorMap& tv, cudaStream_t s) {
  switch (p.d) {
    case 64: return launch_d<T, 64>(p, tq, tk, tv, s);
    case 96: return launch_d<T, 96>(p, tq, tk, tv, s);
    case 128: return launch_d<T, 128>(p, tq, tk, tv, s);
    case 192: return launch_d<T, 192>(p, tq, tk, tv, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

cudaError_t launch_tree_pair(const TreeParams& p, int dtype, const CUtensorMap& tq,
                             const CUtensorMap& tk, const CUtensorMap& tv, cudaStream_t s) {
  return dtype == PVA_BF16 ? launch_type<__nv_bfloat16>(p, tq, tk, tv, s)
                           : launch_type<__half>(p, tq, tk, tv, s);
}

}  // namespace pva
