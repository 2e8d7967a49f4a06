// Tree attention over a KV cache on the 5th-generation tensor cores (tcgen05,
// operands staged by TMA, accumulators in TMEM), f16/bf16.
//
// A key tile of BN keys is read once for up to 128 query rows (nodes x heads of
// the group), 4 * 128 * BN * d operations per 4 * BN * d bytes (half as many again
// in S with rotated queries, see below): below the time the bytes take, so the
// kernel is built to keep the cache read going.  Each CTA takes one piece of the
// line of key tiles (pva_tree.h), every piece equally long, and streams its keys and
// values through a ring as deep as shared memory allows.  Decoding reads at 6.0 TB/s
// (0.89 of the copy rate); drafts of 32 nodes on 1000 to 8000 rows at 5.3 TB/s, with
// 16 us of front end and rotation before and 7 of join after 57 us here.
//
// Per CTA (320 threads):
//   warp 0      TMA producer: walks the piece's segments, publishes each one
//               through a ring in shared memory, and loads the Q tile, then
//               K_j and V_j, into one ring of slots.  Pages shorter than a key
//               tile are copied one page per lane, from the block table.
//   warp 1      MMA issuer and TMEM owner.  S = Q K^T (Q in TMEM) is
//               double-buffered, so S(j+1) runs while tile j is exponentiated;
//               P(j) replaces S(j) and feeds O += P V with A from TMEM.
//   warps 2..9  softmax and epilogue, two threads per query row, each with half
//               of a tile's columns: a tile's latency is what a short request
//               and a piece's last tiles wait for (a thread per row: 22.2
//               against 20.1 us for one request with 8 nodes on 500 rows).
// TMEM: S buffers [0, BN) and [BN, 2 BN), O [2 BN, 2 BN + D), Q after it.
//
// The rotated queries come in two parts, rounded to the storage type and the
// rest rounded again, and S adds the products of both: the second costs d / 16
// MMA steps of a time the copies leave over, and takes one of the three equal
// roundings (queries, weights, output) out of the result.  At d = 256 tensor
// memory has no room for the second part, which stays in shared memory.
//
// Masks: a row sees the cache rows [lo, past) and its ancestors among the new
// rows.  Tiles wholly inside that range of every row of a warp need no mask;
// the others build a bit per key from the range and the row's ancestor mask.
// V rows outside the item's keys are zeroed in shared memory before the
// product (cache rows there may hold anything, and 0 * NaN is NaN); their
// scores are masked whatever they are.
#pragma once

#include "pva_tree_tile.cuh"

namespace pva {
namespace one_tile {

using namespace tile;

constexpr int kThreads = 320;
constexpr int kItemSlots = 4;
constexpr int kSoftmaxWarps = 8;

template <int D>
struct TreeCfg {
  static constexpr int BN = tree_keys(D);
  static constexpr int CH = (D + 63) / 64;        // 128-byte column chunks of a row
  static constexpr int Q_CHUNK = kTcRows * 128;   // bytes of one chunk of the Q tile
  static constexpr int KV_CHUNK = BN * 128;       // bytes of one chunk of a K or V tile
  static constexpr int KV_TILE = CH * KV_CHUNK;   // one ring slot
  static constexpr int Q_PER_SLOT = KV_TILE / Q_CHUNK;
  static_assert(Q_PER_SLOT >= 1, "a Q chunk fits a ring slot");
  static constexpr bool REST_IN_SMEM = D > 192;  // the queries' second part
  static constexpr int TMEM_PARTS = REST_IN_SMEM ? 1 : 2;
  static constexpr int REST = REST_IN_SMEM ? CH * Q_CHUNK : 0;
  static constexpr int Q_SLOTS = (CH + Q_PER_SLOT - 1) / Q_PER_SLOT;  // of one part
  static constexpr int SLOTS_FIT = (232448 - kHeadBytes - REST) / KV_TILE;
  static constexpr int SLOTS = SLOTS_FIT < 16 ? SLOTS_FIT : 16;
  static_assert(SLOTS >= TMEM_PARTS * Q_SLOTS + 2, "ring depth");
  static constexpr int OFF_REST = SLOTS * KV_TILE;
  static constexpr int SMEM = kHeadBytes + OFF_REST + REST;
  static constexpr int TMEM_COLS = 512;
  static constexpr int COL_S = 0;
  static constexpr int COL_O = 2 * BN;
  static constexpr int COL_Q = COL_O + D;
  static_assert(COL_Q + TMEM_PARTS * D / 2 <= TMEM_COLS, "TMEM budget");
  static_assert(SMEM <= 232448, "shared memory budget");
};

template <typename W>
struct ItemSlot {
  typename W::Segment s;
  int last;
};

template <typename W>
struct Bars {
  uint64_t q_tmem, o_ready, o_done, o_free, drain, never;
  uint64_t rest_full, rest_empty;
  uint64_t s_full[2], p_full[2];
  uint64_t meet[4];
  uint64_t ring_full[16], ring_empty[16];
  uint64_t item_full[kItemSlots], item_empty[kItemSlots];
  ItemSlot<W> items[kItemSlots];
  float rows[2][kTcRows][2];  // [turn][row][half]
  uint32_t tmem_base;
  int abort;
};
static_assert(sizeof(Bars<TreeWork>) <= kHeadBytes, "barriers, segments and meeting places");

template <typename T, int D, int CAP, typename W>
__global__ void __launch_bounds__(kThreads, 1)
    pva_tree_tc_kernel(typename W::Params p, const __grid_constant__ typename W::Queries tmap_q,
                       const __grid_constant__ CUtensorMap tmap_k,
                       const __grid_constant__ CUtensorMap tmap_v) {
  using C = TreeCfg<D>;
  constexpr int BN = C::BN;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  static_assert(sizeof(Bars<W>) <= kHeadBytes, "barriers, segments and meeting places");
  if (misplaced<W>(smem_raw, p)) return;
  Bars<W>* bars = reinterpret_cast<Bars<W>*>(smem_raw);
  uint8_t* smem = smem_raw + kHeadBytes;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t* status = p.status;
  volatile int* abort = &bars->abort;
  const int q_slots = C::Q_SLOTS * (C::REST_IN_SMEM ? 1 : p.q_parts);
  const bool rest_in_smem = C::REST_IN_SMEM && p.q_parts == 2;

  if (threadIdx.x == 0) {
    bars->abort = 0;
    mbar_init(&bars->q_tmem, kSoftmaxWarps);
    mbar_init(&bars->o_ready, 1);
    mbar_init(&bars->o_done, 1);
    mbar_init(&bars->o_free, kSoftmaxWarps);
    for (int w = 0; w < 4; ++w) mbar_init(&bars->meet[w], 2);
    mbar_init(&bars->drain, 1);
    mbar_init(&bars->never, 1);
    mbar_init(&bars->rest_full, 1);
    mbar_init(&bars->rest_empty, 1);
    for (int b = 0; b < 2; ++b) {
      mbar_init(&bars->s_full[b], 1);
      mbar_init(&bars->p_full[b], kSoftmaxWarps);
    }
    for (int s = 0; s < C::SLOTS; ++s) {
      mbar_init(&bars->ring_full[s], 1);
      mbar_init(&bars->ring_empty[s], 1);
    }
    for (int s = 0; s < kItemSlots; ++s) {
      mbar_init(&bars->item_full[s], 1);
      mbar_init(&bars->item_empty[s], 1 + kSoftmaxWarps);
    }
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc<C::TMEM_COLS>(&bars->tmem_base);
  if (warp == 0 && lane == 0) {
    W::prefetch(tmap_q);
    prefetch_tensor_map(&tmap_k);
    prefetch_tensor_map(&tmap_v);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  W::start();

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    typename W::Walk walk(p, blockIdx.x);
    const TileCopies tc(p, BN);
    uint32_t loads = 0, published = 0, rests = 0;
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
      return __all_sync(0xffffffffu, mbar_wait<false>(bar, parity, abort, status));
    };
    auto publish = [&](const ItemSlot<W>& v) -> bool {
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
    ItemSlot<W> v;
    v.last = 0;
    while (ok && walk.next(p, v.s)) {
      if (!(ok = publish(v))) break;
      const typename W::Segment& s = v.s;
      for (int qs = 0; ok && qs < q_slots; ++qs, ++loads) {
        const int sl = loads % C::SLOTS;
        if (!(ok = wait(&bars->ring_empty[sl], ((loads / C::SLOTS) & 1) ^ 1))) break;
        if (lane == 0) {
          const int part = qs / C::Q_SLOTS, c_lo = (qs % C::Q_SLOTS) * C::Q_PER_SLOT;
          const int c_hi = min(C::CH, c_lo + C::Q_PER_SLOT);
          mbar_arrive_expect_tx(&bars->ring_full[sl], (uint32_t)(c_hi - c_lo) * W::q_bytes(p, s));
          for (int c = c_lo; c < c_hi; ++c)
            W::load_q(p, s, 0, part, smem + sl * C::KV_TILE + (c - c_lo) * C::Q_CHUNK, tmap_q,
                      &bars->ring_full[sl], c);
        }
        __syncwarp();
      }
      if (rest_in_smem) {
        // once the S MMAs of the segment before are done with it
        if (!ok || !(ok = wait(&bars->rest_empty, (rests & 1) ^ 1))) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(&bars->rest_full, C::REST);
          for (int c = 0; c < C::CH; ++c)
            W::load_q(p, s, 0, 1, smem + C::OFF_REST + c * C::Q_CHUNK, tmap_q, &bars->rest_full, c);
        }
        __syncwarp();
        ++rests;
      }
      // the block of the next tile's copy is looked up while this tile's slots
      // are waited for
      TileCopy copy = tc.template locate<W>(p, s, BN, s.j0, lane);
      for (int j = s.j0; ok && j < s.j0 + s.count; ++j) {
        const TileCopy next = tc.template locate<W>(p, s, BN, j + 1, lane);
        const uint32_t n_copies = __popc(__ballot_sync(0xffffffffu, copy.mine));
#pragma unroll
        for (int kv = 0; kv < 2; ++kv, ++loads) {
          const int sl = loads % C::SLOTS;
          if (!(ok = wait(&bars->ring_empty[sl], ((loads / C::SLOTS) & 1) ^ 1))) break;
          if (lane == 0)
            mbar_arrive_expect_tx(&bars->ring_full[sl], n_copies * C::CH * (uint32_t)tc.box * 128u);
          __syncwarp();
          if (copy.mine) {
            uint8_t* dst = smem + sl * C::KV_TILE + lane * tc.box * 128;
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
    }
    // Drain: every copy this warp issued must land before the CTA exits.
    if (rests) mbar_drain<false>(&bars->rest_full, (rests - 1) & 1, status);
    for (int s = 0; s < C::SLOTS; ++s) {
      const uint32_t fills = loads > (uint32_t)s ? (loads - 1 - s) / C::SLOTS + 1 : 0;
      if (fills) mbar_drain<false>(&bars->ring_full[s], (fills - 1) & 1, status);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    const bool leader = elect_sync();
    const uint32_t idesc_s = idesc_f16<T>(kTcRows, BN, false, false) | W::negate(p);
    constexpr uint32_t idesc_o = idesc_f16<T>(kTcRows, D, false, true);
    const uint64_t kdesc = sdesc_sw128(smem_u32(smem), 16, 1024);
    const uint64_t restdesc = sdesc_sw128(smem_u32(smem + C::OFF_REST), 16, 1024);
    const uint64_t vdesc = sdesc_sw128(smem_u32(smem), C::KV_CHUNK, 1024);
    uint32_t q_cnt = 0, loads = 0, gt = 0, items = 0, taken = 0;
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
      return __all_sync(0xffffffffu, mbar_wait<false>(bar, parity, abort, status));
    };
    auto wait_slot = [&](uint32_t L) -> bool {
      const bool r = wait(&bars->ring_full[L % C::SLOTS], (L / C::SLOTS) & 1);
      tc_fence_after();
      return r;
    };
    auto issue_s = [&](uint32_t T_, uint32_t L, bool last_of_segment) {
      const uint64_t ka = sdesc_advance(kdesc, (L % C::SLOTS) * C::KV_TILE);
      if (leader) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          mma_ts(tmem + C::COL_S + (T_ & 1) * BN, tmem + C::COL_Q + kk * 8,
                 sdesc_advance(ka, (kk >> 2) * C::KV_CHUNK + (kk & 3) * 32), idesc_s,
                 kk > 0 ? 1u : 0u);
        if (C::REST_IN_SMEM) {
          if (rest_in_smem) {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              mma_ss(tmem + C::COL_S + (T_ & 1) * BN,
                     sdesc_advance(restdesc, (kk >> 2) * C::Q_CHUNK + (kk & 3) * 32),
                     sdesc_advance(ka, (kk >> 2) * C::KV_CHUNK + (kk & 3) * 32), idesc_s, 1u);
            if (last_of_segment) mma_commit(&bars->rest_empty);
          }
        } else if (q_slots > C::Q_SLOTS) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            mma_ts(tmem + C::COL_S + (T_ & 1) * BN, tmem + C::COL_Q + D / 2 + kk * 8,
                   sdesc_advance(ka, (kk >> 2) * C::KV_CHUNK + (kk & 3) * 32), idesc_s, 1u);
        }
        mma_commit(&bars->s_full[T_ & 1]);
        mma_commit(&bars->ring_empty[L % C::SLOTS]);
      }
    };
    while (ok) {
      const int isl = taken % kItemSlots;
      if (!(ok = wait(&bars->item_full[isl], (taken / kItemSlots) & 1))) break;
      const int n = bars->items[isl].s.count, last = bars->items[isl].last;
      __syncwarp();
      if (leader) mbar_arrive(&bars->item_empty[isl]);
      ++taken;
      if (last) break;
      if (p.hold_ns && !(ok = __all_sync(0xffffffffu, mbar_wait<false>(&bars->never, 0, abort, status, p.hold_ns))))
        break;
      // Q is in TMEM once every softmax thread has copied its share.
      if (!(ok = wait(&bars->q_tmem, q_cnt & 1))) break;
      if (rest_in_smem && !(ok = wait(&bars->rest_full, q_cnt & 1))) break;
      tc_fence_after();
      if (leader)
        for (int qs = 0; qs < q_slots; ++qs)
          mbar_arrive(&bars->ring_empty[(loads + qs) % C::SLOTS]);
      loads += q_slots;
      for (int j = 0; ok && j < 2 && j < n; ++j) {
        if (!(ok = wait_slot(loads + 2 * j))) break;
        issue_s(gt + j, loads + 2 * j, j + 1 == n);
      }
      if (!ok) break;
      for (int j = 0; ok && j < n; ++j) {
        const uint32_t T_ = gt + j, Lv = loads + 2 * j + 1;
        if (!(ok = wait_slot(Lv))) break;
        if (j == 0 && !(ok = wait(&bars->o_free, (items & 1) ^ 1))) break;
        if (!(ok = wait(&bars->p_full[T_ & 1], (T_ >> 1) & 1))) break;
        tc_fence_after();
        const uint64_t va = sdesc_advance(vdesc, (Lv % C::SLOTS) * C::KV_TILE);
        if (leader) {
#pragma unroll
          for (int kk = 0; kk < BN / 16; ++kk)
            mma_ts(tmem + C::COL_O, tmem + C::COL_S + (T_ & 1) * BN + p_column<BN>(kk),
                   sdesc_advance(va, kk * 16 * 128), idesc_o, (j > 0 || kk > 0) ? 1u : 0u);
          mma_commit(&bars->o_ready);
          if (j + 1 == n) mma_commit(&bars->o_done);
          mma_commit(&bars->ring_empty[Lv % C::SLOTS]);
        }
        if (j + 2 < n) {
          if (!(ok = wait_slot(loads + 2 * (j + 2)))) break;
          issue_s(T_ + 2, loads + 2 * (j + 2), j + 3 == n);
        }
      }
      loads += 2 * n;
      gt += n;
      ++q_cnt;
      ++items;
    }
    // Drain: all issued MMAs complete before TMEM is released.
    if (leader) mma_commit(&bars->drain);
    mbar_drain<false>(&bars->drain, 0, status);
    __syncwarp();
  } else {
    // ------------------------------------------------- softmax + epilogue
    const int half = (warp - 2) >> 2;  // of the columns
    const int quarter = warp & 3;      // TMEM lanes this warp may access
    const int r = quarter * 32 + lane;
    const uint32_t t_lane = tmem + ((uint32_t)(quarter * 32) << 16);
    const float s_mul = CAP ? p.scale / p.softcap : p.scale * kLog2e;
    const float cap_mul = p.softcap * kLog2e;
    RowPair pair{&bars->rows[0][r][0], &bars->meet[quarter], half, abort, status};
    uint32_t gt = 0, taken = 0, done = 0;
    uint32_t lq = 0;  // ring loads accounted for (the producer's order)
    bool ok = true, q_pre = false;
    // Copies the next Q tile from its ring slots into TMEM.
    auto copy_q = [&]() -> bool {
      bool got = true;
      for (int qs = 0; qs < q_slots; ++qs) {
        const uint32_t L = lq + qs;
        got = got && mbar_wait<false>(&bars->ring_full[L % C::SLOTS], (L / C::SLOTS) & 1, abort,
                                      status);
      }
      if (!__all_sync(0xffffffffu, got)) return false;
      // the chunks of both parts, every other one each half's
      const int chunks = q_slots > C::Q_SLOTS ? 2 * C::CH : C::CH;
#pragma unroll 1
      for (int i = half; i < chunks; i += 2) {
        const int part = i / C::CH, c = i - part * C::CH;
        const uint32_t L = lq + part * C::Q_SLOTS + c / C::Q_PER_SLOT;
        const uint32_t t_q = t_lane + C::COL_Q + part * (D / 2) + c * 32;
        const uint8_t* src =
            smem + (L % C::SLOTS) * C::KV_TILE + (c % C::Q_PER_SLOT) * C::Q_CHUNK + r * 128;
        uint32_t w[32];
#pragma unroll
        for (int u = 0; u < 8; ++u) {  // 16-byte unit u of the row, 128-byte swizzle
          const uint4 x = *reinterpret_cast<const uint4*>(src + ((u ^ (r & 7)) << 4));
          w[4 * u] = x.x;
          w[4 * u + 1] = x.y;
          w[4 * u + 2] = x.z;
          w[4 * u + 3] = x.w;
        }
        if (D % 64 == 0 || c + 1 < C::CH) {
          tmem_st32(t_q, w);
        } else {  // a 32-column tail chunk
          uint32_t w16[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) w16[e] = w[e];
          tmem_st16(t_q, w16);
        }
      }
      tmem_wait_st();
      fence_proxy_async_smem();  // the slots are refilled by the TMA unit next
      tc_fence_before();
      warp_arrive(&bars->q_tmem);
      lq += q_slots;
      return true;
    };

    while (ok) {
      const int isl = taken % kItemSlots;
      ok = __all_sync(0xffffffffu, mbar_wait<false>(&bars->item_full[isl],
                                                    (taken / kItemSlots) & 1, abort, status));
      if (!ok) break;
      const ItemSlot<W> it = bars->items[isl];
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->item_empty[isl]);
      ++taken;
      if (it.last) break;
      const typename W::Segment& s = it.s;
      const int n = s.count;
      const int row = W::row(p, s, 0, r);
      const bool own = W::owns(p, s, r, row);
      const int node = own ? row / p.G : 0;
      if (!q_pre && !(ok = copy_q())) break;
      q_pre = false;
      const uint32_t l0 = lq;  // the segment's first K load
      lq += 2 * n;
      const int total = W::total(s);
      const RowView view = W::view(p, s, node);
      const bool any_own = __any_sync(0xffffffffu, own);
      RowState st;

      for (int j = 0; j < n; ++j) {
        const uint32_t T_ = gt + j;
        const int k0 = (s.j0 + j) * BN;
        if (half == 0 && (k0 < s.lo || k0 + BN > total)) {
          // V rows outside the item's keys: zeros
          const uint32_t L = l0 + 2 * j + 1;
          ok = __all_sync(0xffffffffu, mbar_wait<false>(&bars->ring_full[L % C::SLOTS],
                                                        (L / C::SLOTS) & 1, abort, status));
          if (!ok) break;
          zero_v_rows<BN, C::CH>(smem + (L % C::SLOTS) * C::KV_TILE, r, k0, s.lo, total);
        }
        ok = __all_sync(0xffffffffu,
                        mbar_wait<false>(&bars->s_full[T_ & 1], (T_ >> 1) & 1, abort, status));
        if (!ok) break;
        if (any_own) {
          tc_fence_after();
          const uint32_t t_s = t_lane + C::COL_S + (T_ & 1) * BN + half * (BN / 2);
          float alpha;
          ok = softmax_columns<T, BN / 2, CAP, W::kMid>(p, view, s.past, k0 + half * (BN / 2), t_s, s_mul, cap_mul,
                                            W::counts(own), pair, st, alpha);
          if (!ok) break;
          if (j > 0 && __any_sync(0xffffffffu, alpha != 1.0f)) {
            // O must hold PV(j-1) before it is rescaled; PV(j-2) precedes S(j),
            // so the parity of the outstanding phase is unambiguous.
            ok = __all_sync(0xffffffffu,
                            mbar_wait<false>(&bars->o_ready, (T_ - 1) & 1, abort, status));
            if (!ok) break;
            tc_fence_after();
            scale_o(t_lane + C::COL_O, half_columns<D>(half), alpha);
          }
          tmem_wait_st();
        }
        tc_fence_before();
        warp_arrive(&bars->p_full[T_ & 1]);
      }
      if (!ok) break;

      // The next segment's Q goes to TMEM before this one's epilogue, so that
      // its first S MMAs run meanwhile.
      {
        const int nsl = taken % kItemSlots;
        ok = __all_sync(0xffffffffu, mbar_wait<false>(&bars->item_full[nsl],
                                                      (taken / kItemSlots) & 1, abort, status));
        if (!ok) break;
        if (!bars->items[nsl].last) {
          if (!(ok = copy_q())) break;
          q_pre = true;
        }
      }

      ok = __all_sync(0xffffffffu, mbar_wait<false>(&bars->o_done, done & 1, abort, status));
      ++done;
      if (!ok) break;
      tc_fence_after();
      if (any_own) {
        float l;
        if (!(ok = pair.exchange(st.l, l))) break;
        W::template store<T, D>(p, s, t_lane + C::COL_O, own, row, node, half_columns<D>(half), st.m, st.l + l);
      }
      tc_fence_before();
      warp_arrive(&bars->o_free);
      gt += n;
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc<C::TMEM_COLS>(tmem);
  if (threadIdx.x == 0 && *abort) W::give_up(p);  // whoever gave up: nothing is joined
}

}  // namespace one_tile
}  // namespace pva
