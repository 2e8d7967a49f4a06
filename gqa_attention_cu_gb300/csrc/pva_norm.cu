// Norms of query and key heads with the rotary embedding in the same pass
// (pva_norm_rope), and their gradient (pva_norm_rope_backward).
//
// A head row x of d dims gets y = R(n * w) with n = x r, r = (mean x^2 + eps)^-1/2,
// w = offset + weight (the same for all heads of q, or of k) and R the rotation of
// pva_rope.cuh, all in f32 and rounded once.  With g = R^T dy (the rotation by the
// negative angle) the gradients are
//   dx = r (g w - n mean(g w n)),   dweight = sum over rows of g n.
//
// Memory is the floor: each row is read once and written once (twice read in the
// gradient).  A row lies across a few lanes, 16 bytes of each of the two halves that
// turn together per lane, so that its sums take log2(lanes) shuffles and the pairs
// meet in one thread.  A warp works on a token's rows by itself: its lanes copy their
// own packs into their own places of shared memory some row groups ahead
// (asynchronously, and so across tokens, without registers to hold them and without a
// barrier), a token's cos and sin are fetched a pair a lane one token ahead, and gain
// and rotation are one matrix (ca, sb; sa, cb) per pair, made once a token.
//
// 16,001 tokens with 32 + 8 + 8 head rows of 128 bf16, keys and values to the cache: 77
// us, 5.1 TB/s of 394 MB (59 at the copy rate); the gradient of 8190 tokens of 32 + 8
// rows: 61 us, 4.1 TB/s of 252 MB (38).  What bounds them is instructions beside few
// warps: 257 a row group of the forward form, a third of them arithmetic, at 16 warps
// an SM (5 CTAs an SM instead of 4, with 96 registers: 94 us; rows held in registers
// instead of shared memory: 93 us).  Smaller calls: launch and the caller's side.
#include <limits.h>
#include <math.h>

#include "pva_rope.cuh"

using namespace pva;
using namespace pva::host;

namespace pva {
namespace {

struct NormStep {
  RopeTable rt;  // rot 0: no rotation
  const void* x[2];    // q, k [tokens, heads, d] with a token stride; nullptr: none
  const void* dy[2];   // gradient: of the outputs
  void* out[2];        // q_out, k_out; gradient: dq, dk
  const void* w[2];    // [d], or nullptr: gains of one
  long long x_stride[2], dy_stride[2], out_stride[2];  // elements
  int heads[2];        // 0: none
  const void* v;       // copied to the cache
  long long v_stride;
  void* k_cache;       // [blocks, kv heads, page, d]; nullptr: no cache
  void* v_cache;
  const int64_t* slots;
  int page;
  long long n_slots;
  const int64_t* pos;  // [n_axes, tokens]
  int tokens, d;
  int w_f32;           // the gains are f32, else of the rows' type
  float eps, offset, inv_d;
  int parts;           // warps that share a token's rows
  float* partial;      // gradient: [warps' CTAs][2][d] sums of g n
  int want_w[2];       // gradient: the sums are asked for
  float* dw[2];        // [d]
  uint32_t* status;
};

constexpr int kNormCtas = 4, kBackCtas = 3;  // CTAs an SM holds
constexpr int kNormThreads = 128;
constexpr int kNormWarps = kNormThreads / 32;
constexpr int kMaxHalf = 128;  // pairs of a row
constexpr int kFly = 4, kBackFly = 3;  // row groups whose copies are in flight

__device__ __forceinline__ float2 fmul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 ra, rb, rd;\n\t"
      "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
      "mul.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

// VEC floats as pairs for the packed instructions (VEC 1: the second is zero).
template <int VEC>
struct Floats {
  static constexpr int N = (VEC + 1) / 2;
  float2 v[N];
  __device__ __forceinline__ float& operator[](int e) { return e % 2 ? v[e / 2].y : v[e / 2].x; }
  __device__ __forceinline__ float operator[](int e) const { return e % 2 ? v[e / 2].y : v[e / 2].x; }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = make_float2(0.0f, 0.0f);
  }
};

// The first and second members of a unit's pairs, as floats.
template <typename T, int VEC, bool NB>
struct Pairs {
  Floats<VEC> a, b;
  __device__ __forceinline__ void take(Pack<T, VEC> x, Pack<T, VEC> y) {
    if (NB) split_pairs(x, y);
    if (VEC == 1) a.clear(), b.clear();
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      a[e] = load_f(x.v[e]);
      b[e] = load_f(y.v[e]);
    }
  }
  __device__ __forceinline__ void give(Pack<T, VEC>& x, Pack<T, VEC>& y) const {
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      x.v[e] = round_to<T>(a[e]);
      y.v[e] = round_to<T>(b[e]);
    }
    if (NB) join_pairs(x, y);
  }
};

// Sum over the TPR lanes of a row.
template <int TPR>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int o = TPR / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// What a warp works with: TPR lanes a row, U units of 2 VEC dims a lane, and a
// token's cos and sin in shared memory.  Lane a < n_axes reads the position on axis
// a, lane kMaxAxes the slot; the entries of the pairs are fetched a pair a lane, one
// token ahead of the rows.
struct NormShared {
  float gain[2][2 * kMaxHalf];             // of q and k, by dim
  float2 cs[kNormWarps][kMaxHalf];         // of the warps' tokens
};

// NB: pairs of neighbouring dims (also of those that are not turned).
template <typename T, int VEC, int TPR, int U, bool NB>
struct NormLane {
  using P = Pack<T, VEC>;
  static constexpr int FETCH = kMaxHalf / 32;  // pairs a lane fetches
  int group;           // row within the warp's 32 / TPR
  bool in[U];          // the unit exists
  int d0[U], d1[U], pair[U];
  bool turned[U];
  uint32_t axes;       // of the pairs lane, lane + 32, ..., two bits each
  __device__ __forceinline__ NormLane(const NormStep& p) {
    const int lane = threadIdx.x & 31, sub = lane % TPR, half = p.rt.rot / 2;
    group = lane / TPR;
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int u = sub + i * TPR;
      in[i] = u < p.d / (2 * VEC);
      turned[i] = in[i] && u * VEC < half;
      pair[i] = u * VEC;
      d0[i] = !in[i] ? 0 : !turned[i] ? p.rt.rot + (u - half / VEC) * 2 * VEC : NB ? u * 2 * VEC : u * VEC;
      d1[i] = turned[i] && !NB ? d0[i] + half : d0[i] + VEC;
    }
    axes = 0;
    for (int f = 0; f < FETCH; ++f)
      if (lane + 32 * f < half) axes |= (uint32_t)axis_of_pair(p.rt, lane + 32 * f) << (2 * f);
  }
  // lane a < n_axes: the token's position on axis a; lane kMaxAxes: its slot
  __device__ __forceinline__ int64_t fetch_info(const NormStep& p, long long tok) const {
    const int lane = threadIdx.x & 31;
    int64_t x = lane == kMaxAxes ? -1 : 0;
    if (tok < p.tokens) {
      if (p.rt.rot && lane < p.rt.n_axes) x = p.pos[(size_t)lane * p.tokens + tok];
      if (p.slots && lane == kMaxAxes) x = p.slots[tok];
    }
    return x;
  }
  // all positions on the tables and the slot in the cache
  __device__ __forceinline__ bool fine(const NormStep& p, int64_t info) const {
    const int lane = threadIdx.x & 31;
    const bool bad = lane == kMaxAxes ? info < -1 || info >= p.n_slots
                                      : p.rt.rot && lane < p.rt.n_axes && (info < 0 || info >= p.rt.rows);
    return !__any_sync(0xffffffffu, bad);
  }
  struct Entries { float2 cs[FETCH]; };
  __device__ __forceinline__ Entries fetch_entries(const NormStep& p, int64_t info, float sign) const {
    const int lane = threadIdx.x & 31, half = p.rt.rot / 2;
    Entries x;
#pragma unroll
    for (int f = 0; f < FETCH; ++f) {
      x.cs[f] = make_float2(1.0f, 0.0f);
      if (32 * f >= half) continue;
      const int64_t at = __shfl_sync(0xffffffffu, info, axes >> (2 * f) & 3);
      if (lane + 32 * f < half && at >= 0 && at < p.rt.rows) {
        const int64_t i = at * half + lane + 32 * f;
        x.cs[f].x = table_at<false>(p.rt.cos, i, p.rt.is_f16);
        x.cs[f].y = sign * table_at<false>(p.rt.sin, i, p.rt.is_f16);
      }
    }
    return x;
  }
  __device__ __forceinline__ void share(const NormStep& p, const Entries& x, float2* to) const {
    const int lane = threadIdx.x & 31, half = p.rt.rot / 2;
    __syncwarp();
#pragma unroll
    for (int f = 0; f < FETCH; ++f)
      if (lane + 32 * f < half) to[lane + 32 * f] = x.cs[f];
    __syncwarp();
  }
  __device__ __forceinline__ void turn(const float2* cs, int i, Floats<VEC>& c, Floats<VEC>& s) const {
    if (VEC == 1) c.clear(), s.clear();
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const float2 x = turned[i] ? cs[pair[i] + e] : make_float2(1.0f, 0.0f);
      c[e] = x.x;
      s[e] = x.y;
    }
  }
  // where the e-th pair's members lie in the row
  __device__ __forceinline__ int first(int i, int e) const { return NB ? d0[i] + 2 * e : d0[i] + e; }
  __device__ __forceinline__ int second(int i, int e) const { return NB ? d0[i] + 2 * e + 1 : d1[i] + e; }
  __device__ __forceinline__ void gains(const float* w, int i, Floats<VEC>& a, Floats<VEC>& b) const {
    if (VEC == 1) a.clear(), b.clear();
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      a[e] = w[first(i, e)];
      b[e] = w[second(i, e)];
    }
  }
  // This lane's packs of a row on their way to its own place in shared memory (16
  // bytes asynchronously, single elements at once); zeros where there is no row.
  __device__ __forceinline__ void copy_row(const T* src, bool there, P (*to)[U][32]) const {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < U; ++i) {
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const T* from = src + (half ? d1[i] : d0[i]);
        P* dst = &to[half][i][lane];
        const bool valid = there && in[i];
        if constexpr (sizeof(P) == 16) {
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(from),
                       "r"(valid ? 16 : 0)
                       : "memory");
        } else {
          P x;
          x.v[0] = valid ? *from : round_to<T>(0.0f);
          *dst = x;
        }
      }
    }
  }
  __device__ __forceinline__ void take_row(const P (*from)[U][32], Pairs<T, VEC, NB> (&v)[U]) const {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < U; ++i) v[i].take(from[0][i][lane], from[1][i][lane]);
  }
  __device__ __forceinline__ void store_row(T* dst, const P (&x)[U], const P (&y)[U]) const {
#pragma unroll
    for (int i = 0; i < U; ++i)
      if (in[i]) {
        *reinterpret_cast<P*>(dst + d0[i]) = x[i];
        *reinterpret_cast<P*>(dst + d1[i]) = y[i];
      }
  }
};

// The gains of q and k as f32 in shared memory.
template <typename T>
__device__ __forceinline__ void share_gains(const NormStep& p, NormShared& sh) {
  for (int i = threadIdx.x; i < 2 * p.d; i += kNormThreads) {
    const int which = i >= p.d, c = i - which * p.d;
    const void* w = p.w[which];
    sh.gain[which][c] = !w        ? 1.0f
                        : p.w_f32 ? static_cast<const float*>(w)[c] + p.offset
                                  : load_f(static_cast<const T*>(w)[c]) + p.offset;
  }
  __syncthreads();
}

// The row groups (32 / TPR rows of q, k or v of a token) that a warp works on, one
// after another: items are (token, part of its rows), a warp takes every so many.
// Within a kind of rows only `row` moves on.
struct NormCursor {
  long long item;
  int tok, which, row, n;  // this lane's row, of n
  int base;                // the warp's first row of the group
};

// KINDS of rows from kind FIRST on: 0 q, 1 k, 2 v.
template <int RPP>
struct NormWalk {
  long long items, stride;
  int step, parts, group, first, kinds, n0, n1, n2;
  __device__ __forceinline__ NormWalk(const NormStep& p, int group_, int first_, int kinds_)
      : items((long long)p.tokens * p.parts), stride((long long)gridDim.x * kNormWarps), step(p.parts * RPP),
        parts(p.parts), group(group_), first(first_), kinds(kinds_), n0(p.heads[0]), n1(p.heads[1]),
        n2(p.v ? p.heads[1] : 0) {}
  __device__ __forceinline__ int rows_of(int which) const { return which == 0 ? n0 : which == 1 ? n1 : n2; }
  __device__ __forceinline__ bool more(const NormCursor& c) const { return c.item < items; }
  // the first group of kind c.which, or of a later one, that has rows
  __device__ __forceinline__ void settle(NormCursor& c) const {
    while (true) {
      c.tok = parts == 1 ? (int)c.item : (int)(c.item / parts);
      c.base = (int)(c.item - (long long)c.tok * parts) * RPP;
      c.row = c.base + group;
      c.n = rows_of(c.which);
      if (c.base < c.n || !more(c)) return;
      if (++c.which == first + kinds) {
        c.which = first;
        c.item += stride;
      }
    }
  }
  __device__ __forceinline__ NormCursor begin() const {
    NormCursor c;
    c.item = (long long)blockIdx.x * kNormWarps + (threadIdx.x >> 5);
    c.which = first;
    settle(c);
    return c;
  }
  // on to the next group; false: of another kind or token
  __device__ __forceinline__ bool next(NormCursor& c) const {
    c.base += step;
    c.row += step;
    if (c.base < c.n) return true;
    if (++c.which == first + kinds) {
      c.which = first;
      c.item += stride;
    }
    settle(c);
    return false;
  }
};

// FLY row groups have their copies in flight; a lane reads only what it copied.
template <typename T, int VEC, int TPR, int U, int FLY, bool NB>
__global__ void __launch_bounds__(kNormThreads, kNormCtas) pva_norm_rope_kernel(NormStep p) {
  using P = Pack<T, VEC>;
  constexpr int RPP = 32 / TPR, N = Floats<VEC>::N;
  __shared__ NormShared sh;
  __shared__ P stage[kNormWarps][FLY][2][U][32];
  allow_next_grid();
  wait_prior_grid();
  const NormLane<T, VEC, TPR, U, NB> me(p);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const NormWalk<RPP> walk(p, me.group, 0, 3);
  NormCursor ahead = walk.begin(), at = ahead;
  // where the group's rows come from, at its lane's row
  auto source = [&](const NormCursor& c) {
    const T* x = static_cast<const T*>(c.which == 0 ? p.x[0] : c.which == 1 ? p.x[1] : p.v);
    const long long st = c.which == 0 ? p.x_stride[0] : c.which == 1 ? p.x_stride[1] : p.v_stride;
    return x + c.tok * st + (size_t)c.row * p.d;
  };
  const T* src = walk.more(ahead) ? source(ahead) : nullptr;
  const int src_step = walk.step * p.d;
  auto copy = [&](int slot) {
    if (walk.more(ahead)) {
      me.copy_row(src, ahead.row < ahead.n, stage[warp][slot]);
      if (walk.next(ahead))
        src += src_step;
      else if (walk.more(ahead))
        src = source(ahead);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int f = 0; f < FLY - 1; ++f) copy(f);
  int64_t next_info = me.fetch_info(p, walk.more(at) ? at.tok : p.tokens);
  auto entries = me.fetch_entries(p, next_info, 1.0f);
  share_gains<T>(p, sh);
  int slot = 0;
  bool fresh = true, ok = false;  // fresh: another kind of rows, or another token
  long long item = -1;
  int64_t where = -1;
  size_t cache_row = 0;  // of head 0
  T *out = nullptr, *cache = nullptr;
  const int out_step = walk.step * p.d;
  const long long cache_step = (long long)walk.step * p.page * p.d;
  // gain and rotation in one: (a, b) -> r (ca a - sb b, sa a + cb b)
  Floats<VEC> ca[U], sb[U], sa[U], cb[U];
  while (walk.more(at)) {
    copy(slot == 0 ? FLY - 1 : slot - 1);
    const bool arrived = at.item != item;
    if (fresh) {
      if (arrived) {  // a new token: its entries, and the next one's positions on their way
        item = at.item;
        const int64_t info = next_info;
        me.share(p, entries, sh.cs[warp]);
        // (every item has rows: the next one lies a stride ahead)
        next_info = me.fetch_info(p, (item + walk.stride) / p.parts);
        ok = me.fine(p, info);
        where = __shfl_sync(0xffffffffu, info, kMaxAxes);
        if (!ok && lane == 0) atomicOr(p.status, PVA_DEV_ROPE);
        if (ok && where >= 0) {
          const int64_t block = p.n_slots >> 32 ? where / p.page : (int64_t)((uint32_t)where / (uint32_t)p.page);
          cache_row = ((size_t)block * walk.n1 * p.page + (size_t)(where - block * p.page)) * p.d;
        }
      }
      const int which = at.which;
      out = which == 2 ? nullptr : static_cast<T*>(which ? p.out[1] : p.out[0]);
      if (out) out += at.tok * (which ? p.out_stride[1] : p.out_stride[0]) + (size_t)at.row * p.d;
      cache = nullptr;
      if (which > 0 && ok && where >= 0)
        cache = static_cast<T*>(which == 2 ? p.v_cache : p.k_cache) + cache_row + (size_t)at.row * p.page * p.d;
      if (which < 2) {
#pragma unroll
        for (int i = 0; i < U; ++i) {
          Floats<VEC> c, s, wa, wb;
          me.turn(sh.cs[warp], i, c, s);
          me.gains(sh.gain[which], i, wa, wb);
#pragma unroll
          for (int e = 0; e < N; ++e) {
            ca[i].v[e] = fmul2(c.v[e], wa.v[e]);
            sa[i].v[e] = fmul2(s.v[e], wa.v[e]);
            cb[i].v[e] = fmul2(c.v[e], wb.v[e]);
            sb[i].v[e] = make_float2(-s.v[e].x * wb.v[e].x, -s.v[e].y * wb.v[e].y);
          }
        }
      }
    }
    asm volatile("cp.async.wait_group %0;" ::"n"(FLY - 1) : "memory");
    const P(*mine)[U][32] = stage[warp][slot];
    const bool write = ok && at.row < at.n;
    P x[U], y[U];
    if (at.which < 2) {
      Pairs<T, VEC, NB> v[U];
      me.take_row(mine, v);
      float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
      for (int i = 0; i < U; ++i)
#pragma unroll
        for (int e = 0; e < N; ++e) sum = ffma2(v[i].a.v[e], v[i].a.v[e], ffma2(v[i].b.v[e], v[i].b.v[e], sum));
      const float r = rsqrtf(fmaf(row_sum<TPR>(sum.x + sum.y), p.inv_d, p.eps));
      const float2 r2 = make_float2(r, r);
#pragma unroll
      for (int i = 0; i < U; ++i) {
#pragma unroll
        for (int e = 0; e < N; ++e) {
          const float2 a = v[i].a.v[e], b = v[i].b.v[e];
          v[i].a.v[e] = fmul2(r2, ffma2(ca[i].v[e], a, fmul2(sb[i].v[e], b)));
          v[i].b.v[e] = fmul2(r2, ffma2(sa[i].v[e], a, fmul2(cb[i].v[e], b)));
        }
        v[i].give(x[i], y[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < U; ++i) {
        x[i] = mine[0][i][lane];
        y[i] = mine[1][i][lane];
      }
    }
    if (write) {
      if (out) me.store_row(out, x, y);
      if (cache) me.store_row(cache, x, y);
    }
    if (arrived) entries = me.fetch_entries(p, next_info, 1.0f);  // by now the positions are here
    fresh = !walk.next(at);
    if (out) out += out_step;
    if (cache) cache += cache_step;
    slot = slot + 1 == FLY ? 0 : slot + 1;
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// The gradient.  Each warp sums g n over its rows in registers, each CTA over its
// warps, and pva_norm_weights_kernel over the CTAs, always in the same order.
template <typename T, int VEC, int TPR, int U, int FLY, bool NB>
__global__ void __launch_bounds__(kNormThreads, kBackCtas) pva_norm_rope_backward_kernel(NormStep p) {
  using P = Pack<T, VEC>;
  constexpr int RPP = 32 / TPR, N = Floats<VEC>::N;
  extern __shared__ float s_sum[];  // [2][warps][d]
  __shared__ NormShared sh;
  __shared__ P stage[kNormWarps][FLY][2][2][U][32];
  allow_next_grid();
  wait_prior_grid();
  const NormLane<T, VEC, TPR, U, NB> me(p);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  share_gains<T>(p, sh);
#pragma unroll 1
  for (int which = 0; which < 2; ++which) {
    const int n = p.heads[which];
    if (n == 0) continue;
    const NormWalk<RPP> walk(p, me.group, which, 1);
    NormCursor ahead = walk.begin(), at = ahead;
    const T *src = nullptr, *grad = nullptr;
    auto source = [&]() {
      if (!walk.more(ahead)) return;
      src = static_cast<const T*>(p.x[which]) + ahead.tok * p.x_stride[which] + (size_t)ahead.row * p.d;
      grad = static_cast<const T*>(p.dy[which]) + ahead.tok * p.dy_stride[which] + (size_t)ahead.row * p.d;
    };
    source();
    const int row_step = walk.step * p.d;
    auto copy = [&](int slot) {
      if (walk.more(ahead)) {
        const bool there = ahead.row < ahead.n;
        me.copy_row(src, there, stage[warp][slot][0]);
        me.copy_row(grad, there, stage[warp][slot][1]);
        if (walk.next(ahead)) {
          src += row_step;
          grad += row_step;
        } else {
          source();
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int f = 0; f < FLY - 1; ++f) copy(f);
    long long fetched = walk.more(at) ? at.tok : p.tokens;  // the token of info and entries
    int64_t next_info = me.fetch_info(p, fetched);
    auto entries = me.fetch_entries(p, next_info, -1.0f);
    Floats<VEC> wa[U], wb[U], da[U], db[U], c[U], s[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      me.gains(sh.gain[which], i, wa[i], wb[i]);
      da[i].clear();
      db[i].clear();
    }
    long long item = -1;
    int slot = 0;
    bool ok = false;
    T* out = nullptr;
    while (walk.more(at)) {
      copy(slot == 0 ? FLY - 1 : slot - 1);
      const bool arrived = at.item != item;
      if (arrived) {
        item = at.item;
        out = static_cast<T*>(p.out[which]) + at.tok * p.out_stride[which] + (size_t)at.row * p.d;
        if (fetched != at.tok) {  // items without rows of this kind were passed over
          next_info = me.fetch_info(p, at.tok);
          entries = me.fetch_entries(p, next_info, -1.0f);
        }
        me.share(p, entries, sh.cs[warp]);
        ok = me.fine(p, next_info);
        if (!ok && lane == 0) atomicOr(p.status, PVA_DEV_ROPE);
        fetched = (item + walk.stride) / p.parts;
        next_info = me.fetch_info(p, fetched);
#pragma unroll
        for (int i = 0; i < U; ++i) me.turn(sh.cs[warp], i, c[i], s[i]);
      }
      asm volatile("cp.async.wait_group %0;" ::"n"(FLY - 1) : "memory");
      Pairs<T, VEC, NB> v[U], g[U];
      me.take_row(stage[warp][slot][0], v);
      me.take_row(stage[warp][slot][1], g);
      float2 sum = make_float2(0.0f, 0.0f), inner = sum;
#pragma unroll
      for (int i = 0; i < U; ++i) {
#pragma unroll
        for (int e = 0; e < N; ++e) {
          sum = ffma2(v[i].a.v[e], v[i].a.v[e], ffma2(v[i].b.v[e], v[i].b.v[e], sum));
          const float2 ga = g[i].a.v[e], gb = g[i].b.v[e], minus = make_float2(-s[i].v[e].x, -s[i].v[e].y);
          g[i].a.v[e] = ffma2(c[i].v[e], ga, fmul2(minus, gb));
          g[i].b.v[e] = ffma2(s[i].v[e], ga, fmul2(c[i].v[e], gb));
          inner = ffma2(fmul2(g[i].a.v[e], wa[i].v[e]), v[i].a.v[e],
                        ffma2(fmul2(g[i].b.v[e], wb[i].v[e]), v[i].b.v[e], inner));
        }
      }
      const float r = rsqrtf(fmaf(row_sum<TPR>(sum.x + sum.y), p.inv_d, p.eps));
      // n mean(g w n) r = n (r^2 mean(g w x)), with n = x r
      const float m = -(row_sum<TPR>(inner.x + inner.y) * p.inv_d * r * r);
      const float2 r2 = make_float2(r, r), m2 = make_float2(m, m);
      // Lanes without a row work on zeros, whose r is infinite where eps is 0.
      const bool mine = ok && at.row < at.n;
      P x[U], y[U];
#pragma unroll
      for (int i = 0; i < U; ++i) {
#pragma unroll
        for (int e = 0; e < N; ++e) {
          const float2 na = fmul2(v[i].a.v[e], r2), nb = fmul2(v[i].b.v[e], r2);
          if (mine) {
            da[i].v[e] = ffma2(g[i].a.v[e], na, da[i].v[e]);
            db[i].v[e] = ffma2(g[i].b.v[e], nb, db[i].v[e]);
          }
          g[i].a.v[e] = ffma2(fmul2(g[i].a.v[e], wa[i].v[e]), r2, fmul2(na, m2));
          g[i].b.v[e] = ffma2(fmul2(g[i].b.v[e], wb[i].v[e]), r2, fmul2(nb, m2));
        }
        g[i].give(x[i], y[i]);
      }
      if (mine) me.store_row(out, x, y);
      if (arrived) entries = me.fetch_entries(p, next_info, -1.0f);
      walk.next(at);
      out += row_step;
      slot = slot + 1 == FLY ? 0 : slot + 1;
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    if (!p.want_w[which]) continue;
    // the rows of a warp lie TPR lanes apart
#pragma unroll
    for (int i = 0; i < U; ++i) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        float a = da[i][e], b = db[i][e];
#pragma unroll
        for (int o = TPR; o < 32; o <<= 1) {
          a += __shfl_xor_sync(0xffffffffu, a, o);
          b += __shfl_xor_sync(0xffffffffu, b, o);
        }
        if (me.group == 0 && me.in[i]) {
          float* to = s_sum + ((size_t)which * kNormWarps + warp) * p.d;
          to[me.first(i, e)] = a;
          to[me.second(i, e)] = b;
        }
      }
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * p.d; i += kNormThreads) {
    const int which = i / p.d, c = i - which * p.d;
    if (!p.want_w[which]) continue;
    float sum = 0.0f;
#pragma unroll
    for (int x = 0; x < kNormWarps; ++x) sum += s_sum[((size_t)which * kNormWarps + x) * p.d + c];
    p.partial[((size_t)blockIdx.x * 2 + which) * p.d + c] = sum;
  }
}

// dweight: the CTAs' sums, a block for 32 dims of one weight, 32 threads each
// taking every 32nd CTA's.
__global__ void __launch_bounds__(1024) pva_norm_weights_kernel(NormStep p, int ctas) {
  __shared__ float s[32][33];
  allow_next_grid();
  wait_prior_grid();
  const int which = blockIdx.y, c = blockIdx.x * 32 + threadIdx.x;
  if (!p.want_w[which]) return;
  float sum = 0.0f;
  if (c < p.d)
    for (int i = threadIdx.y; i < ctas; i += 32) sum += p.partial[((size_t)i * 2 + which) * p.d + c];
  s[threadIdx.y][threadIdx.x] = sum;
  __syncthreads();
  float x = s[threadIdx.x][threadIdx.y];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  if (threadIdx.x == 0 && blockIdx.x * 32 + threadIdx.y < p.d)
    p.dw[which][blockIdx.x * 32 + threadIdx.y] = x;
}

// Whether `bytes` from p on share some with the rows (they may lie between two of them).
bool span_meets(const void* p, size_t bytes, const RowRange& r, size_t size) {
  if (!p || !r.p) return false;
  const long long st = r.stride * (long long)size, wide = r.width * (long long)size;
  const long long at = (long long)((intptr_t)p - (intptr_t)r.p), end = at + (long long)bytes;
  if (end <= 0 || at >= (r.tokens - 1) * st + wide) return false;
  return at < 0 || at % st < wide || at % st + (long long)bytes > st;
}

int norm_grid(const NormStep& p, int ctas, int num_sms) {
  const long long want = ((long long)p.tokens * p.parts + kNormWarps - 1) / kNormWarps;
  const long long most = (long long)num_sms * ctas;
  return (int)(want < most ? want : most);
}

template <typename T, int VEC, int TPR, int U>
cudaError_t launch_norm(const NormStep& p, bool backward, int grid, cudaStream_t st) {
  constexpr int F = U == 1 ? kFly : 2, FB = U == 1 ? kBackFly : 2;
  auto kern = p.rt.interleaved ? pva_norm_rope_kernel<T, VEC, TPR, U, F, true>
                               : pva_norm_rope_kernel<T, VEC, TPR, U, F, false>;
  auto back = p.rt.interleaved ? pva_norm_rope_backward_kernel<T, VEC, TPR, U, FB, true>
                               : pva_norm_rope_backward_kernel<T, VEC, TPR, U, FB, false>;
  return backward ? launch_dependent(back, dim3(grid), dim3(kNormThreads), sizeof(float) * 2 * kNormWarps * p.d, st, p)
                  : launch_dependent(kern, dim3(grid), dim3(kNormThreads), 0, st, p);
}

// 16-byte accesses where sizes and alignment allow, a row across the least power of
// two of lanes that holds it; single elements, a row a warp, otherwise.
template <typename T>
cudaError_t launch_norm_type(const NormStep& p, bool wide, bool backward, int grid, cudaStream_t st) {
  constexpr int VEC = 16 / sizeof(T);
  if (!wide) return launch_norm<T, 1, 32, 4>(p, backward, grid, st);
  const int units = p.d / (2 * VEC);
  if (units <= 4) return launch_norm<T, VEC, 4, 1>(p, backward, grid, st);
  if (units <= 8) return launch_norm<T, VEC, 8, 1>(p, backward, grid, st);
  if (units <= 16) return launch_norm<T, VEC, 16, 1>(p, backward, grid, st);
  return launch_norm<T, VEC, 32, 1>(p, backward, grid, st);
}

// Rows of a warp pass times the passes in flight, as launch_norm chooses them.
int rows_at_once(const NormStep& p, int dtype, bool wide, bool backward) {
  if (!wide) return 1;
  const int units = p.d / (dtype == PVA_F32 ? 8 : 16);
  const int tpr = units <= 4 ? 4 : units <= 8 ? 8 : units <= 16 ? 16 : 32;
  return 32 / tpr;
}

bool norm_wide(const NormStep& p, int vec) {
  uintptr_t ptrs = (uintptr_t)p.v | (uintptr_t)p.k_cache | (uintptr_t)p.v_cache;
  long long strides = p.v_stride;
  for (int i = 0; i < 2; ++i) {
    ptrs |= (uintptr_t)p.x[i] | (uintptr_t)p.dy[i] | (uintptr_t)p.out[i];
    strides |= p.x_stride[i] | p.dy_stride[i] | p.out_stride[i];
  }
  return (ptrs & 15) == 0 && strides % vec == 0 && p.rt.rot / 2 % vec == 0 &&
         (p.d - p.rt.rot) % (2 * vec) == 0;
}

int enqueue_norm(NormStep& p, int dtype, bool backward, cudaStream_t stream) {
  std::lock_guard<std::mutex> lock(api_mutex());
  int sms = 0;
  int rc = sm_count(&sms);
  if (rc != PVA_OK) return rc;
  const bool wide = norm_wide(p, dtype == PVA_F32 ? 4 : 8);
  // A warp takes a whole token where the GPU is full of them, and as few rows as it
  // has in flight where it is not.
  const int at_once = rows_at_once(p, dtype, wide, backward);
  const int rows = p.heads[0] > p.heads[1] ? p.heads[0] : p.heads[1];
  const int most = (rows + at_once - 1) / at_once;
  const int ctas = backward ? kBackCtas : kNormCtas;
  const long long warps = (long long)sms * ctas * kNormWarps;
  const long long parts = warps / p.tokens;
  p.parts = (int)(parts < 1 ? 1 : parts < most ? parts : most);
  const int grid = norm_grid(p, ctas, sms);
  const bool sums = backward && (p.want_w[0] || p.want_w[1]);
  CallContext c;
  if ((rc = acquire(stream, sums ? sizeof(float) * 2 * p.d * (size_t)grid : 0, &c)) != PVA_OK) return rc;
  p.status = c.status;
  p.partial = reinterpret_cast<float*>(c.buf);
  cudaError_t e = dtype == PVA_F32   ? launch_norm_type<float>(p, wide, backward, grid, stream)
                  : dtype == PVA_F16 ? launch_norm_type<__half>(p, wide, backward, grid, stream)
                                     : launch_norm_type<__nv_bfloat16>(p, wide, backward, grid, stream);
  if (e != cudaSuccess) return cuda_fail(e, "norm launch");
  if (!sums) return PVA_OK;
  e = launch_dependent(pva_norm_weights_kernel, dim3((p.d + 31) / 32, 2), dim3(32, 32), 0, stream, p, grid);
  return e == cudaSuccess ? PVA_OK : cuda_fail(e, "norm weight sums launch");
}

int check_norm(NormStep& p, const void* q_weight, const void* k_weight, float eps, float offset,
               int weight_dtype, int dtype, int d, int rot, const void* cos_cache,
               const void* sin_cache, const int64_t* position_ids, int cache_rows,
               int rotary_interleaved, int n_axes, const int32_t* sections, int axes_interleaved,
               int rotary_dtype) {
  if (!isfinite(eps) || eps < 0.0f || !isfinite(offset))
    return fail(PVA_ERR_INVALID_ARG, "eps must be finite and not negative, weight_offset finite");
  if ((q_weight || k_weight) && weight_dtype != PVA_F32 && weight_dtype != dtype)
    return fail(PVA_ERR_INVALID_ARG, "the weights must be f32 or of the rows' type");
  const size_t w_size = weight_dtype == PVA_F32 ? 4 : 2;
  if (((uintptr_t)q_weight | (uintptr_t)k_weight) % w_size)
    return fail(PVA_ERR_INVALID_ARG, "a weight is not aligned to its elements");
  if (rot != 0) {
    if (!position_ids) return fail(PVA_ERR_INVALID_ARG, "null position_ids pointer");
    const int rc = check_rope(cos_cache, sin_cache, rot, cache_rows, rotary_interleaved, n_axes,
                              sections, axes_interleaved, rotary_dtype, dtype, d, &p.rt);
    if (rc != PVA_OK) return rc;
  }
  p.pos = position_ids;
  p.w[0] = q_weight;
  p.w[1] = k_weight;
  p.w_f32 = weight_dtype == PVA_F32;
  p.eps = eps;
  p.offset = offset;
  p.d = d;
  p.inv_d = 1.0f / (float)d;
  return PVA_OK;
}

}  // namespace
}  // namespace pva

extern "C" int pva_norm_rope(const void* q, const void* k, const void* q_weight,
                             const void* k_weight, void* q_out, void* k_out,
                             const void* cos_cache, const void* sin_cache,
                             const int64_t* position_ids, int tokens, int num_heads,
                             int kv_num_heads, int head_size, int64_t q_stride, int64_t k_stride,
                             int64_t q_out_stride, int64_t k_out_stride, float eps,
                             float weight_offset, int weight_dtype, int rotary_dim, int cache_rows,
                             int rotary_interleaved, int n_axes, const int32_t* sections,
                             int axes_interleaved, int rotary_dtype, const void* v,
                             int64_t v_stride, void* k_cache, void* v_cache,
                             const int64_t* slot_map, int n_blocks, int page_size, int dtype,
                             void* stream) {
  return guarded([&]() -> int {
    const RowsIn rows{q, k, v, q_out, k_out, q_stride, k_stride, v_stride, q_out_stride, k_out_stride,
                      tokens, num_heads, kv_num_heads, head_size, k_cache, v_cache, slot_map, n_blocks,
                      page_size, dtype};
    int rc = check_token_rows(rows);
    if (rc != PVA_OK || tokens == 0) return rc;
    NormStep p{};
    rc = check_norm(p, q_weight, k_weight, eps, weight_offset, weight_dtype, dtype, head_size, rotary_dim,
                    cos_cache, sin_cache, position_ids, cache_rows, rotary_interleaved, n_axes, sections,
                    axes_interleaved, rotary_dtype);
    if (rc != PVA_OK) return rc;
    p.x[0] = q;
    p.x[1] = k;
    p.out[0] = q_out;
    p.out[1] = k_out;
    p.x_stride[0] = q ? q_stride : 0;
    p.x_stride[1] = k ? k_stride : 0;
    p.out_stride[0] = q ? q_out_stride : 0;
    p.out_stride[1] = k_out ? k_out_stride : 0;
    p.heads[0] = q ? num_heads : 0;
    p.heads[1] = k ? kv_num_heads : 0;
    p.tokens = tokens;
    if (k_cache) {
      p.v = v;
      p.v_stride = v_stride;
      p.k_cache = k_cache;
      p.v_cache = v_cache;
      p.slots = slot_map;
      p.page = page_size;
      p.n_slots = (long long)n_blocks * page_size;
    }
    return enqueue_norm(p, dtype, false, static_cast<cudaStream_t>(stream));
  });
}

extern "C" int pva_norm_rope_backward(const void* dq_out, const void* dk_out, const void* q,
                                      const void* k, const void* q_weight, const void* k_weight,
                                      void* dq, void* dk, float* dq_weight, float* dk_weight,
                                      const void* cos_cache, const void* sin_cache,
                                      const int64_t* position_ids, int tokens, int num_heads,
                                      int kv_num_heads, int head_size, int64_t dq_out_stride,
                                      int64_t dk_out_stride, int64_t q_stride, int64_t k_stride,
                                      int64_t dq_stride, int64_t dk_stride, float eps,
                                      float weight_offset, int weight_dtype, int rotary_dim,
                                      int cache_rows, int rotary_interleaved, int n_axes,
                                      const int32_t* sections, int axes_interleaved,
                                      int rotary_dtype, int dtype, void* stream) {
  return guarded([&]() -> int {
    if (tokens < 0 || tokens > INT_MAX - 65536)
      return fail(PVA_ERR_INVALID_ARG, "tokens must be >= 0 and fit in int32");
    if ((q != nullptr) != (dq_out != nullptr) || (q != nullptr) != (dq != nullptr) ||
        (k != nullptr) != (dk_out != nullptr) || (k != nullptr) != (dk != nullptr))
      return fail(PVA_ERR_INVALID_ARG, "a side's rows, output gradients and gradients come together");
    if (tokens && ((dq_weight && !q) || (dk_weight && !k)))  // (no tokens: rows may be NULL)
      return fail(PVA_ERR_INVALID_ARG, "a weight's gradient without its rows");
    if ((dq_weight && !q_weight) || (dk_weight && !k_weight))
      return fail(PVA_ERR_INVALID_ARG, "a weight's gradient without the weight");
    if (((uintptr_t)dq_weight | (uintptr_t)dk_weight) & 3)
      return fail(PVA_ERR_INVALID_ARG, "a weight's gradient is not aligned to its elements");
    // The rows that are read (x) and the output gradients (dy): an output may take the
    // place of its own output gradient, and of nothing else.
    const RowsIn grads{dq_out, dk_out, nullptr, dq, dk, dq_out_stride, dk_out_stride, 0, dq_stride, dk_stride,
                       tokens, num_heads, kv_num_heads, head_size, nullptr, nullptr, nullptr, 0, 0, dtype};
    int rc = tokens ? check_token_rows(grads) : PVA_OK;
    if (rc != PVA_OK) return rc;
    const int d = head_size;
    const long long w[2] = {(long long)num_heads * d, (long long)kv_num_heads * d};
    const size_t size = dtype == PVA_F32 ? 4 : 2;
    if (tokens) {
      if ((q && q_stride < w[0]) || (k && k_stride < w[1]))
        return fail(PVA_ERR_INVALID_ARG, "a token stride is smaller than the token's heads");
      if (((uintptr_t)q | (uintptr_t)k) % size)
        return fail(PVA_ERR_INVALID_ARG, "a tensor is not aligned to its elements");
      const RowRange x[2] = {{q, tokens, q_stride, w[0]}, {k, tokens, k_stride, w[1]}};
      const RowRange out[2] = {{dq, tokens, dq_stride, w[0]}, {dk, tokens, dk_stride, w[1]}};
      for (const RowRange& a : out)
        for (const RowRange& b : x)
          if (rows_meet(a, b, size))
            return fail(PVA_ERR_INVALID_ARG, "a gradient overlaps rows that the call reads");
      const RowRange rows[6] = {x[0], x[1], out[0], out[1], {dq_out, tokens, dq_out_stride, w[0]}, {dk_out, tokens, dk_out_stride, w[1]}};
      for (const float* dw : {dq_weight, dk_weight})
        for (const RowRange& a : rows)
          if (span_meets(dw, sizeof(float) * d, a, size))
            return fail(PVA_ERR_INVALID_ARG, "a weight's gradient overlaps rows of the call");
    }
    if (dq_weight && dk_weight && (uintptr_t)dq_weight < (uintptr_t)(dk_weight + d) &&
        (uintptr_t)dk_weight < (uintptr_t)(dq_weight + d))
      return fail(PVA_ERR_INVALID_ARG, "dq_weight and dk_weight overlap");
    NormStep p{};
    if (tokens || dq_weight || dk_weight) {
      if (d < 2 || d > 256 || d % 2 != 0)
        return fail(PVA_ERR_UNSUPPORTED, "head_size must be even, 2 to 256");
      rc = check_norm(p, q_weight, k_weight, eps, weight_offset, weight_dtype, dtype, d,
                      tokens ? rotary_dim : 0, cos_cache, sin_cache, position_ids, cache_rows,
                      rotary_interleaved, n_axes, sections, axes_interleaved, rotary_dtype);
      if (rc != PVA_OK) return rc;
    }
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (tokens == 0) {  // an empty sum
      for (float* dw : {dq_weight, dk_weight})
        if (dw) {
          const cudaError_t e = cudaMemsetAsync(dw, 0, sizeof(float) * d, st);
          if (e != cudaSuccess) return cuda_fail(e, "weight gradient memset");
        }
      return PVA_OK;
    }
    p.x[0] = q;
    p.x[1] = k;
    p.dy[0] = dq_out;
    p.dy[1] = dk_out;
    p.out[0] = dq;
    p.out[1] = dk;
    p.x_stride[0] = q ? q_stride : 0;
    p.x_stride[1] = k ? k_stride : 0;
    p.dy_stride[0] = q ? dq_out_stride : 0;
    p.dy_stride[1] = k ? dk_out_stride : 0;
    p.out_stride[0] = q ? dq_stride : 0;
    p.out_stride[1] = k ? dk_stride : 0;
    p.heads[0] = q ? num_heads : 0;
    p.heads[1] = k ? kv_num_heads : 0;
    p.tokens = tokens;
    p.want_w[0] = dq_weight != nullptr;
    p.want_w[1] = dk_weight != nullptr;
    p.dw[0] = dq_weight;
    p.dw[1] = dk_weight;
    return enqueue_norm(p, dtype, true, st);
  });
}
