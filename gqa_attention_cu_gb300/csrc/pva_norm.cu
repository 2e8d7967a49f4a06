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
// meet in one thread; a warp works on a token's rows by itself, without a barrier,
// with the token's cos and sin and the gains in registers.
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

constexpr int kNormThreads = 128;
constexpr int kNormWarps = kNormThreads / 32;

// Where the two packs of unit u of a row lie (2 VEC dims of it).
template <int VEC>
struct Unit {
  int d0, d1;
  bool turned;
  __device__ __forceinline__ Unit(const RopeTable& rt, int u) {
    const int half = rt.rot / 2;
    turned = u * VEC < half;
    if (!turned) {
      d0 = rt.rot + (u - half / VEC) * 2 * VEC;
      d1 = d0 + VEC;
    } else if (rt.interleaved) {
      d0 = u * 2 * VEC;
      d1 = d0 + VEC;
    } else {
      d0 = u * VEC;
      d1 = d0 + half;
    }
  }
};

// The pairs of a unit, as floats.
template <typename T, int VEC>
struct Pairs {
  float a[VEC], b[VEC];
  __device__ __forceinline__ void take(Pack<T, VEC> x, Pack<T, VEC> y, bool neighbours) {
    if (neighbours) split_pairs(x, y);
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      a[e] = load_f(x.v[e]);
      b[e] = load_f(y.v[e]);
    }
  }
  __device__ __forceinline__ void give(Pack<T, VEC>& x, Pack<T, VEC>& y, bool neighbours) const {
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      x.v[e] = round_to<T>(a[e]);
      y.v[e] = round_to<T>(b[e]);
    }
    if (neighbours) join_pairs(x, y);
  }
};

// Sum over the TPR lanes of a row.
template <int TPR>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int o = TPR / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// What a lane keeps of a token: cos and sin of its pairs.
template <int VEC, int U>
struct Turn {
  float c[U][VEC], s[U][VEC];
};

// Positions of token tok on all axes, in bounds or not (the same answer in every lane).
__device__ __forceinline__ bool token_position(const NormStep& p, int tok, int64_t (&at)[kMaxAxes]) {
  bool ok = true;
  if (p.rt.rot) {
#pragma unroll
    for (int a = 0; a < kMaxAxes; ++a) {
      at[a] = 0;
      if (a < p.rt.n_axes) {
        at[a] = p.pos[(size_t)a * p.tokens + tok];
        ok = ok && at[a] >= 0 && at[a] < p.rt.rows;
      }
    }
  }
  return ok;
}

// TPR lanes a row, U units of 2 VEC dims a lane.
template <typename T, int VEC, int TPR, int U>
struct NormLane {
  using P = Pack<T, VEC>;
  int sub, group;      // lane within the row, row within the warp's 32 / TPR
  bool in[U];          // the unit exists
  int d0[U], d1[U];
  bool turned[U], neighbours[U];
  uint32_t axes[U];    // two bits a pair
  __device__ __forceinline__ NormLane(const NormStep& p) {
    const int lane = threadIdx.x & 31;
    sub = lane % TPR;
    group = lane / TPR;
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int u = sub + i * TPR;
      const Unit<VEC> unit(p.rt, u);
      in[i] = u < p.d / (2 * VEC);
      d0[i] = in[i] ? unit.d0 : 0;
      d1[i] = in[i] ? unit.d1 : VEC;
      turned[i] = in[i] && unit.turned;
      neighbours[i] = p.rt.interleaved && turned[i];
      axes[i] = 0;
      if (turned[i])
#pragma unroll
        for (int e = 0; e < VEC; ++e) axes[i] |= (uint32_t)axis_of_pair(p.rt, u * VEC + e) << (2 * e);
    }
  }
  // cos and sin of a token (sign -1: the rotation's transpose)
  __device__ __forceinline__ void turn(const NormStep& p, const int64_t (&at)[kMaxAxes], float sign,
                                       Turn<VEC, U>& t) const {
    const int half = p.rt.rot / 2;
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int u = sub + i * TPR;
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        t.c[i][e] = 1.0f;
        t.s[i][e] = 0.0f;
        if (turned[i]) {
          const int a = axes[i] >> (2 * e) & 3;
          const int64_t row = a == 0 ? at[0] : a == 1 ? at[1] : a == 2 ? at[2] : at[3];
          const int64_t k = row * half + u * VEC + e;
          t.c[i][e] = table_at<false>(p.rt.cos, k, p.rt.is_f16);
          t.s[i][e] = sign * table_at<false>(p.rt.sin, k, p.rt.is_f16);
        }
      }
    }
  }
  __device__ __forceinline__ void gains(const NormStep& p, int which, Pairs<T, VEC> (&w)[U]) const {
#pragma unroll
    for (int i = 0; i < U; ++i) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const int da = neighbours[i] ? d0[i] + 2 * e : d0[i] + e;
        const int db = neighbours[i] ? d0[i] + 2 * e + 1 : d1[i] + e;
        float a = 1.0f, b = 1.0f;
        if (p.w[which] && in[i]) {
          if (p.w_f32) {
            a = static_cast<const float*>(p.w[which])[da];
            b = static_cast<const float*>(p.w[which])[db];
          } else {
            a = load_f(static_cast<const T*>(p.w[which])[da]);
            b = load_f(static_cast<const T*>(p.w[which])[db]);
          }
          a += p.offset;
          b += p.offset;
        }
        w[i].a[e] = a;
        w[i].b[e] = b;
      }
    }
  }
  __device__ __forceinline__ void load_row(const T* src, bool there, P (&x)[U], P (&y)[U]) const {
#pragma unroll
    for (int i = 0; i < U; ++i) {
      if (there && in[i]) {
        x[i] = *reinterpret_cast<const P*>(src + d0[i]);
        y[i] = *reinterpret_cast<const P*>(src + d1[i]);
      } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e) x[i].v[e] = y[i].v[e] = round_to<T>(0.0f);
      }
    }
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

// Rows of one warp pass: 32 / TPR head rows; FLY passes have their loads in flight.
template <typename T, int VEC, int TPR, int U, int FLY>
__global__ void __launch_bounds__(kNormThreads) pva_norm_rope_kernel(NormStep p) {
  using P = Pack<T, VEC>;
  constexpr int RPP = 32 / TPR;
  allow_next_grid();
  wait_prior_grid();
  const NormLane<T, VEC, TPR, U> me(p);
  const int lane = threadIdx.x & 31;
  const int nq = p.heads[0], nk = p.heads[1], nv = p.v ? nk : 0;
  const long long items = (long long)p.tokens * p.parts;
  const long long stride = (long long)gridDim.x * kNormWarps;
  for (long long item = (long long)blockIdx.x * kNormWarps + (threadIdx.x >> 5); item < items;
       item += stride) {
    const int tok = (int)(item / p.parts), part = (int)(item - (long long)tok * p.parts);
    int64_t at[kMaxAxes];
    bool ok = token_position(p, tok, at);
    int64_t slot = -1;
    if (p.k_cache) {
      slot = p.slots[tok];
      ok = ok && slot >= -1 && slot < p.n_slots;
    }
    if (!ok) {
      if (lane == 0) atomicOr(p.status, PVA_DEV_ROPE);
      continue;
    }
    const int64_t block = slot < 0 ? 0 : slot / p.page;
    const size_t cache_row = slot < 0 ? 0 : (size_t)(slot - block * p.page);
    Turn<VEC, U> t;
    me.turn(p, at, 1.0f, t);
#pragma unroll 1
    for (int which = 0; which < 2; ++which) {
      const int n = p.heads[which];
      if (n == 0) continue;
      Pairs<T, VEC> w[U];
      me.gains(p, which, w);
      const T* src = static_cast<const T*>(p.x[which]) + (size_t)tok * p.x_stride[which];
      T* out = static_cast<T*>(p.out[which]);
      if (out) out += (size_t)tok * p.out_stride[which];
      for (int r0 = part * RPP * FLY; r0 < n; r0 += p.parts * RPP * FLY) {
        P x[FLY][U], y[FLY][U];
#pragma unroll
        for (int f = 0; f < FLY; ++f) {
          const int row = r0 + f * RPP + me.group;
          me.load_row(src + (size_t)row * p.d, row < n, x[f], y[f]);
        }
#pragma unroll
        for (int f = 0; f < FLY; ++f) {
          const int row = r0 + f * RPP + me.group;
          Pairs<T, VEC> v[U];
          float sum = 0.0f;
#pragma unroll
          for (int i = 0; i < U; ++i) {
            v[i].take(x[f][i], y[f][i], me.neighbours[i]);
#pragma unroll
            for (int e = 0; e < VEC; ++e) sum = fmaf(v[i].a[e], v[i].a[e], fmaf(v[i].b[e], v[i].b[e], sum));
          }
          const float r = rsqrtf(fmaf(row_sum<TPR>(sum), p.inv_d, p.eps));
#pragma unroll
          for (int i = 0; i < U; ++i) {
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
              const float a = v[i].a[e] * r * w[i].a[e], b = v[i].b[e] * r * w[i].b[e];
              v[i].a[e] = t.c[i][e] * a - t.s[i][e] * b;
              v[i].b[e] = t.s[i][e] * a + t.c[i][e] * b;
            }
            v[i].give(x[f][i], y[f][i], me.neighbours[i]);
          }
          if (row < n) {
            if (out) me.store_row(out + (size_t)row * p.d, x[f], y[f]);
            if (which == 1 && slot >= 0)
              me.store_row(static_cast<T*>(p.k_cache) +
                               (((size_t)block * nk + row) * p.page + cache_row) * p.d,
                           x[f], y[f]);
          }
        }
      }
    }
    if (nv && slot >= 0) {
      const T* src = static_cast<const T*>(p.v) + (size_t)tok * p.v_stride;
      for (int row = part * RPP + me.group; row < nv; row += p.parts * RPP) {
        P x[U], y[U];
        me.load_row(src + (size_t)row * p.d, true, x, y);
        me.store_row(static_cast<T*>(p.v_cache) +
                         (((size_t)block * nk + row) * p.page + cache_row) * p.d,
                     x, y);
      }
    }
    (void)nq;
  }
}

// The gradient.  Each warp sums g n over its rows in registers, each CTA over its
// warps, and pva_norm_weights_kernel over the CTAs, always in the same order.
template <typename T, int VEC, int TPR, int U, int FLY>
__global__ void __launch_bounds__(kNormThreads) pva_norm_rope_backward_kernel(NormStep p) {
  using P = Pack<T, VEC>;
  constexpr int RPP = 32 / TPR;
  extern __shared__ float s_sum[];  // [2][warps][d]
  allow_next_grid();
  wait_prior_grid();
  const NormLane<T, VEC, TPR, U> me(p);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long items = (long long)p.tokens * p.parts;
  const long long stride = (long long)gridDim.x * kNormWarps;
#pragma unroll 1
  for (int which = 0; which < 2; ++which) {
    const int n = p.heads[which];
    if (n == 0) continue;
    Pairs<T, VEC> w[U], dw[U];
    me.gains(p, which, w);
#pragma unroll
    for (int i = 0; i < U; ++i)
#pragma unroll
      for (int e = 0; e < VEC; ++e) dw[i].a[e] = dw[i].b[e] = 0.0f;
    for (long long item = (long long)blockIdx.x * kNormWarps + warp; item < items; item += stride) {
      const int tok = (int)(item / p.parts), part = (int)(item - (long long)tok * p.parts);
      int64_t at[kMaxAxes];
      if (!token_position(p, tok, at)) {
        if (lane == 0) atomicOr(p.status, PVA_DEV_ROPE);
        continue;
      }
      Turn<VEC, U> t;
      me.turn(p, at, -1.0f, t);
      const T* src = static_cast<const T*>(p.x[which]) + (size_t)tok * p.x_stride[which];
      const T* grad = static_cast<const T*>(p.dy[which]) + (size_t)tok * p.dy_stride[which];
      T* out = static_cast<T*>(p.out[which]) + (size_t)tok * p.out_stride[which];
      for (int r0 = part * RPP * FLY; r0 < n; r0 += p.parts * RPP * FLY) {
        P x[FLY][U], y[FLY][U], gx[FLY][U], gy[FLY][U];
#pragma unroll
        for (int f = 0; f < FLY; ++f) {
          const int row = r0 + f * RPP + me.group;
          me.load_row(src + (size_t)row * p.d, row < n, x[f], y[f]);
          me.load_row(grad + (size_t)row * p.d, row < n, gx[f], gy[f]);
        }
#pragma unroll
        for (int f = 0; f < FLY; ++f) {
          const int row = r0 + f * RPP + me.group;
          Pairs<T, VEC> v[U], g[U];
          float sum = 0.0f, inner = 0.0f;
#pragma unroll
          for (int i = 0; i < U; ++i) {
            v[i].take(x[f][i], y[f][i], me.neighbours[i]);
            g[i].take(gx[f][i], gy[f][i], me.neighbours[i]);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
              sum = fmaf(v[i].a[e], v[i].a[e], fmaf(v[i].b[e], v[i].b[e], sum));
              const float a = t.c[i][e] * g[i].a[e] - t.s[i][e] * g[i].b[e];
              const float b = t.s[i][e] * g[i].a[e] + t.c[i][e] * g[i].b[e];
              g[i].a[e] = a;
              g[i].b[e] = b;
              inner = fmaf(a * w[i].a[e], v[i].a[e], fmaf(b * w[i].b[e], v[i].b[e], inner));
            }
          }
          const float r = rsqrtf(fmaf(row_sum<TPR>(sum), p.inv_d, p.eps));
          // mean(g w n) r, so that n mean(g w n) r = x r^2 mean(g w x) r
          const float m = row_sum<TPR>(inner) * p.inv_d * r * r;
#pragma unroll
          for (int i = 0; i < U; ++i) {
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
              dw[i].a[e] = fmaf(g[i].a[e], v[i].a[e] * r, dw[i].a[e]);
              dw[i].b[e] = fmaf(g[i].b[e], v[i].b[e] * r, dw[i].b[e]);
              g[i].a[e] = r * (g[i].a[e] * w[i].a[e] - v[i].a[e] * m);
              g[i].b[e] = r * (g[i].b[e] * w[i].b[e] - v[i].b[e] * m);
            }
            g[i].give(x[f][i], y[f][i], me.neighbours[i]);
          }
          if (row < n) me.store_row(out + (size_t)row * p.d, x[f], y[f]);
        }
      }
    }
    if (!p.want_w[which]) continue;
    // the rows of a warp lie TPR lanes apart
#pragma unroll
    for (int i = 0; i < U; ++i) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
#pragma unroll
        for (int o = TPR; o < 32; o <<= 1) {
          dw[i].a[e] += __shfl_xor_sync(0xffffffffu, dw[i].a[e], o);
          dw[i].b[e] += __shfl_xor_sync(0xffffffffu, dw[i].b[e], o);
        }
        if (me.group == 0 && me.in[i]) {
          float* to = s_sum + ((size_t)which * kNormWarps + warp) * p.d;
          to[me.neighbours[i] ? me.d0[i] + 2 * e : me.d0[i] + e] = dw[i].a[e];
          to[me.neighbours[i] ? me.d0[i] + 2 * e + 1 : me.d1[i] + e] = dw[i].b[e];
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

constexpr int kNormCtas = 5;  // CTAs an SM is given

int norm_grid(const NormStep& p, int num_sms) {
  const long long want = ((long long)p.tokens * p.parts + kNormWarps - 1) / kNormWarps;
  const long long most = (long long)num_sms * kNormCtas;
  return (int)(want < most ? want : most);
}

template <typename T, int VEC, int TPR, int U>
cudaError_t launch_norm(const NormStep& p, bool backward, int grid, cudaStream_t st) {
  if (!backward)
    return launch_dependent(pva_norm_rope_kernel<T, VEC, TPR, U, U == 1 ? 4 : 1>, dim3(grid),
                            dim3(kNormThreads), 0, st, p);
  return launch_dependent(pva_norm_rope_backward_kernel<T, VEC, TPR, U, U == 1 ? 2 : 1>, dim3(grid),
                          dim3(kNormThreads), sizeof(float) * 2 * kNormWarps * p.d, st, p);
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
  return 32 / tpr * (backward ? 2 : 4);
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
  const long long warps = (long long)sms * kNormCtas * kNormWarps;
  const long long parts = warps / p.tokens;
  p.parts = (int)(parts < 1 ? 1 : parts < most ? parts : most);
  const int grid = norm_grid(p, sms);
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
