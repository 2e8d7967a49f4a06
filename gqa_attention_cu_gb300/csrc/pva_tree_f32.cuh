// The fp32 attention kernel of the paged caches.
#pragma once

#include "pva_tree_tile.cuh"

namespace pva {
constexpr int kTreeKeysF32 = 32;
namespace f32 {

using tile::RowOut;

// fp32 attention on the CUDA cores, exact fp32 products (no TF32).  A CTA of 4
// warps holds 4 R query rows (R = 2, 4 or 6, as many as the step can have) and
// streams tiles of 32 keys, the next tile on its way (cp.async) while one is
// worked on.  A warp owns R rows throughout: its threads score up to 3 rows x 2
// keys each, then its lanes hold a key each for the softmax, then 4 (or 8)
// channels of each of its rows for the weighted sum, so warps meet only where a
// tile is complete.  Each step waits on shared memory and shuffles, so what
// counts is how many warps an SM has to switch between: 24 rows and three CTAs
// an SM against 32 rows and two, 146 against 188 us (7 nodes x 3 query heads on
// 20,000 rows of 3 sequences x 4 kv heads, d = 96); 8 rows and four CTAs for one
// node, 34 against 50 us (8 sequences of 1000 to 2000 rows).  Keys outside the
// item's range are zeros in shared memory, whatever the cache holds there.
constexpr int kWarps = 4;

__host__ __device__ constexpr int row_stride(int d) { return (d + 3) / 4 * 4 + 4; }

inline size_t smem_bytes(int rows, int d) {
  return sizeof(float) * ((size_t)(rows + 4 * kTreeKeysF32) * row_stride(d) + rows * 36);
}
// CTAs an SM holds by their shared memory (1 KB of it each is the system's) and
// by their registers: 4 of 8 rows, 3 of 16 or 24.
inline int ctas(int rows, int d) {
  const int by_smem = (int)((228 * 1024) / (smem_bytes(rows, d) + 2048)), by_regs = rows <= 8 ? 4 : 3;
  return by_smem < by_regs ? by_smem : by_regs;
}

__device__ __forceinline__ void copy_async16(void* dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src),
               "r"(valid ? 16 : 0)
               : "memory");
}

// C: 16-byte channel groups a lane sums (1: d <= 128, 2: d <= 256); WIDE: rows of
// the cache lie on 16-byte boundaries.
template <int R, int C, bool WIDE, typename W>
__global__ void __launch_bounds__(kWarps * 32) pva_tree_f32_kernel(typename W::Params p) {
  constexpr int kRows = kWarps * R;
  extern __shared__ float smem[];
  const int d = p.d, stride = row_stride(d), groups = (d + 3) / 4;
  constexpr int kTile = kTreeKeysF32;
  float* sq = smem;                               // [kRows][stride]
  float* skv = sq + kRows * stride;               // [2][K, V][32][stride]
  float* sp = skv + 4 * kTile * stride;           // [kRows][36] weights
  __shared__ typename W::Segment s_segment;
  __shared__ int s_more;
  W::start();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const float NEG_INF = __int_as_float(0xff800000);
  const float* kc = static_cast<const float*>(p.k_cache);
  const float* vc = static_cast<const float*>(p.v_cache);
  // the padding channels of every row stay zero
  for (int e = tid; e < (kRows + 4 * kTile) * (stride - d); e += kWarps * 32)
    smem[e / (stride - d) * stride + d + e % (stride - d)] = 0.0f;
  typename W::Walk walk(p, blockIdx.x);  // the first warp's counts
  while (true) {
    __syncthreads();
    if (warp == 0) {
      typename W::Segment next;
      const bool more = walk.next(p, next);
      if (lane == 0) {
        s_more = more;
        s_segment = next;
      }
    }
    __syncthreads();
    if (!s_more) break;
    const typename W::Segment s = s_segment;
    const int n_rows = min(p.rows, s.n * p.G - s.t * p.rows);
    const int total = W::total(s);
    auto load = [&](int j) {  // key tile j into its buffer
      float* dst = skv + (j & 1) * 2 * kTile * stride;
      // a warp takes every fourth key, its lanes the row's channels
      for (int i = warp; i < kTile; i += kWarps) {
        const int key = j * kTile + i;
        const bool valid = key >= s.lo && key < total;
        size_t at = 0;
        if (valid) {
          const int in = key / p.page;
          const int block = W::block(p, s, in);
          at = (((size_t)block * p.Hkv + s.h) * p.page + (key - in * p.page)) * d;
        }
        if (WIDE) {
          for (int c = lane; c < groups; c += 32) {
            copy_async16(dst + i * stride + 4 * c, kc + at + 4 * c, valid);
            copy_async16(dst + (kTile + i) * stride + 4 * c, vc + at + 4 * c, valid);
          }
        } else {
          for (int c = lane; c < d; c += 32) {
            dst[i * stride + c] = valid ? kc[at + c] : 0.0f;
            dst[(kTile + i) * stride + c] = valid ? vc[at + c] : 0.0f;
          }
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    load(s.j0);
    // This warp's row r is row warp + 4 r of the item (dealt out, so that no warp
    // idles), in slot warp R + r of shared memory (side by side, so that the lanes'
    // reads of different rows meet different banks).
    const int my_rows = n_rows > warp ? (n_rows - warp + kWarps - 1) / kWarps : 0;
    auto row_of = [&](int r) { return warp + kWarps * r; };
    auto slot_of = [&](int r) { return warp * R + r; };
#pragma unroll 1
    for (int r = 0; r < R; ++r) {
      const float* q0 = r < my_rows ? W::q_row(p, s, s.t * p.rows + row_of(r)) : nullptr;
      for (int c = lane; c < d; c += 32) sq[slot_of(r) * stride + c] = q0 ? q0[c] : 0.0f;
    }
    float m[R], l[R], acc[R][4 * C];
    int row_lo[R], row_hi[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      m[r] = NEG_INF;
      l[r] = 0.0f;
#pragma unroll
      for (int u = 0; u < 4 * C; ++u) acc[r][u] = 0.0f;
      const int node = r < my_rows ? (s.t * p.rows + row_of(r)) / p.G : 0;
      const tile::RowView view = W::view(p, s, node);
      row_lo[r] = view.lo;
      row_hi[r] = view.hi;
    }
    for (int j = s.j0; j < s.j0 + s.count; ++j) {
      if (j + 1 < s.j0 + s.count) {
        load(j + 1);
        asm volatile("cp.async.wait_group 1;" ::: "memory");
      } else {
        asm volatile("cp.async.wait_group 0;" ::: "memory");
      }
      __syncthreads();  // tile j (and Q) is complete
      const float* sk = skv + (j & 1) * 2 * kTile * stride;
      const float* sv = sk + kTile * stride;
      if (my_rows > 0) {  // warp-uniform
        // scores: LANES lanes side by side on a row's keys, RT rows a thread
        constexpr int LANES = R % 4 == 0 ? 8 : 16, RT = R * LANES / 32, KT = kTile / LANES;
        const int y = lane / LANES, x = lane % LANES;
        float sc[RT][KT] = {};
        const float* qa = sq + slot_of(RT * y) * stride;
#pragma unroll 4
        for (int c = 0; c < groups; ++c) {
          float4 a[RT];
#pragma unroll
          for (int r = 0; r < RT; ++r)
            a[r] = *reinterpret_cast<const float4*>(qa + r * stride + 4 * c);
#pragma unroll
          for (int k = 0; k < KT; ++k) {
            const float4 b = *reinterpret_cast<const float4*>(sk + (x + LANES * k) * stride + 4 * c);
#pragma unroll
            for (int r = 0; r < RT; ++r)
              sc[r][k] = fmaf(a[r].w, b.w,
                              fmaf(a[r].z, b.z, fmaf(a[r].y, b.y, fmaf(a[r].x, b.x, sc[r][k]))));
          }
        }
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
          for (int k = 0; k < KT; ++k) sp[slot_of(RT * y + r) * 36 + x + LANES * k] = sc[r][k];
        __syncwarp();
        // softmax: lane = key
        const int key = j * kTile + lane, other = key - s.past;
        float w[R], top[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
          bool seen = key >= row_lo[r] && key < row_hi[r];
          if (p.parents && other >= 0 && other < s.n && r < my_rows) {
            const int node = (s.t * p.rows + row_of(r)) / p.G;
            seen = (p.mask[((size_t)s.b * p.T + node) * p.W32 + (other >> 5)] >> (other & 31)) & 1;
          }
          float v = sp[slot_of(r) * 36 + lane] * p.scale;
          if (p.softcap != 0.0f) v = p.softcap * tanhf(v / p.softcap);
          w[r] = seen ? v * 1.4426950408889634f : NEG_INF;  // base-2 units, as the join expects
          top[r] = w[r];
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
#pragma unroll
          for (int r = 0; r < R; ++r) top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], o));
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const float m_new = fmaxf(m[r], top[r]);
          const float base = m_new == NEG_INF ? 0.0f : m_new;
          const float alpha = exp2f(m[r] - base);
          m[r] = m_new;
          w[r] = exp2f(w[r] - base);  // 0 where unseen
          top[r] = w[r];
          l[r] *= alpha;
#pragma unroll
          for (int u = 0; u < 4 * C; ++u) acc[r][u] *= alpha;
          sp[slot_of(r) * 36 + lane] = w[r];
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
#pragma unroll
          for (int r = 0; r < R; ++r) top[r] += __shfl_xor_sync(0xffffffffu, top[r], o);
#pragma unroll
        for (int r = 0; r < R; ++r) l[r] += top[r];
        __syncwarp();
        // weighted sums: lane = channels 4 lane .. (and 128 on)
#pragma unroll 2
        for (int i = 0; i < kTile; i += 4) {
          float4 v[4][C];
#pragma unroll
          for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int u = 0; u < C; ++u)
              if (lane + 32 * u < groups)
                v[k][u] = *reinterpret_cast<const float4*>(sv + (i + k) * stride + 4 * (lane + 32 * u));
#pragma unroll
          for (int r = 0; r < R; ++r) {
            const float4 wr = *reinterpret_cast<const float4*>(sp + slot_of(r) * 36 + i);
            const float wk[4] = {wr.x, wr.y, wr.z, wr.w};
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
              for (int u = 0; u < C; ++u) {
                acc[r][4 * u + 0] = fmaf(wk[k], v[k][u].x, acc[r][4 * u + 0]);
                acc[r][4 * u + 1] = fmaf(wk[k], v[k][u].y, acc[r][4 * u + 1]);
                acc[r][4 * u + 2] = fmaf(wk[k], v[k][u].z, acc[r][4 * u + 2]);
                acc[r][4 * u + 3] = fmaf(wk[k], v[k][u].w, acc[r][4 * u + 3]);
              }
          }
        }
      }
      __syncthreads();  // before tile j + 2 goes over tile j
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (r >= my_rows) break;
      const int lr = row_of(r);
      const RowOut to = W::row_out(p, s, s.t * p.rows + lr, lr);
      const bool whole = to.ml == nullptr;
      float* o = to.o;
      const float f = !whole ? 1.0f : l[r] != 0.0f ? 1.0f / l[r] : 0.0f;
      if (!whole && lane == 0) *to.ml = make_float2(m[r], l[r]);
#pragma unroll
      for (int u = 0; u < 4 * C; ++u) {
        const int c = 4 * (lane + 32 * (u >> 2)) + (u & 3);
        if (c < d) o[c] = acc[r][u] * f;
      }
    }
  }
}

template <int R, typename W>
cudaError_t launch_rows(const typename W::Params& p, cudaStream_t s) {
  const size_t smem = smem_bytes(kWarps * R, p.d);
  const bool wide = p.d % 4 == 0 && (((uintptr_t)p.k_cache | (uintptr_t)p.v_cache) & 15) == 0;
  auto kern = p.d <= 128 ? (wide ? pva_tree_f32_kernel<R, 1, true, W> : pva_tree_f32_kernel<R, 1, false, W>)
                         : (wide ? pva_tree_f32_kernel<R, 2, true, W> : pva_tree_f32_kernel<R, 2, false, W>);
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  return launch_dependent(kern, dim3(p.pieces), dim3(kWarps * 32), smem, s, p);
}
template <typename W>
cudaError_t launch(const typename W::Params& p, cudaStream_t s) {
  return p.rows == 8    ? launch_rows<2, W>(p, s)
         : p.rows == 16 ? launch_rows<4, W>(p, s)
                        : launch_rows<6, W>(p, s);
}

}  // namespace f32
}  // namespace pva
