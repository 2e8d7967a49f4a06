// The paired kernel (pva_tree_pair.cuh) with the work of pva_gqa_prefix, without a softcap
// (which the one-tile kernel does faster).
#include "pva_prefix.cuh"
#include "pva_tree_pair.cuh"

namespace pva {
namespace {

using namespace paired;

template <typename T, int D>
cudaError_t launch_d(const PrefixParams& p, const PrefixQueries& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                     cudaStream_t s) {
  constexpr int smem = PairCfg<D, 1>::SMEM;
  auto kern = pva_tree_pair_kernel<T, D, 1, kNoCap, PrefixWork>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  return launch_dependent(kern, dim3(p.pieces), dim3(kThreads), smem, s, p, tq, tk, tv);
}

template <typename T>
cudaError_t launch_type(const PrefixParams& p, const PrefixQueries& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                        cudaStream_t s) {
  switch (p.d) {
    case 64: return launch_d<T, 64>(p, tq, tk, tv, s);
    case 96: return launch_d<T, 96>(p, tq, tk, tv, s);
    case 128: return launch_d<T, 128>(p, tq, tk, tv, s);
    case 192: return launch_d<T, 192>(p, tq, tk, tv, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

cudaError_t launch_prefix_pair(const PrefixParams& p, int dtype, const PrefixQueries& tq, const CUtensorMap& tk,
                               const CUtensorMap& tv, cudaStream_t s) {
  if (p.softcap != 0.0f) return cudaErrorInvalidValue;
  return dtype == PVA_BF16 ? launch_type<__nv_bfloat16>(p, tq, tk, tv, s) : launch_type<__half>(p, tq, tk, tv, s);
}

}  // namespace pva
