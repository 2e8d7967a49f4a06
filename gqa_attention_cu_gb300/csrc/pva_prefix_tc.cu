// The one-tile kernel (pva_tree_tc.cuh) with the work of pva_gqa_prefix.
#include "pva_prefix.cuh"
#include "pva_tree_tc.cuh"

namespace pva {
namespace {

using namespace one_tile;

template <typename T, int D>
cudaError_t launch_d(const PrefixParams& p, const PrefixQueries& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                     cudaStream_t s) {
  constexpr int smem = TreeCfg<D>::SMEM;
  const int cap = cap_form(p.softcap);
  auto kern = cap == kNoCap ? pva_tree_tc_kernel<T, D, kNoCap, PrefixWork>
              : cap == kCap ? pva_tree_tc_kernel<T, D, kCap, PrefixWork>
                            : pva_tree_tc_kernel<T, D, kLargeCap, PrefixWork>;
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
    case 256: return launch_d<T, 256>(p, tq, tk, tv, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

cudaError_t launch_prefix_tc(const PrefixParams& p, int dtype, const PrefixQueries& tq, const CUtensorMap& tk,
                             const CUtensorMap& tv, cudaStream_t s) {
  return dtype == PVA_BF16 ? launch_type<__nv_bfloat16>(p, tq, tk, tv, s) : launch_type<__half>(p, tq, tk, tv, s);
}

}  // namespace pva
