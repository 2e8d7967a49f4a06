// The paired kernel of pva_gqa_tree (pva_tree_pair.cuh) for its types and head sizes.
#include "pva_tree_pair.cuh"

namespace pva {
namespace {

using namespace paired;

template <typename T, int D, int PARTS>
cudaError_t launch_parts(const TreeParams& p, const CUtensorMap& tq, const CUtensorMap& tk,
                         const CUtensorMap& tv, cudaStream_t s) {
  constexpr int smem = PairCfg<D, PARTS>::SMEM;
  const int cap = cap_form(p.softcap);
  auto kern = cap == kNoCap ? pva_tree_pair_kernel<T, D, PARTS, kNoCap, TreeWork>
              : cap == kCap ? pva_tree_pair_kernel<T, D, PARTS, kCap, TreeWork>
                            : pva_tree_pair_kernel<T, D, PARTS, kLargeCap, TreeWork>;
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
