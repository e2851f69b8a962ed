// dense_tc_launch.cuh -- launches of the tensor-core product for one element
// type (included by one source file per type, which compile in parallel).
#pragma once

#include "dense_tc.cuh"

namespace conv {
namespace dtc {

template <typename T, int CG, int NT, int MODE, bool A_MN, bool B_MN>
cudaError_t go(const DenseTcArgs& args, const DenseTcMaps& maps, int blocks, cudaStream_t s) {
  using C = Cfg<CG, NT>;
  auto kern = dense_tc<T, CG, NT, MODE, A_MN, B_MN>;
  cudaError_t err = opt_in_smem(reinterpret_cast<const void*>(kern), C::kSmem);
  if (err != cudaSuccess) return err;
  return launch_overlapped(kern, dim3(static_cast<unsigned>(blocks)), C::kThreads, C::kSmem, CG, s, args, maps);
}

// The operand orders that occur: the layer's, its input gradient's, its weight gradient's.
template <typename T, int CG, int NT, int MODE>
cudaError_t by_order(int a_mn, int b_mn, const DenseTcArgs& args, const DenseTcMaps& maps, int blocks, cudaStream_t s) {
  if (a_mn) return b_mn ? go<T, CG, NT, MODE, true, true>(args, maps, blocks, s) : cudaErrorInvalidValue;
  return b_mn ? go<T, CG, NT, MODE, false, true>(args, maps, blocks, s)
              : go<T, CG, NT, MODE, false, false>(args, maps, blocks, s);
}
template <typename T, int CG, int NT>
cudaError_t by_mode(int mode, int a_mn, int b_mn, const DenseTcArgs& args, const DenseTcMaps& maps, int blocks,
                    cudaStream_t s) {
  switch (mode) {
    case EPI_GATED:
      return a_mn || b_mn ? cudaErrorInvalidValue : go<T, CG, NT, EPI_GATED, false, false>(args, maps, blocks, s);
    case EPI_GATED_BWD:
      return a_mn || !b_mn ? cudaErrorInvalidValue : go<T, CG, NT, EPI_GATED_BWD, false, true>(args, maps, blocks, s);
    default: return by_order<T, CG, NT, EPI_LINEAR>(a_mn, b_mn, args, maps, blocks, s);
  }
}

template <typename T>
cudaError_t by_tile(const DenseTcPlan& t, int mode, int a_mn, int b_mn, const DenseTcArgs& args, const DenseTcMaps& maps,
                    cudaStream_t s) {
  if (t.cg == 2) return by_mode<T, 2, 256>(mode, a_mn, b_mn, args, maps, t.blocks, s);
  return by_mode<T, 1, 128>(mode, a_mn, b_mn, args, maps, t.blocks, s);
}

}  // namespace dtc
}  // namespace conv
