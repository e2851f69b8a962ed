// dense_tc_launch.cuh -- launches of the tensor-core product for one element
// type (included by one source file per type, which compile in parallel).
#pragma once

#include "dense_tc.cuh"

namespace conv {
namespace dtc {

template <typename T, int CG, int NT, int MODE>
cudaError_t go(const DenseTcArgs& args, const DenseTcMaps& maps, int blocks, cudaStream_t s) {
  using C = Cfg<CG, NT>;
  auto kern = dense_tc<T, CG, NT, MODE>;
  cudaError_t err = opt_in_smem(reinterpret_cast<const void*>(kern), C::kSmem);
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = CG;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = CG > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, args, maps);
}

template <typename T, int CG, int NT>
cudaError_t by_mode(int mode, const DenseTcArgs& args, const DenseTcMaps& maps, int blocks, cudaStream_t s) {
  switch (mode) {
    case EPI_GATED: return go<T, CG, NT, EPI_GATED>(args, maps, blocks, s);
    case EPI_GATED_BWD: return go<T, CG, NT, EPI_GATED_BWD>(args, maps, blocks, s);
    case EPI_PARTIAL: return go<T, CG, NT, EPI_PARTIAL>(args, maps, blocks, s);
    default: return go<T, CG, NT, EPI_LINEAR>(args, maps, blocks, s);
  }
}

template <typename T>
cudaError_t by_tile(const DenseTcPlan& t, int mode, const DenseTcArgs& args, const DenseTcMaps& maps, cudaStream_t s) {
  if (t.cg == 2) return by_mode<T, 2, 256>(mode, args, maps, t.blocks, s);
  return by_mode<T, 1, 128>(mode, args, maps, t.blocks, s);
}

}  // namespace dtc
}  // namespace conv
