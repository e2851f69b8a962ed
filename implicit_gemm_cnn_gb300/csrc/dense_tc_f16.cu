// dense_tc_f16.cu -- the tensor-core products of binary16 operands.
#include "dense_tc_launch.cuh"

namespace conv {
cudaError_t launch_dense_tc_f16(const DenseTcPlan& t, int mode, int a_mn, int b_mn, const DenseTcArgs& args,
                                const DenseTcMaps& maps, cudaStream_t s) {
  return dtc::by_tile<__half>(t, mode, a_mn, b_mn, args, maps, s);
}
}  // namespace conv
