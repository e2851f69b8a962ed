// dense_internal.h -- launch interfaces between the dense operators' host side
// (dense_api.cu) and their kernels.
#pragma once

#include "conv_internal.h"
#include "dense_common.cuh"
#include "linear.h"

namespace conv {

// Programmatic dependent launch: a kernel's start (its set-up, before
// griddep_wait) overlaps the end of the kernel before it in the stream.  Every
// dense kernel calls griddep_wait before it touches memory that another kernel
// writes or reads, so any kernel may stand before it.
__device__ __forceinline__ void griddep_wait() { asm volatile("griddepcontrol.wait;\n" ::: "memory"); }
__device__ __forceinline__ void griddep_launch() { asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory"); }
template <typename... P, typename... A>
cudaError_t launch_overlapped(void (*kern)(P...), dim3 grid, int threads, size_t smem, int cluster, cudaStream_t s,
                              A&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<P>(args)...);
}

// CUDA-core product (dense_ffma.cu): any type, stride and alignment.
struct DenseFfmaPlan {
  int bm, bn;            // tile
  int split;             // k ranges
  long long k_per_split;
};
DenseFfmaPlan dense_ffma_plan(const DenseGemm& g, int sm, bool ranges);
cudaError_t launch_dense_ffma(const DenseFfmaPlan& p, const DenseGemm& g, int dtype, cudaStream_t s);

// Tensor-core product: 16-bit operands on 16-byte boundaries (dense_tc.cuh), or
// the three bfloat16 planes of float32 ones (dense_tc32.cu).
struct DenseTcPlan {
  int cg, nt;       // SMs per tile, MMA columns: tiles of 128 * cg x nt (nt / 2 gated)
  int tiles, whole; // tiles; the first ones, done whole
  int split;        // k ranges of the others
  int kb_range;     // 64-term blocks of a range
  int blocks;       // persistent blocks
  size_t part_bytes;  // the ranges' sums
};
DenseTcPlan dense_tc_plan(const DenseGemm& g, int dtype, int sm);
cudaError_t launch_dense_tc(const DenseTcPlan& t, const DenseGemm& g, int dtype, void* part, cudaStream_t s);
cudaError_t dense_error_word(uint32_t* word, int reset);

// Few rows (dense_few.cu): at most 16, any alignment.  `follows`:
// the kernel before in the stream is this call's own, and writes no weights: the
// launch overlaps its end, the first weights' loads included.
constexpr int kFewRows = 16;
cudaError_t launch_dense_few(const DenseGemm& g, int dtype, bool follows, int sm, cudaStream_t s);

// Adds the k ranges' planes in order and applies the epilogue.
cudaError_t launch_dense_reduce(const DenseGemm& g, int dtype, cudaStream_t s);

// Operands' copies, in one launch: 16-bit rows copied to a pitch of `ld`
// elements, or (planes) the three bfloat16 planes of float32 rows, rows of ld (a
// multiple of 64) elements, planes rows * ld elements apart, the second and third
// multiplied by these powers of two.
constexpr int kPlaneScale1 = 7, kPlaneScale2 = 16;
struct CopyJob {
  const void* in;
  void* out;
  long long ld_in, ld, rows, cols;
};
constexpr int kCopyJobs = 6;
cudaError_t launch_dense_copies(const CopyJob* jobs, int count, bool planes, cudaStream_t s);

// dz = dy * act'(pre) in the element type (`dz`, may be nullptr: not wanted;
// planes: as the three planes of CopyJob) and float32 column sums of the unrounded dz over row blocks
// (part [blocks][cols]), summed in order into dbias by the second kernel.
constexpr int kColRowsMin = 32;
int dense_col_blocks(long long rows, long long cols, int sm);
cudaError_t launch_dense_dz(const void* dy, long long ld_dy, const float* pre, void* dz, long long ld_dz, bool planes, void* dbias,
                            float* part, int blocks, long long rows, long long cols, int act, float alpha, float beta,
                            int dtype, cudaStream_t s);

// Clipping (clip.cu).
size_t clip_scratch_bytes(long long count, const int64_t* sizes);
cudaError_t launch_clip(long long count, const void* const* in, void* const* out, const int64_t* sizes,
                        const int32_t* dtypes, float max_norm, float eps, float* norm, void* scratch, int sm,
                        cudaStream_t s);

}  // namespace conv
