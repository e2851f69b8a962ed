// dense_internal.h -- launch interfaces between the dense operators' host side
// (dense_api.cu) and their kernels.
#pragma once

#include "conv_internal.h"
#include "dense_common.cuh"
#include "linear.h"

namespace conv {

// CUDA-core product (dense_ffma.cu): any type, stride and alignment.
struct DenseFfmaPlan {
  int bm, bn;            // tile
  int split;             // k ranges
  long long k_per_split;
};
DenseFfmaPlan dense_ffma_plan(const DenseGemm& g, int sm);
cudaError_t launch_dense_ffma(const DenseFfmaPlan& p, const DenseGemm& g, int dtype, cudaStream_t s);

// Tensor-core product (dense_tc.cuh): 16-bit operands on 16-byte boundaries.
struct DenseTcPlan {
  int cg, nt;       // SMs per tile, MMA columns: tiles of 128 * cg x nt (nt / 2 gated)
  int split;        // k ranges
  int kb_range;     // 64-term blocks of a range
  long long tiles;
  int blocks;       // persistent blocks
};
DenseTcPlan dense_tc_plan(const DenseGemm& g, int sm);
cudaError_t launch_dense_tc(const DenseTcPlan& t, const DenseGemm& g, int dtype, cudaStream_t s);
cudaError_t dense_error_word(uint32_t* word, int reset);

// Few rows (dense_few.cu): at most 16 (8 of float32), any alignment.  `follows`:
// the kernel before in the stream is this call's own, and writes no weights: the
// launch overlaps its end, the first weights' loads included.
constexpr int dense_few_rows(int dtype) { return dtype == CONV_F32 ? 8 : 16; }
cudaError_t launch_dense_few(const DenseGemm& g, int dtype, bool follows, cudaStream_t s);

// Adds the k ranges' planes in order and applies the epilogue.
cudaError_t launch_dense_reduce(const DenseGemm& g, int dtype, cudaStream_t s);

// Rows copied to a pitch of `ld_out` elements (16-bit elements).
cudaError_t launch_dense_repack(const void* in, long long ld_in, void* out, long long ld_out, long long rows,
                                long long cols, cudaStream_t s);

// dz = dy * act'(pre) in the element type (`dz`, may be nullptr: not wanted)
// and float32 column sums of the unrounded dz over row blocks
// (part [blocks][cols]), summed in order into dbias by the second kernel.
constexpr int kColRowsMin = 64;
int dense_col_blocks(long long rows, long long cols, int sm);
cudaError_t launch_dense_dz(const void* dy, long long ld_dy, const float* pre, void* dz, long long ld_dz, void* dbias,
                            float* part, int blocks, long long rows, long long cols, int act, float alpha, float beta,
                            int dtype, cudaStream_t s);

// Clipping (clip.cu).
size_t clip_scratch_bytes(long long count, const int64_t* sizes);
cudaError_t launch_clip(long long count, const void* const* in, void* const* out, const int64_t* sizes,
                        const int32_t* dtypes, float max_norm, float eps, float* norm, void* scratch, int sm,
                        cudaStream_t s);

}  // namespace conv
