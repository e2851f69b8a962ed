/*
 * linear.h -- C ABI of the dense operators of libconv on one NVIDIA GB300
 * (sm_103a): the linear layer, the gated feed-forward block and the clipping
 * of gradients by their global norm.  They are what surrounds the convolutions
 * of conv.h in a network with [rows][features] activations (a row is a token,
 * a frame or a pixel): the layer itself, its backward pass, and the step
 * between the gradients and the optimizer.
 *
 * Conventions are those of conv.h: statuses, element types and activations of
 * conv_dtype / conv_act, caller-owned device memory, host-side validation
 * before anything is enqueued, work enqueued on `stream` only (NULL: the legacy
 * default stream), nothing synchronised, nothing allocated.  Sums are float32;
 * 16-bit results are rounded once, to nearest even.  No kernel uses atomics:
 * results are bit-identical from run to run on one device.
 *
 * float32 products of more than 16 rows (of more than 8 where rows are no whole
 * 16-byte pieces; all of a backward pass) multiply their operands as three
 * bfloat16 parts each (all 24 bits of their significands), with sums at least as
 * exact as float32 ones; of a subnormal operand two units of its last place
 * (2^-148) may be lost.
 * Infinities and NaN come out as the formula gives them, whatever the kernel;
 * a sum of products whose absolute values come within 1% of the end of float32's
 * range may be infinite there (the product of the first parts may pass the whole
 * one by 2^-7).
 *
 * Matrices are row-major.  A row stride counts elements from one row to the
 * next; 0 stands for dense rows (stride = width).  Strides of any size, and
 * addresses at any multiple of the element's size, are legal (others are
 * CONV_ERR_ARG).  16-bit operands whose address or row stride in bytes is
 * no multiple of 16 are first copied into scratch rows that are; the scratch
 * queries go by the strides, and by CONV_LINEAR_FLAG_UNALIGNED for addresses
 * (without that flag, or the scratch it asks for, an unaligned address is read
 * by the CUDA-core kernel, which is slower; the scratch of an aligned call is
 * enough for it).
 */
#ifndef CONV_GB300_LINEAR_H
#define CONV_GB300_LINEAR_H

#include "conv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Activations of the dense operators: conv_act, and
 *   gelu       t * Phi(t), Phi the normal distribution function;
 *   gelu_tanh  t/2 * (1 + tanh(sqrt(2/pi) * (t + 0.044715 t^3))).
 * Derivatives at a corner: relu 0 at 0, leaky_relu 1 at 0; hard_sigmoid,
 * hard_swish and clip have the slope of their flat side at their corners. */
#define CONV_ACT_GELU 9
#define CONV_ACT_GELU_TANH 10

/* flags of the problems below */
#define CONV_LINEAR_FLAG_RESIDUAL_LAST 0x1u /* y = act(x W^T + bias) + residual, not
                                               act(x W^T + bias + residual)          */
#define CONV_LINEAR_FLAG_UNALIGNED 0x2u     /* scratch for copies of every 16-bit operand:
                                               addresses need not be 16-byte aligned */
#define CONV_LINEAR_FLAG_FORCE_FFMA 0x4u    /* testing: the CUDA-core kernel always  */
#define CONV_LINEAR_FLAG_NO_FEW_ROWS 0x8u   /* testing: never the kernel for few rows */

/* ---- linear ---------------------------------------------------------------
 *   z[r][o] = sum_i x[r][i] w[o][i] + bias[o] + residual[r][o],   y = act(z)
 * x [rows][c_in], w [c_out][c_in], bias [c_out], residual, y [rows][c_out]. */
typedef struct conv_linear_problem {
  int64_t rows, c_in, c_out;        /* rows >= 0 (0: nothing to do); others >= 1 */
  int64_t x_stride, w_stride, residual_stride, y_stride; /* row strides, 0: dense */
  int32_t act;                      /* conv_act, CONV_ACT_GELU, CONV_ACT_GELU_TANH */
  float act_alpha, act_beta;        /* see conv_act                            */
  int32_t dtype;                    /* conv_dtype of every operand             */
  int32_t has_bias;                 /* bias pointer is read iff nonzero        */
  int32_t has_residual;             /* residual pointer is read iff nonzero    */
  uint32_t flags;                   /* CONV_LINEAR_FLAG_*                      */
} conv_linear_problem;

/* Scratch bytes of conv_linear_forward / conv_linear_backward on the current
 * device.  Errors: CONV_ERR_NULL, CONV_ERR_SHAPE (a size out of range, a row
 * stride below the width), CONV_ERR_OVERFLOW, CONV_ERR_DTYPE, CONV_ERR_ACT,
 * CONV_ERR_ARG (unknown flags), CONV_ERR_DEVICE. */
CONV_API conv_status conv_linear_scratch_bytes(const conv_linear_problem* p, size_t* bytes);
CONV_API conv_status conv_linear_backward_scratch_bytes(const conv_linear_problem* p, size_t* bytes);

/* One line on the kernels that conv_linear_forward (pass 0) or the products dx
 * and dw of conv_linear_backward (pass 1, 2) run on a device with `sm_count`
 * SMs, operands 16-byte aligned.  Host only. */
CONV_API conv_status conv_linear_describe_plan(const conv_linear_problem* p, int32_t pass, int32_t sm_count,
                                               char* buf, size_t len);

/* Enqueue the layer.  `pre`, if not NULL, receives the activation's argument
 * (z; with CONV_LINEAR_FLAG_RESIDUAL_LAST, z without the residual) in float32,
 * [rows][c_out] dense, for conv_linear_backward: float32, because 16 bits here
 * would add a rounding error of the size of the result's own to every gradient.
 * Errors: those of conv_linear_scratch_bytes; CONV_ERR_NULL, CONV_ERR_ARG (an
 * address no multiple of its element's size), CONV_ERR_SCRATCH (too small, or
 * not 256-byte aligned), CONV_ERR_ALIAS (y, pre or scratch
 * overlaps an operand; columns side by side in one wider matrix do not),
 * CONV_ERR_CUDA. */
CONV_API conv_status conv_linear_forward(const conv_linear_problem* p, const void* x, const void* w,
                                         const void* bias, const void* residual, void* y, float* pre,
                                         void* scratch, size_t scratch_bytes, void* stream);

/* Enqueue the gradients for dy (row stride p->y_stride):
 *   dz = dy * act'(pre),  dx = dz w,  dw = dz^T x,  dbias = sum over rows of dz,
 *   dresidual = dz (dy with CONV_LINEAR_FLAG_RESIDUAL_LAST).
 * Outputs are dense, of the problem's element type; NULL ones are not computed.
 * dz is rounded to the element type before the two products (they run on the
 * tensor cores); dbias sums the unrounded values.  `pre` may be NULL for the
 * identity.  x may be NULL without dw, w without dx.  With rows = 0, dw and
 * dbias are set to zero.  Errors: as conv_linear_forward. */
CONV_API conv_status conv_linear_backward(const conv_linear_problem* p, const void* x, const void* w,
                                          const float* pre, const void* dy, void* dx, void* dw, void* dbias,
                                          void* dresidual, void* scratch, size_t scratch_bytes, void* stream);

/* ---- gated feed-forward block ----------------------------------------------
 *   g = x Wg^T,  u = x Wu^T,  h = act(g) * u,  y = h Wd^T + residual
 * x [rows][c_in], Wg and Wu [hidden][c_in], Wd [c_out][hidden] (dense),
 * residual, y [rows][c_out].  g, u and h = act(g) * u are float32; h is rounded
 * to the element type once, as the second product's operand. */
typedef struct conv_gated_problem {
  int64_t rows, c_in, hidden, c_out;
  int64_t x_stride, residual_stride, y_stride; /* row strides, 0: dense */
  int32_t act;
  float act_alpha, act_beta;
  int32_t dtype;
  int32_t has_residual;
  uint32_t flags;                   /* CONV_LINEAR_FLAG_* (not RESIDUAL_LAST)  */
} conv_gated_problem;

/* Bytes of scratch, and of `saved` (g and u in float32, h; the layout is the
 * library's own).  Errors: as conv_linear_scratch_bytes. */
CONV_API conv_status conv_gated_scratch_bytes(const conv_gated_problem* p, size_t* bytes);
CONV_API conv_status conv_gated_backward_scratch_bytes(const conv_gated_problem* p, size_t* bytes);
CONV_API conv_status conv_gated_saved_bytes(const conv_gated_problem* p, size_t* bytes);

/* Enqueue the block.  `saved`, if not NULL, is conv_gated_saved_bytes bytes,
 * 256-byte aligned, that conv_gated_backward reads. */
CONV_API conv_status conv_gated_forward(const conv_gated_problem* p, const void* x, const void* w_gate,
                                        const void* w_up, const void* w_down, const void* residual, void* y,
                                        void* saved, void* scratch, size_t scratch_bytes, void* stream);

/* Enqueue the gradients for dy (row stride p->y_stride):
 *   dh = dy Wd, dg = dh * u * act'(g), du = dh * act(g),
 *   dx = dg Wg + du Wu, dWg = dg^T x, dWu = du^T x, dWd = dy^T h
 * (the residual's gradient is dy itself).  dg and du are rounded to the element
 * type once, as operands; dh stays in float32.  Outputs are dense; NULL ones are
 * not computed.  With rows = 0 the weights' gradients are set to zero. */
CONV_API conv_status conv_gated_backward(const conv_gated_problem* p, const void* x, const void* w_gate,
                                         const void* w_up, const void* w_down, const void* saved, const void* dy,
                                         void* dx, void* dw_gate, void* dw_up, void* dw_down, void* scratch,
                                         size_t scratch_bytes, void* stream);

/* ---- gradient clipping -----------------------------------------------------
 *   norm = sqrt(sum over all tensors and elements of g^2)
 *   out = g * min(1, max_norm / (norm + eps)),  rounded once to g's type
 * over `count` tensors, tensor i with sizes[i] >= 0 elements of type dtypes[i]
 * (conv_dtype) at in[i], written to out[i] (out[i] == in[i]: in place; out ==
 * NULL: the norm alone).  The four arrays are host memory, read during the
 * call.  The sum neither overflows nor underflows for any finite elements (it
 * is carried in float64 over blocks scaled by their largest element).  A NaN
 * or an infinity makes the norm NaN or infinite, and the outputs what the
 * formula gives: NaN for a NaN norm, zeros (NaN where g is infinite) for an
 * infinite one.  norm: one float32 on the device.
 * Errors: CONV_ERR_NULL, CONV_ERR_SHAPE (count or a size < 0, or too large),
 * CONV_ERR_DTYPE, CONV_ERR_ARG (max_norm or eps negative or NaN; an address no
 * multiple of its element's size), CONV_ERR_SCRATCH, CONV_ERR_ALIAS (an output
 * overlaps another tensor's input or output, other than out[i] == in[i];
 * norm or scratch overlaps a tensor), CONV_ERR_DEVICE, CONV_ERR_CUDA. */
CONV_API conv_status conv_clip_scratch_bytes(int64_t count, const int64_t* sizes, size_t* bytes);
CONV_API conv_status conv_clip_grads(int64_t count, const void* const* in, void* const* out, const int64_t* sizes,
                                     const int32_t* dtypes, float max_norm, float eps, float* norm,
                                     void* scratch, size_t scratch_bytes, void* stream);

/* As conv_device_error, for the tensor-core kernel of this header: nonzero when
 * it gave up a bounded wait (its output is then incomplete). */
CONV_API conv_status conv_linear_device_error(uint32_t* word, int32_t reset);

#ifdef __cplusplus
}
#endif

#endif /* CONV_GB300_LINEAR_H */
