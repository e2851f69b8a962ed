/*
 * rows.h -- C ABI of libconv's operators on [rows][features] activations that
 * stand between the dense layers of linear.h on one NVIDIA GB300 (sm_103a):
 * layer norm with its backward pass, dropout with the residual added, the
 * quantisation of rows to 8 bits and the linear layer on them.  A block in
 * training is norm, products, dropout + residual; the same block served is
 * norm, 8-bit products.
 *
 * Conventions are those of linear.h: statuses and element types of conv_dtype,
 * caller-owned device memory, host-side validation before anything is enqueued,
 * work enqueued on `stream` only (NULL: the legacy default stream), nothing
 * synchronised, nothing allocated, no atomics (results are bit-identical from
 * run to run on one device).  Row strides count elements, 0 stands for dense
 * rows; strides of any size and addresses at any multiple of the element's size
 * are legal (rows of whole 16-byte pieces are the quickest).  Sums, statistics
 * and epilogues are float32; results are rounded once, to nearest even.  An
 * output that overlaps an input is CONV_ERR_ALIAS.  rows = 0 is legal.
 */
#ifndef CONV_GB300_ROWS_H
#define CONV_GB300_ROWS_H

#include "linear.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- layer norm ------------------------------------------------------------
 *   mean = sum_i x[r][i] / width,  var = sum_i (x[r][i] - mean)^2 / width
 *   y[r][i] = (x[r][i] - mean) / sqrt(var + eps) * weight[i] + bias[i]
 * x, y [rows][width]; weight, bias [width], each used iff has_* is nonzero. The
 * variance is summed from the differences to the mean, and the rounding of the
 * mean is taken out of them, so that a mean far larger than the spread costs no
 * bits of y.  (A row's sum of squared differences has to fit float32.) */
typedef struct conv_norm_problem {
  int64_t rows, width;              /* rows >= 0, width >= 1                   */
  int64_t x_stride, y_stride;       /* row strides, 0: dense; y_stride is dy's in the backward pass */
  float eps;                        /* >= 0, finite                            */
  int32_t dtype;                    /* conv_dtype of every operand             */
  int32_t has_weight, has_bias;
  uint32_t flags;                   /* CONV_NORM_FLAG_*                        */
} conv_norm_problem;

#define CONV_NORM_FLAG_STREAM 0x1u  /* testing: the kernels of rows too wide for registers */

/* `stats`, if not NULL, receives the mean and 1 / sqrt(var + eps) of each row
 * (float32, [rows][2], 8-byte aligned) for conv_norm_backward.
 * Errors: CONV_ERR_NULL, CONV_ERR_SHAPE, CONV_ERR_OVERFLOW, CONV_ERR_DTYPE,
 * CONV_ERR_ARG (eps negative, infinite or NaN; unknown flags; an address inside
 * an element), CONV_ERR_ALIAS, CONV_ERR_DEVICE, CONV_ERR_CUDA. */
CONV_API conv_status conv_norm_forward(const conv_norm_problem* p, const void* x, const void* weight, const void* bias,
                                       void* y, float* stats, void* stream);

/* The gradients for dy (row stride p->y_stride), with xhat = (x - mean) * rstd and g = dy * weight (the saved mean is
 * rounded; what that leaves in xhat is summed over the row and taken out again):
 *   dx = rstd (g - sum_i g / width - xhat sum_i (g xhat) / width)
 *   dweight = sum over rows of dy xhat,   dbias = sum over rows of dy
 * Outputs are dense, of the problem's element type; NULL ones are not computed.  weight is read iff
 * p->has_weight and dx is wanted.  With rows = 0, dweight and dbias are set to zero.  Scratch: the sums of blocks of
 * rows (and 16 bytes for each row too wide for registers), 256-byte aligned.  Errors: as above, and CONV_ERR_SCRATCH. */
CONV_API conv_status conv_norm_backward_scratch_bytes(const conv_norm_problem* p, size_t* bytes);
CONV_API conv_status conv_norm_backward(const conv_norm_problem* p, const void* x, const void* weight, const float* stats,
                                        const void* dy, void* dx, void* dweight, void* dbias, void* scratch,
                                        size_t scratch_bytes, void* stream);

/* ---- dropout ---------------------------------------------------------------
 *   y[r][i] = residual[r][i] + (u[r][i] < t ? 0 : x[r][i] * 65536 / (65536 - t)),   t = round(65536 p)
 * u are the 16-bit halves, low half first, of Philox4x32-10's four words (Salmon,
 * Moraes, Dror, Shaw, "Parallel random numbers: as easy as 1, 2, 3", SC 2011)
 * for the counter (i / 8, r, offset, offset >> 32) and the key (seed, seed >> 32):
 * one counter per row and 8 columns.  A mask is never stored: the backward pass
 * draws it again from the same seed and offset.  Calls that are to draw apart
 * take different offsets (or seeds).  p is thus a multiple of 2^-16, and the
 * scale its own, so that the expectation of y is x exactly; a dropped value is
 * zero even where x is infinite or NaN.  With t = 65536 nothing is kept. */
typedef struct conv_dropout_problem {
  int64_t rows, width;              /* rows >= 0, width >= 1                   */
  int64_t x_stride, residual_stride, y_stride; /* row strides, 0: dense        */
  uint64_t seed, offset;
  double p;                         /* 0 <= p <= 1                             */
  int32_t dtype;
  int32_t has_residual;
  uint32_t flags;                   /* 0                                       */
} conv_dropout_problem;

/* `state`, if not NULL, is two uint64 on the device, a seed and an offset, read
 * when the kernel runs: the seed stands for p->seed, the offset is added to
 * p->offset (modulo 2^64).  A captured graph draws anew when they change.
 * Errors: as conv_norm_forward; CONV_ERR_ARG also for p outside [0, 1]. */
CONV_API conv_status conv_dropout_forward(const conv_dropout_problem* p, const void* x, const void* residual, void* y,
                                          const uint64_t* state, void* stream);
/* dx = u < t ? 0 : dy * 65536 / (65536 - t), for dy and dx with the strides
 * p->y_stride and p->x_stride (the residual's gradient is dy). */
CONV_API conv_status conv_dropout_backward(const conv_dropout_problem* p, const void* dy, void* dx, const uint64_t* state,
                                           void* stream);

/* ---- rows in 8 bits --------------------------------------------------------
 *   scale[r] = max_i |x[r][i]| * (1 / 127) (both rounded to float32),  q[r][i] = x[r][i] / scale[r]
 * rounded to the nearest whole number, ties to even, as the exact quotient
 * rounds, within [-127, 127].  A row of zeros has scale 0 and zeros; so has a
 * row whose scale is below float32's smallest value.  A row with an infinity or
 * a NaN has scale NaN and zeros.  The rows of a weight matrix are quantised by
 * the same call: a scale for each output.  Errors: as conv_norm_forward. */
typedef struct conv_quantize_problem {
  int64_t rows, width;              /* rows >= 0, width >= 1                   */
  int64_t x_stride, q_stride;       /* row strides, 0: dense                   */
  int32_t dtype;                    /* conv_dtype of x                         */
  uint32_t flags;                   /* 0                                       */
} conv_quantize_problem;

CONV_API conv_status conv_quantize_rows(const conv_quantize_problem* p, const void* x, int8_t* q, float* scale, void* stream);

/* ---- linear on 8-bit rows ----------------------------------------------------
 *   z[r][o] = (sum_i xq[r][i] w[o][i]) * x_scale[r] * w_scale[o] + bias[o] + residual[r][o],   y = act(z)
 * w [c_out][c_in] int8 (all 256 values), w_scale [c_out] float32; xq [rows][c_in]
 * int8 with x_scale [rows] float32, or (x_quantized = 0) the rows of x, of the
 * problem's type, quantised as by conv_quantize_rows first.  The sum is the exact
 * integer, for every operand; what follows is float32.  Activations, residual,
 * order and flags as conv_linear_forward.  What 8 bits save is memory; time only
 * for some tens of rows and fewer, where reading the weights is the work (the
 * products run at the 16-bit rate, and many rows' operands are widened first). */
typedef struct conv_int8_problem {
  int64_t rows, c_in, c_out;        /* rows >= 0, 1 <= c_in <= 131071 (the sum fits 32 bits), c_out >= 1 */
  int64_t x_stride, w_stride, residual_stride, y_stride; /* row strides, 0: dense */
  int32_t act;                      /* conv_act, CONV_ACT_GELU, CONV_ACT_GELU_TANH */
  float act_alpha, act_beta;
  int32_t dtype;                    /* conv_dtype of bias, residual, y, and of x that is not quantised */
  int32_t x_quantized;
  int32_t has_bias, has_residual;
  uint32_t flags;                   /* CONV_LINEAR_FLAG_RESIDUAL_LAST, CONV_INT8_FLAG_* */
} conv_int8_problem;

#define CONV_INT8_FLAG_FEW 0x10u   /* testing: the kernel for few rows (at most 2^20 of them)  */
#define CONV_INT8_FLAG_MID 0x20u   /* testing: that for some tens to hundreds (at most 2^20,
                                      weights in rows on 16-byte boundaries) */
#define CONV_INT8_FLAG_MANY 0x40u  /* testing: that for many                                    */
/* A flag whose kernel cannot run the call is passed over (conv_int8_describe_plan says what runs). */

/* Scratch bytes on the current device, enough for operands at any address: between 17 and 128 rows that may be 2 c_in c_out
 * bytes for weights off 16-byte boundaries (64 rows of 4096 -> 12288: 101 MB, of which weights on such boundaries use half a
 * megabyte).  Errors: as conv_linear_scratch_bytes. */
CONV_API conv_status conv_int8_scratch_bytes(const conv_int8_problem* p, size_t* bytes);
/* One line on the kernels that a device with `sm_count` SMs runs, weights 16-byte
 * aligned.  Host only. */
CONV_API conv_status conv_int8_describe_plan(const conv_int8_problem* p, int32_t sm_count, char* buf, size_t len);
/* x_scale is read iff p->x_quantized.  Errors: those of conv_int8_scratch_bytes;
 * CONV_ERR_NULL, CONV_ERR_ARG, CONV_ERR_SCRATCH (too small, or not 256-byte
 * aligned), CONV_ERR_ALIAS, CONV_ERR_CUDA. */
CONV_API conv_status conv_int8_forward(const conv_int8_problem* p, const void* x, const float* x_scale, const int8_t* w,
                                       const float* w_scale, const void* bias, const void* residual, void* y,
                                       void* scratch, size_t scratch_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* CONV_GB300_ROWS_H */
