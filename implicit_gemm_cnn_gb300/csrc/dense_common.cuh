// dense_common.cuh -- the products behind the dense operators (linear.h): one
// description for every kernel, the activations with their derivatives, and
// the epilogue of one output element.
//
// Every product is D[m][n] = sum_k A[m][k] * B[n][k], each operand stored with
// k contiguous ("k-major": element (m, k) at m * ld + k) or with m / n
// contiguous ("mn-major": at k * ld + m), so the layer, its input gradient and
// its weight gradient are the same kernels on operands as they lie:
//   y  = x W^T      A = x  k-major,  B = W k-major
//   dx = dz W       A = dz k-major,  B = W mn-major (the sum runs over outputs)
//   dW = dz^T x     A = dz mn-major, B = x mn-major (the sum runs over rows)
#pragma once

#include "conv_common.cuh"

namespace conv {

constexpr int ACT_GELU = 9;
constexpr int ACT_GELU_TANH = 10;

enum DenseEpiMode {
  EPI_LINEAR = 0,     // bias, residual, activation; y, and the activation's argument if wanted
  EPI_GATED = 1,      // two products g, u: y = act(g) * u; g and u if wanted
  EPI_GATED_BWD = 2   // the product dh, and g, u as saved: y = dh * u * act'(g), y2 = dh * act(g)
};

struct DenseEpi {
  int mode;
  int act;
  float alpha, beta;
  int residual_last;
  const void* bias;      // [N] or nullptr
  const void* residual;  // [M][ldr] or nullptr
  void* y;
  void* y2;              // EPI_GATED_BWD, or the second product's output (batch = 2)
  float* pre;            // EPI_LINEAR, EPI_GATED: written if not nullptr; EPI_GATED_BWD: g, read
  float* pre2;           // u
  long long ldr, ldy, ldp;
};

struct DenseGemm {
  int M, N, K;           // of one product; K of one segment
  int a_mn, b_mn;        // operand is mn-major
  int segs;              // 1, or 2: the sum runs over (a[0], b[0]), then (a[1], b[1])
  int batch;             // 1, or 2: products a[i] b[i] into y, y2
  int dual;              // EPI_GATED: products a[0] b[0] and a[0] b[1]
  const void* a[2];
  const void* b[2];
  long long lda, ldb;
  int a_pad, b_pad;      // mn-major: the library's own rows, which go on to a multiple of 64 (what is there is no result)
  DenseEpi epi;
  // k ranges of the CUDA-core kernel: `split` of `k_per_split` terms of the whole sum (segs * K), each
  // into plane s of `part` (float32 [split][products][M][N]); 1: the whole sum
  int split;
  long long k_per_split;
  float* part;
};
__host__ __device__ inline int dense_products(const DenseGemm& g) { return g.dual ? 2 : g.batch; }

// act(t) and act'(t).  FAST: sigmoid, tanh and their like by the hardware's
// exponential and reciprocal (a few units in 2^-22), for results that are
// rounded to 16 bits, whose unit is 2^-9 or 2^-12.  Derivatives multiply by t
// where act' has long tails of zeros; t is clamped there, so that a large t
// gives 0, not 0 * inf.
template <bool FAST>
__device__ __forceinline__ float dense_sigmoid(float t) {
  if constexpr (FAST) return __fdividef(1.0f, 1.0f + __expf(-t));
  else return sigmoid_f32(t);
}
// Phi(t) and exp(-t^2 / 2) for results of 16 bits: the rational approximation of erf of Abramowitz and Stegun, Handbook of
// Mathematical Functions, 7.1.26 (error below 1.5e-7), with x = |t| / sqrt(2); one exponential, one reciprocal.
__device__ __forceinline__ float dense_cdf_fast(float t, float* e) {
  const float x = fabsf(t) * 0.70710678f;
  const float k = __fdividef(1.0f, fmaf(0.3275911f, x, 1.0f));
  *e = __expf(-x * x);
  const float poly = k * fmaf(k, fmaf(k, fmaf(k, fmaf(k, 1.061405429f, -1.453152027f), 1.421413741f), -0.284496736f), 0.254829592f);
  const float tail = 0.5f * poly * *e;  // Phi(-|t|)
  return t >= 0.0f ? 1.0f - tail : tail;
}
template <int ACT, bool FAST>
__device__ __forceinline__ float dense_act_fn(float t, float alpha, float beta) {
  if constexpr (ACT == ACT_GELU) {
    float e;
    if constexpr (FAST) return t * dense_cdf_fast(t, &e);
    else return t * normcdff(t);
  } else if constexpr (ACT == ACT_GELU_TANH) {
    // t/2 (1 + tanh v) = t * sigmoid(2v)
    const float v2 = 1.5957691216f * t * fmaf(0.044715f * t, t, 1.0f);
    return t * dense_sigmoid<FAST>(v2);
  } else if constexpr (ACT == ACT_SILU) return t * dense_sigmoid<FAST>(t);
  else if constexpr (ACT == ACT_SIGMOID) return dense_sigmoid<FAST>(t);
  // (written so that a NaN stays one: a training step has to show it)
  else if constexpr (ACT == ACT_RELU) return t < 0.0f ? 0.0f : t;
  else if constexpr (ACT == ACT_CLIP) return t < alpha ? alpha : (t > beta ? beta : t);
  else if constexpr (ACT == ACT_HARD_SIGMOID || ACT == ACT_HARD_SWISH) {
    const float s = ACT == ACT_HARD_SWISH ? fmaf(t, 1.0f / 6.0f, 0.5f) : fmaf(alpha, t, beta);
    const float c = s < 0.0f ? 0.0f : (s > 1.0f ? 1.0f : s);
    return ACT == ACT_HARD_SWISH ? t * c : c;
  } else return act_fn<ACT>(t, alpha, beta);
}
template <int ACT, bool FAST>
__device__ __forceinline__ float dense_act_grad(float t, float alpha, float beta) {
  if constexpr (ACT == ACT_RELU) return t > 0.0f ? 1.0f : (t == t ? 0.0f : t);
  else if constexpr (ACT == ACT_SILU) {
    const float s = dense_sigmoid<FAST>(t), c = fminf(fmaxf(t, -100.0f), 100.0f);
    return s * (1.0f + c * (1.0f - s));
  } else if constexpr (ACT == ACT_SIGMOID) {
    const float s = dense_sigmoid<FAST>(t);
    return s * (1.0f - s);
  } else if constexpr (ACT == ACT_TANH) {
    const float h = tanhf(t);
    return 1.0f - h * h;
  } else if constexpr (ACT == ACT_HARD_SWISH) {
    return t <= -3.0f ? 0.0f : (t >= 3.0f ? 1.0f : fmaf(t, 1.0f / 3.0f, 0.5f));
  } else if constexpr (ACT == ACT_HARD_SIGMOID) {
    const float s = fmaf(alpha, t, beta);
    return s > 0.0f && s < 1.0f ? alpha : (t == t ? 0.0f : t);
  } else if constexpr (ACT == ACT_CLIP) return t > alpha && t < beta ? 1.0f : (t == t ? 0.0f : t);
  else if constexpr (ACT == ACT_LEAKY_RELU) return t >= 0.0f ? 1.0f : (t == t ? alpha : t);
  else if constexpr (ACT == ACT_GELU) {
    const float c = fminf(fmaxf(t, -40.0f), 40.0f);
    float e, cdf;
    if constexpr (FAST) {
      cdf = dense_cdf_fast(t, &e);
    } else {
      cdf = normcdff(t);
      e = expf(-0.5f * c * c);
    }
    return fmaf(c, 0.3989422804f * e, cdf);
  } else if constexpr (ACT == ACT_GELU_TANH) {
    const float c = fminf(fmaxf(t, -40.0f), 40.0f);
    const float s = dense_sigmoid<FAST>(1.5957691216f * t * fmaf(0.044715f * t, t, 1.0f));
    const float dv2 = 1.5957691216f * fmaf(0.134145f * c, c, 1.0f);
    return fmaf(c * s * (1.0f - s), dv2, s);
  } else return t == t ? 1.0f : t;
}

// One activation, chosen at run time, over N register values (one branch for
// all of them, as in activate_n).
template <bool FAST, int N>
__device__ __forceinline__ void dense_activate(float (&v)[N], int act, float alpha, float beta) {
#define CONV_ACT_CASE(A)                                                                               \
  case A: {                                                                                            \
    _Pragma("unroll") for (int i = 0; i < N; ++i) v[i] = dense_act_fn<A, FAST>(v[i], alpha, beta);     \
    break;                                                                                             \
  }
  switch (act) {
    CONV_ACT_CASE(ACT_RELU) CONV_ACT_CASE(ACT_SILU) CONV_ACT_CASE(ACT_SIGMOID) CONV_ACT_CASE(ACT_TANH)
    CONV_ACT_CASE(ACT_HARD_SWISH) CONV_ACT_CASE(ACT_HARD_SIGMOID) CONV_ACT_CASE(ACT_CLIP)
    CONV_ACT_CASE(ACT_LEAKY_RELU) CONV_ACT_CASE(ACT_GELU) CONV_ACT_CASE(ACT_GELU_TANH)
    default: break;
  }
#undef CONV_ACT_CASE
}
// v[i] -> act(v[i]), d[i] = act'(v[i])
template <bool FAST, int N>
__device__ __forceinline__ void dense_activate_grad(float (&v)[N], float (&d)[N], int act, float alpha, float beta) {
#define CONV_ACT_CASE(A)                                              \
  case A: {                                                           \
    _Pragma("unroll") for (int i = 0; i < N; ++i) {                   \
      d[i] = dense_act_grad<A, FAST>(v[i], alpha, beta);              \
      v[i] = dense_act_fn<A, FAST>(v[i], alpha, beta);                \
    }                                                                 \
    break;                                                            \
  }
  switch (act) {
    CONV_ACT_CASE(ACT_RELU) CONV_ACT_CASE(ACT_SILU) CONV_ACT_CASE(ACT_SIGMOID) CONV_ACT_CASE(ACT_TANH)
    CONV_ACT_CASE(ACT_HARD_SWISH) CONV_ACT_CASE(ACT_HARD_SIGMOID) CONV_ACT_CASE(ACT_CLIP)
    CONV_ACT_CASE(ACT_LEAKY_RELU) CONV_ACT_CASE(ACT_GELU) CONV_ACT_CASE(ACT_GELU_TANH)
    CONV_ACT_CASE(ACT_IDENTITY)
    default: break;
  }
#undef CONV_ACT_CASE
}

// The same over 32 values in local memory, four at a time: for the accurate forms, whose code, unrolled 32 times, takes
// longer to fetch than to run.
static __device__ __noinline__ void dense_activate_array(float* v, int act, float alpha, float beta) {
#pragma unroll 1
  for (int i = 0; i < 32; i += 4) {
    float t[4] = {v[i], v[i + 1], v[i + 2], v[i + 3]};
    dense_activate<false, 4>(t, act, alpha, beta);
    v[i] = t[0]; v[i + 1] = t[1]; v[i + 2] = t[2]; v[i + 3] = t[3];
  }
}
static __device__ __noinline__ void dense_activate_grad_array(float* v, float* d, int act, float alpha, float beta) {
#pragma unroll 1
  for (int i = 0; i < 32; i += 4) {
    float t[4] = {v[i], v[i + 1], v[i + 2], v[i + 3]}, s[4];
    dense_activate_grad<false, 4>(t, s, act, alpha, beta);
    v[i] = t[0]; v[i + 1] = t[1]; v[i + 2] = t[2]; v[i + 3] = t[3];
    d[i] = s[0]; d[i + 1] = s[1]; d[i + 2] = s[2]; d[i + 3] = s[3];
  }
}

// The epilogue of N elements of one row m, columns col[i] (all valid): v the
// first product's sums, u the second's (EPI_GATED).  `which`: the product of a
// batch.  For the kernels whose output accesses are elementwise.
template <typename T, int N>
__device__ __forceinline__ void dense_epilogue(const DenseEpi& e, int which, int m, const int (&col)[N],
                                               const bool (&ok)[N], float (&v)[N], float (&u)[N]) {
  constexpr bool FAST = sizeof(T) == 2;
  const long long yo = m * e.ldy, po = m * e.ldp;
  T* y = static_cast<T*>(which ? e.y2 : e.y);
  if (e.mode == EPI_GATED) {
    if (e.pre) {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (ok[i]) { e.pre[po + col[i]] = v[i]; e.pre2[po + col[i]] = u[i]; }
    }
    dense_activate<FAST, N>(v, e.act, e.alpha, e.beta);
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (ok[i]) y[yo + col[i]] = from_f32<T>(v[i] * u[i]);
  } else if (e.mode == EPI_GATED_BWD) {
    float a[N], d[N];
#pragma unroll
    for (int i = 0; i < N; ++i) a[i] = ok[i] ? e.pre[po + col[i]] : 0.0f;
    dense_activate_grad<FAST, N>(a, d, e.act, e.alpha, e.beta);
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (ok[i]) {
        y[yo + col[i]] = from_f32<T>(v[i] * e.pre2[po + col[i]] * d[i]);
        static_cast<T*>(e.y2)[yo + col[i]] = from_f32<T>(v[i] * a[i]);
      }
  } else {
    if (e.bias) {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (ok[i]) v[i] = __fadd_rn(v[i], to_f32(static_cast<const T*>(e.bias)[col[i]]));
    }
    const T* r = static_cast<const T*>(e.residual) + m * e.ldr;
    if (e.residual && !e.residual_last) {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (ok[i]) v[i] = __fadd_rn(v[i], to_f32(r[col[i]]));
    }
    if (e.pre) {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (ok[i]) e.pre[po + col[i]] = v[i];
    }
    dense_activate<FAST, N>(v, e.act, e.alpha, e.beta);
    if (e.residual && e.residual_last) {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (ok[i]) v[i] = __fadd_rn(v[i], to_f32(r[col[i]]));
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (ok[i]) y[yo + col[i]] = from_f32<T>(v[i]);
  }
}

}  // namespace conv
