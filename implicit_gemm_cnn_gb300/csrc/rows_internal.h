// rows_internal.h -- launch interfaces between the row operators' host side
// (rows_api.cu) and their kernels, and the accesses that these share.
#pragma once

#include "dense_internal.h"
#include "rows.h"

namespace conv {

// An access of B bytes: 16, or 4 or 2 where rows are no whole 16-byte pieces.
template <int B> struct RawOf { using type = uint32_t; };
template <> struct RawOf<16> { using type = uint4; };
template <int B> using Raw = typename RawOf<B>::type;

// The access at p if i < n, else zeros: one predicated instruction.  (As a condition around a 2-byte load the compiler made a
// branch of each and waited for one value before it asked for the next: 5000 rows of 1003 bfloat16 took 20 us.)
template <int B>
__device__ __forceinline__ Raw<B> load_raw(const void* p, int i, int n) {
  if constexpr (B == 16) {
    uint4 r;
    asm volatile("{\n .reg .pred p;\n setp.lt.s32 p, %5, %6;\n mov.b32 %0, 0;\n mov.b32 %1, 0;\n mov.b32 %2, 0;\n mov.b32 %3, 0;\n"
                 " @p ld.global.v4.b32 {%0, %1, %2, %3}, [%4];\n}\n"
                 : "=&r"(r.x), "=&r"(r.y), "=&r"(r.z), "=&r"(r.w)
                 : "l"(p), "r"(i), "r"(n));
    return r;
  } else {
    uint32_t r;
    if constexpr (B == 4)
      asm volatile("{\n .reg .pred p;\n setp.lt.s32 p, %2, %3;\n mov.b32 %0, 0;\n @p ld.global.b32 %0, [%1];\n}\n"
                   : "=&r"(r)
                   : "l"(p), "r"(i), "r"(n));
    else
      asm volatile("{\n .reg .pred p;\n setp.lt.s32 p, %2, %3;\n mov.b32 %0, 0;\n @p ld.global.u16 %0, [%1];\n}\n"
                   : "=&r"(r)
                   : "l"(p), "r"(i), "r"(n));
    return r;
  }
}
template <int B>
__device__ __forceinline__ void store_raw(void* p, const Raw<B>& r) {
  if constexpr (B == 2) *static_cast<uint16_t*>(p) = static_cast<uint16_t>(r);
  else *static_cast<Raw<B>*>(p) = r;
}
// The same bits, as far as the compiler knows other ones: packed values are unpacked again at each use, instead of living
// unpacked in twice the registers.
template <int B>
__device__ __forceinline__ void keep_packed(Raw<B>& r) {
  if constexpr (B == 16) asm volatile("" : "+r"(r.x), "+r"(r.y), "+r"(r.z), "+r"(r.w));
  else asm volatile("" : "+r"(r));
}

// 16-bit values by their bits.
template <typename T>
__device__ __forceinline__ float half_bits_f32(uint16_t h) {
  if constexpr (std::is_same<T, __nv_bfloat16>::value) return __uint_as_float(static_cast<uint32_t>(h) << 16);
  else return __half2float(__ushort_as_half(h));
}
template <typename T>
__device__ __forceinline__ uint32_t pack_halves(float lo, float hi) {
  if constexpr (std::is_same<T, __half>::value) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}
// One access's values as float32, and back.
template <typename T, int B>
__device__ __forceinline__ void raw_to_f32(const Raw<B>& q, float* v) {
  if constexpr (sizeof(T) == 4) {
    if constexpr (B == 4) v[0] = __uint_as_float(q);
    else { v[0] = __uint_as_float(q.x); v[1] = __uint_as_float(q.y); v[2] = __uint_as_float(q.z); v[3] = __uint_as_float(q.w); }
  } else if constexpr (B == 2) {
    v[0] = half_bits_f32<T>(static_cast<uint16_t>(q));
  } else {
    constexpr int W = B / 4;
    uint32_t w[W];
    if constexpr (B == 4) w[0] = q;
    else { w[0] = q.x; w[1] = q.y; w[2] = q.z; w[3] = q.w; }
#pragma unroll
    for (int i = 0; i < W; ++i) {
      if constexpr (std::is_same<T, __nv_bfloat16>::value) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      } else {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
      }
    }
  }
}
template <typename T, int B>
__device__ __forceinline__ Raw<B> f32_to_raw(const float* v) {
  if constexpr (sizeof(T) == 4) {
    if constexpr (B == 4) return __float_as_uint(v[0]);
    else return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
  } else if constexpr (B == 2) {
    return pack_halves<T>(v[0], 0.0f);
  } else if constexpr (B == 4) {
    return pack_halves<T>(v[0], v[1]);
  } else {
    return make_uint4(pack_halves<T>(v[0], v[1]), pack_halves<T>(v[2], v[3]), pack_halves<T>(v[4], v[5]),
                      pack_halves<T>(v[6], v[7]));
  }
}

// float32 arithmetic on two values an instruction, where V is even.
__device__ __forceinline__ unsigned long long pair(float a, float b) {
  unsigned long long r;
  asm("mov.b64 %0, {%1, %2};\n" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpair(unsigned long long p, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;\n" : "=f"(a), "=f"(b) : "l"(p));
}
// d = a b + c, a b, a + b; scalars stand for all V values
template <int V>
__device__ __forceinline__ void fma_n(float (&d)[V], const float (&a)[V], const float (&b)[V], const float (&c)[V]) {
  if constexpr (V % 2 == 0) {
#pragma unroll
    for (int i = 0; i < V; i += 2) {
      unsigned long long r;
      asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(r) : "l"(pair(a[i], a[i + 1])), "l"(pair(b[i], b[i + 1])), "l"(pair(c[i], c[i + 1])));
      unpair(r, d[i], d[i + 1]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) d[i] = fmaf(a[i], b[i], c[i]);
  }
}
template <int V>
__device__ __forceinline__ void mul_n(float (&d)[V], const float (&a)[V], const float (&b)[V]) {
  if constexpr (V % 2 == 0) {
#pragma unroll
    for (int i = 0; i < V; i += 2) {
      unsigned long long r;
      asm("mul.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(pair(a[i], a[i + 1])), "l"(pair(b[i], b[i + 1])));
      unpair(r, d[i], d[i + 1]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) d[i] = a[i] * b[i];
  }
}
template <int V>
__device__ __forceinline__ void add_n(float (&d)[V], const float (&a)[V], const float (&b)[V]) {
  if constexpr (V % 2 == 0) {
#pragma unroll
    for (int i = 0; i < V; i += 2) {
      unsigned long long r;
      asm("add.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(pair(a[i], a[i + 1])), "l"(pair(b[i], b[i + 1])));
      unpair(r, d[i], d[i + 1]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) d[i] = a[i] + b[i];
  }
}
template <int V>
struct Same {
  float v[V];
  __device__ __forceinline__ explicit Same(float f) {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = f;
  }
};
// Sums of V values, two at a time (few registers; a warp's other work hides the chain).
template <int V>
struct Sum {
  static constexpr int W = V % 2 == 0 ? 2 : 1;
  float s[W] = {};
  __device__ __forceinline__ void add(const float (&v)[V]) {
#pragma unroll
    for (int i = 0; i < V; i += W) add_n(s, s, reinterpret_cast<const float(&)[W]>(v[i]));
  }
  __device__ __forceinline__ void add(const float (&a)[V], const float (&b)[V]) {  // products
#pragma unroll
    for (int i = 0; i < V; i += W) fma_n(s, reinterpret_cast<const float(&)[W]>(a[i]), reinterpret_cast<const float(&)[W]>(b[i]), s);
  }
  __device__ __forceinline__ float value() const { return W == 2 ? s[0] + s[W - 1] : s[0]; }
};
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}

// Two sums: one goes on in the lower half of the warp, the other in the upper.
__device__ __forceinline__ void warp_sum2(float& a, float& b) {
  const bool high = threadIdx.x % 32 >= 16;
  float s = (high ? b : a) + __shfl_xor_sync(0xffffffffu, high ? a : b, 16);
#pragma unroll
  for (int d = 8; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
  a = __shfl_sync(0xffffffffu, s, 0);
  b = __shfl_sync(0xffffffffu, s, 16);
}

// The widest access (bytes) that addresses, row strides and the width all are multiples of; 2-byte types: 16, 4 or 2,
// float32: 16 or 4.
inline int access_bytes(int es, long long width, std::initializer_list<const void*> ptrs,
                        std::initializer_list<long long> strides) {
  unsigned long long all = static_cast<unsigned long long>(width) * es;
  for (const void* p : ptrs) all |= reinterpret_cast<uintptr_t>(p);
  for (long long s : strides) all |= static_cast<unsigned long long>(s) * es;
  return all % 16 == 0 ? 16 : all % 4 == 0 ? 4 : es;
}

// Layer norm (norm_fwd.cu, norm_bwd.cu).
struct NormArgs {
  const void *x, *w, *b, *dy;
  void *y, *dx, *dw, *db;
  float* stats;             // [rows][2]: written forward (or nullptr), read backward
  float* part;              // backward: the scratch, float32 [blocks][2][width] and, of wide rows, [rows][4]
  long long rows, width, ldx, ldy;
  float eps;
};
cudaError_t launch_norm_forward(const NormArgs& a, int dtype, bool stream, int sm, cudaStream_t s);
size_t norm_backward_scratch(long long rows, long long width, int es, bool stream, int sm);  // bytes
cudaError_t launch_norm_backward(const NormArgs& a, int dtype, bool stream, int sm, cudaStream_t s);

// Dropout (dropout.cu).
struct DropoutArgs {
  const void *x, *residual;
  void* y;
  long long rows, width, ldx, ldr, ldy;
  uint64_t seed, offset;
  const uint64_t* state;
  uint32_t drop;            // of 65536
};
cudaError_t launch_dropout(const DropoutArgs& a, int dtype, int sm, cudaStream_t s);

// Rows in 8 bits (quantize.cu).
struct QuantizeArgs {
  const void* x;
  void* q;                  // int8, or (wide) the same whole numbers as halves
  float* scale;
  long long rows, width, ldx, ldq;
};
cudaError_t launch_quantize(const QuantizeArgs& a, int dtype, bool wide, int sm, cudaStream_t s);

// 8-bit rows as halves, in rows of `ld` values (a multiple of 64); or as they are (a multiple of 16), what lies behind a row's
// end unspecified.
struct WidenArgs {
  const int8_t* in;
  void* out;
  long long rows, cols, ld_in, ld;
};
// `follows`: the kernel before in the stream is this call's own, and touches neither `in` nor `out`.
cudaError_t launch_widen(const WidenArgs& a, bool wide, bool follows, int sm, cudaStream_t s);

// The 8-bit product (int8_*.cu).
struct Int8Args {
  const int8_t *x, *w;
  const float *x_scale, *w_scale;
  long long ldx, ldw;
  int M, N, K;
  DenseEpi epi;
};
// (the kernel for few rows) x in whole 16-byte pieces on 16-byte boundaries, its rows padded to that.  `follows`: the kernel before in the stream is this call's own, and writes no weights.
cudaError_t launch_int8_few(const Int8Args& g, int dtype, bool follows, int sm, cudaStream_t s);
// For some tens of rows: x as halves, the weights as they are.
struct Int8MidPlan {
  int nt, row_tiles, tiles;  // rows of a tile; tiles of rows and of outputs
  int split, kb_range;       // blocks of a cluster, and the 128-term stages of each
};
Int8MidPlan int8_mid_plan(int M, int N, int K, int sm);
cudaError_t launch_int8_mid(const Int8MidPlan& t, const Int8Args& g, const __half* x, int dtype, cudaStream_t s);

// On the tensor cores: x [M][ldx] and w [N][ldw] as halves, rows of a multiple of 64 on 128-byte boundaries.  `part`: the k
// ranges' sums (t.part_bytes).
DenseTcPlan int8_tc_plan(int M, int N, int K, int sm);
cudaError_t launch_int8_tc(const DenseTcPlan& t, const Int8Args& g, const __half* x, const __half* w, int dtype, void* part,
                           cudaStream_t s);

}  // namespace conv
