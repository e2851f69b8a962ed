// quantize.cu -- rows in 8 bits: the largest value of a row, then its quotients;
// and 8-bit rows as the halves that the tensor cores multiply.
//
// A row is read once, into registers (norm.cuh).  What bounds it is the issue of
// instructions as much as memory (ncu: 64 to 70% of the slots).  Measured:
// 8192 x 4096 bfloat16 to bytes 23.4 us (4.3 TB/s), float32 32.7 (5.1), 1 x 4096 1.6;
// value by value 15370 x 1003 bfloat16 22.6 (2.0), float32 25.8 (3.0); 2000 x 20000
// bfloat16 44 (2.7), 2000 x 40000, too wide for registers, 141 (1.7).  Cold: 2048 x
// 4096 to halves 10.7 us, 4096 x 4096 bytes to halves 9.6 (5.2 TB/s).
#include <algorithm>

#include "int8.cuh"
#include "norm.cuh"

namespace conv {
namespace {
using namespace norm;

// x / scale to the nearest whole number, ties to even, as the exact quotient rounds.  `inv` is 1 / scale rounded, so the
// first guess q is off by at most one.  What it leaves, x - q scale, is one fused step: it is a multiple of scale's last
// place and at most scale, so exact, for |x| >= scale; below that q is 0 (x itself) or 1, where the difference may round
// onto half a scale and no further, and the tie goes to 0, as the quotient does.  (16-bit values tie often: x / scale is
// 127 times a quotient of two short numbers.)
constexpr float kMagic = 12582912.0f;  // 1.5 * 2^23: the last place of a sum with it is 1, its last byte the integer

// A row's scale, from the largest of the bits of its absolute values (they are ordered as the values are, infinities and NaN
// above them), and the quotients by it.
struct RowScale {
  float scale, inv, half;
  bool small;
  __device__ __forceinline__ explicit RowScale(uint32_t most) {
    const bool finite = most < 0x7f800000u;
    constexpr float kStep = 1.0f / 127.0f;  // (a product, as torch makes of a float32 device tensor / 127: scales made there are the same bits)
    scale = finite ? __uint_as_float(most) * kStep : __uint_as_float(0x7fffffffu);
    small = scale < 0x1p-100f;
    inv = finite && scale > 0.0f && !small ? __fdiv_rn(1.0f, scale) : 0.0f;
    half = 0.5f * scale;
  }
  // The whole numbers of V values, as the bits of their sums with kMagic.
  template <int V>
  __device__ __forceinline__ void of(const float (&v)[V], int (&bits)[V]) const {
    if (inv == 0.0f) {
#pragma unroll
      for (int i = 0; i < V; ++i) bits[i] = slow(v[i]);
      return;
    }
    float t[V], q[V], left[V];
    const Same<V> by(inv), magic(kMagic), back(-kMagic), less(-scale);
    fma_n(t, v, by.v, magic.v);
    add_n(q, t, back.v);
    fma_n(left, q, less.v, v);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int b = __float_as_int(t[i]);
      // |left| - half is exact near zero.  Above zero, or zero at an odd q: one further, towards left's side.
      const int d = __float_as_int(fabsf(left[i]) - half) + (b & 1);
      bits[i] = d > 0 ? b + ((__float_as_int(left[i]) >> 31) | 1) : b;
    }
  }
  // Rows without a scale (zeros, infinities, NaN), and scales whose inverse or half would not be exact or finite: x and
  // scale times 2^64.
  __device__ __noinline__ int slow(float x) const {
    if (!small || scale == 0.0f) return __float_as_int(kMagic);
    const float s = scale * 0x1p64f;
    x *= 0x1p64f;
    float q = rintf(__fdiv_rn(x, s));
    const float left = fmaf(-q, s, x);
    const bool odd = static_cast<int>(q) & 1;
    if (left > 0.5f * s || (left == 0.5f * s && odd)) q += 1.0f;
    else if (left < -0.5f * s || (left == -0.5f * s && odd)) q -= 1.0f;
    return __float_as_int(fminf(fmaxf(q, -127.0f), 127.0f) + kMagic);
  }
};

// V whole numbers (their sums with kMagic), as bytes or halves.
template <int V>
__device__ __forceinline__ void store_whole(void* q, long long at, const int (&v)[V], int wide) {
  if (wide) {
    __half* to = static_cast<__half*>(q) + at;
    float f[V];
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = __int_as_float(v[i]) - kMagic;
    if constexpr (V == 1) *to = __float2half_rn(f[0]);
    else {
      uint32_t w[V / 2];
#pragma unroll
      for (int i = 0; i < V / 2; ++i) w[i] = pack_halves<__half>(f[2 * i], f[2 * i + 1]);
      if constexpr (V == 8) *reinterpret_cast<uint4*>(to) = make_uint4(w[0], w[1], w[2], w[3]);
      else if constexpr (V == 4) *reinterpret_cast<uint2*>(to) = make_uint2(w[0], w[1]);
      else *reinterpret_cast<uint32_t*>(to) = w[0];
    }
  } else {
    int8_t* to = static_cast<int8_t*>(q) + at;
    auto four = [&](int i) {  // the last bytes of four of them
      return __byte_perm(__byte_perm(v[i], v[i + 1], 0x0040), __byte_perm(v[i + 2], v[i + 3], 0x0040), 0x5410);
    };
    if constexpr (V == 8) *reinterpret_cast<uint2*>(to) = make_uint2(four(0), four(4));
    else if constexpr (V == 4) *reinterpret_cast<uint32_t*>(to) = four(0);
    else if constexpr (V == 2) *reinterpret_cast<uint16_t*>(to) = static_cast<uint16_t>(__byte_perm(v[0], v[1], 0x0040));
    else *to = static_cast<int8_t>(v[0]);
  }
}

// The largest of the absolute values' bits of an access, as float32's bits or (packed 16-bit values) two of 16 bits.
template <typename T, int B>
__device__ __forceinline__ uint32_t larger(uint32_t most, const Raw<B>& raw) {
  auto word = [&](uint32_t w) {
    if constexpr (sizeof(T) == 4) most = max(most, w & 0x7fffffffu);
    else most = __vmaxu2(most, w & 0x7fff7fffu);
  };
  if constexpr (B == 16) {
    word(raw.x); word(raw.y); word(raw.z); word(raw.w);
  } else {
    word(raw);
  }
  return most;
}
template <typename T>
__device__ __forceinline__ uint32_t largest_bits(uint32_t most) {
  if constexpr (sizeof(T) == 4) return most;
  else return __float_as_uint(half_bits_f32<T>(static_cast<uint16_t>(max(most & 0xffffu, most >> 16))));
}

// Rows in registers, as layer norm's (norm.cuh).
template <typename T, int B, int N, bool WARP>
__global__ void __maxnreg__(registers(B, N)) quantize_rows(const QuantizeArgs a, const int wide) {
  constexpr int V = B / sizeof(T);
  __shared__ uint32_t red[2][32];
  int turn = 0;
  const int G = WARP ? 32 : blockDim.x, t = WARP ? threadIdx.x % 32 : threadIdx.x;
  const int n = (static_cast<int>(a.width) / V - t + G - 1) / G;  // this thread's accesses
  griddep_wait();
  griddep_launch();
  const long long step = static_cast<long long>(gridDim.x) * (WARP ? kWarps : 1);
  for (long long r = static_cast<long long>(blockIdx.x) * (WARP ? kWarps : 1) + (WARP ? threadIdx.x / 32 : 0); r < a.rows;
       r += step) {
    const T* x = static_cast<const T*>(a.x) + r * a.ldx + t * V;
    Raw<B> raw[N];
#pragma unroll
    for (int i = 0; i < N; ++i)
      raw[i] = load_raw<B>(x + i * G * V, i, n);
    uint32_t most = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) most = larger<T, B>(most, raw[i]);
    most = __reduce_max_sync(0xffffffffu, largest_bits<T>(most));
    if (!WARP && blockDim.x > 32) {
      if (threadIdx.x % 32 == 0) red[turn][threadIdx.x / 32] = most;
      __syncthreads();
      most = __reduce_max_sync(0xffffffffu, threadIdx.x % 32 < blockDim.x / 32 ? red[turn][threadIdx.x % 32] : 0u);
      turn ^= 1;
    }
    const RowScale s(most);
    if (t == 0) a.scale[r] = s.scale;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (i < n) {
        float v[V];
        if constexpr (N >= 4) keep_packed<B>(raw[i]);
        raw_to_f32<T, B>(raw[i], v);
        int bits[V];
        s.of(v, bits);
        store_whole<V>(a.q, r * a.ldq + (i * G + t) * V, bits, wide);
      }
    }
  }
}
// Rows of any width: two passes over the row.
template <typename T>
__global__ void __launch_bounds__(1024) quantize_rows_stream(const QuantizeArgs a, const int wide) {
  __shared__ uint32_t red[2][32];
  int turn = 0;
  griddep_wait();
  griddep_launch();
  for (long long r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + r * a.ldx;
    uint32_t most = 0;
    for (long long c = threadIdx.x; c < a.width; c += blockDim.x) most = max(most, __float_as_uint(fabsf(to_f32(x[c]))));
    most = __reduce_max_sync(0xffffffffu, most);
    if (threadIdx.x % 32 == 0) red[turn][threadIdx.x / 32] = most;
    __syncthreads();
    most = __reduce_max_sync(0xffffffffu, red[turn][threadIdx.x % 32]);
    turn ^= 1;
    const RowScale s(most);
    if (threadIdx.x == 0) a.scale[r] = s.scale;
    for (long long c = threadIdx.x; c < a.width; c += blockDim.x) {
      const float v[1] = {to_f32(x[c])};
      int bits[1];
      s.of(v, bits);
      store_whole<1>(a.q, r * a.ldq + c, bits, wide);
    }
  }
}

template <typename T, int B, int N>
cudaError_t quantize_go(const QuantizeArgs& a, const Shape& sh, int wide, int sm, cudaStream_t s) {
  const long long per = sh.warp ? kWarps : 1;
  const unsigned blocks = static_cast<unsigned>(std::min((a.rows + per - 1) / per, static_cast<long long>(sm) * (2048 / sh.threads)));
  return launch_overlapped(sh.warp ? quantize_rows<T, B, N, true> : quantize_rows<T, B, N, false>, dim3(blocks), sh.threads, 0, 1,
                           s, a, wide);
}
template <typename T, int B>
cudaError_t quantize_by_accesses(const QuantizeArgs& a, const Shape& sh, int wide, int sm, cudaStream_t s) {
  switch (sh.accesses) {
    case 1: return quantize_go<T, B, 1>(a, sh, wide, sm, s);
    case 2: return quantize_go<T, B, 2>(a, sh, wide, sm, s);
    case 4: return quantize_go<T, B, 4>(a, sh, wide, sm, s);
    case 8: return quantize_go<T, B, 8>(a, sh, wide, sm, s);
    default:
      if constexpr (B < 16) {
        if (sh.accesses == 16) return quantize_go<T, B, 16>(a, sh, wide, sm, s);
      }
      if constexpr (B == 2) return quantize_go<T, B, 32>(a, sh, wide, sm, s);
      return cudaErrorInvalidValue;
  }
}
template <typename T>
cudaError_t quantize_by_type(const QuantizeArgs& a, int wide, int sm, cudaStream_t s) {
  // q's accesses have as many values as x's
  const int es = sizeof(T), qs = wide ? 2 : 1;
  int bytes = access_bytes(es, a.width, {a.x}, {a.rows > 1 ? a.ldx : 0});
  auto q_fits = [&](int b) {
    return (reinterpret_cast<uintptr_t>(a.q) | static_cast<uintptr_t>(a.rows > 1 ? a.ldq * qs : 0)) % (b / es * qs) == 0;
  };
  if (bytes == 16 && !q_fits(16)) bytes = 4;
  if (bytes == 4 && !q_fits(4)) bytes = es;
  const Shape sh = shape_of(a.rows, a.width, bytes, es, sm);
  if (sh.accesses == 0)
    return launch_overlapped(quantize_rows_stream<T>, dim3(static_cast<unsigned>(std::min<long long>(a.rows, 2LL * sm))), 1024, 0, 1, s, a, wide);
  if (bytes == 16) return quantize_by_accesses<T, 16>(a, sh, wide, sm, s);
  if constexpr (sizeof(T) == 2) {
    if (bytes == 2) return quantize_by_accesses<T, 2>(a, sh, wide, sm, s);
  }
  return quantize_by_accesses<T, 4>(a, sh, wide, sm, s);
}

// A warp widens 1024 bytes of a row: a lane 8 at a time, four of these on the way (16 bytes at a time its two stores would
// leave gaps: 50 MB took 13 us).  `early`: the kernel before is the same call's, and writes none of this one's operands.  It
// is then waited for at the end, so that who waits for this kernel has waited for that one too.
template <bool WIDE>
__global__ void __launch_bounds__(256) widen_rows(const WidenArgs a, const int early) {
  if (!early) griddep_wait();
  griddep_launch();
  const long long chunks = (a.cols + 1023) / 1024, warps = static_cast<long long>(gridDim.x) * 8;
  const int lane = threadIdx.x % 32;
  const int8_t* const end = a.in + (a.rows - 1) * a.ld_in + a.cols;
  for (long long i = static_cast<long long>(blockIdx.x) * 8 + threadIdx.x / 32; i < a.rows * chunks; i += warps) {
    const long long r = i / chunks, c = i % chunks * 1024 + lane * 8;
    const int8_t* p = a.in + r * a.ld_in + c;
    uint2 v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[k] = make_uint2(0, 0);
      if (c + 256 * k >= a.cols) continue;
      const int8_t* at = p + 256 * k;
      if (reinterpret_cast<uintptr_t>(at) % 8 == 0 && at + 8 <= end) {
        v[k] = *reinterpret_cast<const uint2*>(at);
      } else {
        const uint4 q = load_any(at, a.in, end);
        v[k] = make_uint2(q.x, q.y);
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (c + 256 * k >= a.cols) continue;
      const long long to = r * a.ld + c + 256 * k;  // (rows of a multiple of 16: 8 values from here exist)
      if constexpr (WIDE) {
        uint4 h;
        widen(v[k].x, h.x, h.y);
        widen(v[k].y, h.z, h.w);
        *reinterpret_cast<uint4*>(static_cast<__half*>(a.out) + to) = h;
      } else {
        *reinterpret_cast<uint2*>(static_cast<int8_t*>(a.out) + to) = v[k];
      }
    }
  }
  if (early) griddep_wait();
}

}  // namespace

cudaError_t launch_widen(const WidenArgs& a, bool wide, bool follows, int sm, cudaStream_t s) {
  const long long warps = a.rows * ((a.cols + 1023) / 1024);
  return launch_overlapped(wide ? widen_rows<true> : widen_rows<false>, dim3(static_cast<unsigned>(std::min((warps + 7) / 8, 16LL * sm))), 256, 0, 1, s, a, follows ? 1 : 0);
}

cudaError_t launch_quantize(const QuantizeArgs& a, int dtype, bool wide, int sm, cudaStream_t s) {
  return dtype == CONV_F32 ? quantize_by_type<float>(a, wide, sm, s) : dtype == CONV_F16 ? quantize_by_type<__half>(a, wide, sm, s)
                                                                                         : quantize_by_type<__nv_bfloat16>(a, wide, sm, s);
}

}  // namespace conv
