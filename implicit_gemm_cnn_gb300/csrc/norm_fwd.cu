// norm_fwd.cu -- layer norm, forward.
//
// A row is read once, into registers, as it lies in memory (16-bit values stay
// packed), and walked three times there: the mean of a warp's values, their
// differences to it and the squares, the output.  The warps' means and squares
// are joined after one barrier (Chan, Golub and LeVeque's formula: the squares
// about the whole mean are those about the parts' means and the parts' weighted
// squared distances), so no sum of squares is about a mean far from its values.
// What bounds it is memory, a read and a write of each value, and the some 130
// instructions for 8 values nearly as much (ncu: issue slots 60%).  Measured:
// 8192 x 4096 bfloat16 28 us (4.8 TB/s), 16384 x 8192 102 (5.3), 1 x 4096 2.1;
// float32 8192 x 4096 46 (5.8), 4096 x 16384 108 (5.0), 1001 x 515 4.3.  Rows of no
// whole 16-byte pieces go value by value: 5000 x 1003 bfloat16 16, 5000 x 12001 158,
// 15370 x 1003 float32 33 (floors 3, 36, 18); rows too wide for registers too, in
// three walks: 1000 x 9001 float32 38, 2000 x 20000 bfloat16, in registers, 54
// (floors 11 and 24).  At the limit of 64 registers the variants of four 16-byte
// accesses a thread spill 16 to 48 bytes, those of 16 values 4 to 48, and those of
// 32 values, at 128 registers, some 100.
#include <algorithm>

#include "norm.cuh"

namespace conv {
namespace {
using namespace norm;

// AFFINE: with weight and bias both.
template <typename T, int B, int N, bool WARP, bool AFFINE>
__global__ void __maxnreg__(registers(B, N)) norm_forward(const NormArgs a) {
  constexpr int V = B / sizeof(T);
  __shared__ float4 red[2][32];  // warps' means, what these are off, squares about both, and counts
  int turn = 0;
  const int G = WARP ? 32 : blockDim.x, t = WARP ? threadIdx.x % 32 : threadIdx.x;
  const int all = static_cast<int>(a.width) / V;   // accesses of a row
  const int n = (all - t + G - 1) / G;             // this thread's
  // a warp's values: those of its 32 threads, which follow one another
  const int whole = all / G, rest = min(max(all - whole * G - static_cast<int>(threadIdx.x / 32) * 32, 0), 32);
  const float count = WARP ? static_cast<float>(a.width) : static_cast<float>((32 * whole + rest) * V);
  const float inv = count > 0.0f ? 1.0f / count : 0.0f, inv_width = 1.0f / static_cast<float>(a.width);
  const int warps = blockDim.x / 32, lane = threadIdx.x % 32;
  const int slot = lane & (warps > 1 ? (1 << (32 - __clz(warps - 1))) - 1 : 0);  // lanes repeat the warps
  griddep_wait();
  griddep_launch();
  const long long step = static_cast<long long>(gridDim.x) * (WARP ? kWarps : 1);
  for (long long r = static_cast<long long>(blockIdx.x) * (WARP ? kWarps : 1) + (WARP ? threadIdx.x / 32 : 0); r < a.rows;
       r += step) {
    const T* x = static_cast<const T*>(a.x) + r * a.ldx + t * V;
    Raw<B> raw[N];
#pragma unroll
    for (int i = 0; i < N; ++i) raw[i] = load_raw<B>(x + i * G * V, i, n);
    Sum<V> sum, diff, square;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float v[V];
      raw_to_f32<T, B>(raw[i], v);
      sum.add(v);
    }
    float mean = warp_sum(sum.value()) * inv;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float v[V];
      if constexpr (N >= 4) keep_packed<B>(raw[i]);
      raw_to_f32<T, B>(raw[i], v);
      const Same<V> minus(i < n ? -mean : 0.0f);  // (values that are not there stay zeros)
      add_n(v, v, minus.v);
      diff.add(v);
      square.add(v, v);
    }
    // the mean's rounding, and the squares about the mean without it
    float off = diff.value(), var = square.value();
    warp_sum2(off, var);
    var = fmaf(-off * inv, off, var);
    off *= inv;
    if (!WARP && warps > 1) {
      if (lane == 0) red[turn][threadIdx.x / 32] = make_float4(mean, off, var, count);
      __syncthreads();
      mean = red[turn][0].x;
      const float4 f = slot < warps ? red[turn][slot] : make_float4(mean, 0.0f, 0.0f, 0.0f);
      const float dist = (f.x - mean) + f.y;  // a warp's mean from the first one's
      off = f.w * dist;
      for (int d = 1; d < warps; d *= 2) off += __shfl_xor_sync(0xffffffffu, off, d);
      off *= inv_width;
      var = fmaf(f.w * (dist - off), dist - off, f.z);
      for (int d = 1; d < warps; d *= 2) var += __shfl_xor_sync(0xffffffffu, var, d);
      turn ^= 1;
    }
    var *= inv_width;
    var = var < 0.0f ? 0.0f : var;  // (a NaN stays)
    const float rstd = 1.0f / sqrtf(var + a.eps);
    if (a.stats && t == 0) *reinterpret_cast<float2*>(a.stats + 2 * r) = make_float2(mean + off, rstd);
    T* y = static_cast<T*>(a.y) + r * a.ldy + t * V;
    const T* w = static_cast<const T*>(a.w) + t * V;
    const T* b = static_cast<const T*>(a.b) + t * V;
    // The mean's two parts are taken off one after the other: their rounded sum is off by 2^-24 of the mean, and a value's
    // distance from the mean may be less than that (16384 halves of 1024 but for one of 1025: 2^-14).
    const Same<V> centre(-mean), rest(-off), scale(rstd);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float v[V], f[V];
      if constexpr (N >= 4) keep_packed<B>(raw[i]);
      raw_to_f32<T, B>(raw[i], v);
      add_n(v, v, centre.v);
      add_n(v, v, rest.v);
      if (AFFINE || a.w) {
        raw_to_f32<T, B>(load_raw<B>(w + i * G * V, i, n), f);
        mul_n(f, f, scale.v);
      } else {
#pragma unroll
        for (int j = 0; j < V; ++j) f[j] = rstd;
      }
      if (AFFINE || a.b) {
        float g[V];
        raw_to_f32<T, B>(load_raw<B>(b + i * G * V, i, n), g);
        fma_n(v, v, f, g);
      } else {
        mul_n(v, v, f);
      }
      if (i < n) store_raw<B>(y + i * G * V, f32_to_raw<T, B>(v));
    }
  }
}

// Rows of any width: three passes over the row, which the caches hold.
template <typename T>
__global__ void __launch_bounds__(1024) norm_forward_stream(const NormArgs a) {
  __shared__ float red1[2][1][32], red2[2][2][32];
  int turn1 = 0, turn2 = 0;
  griddep_wait();
  griddep_launch();
  for (long long r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + r * a.ldx;
    T* y = static_cast<T*>(a.y) + r * a.ldy;
    float mean[1] = {0.0f}, s[2] = {0.0f, 0.0f};
    for (long long c = threadIdx.x; c < a.width; c += blockDim.x) mean[0] += to_f32(x[c]);
    block_sum<1>(mean, red1, turn1);
    const float n = static_cast<float>(a.width);
    mean[0] /= n;
    for (long long c = threadIdx.x; c < a.width; c += blockDim.x) {
      const float d = to_f32(x[c]) - mean[0];
      s[0] += d;
      s[1] = fmaf(d, d, s[1]);
    }
    block_sum<2>(s, red2, turn2);
    const float off = s[0] / n;
    float var = fmaf(-off, off, s[1] / n);
    var = var < 0.0f ? 0.0f : var;
    const float rstd = 1.0f / sqrtf(var + a.eps);
    if (a.stats && threadIdx.x == 0) *reinterpret_cast<float2*>(a.stats + 2 * r) = make_float2(mean[0] + off, rstd);
    for (long long c = threadIdx.x; c < a.width; c += blockDim.x) {
      float o = (to_f32(x[c]) - mean[0] - off) * rstd;
      if (a.w) o *= to_f32(static_cast<const T*>(a.w)[c]);
      if (a.b) o += to_f32(static_cast<const T*>(a.b)[c]);
      y[c] = from_f32<T>(o);
    }
  }
}

template <typename T, int B, int N>
cudaError_t go(const NormArgs& a, const Shape& sh, int sm, cudaStream_t s) {
  const long long per = sh.warp ? kWarps : 1;
  const unsigned blocks = static_cast<unsigned>(std::min((a.rows + per - 1) / per, static_cast<long long>(sm) * (2048 / sh.threads)));
  auto kern = a.w && a.b ? (sh.warp ? norm_forward<T, B, N, true, true> : norm_forward<T, B, N, false, true>)
                         : (sh.warp ? norm_forward<T, B, N, true, false> : norm_forward<T, B, N, false, false>);
  return launch_overlapped(kern, dim3(blocks), sh.threads, 0, 1, s, a);
}
template <typename T, int B>
cudaError_t by_accesses(const NormArgs& a, const Shape& sh, int sm, cudaStream_t s) {
  switch (sh.accesses) {
    case 1: return go<T, B, 1>(a, sh, sm, s);
    case 2: return go<T, B, 2>(a, sh, sm, s);
    case 4: return go<T, B, 4>(a, sh, sm, s);
    case 8: return go<T, B, 8>(a, sh, sm, s);
    default:
      if constexpr (B < 16) {
        if (sh.accesses == 16) return go<T, B, 16>(a, sh, sm, s);
      }
      if constexpr (B == 2) return go<T, B, 32>(a, sh, sm, s);
      return cudaErrorInvalidValue;
  }
}
template <typename T>
cudaError_t by_type(const NormArgs& a, bool stream, int sm, cudaStream_t s) {
  const int bytes = access_bytes(sizeof(T), a.width, {a.x, a.w, a.b, a.y}, {a.rows > 1 ? a.ldx : 0, a.rows > 1 ? a.ldy : 0});
  const Shape sh = shape_of(a.rows, a.width, bytes, sizeof(T), sm);
  if (stream || sh.accesses == 0)
    return launch_overlapped(norm_forward_stream<T>, dim3(static_cast<unsigned>(std::min<long long>(a.rows, 2LL * sm))), 1024, 0, 1, s, a);
  if (bytes == 16) return by_accesses<T, 16>(a, sh, sm, s);
  if constexpr (sizeof(T) == 2) {
    if (bytes == 2) return by_accesses<T, 2>(a, sh, sm, s);
  }
  return by_accesses<T, 4>(a, sh, sm, s);
}

}  // namespace

cudaError_t launch_norm_forward(const NormArgs& a, int dtype, bool stream, int sm, cudaStream_t s) {
  return dtype == CONV_F32 ? by_type<float>(a, stream, sm, s) : dtype == CONV_F16 ? by_type<__half>(a, stream, sm, s)
                                                                                  : by_type<__nv_bfloat16>(a, stream, sm, s);
}

}  // namespace conv
