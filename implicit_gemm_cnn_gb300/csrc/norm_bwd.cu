// norm_bwd.cu -- layer norm, backward.
//
// dx needs two sums over a row, dweight and dbias sums over columns.  A third sum
// over the row, of the differences to the saved mean, is what that mean's rounding
// left in them; it is taken out of xhat before dweight and dx are made of it.  A block of
// 512 threads keeps the columns' sums in registers: a group of threads spans the
// row, 8 to 32 values each (float32: 4 to 16), and where the row is short a
// block has several groups.  A group takes R rows at a time and reduces their
// sums in one go (a barrier and some 20 shuffles for all of them).  Rows of
// whole 16-byte pieces come through shared memory, two batches of 64 KB ahead
// (cp.async; a thread reads back only what it copied itself, so no barrier
// stands between): the memory works under the arithmetic, some 115 instructions
// for 8 values.  Other rows are loaded straight into registers.  Groups and
// blocks leave their columns' sums to a second kernel, which adds them in order.
//
// What bounds it is memory, two reads and a write.  Measured with the second
// kernel: 16384 x 8192 bfloat16 140 us (5.7 TB/s; with the mean's rounding left in
// 135, without the batches ahead 172), 8192 x 4096 45.3 (4.4; 42.8), 1001 x 515
// float32 7.2, 5000 x 1003 bfloat16 19.0.  Rows too wide for registers go value by
// value, dx and the columns' sums in kernels of their own: 4096 x 16384 float32 305
// (floor 120), 2000 x 20000 bfloat16 165.  Rows of no whole 16-byte pieces go value
// by value as well, 15370 x 1003 float32 49 (28); from 8193 to 16384 values of 16
// bits, 32 a thread, such a kernel spills 550 bytes with a weight and 170 without
// (pairs of values: 80 and none), 5000 x 12001 bfloat16 275 (54).
#include <algorithm>

#include "norm.cuh"

namespace conv {
namespace {
using namespace norm;

constexpr int kThreads = 512;
constexpr int kStages = 3;        // batches of rows in shared memory
constexpr int kColumns = 32;      // of a block that adds the partial sums
constexpr int kRanges = 32;       // and the ranges of parts that it adds at once
constexpr int kStreamRows = 64;   // rows of a block of the wide rows' column sums, at least

// C sums (C a power of two) over the warp, halving the values with each step: afterwards v[0] of lane l is the sum of
// value l % C.
template <int C>
__device__ __forceinline__ void warp_sums(float (&v)[C]) {
  const int lane = threadIdx.x % 32;
  int bit = 1;
#pragma unroll
  for (int n = C; n > 1; n /= 2, bit *= 2) {
    const bool high = lane & bit;
#pragma unroll
    for (int i = 0; i < n / 2; ++i) {  // even values stay with the lanes whose bit is clear
      const float send = high ? v[2 * i] : v[2 * i + 1], keep = high ? v[2 * i + 1] : v[2 * i];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, send, bit);
    }
  }
#pragma unroll
  for (; bit < 32; bit *= 2) v[0] += __shfl_xor_sync(0xffffffffu, v[0], bit);
}

// 16 bytes from global to shared memory if `ok`, else zeros, under way until its group is waited for.
__device__ __forceinline__ void copy_ahead(uint4* to, const void* from, bool ok) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(to))), "l"(from),
               "r"(ok ? 16 : 0)
               : "memory");
}

// `sums`: the weight's and the bias's gradients are wanted.  `warps`: of a group.
template <typename T, int B, int E, int R, bool WEIGHT>
__global__ void __launch_bounds__(kThreads, 1) norm_backward(const NormArgs a, const int sums, const int warps) {
  constexpr int V = B / sizeof(T), N = E / V;
  constexpr bool HOLD = E * sizeof(T) <= 32;               // the weights in registers; else from the cache, row by row
  constexpr bool AHEAD = B == 16;
  constexpr int C = 4 * R;                                 // sums of R rows: three each, and none
  extern __shared__ uint4 ahead[];                         // batches [kStages][R][x, dy][N][threads]; then the groups' sums
  __shared__ float red[2][kThreads / 32][C];
  int turn = 0;
  const int G = warps * 32, group = threadIdx.x / G, groups = blockDim.x / G, t = threadIdx.x - group * G;
  const int lane = threadIdx.x % 32, warp0 = group * warps;
  const int width = static_cast<int>(a.width);
  griddep_wait();
  griddep_launch();
  const int n = (width / V - t + G - 1) / G;               // this thread's accesses
  auto load_weight = [&](int i) { return load_raw<B>(static_cast<const T*>(a.w) + (i * G + t) * V, i, n); };
  float w[HOLD && WEIGHT ? N : 1][V] = {};
  auto times_weight = [&](int i, float (&g)[V]) {
    if constexpr (!WEIGHT) {
    } else if constexpr (HOLD) {
      mul_n(g, g, w[i]);
    } else {
      float f[V];
      raw_to_f32<T, B>(load_weight(i), f);
      mul_n(g, g, f);
    }
  };
  float dw[N][V], db[N][V];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if constexpr (HOLD && WEIGHT) raw_to_f32<T, B>(load_weight(i), w[i]);
#pragma unroll
    for (int j = 0; j < V; ++j) dw[i][j] = db[i][j] = 0.0f;
  }
  const float inv = 1.0f / static_cast<float>(width);
  const long long step = static_cast<long long>(gridDim.x) * groups;
  const T* const x0 = static_cast<const T*>(a.x) + t * V;
  const T* const dy0 = static_cast<const T*>(a.dy) + t * V;
  T* const dx0 = static_cast<T*>(a.dx) + t * V;
  const long long first = static_cast<long long>(blockIdx.x) * groups;
  auto place = [&](int stage, int k, int which, int i) {
    return ahead + (((stage * R + k) * 2 + which) * N + i) * static_cast<int>(blockDim.x) + threadIdx.x;
  };
  auto fetch = [&](long long base, int stage) {
    if constexpr (AHEAD) {
#pragma unroll
      for (int k = 0; k < R; ++k) {
        const long long r = base + group + k * step;
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const bool ok = r < a.rows && i < n;
          copy_ahead(place(stage, k, 0, i), ok ? x0 + r * a.ldx + i * G * V : a.x, ok);
          copy_ahead(place(stage, k, 1, i), ok ? dy0 + r * a.ldy + i * G * V : a.dy, ok);
        }
      }
      asm volatile("cp.async.commit_group;\n" ::: "memory");
    }
  };
  float2 stats[R];  // of the batch after this one
  auto fetch_stats = [&](long long base) {
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const long long r = base + group + k * step;
      stats[k] = r < a.rows ? *reinterpret_cast<const float2*>(a.stats + 2 * r) : make_float2(0.0f, 0.0f);
    }
  };
  int stage = 0;
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) fetch(first + i * R * step, i);
  fetch_stats(first);
  // every group of a block takes the same number of turns (they meet at barriers)
  for (long long base = first; base < a.rows; base += R * step) {
    Raw<B> rx[R][N], rd[R][N];
    float mean[R], rstd[R];
#pragma unroll
    for (int k = 0; k < R; ++k) {
      mean[k] = stats[k].x;
      rstd[k] = stats[k].y;
    }
    fetch_stats(base + R * step);
    if constexpr (AHEAD) {
      const int before = stage == 0 ? kStages - 1 : stage - 1;
      fetch(base + (kStages - 1) * R * step, before);  // (this thread has read the batch that was there)
      asm volatile("cp.async.wait_group %0;\n" ::"n"(kStages - 1) : "memory");
    }
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const long long r = base + group + k * step;
      const T *x = x0 + r * a.ldx, *dy = dy0 + r * a.ldy;
      const int here = r < a.rows ? n : 0;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        if constexpr (AHEAD) {
          rx[k][i] = *place(stage, k, 0, i);
          rd[k][i] = *place(stage, k, 1, i);
        } else {
          rx[k][i] = load_raw<B>(x + i * G * V, i, here);
          rd[k][i] = load_raw<B>(dy + i * G * V, i, here);
        }
      }
    }
    float s[C];
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const Same<V> scale(rstd[k]);
      Sum<V> s1, s2, s3;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        float h[V], g[V];
        raw_to_f32<T, B>(rx[k][i], h);
        raw_to_f32<T, B>(rd[k][i], g);
        const Same<V> minus(i < n ? -mean[k] : 0.0f);  // (values that are not there stay zeros)
        add_n(h, h, minus.v);
        if constexpr (V == 1) h[0] = __fmul_rn(h[0], rstd[k]);  // (no part of the sum's addition: every variant has the same sum)
        else mul_n(h, h, scale.v);
        s3.add(h);
        add_n(db[i], db[i], g);
        times_weight(i, g);
        s1.add(g);
        s2.add(g, h);
      }
      s[4 * k] = s1.value();
      s[4 * k + 1] = s2.value();
      s[4 * k + 2] = s3.value();
      s[4 * k + 3] = 0.0f;
    }
    const int now = stage;
    stage = stage == kStages - 1 ? 0 : stage + 1;
    warp_sums<C>(s);
    float sum = s[0];  // of value lane % C
    if (warps > 1) {
      if (lane < C) red[turn][threadIdx.x / 32][lane] = sum;
      __syncthreads();
      sum = 0.0f;
      for (int k = lane / C; k < warps; k += 32 / C) sum += red[turn][warp0 + k][lane % C];
#pragma unroll
      for (int d = C; d < 32; d *= 2) sum += __shfl_xor_sync(0xffffffffu, sum, d);
      turn ^= 1;
    }
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const long long r = base + group + k * step;
      const float c1 = __shfl_sync(0xffffffffu, sum, 4 * k) * inv, off = __shfl_sync(0xffffffffu, sum, 4 * k + 2) * inv;
      const float c2 = fmaf(-off, c1, __shfl_sync(0xffffffffu, sum, 4 * k + 1) * inv);
      T* dx = dx0 + r * a.width;
      // xhat = (x - mean) rstd - off,  dx = rstd (g - c1 - xhat c2); (rstd^2 c2 as one factor would leave float32's range
      // where rstd is 1e18)
      const Same<V> minus(-mean[k]), scale(rstd[k]), less(-off), slope(-rstd[k] * c2), shift(-rstd[k] * c1);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        float x[V], g[V];
        if constexpr (AHEAD) {
          rx[k][i] = *place(now, k, 0, i);
          rd[k][i] = *place(now, k, 1, i);
        } else {
          keep_packed<B>(rx[k][i]);
          keep_packed<B>(rd[k][i]);
        }
        raw_to_f32<T, B>(rx[k][i], x);
        raw_to_f32<T, B>(rd[k][i], g);
        add_n(x, x, minus.v);
        fma_n(x, x, scale.v, less.v);
        fma_n(dw[i], g, x, dw[i]);  // (of values that are not there g is zero, or nobody reads dw)
        times_weight(i, g);
        fma_n(x, x, slope.v, shift.v);
        fma_n(g, g, scale.v, x);
        if (a.dx && r < a.rows && i < n) store_raw<B>(dx + i * G * V, f32_to_raw<T, B>(g));
      }
    }
  }
  if constexpr (AHEAD) asm volatile("cp.async.wait_all;\n" ::: "memory");
  if (!sums) return;
  float* const join = reinterpret_cast<float*>(ahead);
  if (groups > 1) __syncthreads();  // (other threads' batches were there)
  float* part = a.part + static_cast<long long>(blockIdx.x) * 2 * width;
  float* to = groups > 1 ? join + group * 2 * width : part;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int c = (i * G + t) * V;
    if (c < width) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        to[c + j] = dw[i][j];
        to[width + c + j] = db[i][j];
      }
    }
  }
  if (groups == 1) return;
  __syncthreads();
  for (int c = threadIdx.x; c < 2 * width; c += blockDim.x) {
    float s = 0.0f;
    for (int k = 0; k < groups; ++k) s += join[k * 2 * width + c];
    part[c] = s;
  }
}

// Rows of any width: two passes over the row, one over x alone where dx is not wanted.  `rows` (if not nullptr) receives for
// the columns' sums a row's mean, rstd, and what the mean's rounding left in its xhat.  (No early launch of what follows: that
// kernel's blocks, waiting among this one's, cost 40 us of 4096 rows of 16384 float32.)
template <typename T, bool WEIGHT>
__global__ void __launch_bounds__(1024) norm_backward_stream(const NormArgs a, float4* const rows) {
  __shared__ float red[2][3][32];
  int turn = 0;
  griddep_wait();
  const int width = static_cast<int>(a.width);
  for (long long r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + r * a.ldx;
    const T* dy = static_cast<const T*>(a.dy) + r * a.ldy;
    T* dx = static_cast<T*>(a.dx) + r * a.width;
    const float2 stats = *reinterpret_cast<const float2*>(a.stats + 2 * r);
    const float mean = stats.x, rstd = stats.y;
    auto gradient = [&](int c) {
      const float g = to_f32(dy[c]);
      return WEIGHT ? g * to_f32(static_cast<const T*>(a.w)[c]) : g;
    };
    float s[3] = {0.0f, 0.0f, 0.0f};
    if (a.dx) {
#pragma unroll 4
      for (int c = threadIdx.x; c < width; c += 1024) {
        const float g = gradient(c), h = __fmul_rn(to_f32(x[c]) - mean, rstd);  // (rounded by itself: the same sum below)
        s[0] += g;
        s[1] = fmaf(g, h, s[1]);
        s[2] += h;
      }
    } else {
#pragma unroll 4
      for (int c = threadIdx.x; c < width; c += 1024) s[2] += __fmul_rn(to_f32(x[c]) - mean, rstd);
    }
    block_sum<3>(s, red, turn);
    const float n = static_cast<float>(width), c1 = s[0] / n, off = s[2] / n, c2 = fmaf(-off, c1, s[1] / n);
    if (rows && threadIdx.x == 0) rows[r] = make_float4(mean, rstd, off, 0.0f);
    if (!a.dx) continue;
#pragma unroll 4
    for (int c = threadIdx.x; c < width; c += 1024)
      dx[c] = from_f32<T>(rstd * (gradient(c) - c1 - fmaf(to_f32(x[c]) - mean, rstd, -off) * c2));
  }
}
// The column sums of wide rows: a block has 256 columns of one range of rows.
template <typename T>
__global__ void __launch_bounds__(256) norm_columns_stream(const NormArgs a, const float4* const rows, const long long per) {
  griddep_wait();
  griddep_launch();
  const long long c = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
  if (c >= a.width) return;
  const long long r0 = blockIdx.y * per, r1 = min(a.rows, r0 + per);
  float dw = 0.0f, db = 0.0f;
#pragma unroll 8
  for (long long r = r0; r < r1; ++r) {
    const float4 f = rows[r];
    const float g = to_f32(static_cast<const T*>(a.dy)[r * a.ldy + c]);
    dw = fmaf(g, fmaf(to_f32(static_cast<const T*>(a.x)[r * a.ldx + c]) - f.x, f.y, -f.z), dw);
    db += g;
  }
  float* part = a.part + static_cast<long long>(blockIdx.y) * 2 * a.width;
  part[c] = dw;
  part[a.width + c] = db;
}

// Adds the blocks' sums in their order: ranges of blocks for 32 columns, then the ranges.
template <typename T>
__global__ void __launch_bounds__(kRanges * kColumns) norm_join(const NormArgs a, const int parts) {
  __shared__ float red[kRanges][kColumns + 1];
  griddep_wait();
  griddep_launch();
  const int lane = threadIdx.x % kColumns, k = threadIdx.x / kColumns;
  const long long c = static_cast<long long>(blockIdx.x) * kColumns + lane;  // of both gradients, one after the other
  const int per = (parts + kRanges - 1) / kRanges, p1 = min(parts, (k + 1) * per);
  float s = 0.0f;
  if (c < 2 * a.width) {
#pragma unroll 4
    for (int p = k * per; p < p1; ++p) s += a.part[static_cast<long long>(p) * 2 * a.width + c];
  }
  red[k][lane] = s;
  __syncthreads();
  // a warp adds the ranges of a column
  s = warp_sum(red[lane][k]);
  const long long to = static_cast<long long>(blockIdx.x) * kColumns + k;
  if (lane != 0 || to >= 2 * a.width) return;
  if (to < a.width) {
    if (a.dw) static_cast<T*>(a.dw)[to] = from_f32<T>(s);
  } else if (a.db) {
    static_cast<T*>(a.db)[to - a.width] = from_f32<T>(s);
  }
}

// A group spans the row with `values` a thread; a block has as many groups as fit.  values 0: the row does not fit.
struct BackShape {
  int values, warps, groups, threads, blocks;
};
BackShape back_shape(long long rows, long long width, int es, int sm) {
  BackShape s = {};
  const int base = 16 / es;  // values of 16 bytes
  // no more a thread than the row needs (twice as many where half would do, bfloat16: 1024 wide 39.3 us in place of 38.0,
  // 2048 wide 39.9 and 38.8, 4096 wide 40.9 and 40.6, 515 wide 114 and 96)
  for (int v = base; v <= 4 * base && s.values == 0; v *= 2)
    if (width <= static_cast<long long>(kThreads) * v) s.values = v;
  if (s.values == 0) return s;
  s.warps = static_cast<int>((width + 32LL * s.values - 1) / (32LL * s.values));
  s.groups = kThreads / (32 * s.warps);
  s.threads = 32 * s.warps * s.groups;
  s.blocks = static_cast<int>(std::min<long long>((rows + s.groups - 1) / s.groups, sm));
  return s;
}
bool streams(long long width, int es, bool stream) { return stream || back_shape(1, width, es, 1).values == 0; }
// Blocks of rows whose sums of dweight and dbias go to `part`.
long long parts_of(long long rows, long long width, int es, bool stream, int sm) {
  if (streams(width, es, stream)) {
    const long long strips = (width + 255) / 256;
    return std::max<long long>(1, std::min({8LL * sm / strips, (rows + kStreamRows - 1) / kStreamRows, 65535LL}));
  }
  return back_shape(rows, width, es, sm).blocks;
}
size_t part_floats(long long parts, long long width) { return (static_cast<size_t>(parts) * 2 * width + 3) / 4 * 4; }

template <typename T, int B, int E, int R>
cudaError_t go(const NormArgs& a, const BackShape& sh, int sums, cudaStream_t s) {
  auto kern = a.w ? norm_backward<T, B, E, R, true> : norm_backward<T, B, E, R, false>;
  size_t smem = sums && sh.groups > 1 ? static_cast<size_t>(sh.groups) * 2 * a.width * sizeof(float) : 0;
  if (B == 16) smem = std::max(smem, static_cast<size_t>(kStages) * R * 2 * E * sizeof(T) * sh.threads);
  if (smem > 32768) {  // (with the fixed part more than 48 KB)
    const cudaError_t err = opt_in_smem(reinterpret_cast<const void*>(kern), smem);
    if (err != cudaSuccess) return err;
  }
  return launch_overlapped(kern, dim3(static_cast<unsigned>(sh.blocks)), sh.threads, smem, 1, s, a, sums, sh.warps);
}
// Rows at a time: 64 bytes of x in flight a thread where registers have room (2-byte accesses take a register each).
template <typename T, int B>
cudaError_t by_values(const NormArgs& a, const BackShape& sh, int sums, cudaStream_t s) {
  constexpr int P = 16 / sizeof(T);
  if (sh.values == P) return go<T, B, P, B == 2 ? 2 : 4>(a, sh, sums, s);
  if (sh.values == 2 * P) return go<T, B, 2 * P, B == 2 ? 1 : 2>(a, sh, sums, s);
  return go<T, B, 4 * P, 1>(a, sh, sums, s);
}
template <typename T>
cudaError_t by_type(const NormArgs& a, bool stream, int sm, cudaStream_t s) {
  const int sums = a.dw || a.db;
  const int parts = static_cast<int>(parts_of(a.rows, a.width, sizeof(T), stream, sm));
  cudaError_t err = cudaSuccess;
  if (streams(a.width, sizeof(T), stream)) {
    float4* const rows = sums ? reinterpret_cast<float4*>(a.part + part_floats(parts, a.width)) : nullptr;
    if (a.dx || sums)
      err = launch_overlapped(a.w ? norm_backward_stream<T, true> : norm_backward_stream<T, false>,
                              dim3(static_cast<unsigned>(std::min<long long>(a.rows, 2LL * sm))), 1024, 0, 1, s, a, rows);
    if (err == cudaSuccess && sums)
      err = launch_overlapped(norm_columns_stream<T>, dim3(static_cast<unsigned>((a.width + 255) / 256), static_cast<unsigned>(parts)),
                              256, 0, 1, s, a, rows, (a.rows + parts - 1) / parts);
  } else if (a.dx || sums) {
    const BackShape sh = back_shape(a.rows, a.width, sizeof(T), sm);
    const int bytes = access_bytes(sizeof(T), a.width, {a.x, a.w, a.dy, a.dx},
                                   {a.rows > 1 ? a.ldx : 0, a.rows > 1 ? a.ldy : 0});
    if (bytes == 16) err = by_values<T, 16>(a, sh, sums, s);
    else if constexpr (sizeof(T) == 2)
      err = bytes == 2 ? by_values<T, 2>(a, sh, sums, s) : by_values<T, 4>(a, sh, sums, s);
    else err = by_values<T, 4>(a, sh, sums, s);
  }
  if (err != cudaSuccess || !sums) return err;
  return launch_overlapped(norm_join<T>, dim3(static_cast<unsigned>((2 * a.width + kColumns - 1) / kColumns)), kRanges * kColumns, 0, 1, s,
                           a, parts);
}

}  // namespace

size_t norm_backward_scratch(long long rows, long long width, int es, bool stream, int sm) {
  return part_floats(parts_of(rows, width, es, stream, sm), width) * sizeof(float) +
         (streams(width, es, stream) ? static_cast<size_t>(rows) * sizeof(float4) : 0);
}

cudaError_t launch_norm_backward(const NormArgs& a, int dtype, bool stream, int sm, cudaStream_t s) {
  return dtype == CONV_F32 ? by_type<float>(a, stream, sm, s) : dtype == CONV_F16 ? by_type<__half>(a, stream, sm, s)
                                                                                  : by_type<__nv_bfloat16>(a, stream, sm, s);
}

}  // namespace conv
