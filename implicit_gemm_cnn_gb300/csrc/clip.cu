// clip.cu -- the global norm of many tensors, and the tensors scaled to it.
//
// Two passes over the data, bound by its bytes: one that reads everything into
// one float64 sum per block, and one that adds those sums in their order, then
// reads everything again and writes it scaled.  The tensors' addresses and
// sizes travel as kernel parameters (no copy to the device, nothing kept
// between calls); work is cut into chunks of kChunk elements of one tensor, so
// that short and long tensors fill the same grid.
//
// Measured, 300 tensors, 800 million bfloat16: the norm 253 us (6.3 TB/s, 93% of
// measured), the scaling 495 us (6.5 TB/s).  40 tensors of 150 thousand float32
// in all: 6 and 8 us, less than the call's host side (some 1.2 us a tensor).
//
// The sum: a thread squares and adds kVecs 16-byte vectors in float32 and adds
// that to a float64; no conversion per element (the FP64 units do two
// operations a clock per SM).  With float32's range the squares could overflow
// or vanish, so a group whose largest element lies outside [2^-40, 2^55] is
// taken again, scaled by a power of two: inside that range 32 squares stay
// below 2^115, and what vanishes is below 2^-126 beside at least 2^-80.
#include <algorithm>

#include "dense_internal.h"

namespace conv {
namespace {

constexpr int kThreads = 256;
constexpr int kVecs = 4;          // 16-byte vectors a thread has in flight
constexpr int kChunk = 16384;     // elements

template <int CAP>
struct ClipTable {
  const void* in[CAP];
  void* out[CAP];
  long long size[CAP];
  int first[CAP + 1];   // a tensor's first chunk; first[count] = all chunks
  uint8_t type[CAP];
  int count;
};

template <int CAP>
__device__ __forceinline__ int find_tensor(const ClipTable<CAP>& t, int chunk) {
  int lo = 0, hi = t.count;  // first[lo] <= chunk < first[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (t.first[mid] <= chunk) lo = mid; else hi = mid;
  }
  return lo;
}

// Elements of a 16-byte vector as float32.
template <typename T>
__device__ __forceinline__ void unpack(const uint4& q, float (&v)[16 / sizeof(T)]) {
  if constexpr (sizeof(T) == 4) {
    v[0] = __uint_as_float(q.x); v[1] = __uint_as_float(q.y); v[2] = __uint_as_float(q.z); v[3] = __uint_as_float(q.w);
  } else {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
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
template <typename T>
__device__ __forceinline__ uint4 pack(const float (&v)[16 / sizeof(T)]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 4) w[i] = __float_as_uint(v[i]);
    else if constexpr (std::is_same<T, __nv_bfloat16>::value) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    } else {
      const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// The sum of squares of N values, in float64 range.
template <bool WIDE, int N>
__device__ __forceinline__ double squares(const float (&v)[N]) {
  float s = 0.0f, m = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    s = fmaf(v[i], v[i], s);
    if (WIDE) m = fmaxf(m, fabsf(v[i]));
  }
  if (WIDE && (m > 0x1p55f || (m < 0x1p-40f && m > 0.0f)) && m <= 3.402823466e38f && !(s != s)) {
    const float f = m > 1.0f ? 0x1p-80f : 0x1p100f;
    float t = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float x = v[i] * f;
      t = fmaf(x, x, t);
    }
    return static_cast<double>(t) * (m > 1.0f ? 0x1p160 : 0x1p-200);
  }
  return s;
}

// The part of a tensor that chunk c of it covers.  Chunks begin on 16-byte
// boundaries: all of them are shifted by the `head` elements before the first
// one, which the first chunk takes as well.
struct Span {
  long long body, end;  // vectors from `body` on; the last end - body elements may be no whole vector
  int head;
};
template <typename T>
__device__ __forceinline__ Span span_of(const void* base, long long size, int c) {
  constexpr int V = 16 / sizeof(T);
  Span s;
  const int mis = static_cast<int>(reinterpret_cast<uintptr_t>(base) % 16 / sizeof(T));
  const int head = static_cast<int>(min(static_cast<long long>((V - mis) % V), size));
  s.head = c == 0 ? head : 0;
  s.body = min(static_cast<long long>(c) * kChunk + head, size);
  s.end = min(s.body + kChunk, size);
  return s;
}

template <typename T>
__device__ __forceinline__ double chunk_squares(const void* base, long long size, int c) {
  constexpr int V = 16 / sizeof(T);
  constexpr bool WIDE = !std::is_same<T, __half>::value;  // half's squares need no scaling
  const T* p = static_cast<const T*>(base);
  const Span sp = span_of<T>(base, size, c);
  double acc = 0.0;
  const int vecs = static_cast<int>((sp.end - sp.body) / V);
  const uint4* q = reinterpret_cast<const uint4*>(p + sp.body);
  for (int i0 = threadIdx.x; i0 < vecs; i0 += kThreads * kVecs) {
    uint4 r[kVecs];
#pragma unroll
    for (int u = 0; u < kVecs; ++u)
      r[u] = i0 + u * kThreads < vecs ? __ldg(q + i0 + u * kThreads) : make_uint4(0, 0, 0, 0);
    float v[kVecs * V];
#pragma unroll
    for (int u = 0; u < kVecs; ++u) {
      float w[V];
      unpack<T>(r[u], w);
#pragma unroll
      for (int j = 0; j < V; ++j) v[u * V + j] = w[j];
    }
    acc += squares<WIDE, kVecs * V>(v);
  }
  const int tail = static_cast<int>(sp.end - sp.body) - vecs * V;
  const int t = threadIdx.x;
  if (t < sp.head + tail) {
    const float v[1] = {to_f32(p[t < sp.head ? t : sp.body + vecs * V + (t - sp.head)])};
    acc += squares<WIDE, 1>(v);
  }
  return acc;
}

__device__ __forceinline__ double block_sum(double v) {
  __shared__ double part[kThreads / 32];
#pragma unroll
  for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = v;
  __syncthreads();
  double s = 0.0;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) s += part[i];
  return s;
}

template <int CAP>
__global__ void __launch_bounds__(kThreads) clip_norm(const __grid_constant__ ClipTable<CAP> t, double* part) {
  griddep_wait();
  griddep_launch();
  double acc = 0.0;
  const int chunks = t.first[t.count];
  for (int c = blockIdx.x; c < chunks; c += gridDim.x) {
    const int i = find_tensor(t, c);
    const int own = c - t.first[i];
    switch (t.type[i]) {
      case CONV_F32: acc += chunk_squares<float>(t.in[i], t.size[i], own); break;
      case CONV_F16: acc += chunk_squares<__half>(t.in[i], t.size[i], own); break;
      default: acc += chunk_squares<__nv_bfloat16>(t.in[i], t.size[i], own); break;
    }
  }
  acc = block_sum(acc);
  if (threadIdx.x == 0) part[blockIdx.x] = acc;
}

template <typename T>
__device__ __forceinline__ void chunk_scale(const void* base, void* out, long long size, int c, float scale) {
  constexpr int V = 16 / sizeof(T);
  const T* p = static_cast<const T*>(base);
  T* o = static_cast<T*>(out);
  const Span sp = span_of<T>(base, size, c);
  const int t = threadIdx.x;
  if (reinterpret_cast<uintptr_t>(o + sp.body) % 16 == 0) {
    const int vecs = static_cast<int>((sp.end - sp.body) / V);
    const uint4* q = reinterpret_cast<const uint4*>(p + sp.body);
    uint4* w = reinterpret_cast<uint4*>(o + sp.body);
    for (int i0 = t; i0 < vecs; i0 += kThreads * kVecs) {
      uint4 r[kVecs];
#pragma unroll
      for (int u = 0; u < kVecs; ++u)
        if (i0 + u * kThreads < vecs) r[u] = __ldcs(q + i0 + u * kThreads);
#pragma unroll
      for (int u = 0; u < kVecs; ++u)
        if (i0 + u * kThreads < vecs) {
          float v[V];
          unpack<T>(r[u], v);
#pragma unroll
          for (int j = 0; j < V; ++j) v[j] *= scale;
          __stcs(w + i0 + u * kThreads, pack<T>(v));
        }
    }
    const int tail = static_cast<int>(sp.end - sp.body) - vecs * V;
    if (t < sp.head + tail) {
      const long long at = t < sp.head ? t : sp.body + vecs * V + (t - sp.head);
      o[at] = from_f32<T>(to_f32(p[at]) * scale);
    }
  } else {  // in and out lie differently within 16 bytes: element by element
    if (t < sp.head) o[t] = from_f32<T>(to_f32(p[t]) * scale);
    for (long long i = sp.body + t; i < sp.end; i += kThreads) o[i] = from_f32<T>(to_f32(p[i]) * scale);
  }
}

// Every block adds the sums in the same order.  Chunks run from the last to the
// first: the norm pass left the last ones in the L2 cache.
template <int CAP>
__global__ void __launch_bounds__(kThreads) clip_scale(const __grid_constant__ ClipTable<CAP> t, const double* part,
                                                       int parts, float max_norm, float eps, float* norm) {
  griddep_wait();
  griddep_launch();
  double s = 0.0;
  for (int i = threadIdx.x; i < parts; i += kThreads) s += part[i];
  const double total = sqrt(block_sum(s));
  if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = static_cast<float>(total);
  const double ratio = static_cast<double>(max_norm) / (total + static_cast<double>(eps));
  // min(1, ratio) that keeps a NaN; 0 / 0 (no gradient, no bound, no eps) scales by 1
  float scale = ratio >= 1.0 ? 1.0f : static_cast<float>(ratio);
  if (total == 0.0) scale = 1.0f;
  const int chunks = t.first[t.count];
  for (int k = blockIdx.x; k < chunks; k += gridDim.x) {
    const int c = chunks - 1 - k;
    const int i = find_tensor(t, c);
    const int own = c - t.first[i];
    switch (t.type[i]) {
      case CONV_F32: chunk_scale<float>(t.in[i], t.out[i], t.size[i], own, scale); break;
      case CONV_F16: chunk_scale<__half>(t.in[i], t.out[i], t.size[i], own, scale); break;
      default: chunk_scale<__nv_bfloat16>(t.in[i], t.out[i], t.size[i], own, scale); break;
    }
  }
}

constexpr int kSmall = 64, kLarge = 1024;  // 1.9 and 30 KB of parameters
constexpr int kMaxBlocks = 2048;           // sums of one launch

// The non-empty tensors [at, ...) that fit a table; returns where the next one begins.
template <int CAP>
long long fill(ClipTable<CAP>* t, long long at, long long count, const void* const* in, void* const* out,
               const int64_t* sizes, const int32_t* dtypes) {
  t->count = 0;
  long long chunks = 0;
  for (; at < count && t->count < CAP; ++at) {
    if (sizes[at] == 0) continue;
    const long long c = (sizes[at] + kChunk - 1) / kChunk;
    if (t->count > 0 && chunks + c > (1LL << 30)) break;
    const int i = t->count++;
    t->in[i] = in[at];
    t->out[i] = out ? out[at] : nullptr;
    t->size[i] = sizes[at];
    t->type[i] = static_cast<uint8_t>(dtypes[at]);
    t->first[i] = static_cast<int>(chunks);
    chunks += c;
  }
  t->first[t->count] = static_cast<int>(chunks);
  return at;
}

template <int CAP>
cudaError_t run(long long count, const void* const* in, void* const* out, const int64_t* sizes, const int32_t* dtypes,
                float max_norm, float eps, float* norm, double* part, int sm, cudaStream_t s) {
  ClipTable<CAP> t;
  auto blocks_of = [&] { return std::min({std::max(t.first[t.count], 1), 8 * sm, kMaxBlocks}); };
  int parts = 0, launches = 0;
  long long at = 0;
  do {
    at = fill(&t, at, count, in, out, sizes, dtypes);
    const int blocks = blocks_of();
    const cudaError_t err = launch_overlapped(clip_norm<CAP>, dim3(static_cast<unsigned>(blocks)), kThreads, 0, 1, s, t,
                                              part + parts);
    if (err != cudaSuccess) return err;
    parts += blocks;
    ++launches;
  } while (at < count);
  if (!out) {
    t.count = 0;
    t.first[0] = 0;
  } else if (launches > 1) {  // (else the table is the norm's)
    at = fill(&t, 0, count, in, out, sizes, dtypes);
  }
  for (bool first = true;; first = false) {
    const cudaError_t err = launch_overlapped(clip_scale<CAP>, dim3(static_cast<unsigned>(blocks_of())), kThreads, 0, 1, s, t,
                                              part, parts, max_norm, eps, first ? norm : static_cast<float*>(nullptr));
    if (err != cudaSuccess) return err;
    if (!out || at >= count) break;
    at = fill(&t, at, count, in, out, sizes, dtypes);
  }
  return cudaSuccess;
}

}  // namespace

size_t clip_scratch_bytes(long long count, const int64_t* sizes) {
  // one float64 per block of every norm launch: a launch ends at kLarge tensors or 2^30 chunks
  long long launches = 1, tensors = 0, chunks = 0;
  for (long long i = 0; i < count; ++i) {
    if (sizes[i] == 0) continue;
    const long long c = (sizes[i] + kChunk - 1) / kChunk;
    if (tensors == kLarge || (tensors > 0 && chunks + c > (1LL << 30))) { ++launches; tensors = 0; chunks = 0; }
    ++tensors;
    chunks += c;
  }
  return static_cast<size_t>(launches) * kMaxBlocks * sizeof(double);
}

cudaError_t launch_clip(long long count, const void* const* in, void* const* out, const int64_t* sizes,
                        const int32_t* dtypes, float max_norm, float eps, float* norm, void* scratch, int sm,
                        cudaStream_t s) {
  double* part = static_cast<double*>(scratch);
  return count <= kSmall ? run<kSmall>(count, in, out, sizes, dtypes, max_norm, eps, norm, part, sm, s)
                         : run<kLarge>(count, in, out, sizes, dtypes, max_norm, eps, norm, part, sm, s);
}

}  // namespace conv
