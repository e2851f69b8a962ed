// dense_ffma.cu -- the dense products on the CUDA cores: 16-bit operands off
// 16-byte boundaries where there is no scratch for their copies, and any problem
// that asks for this kernel (CONV_LINEAR_FLAG_FORCE_FFMA).  Also the ordered sum
// of its k ranges, the operands' copies, and the elementwise helpers of the
// backward passes.
//
// A block computes a BM x BN tile of D = A B^T in register tiles of TM x TN per
// thread, operands staged k-row by k-row in shared memory (As[k][m], Bs[k][n])
// as float32, the next stage's values held in registers while the current one
// is multiplied.  A thread's rows and columns are groups of four, half a tile
// apart, so that its shared-memory reads are 16 bytes and free of bank
// conflicts.  The same split serves the gated product: the column groups of
// the first half are gate columns, those of the second half the up columns of
// the same positions, so g and u of one element meet in one thread.
//
// Measured: 1001 x 515 -> 1030 float32 51 us (20.7 TFLOP/s, 272 tiles of 64 x
// 64 on 152 SMs), where the tensor-core kernel takes 26.
#include <algorithm>

#include "dense_internal.h"

namespace conv {
namespace {

constexpr int kThreads = 256;
constexpr int kBK = 16;

// One operand's stage: R = 16 * T / kThreads values per thread.  k-major: 16
// consecutive k of a row (64 or 32 bytes) per 16 lanes; mn-major: whole rows of
// consecutive m.
template <typename T, int TILE>
struct Loader {
  static constexpr int R = TILE * kBK / kThreads;
  const T* p;
  long long step_i, step_k;  // between a thread's values; between stages
  int r0, k0, dr, dk;        // the first value's row and k in the tile, and their steps
  __device__ __forceinline__ void init(const void* base, long long ld, int mn, int row, long long k, int tid) {
    if (mn) {
      r0 = tid % TILE; k0 = tid / TILE; dr = 0; dk = kThreads / TILE;
      p = static_cast<const T*>(base) + (k + k0) * ld + row + r0;
      step_i = dk * ld; step_k = kBK * ld;
    } else {
      r0 = tid / kBK; k0 = tid % kBK; dr = kThreads / kBK; dk = 0;
      p = static_cast<const T*>(base) + (row + r0) * ld + k + k0;
      step_i = dr * ld; step_k = kBK;
    }
  }
  // values of the stage; `rows`, `ks`: how many of the tile's rows and of the stage's k exist
  __device__ __forceinline__ void load(float (&v)[R], int rows, long long ks) {
#pragma unroll
    for (int i = 0; i < R; ++i)
      v[i] = (r0 + i * dr < rows && k0 + i * dk < ks) ? to_f32(p[i * step_i]) : 0.0f;
    p += step_k;
  }
  template <int P>
  __device__ __forceinline__ void store(float (&s)[kBK][P], const float (&v)[R], int at) const {
#pragma unroll
    for (int i = 0; i < R; ++i) s[k0 + i * dk][at + r0 + i * dr] = v[i];
  }
};

template <typename T, int BM, int BN, bool DUAL>
__global__ void __launch_bounds__(kThreads, BM * BN >= 128 * 128 ? 1 : 2) dense_ffma(const DenseGemm g) {
  constexpr int TM = BM / 16, TN = BN / 16;
  constexpr int BNL = DUAL ? BN / 2 : BN;  // columns of the output tile
  griddep_wait();
  griddep_launch();
  __shared__ float As[2][kBK][BM + 4];
  __shared__ float Bs[2][kBK][BN + 4];
  const int tid = threadIdx.x, tx = tid % 16, ty = tid / 16;
  const int products = DUAL ? 1 : g.batch;
  const int which = blockIdx.z % products, range = blockIdx.z / products;
  const int ntiles = (g.N + BNL - 1) / BNL;
  const int m0 = static_cast<int>(blockIdx.x / ntiles) * BM, n0 = static_cast<int>(blockIdx.x % ntiles) * BNL;
  const int rows_a = min(BM, g.M - m0), rows_b = min(BNL, g.N - n0);

  float acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = 0.0f;

  const long long k_end_all = static_cast<long long>(g.segs) * g.K;
  const long long k_lo = range * g.k_per_split;
  const long long k_hi = min(k_lo + g.k_per_split, k_end_all);
  for (int seg = 0; seg < g.segs; ++seg) {
    // this segment's part of the range
    const long long lo = max(k_lo - static_cast<long long>(seg) * g.K, 0LL);
    const long long hi = min(k_hi - static_cast<long long>(seg) * g.K, static_cast<long long>(g.K));
    if (lo >= hi) continue;
    Loader<T, BM> la;
    Loader<T, BNL> lb, lb2;
    const int op = g.segs > 1 ? seg : which;
    la.init(g.a[op], g.lda, g.a_mn, m0, lo, tid);
    lb.init(g.b[op], g.ldb, g.b_mn, n0, lo, tid);
    if (DUAL) lb2.init(g.b[1], g.ldb, g.b_mn, n0, lo, tid);
    float va[Loader<T, BM>::R], vb[Loader<T, BNL>::R], vb2[DUAL ? Loader<T, BNL>::R : 1];
    auto load = [&](long long k) {
      la.load(va, rows_a, hi - k);
      lb.load(vb, rows_b, hi - k);
      if constexpr (DUAL) lb2.load(vb2, rows_b, hi - k);
    };
    auto store = [&](int s) {
      la.store(As[s], va, 0);
      lb.store(Bs[s], vb, 0);
      if constexpr (DUAL) lb2.store(Bs[s], vb2, BNL);
    };
    __syncthreads();  // the previous segment's last stage has been read
    load(lo);
    store(0);
    __syncthreads();
    int s = 0;
    for (long long k = lo; k < hi; k += kBK) {
      const bool more = k + kBK < hi;
      if (more) load(k + kBK);
#pragma unroll
      for (int kk = 0; kk < kBK; ++kk) {
        float a[TM], b[TN];
#pragma unroll
        for (int i = 0; i < TM; i += 4)
          *reinterpret_cast<float4*>(a + i) = *reinterpret_cast<const float4*>(&As[s][kk][i / 4 * (BM / 2) + ty * 4]);
#pragma unroll
        for (int j = 0; j < TN; j += 4)
          *reinterpret_cast<float4*>(b + j) = *reinterpret_cast<const float4*>(&Bs[s][kk][j / 4 * (BN / 2) + tx * 4]);
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
          for (int j = 0; j < TN; ++j) acc[i][j] = fmaf(a[i], b[j], acc[i][j]);
      }
      if (more) {
        store(s ^ 1);  // read last before the previous barrier
        __syncthreads();
        s ^= 1;
      }
    }
  }

  constexpr int NC = DUAL ? TN / 2 : TN;
  int col[NC];
  bool okc[NC];
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    col[j] = n0 + (DUAL ? 0 : j / 4 * (BN / 2)) + tx * 4 + j % 4;
    okc[j] = col[j] < g.N;
  }
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    const int m = m0 + i / 4 * (BM / 2) + ty * 4 + i % 4;
    if (m >= g.M) continue;
    if (g.split > 1) {
      const long long plane = static_cast<long long>(g.M) * g.N;
      const int planes = DUAL ? 2 : products;
      float* part = g.part + (static_cast<long long>(range) * planes + which) * plane + static_cast<long long>(m) * g.N;
#pragma unroll
      for (int j = 0; j < NC; ++j)
        if (okc[j]) {
          part[col[j]] = acc[i][j];
          if constexpr (DUAL) part[plane + col[j]] = acc[i][j + NC];
        }
    } else {
      float v[NC], u[NC];
#pragma unroll
      for (int j = 0; j < NC; ++j) {
        v[j] = acc[i][j];
        u[j] = DUAL ? acc[i][j + (DUAL ? NC : 0)] : 0.0f;
      }
      dense_epilogue<T, NC>(g.epi, which, m, col, okc, v, u);
    }
  }
}

// y[m][n] from the planes of the k ranges: four columns per thread.
template <typename T>
__global__ void __launch_bounds__(256) dense_reduce(const DenseGemm g) {
  griddep_wait();
  griddep_launch();
  const long long quads = (static_cast<long long>(g.N) + 3) / 4;
  const long long idx = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
  if (idx >= quads * g.M) return;
  const int which = blockIdx.y;
  const int m = static_cast<int>(idx / quads), n = static_cast<int>(idx % quads) * 4;
  const long long plane = static_cast<long long>(g.M) * g.N;
  const int planes = g.dual ? 2 : g.batch;
  const float* p = g.part + which * plane + static_cast<long long>(m) * g.N + n;
  float v[4] = {0, 0, 0, 0}, u[4] = {0, 0, 0, 0};
  int col[4];
  bool ok[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) { col[j] = n + j; ok[j] = n + j < g.N; }
  const bool vec = g.N % 4 == 0;  // planes are 16-byte aligned then
#pragma unroll 4
  for (int s = 0; s < g.split; ++s) {  // (loads of four ranges in flight; added in order)
    if (vec) {
      const float4 t = *reinterpret_cast<const float4*>(p);
      v[0] += t.x; v[1] += t.y; v[2] += t.z; v[3] += t.w;
      if (g.dual) {
        const float4 q = *reinterpret_cast<const float4*>(p + plane);
        u[0] += q.x; u[1] += q.y; u[2] += q.z; u[3] += q.w;
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (ok[j]) {
          v[j] += p[j];
          if (g.dual) u[j] += p[plane + j];
        }
    }
    p += planes * plane;
  }
  dense_epilogue<T, 4>(g.epi, which, m, col, ok, v, u);
}

// The three planes of 4 values: v = p0 + 2^-kPlaneScale1 p1 + 2^-kPlaneScale2 p2, exactly, for every float32 down to the
// smallest subnormal: unscaled, p1 and p2 of values below 2^-110 would end where bfloat16's range does (2^-133).  |p1| and
// |p2| stay below |v| / 2 (of a value below 2^-134, below 2^-126).  An infinity or a NaN is its own first plane; a value that
// would round up to infinity is cut instead, and one that would round to zero becomes the smallest p0 (an infinity times it is
// one, not NaN).
__device__ __forceinline__ void put_planes(const float (&v)[4], __nv_bfloat16* out, long long plane) {
  constexpr float kUp1 = 1u << kPlaneScale1, kUp2 = 1u << (kPlaneScale2 - kPlaneScale1);
  uint16_t h[3][4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    __nv_bfloat16 p0 = __float2bfloat16_rn(v[j]);
    const bool finite = fabsf(v[j]) <= 3.402823466e38f;
    if (finite && __hisinf(p0)) p0 = __float2bfloat16_rz(v[j]);
    if (__bfloat162float(p0) == 0.0f && v[j] != 0.0f)
      p0 = __ushort_as_bfloat16(static_cast<uint16_t>((__float_as_uint(v[j]) >> 16) & 0x8000u | 1u));
    const float r1 = finite ? (v[j] - __bfloat162float(p0)) * kUp1 : 0.0f;
    const __nv_bfloat16 p1 = __float2bfloat16_rn(r1);
    const __nv_bfloat16 p2 = __float2bfloat16_rn((r1 - __bfloat162float(p1)) * kUp2);
    h[0][j] = __bfloat16_as_ushort(p0);
    h[1][j] = __bfloat16_as_ushort(p1);
    h[2][j] = __bfloat16_as_ushort(p2);
  }
#pragma unroll
  for (int q = 0; q < 3; ++q)
    *reinterpret_cast<uint2*>(out + q * plane) =
        make_uint2(h[q][0] | (static_cast<uint32_t>(h[q][1]) << 16), h[q][2] | (static_cast<uint32_t>(h[q][3]) << 16));
}

// Operands' copies, bound by their bytes (30 MB of weights with odd rows 13 us).  A warp takes 256 columns of a row at a
// time: 16-bit rows as they are, or float32 rows as three planes (rows of the planes are a multiple of 64 long, so whole
// groups of four are written).  Blocks walk over the jobs' pieces together.
struct CopyJobs {
  CopyJob job[kCopyJobs];
  long long first[kCopyJobs + 1];
  int count;
};
template <bool PLANES>
__global__ void __launch_bounds__(256) dense_copies(const __grid_constant__ CopyJobs c) {
  griddep_wait();
  griddep_launch();
  const int lane = threadIdx.x % 32;
  const long long warps = static_cast<long long>(gridDim.x) * 8;
  int j = 0;
  for (long long w = static_cast<long long>(blockIdx.x) * 8 + threadIdx.x / 32; w < c.first[c.count]; w += warps) {
    while (w >= c.first[j + 1]) ++j;
    const CopyJob& job = c.job[j];
    const long long chunks = (job.cols + 255) / 256, i = w - c.first[j];
    const long long r = i / chunks, c0 = i % chunks * 256;
    if constexpr (PLANES) {
      const float* src = static_cast<const float*>(job.in) + r * job.ld_in;
      __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(job.out) + r * job.ld;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const long long col = c0 + h * 128 + lane * 4;
        if (col >= job.cols) continue;
        float v[4];
        if (col + 4 <= job.cols && reinterpret_cast<uintptr_t>(src + col) % 16 == 0) {
          const float4 f = *reinterpret_cast<const float4*>(src + col);
          v[0] = f.x; v[1] = f.y; v[2] = f.z; v[3] = f.w;
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k) v[k] = col + k < job.cols ? src[col + k] : 0.0f;
        }
        put_planes(v, dst + col, job.rows * job.ld);
      }
    } else {
      // A lane writes eight values (16 bytes): out of the two aligned 16-byte pieces that they lie in, where both are
      // inside the matrix, shifted together; else one by one.
      const char* first = static_cast<const char*>(job.in);
      const char* end = first + ((job.rows - 1) * job.ld_in + job.cols) * 2;
      const long long col = c0 + 8 * lane;
      if (col >= job.cols) continue;
      const char* src = first + (r * job.ld_in + col) * 2;
      uint16_t* dst = static_cast<uint16_t*>(job.out) + r * job.ld + col;
      const uint32_t off = reinterpret_cast<uintptr_t>(src) % 16;
      const char* at = src - off;
      uint32_t w[4];
      if (at >= first && at + 32 <= end) {
        const uint4 lo = __ldg(reinterpret_cast<const uint4*>(at)), hi = __ldg(reinterpret_cast<const uint4*>(at) + 1);
        const uint32_t q[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
        const int word = off / 4;
        const uint32_t bits = 8 * (off % 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t a = 0, b = 0;
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (k == word) { a = q[i + k]; b = q[i + k + 1]; }
          w[i] = __funnelshift_r(a, b, bits);
        }
      } else {
        const uint16_t* h = reinterpret_cast<const uint16_t*>(src);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t a = col + 2 * i < job.cols ? h[2 * i] : 0, b = col + 2 * i + 1 < job.cols ? h[2 * i + 1] : 0;
          w[i] = a | (b << 16);
        }
      }
      // (the copy's rows are a multiple of 64 long; what lies past the columns there is never read as a term)
      *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

// dz and the column sums of a row block, bound by the bytes (dy, pre in; dz out: 8192 x 8192 bfloat16 102 us, 5.2 TB/s).
// A warp takes 32 * V columns of every eighth row of the block (V columns per lane: 16 bytes of 16-bit values, or of
// float32), two rows in flight; the eight warps' partial sums are added in order.  VEC: every row of dy, pre and dz begins
// on a 16-byte boundary.
template <typename T, bool VEC, bool PLANES>
__global__ void __launch_bounds__(256, 3) dense_dz(const T* dy, long long ld_dy, const float* pre, void* dz, long long ld_dz,
                                                   float* part, int rows_per_block, long long rows, long long cols,
                                                int act, float alpha, float beta) {
  constexpr bool FAST = sizeof(T) == 2;
  constexpr int V = VEC ? 16 / sizeof(T) : PLANES ? 4 : 2;
  griddep_wait();
  griddep_launch();
  constexpr int U = 2;
  __shared__ float sums[8][32 * V];
  const int tx = threadIdx.x % 32, ty = threadIdx.x / 32;
  const long long c = (static_cast<long long>(blockIdx.x) * 32 + tx) * V;
  const long long r0 = static_cast<long long>(blockIdx.y) * rows_per_block;
  const long long r1 = min(r0 + rows_per_block, rows);
  const int n = static_cast<int>(min(static_cast<long long>(V), cols - c));  // columns that exist
  const bool wide = VEC && n == V;
  float sum[V];
#pragma unroll
  for (int j = 0; j < V; ++j) sum[j] = 0.0f;
  for (long long r = r0 + ty; r < r1; r += 8 * U) {
    T raw[U][V];
    float t[U][V];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const long long row = r + 8 * u;
      if (row >= r1) continue;
      const T* src = dy + row * ld_dy + c;
      const float* arg = pre + row * cols + c;
      if (wide) {
        if constexpr (VEC) {
          *reinterpret_cast<uint4*>(raw[u]) = __ldcs(reinterpret_cast<const uint4*>(src));
          if (act != ACT_IDENTITY) {
#pragma unroll
            for (int q = 0; q < V / 4; ++q)
              *reinterpret_cast<float4*>(&t[u][4 * q]) = __ldcs(reinterpret_cast<const float4*>(arg) + q);
          }
        }
      } else {
#pragma unroll
        for (int j = 0; j < V; ++j)
          if (j < n) {
            raw[u][j] = src[j];
            if (act != ACT_IDENTITY) t[u][j] = arg[j];
          }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const long long row = r + 8 * u;
      if (row >= r1) continue;
      float v[V];
#pragma unroll
      for (int j = 0; j < V; ++j) v[j] = j < n ? to_f32(raw[u][j]) : 0.0f;
      if (act != ACT_IDENTITY) {
        float a[V], d[V];
#pragma unroll
        for (int j = 0; j < V; ++j) a[j] = j < n ? t[u][j] : 0.0f;
        dense_activate_grad<FAST, V>(a, d, act, alpha, beta);
#pragma unroll
        for (int j = 0; j < V; ++j) v[j] = j < n ? v[j] * d[j] : 0.0f;
      }
      if constexpr (PLANES) {
        if (dz && n > 0) put_planes(v, static_cast<__nv_bfloat16*>(dz) + row * ld_dz + c, rows * ld_dz);
      } else if (dz) {
        T out[V];
#pragma unroll
        for (int j = 0; j < V; ++j) out[j] = from_f32<T>(v[j]);
        T* dst = static_cast<T*>(dz) + row * ld_dz + c;
        if (wide) {
          if constexpr (VEC) *reinterpret_cast<uint4*>(dst) = *reinterpret_cast<const uint4*>(out);
        } else {
#pragma unroll
          for (int j = 0; j < V; ++j)
            if (j < n) dst[j] = out[j];
        }
      }
#pragma unroll
      for (int j = 0; j < V; ++j) sum[j] += v[j];
    }
  }
  if (!part) return;
#pragma unroll
  for (int j = 0; j < V; ++j) sums[ty][tx * V + j] = sum[j];
  __syncthreads();
  for (int i = threadIdx.x; i < 32 * V; i += 256) {
    float s = sums[0][i];
#pragma unroll
    for (int w = 1; w < 8; ++w) s += sums[w][i];
    const long long col = static_cast<long long>(blockIdx.x) * 32 * V + i;
    if (col < cols) part[static_cast<long long>(blockIdx.y) * cols + col] = s;
  }
}
template <typename T>
__global__ void __launch_bounds__(256) dense_colsum(const float* part, T* out, int blocks, long long cols) {
  griddep_wait();
  griddep_launch();
  const long long c = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
  if (c >= cols) return;
  float s = 0.0f;
#pragma unroll 8
  for (int b = 0; b < blocks; ++b) s += part[b * cols + c];  // (eight loads in flight, added in order)
  out[c] = from_f32<T>(s);
}

template <typename T, int BM, int BN, bool DUAL>
cudaError_t go(const DenseGemm& g, cudaStream_t s) {
  const int bnl = DUAL ? BN / 2 : BN;
  const dim3 grid(static_cast<unsigned>(((g.N + bnl - 1LL) / bnl) * ((g.M + BM - 1LL) / BM)), 1,
                  static_cast<unsigned>((DUAL ? 1 : g.batch) * g.split));
  return launch_overlapped(dense_ffma<T, BM, BN, DUAL>, grid, kThreads, 0, 1, s, g);
}
template <typename T>
cudaError_t by_tile(const DenseFfmaPlan& p, const DenseGemm& g, cudaStream_t s) {
  if (g.dual) return p.bm == 128 ? go<T, 128, 128, true>(g, s) : go<T, 64, 128, true>(g, s);
  return p.bm == 128 ? go<T, 128, 128, false>(g, s) : go<T, 64, 64, false>(g, s);
}

template <typename T>
cudaError_t dz_go(const void* dy, long long ld_dy, const float* pre, void* dz, long long ld_dz, bool planes, void* dbias,
                  float* part, int blocks, long long rows, long long cols, int act, float alpha, float beta, cudaStream_t s) {
  const int per = static_cast<int>((rows + blocks - 1) / blocks);
  auto on16 = [](const void* p, long long bytes) { return reinterpret_cast<uintptr_t>(p) % 16 == 0 && bytes % 16 == 0; };
  const bool vec = on16(dy, ld_dy * sizeof(T)) && on16(pre, cols * 4) && (planes || on16(dz, ld_dz * sizeof(T)));
  const long long strip = 32 * (vec ? 16 / static_cast<long long>(sizeof(T)) : planes ? 4 : 2);
  const dim3 grid(static_cast<unsigned>((cols + strip - 1) / strip), static_cast<unsigned>((rows + per - 1) / per));
  auto kern = vec ? dense_dz<T, true, false> : dense_dz<T, false, false>;
  if constexpr (sizeof(T) == 4) {
    if (planes) kern = vec ? dense_dz<T, true, true> : dense_dz<T, false, true>;
  }
  cudaError_t err = launch_overlapped(kern, grid, 256, 0, 1, s, static_cast<const T*>(dy), ld_dy, pre, dz, ld_dz,
                                      dbias ? part : nullptr, per, rows, cols, act, alpha, beta);
  if (err != cudaSuccess || !dbias) return err;
  return launch_overlapped(dense_colsum<T>, dim3(static_cast<unsigned>((cols + 255) / 256)), 256, 0, 1, s, part,
                           static_cast<T*>(dbias), static_cast<int>(grid.y), cols);
}

}  // namespace

DenseFfmaPlan dense_ffma_plan(const DenseGemm& g, int sm, bool ranges) {
  DenseFfmaPlan p;
  auto tiles = [&](int bm, int bnl) {
    return ((g.M + bm - 1LL) / bm) * ((g.N + bnl - 1LL) / bnl) * g.batch;
  };
  const int bnl_large = g.dual ? 64 : 128, bnl_small = 64;
  // large tiles where they fill the device twice over; else small ones
  if (tiles(128, bnl_large) >= 2LL * sm) { p.bm = 128; p.bn = bnl_large; }
  else { p.bm = 64; p.bn = bnl_small; }
  const long long t = tiles(p.bm, p.bn), k = static_cast<long long>(g.segs) * g.K;
  // two blocks per SM; k in ranges of at least 128 terms where the tiles are fewer
  long long split = 1;
  if (ranges && t < 2LL * sm && k >= 256) split = std::min<long long>({(2LL * sm) / t, k / 128, 16});
  if (split < 1) split = 1;
  p.k_per_split = ((k + split - 1) / split + kBK - 1) / kBK * kBK;
  p.split = static_cast<int>((k + p.k_per_split - 1) / p.k_per_split);
  if (p.split <= 1) { p.split = 1; p.k_per_split = k; }
  return p;
}

cudaError_t launch_dense_ffma(const DenseFfmaPlan& p, const DenseGemm& g, int dtype, cudaStream_t s) {
  switch (dtype) {
    case CONV_F32: return by_tile<float>(p, g, s);
    case CONV_F16: return by_tile<__half>(p, g, s);
    default: return by_tile<__nv_bfloat16>(p, g, s);
  }
}

cudaError_t launch_dense_reduce(const DenseGemm& g, int dtype, cudaStream_t s) {
  const long long quads = (static_cast<long long>(g.N) + 3) / 4 * g.M;
  const dim3 grid(static_cast<unsigned>((quads + 255) / 256), static_cast<unsigned>(g.dual ? 1 : g.batch));
  switch (dtype) {
    case CONV_F32: return launch_overlapped(dense_reduce<float>, grid, 256, 0, 1, s, g);
    case CONV_F16: return launch_overlapped(dense_reduce<__half>, grid, 256, 0, 1, s, g);
    default: return launch_overlapped(dense_reduce<__nv_bfloat16>, grid, 256, 0, 1, s, g);
  }
}

cudaError_t launch_dense_copies(const CopyJob* jobs, int count, bool planes, cudaStream_t s) {
  if (count == 0) return cudaSuccess;
  CopyJobs c = {};
  c.count = count;
  for (int i = 0; i < count; ++i) {
    c.job[i] = jobs[i];
    c.first[i + 1] = c.first[i] + jobs[i].rows * ((jobs[i].cols + 255) / 256);
  }
  const unsigned blocks = static_cast<unsigned>(std::min<long long>((c.first[count] + 7) / 8, 1 << 14));
  return launch_overlapped(planes ? dense_copies<true> : dense_copies<false>, dim3(blocks), 256, 0, 1, s, c);
}

int dense_col_blocks(long long rows, long long cols, int sm) {
  // row blocks of at least kColRowsMin rows, about 8 blocks per SM in all
  const long long strips = (cols + 255) / 256;
  const long long want = std::max<long long>(1, 8LL * sm / strips);
  return static_cast<int>(std::max<long long>(1, std::min<long long>({want, (rows + kColRowsMin - 1) / kColRowsMin, 65535})));
}

cudaError_t launch_dense_dz(const void* dy, long long ld_dy, const float* pre, void* dz, long long ld_dz, bool planes,
                            void* dbias, float* part, int blocks, long long rows, long long cols, int act, float alpha,
                            float beta, int dtype, cudaStream_t s) {
  auto go = dtype == CONV_F32 ? dz_go<float> : dtype == CONV_F16 ? dz_go<__half> : dz_go<__nv_bfloat16>;
  return go(dy, ld_dy, pre, dz, ld_dz, planes, dbias, part, blocks, rows, cols, act, alpha, beta, s);
}

}  // namespace conv
