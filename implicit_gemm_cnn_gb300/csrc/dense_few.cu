// dense_few.cu -- the dense products for few rows (at most 16; one row is one
// generated token), bound by reading the weights once.
//
// A block takes 16 output features (of both projections in the gated product),
// its eight warps every eighth piece of k.  The weights go from memory straight
// into registers: nothing is reused, so shared memory would only add a step.
// 16-bit types multiply by mma.sync m16n8k16 with the weights as the 16-row
// operand and the rows of x as the 8 columns; a lane loads 16 consecutive bytes
// of a weight row and of an x row, and the eight values become the k's of two
// MMAs (both operands in the same order, so which k is which does not matter).
// The tensor cores' rate is beside the point: one MMA per kilobyte.  float32
// multiplies on the CUDA cores.  The warps' sums meet in shared memory and are
// added in order.
//
// Measured, back to back in a graph (the tcgen05 kernel, whose 128-row tiles
// need barriers and k ranges through memory, in brackets): one row of 2048 ->
// 8192 7.8 us (10.1), of 4096 -> 4096 7.5 (11.9), of 1024 -> 1024 2.4 (6.2); one
// row of 4096 -> 12288 18.4, 5.5 TB/s.  From 9 rows on the two come together,
// because every block reads all of x: few_rows in dense_api.cu has the rule.
// One row of a 4096 x 12288 gated block, two launches, the second's first loads
// under the first's end: 50 us, 6.0 TB/s.
#include <algorithm>

#include "dense_internal.h"

namespace conv {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kOuts = 16;   // output features of a block

// 16 bytes read once.
__device__ __forceinline__ uint4 load_once(const void* p) {
  uint4 r;
  asm volatile("ld.global.nc.L1::no_allocate.L2::256B.v4.u32 {%0, %1, %2, %3}, [%4];\n"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p));
  return r;
}
// `n` of 8 (n >= 8: all) 16-bit values at p.  VEC: p is on a 16-byte boundary and n is 0 or 8 at least.
template <bool VEC, bool ONCE>
__device__ __forceinline__ uint4 load8(const uint16_t* p, long long n) {
  if constexpr (VEC) {
    if (n <= 0) return make_uint4(0, 0, 0, 0);
    return ONCE ? load_once(p) : *reinterpret_cast<const uint4*>(p);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t lo = 2 * i < n ? p[2 * i] : 0, hi = 2 * i + 1 < n ? p[2 * i + 1] : 0;
      w[i] = lo | (hi << 16);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
}

template <typename T>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  if constexpr (std::is_same<T, __half>::value)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};\n"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};\n"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The sums of a block's outputs: red[product][warp][output][row] in shared memory.  The epilogue: one thread per
// (output, row).
template <typename T, int ROWS, bool DUAL>
__device__ __forceinline__ void finish(const DenseGemm& g, const float* red, int n0) {
  for (int i = threadIdx.x; i < kOuts * ROWS; i += kThreads) {
    const int o = i % kOuts, r = i / kOuts;
    if (r >= g.M || n0 + o >= g.N) continue;
    float v[1] = {0.0f}, u[1] = {0.0f};
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      v[0] += red[(w * kOuts + o) * ROWS + r];
      if (DUAL) u[0] += red[((kWarps + w) * kOuts + o) * ROWS + r];
    }
    const int col[1] = {n0 + o};
    const bool ok[1] = {true};
    dense_epilogue<T, 1>(g.epi, 0, r, col, ok, v, u);
  }
}

// NB: 8-row groups of x (1 or 2).  A piece is 32 * CH terms.  Blocks walk over the groups of outputs, the next group's
// first weights on their way while one group's sums are joined.
template <typename T, int NB, bool DUAL, bool VEC>
__global__ void __launch_bounds__(kThreads, 2) few_mma(const DenseGemm g, const int early) {
  constexpr int P = DUAL ? 2 : 1;
  constexpr int CH = DUAL ? 2 : 4;
  __shared__ float red[2][P * kWarps * kOuts * NB * 8];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, gq = lane / 4, t = lane % 4;
  const long long K = g.K;
  // this lane's two weight rows (of each product) and its x rows; rows past the end read the last one and are not stored
  const uint16_t* w[P][2];
  auto rows_of = [&](int n0) {
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        w[p][h] = static_cast<const uint16_t*>(g.b[p]) + static_cast<long long>(min(n0 + gq + 8 * h, g.N - 1)) * g.ldb + t * 8;
  };
  const uint16_t* x[NB];
  bool has[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    has[b] = gq + 8 * b < g.M;
    x[b] = static_cast<const uint16_t*>(g.a[0]) + static_cast<long long>(has[b] ? gq + 8 * b : 0) * g.lda + t * 8;
  }
  uint4 cur[P][2][CH], next[P][2][CH];
  auto load_w = [&](uint4 (&q)[P][2][CH], long long k) {
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int p = 0; p < P; ++p)
#pragma unroll
        for (int h = 0; h < 2; ++h) q[p][h][c] = load8<VEC, true>(w[p][h] + k + 32 * c, K - (k + 32 * c + t * 8));
  };
  const long long piece = 32 * CH, step = piece * kWarps, k0 = warp * piece;
  int n0 = blockIdx.x * kOuts, turn = 0;
  rows_of(n0);
  // `early`: the kernel before is the same call's, whose output x is and the weights are not
  if (!early) griddep_wait();
  if (k0 < K) load_w(cur, k0);
  griddep_wait();
  griddep_launch();
  while (n0 < g.N) {
    float acc[P][NB][4];
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[p][b][i] = 0.0f;
    const int n1 = n0 + static_cast<int>(gridDim.x) * kOuts;
    for (long long k = k0; k < K; k += step) {
      if (k + step < K) load_w(next, k + step);
      else if (n1 < g.N) {
        rows_of(n1);
        load_w(next, k0);
      }
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const long long left = K - (k + 32 * c + t * 8);
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const uint4 xv = load8<VEC, false>(x[b] + k + 32 * c, has[b] ? left : 0);
#pragma unroll
          for (int p = 0; p < P; ++p) {
            mma16816<T>(acc[p][b], cur[p][0][c].x, cur[p][1][c].x, cur[p][0][c].y, cur[p][1][c].y, xv.x, xv.y);
            mma16816<T>(acc[p][b], cur[p][0][c].z, cur[p][1][c].z, cur[p][0][c].w, cur[p][1][c].w, xv.z, xv.w);
          }
        }
      }
#pragma unroll
      for (int p = 0; p < P; ++p)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int c = 0; c < CH; ++c) cur[p][h][c] = next[p][h][c];
    }
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          red[turn][((p * kWarps + warp) * kOuts + gq + 8 * (i / 2)) * (NB * 8) + b * 8 + 2 * t + i % 2] = acc[p][b][i];
    __syncthreads();  // (the other buffer's sums were read before this)
    finish<T, NB * 8, DUAL>(g, red[turn], n0);
    turn ^= 1;
    n0 = n1;
  }
}

// float32: a warp multiplies pieces of 128 terms (four per lane) of the block's outputs with every row.  ROWS: rows
// compiled for (at least g.M).  Outputs are taken OG at a time, so that their sums stay in registers.
template <int ROWS, bool DUAL, bool VEC>
__global__ void __launch_bounds__(kThreads) few_f32(const DenseGemm g) {
  constexpr int P = DUAL ? 2 : 1;
  constexpr int OG = (ROWS > 8 ? 4 : 8) / P;
  __shared__ float red[P * kWarps * kOuts * ROWS];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int n0 = blockIdx.x * kOuts;
  griddep_wait();
  griddep_launch();
  auto load4 = [&](const float* p, long long k, float (&v)[4]) {
    if (VEC) {
      const float4 f = k < g.K ? __ldg(reinterpret_cast<const float4*>(p + k)) : make_float4(0, 0, 0, 0);
      v[0] = f.x; v[1] = f.y; v[2] = f.z; v[3] = f.w;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = k + i < g.K ? p[k + i] : 0.0f;
    }
  };
  for (int o0 = 0; o0 < kOuts; o0 += OG) {
    float acc[P][OG][ROWS];
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
      for (int o = 0; o < OG; ++o)
#pragma unroll
        for (int r = 0; r < ROWS; ++r) acc[p][o][r] = 0.0f;
    for (long long k = warp * 128 + lane * 4; k < (g.K + 127LL) / 128 * 128; k += kWarps * 128) {
      float wv[P][OG][4];
#pragma unroll
      for (int p = 0; p < P; ++p)
#pragma unroll
        for (int o = 0; o < OG; ++o)
          load4(static_cast<const float*>(g.b[p]) + static_cast<long long>(min(n0 + o0 + o, g.N - 1)) * g.ldb, k, wv[p][o]);
#pragma unroll
      for (int r = 0; r < ROWS; ++r) {
        float xv[4];
        load4(static_cast<const float*>(g.a[0]) + static_cast<long long>(min(r, g.M - 1)) * g.lda, k, xv);
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
          for (int o = 0; o < OG; ++o)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[p][o][r] = fmaf(wv[p][o][i], xv[i], acc[p][o][r]);
      }
    }
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
      for (int o = 0; o < OG; ++o)
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
          float v = acc[p][o][r];
#pragma unroll
          for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
          if (lane == 0) red[((p * kWarps + warp) * kOuts + o0 + o) * ROWS + r] = v;
        }
  }
  __syncthreads();
  finish<float, ROWS, DUAL>(g, red, n0);
}

int groups_of(const DenseGemm& g) { return static_cast<int>((static_cast<long long>(g.N) + kOuts - 1) / kOuts); }
template <typename T, bool DUAL>
cudaError_t go16(const DenseGemm& g, bool vec, bool follows, int sm, cudaStream_t s) {
  // two blocks per SM at most, each with as many groups of outputs as any other
  const int groups = groups_of(g), rounds = (groups + 2 * sm - 1) / (2 * sm), blocks = (groups + rounds - 1) / rounds;
  auto kern = g.M <= 8 ? (vec ? few_mma<T, 1, DUAL, true> : few_mma<T, 1, DUAL, false>)
                       : (vec ? few_mma<T, 2, DUAL, true> : few_mma<T, 2, DUAL, false>);
  return launch_overlapped(kern, dim3(static_cast<unsigned>(blocks)), kThreads, 0, 1, s, g, follows ? 1 : 0);
}
template <int ROWS, bool DUAL>
cudaError_t go32(const DenseGemm& g, bool vec, cudaStream_t s) {
  return launch_overlapped(vec ? few_f32<ROWS, DUAL, true> : few_f32<ROWS, DUAL, false>,
                           dim3(static_cast<unsigned>(groups_of(g))), kThreads, 0, 1, s, g);
}

}  // namespace

cudaError_t launch_dense_few(const DenseGemm& g, int dtype, bool follows, int sm, cudaStream_t s) {
  const int es = dtype == CONV_F32 ? 4 : 2, per = 16 / es;
  auto on16 = [&](const void* p, long long ld) { return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % per == 0; };
  // whole 16-byte pieces: rows on 16-byte boundaries, k a multiple of a piece
  const bool vec = g.K % per == 0 && on16(g.a[0], g.M > 1 ? g.lda : 0) && on16(g.b[0], g.ldb) &&
                   (!g.dual || on16(g.b[1], g.ldb));
  if (dtype == CONV_F16) return g.dual ? go16<__half, true>(g, vec, follows, sm, s) : go16<__half, false>(g, vec, follows, sm, s);
  if (dtype == CONV_BF16)
    return g.dual ? go16<__nv_bfloat16, true>(g, vec, follows, sm, s) : go16<__nv_bfloat16, false>(g, vec, follows, sm, s);
  if (g.M <= 1) return g.dual ? go32<1, true>(g, vec, s) : go32<1, false>(g, vec, s);
  if (g.M <= 4) return g.dual ? go32<4, true>(g, vec, s) : go32<4, false>(g, vec, s);
  if (g.M <= 8) return g.dual ? go32<8, true>(g, vec, s) : go32<8, false>(g, vec, s);
  return g.dual ? go32<16, true>(g, vec, s) : go32<16, false>(g, vec, s);
}

}  // namespace conv
