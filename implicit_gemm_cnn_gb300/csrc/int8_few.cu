// int8_few.cu -- the 8-bit product for few rows (one row is one generated
// token): the weights, a byte each, go straight into registers, once for each
// tile of at most 32 rows of x (128 rows: four times, mostly out of L2).
//
// sm_103's 8-bit tensor-core kinds are gone (tcgen05 has no kind::i8 here), its
// CUDA cores' dp4a is slow, but 16-bit floats hold every 8-bit integer: a byte u
// = b + 128 put below 0x64 is the half 1024 + u, and one subtraction of 1152
// leaves b.  The products, of 2^14 at most each, are summed by mma.sync m16n8k16
// in float32, which is exact up to 2^24, so 1024 terms; each piece's sums (at
// most 256 terms) then move into int32.
//
// A block takes 16 output features at a time, its eight warps every eighth piece
// of k.  The weights are the 16-row operand, the rows of x the 8 columns (a tile
// has NB = 1, 2 or 4 groups of 8 rows); a lane loads 16 consecutive bytes of a
// weight row and of an x row, which are the k's of four MMAs (both operands in the
// same order, so which k is which does not matter).  The warps' sums meet in shared
// memory.
//
// A piece is CH chunks of 64 terms: four of them (256 terms of 16 outputs, 4 KB a
// warp in flight and as much at work) for tiles of at most 16 rows, two for tiles of
// 32, whose sums take the registers; half as many where the weights' rows are no whole
// 16-byte pieces, since each chunk is then two loads (put together on arrival).
//
// What bounds it: the weights' loads, and the barriers of each 16 outputs.  One
// row of 4096 -> 12288 14.4 us (50 MB: 3.5 TB/s), 16 rows 17.4, 32 rows 25.6;
// 2048 -> 8192 6.8, 8.1, 10.9; 4003 -> 12288, x quantised by the call, 25, 31, 42.
// (linear's kernel for few rows reads the same layer in 16 bits at 5.6 TB/s, so one
// row in 8 bits saves a sixth of its 18.0 us, not half.)
// Pieces of 256 terms and two blocks an SM are the quickest for one row: pieces of
// 64 terms took 18.7 us, of 512 17.9; 32 or 64 outputs a block 16.7 and 17.7.
#include <algorithm>

#include "int8.cuh"

namespace conv {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kOuts = 16;  // output features of a block at a time
constexpr int kPerSm = 2;  // blocks

__device__ __forceinline__ uint4 load_once(const void* p) {
  uint4 r;
  asm volatile("ld.global.nc.L1::no_allocate.L2::256B.v4.u32 {%0, %1, %2, %3}, [%4];\n"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p));
  return r;
}
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};\n"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The 16 bytes at a 16-byte boundary, those of [first, end) of them (others are zero).
__device__ __noinline__ uint4 edge_piece(const int8_t* at, const int8_t* first, const int8_t* end) {
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 16; ++i)
    if (at + i >= first && at + i < end) w[i / 4] |= static_cast<uint32_t>(static_cast<uint8_t>(at[i])) << (8 * (i % 4));
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// A piece at any address: the two at 16-byte boundaries that it lies in, under way until they are put together.  (Put together
// where they are loaded, each waited for the one before: one row of 4003 -> 12288 took 37 us, now 24.)
struct Halves {
  uint4 lo, hi;
  __device__ __forceinline__ void load(const int8_t* p, bool ok, const int8_t* first, const int8_t* end) {
    const uint32_t off = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p)) % 16;
    const int8_t* at = p - off;
    const bool begins = at >= first, more = ok && off != 0;
    lo = load_raw<16>(at, 0, ok && begins && at + 16 <= end);
    hi = load_raw<16>(at + 16, 0, more && at + 32 <= end);
    if (ok && !(begins && at + 16 <= end)) lo = edge_piece(at, first, end);
    if (more && at + 32 > end) hi = edge_piece(at + 16, first, end);
  }
  __device__ __forceinline__ uint4 value(uint32_t off) const {
    const uint32_t q[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    uint32_t r[6], s[5];
#pragma unroll
    for (int i = 0; i < 6; ++i) r[i] = off & 8 ? q[i + 2] : q[i];
#pragma unroll
    for (int i = 0; i < 5; ++i) s[i] = off & 4 ? r[i + 1] : r[i];
    const uint32_t by = 8 * (off % 4);
    return make_uint4(__funnelshift_r(s[0], s[1], by), __funnelshift_r(s[1], s[2], by), __funnelshift_r(s[2], s[3], by),
                      __funnelshift_r(s[3], s[4], by));
  }
};
struct Whole {
  uint4 v;
  __device__ __forceinline__ void load(const int8_t* p, bool ok, const int8_t*, const int8_t*) {
    v = make_uint4(0, 0, 0, 0);
    if (ok) v = load_once(p);
  }
  __device__ __forceinline__ uint4 value(uint32_t) const { return v; }
};

// NB: groups of 8 rows; CH: 64-term chunks of a piece.  PIECES: the rows of w are whole 16-byte pieces.
template <typename T, int NB, int CH, bool PIECES>
__global__ void __launch_bounds__(kThreads, kPerSm) int8_few(const Int8Args g, const int early) {
  using Piece = typename std::conditional<PIECES, Whole, Halves>::type;
  constexpr int ROWS = 8 * NB;
  __shared__ int red[kWarps][kOuts][ROWS + 1];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, gq = lane / 4, t = lane % 4;
  const int m0 = blockIdx.y * ROWS;
  const long long K = g.K;
  const int8_t* const w_end = g.w + (g.N - 1) * g.ldw + K;
  // this lane's weight rows and x rows; rows past the end read the last one and are not stored
  const int8_t* w[2];
  uint32_t off[2], next_off[2];  // of a row's pieces from 16-byte boundaries
  auto rows_of = [&](int n0) {
#pragma unroll
    for (int h = 0; h < 2; ++h) w[h] = g.w + static_cast<long long>(min(n0 + gq + 8 * h, g.N - 1)) * g.ldw + t * 16;
#pragma unroll
    for (int h = 0; h < 2; ++h) next_off[h] = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(w[h])) % 16;
  };
  const int8_t* x[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) x[b] = g.x + static_cast<long long>(min(m0 + gq + 8 * b, g.M - 1)) * g.ldx + t * 16;
  Piece cur[2][CH], next[2][CH];
  auto load_w = [&](Piece (&q)[2][CH], long long k) {
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int h = 0; h < 2; ++h) q[h][c].load(w[h] + k + 64 * c, k + 64 * c + t * 16 < K, g.w, w_end);
  };
  const long long piece = 64 * CH, step = piece * kWarps, k0 = warp * piece;
  int n0 = blockIdx.x * kOuts;
  rows_of(n0);
  off[0] = next_off[0];
  off[1] = next_off[1];
  // `early`: the kernel before is the same call's, and writes no weights
  if (!early) griddep_wait();
  if (k0 < K) load_w(cur, k0);
  griddep_wait();
  griddep_launch();
  while (n0 < g.N) {
    int sum[NB][4];
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int i = 0; i < 4; ++i) sum[b][i] = 0;
    const int n1 = n0 + static_cast<int>(gridDim.x) * kOuts;
    for (long long k = k0; k < K; k += step) {
      if (k + step < K) load_w(next, k + step);
      else if (n1 < g.N) {
        rows_of(n1);
        load_w(next, k0);
      }
      float acc[NB][4];
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[b][i] = 0.0f;
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const long long left = K - (k + 64 * c + t * 16);
        uint32_t a[2][8];
#pragma unroll
        for (int h = 0; h < 2; ++h) widen16(cur[h][c].value(off[h]), a[h]);
        uint4 xb[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const int8_t* const p = x[b] + k + 64 * c;
          if constexpr (PIECES) {
            xb[b] = make_uint4(0, 0, 0, 0);
            if (left > 0) xb[b] = *reinterpret_cast<const uint4*>(p);
          } else {  // (as a branch each waited for its value, which is cut off right away: 12 rows of 2003 -> 5001 14.4 us, now 13.0)
            xb[b] = load_raw<16>(p, 0, left > 0);
          }
        }
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          if constexpr (!PIECES) xb[b] = first_bytes(xb[b], left);  // (of the weights, what follows the row is there)
          uint32_t xv[8];
          widen16(xb[b], xv);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            mma(acc[b], a[0][2 * j], a[1][2 * j], a[0][2 * j + 1], a[1][2 * j + 1], xv[2 * j], xv[2 * j + 1]);
        }
      }
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i) sum[b][i] += __float2int_rn(acc[b][i]);  // (few of them)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int c = 0; c < CH; ++c) cur[h][c] = next[h][c];
      off[0] = next_off[0];
      off[1] = next_off[1];
    }
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int i = 0; i < 4; ++i) red[warp][gq + 8 * (i / 2)][8 * b + 2 * t + i % 2] = sum[b][i];
    __syncthreads();
    for (int i = threadIdx.x; i < kOuts * ROWS; i += kThreads) {
      const int r = i / kOuts, m = m0 + r, n = n0 + i % kOuts;
      if (m >= g.M || n >= g.N) continue;
      int total = 0;
#pragma unroll
      for (int k = 0; k < kWarps; ++k) total += red[k][i % kOuts][r];
      float v[1] = {static_cast<float>(total) * g.x_scale[m] * g.w_scale[n]}, u[1];
      const int col[1] = {n};
      const bool ok[1] = {true};
      dense_epilogue<T, 1>(g.epi, 0, m, col, ok, v, u);
    }
    __syncthreads();
    n0 = n1;
  }
}

template <typename T, int NB, int CH>
cudaError_t go(const Int8Args& g, bool pieces, bool follows, int sm, cudaStream_t s) {
  // as many blocks as run at once at most, each with as many groups of outputs as any other
  const int groups = (g.N + kOuts - 1) / kOuts, rounds = (groups + kPerSm * sm - 1) / (kPerSm * sm);
  const dim3 grid(static_cast<unsigned>((groups + rounds - 1) / rounds), static_cast<unsigned>((g.M + 8 * NB - 1) / (8 * NB)));
  // (weights in two halves: half the chunks)
  return launch_overlapped(pieces ? int8_few<T, NB, CH, true> : int8_few<T, NB, CH / 2, false>, grid, kThreads, 0, 1, s, g,
                           follows ? 1 : 0);
}
// A tile has 8, 16 or 32 rows, and a lane its share of their sums: with 32 of them registers leave room for half the piece.
template <typename T>
cudaError_t by_rows(const Int8Args& g, bool pieces, bool follows, int sm, cudaStream_t s) {
  if (g.M <= 8) return go<T, 1, 4>(g, pieces, follows, sm, s);
  if (g.M <= 16) return go<T, 2, 4>(g, pieces, follows, sm, s);
  return go<T, 4, 2>(g, pieces, follows, sm, s);
}

}  // namespace

cudaError_t launch_int8_few(const Int8Args& g, int dtype, bool follows, int sm, cudaStream_t s) {
  const bool pieces = g.K % 16 == 0 && reinterpret_cast<uintptr_t>(g.w) % 16 == 0 && (g.N == 1 || g.ldw % 16 == 0);
  if (dtype == CONV_F32) return by_rows<float>(g, pieces, follows, sm, s);
  return dtype == CONV_F16 ? by_rows<__half>(g, pieces, follows, sm, s) : by_rows<__nv_bfloat16>(g, pieces, follows, sm, s);
}

}  // namespace conv
