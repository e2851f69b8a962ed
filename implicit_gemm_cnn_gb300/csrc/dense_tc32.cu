// dense_tc32.cu -- the dense products of float32 operands on the tensor cores.
//
// A float32 value is the exact sum of three bfloat16 values, each the rounding
// of what the ones before leave (8 significand bits each, 24 in all).  A pass
// over the operands writes the three as planes, the second times 2^7 and the
// third times 2^16: bfloat16 has float32's exponents, so the remainders of small
// values would have no room.  (2^8 for the second would let sums of parts
// overflow that the whole sum does not.)  A product then is
//   a b = a0 b0 + 2^-7 (a0 b1 + a1 b0 + 2^-7 a1 b1) + 2^-16 (a0 b2 + a2 b0)
// without a1 b2, a2 b1 and a2 b2, which are below 2^-24 of |a b| (of a factor
// below 2^-124, 1.5 * 2^-149 of the other): six bfloat16 products, still three
// times the CUDA cores' float32 rate and more.  The accumulator is divided by
// the powers of two as the MMAs go on (scale-input-d), at no cost in time.
//
// The tensor cores cut their float32 accumulator instead of rounding it (the
// sum of 1024 positive terms came out 2.2e-6 low, 64 terms 8e-8), so no
// accumulator lives long: each 64 terms start a new one, and the epilogue warps
// add the finished 64-term sums up in registers, rounding to nearest.  That work
// overlaps the next stage's MMAs (two pairs of accumulators).  The five small
// products have an accumulator of their own: an infinity's remainders are zero,
// and where a0 b0 is infinite or NaN it alone is the result.  (One accumulator
// for all six took 2% less time, and gave NaN for infinity times anything; its
// sums of positive terms were 4e-8 low on the average, these are not.)
//
// Measured: 4096 x 4096 x 4096 551 us, 249 TFLOP/s (4.1 times the CUDA cores'
// rate; the six products alone are 1.5 PFLOP/s of bfloat16); 1024 positive terms
// at most 1.8e-7 off.  A stage's MMAs take 1536 clocks, its copies 96 KB.  Small
// products wait for the launches and the epilogue (1001 x 515 -> 1030 with gelu:
// 26 us, of which the MMAs 8).
//
// Otherwise as dense_tc.cuh, with tiles of 128 x 64 or 128 x 128 on one SM: a
// stage is three planes of both operands, 96 KB, for 24 MMAs.
#include <string.h>

#include <algorithm>

#include "dense_tc.cuh"

namespace conv {
namespace {
using namespace dtc;

constexpr int kEpiWarps = 4;
constexpr int kThreads32 = 64 + 32 * kEpiWarps;
constexpr int kPlaneBytes = 128 * 128;          // one plane of a 128-row operand tile, 64 terms
constexpr int kStage32 = 6 * kPlaneBytes;
constexpr int kStages32 = 2;
constexpr int kBuf32 = 4096;                    // a staging tile of 32 rows of 32 float32
constexpr int kLarge32 = 128;                   // columns from an accumulator's small products to its large one
constexpr int kAcc32 = 2 * kLarge32;
constexpr int kStaging32 = kEpiWarps * 2 * kBuf32;
constexpr int kSmem32 = kStages32 * kStage32 + kStaging32 + 2032;

template <int MODE, bool A_MN, bool B_MN>
__global__ void __launch_bounds__(kThreads32, 1)
    dense_tc32(const __grid_constant__ DenseTcArgs p, const __grid_constant__ DenseTcMaps maps) {
  const int nt = p.nt, out_cols = MODE == EPI_GATED ? nt / 2 : nt;
  extern __shared__ uint8_t smem_raw[];
  __shared__ volatile int abort_flag;
  __shared__ uint32_t tmem_slot;
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t staging = base + kStages32 * kStage32;
  const uint32_t bars = staging + kStaging32;
  auto full = [&](int s) { return bars + 8u * s; };
  auto empty = [&](int s) { return bars + 8u * (kStages32 + s); };
  auto acc_full = [&](int b) { return bars + 8u * (2 * kStages32 + b); };
  auto acc_empty = [&](int b) { return bars + 8u * (2 * kStages32 + 2 + b); };
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0), lane = threadIdx.x % 32;
  if (warp == 0 && lane == 0) {
    for (int s = 0; s < kStages32; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(acc_full(b), 1);
      mbar_init(acc_empty(b), kEpiWarps);
    }
    abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    fence_proxy_async();
  }
  if (warp == 1) alloc_tmem<1>(smem_u32(&tmem_slot), 2 * kAcc32);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_slot, 0);
  griddep_wait();
  griddep_launch();
  const int first = blockIdx.x, step = gridDim.x;

  if (warp == 0) {
    if (elect_one()) {
      // k-major: a box of 128 (nt) rows x 64 terms x 3 planes; mn-major: of 64 columns x 64 terms x 3 planes, one after
      // another
      const int b_boxes = nt / 64;
      const uint32_t stage_bytes = 3 * (kPlaneBytes + nt * 128);
      int s = 0;
      uint32_t parity = 1;
      bool ok = true;
      for (int u = first; u < p.units && ok; u += step) {
        const Tile t = tile_of(p, u);
        const int kb0 = t.kb0, kb1 = kb0 + t.kbs;
        const int m0 = t.m * 128, n0 = t.n * out_cols;
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!wait_phase(p.err, empty(s), parity, &abort_flag, 1u)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(full(s), stage_bytes);
          const int seg = kb >= p.kb_seg ? 1 : 0, k0 = (kb - seg * p.kb_seg) * kBK;
          const int op = p.segs > 1 ? seg : t.batch;
          const uint32_t a = base + s * kStage32, b = a + 3 * kPlaneBytes;
          if constexpr (A_MN) {
            load_3d<1>(a, &maps.a[op], m0, k0, 0, full(s));
            load_3d<1>(a + 3 * 8192, &maps.a[op], m0 + 64, k0, 0, full(s));
          } else {
            load_3d<1>(a, &maps.a[op], k0, m0, 0, full(s));
          }
          if constexpr (MODE == EPI_GATED) {
            load_3d<1>(b, &maps.b[0], k0, n0, 0, full(s));
            load_3d<1>(b + 3 * out_cols * 128, &maps.b[1], k0, n0, 0, full(s));
          } else if constexpr (B_MN) {
            for (int i = 0; i < b_boxes; ++i) load_3d<1>(b + i * 3 * 8192, &maps.b[op], n0 + 64 * i, k0, 0, full(s));
          } else {
            load_3d<1>(b, &maps.b[op], k0, n0, 0, full(s));
          }
          if (++s == kStages32) { s = 0; parity ^= 1; }
        }
      }
      for (int left = kStages32; left > 0 && ok; --left) {
        ok = wait_phase(p.err, empty(s), parity, &abort_flag, 1u);
        if (++s == kStages32) { s = 0; parity ^= 1; }
      }
      if (!ok)  // copies in flight end within microseconds; the block does not return before
        for (int i = 0; i < 1000; ++i) __nanosleep(10000);
    }
  } else if (warp == 1) {
    if (elect_one()) {
      // The gated product's B is two boxes (gate, up), each of three planes: two MMAs of half the columns.
      constexpr int kHalves = MODE == EPI_GATED ? 2 : 1;
      const int cols = nt / kHalves;
      const uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(A_MN) << 15) |
                             (static_cast<uint32_t>(B_MN) << 16) | (static_cast<uint32_t>(cols >> 3) << 17) | (8u << 24);
      constexpr int kAStep = A_MN ? 2048 >> 4 : 32 >> 4, kBStep = B_MN ? 2048 >> 4 : 32 >> 4;
      // planes lie one after another within a box: mn-major 64-column blocks are three planes apart
      const uint64_t a0 = smem_desc(base, A_MN ? 3 * 8192 : 16, 1024, 2);
      const uint64_t b0 = smem_desc(base + 3 * kPlaneBytes, B_MN ? 3 * 8192 : 16, 1024, 2);
      const uint64_t a_plane = (A_MN ? 8192 : kPlaneBytes) >> 4;
      const uint64_t b_plane = (B_MN ? 8192 : cols * 128) >> 4;
      int s = 0, it = 0;
      uint32_t parity = 0;
      bool ok = true;
      for (int u = first; u < p.units && ok; u += step) {
        const int kbs = tile_of(p, u).kbs;
        for (int kb = 0; kb < kbs; ++kb, ++it) {
          const int buf = it & 1;
          if (!wait_phase(p.err, acc_empty(buf), ((it >> 1) & 1) ^ 1, &abort_flag, 2u) ||
              !wait_phase(p.err, full(s), parity, &abort_flag, 4u)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t off = static_cast<uint64_t>(s) * (kStage32 >> 4);
#pragma unroll
          for (int h = 0; h < kHalves; ++h) {
            const uint32_t d = tmem + buf * kAcc32 + h * cols;
            const uint64_t a = a0 + off, b = b0 + off + h * 3 * b_plane;
            // the small products, each order's scale taken off as the next one begins; beside them the large one
            mma_terms<-1, kAStep, kBStep>(d, a, b + 2 * b_plane, idesc);
            mma_terms<0, kAStep, kBStep>(d, a + 2 * a_plane, b, idesc);
            mma_terms<kPlaneScale2 - 2 * kPlaneScale1, kAStep, kBStep>(d, a + a_plane, b + b_plane, idesc);
            mma_terms<kPlaneScale1, kAStep, kBStep>(d, a, b + b_plane, idesc);
            mma_terms<0, kAStep, kBStep>(d, a + a_plane, b, idesc);
            mma_terms<-1, kAStep, kBStep>(d + kLarge32, a, b, idesc);
          }
          commit<1>(empty(s));
          commit<1>(acc_full(buf));
          if (++s == kStages32) { s = 0; parity ^= 1; }
        }
      }
      if (abort_flag)
        for (int i = 0; i < 1000; ++i) __nanosleep(10000);
    }
  } else {
    const int quarter = warp & 3;
    const uint32_t mine = staging + (warp - 2) * 2 * kBuf32;
    const DenseEpi& e = p.epi;
    int turn = 0, it = 0;
    // 32 float32 columns of this lane's row
    auto put = [&](const float (&v)[32], const CUtensorMap* map, float* out, long long ld, bool tma, int n, int m_warp) {
      if (tma) {
        if (lane == 0) bulk_wait_read<1>();
        __syncwarp();
        const uint32_t b = mine + (turn & 1) * kBuf32;
        ++turn;
#pragma unroll
        for (int q = 0; q < 8; ++q)
          sts_v4(b + lane * 128 + ((q ^ (lane & 7)) << 4),
                 make_uint4(__float_as_uint(v[4 * q]), __float_as_uint(v[4 * q + 1]), __float_as_uint(v[4 * q + 2]),
                            __float_as_uint(v[4 * q + 3])));
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) {
          store_2d(map, b, n, m_warp);
          bulk_commit();
        }
      } else {
        // rows of any alignment: through shared memory, so that a store instruction covers one row's consecutive columns
        if (lane == 0) bulk_wait_read<0>();
        __syncwarp();
        float* tile = static_cast<float*>(__cvta_shared_to_generic(mine));
#pragma unroll
        for (int i = 0; i < 32; ++i) tile[lane * 33 + i] = v[i];
        __syncwarp();
        out += static_cast<long long>(m_warp) * ld + n;
        const int rows = min(32, p.M - m_warp);
        if (n + lane < p.N)
          for (int r = 0; r < rows; ++r) out[r * ld + lane] = tile[r * 33 + lane];
        __syncwarp();
      }
    };
    auto activate = [&](float (&v)[32]) {
      if (e.act == ACT_IDENTITY) return;
      float t[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) t[i] = v[i];
      dense_activate_array(t, e.act, e.alpha, e.beta);
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = t[i];
    };
    // 32 float32 values of a row, `n` of which exist, at any alignment
    auto add_row = [&](float (&v)[32], const float* row, int n) {
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (i < n) v[i] = __fadd_rn(v[i], row[i]);
    };
    for (int u = first; u < p.units; u += step) {
      const Tile t = tile_of(p, u);
      const int kbs = t.kbs;
      const int m_warp = t.m * 128 + quarter * 32, m = m_warp + lane, n_tile = t.n * out_cols;
      float acc[4][32];
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int i = 0; i < 32; ++i) acc[c][i] = 0.0f;
      bool ok = true;
      for (int kb = 0; kb < kbs; ++kb, ++it) {
        const int buf = it & 1;
        if (!warp_wait(p.err, acc_full(buf), (it >> 1) & 1, &abort_flag, 8u)) {
          ok = false;
          break;
        }
        __syncwarp();
        tc_fence_after();
        const uint32_t at = tmem + buf * kAcc32 + (static_cast<uint32_t>(quarter * 32) << 16);
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (32 * c < nt) {
            float small[32], v[32];
            tmem_ld32(at + 32 * c, small);
            tmem_ld32(at + kLarge32 + 32 * c, v);
            tmem_arrived(small);
            tmem_arrived(v);
            // (an infinite or NaN large product is the sum: infinity times a remainder of zero would be NaN)
#pragma unroll
            for (int i = 0; i < 32; ++i)
              acc[c][i] += fabsf(v[i]) <= 3.402823466e38f ? fmaf(small[i], 1.0f / (1u << kPlaneScale1), v[i]) : v[i];
          }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(acc_empty(buf));
      }
      if (!ok) break;
      if (m_warp >= p.M) continue;
      if (t.slot >= 0) {  // a k range: its sums as they are
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (32 * c < nt) put(acc[c], &maps.part, nullptr, 0, true, 32 * c, t.slot * 128 + quarter * 32);
        continue;
      }
      // one copy of the code for all pieces: the next piece's sums move into acc[0]
#pragma unroll 1
      for (int c = 0; 32 * c < out_cols; ++c) {
        if (c > 0) {
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            acc[0][i] = acc[1][i];
            if (MODE != EPI_GATED) acc[1][i] = acc[2][i];
            acc[2][i] = acc[3][i];
          }
        }
        const int n = n_tile + 32 * c, left = p.N - n;
        if (left <= 0) break;
        const bool row_ok = m < p.M;
        if constexpr (MODE == EPI_GATED) {
          // gate columns are the tile's first half, up columns its second
          float up[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) up[i] = nt == 64 ? acc[1][i] : acc[2][i];
          if (e.pre) {
            put(acc[0], &maps.pre[0], e.pre, e.ldp, p.align_pre != 0, n, m_warp);
            put(up, &maps.pre[1], e.pre2, e.ldp, p.align_pre != 0, n, m_warp);
          }
          activate(acc[0]);
#pragma unroll
          for (int i = 0; i < 32; ++i) up[i] *= acc[0][i];
          put(up, &maps.y[0], static_cast<float*>(e.y), e.ldy, p.align_y != 0, n, m_warp);
        } else if constexpr (MODE == EPI_GATED_BWD) {
          float g[32], slope[32];
          const float* gp = e.pre + static_cast<long long>(m) * e.ldp + n;
          const float* up = e.pre2 + static_cast<long long>(m) * e.ldp + n;
#pragma unroll
          for (int i = 0; i < 32; ++i) g[i] = row_ok && i < left ? gp[i] : 0.0f;
          dense_activate_grad_array(g, slope, e.act, e.alpha, e.beta);
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            slope[i] *= acc[0][i] * (row_ok && i < left ? up[i] : 0.0f);
            g[i] *= acc[0][i];
          }
          put(slope, &maps.y[0], static_cast<float*>(e.y), e.ldy, p.align_y != 0, n, m_warp);
          put(g, &maps.y[1], static_cast<float*>(e.y2), e.ldy, p.align_y != 0, n, m_warp);
        } else {
          const float* res = e.residual && row_ok ? static_cast<const float*>(e.residual) + static_cast<long long>(m) * e.ldr + n
                                                  : nullptr;
          if (e.bias) add_row(acc[0], static_cast<const float*>(e.bias) + n, left);
          if (res && !e.residual_last) add_row(acc[0], res, left);
          if (e.pre) put(acc[0], &maps.pre[0], e.pre, e.ldp, p.align_pre != 0, n, m_warp);
          activate(acc[0]);
          if (res && e.residual_last) add_row(acc[0], res, left);
          put(acc[0], &maps.y[t.batch], static_cast<float*>(t.batch ? e.y2 : e.y), e.ldy, p.align_y != 0, n, m_warp);
        }
      }
    }
    if (lane == 0) bulk_wait_all();
    __syncwarp();
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    free_tmem<1>(tmem, 2 * kAcc32);
  }
}

template <int MODE, bool A_MN, bool B_MN>
cudaError_t go32(const DenseTcArgs& args, const DenseTcMaps& maps, int blocks, cudaStream_t s) {
  auto kern = dense_tc32<MODE, A_MN, B_MN>;
  cudaError_t err = opt_in_smem(reinterpret_cast<const void*>(kern), kSmem32);
  if (err != cudaSuccess) return err;
  return launch_overlapped(kern, dim3(static_cast<unsigned>(blocks)), kThreads32, kSmem32, 1, s, args, maps);
}
template <int MODE>
cudaError_t order32(int a_mn, int b_mn, const DenseTcArgs& args, const DenseTcMaps& maps, int blocks, cudaStream_t s) {
  if (a_mn) return b_mn ? go32<MODE, true, true>(args, maps, blocks, s) : cudaErrorInvalidValue;
  return b_mn ? go32<MODE, false, true>(args, maps, blocks, s) : go32<MODE, false, false>(args, maps, blocks, s);
}

}  // namespace

cudaError_t launch_dense_tc32(int mode, int a_mn, int b_mn, const DenseTcArgs& args, const DenseTcMaps& maps, int blocks,
                              cudaStream_t s) {
  switch (mode) {
    case EPI_GATED:
      return a_mn || b_mn ? cudaErrorInvalidValue : go32<EPI_GATED, false, false>(args, maps, blocks, s);
    case EPI_GATED_BWD:
      return a_mn || !b_mn ? cudaErrorInvalidValue : go32<EPI_GATED_BWD, false, true>(args, maps, blocks, s);
    default: return order32<EPI_LINEAR>(a_mn, b_mn, args, maps, blocks, s);
  }
}

}  // namespace conv
