// int8_tc.cu -- the 8-bit product of many rows, on the fifth-generation tensor
// cores.
//
// sm_103a has no kind::i8; its halves hold every 8-bit integer, so a pass over
// the operands writes them as halves (quantize.cu) and the product runs at the
// 16-bit rate: tiles, rings, and roles as in dense_tc.cuh.  What is different is
// the sum.  A float32 accumulator is exact while sums stay within 2^24, which
// 1024 products of 2^14 cannot pass: every 16 stages (of 64 terms) start a new
// accumulator, and the epilogue warps add the finished ones up as int32 in
// registers, under the next 1024 terms' MMAs.  (A stage of a pair's 256 x 256
// tile takes 512 clocks, so 16 of them 8192; a warp reads its 128 columns and
// adds them in some 1000.)
//
// What bounds it is the tensor pipe: 77% of its rate (4864 x 4096 -> 4096 97 us,
// 1.68 PFLOP/s), where the one accumulator of a 16-bit product leaves 84.  With the
// passes before it 2048 x 4096 -> 4096 takes 58 us, 8192 x 4096 -> 12288 492 at full
// clock and 540 to 585 in longer runs, at the power limit.  (linear, whose operands are
// halves already: 40 and 414 beside 60 and 540, one after the other on one machine.)
// A pair's variants spill: 300 bytes for 16-bit results, 180 for float32.
#include <string.h>

#include <algorithm>

#include "dense_tc.cuh"
#include "int8.cuh"

namespace conv {
namespace {
using namespace dtc;

constexpr int kExact = 16;       // stages of an accumulator
constexpr int kFactors = 1024;   // a warp's scales and bias of 128 columns

template <int CG, int NT>
struct Cfg8 {
  static constexpr int kEpiWarps = NT >= 256 ? 8 : 4;
  static constexpr int kThreads = 64 + 32 * kEpiWarps;
  static constexpr int kABytes = 128 * 128;
  static constexpr int kStageBytes = kABytes + NT / CG * 128;
  static constexpr int kStaging = kEpiWarps * (kBufBytes + kFactors);
  static constexpr int kFit = (232448 - 2048 - kStaging) / kStageBytes;
  static constexpr int kStages = kFit > 8 ? 8 : kFit;
  static constexpr int kSmem = kStages * kStageBytes + kStaging + 2032;  // 1024 to align, the rest for barriers
};

struct Int8TcMaps {
  CUtensorMap a, b;
};
struct Int8TcArgs {
  DenseTcArgs t;
  const float *x_scale, *w_scale;
};

// An arrival in the pair's first block that orders no memory accesses: the loads from tensor memory before it have been waited
// for, and the fence of tcgen05 stands between.  (One that releases waits for the warp's stores of the tile before: with it
// a drain took a warp 8000 clocks, 4864 x 4096 -> 4096 115 us.)
__device__ __forceinline__ void mbar_arrive_relaxed(uint32_t bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];\n" ::"r"(bar) : "memory");
}

// Values n..n+31 of a row of T, `left` of which exist, added to v.
template <typename T>
__device__ __forceinline__ void add_values(float (&v)[32], const T* p, bool vec, int left) {
  if constexpr (sizeof(T) == 2) {
    uint32_t w[16];
    load_row32(p, vec, left, w);
    add_row32<T>(v, w);
  } else {
    if (vec && left >= 32) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float4 f = __ldg(reinterpret_cast<const float4*>(p) + i);
        v[4 * i] += f.x; v[4 * i + 1] += f.y; v[4 * i + 2] += f.z; v[4 * i + 3] += f.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (i < left) v[i] += p[i];
    }
  }
}

template <typename T, int CG, int NT>
__global__ void __launch_bounds__(Cfg8<CG, NT>::kThreads, 1)
    int8_tc(const __grid_constant__ Int8TcArgs q, const __grid_constant__ Int8TcMaps maps) {
  using C = Cfg8<CG, NT>;
  const DenseTcArgs& p = q.t;
  const int nt = p.nt, b_rows = nt / CG;
  extern __shared__ uint8_t smem_raw[];
  __shared__ volatile int abort_flag;
  __shared__ uint32_t tmem_slot;
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t staging = base + C::kStages * C::kStageBytes;
  const uint32_t bars = staging + C::kStaging;
  auto full = [&](int s) { return bars + 8u * s; };
  auto empty = [&](int s) { return bars + 8u * (C::kStages + s); };
  auto acc_full = [&](int b) { return bars + 8u * (2 * C::kStages + b); };
  auto acc_empty = [&](int b) { return bars + 8u * (2 * C::kStages + 2 + b); };
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0), lane = threadIdx.x % 32;
  const uint32_t rank = CG == 2 ? cluster_rank() : 0;

  if (warp == 0 && lane == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(acc_full(b), 1);
      mbar_init(acc_empty(b), C::kEpiWarps * CG);
    }
    abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    fence_proxy_async();
  }
  if (warp == 1) alloc_tmem<CG>(smem_u32(&tmem_slot), 2 * NT);
  tc_fence_before();
  if constexpr (CG == 2) cluster_sync_all(); else __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_slot, 0);
  griddep_wait();
  griddep_launch();
  const int first = blockIdx.x / CG, step = gridDim.x / CG;

  if (warp == 0) {
    if (elect_one()) {
      const uint32_t stage_bytes = CG * (p.a_rows * 128 + b_rows * 128);
      const uint32_t bar0 = CG == 2 ? map_rank(full(0), 0) : full(0);  // the first block's
      int s = 0;
      uint32_t parity = 1;
      bool ok = true;
      for (int u = first; u < p.units && ok; u += step) {
        const Tile t = tile_of(p, u);
        const int m0 = t.m * (128 * CG) + static_cast<int>(rank) * 128;
        const int n0 = t.n * nt + static_cast<int>(rank) * b_rows;
        int k0 = t.kb0 * kBK;
        for (int kb = 0; kb < t.kbs; ++kb, k0 += kBK) {
          if (!mbar_try_wait(empty(s), parity) && !wait_phase(p.err, empty(s), parity, &abort_flag, 1u)) {
            ok = false;
            break;
          }
          const uint32_t bar = bar0 + 8u * s;
          if (rank == 0) mbar_arrive_expect_tx(bar, stage_bytes);
          const uint32_t a = base + s * C::kStageBytes;
          load_2d<CG>(a, &maps.a, k0, m0, bar);
          load_2d<CG>(a + C::kABytes, &maps.b, k0, n0, bar);
          if (++s == C::kStages) { s = 0; parity ^= 1; }
        }
      }
      // every stage handed out has been released (no arrival is under way when the block ends)
      for (int left = C::kStages; left > 0 && ok; --left) {
        ok = wait_phase(p.err, empty(s), parity, &abort_flag, 1u);
        if (++s == C::kStages) { s = 0; parity ^= 1; }
      }
      if (!ok)  // copies in flight end within microseconds; the block does not return before
        for (int i = 0; i < 1000; ++i) __nanosleep(10000);
    }
  } else if (warp == 1) {
    if (rank == 0 && elect_one()) {
      // D float32, A and B halves, both k-major, N / 8, M / 16
      const uint32_t idesc = (1u << 4) | (static_cast<uint32_t>(nt >> 3) << 17) | (static_cast<uint32_t>(128 * CG >> 4) << 24);
      const uint64_t a0 = smem_desc(base, 16, 1024, 2), b0 = smem_desc(base + C::kABytes, 16, 1024, 2);
      int s = 0, it = 0;
      uint32_t parity = 0;
      bool ok = true;
      for (int u = first; u < p.units && ok; u += step) {
        const int kbs = tile_of(p, u).kbs;
        for (int kb0 = 0; kb0 < kbs && ok; kb0 += kExact, ++it) {
          const int buf = it & 1, n = min(kExact, kbs - kb0);
          if (!wait_phase(p.err, acc_empty(buf), ((it >> 1) & 1) ^ 1, &abort_flag, 2u)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t d = tmem + buf * NT;
          for (int kb = 0; kb < n; ++kb) {
            if (!mbar_try_wait(full(s), parity) && !wait_phase(p.err, full(s), parity, &abort_flag, 4u)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint64_t off = static_cast<uint64_t>(s) * (C::kStageBytes >> 4);
            mma_stage<CG, 2, 2>(d, a0 + off, b0 + off, idesc, kb, empty(s));
            if (++s == C::kStages) { s = 0; parity ^= 1; }
          }
          if (ok) commit<CG>(acc_full(buf));
        }
      }
      if (abort_flag)
        for (int i = 0; i < 1000; ++i) __nanosleep(10000);
    }
  } else {
    const int quarter = warp & 3, half = (warp - 2) >> 2;
    constexpr int kParts = C::kEpiWarps / 4;       // warps that share a quarter's columns
    const uint32_t mine = staging + (warp - 2) * (kBufBytes + kFactors), factors = mine + kBufBytes;
    const DenseEpi& e = p.epi;
    // 32 columns of a lane's row: on 16-byte boundaries the lane writes them itself; else through shared memory, so that a
    // store instruction covers consecutive columns of one row.
    auto put = [&](const float (&v)[32], T* y, int n, int left, int m_warp) {
      if (p.align_y) {
        if (m_warp + lane >= p.M) return;
        uint8_t* row = reinterpret_cast<uint8_t*>(y + static_cast<long long>(m_warp + lane) * e.ldy + n);
        if constexpr (sizeof(T) == 4) {
          store_row32<4>(row, reinterpret_cast<const uint32_t(&)[32]>(v), left, p.align_y);
        } else {
          uint32_t w[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) w[i] = pack_pair<T>(v[2 * i], v[2 * i + 1]);
          store_row32<2>(row, w, left, p.align_y);
        }
        return;
      }
      T* out = y + static_cast<long long>(m_warp) * e.ldy + n + lane;
#pragma unroll
      for (int h = 0; h < 2; ++h) {  // 16 rows at a time
        if (lane / 16 == h) {
#pragma unroll
          for (int i = 0; i < 32; ++i) sts_u32(mine + (lane % 16) * 132 + 4 * i, __float_as_uint(v[i]));
        }
        __syncwarp();
        const int rows = min(16, p.M - m_warp - 16 * h);
        if (lane < left) {
#pragma unroll 4
          for (int r = 0; r < rows; ++r) out[(16 * h + r) * e.ldy] = from_f32<T>(lds_f32(mine + r * 132 + 4 * lane));
        }
        __syncwarp();
      }
    };
    const bool vec_r = (e.ldr * sizeof(T)) % 16 == 0 && reinterpret_cast<uintptr_t>(e.residual) % 16 == 0;
    const int pieces = nt / 32, per_warp = (pieces + kParts - 1) / kParts;
    const int c0 = half * per_warp, mine_n = min(per_warp, pieces - c0);  // of the (up to 4) pieces of 32 columns
    int it = 0;
    for (int u = first; u < p.units; u += step) {
      const Tile t = tile_of(p, u);
      const int m_warp = t.m * (128 * CG) + static_cast<int>(rank) * 128 + quarter * 32;
      const int m = m_warp + lane, n_warp = t.n * nt + 32 * c0;
      const bool rows = m_warp < p.M;
      float xs = 0.0f;
      if (t.slot < 0) {  // the factors of this warp's columns, four a lane
        if (m < p.M) xs = q.x_scale[m];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int n = n_warp + 4 * lane + i;
          const bool ok = n < p.N && 4 * lane + i < 32 * mine_n;
          sts_u32(factors + 16 * lane + 4 * i, __float_as_uint(ok ? q.w_scale[n] : 0.0f));
          sts_u32(factors + 512 + 16 * lane + 4 * i,
                  __float_as_uint(ok && e.bias ? to_f32(static_cast<const T*>(e.bias)[n]) : 0.0f));
        }
        __syncwarp();
      }
      int sum[4][32];
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int i = 0; i < 32; ++i) sum[c][i] = 0;
      bool ok = true;
      const int calls = (t.kbs + kExact - 1) / kExact;
      for (int kb0 = 0; kb0 < t.kbs; kb0 += kExact, ++it) {
        const int buf = it & 1;
        if (!warp_wait(p.err, acc_full(buf), (it >> 1) & 1, &abort_flag, 8u, false, 128, kWaitNs)) {
          ok = false;
          break;
        }
        __syncwarp();
        tc_fence_after();
        const uint32_t at = tmem + buf * NT + (static_cast<uint32_t>(quarter * 32) << 16) + 32 * c0;
        // 16 columns are on their way while 16 are added
        uint32_t v[2][16];
        tmem_ld16_nowait(at, v[0]);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (j / 2 >= mine_n) break;
          tmem_arrived16(v[j % 2]);
          if (j + 1 < 2 * mine_n) tmem_ld16_nowait(at + 16 * (j + 1), v[(j + 1) % 2]);
          add_whole(sum[j / 2] + j % 2 * 16, reinterpret_cast<const float(&)[16]>(v[j % 2]));
        }
        // the accumulator has been read: the next but one may have it
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if constexpr (CG == 2) mbar_arrive_relaxed(map_rank(acc_empty(buf), 0));
          else mbar_arrive(acc_empty(buf));
        }
      }
      if (!ok) break;
      if (!rows) continue;
      // one copy of the code for all pieces: the next piece's sums move into sum[0]
#pragma unroll 1
      for (int c = 0; c < mine_n; ++c) {
        if (c > 0) {
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            sum[0][i] = sum[1][i];
            sum[1][i] = sum[2][i];
            sum[2][i] = sum[3][i];
          }
        }
#pragma unroll
        for (int i = 0; i < 32; ++i) sum[0][i] = whole_value(sum[0][i], calls);
        if (t.slot >= 0) {  // a k range: its sums as they are
          const int row = t.slot * (128 * CG) + static_cast<int>(rank) * 128 + quarter * 32 + lane;
          store_row32<4>(reinterpret_cast<uint8_t*>(p.part + static_cast<long long>(row) * nt + 32 * (c0 + c)),
                         reinterpret_cast<const uint32_t(&)[32]>(sum[0]), 32, 32);
          continue;
        }
        const int n = n_warp + 32 * c, left = p.N - n;
        if (left <= 0) break;
        float v[32];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          uint32_t f[4], b[4];
          lds_v4(factors + 128 * c + 16 * i, f);
          lds_v4(factors + 512 + 128 * c + 16 * i, b);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            v[4 * i + j] = static_cast<float>(sum[0][4 * i + j]) * xs * __uint_as_float(f[j]);
            if (e.bias) v[4 * i + j] += __uint_as_float(b[j]);
          }
        }
        const T* res = static_cast<const T*>(e.residual) + static_cast<long long>(m) * e.ldr + n;
        const int here = m < p.M ? left : 0;
        if (e.residual && !e.residual_last) add_values(v, res, vec_r, here);
        if constexpr (sizeof(T) == 2) dense_activate<true, 32>(v, e.act, e.alpha, e.beta);
        else if (e.act != ACT_IDENTITY) {
          float a[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) a[i] = v[i];
          dense_activate_array(a, e.act, e.alpha, e.beta);
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = a[i];
        }
        if (e.residual && e.residual_last) add_values(v, res, vec_r, here);
        put(v, static_cast<T*>(e.y), n, left, m_warp);
      }
      __syncwarp();  // (the factors are written again)
    }
  }

  __syncwarp();
  tc_fence_before();
  if constexpr (CG == 2) cluster_sync_all(); else __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    free_tmem<CG>(tmem, 2 * NT);
  }
}

// Adds the k ranges' sums of the tiles that were cut, and runs their epilogue: four columns per thread.
template <typename T>
__global__ void __launch_bounds__(256) int8_join(const __grid_constant__ Int8TcArgs q, int tile_rows) {
  griddep_wait();
  griddep_launch();
  const DenseTcArgs& p = q.t;
  const int quads = p.nt / 4;
  const long long per = static_cast<long long>(tile_rows) * quads;
  const long long i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
  const int k = static_cast<int>(i / per);
  if (p.whole + static_cast<long long>(k) * p.split >= p.units) return;
  const int at = static_cast<int>(i - k * per), row = at / quads, c = at % quads * 4;
  const Tile t = tile_of(p, p.whole + k * p.split);
  const int m = t.m * tile_rows + row, n = t.n * p.nt + c;
  if (m >= p.M || n >= p.N) return;
  const long long tile = static_cast<long long>(tile_rows) * p.nt;
  const int* src = reinterpret_cast<const int*>(p.part) + (static_cast<long long>(k) * p.split * tile_rows + row) * p.nt + c;
  int sum[4] = {0, 0, 0, 0};
#pragma unroll 4
  for (int s = 0; s < p.split; ++s) {
    const int4 f = *reinterpret_cast<const int4*>(src + s * tile);
    sum[0] += f.x; sum[1] += f.y; sum[2] += f.z; sum[3] += f.w;
  }
  int col[4];
  bool ok[4];
  float v[4], u[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    col[j] = n + j;
    ok[j] = n + j < p.N;
    v[j] = ok[j] ? static_cast<float>(sum[j]) * q.x_scale[m] * q.w_scale[n + j] : 0.0f;
  }
  dense_epilogue<T, 4>(p.epi, 0, m, col, ok, v, u);
}

template <typename T, int CG, int NT>
cudaError_t go(const Int8TcArgs& args, const Int8TcMaps& maps, int blocks, cudaStream_t s) {
  using C = Cfg8<CG, NT>;
  auto kern = int8_tc<T, CG, NT>;
  const cudaError_t err = opt_in_smem(reinterpret_cast<const void*>(kern), C::kSmem);
  if (err != cudaSuccess) return err;
  return launch_overlapped(kern, dim3(static_cast<unsigned>(blocks)), C::kThreads, C::kSmem, CG, s, args, maps);
}
template <typename T>
cudaError_t run(const DenseTcPlan& t, const Int8TcArgs& args, const Int8TcMaps& maps, cudaStream_t s) {
  const cudaError_t err = t.cg == 2 ? go<T, 2, 256>(args, maps, t.blocks, s) : go<T, 1, 128>(args, maps, t.blocks, s);
  const int cut = t.tiles - t.whole;
  if (err != cudaSuccess || cut == 0) return err;
  const int tile_rows = 128 * t.cg;
  const long long threads = static_cast<long long>(cut) * tile_rows * (t.nt / 4);
  return launch_overlapped(int8_join<T>, dim3(static_cast<unsigned>((threads + 255) / 256)), 256, 0, 1, s, args, tile_rows);
}

}  // namespace

DenseTcPlan int8_tc_plan(int M, int N, int K, int sm) {
  DenseGemm g;
  memset(&g, 0, sizeof(g));
  g.M = M; g.N = N; g.K = K;
  g.segs = g.batch = 1;
  return dense_tc_plan(g, CONV_F16, sm);
}

cudaError_t launch_int8_tc(const DenseTcPlan& t, const Int8Args& g, const __half* x, const __half* w, int dtype, void* part,
                           cudaStream_t s) {
  Int8TcArgs a;
  Int8TcMaps maps;
  memset(&a, 0, sizeof(a));
  memset(&maps, 0, sizeof(maps));
  DenseTcArgs& p = a.t;
  p.M = g.M; p.N = g.N;
  p.segs = p.batch = 1;
  p.nt = t.nt;
  p.kb_seg = p.kb_total = (g.K + kBK - 1) / kBK;
  p.kb_range = t.kb_range;
  p.split = t.split;
  p.mtiles = static_cast<int>((g.M + 128LL * t.cg - 1) / (128 * t.cg));
  p.ntiles = static_cast<int>((static_cast<long long>(g.N) + t.nt - 1) / t.nt);
  p.whole = t.whole;
  p.units = t.whole + (t.tiles - t.whole) * t.split;
  p.group = 16;
  p.epi = g.epi;
  p.part = static_cast<float*>(part);
  p.a_rows = std::min(128, (g.M + 7) / 8 * 8);
  const uintptr_t rows = reinterpret_cast<uintptr_t>(g.epi.y) | static_cast<uintptr_t>(g.epi.ldy * (dtype == CONV_F32 ? 4 : 2));
  p.align_y = rows % 32 == 0 ? 32 : rows % 16 == 0 ? 16 : 0;
  p.err = dense_error_address();
  if (!p.err) return cudaErrorNotSupported;
  a.x_scale = g.x_scale;
  a.w_scale = g.w_scale;
  if (!dense_encode(&maps.a, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, x, g.K, g.M, g.ldx, p.a_rows) ||
      !dense_encode(&maps.b, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, w, g.K, g.N, g.ldw, t.nt / t.cg))
    return cudaErrorInvalidValue;
  return dtype == CONV_F32 ? run<float>(t, a, maps, s) : dtype == CONV_F16 ? run<__half>(t, a, maps, s) : run<__nv_bfloat16>(t, a, maps, s);
}

}  // namespace conv
