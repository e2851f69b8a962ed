// dense_tc.cuh -- the dense products of 16-bit operands on the fifth-generation
// tensor cores (tcgen05, accumulators in tensor memory, operands by TMA).
//
// A tile of D = A B^T is 128 * CG rows by NT columns (CG = 2: a pair of SMs, one
// cluster, works on one tile; each holds 128 rows of A and half of B, and one
// cta_group::2 MMA per 16 terms multiplies both).  Persistent blocks walk over
// the tiles:
//   warp 0     loads 64-term stages of A and B into a ring (128-byte swizzle),
//   warp 1     issues the MMAs (of the pair: in the first block only),
//   the others read finished accumulators and run the epilogue; there are two
//              accumulators, so one tile's epilogue runs under the next one's
//              MMAs.
// Operands are read as they lie: k-major ones as rows of 64 terms, mn-major
// ones as 64 x 64 boxes whose rows run along m or n (the MMA transposes on the
// fly), so neither the layer nor its two gradients need a transposed copy.  The
// gated product loads half a tile of gate columns and half a tile of up
// columns as one B: g and u of an element arrive in one lane of one
// accumulator.  Edges need no code: TMA fills zeros past a matrix's end and
// does not write past the output's.
#pragma once

#include <cuda.h>

#include "dense_internal.h"
#include "tc_ptx.cuh"

namespace conv {

struct DenseTcMaps {
  CUtensorMap a[2], b[2];
  CUtensorMap y[2];    // outputs, boxes of 64 columns x 32 rows
  CUtensorMap pre[2];  // float32 outputs (g, u or the activation's argument, or the ranges' planes): 32 x 32
};

struct DenseTcArgs {
  int M, N;
  int segs, batch, dual, a_mn, b_mn;
  int kb_seg;               // 64-term blocks of a segment
  int kb_total, kb_range;   // of the sum; of a k range
  int split;
  int mtiles, ntiles, tiles, units, group;
  int tma_y, tma_pre;       // those outputs lie on 16-byte boundaries: written by TMA
  DenseEpi epi;
  float* part;
  uint32_t* err;
};

namespace dtc {
using namespace tcx;

constexpr int kBK = 64;
constexpr int kBufBytes = 4096;  // a 32-row staging tile of 128-byte rows

template <int CG, int NT>
struct Cfg {
  static constexpr int kEpiWarps = NT >= 256 ? 8 : 4;
  static constexpr int kThreads = 64 + 32 * kEpiWarps;
  static constexpr int kBRows = NT / CG;
  static constexpr int kABytes = 128 * 128;
  static constexpr int kStageBytes = kABytes + kBRows * 128;
  static constexpr int kStaging = kEpiWarps * 2 * kBufBytes;
  static constexpr int kStages = (232448 - 2048 - kStaging) / kStageBytes > 8 ? 8 : (232448 - 2048 - kStaging) / kStageBytes;
  static constexpr int kSmem = kStages * kStageBytes + kStaging + 2048;  // 1024 to align, 1024 for barriers
  static constexpr int kTmemCols = 2 * NT < 32 ? 32 : 2 * NT;
};

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;\n" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}
// The shared-memory address of the same variable in block `rank` of the cluster.
__device__ __forceinline__ uint32_t map_rank(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];\n" ::"r"(bar) : "memory");
}
template <int CG>
__device__ __forceinline__ void load_2d(uint32_t dst, const void* map, int c0, int c1, uint32_t bar) {
  if constexpr (CG == 2)
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, "
        "%3}], [%4];\n" ::"r"(dst), "l"(map), "r"(c0), "r"(c1), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];\n" ::"r"(dst),
        "l"(map), "r"(c0), "r"(c1), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void store_2d(const void* map, uint32_t src, int c0, int c1) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];\n" ::"l"(map), "r"(c0),
               "r"(c1), "r"(src)
               : "memory");
}
__device__ __forceinline__ void store_3d(const void* map, uint32_t src, int c0, int c1, int c2) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];\n" ::"l"(map),
               "r"(c0), "r"(c1), "r"(c2), "r"(src)
               : "memory");
}
// One MMA, by one lane of the converged warp; and the arrival on `bar` (of
// every block of the pair) when all MMAs issued so far are done.
template <int CG>
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  if constexpr (CG == 2)
    asm volatile(
        "{\n .reg .pred p, e;\n elect.sync _|e, 0xffffffff;\n setp.ne.b32 p, %4, 0;\n"
        " @e tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
  else
    mma_f16_elect(d, a, b, idesc, acc);
}
template <int CG>
__device__ __forceinline__ void commit(uint32_t bar) {
  if constexpr (CG == 2)
    asm volatile(
        "{\n .reg .pred e;\n .reg .b16 m;\n elect.sync _|e, 0xffffffff;\n mov.b16 m, 3;\n"
        " @e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], m;\n}\n" ::"r"(bar)
        : "memory");
  else
    mma_commit_elect(bar);
}
template <int CG>
__device__ __forceinline__ void alloc_tmem(uint32_t slot, uint32_t cols) {
  if constexpr (CG == 2) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(slot), "r"(cols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;\n" ::: "memory");
  } else
    tmem_alloc(slot, cols);
}
template <int CG>
__device__ __forceinline__ void free_tmem(uint32_t base, uint32_t cols) {
  if constexpr (CG == 2)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;\n" ::"r"(base), "r"(cols) : "memory");
  else
    tmem_dealloc(base, cols);
}
// 32 columns of the warp's 32 lanes; no wait.
__device__ __forceinline__ void tmem_ld32(uint32_t addr, float (&v)[32]) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]),
        "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]),
        "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

// Waits for the loads above; the values are operands, so that nothing that uses them moves before the wait.
__device__ __forceinline__ void tmem_arrived(float (&v)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;\n"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]), "+f"(v[8]),
                 "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]), "+f"(v[16]),
                 "+f"(v[17]), "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]), "+f"(v[23]), "+f"(v[24]),
                 "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28]), "+f"(v[29])
               :
               : "memory");
  asm volatile("" : "+f"(v[30]), "+f"(v[31]));
}

template <typename T>
__device__ __forceinline__ uint32_t pack_pair(float lo, float hi) {
  if constexpr (std::is_same<T, __half>::value) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}
// 32 consecutive 16-bit values as float32; `n` of them exist.
template <typename T>
__device__ __forceinline__ void load_row32(const T* p, bool vec, int n, float (&v)[32]) {
  if (vec && n >= 32) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint4 w = __ldg(reinterpret_cast<const uint4*>(p) + q);
      const uint32_t r[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[q * 8 + 2 * i] = to_f32(*reinterpret_cast<const T*>(&r[i]));
        v[q * 8 + 2 * i + 1] = to_f32(reinterpret_cast<const T*>(&r[i])[1]);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = i < n ? to_f32(p[i]) : 0.0f;
  }
}
__device__ __forceinline__ void load_row32f(const float* p, bool vec, int n, float (&v)[32]) {
  if (vec && n >= 32) {
#pragma unroll
    for (int q = 0; q < 8; ++q) *reinterpret_cast<float4*>(v + 4 * q) = __ldg(reinterpret_cast<const float4*>(p) + q);
  } else {
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = i < n ? p[i] : 0.0f;
  }
}

// Where unit u's tile lies: blocks of `group` tile rows are walked column by
// column, so that the tiles in flight share operands in L2.
struct Tile {
  int m, n, batch, range;
};
__device__ __forceinline__ Tile tile_of(const DenseTcArgs& p, int u) {
  Tile t;
  t.range = u / p.tiles;
  int i = u - t.range * p.tiles;
  const int per = p.mtiles * p.ntiles;
  t.batch = i / per;
  i -= t.batch * per;
  const int g = i / (p.group * p.ntiles), first = g * p.group;
  const int rows = min(p.group, p.mtiles - first);
  i -= g * p.group * p.ntiles;
  t.n = i / rows;
  t.m = first + i - t.n * rows;
  return t;
}

template <typename T, int CG, int NT, int MODE>
__global__ void __launch_bounds__(Cfg<CG, NT>::kThreads, 1)
    dense_tc(const __grid_constant__ DenseTcArgs p, const __grid_constant__ DenseTcMaps maps) {
  using C = Cfg<CG, NT>;
  constexpr int kOutCols = MODE == EPI_GATED ? NT / 2 : NT;  // output columns of a tile
  extern __shared__ uint8_t smem_raw[];
  __shared__ volatile int abort_flag;
  __shared__ uint32_t tmem_slot;
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  const uint32_t staging = base + C::kStages * C::kStageBytes;
  const uint32_t bars = staging + C::kStaging;
  auto full = [&](int s) { return bars + 8u * s; };
  auto empty = [&](int s) { return bars + 8u * (C::kStages + s); };
  auto acc_full = [&](int b) { return bars + 8u * (2 * C::kStages + b); };
  auto acc_empty = [&](int b) { return bars + 8u * (2 * C::kStages + 2 + b); };
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
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
  if (warp == 1) alloc_tmem<CG>(smem_u32(&tmem_slot), C::kTmemCols);
  tc_fence_before();
  if constexpr (CG == 2) cluster_sync_all(); else __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  const int first = blockIdx.x / CG, step = gridDim.x / CG;

  if (warp == 0) {
    if (lane == 0) {
      int it = 0;
      bool ok = true;
      for (int u = first; u < p.units && ok; u += step) {
        const Tile t = tile_of(p, u);
        const int kb0 = t.range * p.kb_range, kb1 = min(kb0 + p.kb_range, p.kb_total);
        const int m0 = t.m * (128 * CG) + static_cast<int>(rank) * 128;
        for (int kb = kb0; kb < kb1; ++kb, ++it) {
          const int s = it % C::kStages;
          if (!wait_phase(p.err, empty(s), ((it / C::kStages) & 1) ^ 1, &abort_flag, 1u)) { ok = false; break; }
          const uint32_t bar = CG == 2 ? map_rank(full(s), 0) : full(s);
          if (rank == 0) mbar_arrive_expect_tx(full(s), CG * C::kStageBytes);
          const int seg = kb >= p.kb_seg ? 1 : 0;
          const int k0 = (kb - seg * p.kb_seg) * kBK;
          const int op = p.segs > 1 ? seg : t.batch;
          const uint32_t a = base + s * C::kStageBytes, b = a + C::kABytes;
          if (p.a_mn) {
            load_2d<CG>(a, &maps.a[op], m0, k0, bar);
            load_2d<CG>(a + 8192, &maps.a[op], m0 + 64, k0, bar);
          } else {
            load_2d<CG>(a, &maps.a[op], k0, m0, bar);
          }
          if constexpr (MODE == EPI_GATED) {
            if constexpr (CG == 2) {  // the first block's half of B is the gate's, the second's the up projection's
              load_2d<CG>(b, &maps.b[rank], k0, t.n * kOutCols, bar);
            } else {
              load_2d<CG>(b, &maps.b[0], k0, t.n * kOutCols, bar);
              load_2d<CG>(b + kOutCols * 128, &maps.b[1], k0, t.n * kOutCols, bar);
            }
          } else {
            const int n0 = t.n * NT + static_cast<int>(rank) * C::kBRows;
            if (p.b_mn) {
#pragma unroll
              for (int i = 0; i < C::kBRows / 64; ++i) load_2d<CG>(b + i * 8192, &maps.b[op], n0 + 64 * i, k0, bar);
            } else {
              load_2d<CG>(b, &maps.b[op], k0, n0, bar);
            }
          }
        }
      }
      // every stage handed out has been released (no arrival is under way when the block ends)
      for (int i = 0; i < C::kStages && ok; ++i, ++it)
        ok = wait_phase(p.err, empty(it % C::kStages), ((it / C::kStages) & 1) ^ 1, &abort_flag, 1u);
      if (!ok)  // copies in flight end within microseconds; the block does not return before
        for (int i = 0; i < 1000; ++i) __nanosleep(10000);
    }
  } else if (warp == 1) {
    if (rank == 0) {
      // D float32, A and B of type T, transposes, N / 8, M / 16
      const uint32_t kind = std::is_same<T, __nv_bfloat16>::value ? 1u : 0u;
      const uint32_t idesc = (1u << 4) | (kind << 7) | (kind << 10) | (static_cast<uint32_t>(p.a_mn) << 15) |
                             (static_cast<uint32_t>(p.b_mn) << 16) | (static_cast<uint32_t>(NT >> 3) << 17) |
                             (static_cast<uint32_t>(128 * CG >> 4) << 24);
      // 128-byte swizzle.  k-major: 8-row groups 1024 bytes apart, 16 terms are 32 bytes of a row.  mn-major: 64-wide
      // blocks 8192 bytes apart (the leading offset), groups of 8 terms 1024 apart, 16 terms are 2048 bytes.
      const uint32_t a_step = p.a_mn ? 2048 >> 4 : 32 >> 4, b_step = p.b_mn ? 2048 >> 4 : 32 >> 4;
      const uint64_t a_hi = smem_desc(0, p.a_mn ? 8192 : 16, 1024, 2), b_hi = smem_desc(0, p.b_mn ? 8192 : 16, 1024, 2);
      int it = 0, tile_it = 0;
      bool ok = true;
      for (int u = first; u < p.units && ok; u += step, ++tile_it) {
        const int range = u / p.tiles;
        const int kb0 = range * p.kb_range, kb1 = min(kb0 + p.kb_range, p.kb_total);
        const int buf = tile_it & 1;
        if (!wait_phase(p.err, acc_empty(buf), ((tile_it >> 1) & 1) ^ 1, &abort_flag, 2u)) break;
        __syncwarp();
        tc_fence_after();
        const uint32_t d = tmem + buf * NT;
        for (int kb = kb0; kb < kb1; ++kb, ++it) {
          const int s = it % C::kStages;
          if (!wait_phase(p.err, full(s), (it / C::kStages) & 1, &abort_flag, 4u)) { ok = false; break; }
          __syncwarp();
          tc_fence_after();
          const uint32_t a = base + s * C::kStageBytes, b = a + C::kABytes;
          const uint64_t ad = a_hi | (a >> 4), bd = b_hi | (b >> 4);
#pragma unroll
          for (int k = 0; k < kBK / 16; ++k)
            mma<CG>(d, ad + k * a_step, bd + k * b_step, idesc, kb > kb0 || k > 0);
          commit<CG>(empty(s));
        }
        if (ok) commit<CG>(acc_full(buf));
      }
      if (abort_flag)
        for (int i = 0; i < 1000; ++i) __nanosleep(10000);
      __syncwarp();
    }
  } else {
    const int quarter = warp & 3, half = (warp - 2) >> 2;
    constexpr int kParts = C::kEpiWarps / 4;       // warps that share a quarter's columns
    constexpr int kCols = kOutCols / kParts;       // output columns of this warp
    static_assert(kCols % 64 == 0, "whole staging tiles");
    const uint32_t mine = staging + (warp - 2) * 2 * kBufBytes;
    const DenseEpi& e = p.epi;
    int ring = 0;
    // the next staging tile, free of its last store
    auto acquire = [&]() {
      if (lane == 0) bulk_wait_read<1>();
      __syncwarp();
      const uint32_t b = mine + (ring & 1) * kBufBytes;
      ++ring;
      return b;
    };
    auto publish = [&]() {
      fence_proxy_async();
      __syncwarp();
    };
    // 64 16-bit columns (32 words) of this lane's row
    auto put16 = [&](const uint32_t (&w)[32], const CUtensorMap* map, T* y, int n, int m_warp) {
      if (p.tma_y) {
        const uint32_t b = acquire();
#pragma unroll
        for (int q = 0; q < 8; ++q)
          sts_v4(b + lane * 128 + ((q ^ (lane & 7)) << 4), make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]));
        publish();
        if (lane == 0) {
          store_2d(map, b, n, m_warp);
          bulk_commit();
        }
      } else if (m_warp + lane < p.M) {
        T* row = y + static_cast<long long>(m_warp + lane) * e.ldy + n;
#pragma unroll
        for (int j = 0; j < 64; ++j)
          if (n + j < p.N) {
            const uint16_t v = static_cast<uint16_t>(w[j / 2] >> (16 * (j & 1)));
            row[j] = *reinterpret_cast<const T*>(&v);
          }
      }
    };
    // 32 float32 columns of this lane's row (plane >= 0: of the ranges' planes)
    auto put32 = [&](const float (&v)[32], const CUtensorMap* map, float* out, long long ld, int n, int m_warp, int plane) {
      if (n >= p.N) return;
      if (p.tma_pre) {
        const uint32_t b = acquire();
#pragma unroll
        for (int q = 0; q < 8; ++q)
          sts_v4(b + lane * 128 + ((q ^ (lane & 7)) << 4),
                 make_uint4(__float_as_uint(v[4 * q]), __float_as_uint(v[4 * q + 1]), __float_as_uint(v[4 * q + 2]),
                            __float_as_uint(v[4 * q + 3])));
        publish();
        if (lane == 0) {
          if (plane >= 0) store_3d(map, b, n, m_warp, plane);
          else store_2d(map, b, n, m_warp);
          bulk_commit();
        }
      } else if (m_warp + lane < p.M) {
        float* row = out + (plane >= 0 ? static_cast<long long>(plane) * p.M * p.N : 0) +
                     static_cast<long long>(m_warp + lane) * ld + n;
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (n + j < p.N) row[j] = v[j];
      }
    };
    const bool vec_r = e.residual && e.ldr % 8 == 0 && reinterpret_cast<uintptr_t>(e.residual) % 16 == 0;
    const bool vec_b = reinterpret_cast<uintptr_t>(e.bias) % 16 == 0;
    const bool vec_p = e.ldp % 4 == 0 && reinterpret_cast<uintptr_t>(e.pre) % 16 == 0 &&
                       reinterpret_cast<uintptr_t>(e.pre2) % 16 == 0;
    int tile_it = 0;
    for (int u = first; u < p.units; u += step, ++tile_it) {
      const Tile t = tile_of(p, u);
      const int buf = tile_it & 1;
      if (!wait_phase(p.err, acc_full(buf), (tile_it >> 1) & 1, &abort_flag, 8u, false, 64,
                      kWaitNs + 1000ull * p.kb_range))  // a stage takes below a microsecond
        break;
      tc_fence_after();
      const uint32_t acc = tmem + buf * NT + (static_cast<uint32_t>(quarter * 32) << 16);
      const int m_warp = t.m * (128 * CG) + static_cast<int>(rank) * 128 + quarter * 32;
      const int m = m_warp + lane;
      const int col0 = half * kCols;
#pragma unroll 1
      for (int c = 0; c < kCols; c += 64) {
        const int n = t.n * kOutCols + col0 + c;
        const bool dead = n >= p.N || m_warp >= p.M;  // nothing of this piece exists
        uint32_t w0[32], w1[32];
#pragma unroll
        for (int sub = 0; sub < 2; ++sub) {
          float v[32];
          tmem_ld32(acc + col0 + c + sub * 32, v);
          const int ns = n + sub * 32, left = p.N - ns;  // columns that exist
          const bool row_ok = m < p.M && left > 0;
          if constexpr (MODE == EPI_PARTIAL) {
            tmem_arrived(v);
            if (!dead) put32(v, &maps.pre[0], p.part, p.N, ns, m_warp, t.range * (p.dual ? 2 : p.batch) + t.batch);
          } else if constexpr (MODE == EPI_GATED) {
            float g[32];
            tmem_ld32(acc + NT / 2 + col0 + c + sub * 32, g);
            tmem_arrived(v);
            tmem_arrived(g);
            if (dead) continue;
            if (e.pre) {
              put32(v, &maps.pre[0], e.pre, e.ldp, ns, m_warp, -1);
              put32(g, &maps.pre[1], e.pre2, e.ldp, ns, m_warp, -1);
            }
            dense_activate<true, 32>(v, e.act, e.alpha, e.beta);
#pragma unroll
            for (int i = 0; i < 16; ++i) w0[sub * 16 + i] = pack_pair<T>(v[2 * i] * g[2 * i], v[2 * i + 1] * g[2 * i + 1]);
          } else if constexpr (MODE == EPI_GATED_BWD) {
            float g[32], gr[32], uu[32];
            const long long at = static_cast<long long>(m) * e.ldp + ns;
            if (row_ok) {
              load_row32f(e.pre + at, vec_p, left, g);
              load_row32f(e.pre2 + at, vec_p, left, uu);
            } else {
#pragma unroll
              for (int i = 0; i < 32; ++i) g[i] = uu[i] = 0.0f;
            }
            dense_activate_grad<true, 32>(g, gr, e.act, e.alpha, e.beta);
            tmem_arrived(v);
            if (dead) continue;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              w0[sub * 16 + i] = pack_pair<T>(v[2 * i] * uu[2 * i] * gr[2 * i], v[2 * i + 1] * uu[2 * i + 1] * gr[2 * i + 1]);
              w1[sub * 16 + i] = pack_pair<T>(v[2 * i] * g[2 * i], v[2 * i + 1] * g[2 * i + 1]);
            }
          } else {
            float r[32];
            if (e.residual) {
              if (row_ok) load_row32(static_cast<const T*>(e.residual) + static_cast<long long>(m) * e.ldr + ns, vec_r, left, r);
              else {
#pragma unroll
                for (int i = 0; i < 32; ++i) r[i] = 0.0f;
              }
            }
            tmem_arrived(v);
            if (dead) continue;
            if (e.bias) {
              float bv[32];
              load_row32(static_cast<const T*>(e.bias) + ns, vec_b, left, bv);
#pragma unroll
              for (int i = 0; i < 32; ++i) v[i] += bv[i];
            }
            if (e.residual && !e.residual_last) {
#pragma unroll
              for (int i = 0; i < 32; ++i) v[i] += r[i];
            }
            if (e.pre) put32(v, &maps.pre[0], e.pre, e.ldp, ns, m_warp, -1);
            dense_activate<true, 32>(v, e.act, e.alpha, e.beta);
            if (e.residual && e.residual_last) {
#pragma unroll
              for (int i = 0; i < 32; ++i) v[i] += r[i];
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) w0[sub * 16 + i] = pack_pair<T>(v[2 * i], v[2 * i + 1]);
          }
        }
        if (c + 64 >= kCols) {  // the accumulator has been read: the next but one tile may have it
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            if constexpr (CG == 2) mbar_arrive_cluster(map_rank(acc_empty(buf), 0));
            else mbar_arrive(acc_empty(buf));
          }
        }
        if constexpr (MODE != EPI_PARTIAL) {
          if (!dead) {
            if constexpr (MODE == EPI_GATED_BWD) {
              put16(w0, &maps.y[0], static_cast<T*>(e.y), n, m_warp);
              put16(w1, &maps.y[1], static_cast<T*>(e.y2), n, m_warp);
            } else {
              put16(w0, &maps.y[t.batch], static_cast<T*>(t.batch ? e.y2 : e.y), n, m_warp);
            }
          }
        }
      }
    }
    if (lane == 0) bulk_wait_all();
    __syncwarp();
  }

  __syncwarp();
  tc_fence_before();
  if constexpr (CG == 2) cluster_sync_all(); else __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    free_tmem<CG>(tmem, C::kTmemCols);
  }
}

}  // namespace dtc
}  // namespace conv
