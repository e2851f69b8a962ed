// dense_tc.cuh -- the dense products of 16-bit operands on the fifth-generation
// tensor cores (tcgen05, accumulators in tensor memory, operands by TMA).
//
// A tile of D = A B^T is 128 * CG rows by nt columns (CG = 2: a pair of SMs, one
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
// accumulator.  TMA fills zeros past a matrix's end, so edges need no code in the
// loops.
//
// What bounds it: long sums, the MMAs, then the power limit.  A pair's tile of
// 256 x 256 takes 32 KB into each SM per 512 clocks of MMAs, which is what the
// path from L2 carries (64 bytes a clock); smaller tiles wait for it.  8192 x
// 4096 -> 12288, bfloat16, full speed: 430 to 440 us, 1.9 PFLOP/s (98% of
// measured), both operands mn-major 420 (768 tiles: the tenth round full, the
// rest in ranges); over seconds the clock falls to 1.5 GHz and both to 1.6 to
// 1.7.  Short sums wait for the epilogue: 32 columns of 32 rows take a warp
// some 900 clocks, with gelu and its argument's store 2900, beside 608 clocks
// per 64 terms.  What made it: the issuing loops.  As first written, with
// operand orders read at run time and the branch on a lane's number, a stage
// took 530 clocks to issue whatever the tile.
#pragma once

#include <cuda.h>

#include "dense_internal.h"
#include "tc_ptx.cuh"

namespace conv {

struct DenseTcMaps {
  CUtensorMap a[2], b[2];
  CUtensorMap y[2], pre[2], part;  // float32 products: the outputs, boxes of 32 columns x 32 rows
};

struct DenseTcArgs {
  int M, N;
  int nt;                   // MMA columns of a tile: a multiple of 32 (64 gated), at most the kernel's NT
  int segs, batch;
  int a_rows;               // k-major A: rows of a copy (128; fewer where M has no more: the rest of the tile is not stored)
  int a_3d, b_3d;           // mn-major: all of a stage's 64-wide boxes in one copy
  int kb_seg;               // 64-term blocks of a segment
  int kb_total, kb_range;   // of the sum; of a k range
  // Units of work: `whole` tiles with their epilogue, then the others (the last, partly filled round of blocks) as
  // `split` k ranges each, whose raw sums go to `part`, one tile after another (a second kernel adds them)
  int whole, split, units;
  int mtiles, ntiles, group;
  int align_y, align_pre;   // the rows' boundaries: 32 or 16 bytes, 0: neither
  DenseEpi epi;
  float* part;
  uint32_t* err;
};

namespace dtc {
using namespace tcx;

constexpr int kBK = 64;
constexpr int kBufBytes = 2304;   // a warp's staging: 32 rows of 32 16-bit values, or 16 of 32 float32, a word apart
constexpr int kBiasBytes = 256;   // and the bias of its (up to 128) columns

template <int CG, int NT>
struct Cfg {
  static constexpr int kEpiWarps = NT >= 256 ? 8 : 4;
  static constexpr int kThreads = 64 + 32 * kEpiWarps;
  static constexpr int kABytes = 128 * 128;
  static constexpr int kStageBytes = kABytes + NT / CG * 128;
  static constexpr int kStaging = kEpiWarps * (kBufBytes + kBiasBytes);
  static constexpr int kFit = (232448 - 2048 - kStaging) / kStageBytes;
  static constexpr int kStages = kFit > 8 ? 8 : kFit;
  static constexpr int kSmem = kStages * kStageBytes + kStaging + 2032;  // 1024 to align, the rest for barriers
};

// A wait of a whole warp: one lane polls (32 polling lanes, of eight warps, take shared-memory cycles from the MMAs).
__device__ __forceinline__ bool warp_wait(uint32_t* err, uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                          uint32_t code, bool ignore_abort = false, uint32_t sleep_ns = 0,
                                          unsigned long long limit_ns = kWaitNs) {
  int ok = 1;
  if (threadIdx.x % 32 == 0) ok = wait_phase(err, bar, parity, abort_flag, code, ignore_abort, sleep_ns, limit_ns);
  ok = __shfl_sync(0xffffffffu, ok, 0);
  return ok != 0;
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;\n" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}
// One lane of a converged warp.  (A branch on the lane's number would do, but not tell the compiler that one lane alone
// is inside: it then guards every TMA and MMA instruction against several.)
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n selp.u32 %0, 1, 0, e;\n}\n" : "=r"(p));
  return p != 0;
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
template <int CG>
__device__ __forceinline__ void load_3d(uint32_t dst, const void* map, int c0, int c1, int c2, uint32_t bar) {
  if constexpr (CG == 2)
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, "
        "%3, %4}], [%5];\n" ::"r"(dst), "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
        "[%5];\n" ::"r"(dst), "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
        : "memory");
}
// 32 bytes from or to global memory (on a 32-byte boundary).  What an epilogue reads or writes passes through L2 once: it
// is the first to go, so that the operands' tiles, which are read by many blocks, stay.
__device__ __forceinline__ void load_32b(const void* p, uint32_t* r) {
  asm volatile("ld.global.L2::evict_first.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "l"(p)
               : "memory");
}
__device__ __forceinline__ void store_32b(void* p, const uint32_t* r) {
  asm volatile("st.global.L2::evict_first.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};\n" ::"l"(p), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ void store_16b(void* p, const uint32_t* r) {
  asm volatile("st.global.v4.b32 [%0], {%1, %2, %3, %4};\n" ::"l"(p), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]) : "memory");
}
__device__ __forceinline__ void prefetch_l2(const void* p) {
  asm volatile("prefetch.global.L2 [%0];\n" ::"l"(p) : "memory");
}
// 32 values of B bytes each (packed into words) of a row, `left` of which exist, on boundaries of `align` (16 or 32)
// bytes.
template <int B>
__device__ __forceinline__ void store_row32(uint8_t* row, const uint32_t (&w)[8 * B], int left, int align) {
  constexpr int kPer = 32 / B;  // values of 32 bytes
#pragma unroll
  for (int j = 0; j < B; ++j) {
    if (left >= kPer * (j + 1)) {
      if (align == 32) store_32b(row + 32 * j, w + 8 * j);
      else {
        store_16b(row + 32 * j, w + 8 * j);
        store_16b(row + 32 * j + 16, w + 8 * j + 4);
      }
    } else {
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (kPer * j + i < left) {
          if constexpr (B == 4) reinterpret_cast<uint32_t*>(row)[kPer * j + i] = w[8 * j + i];
          else reinterpret_cast<uint16_t*>(row)[kPer * j + i] = static_cast<uint16_t>(w[8 * j + i / 2] >> (16 * (i & 1)));
        }
    }
  }
}
__device__ __forceinline__ void store_2d(const void* map, uint32_t src, int c0, int c1) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];\n" ::"l"(map), "r"(c0),
               "r"(c1), "r"(src)
               : "memory");
}
// The MMAs of one 64-term stage, then the arrival on `bar` (of every block of the pair) when they are done.
template <int CG, int A_STEP, int B_STEP>
__device__ __forceinline__ void mma_stage(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc, uint32_t bar) {
#define CONV_MMA_STAGE(GROUP, COMMIT)                                                                    \
  asm volatile(                                                                                          \
      "{\n .reg .pred p, q;\n .reg .b64 a1, a2, a3, b1, b2, b3;\n .reg .b16 m;\n"                        \
      " setp.ne.b32 p, %6, 0;\n setp.eq.b32 q, 0, 0;\n mov.b16 m, 3;\n"    \
      " add.s64 a1, %1, %3;\n add.s64 b1, %2, %4;\n add.s64 a2, a1, %3;\n add.s64 b2, b1, %4;\n"         \
      " add.s64 a3, a2, %3;\n add.s64 b3, b2, %4;\n"                                                     \
      " tcgen05.mma.cta_group::" GROUP ".kind::f16 [%0], %1, %2, %5, p;\n"                            \
      " tcgen05.mma.cta_group::" GROUP ".kind::f16 [%0], a1, b1, %5, q;\n"                            \
      " tcgen05.mma.cta_group::" GROUP ".kind::f16 [%0], a2, b2, %5, q;\n"                            \
      " tcgen05.mma.cta_group::" GROUP ".kind::f16 [%0], a3, b3, %5, q;\n"                            \
      " tcgen05.commit.cta_group::" GROUP ".mbarrier::arrive::one.shared::cluster" COMMIT ";\n}\n" ::"r"(d), \
      "l"(a), "l"(b), "n"(A_STEP), "n"(B_STEP), "r"(idesc), "r"(acc), "r"(bar)                           \
      : "memory")
  if constexpr (CG == 2) CONV_MMA_STAGE("2", ".multicast::cluster.b64 [%7], m");
  else CONV_MMA_STAGE("1", ".b64 [%7]");
#undef CONV_MMA_STAGE
}
// One MMA onto the accumulator's values divided by 2^DOWN (one SM).
template <int DOWN>
__device__ __forceinline__ void mma_onto(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc) {
  asm volatile("{\n .reg .pred p;\n setp.eq.b32 p, 0, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p, %4;\n}\n" ::"r"(d),
               "l"(a), "l"(b), "r"(idesc), "n"(DOWN)
               : "memory");
}
// The MMAs of 64 terms alone (one SM).  DOWN < 0: a new sum; else onto the one that is there, divided by 2^DOWN.
template <int DOWN, int A_STEP, int B_STEP>
__device__ __forceinline__ void mma_terms(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc) {
  if constexpr (DOWN > 0) mma_onto<DOWN>(d, a, b, idesc);
  else mma_f16(d, a, b, idesc, DOWN == 0);
  mma_f16(d, a + A_STEP, b + B_STEP, idesc, 1);
  mma_f16(d, a + 2 * A_STEP, b + 2 * B_STEP, idesc, 1);
  mma_f16(d, a + 3 * A_STEP, b + 3 * B_STEP, idesc, 1);
}
template <int CG>
__device__ __forceinline__ void commit(uint32_t bar) {
  if constexpr (CG == 2)
    asm volatile(
        "{\n .reg .b16 m;\n mov.b16 m, 3;\n"
        " tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], m;\n}\n" ::"r"(bar)
        : "memory");
  else
    mma_commit(bar);
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
// 32 consecutive 16-bit values, packed; `n` of them exist (n <= 0: none).
template <typename T>
__device__ __forceinline__ void load_row32(const T* p, bool vec, int n, uint32_t (&w)[16]) {
  if (vec && n >= 32) {
#pragma unroll
    for (int q = 0; q < 4; ++q) *reinterpret_cast<uint4*>(w + 4 * q) = __ldg(reinterpret_cast<const uint4*>(p) + q);
  } else {
    const uint16_t* h = reinterpret_cast<const uint16_t*>(p);
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = pack2(2 * i < n ? h[2 * i] : 0, 2 * i + 1 < n ? h[2 * i + 1] : 0);
  }
}
template <typename T>
__device__ __forceinline__ void add_row32(float (&v)[32], const uint32_t (&w)[16]) {
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    v[2 * i] += to_f32(*reinterpret_cast<const T*>(&w[i]));
    v[2 * i + 1] += to_f32(reinterpret_cast<const T*>(&w[i])[1]);
  }
}

__device__ __forceinline__ void lds_v4(uint32_t addr, uint32_t* r) {
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];\n" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void sts_u32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared.u32 [%0], %1;\n" ::"r"(addr), "r"(v) : "memory");
}

// Unit u: its tile (blocks of `group` tile rows are walked column by column, so that the tiles in flight share operands
// in L2) and its 64-term blocks.
struct Tile {
  int m, n, batch;
  int slot;      // raw sums: the place in `part`; -1: the whole tile
  int kb0, kbs;
};
__device__ __forceinline__ Tile tile_of(const DenseTcArgs& p, int u) {
  Tile t;
  int i = u;
  t.slot = -1;
  t.kb0 = 0;
  t.kbs = p.kb_total;
  if (u >= p.whole) {
    t.slot = u - p.whole;
    const int q = t.slot / p.split;
    i = p.whole + q;
    t.kb0 = (t.slot - q * p.split) * p.kb_range;
    t.kbs = min(p.kb_range, p.kb_total - t.kb0);
  }
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

template <typename T, int CG, int NT, int MODE, bool A_MN, bool B_MN>
__global__ void __launch_bounds__(Cfg<CG, NT>::kThreads, 1)
    dense_tc(const __grid_constant__ DenseTcArgs p, const __grid_constant__ DenseTcMaps maps) {
  using C = Cfg<CG, NT>;
  const int nt = p.nt, out_cols = MODE == EPI_GATED ? nt / 2 : nt;  // a tile's columns of the output
  const int b_rows = nt / CG;                                      // rows of B in this block
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

  // The two issuing loops are one thread's: every instruction of theirs counts (a stage's MMAs take 512 clocks at most).
  // Operand orders are compiled in, addresses are carried from stage to stage.
  if (warp == 0) {
    if (elect_one()) {
      // bytes of a stage, both blocks' together: whole boxes, past the matrices' ends too
      const int b_boxes = (b_rows + 63) / 64;
      const uint32_t stage_bytes = CG * ((A_MN ? C::kABytes : p.a_rows * 128) + (B_MN ? b_boxes * 8192 : b_rows * 128));
      const uint32_t bar0 = CG == 2 ? map_rank(full(0), 0) : full(0);  // the first block's
      const bool a_3d = A_MN && p.a_3d, b_3d = B_MN && p.b_3d;
      int s = 0, left = 0;
      uint32_t parity = 1;
      bool ok = true;
      for (int u = first; u < p.units && ok; u += step) {
        const Tile t = tile_of(p, u);
        const int kb0 = t.kb0, kb1 = kb0 + t.kbs;
        const int m0 = t.m * (128 * CG) + static_cast<int>(rank) * 128;
        const int n0 = MODE == EPI_GATED ? t.n * out_cols : t.n * nt + static_cast<int>(rank) * b_rows;
        for (int kb = kb0; kb < kb1 && ok;) {
          const int seg = kb >= p.kb_seg ? 1 : 0;
          const int op = p.segs > 1 ? seg : t.batch;
          const CUtensorMap* am = &maps.a[op];
          const CUtensorMap* bm = &maps.b[MODE == EPI_GATED && CG == 2 ? rank : op];
          int k0 = (kb - seg * p.kb_seg) * kBK;
          const int end = seg ? kb1 : min(kb1, p.kb_seg);
          for (; kb < end; ++kb, k0 += kBK) {
            if (!mbar_try_wait(empty(s), parity) && !wait_phase(p.err, empty(s), parity, &abort_flag, 1u)) {
              ok = false;
              break;
            }
            const uint32_t bar = bar0 + 8u * s;
            if (rank == 0) mbar_arrive_expect_tx(bar0 + 8u * s, stage_bytes);
            const uint32_t a = base + s * C::kStageBytes, b = a + C::kABytes;
            if constexpr (A_MN) {
              if (a_3d) load_3d<CG>(a, am, 0, k0, m0 / 64, bar);
              else {
                load_2d<CG>(a, am, m0, k0, bar);
                load_2d<CG>(a + 8192, am, m0 + 64, k0, bar);
              }
            } else {
              load_2d<CG>(a, am, k0, m0, bar);
            }
            if constexpr (MODE == EPI_GATED) {
              // of a pair, the first block's half of B is the gate's, the second's the up projection's
              load_2d<CG>(b, bm, k0, n0, bar);
              if constexpr (CG == 1) load_2d<CG>(b + out_cols * 128, &maps.b[1], k0, n0, bar);
            } else if constexpr (B_MN) {
              if (b_3d) load_3d<CG>(b, bm, 0, k0, n0 / 64, bar);
              else
                for (int i = 0; i < b_boxes; ++i) load_2d<CG>(b + i * 8192, bm, n0 + 64 * i, k0, bar);
            } else {
              load_2d<CG>(b, bm, k0, n0, bar);
            }
            if (++s == C::kStages) { s = 0; parity ^= 1; }
          }
        }
      }
      // every stage handed out has been released (no arrival is under way when the block ends)
      for (left = C::kStages; left > 0 && ok; --left) {
        ok = wait_phase(p.err, empty(s), parity, &abort_flag, 1u);
        if (++s == C::kStages) { s = 0; parity ^= 1; }
      }
      if (!ok)  // copies in flight end within microseconds; the block does not return before
        for (int i = 0; i < 1000; ++i) __nanosleep(10000);
    }
  } else if (warp == 1) {
    if (rank == 0 && elect_one()) {
      // D float32, A and B of type T, transposes, N / 8, M / 16
      const uint32_t kind = std::is_same<T, __nv_bfloat16>::value ? 1u : 0u;
      const uint32_t idesc = (1u << 4) | (kind << 7) | (kind << 10) | (static_cast<uint32_t>(A_MN) << 15) |
                             (static_cast<uint32_t>(B_MN) << 16) | (static_cast<uint32_t>(nt >> 3) << 17) |
                             (static_cast<uint32_t>(128 * CG >> 4) << 24);
      // 128-byte swizzle.  k-major: 8-row groups 1024 bytes apart, 16 terms are 32 bytes of a row.  mn-major: 64-wide
      // blocks 8192 bytes apart (the leading offset), groups of 8 terms 1024 apart, 16 terms are 2048 bytes.
      constexpr int kAStep = A_MN ? 2048 >> 4 : 32 >> 4, kBStep = B_MN ? 2048 >> 4 : 32 >> 4;
      const uint64_t a0 = smem_desc(base, A_MN ? 8192 : 16, 1024, 2);
      const uint64_t b0 = smem_desc(base + C::kABytes, B_MN ? 8192 : 16, 1024, 2);
      int s = 0, tile_it = 0;
      uint32_t parity = 0;
      bool ok = true;
      for (int u = first; u < p.units && ok; u += step, ++tile_it) {
        const int kbs = tile_of(p, u).kbs;
        const int buf = tile_it & 1;
        if (!wait_phase(p.err, acc_empty(buf), ((tile_it >> 1) & 1) ^ 1, &abort_flag, 2u)) break;
        tc_fence_after();
        const uint32_t d = tmem + buf * NT;
        for (int kb = 0; kb < kbs; ++kb) {
          if (!mbar_try_wait(full(s), parity) && !wait_phase(p.err, full(s), parity, &abort_flag, 4u)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t off = static_cast<uint64_t>(s) * (C::kStageBytes >> 4);
          mma_stage<CG, kAStep, kBStep>(d, a0 + off, b0 + off, idesc, kb, empty(s));
          if (++s == C::kStages) { s = 0; parity ^= 1; }
        }
        if (ok) commit<CG>(acc_full(buf));
      }
      if (abort_flag)
        for (int i = 0; i < 1000; ++i) __nanosleep(10000);
    }
  } else {
    const int quarter = warp & 3, half = (warp - 2) >> 2;
    constexpr int kParts = C::kEpiWarps / 4;       // warps that share a quarter's columns
    const uint32_t mine = staging + (warp - 2) * (kBufBytes + kBiasBytes);
    const DenseEpi& e = p.epi;
    // A lane holds 32 columns of one row.  On 16-byte boundaries it writes them itself, in whole sectors: nothing to wait
    // for.  (Staged tiles that TMA stores took 400 to 1300 clocks each until their place was free again.)  Rows of other
    // alignments go through shared memory: a store instruction covers 32 consecutive columns of one row.
    auto put16 = [&](const uint32_t (&w)[16], T* y, int n, int left, int m_warp) {
      if (p.align_y) {
        if (m_warp + lane < p.M)
          store_row32<2>(reinterpret_cast<uint8_t*>(y + static_cast<long long>(m_warp + lane) * e.ldy + n), w, left, p.align_y);
        return;
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) sts_u32(mine + lane * 68 + 4 * i, w[i]);
      __syncwarp();
      uint16_t* out = reinterpret_cast<uint16_t*>(y + static_cast<long long>(m_warp) * e.ldy + n) + lane;
      const int rows = min(32, p.M - m_warp);
      if (lane < left) {
#pragma unroll 8
        for (int r = 0; r < rows; ++r) out[r * e.ldy] = lds_u16(mine + r * 68 + 2 * lane);
      }
      __syncwarp();
    };
    auto put32 = [&](const float (&v)[32], float* out, int n, int left, int m_warp) {
      if (p.align_pre) {
        if (m_warp + lane < p.M)
          store_row32<4>(reinterpret_cast<uint8_t*>(out + static_cast<long long>(m_warp + lane) * e.ldp + n),
                         reinterpret_cast<const uint32_t(&)[32]>(v), left, p.align_pre);
        return;
      }
      out += static_cast<long long>(m_warp) * e.ldp + n + lane;
#pragma unroll
      for (int h = 0; h < 2; ++h) {  // 16 rows at a time
        if (lane / 16 == h) {
#pragma unroll
          for (int i = 0; i < 32; ++i) sts_u32(mine + (lane % 16) * 132 + 4 * i, __float_as_uint(v[i]));
        }
        __syncwarp();
        const int rows = min(16, p.M - m_warp - 16 * h);
        if (lane < left) {
#pragma unroll 8
          for (int r = 0; r < rows; ++r) out[(16 * h + r) * e.ldp] = lds_f32(mine + r * 132 + 4 * lane);
        }
        __syncwarp();
      }
    };
    const bool vec_r = e.ldr % 8 == 0 && reinterpret_cast<uintptr_t>(e.residual) % 16 == 0;
    const int chunks = out_cols / 32, per_warp = (chunks + kParts - 1) / kParts;
    const int c0 = half * per_warp, c1 = min(c0 + per_warp, chunks);
    const int raw0 = half * (nt / 32 / kParts), raw1 = kParts == 1 || half ? nt / 32 : raw0 + nt / 32 / kParts;
    int tile_it = 0;
    for (int u = first; u < p.units; u += step, ++tile_it) {
      const Tile t = tile_of(p, u);
      const int buf = tile_it & 1;
      const int m_warp = t.m * (128 * CG) + static_cast<int>(rank) * 128 + quarter * 32;
      const int m = m_warp + lane, n_tile = t.n * out_cols;
      // pieces that exist: this warp's rows, and columns below N
      const int c_end = t.slot < 0 && m_warp < p.M ? min(c1, (p.N - n_tile + 31) / 32) : c0;
      // Short sums: g and u come into L2 under the tile's MMAs (679 terms: 141 -> 112 us at 2603 x 8966; sums of 4096
      // terms hide the loads anyway, and took 536 instead of 511 us at 8192 x 12288).
      if (MODE == EPI_GATED_BWD && p.kb_total <= 32) {
        const long long at = static_cast<long long>(min(m, p.M - 1)) * e.ldp + n_tile;
        for (int c = c0; c < c_end; ++c) {
          prefetch_l2(e.pre + at + 32 * c);
          prefetch_l2(e.pre2 + at + 32 * c);
        }
      }
      if (MODE == EPI_LINEAR && e.bias) {  // 16-bit, four columns a lane
        const uint16_t* h = static_cast<const uint16_t*>(e.bias);
        const int at = n_tile + 32 * c0 + 4 * lane;
        uint16_t b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) b[i] = at + i < p.N ? h[at + i] : static_cast<uint16_t>(0);
        sts_u32(mine + kBufBytes + 8 * lane, pack2(b[0], b[1]));
        sts_u32(mine + kBufBytes + 8 * lane + 4, pack2(b[2], b[3]));
        __syncwarp();
      }
      uint32_t res[16];
      const T* res_row = static_cast<const T*>(e.residual) + static_cast<long long>(m) * e.ldr + n_tile;
      auto fetch_residual = [&](int c) {
        load_row32(res_row + 32 * c, vec_r, m < p.M && c < c_end ? p.N - n_tile - 32 * c : 0, res);
      };
      if (MODE == EPI_LINEAR && e.residual) fetch_residual(c0);
      if (!warp_wait(p.err, acc_full(buf), (tile_it >> 1) & 1, &abort_flag, 8u, false, 128,
                      kWaitNs + 1000ull * p.kb_total)) {  // a stage takes below a microsecond
        break;
      }
      __syncwarp();
      tc_fence_after();
      const uint32_t acc = tmem + buf * NT + (static_cast<uint32_t>(quarter * 32) << 16);
      if (t.slot >= 0 && m_warp < p.M) {  // a k range: its sums as they are
        const int row = t.slot * (128 * CG) + static_cast<int>(rank) * 128 + quarter * 32;
#pragma unroll 1
        for (int c = raw0; c < raw1; ++c) {
          float v[32];
          tmem_ld32(acc + 32 * c, v);
          tmem_arrived(v);
          store_row32<4>(reinterpret_cast<uint8_t*>(p.part + static_cast<long long>(row + lane) * nt + 32 * c),
                         reinterpret_cast<const uint32_t(&)[32]>(v), 32, 32);
        }
      }
#pragma unroll 1
      for (int c = c0; c < c_end; ++c) {
        const int n = n_tile + 32 * c, left = p.N - n;
        float v[32];
        uint32_t w[16];
        tmem_ld32(acc + 32 * c, v);
        if constexpr (MODE == EPI_GATED) {
          float g[32];
          tmem_ld32(acc + nt / 2 + 32 * c, g);
          tmem_arrived(v);
          tmem_arrived(g);
          if (e.pre) {
            put32(v, e.pre, n, left, m_warp);
            put32(g, e.pre2, n, left, m_warp);
          }
          dense_activate<true, 32>(v, e.act, e.alpha, e.beta);
#pragma unroll
          for (int i = 0; i < 16; ++i) w[i] = pack_pair<T>(v[2 * i] * g[2 * i], v[2 * i + 1] * g[2 * i + 1]);
          put16(w, static_cast<T*>(e.y), n, left, m_warp);
        } else if constexpr (MODE == EPI_GATED_BWD) {
          // the library's own rows: a multiple of 64 long, so 8 values that begin below N exist
          float g[32], u[32], slope[32];
          const long long at = static_cast<long long>(min(m, p.M - 1)) * e.ldp + n;
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (8 * j < left) {
              load_32b(e.pre + at + 8 * j, reinterpret_cast<uint32_t*>(g) + 8 * j);
              load_32b(e.pre2 + at + 8 * j, reinterpret_cast<uint32_t*>(u) + 8 * j);
            } else {
#pragma unroll
              for (int i = 0; i < 8; ++i) g[8 * j + i] = u[8 * j + i] = 0.0f;
            }
          dense_activate_grad<true, 32>(g, slope, e.act, e.alpha, e.beta);
          tmem_arrived(v);
#pragma unroll
          for (int i = 0; i < 16; ++i)
            w[i] = pack_pair<T>(v[2 * i] * u[2 * i] * slope[2 * i], v[2 * i + 1] * u[2 * i + 1] * slope[2 * i + 1]);
          put16(w, static_cast<T*>(e.y), n, left, m_warp);
#pragma unroll
          for (int i = 0; i < 16; ++i) w[i] = pack_pair<T>(v[2 * i] * g[2 * i], v[2 * i + 1] * g[2 * i + 1]);
          put16(w, static_cast<T*>(e.y2), n, left, m_warp);
        } else {
          uint32_t bias[16];
          if (e.bias) {
#pragma unroll
            for (int i = 0; i < 4; ++i) lds_v4(mine + kBufBytes + 64 * (c - c0) + 16 * i, bias + 4 * i);
          }
          tmem_arrived(v);
          if (e.bias) add_row32<T>(v, bias);
          if (e.residual && !e.residual_last) {
            add_row32<T>(v, res);
            fetch_residual(c + 1);
          }
          if (e.pre) put32(v, e.pre, n, left, m_warp);
          dense_activate<true, 32>(v, e.act, e.alpha, e.beta);
          if (e.residual && e.residual_last) {
            add_row32<T>(v, res);
            fetch_residual(c + 1);
          }
#pragma unroll
          for (int i = 0; i < 16; ++i) w[i] = pack_pair<T>(v[2 * i], v[2 * i + 1]);
          put16(w, static_cast<T*>(t.batch ? e.y2 : e.y), n, left, m_warp);
        }
      }
      // the accumulator has been read: the next but one tile may have it
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if constexpr (CG == 2) mbar_arrive_cluster(map_rank(acc_empty(buf), 0));
        else mbar_arrive(acc_empty(buf));
      }
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

}  // namespace dtc
}  // namespace conv
