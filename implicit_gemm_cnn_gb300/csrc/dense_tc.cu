// dense_tc.cu -- the tensor-core product's host side: tile choice, tensor maps,
// launch, and the error word of its bounded waits.
#include <string.h>

#include <algorithm>
#include <mutex>

#include <cudaTypedefs.h>

#include "dense_tc.cuh"

namespace conv {

cudaError_t launch_dense_tc_f16(const DenseTcPlan& t, int mode, int a_mn, int b_mn, const DenseTcArgs& args,
                                const DenseTcMaps& maps, cudaStream_t s);
cudaError_t launch_dense_tc_bf16(const DenseTcPlan& t, int mode, int a_mn, int b_mn, const DenseTcArgs& args,
                                 const DenseTcMaps& maps, cudaStream_t s);

cudaError_t launch_dense_tc32(int mode, int a_mn, int b_mn, const DenseTcArgs& args, const DenseTcMaps& maps, int blocks,
                              cudaStream_t s);

namespace {

__device__ uint32_t g_dense_err;

// The driver's tensor-map encoder, looked up once.
PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    else
      cudaGetLastError();
  });
  return fn;
}
// The error word's address on the current device, looked up once per device.
uint32_t* error_word() {
  static std::mutex mu;
  static uint32_t* at[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
    cudaGetLastError();
    return nullptr;
  }
  std::lock_guard<std::mutex> lock(mu);
  if (!at[dev]) {
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, g_dense_err) != cudaSuccess) {
      cudaGetLastError();
      return nullptr;
    }
    at[dev] = static_cast<uint32_t*>(p);
  }
  return at[dev];
}

// A row-major matrix as a tensor map with boxes of 128 bytes of a row x box_rows rows, swizzled over as many bytes, zeros
// outside.
bool encode(CUtensorMap* map, CUtensorMapDataType type, const void* base, long long inner, long long rows, long long ld,
            int box_rows) {
  const size_t es = type == CU_TENSOR_MAP_DATA_TYPE_FLOAT32 ? 4 : 2;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(inner), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld) * es};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(128 / es), static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t step[2] = {1, 1};
  return encoder()(map, type, 2, const_cast<void*>(base), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                   CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// An mn-major operand's matrix (rows of `inner` values, existing to a multiple of 64) as a map of 64-wide column blocks:
// one copy brings `blocks` of them, one after another.
bool encode_blocks(CUtensorMap* map, CUtensorMapDataType type, const void* base, long long inner, long long rows,
                   long long ld, int blocks) {
  const cuuint64_t dims[3] = {64, static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>((inner + 63) / 64)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(ld) * 2, 128};
  const cuuint32_t box[3] = {64, 64, static_cast<cuuint32_t>(blocks)};
  const cuuint32_t step[3] = {1, 1, 1};
  return encoder()(map, type, 3, const_cast<void*>(base), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                   CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// Three bfloat16 planes of a matrix (rows * ld elements apart), boxes of 64 x box_rows of all three.
bool encode_planes(CUtensorMap* map, const void* base, long long inner, long long rows, long long ld, int box_rows) {
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(inner), static_cast<cuuint64_t>(rows), 3};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(ld) * 2, static_cast<cuuint64_t>(ld) * 2 * rows};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_rows), 3};
  const cuuint32_t step[3] = {1, 1, 1};
  return encoder()(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, step,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The tile and the k ranges of least time by this model, in clocks, fitted to full waves of 4096-term sums (bfloat16,
// 1.85 GHz): 64 terms of a pair's tile take 165 + 1.73 nt (608 at nt = 256, 386 at 128: 512 and 256 are the MMAs
// alone), of one SM's 190 + 1.76 nt (415 at 128: its stage is as many bytes as the pair's of 256); a tile adds 600, a
// launch 6000.  Tiles run in rounds of one per block.  The last round, if it is not full, may be cut into k ranges, so
// that it takes a part of a round's time; their sums pass through L2 twice, at some 4000 bytes a clock, and cost a launch.
// float32 (dense_tc32.cu): one SM's tiles of 64 or 128 columns, six products; a stage of 64 terms takes 13 nt clocks, or
// the 1000 of its copies and hand-overs.
DenseTcPlan search(const DenseGemm& g, int f32, int sm) {
  DenseTcPlan best = {};
  const int kb = static_cast<int>((static_cast<long long>(g.K) + dtc::kBK - 1) / dtc::kBK) * g.segs;
  double best_t = 0.0;
  for (int cg = f32 ? 1 : 2; cg >= 1; --cg) {
    const long long slots = sm / cg;
    if (slots < 1) continue;  // (one SM has no pair)
    for (int nt = cg == 2 ? 256 : 128; nt >= 64; nt -= 32) {
      if ((g.dual || f32) && nt % 64) continue;
      if (g.b_mn && nt / cg % 64) continue;  // copied in blocks of 64 columns: other widths would load more than they use
      const int cols = g.dual ? nt / 2 : nt;
      const long long tiles = ((g.M + 128LL * cg - 1) / (128 * cg)) * ((static_cast<long long>(g.N) + cols - 1) / cols) * g.batch;
      const double per = f32 ? std::max(13.0 * nt, 1000.0) : cg == 2 ? 165.0 + 1.73 * nt : 190.0 + 1.76 * nt;
      const long long rest = tiles % slots;
      for (int split = 1; split <= 16; ++split) {
        if (split > 1 && (kb / split < 4 || rest == 0)) break;
        const int range = (kb + split - 1) / split;
        if ((kb + range - 1) / range != split) continue;  // every range holds terms
        const long long whole = split > 1 ? tiles - rest : tiles, ranges = (tiles - whole) * split;
        if (split > 1 && ranges > 2 * slots) break;
        const double bytes = split > 1 ? static_cast<double>(ranges) * 128 * cg * nt * 4 : 0.0;
        double t = static_cast<double>((whole + slots - 1) / slots) * (kb * per + 600.0) + 6000.0;
        if (split > 1)
          t += static_cast<double>((ranges + slots - 1) / slots) * (range * per + 600.0) + 4000.0 + 2.0 * bytes / 4000.0;
        if (!best.cg || t < best_t) {
          best_t = t;
          best.cg = cg; best.nt = nt; best.split = split; best.kb_range = range;
          best.tiles = static_cast<int>(tiles);
          best.whole = static_cast<int>(whole);
          best.blocks = static_cast<int>(std::min(whole + ranges, slots)) * cg;
          best.part_bytes = static_cast<size_t>(bytes);
        }
      }
    }
  }
  return best;
}

// Adds the k ranges' sums of the tiles that were cut, in order, and runs their epilogue: four columns per thread (28 tiles
// of 256 x 256 in two ranges: 10 us, where a fourth round of whole tiles would be 20).
template <typename T>
__global__ void __launch_bounds__(256) dense_join(const __grid_constant__ DenseTcArgs p, const float* part, int tile_rows,
                                                  int dual) {
  griddep_wait();
  griddep_launch();
  const int out_cols = dual ? p.nt / 2 : p.nt, quads = out_cols / 4;
  const long long per = static_cast<long long>(tile_rows) * quads;
  const long long i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
  const int q = static_cast<int>(i / per);
  if (p.whole + static_cast<long long>(q) * p.split >= p.units) return;
  const int at = static_cast<int>(i - q * per), row = at / quads, c = at % quads * 4;
  const dtc::Tile t = dtc::tile_of(p, p.whole + q * p.split);
  const int m = t.m * tile_rows + row, n = t.n * out_cols + c;
  if (m >= p.M || n >= p.N) return;
  const long long tile = static_cast<long long>(tile_rows) * p.nt;
  const float* src = part + (static_cast<long long>(q) * p.split * tile_rows + row) * p.nt + c;
  float v[4] = {0.0f, 0.0f, 0.0f, 0.0f}, u[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
  for (int s = 0; s < p.split; ++s) {
    const float4 f = *reinterpret_cast<const float4*>(src + s * tile);
    v[0] += f.x; v[1] += f.y; v[2] += f.z; v[3] += f.w;
    if (dual) {
      const float4 h = *reinterpret_cast<const float4*>(src + s * tile + p.nt / 2);
      u[0] += h.x; u[1] += h.y; u[2] += h.z; u[3] += h.w;
    }
  }
  int col[4];
  bool ok[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    col[j] = n + j;
    ok[j] = n + j < p.N;
  }
  dense_epilogue<T, 4>(p.epi, t.batch, m, col, ok, v, u);
}

// The plans of the shapes used last (a search takes microseconds, a small product too).
struct PlanKey {
  int M, N, K, segs, batch, dual, b_mn, f32, sm;
  bool operator==(const PlanKey& o) const {
    return M == o.M && N == o.N && K == o.K && segs == o.segs && batch == o.batch && dual == o.dual &&
           b_mn == o.b_mn && f32 == o.f32 && sm == o.sm;
  }
};
std::mutex g_plan_mu;
struct {
  PlanKey key;
  DenseTcPlan plan;
} g_plans[256];

}  // namespace

DenseTcPlan dense_tc_plan(const DenseGemm& g, int dtype, int sm) {
  const int f32 = dtype == CONV_F32;
  const PlanKey key{g.M, g.N, g.K, g.segs, g.batch, g.dual, g.b_mn, f32, sm};
  uint32_t h = 2166136261u;
  for (int v : {key.M, key.N, key.K, key.segs, key.batch, key.dual, key.b_mn, key.f32}) h = (h ^ static_cast<uint32_t>(v)) * 16777619u;
  auto& slot = g_plans[(h ^ (h >> 15)) % 256];
  {
    std::lock_guard<std::mutex> lock(g_plan_mu);
    if (slot.key == key) return slot.plan;  // (an empty slot's sm is 0)
  }
  const DenseTcPlan plan = search(g, f32, sm);
  std::lock_guard<std::mutex> lock(g_plan_mu);
  slot.key = key;
  slot.plan = plan;
  return plan;
}

cudaError_t launch_dense_tc(const DenseTcPlan& t, const DenseGemm& g, int dtype, void* part, cudaStream_t s) {
  if (!encoder()) return cudaErrorNotSupported;
  DenseTcArgs p;
  DenseTcMaps maps;
  memset(&p, 0, sizeof(p));
  memset(&maps, 0, sizeof(maps));
  p.M = g.M; p.N = g.N;
  p.segs = g.segs; p.batch = g.batch;
  p.nt = t.nt;
  p.kb_seg = static_cast<int>((static_cast<long long>(g.K) + dtc::kBK - 1) / dtc::kBK);
  p.kb_total = p.kb_seg * g.segs;
  p.kb_range = t.kb_range;
  p.split = t.split;
  const int cols = g.dual ? t.nt / 2 : t.nt;
  p.mtiles = static_cast<int>((g.M + 128LL * t.cg - 1) / (128 * t.cg));
  p.ntiles = static_cast<int>((static_cast<long long>(g.N) + cols - 1) / cols);
  p.whole = t.whole;
  p.units = t.whole + (t.tiles - t.whole) * t.split;
  p.group = 16;  // 8 to 19 rows of tiles measured alike, 1 and 32 some 5% slower
  p.epi = g.epi;
  p.err = error_word();
  if (!p.err) return cudaErrorNotSupported;
  const bool f32 = dtype == CONV_F32;
  const CUtensorMapDataType type = dtype == CONV_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const int b_rows = g.dual && t.cg == 1 ? t.nt / 2 : t.nt / t.cg;
  const int as = std::max(g.segs, g.batch), bs = g.segs > 1 || g.batch > 1 || g.dual ? 2 : 1;
  p.a_rows = f32 ? 128 : std::min(128, (g.M + 7) / 8 * 8);
  // one copy per operand and stage where the blocks of 64 divide the matrix and the block's share of the tile
  p.a_3d = g.a_mn && (g.M % 64 == 0 || g.a_pad) && !f32;
  p.b_3d = g.b_mn && (g.N % 64 == 0 || g.b_pad) && b_rows % 64 == 0 && !f32;
  bool ok = true;
  auto operand = [&](CUtensorMap* map, const void* base, int mn, bool blocks, long long rows, long long ld, int box_rows,
                     int box_blocks) {
    if (f32)
      return mn ? encode_planes(map, base, rows, g.K, ld, 64) : encode_planes(map, base, g.K, rows, ld, box_rows);
    if (blocks) return encode_blocks(map, type, base, rows, g.K, ld, box_blocks);
    return mn ? encode(map, type, base, rows, g.K, ld, 64) : encode(map, type, base, g.K, rows, ld, box_rows);
  };
  for (int i = 0; i < as; ++i) ok = ok && operand(&maps.a[i], g.a[i], g.a_mn, p.a_3d, g.M, g.lda, p.a_rows, 2);
  for (int i = 0; i < bs; ++i) ok = ok && operand(&maps.b[i], g.b[i], g.b_mn, p.b_3d, g.N, g.ldb, b_rows, b_rows / 64);
  const int mode = g.epi.mode;
  const int tile_rows = 128 * t.cg, cut = t.tiles - t.whole;
  const bool two = mode == EPI_GATED_BWD || g.batch > 1, saves = mode != EPI_GATED_BWD && g.epi.pre;
  const int es = f32 ? 4 : 2;
  auto align = [](const void* a, const void* b, long long row_bytes) {
    const uintptr_t all = reinterpret_cast<uintptr_t>(a) | reinterpret_cast<uintptr_t>(b) | static_cast<uintptr_t>(row_bytes);
    return all % 32 == 0 ? 32 : all % 16 == 0 ? 16 : 0;
  };
  p.align_y = align(g.epi.y, two ? g.epi.y2 : nullptr, g.epi.ldy * es);
  p.align_pre = align(g.epi.pre, mode == EPI_LINEAR ? nullptr : g.epi.pre2, g.epi.ldp * 4);
  if (mode == EPI_GATED_BWD && (p.align_pre != 32 || !p.align_y)) return cudaErrorInvalidValue;  // the library's own layout
  p.part = static_cast<float*>(part);
  if (f32) {
    auto out = [&](CUtensorMap* map, const void* base, long long cols, long long rows, long long ld) {
      return encode(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, base, cols, rows, ld, 32);
    };
    if (cut > 0) ok = ok && out(&maps.part, part, t.nt, static_cast<long long>(cut) * t.split * tile_rows, t.nt);
    if (p.align_y) {
      ok = ok && out(&maps.y[0], g.epi.y, g.N, g.M, g.epi.ldy);
      if (two) ok = ok && out(&maps.y[1], g.epi.y2, g.N, g.M, g.epi.ldy);
    }
    if (saves && p.align_pre) {
      ok = ok && out(&maps.pre[0], g.epi.pre, g.N, g.M, g.epi.ldp);
      if (mode == EPI_GATED) ok = ok && out(&maps.pre[1], g.epi.pre2, g.N, g.M, g.epi.ldp);
    }
  }
  if (!ok) return cudaErrorInvalidValue;
  const cudaError_t err = f32 ? launch_dense_tc32(mode, g.a_mn, g.b_mn, p, maps, t.blocks, s)
                          : dtype == CONV_F16 ? launch_dense_tc_f16(t, mode, g.a_mn, g.b_mn, p, maps, s)
                                              : launch_dense_tc_bf16(t, mode, g.a_mn, g.b_mn, p, maps, s);
  if (err != cudaSuccess || cut == 0) return err;
  const long long threads = static_cast<long long>(cut) * tile_rows * (cols / 4);
  const dim3 grid(static_cast<unsigned>((threads + 255) / 256));
  auto join = f32 ? dense_join<float> : dtype == CONV_F16 ? dense_join<__half> : dense_join<__nv_bfloat16>;
  return launch_overlapped(join, grid, 256, 0, 1, s, p, static_cast<const float*>(part), tile_rows, g.dual);
}

cudaError_t dense_error_word(uint32_t* word, int reset) {
  cudaError_t err = cudaDeviceSynchronize();
  if (err != cudaSuccess) return err;
  err = cudaMemcpyFromSymbol(word, g_dense_err, sizeof(uint32_t));
  if (err != cudaSuccess || !reset) return err;
  const uint32_t zero = 0;
  return cudaMemcpyToSymbol(g_dense_err, &zero, sizeof(uint32_t));
}

}  // namespace conv
