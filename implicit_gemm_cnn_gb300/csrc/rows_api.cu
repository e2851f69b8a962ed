// rows_api.cu -- the C ABI of the row operators (rows.h): validation, planning
// and dispatch.  Everything here runs on the host; a call only enqueues.
#include <math.h>
#include <stdio.h>
#include <string.h>

#include <algorithm>

#include "dense_host.h"
#include "rows_internal.h"

using namespace conv;

namespace {

conv_status rows_ok(int64_t rows, int64_t width) {
  return rows < 0 || width < 1 || rows > kI32 - 65536 || width > kI32 - 65536 ? CONV_ERR_SHAPE : CONV_OK;
}
bool type_ok(int dtype) { return dtype >= CONV_F32 && dtype <= CONV_BF16; }

// ---- layer norm ---------------------------------------------------------------
struct NormShape {
  long long ldx, ldy;
};
conv_status validate(const conv_norm_problem* p, NormShape* s) {
  if (!p) return CONV_ERR_NULL;
  if (!type_ok(p->dtype)) return CONV_ERR_DTYPE;
  if ((p->flags & ~CONV_NORM_FLAG_STREAM) || !(p->eps >= 0.0f) || isinf(p->eps)) return CONV_ERR_ARG;
  if (rows_ok(p->rows, p->width) != CONV_OK || !stride_of(p->x_stride, p->width, &s->ldx) ||
      !stride_of(p->y_stride, p->width, &s->ldy))
    return CONV_ERR_SHAPE;
  return elems_ok(p->rows, s->ldx) && elems_ok(p->rows, s->ldy) ? CONV_OK : CONV_ERR_OVERFLOW;
}
bool norm_streams(const conv_norm_problem* p) { return (p->flags & CONV_NORM_FLAG_STREAM) != 0; }
size_t norm_scratch(const conv_norm_problem* p, int sm) {
  return p->rows == 0 ? 0 : align256(norm_backward_scratch(p->rows, p->width, static_cast<int>(elem_size(p->dtype)), norm_streams(p), sm));
}

// ---- dropout ------------------------------------------------------------------
struct DropoutShape {
  long long ldx, ldr, ldy;
};
conv_status validate(const conv_dropout_problem* p, DropoutShape* s) {
  if (!p) return CONV_ERR_NULL;
  if (!type_ok(p->dtype)) return CONV_ERR_DTYPE;
  if (p->flags || !(p->p >= 0.0 && p->p <= 1.0)) return CONV_ERR_ARG;
  if (rows_ok(p->rows, p->width) != CONV_OK || !stride_of(p->x_stride, p->width, &s->ldx) ||
      !stride_of(p->residual_stride, p->width, &s->ldr) || !stride_of(p->y_stride, p->width, &s->ldy))
    return CONV_ERR_SHAPE;
  return elems_ok(p->rows, s->ldx) && elems_ok(p->rows, s->ldy) && (!p->has_residual || elems_ok(p->rows, s->ldr)) ? CONV_OK
                                                                                                                    : CONV_ERR_OVERFLOW;
}
conv_status enqueue_dropout(const conv_dropout_problem* p, const void* x, long long ldx, const void* residual, long long ldr, void* y,
                            long long ldy, const uint64_t* state, void* stream) {
  if (p->rows == 0) return CONV_OK;
  if (!x || !y || (p->has_residual && !residual)) return CONV_ERR_NULL;
  const size_t es = elem_size(p->dtype), width = p->width * es;
  if (!p->has_residual) residual = nullptr;
  Ranges ranges;
  ranges.add_in(x, p->rows, width, ldx * es);
  ranges.add_in(residual, p->rows, width, ldr * es);
  ranges.add_in(state, 16);
  ranges.add_out(y, p->rows, width, ldy * es);
  if (ranges.clash()) return CONV_ERR_ALIAS;
  if (misplaced(es, {x, residual, y}) || misplaced(8, {state})) return CONV_ERR_ARG;
  int dev, sm;
  const conv_status st = current_device(&dev, &sm);
  if (st != CONV_OK) return st;
  DropoutArgs a = {};
  a.x = x; a.residual = residual; a.y = y;
  a.rows = p->rows; a.width = p->width;
  a.ldx = ldx; a.ldr = ldr; a.ldy = ldy;
  a.seed = p->seed; a.offset = p->offset; a.state = state;
  a.drop = static_cast<uint32_t>(lrint(p->p * 65536.0));
  CONV_TRY(launch_dropout(a, p->dtype, sm, static_cast<cudaStream_t>(stream)));
  return CONV_OK;
}

// ---- 8 bits -------------------------------------------------------------------
conv_status validate(const conv_quantize_problem* p, long long* ldx, long long* ldq) {
  if (!p) return CONV_ERR_NULL;
  if (!type_ok(p->dtype)) return CONV_ERR_DTYPE;
  if (p->flags) return CONV_ERR_ARG;
  if (rows_ok(p->rows, p->width) != CONV_OK || !stride_of(p->x_stride, p->width, ldx) || !stride_of(p->q_stride, p->width, ldq))
    return CONV_ERR_SHAPE;
  return elems_ok(p->rows, *ldx) && elems_ok(p->rows, *ldq) ? CONV_OK : CONV_ERR_OVERFLOW;
}

constexpr long long kMaxTerms = 131071;  // 2^14 each: the sum stays below 2^31
constexpr uint32_t kInt8Flags = CONV_LINEAR_FLAG_RESIDUAL_LAST | CONV_INT8_FLAG_FEW | CONV_INT8_FLAG_MID | CONV_INT8_FLAG_MANY;

struct Int8Shape {
  long long ldx, ldw, ldr, ldy;
};
conv_status validate(const conv_int8_problem* p, Int8Shape* s) {
  if (!p) return CONV_ERR_NULL;
  if (!type_ok(p->dtype)) return CONV_ERR_DTYPE;
  if (p->act < CONV_ACT_IDENTITY || p->act > CONV_ACT_GELU_TANH) return CONV_ERR_ACT;
  if (p->flags & ~kInt8Flags) return CONV_ERR_ARG;
  if (rows_ok(p->rows, p->c_in) != CONV_OK || rows_ok(p->c_out, p->c_out) != CONV_OK || p->c_in > kMaxTerms) return CONV_ERR_SHAPE;
  if (!stride_of(p->x_stride, p->c_in, &s->ldx) || !stride_of(p->w_stride, p->c_in, &s->ldw) ||
      !stride_of(p->residual_stride, p->c_out, &s->ldr) || !stride_of(p->y_stride, p->c_out, &s->ldy))
    return CONV_ERR_SHAPE;
  return elems_ok(p->rows, s->ldx) && elems_ok(p->c_out, s->ldw) && elems_ok(p->rows, s->ldy) &&
                 (!p->has_residual || elems_ok(p->rows, s->ldr))
             ? CONV_OK
             : CONV_ERR_OVERFLOW;
}

// Which kernel: the weights straight into registers (few rows), through shared memory (mid), or as halves first (many).
// The second takes weights in rows on 16-byte boundaries only (TMA).  The first works on 32 rows and 16 outputs at a time, two
// blocks an SM.  From 17 rows on the choice goes by what these take (fitted to the measurements): the first, in r rounds of such
// blocks, 0.6 + 1.5 r (k + 1) us for k times 1024 terms, the second 9.2 + 0.8 k.  The fit ends at 128 rows, a tile of the
// second, and so does the choice: above, small layers would still be quicker without a pass over the weights (x quantised by
// the call, few / mid / many: 129 rows 1024->1024 6.6 / 10.8 / 9.5, 2048->2048 14.3 / 12.9 / 13.3; 256 rows 8.5 / 12.9 / 9.7
// and 21.3 / 15.8 / 13.8).
// Measured (us, few / mid / many):
//              16 rows        32             64             96             128            256
//   1024->1024                                3 /  9 /  9    4 / 11 /  9    4 / 12 /  9
//   8192->1024                               13 / 15 / 16   15 / 19 / 16   15 / 20 / 17
//   2048->2048                                6 / 11 / 13   10 / 12 / 13   10 / 14 / 13
//   4096->2048                                9 / 13 / 15   16 / 14 / 15   17 / 16 / 16
//   2048->4096                               11 / 12 / 14   15 / 13 / 15   19 / 16 / 15
//   2048->8192  8 / 12 / 17   11 / 13 / 17   19 / 13 / 17                   - / 17 / 17    - / 20 / 20
//   4096->6144                17 / 16 / -
//   4096->12288 17 / 20 / 44  26 / 21 / 44   46 / 21 / 44                   - / 29 / 45    - / 53 / 51
// Weights in rows of no whole 16-byte pieces: the first r (3 + 2.9 k), the third 8.5 + 0.5 k + 0.75 for each MB of weights (few
// / many, x quantised by the call):
//   24 rows: 1001->1000 7 / 9, 2003->1024 9 / 13, 8003->1024 24 / 19, 2003->5001 18 / 19, 4003->5001 29 / 25, 4003->12288 42 / 53
//   64 rows: 1001->4001 13 / 14, 2003->2048 11 / 15, 8003->1024 27 / 19, 2003->5001 28 / 19, 4003->12288 78 / 54
//  128 rows: 1001->1000 8 / 12, 503->4001 16 / 12, 2003->2048 18 / 16;   12 rows: 4003->12288 29 / 53, 4003->5001 21 / 25
enum Int8Kernel { I8_FEW, I8_MID, I8_MANY };
constexpr long long kGridMost = 1 << 20;  // rows that the first two have grids for
Int8Kernel int8_kernel(const conv_int8_problem* p, const Int8Shape& sh, bool aligned, int sm) {
  const bool mid = aligned && sh.ldw % 16 == 0 && p->rows <= kGridMost;
  if (p->flags & CONV_INT8_FLAG_FEW && p->rows <= kGridMost) return I8_FEW;
  if (p->flags & CONV_INT8_FLAG_MID && mid) return I8_MID;
  if (p->flags & CONV_INT8_FLAG_MANY) return I8_MANY;
  if (p->rows <= 16) return I8_FEW;
  if (p->rows > 128) return I8_MANY;
  const long long blocks = (p->rows + 31) / 32 * ((p->c_out + 15) / 16), rounds = (blocks + 2LL * sm - 1) / (2LL * sm);
  const double k = p->c_in / 1024.0, mb = static_cast<double>(p->c_in) * static_cast<double>(p->c_out) * 1e-6;
  const double few = mid && p->c_in % 16 == 0 ? 0.6 + 1.5 * rounds * (k + 1.0) : rounds * (3.0 + 2.9 * k);
  const double other = mid ? 9.2 + 0.8 * k : 8.5 + 0.5 * k + 0.75 * mb;
  return few < other ? I8_FEW : mid ? I8_MID : I8_MANY;
}

struct Int8Plan {
  Int8Kernel kernel;
  bool pad;                 // few rows, 8-bit ones: x is copied to rows of whole 16-byte pieces
  Int8MidPlan mid;
  DenseTcPlan tc;
  long long ldq, ldw;       // rows of the quantised x (bytes, or halves), and of the weights as halves
  size_t q_off, scale_off, w_off, part_off, total;
  int launches;
};
// `aligned`: the weights' address is on a 16-byte boundary; `x_aligned`: that of x.
Int8Plan plan_int8(const conv_int8_problem* p, const Int8Shape& sh, bool aligned, bool x_aligned, int sm) {
  Int8Plan r = {};
  if (p->rows == 0) return r;
  auto take = [&](size_t bytes) {
    const size_t at = r.total;
    r.total = align256(at + bytes);
    return at;
  };
  r.kernel = int8_kernel(p, sh, aligned, sm);
  r.launches = 1;
  if (!p->x_quantized) {
    r.scale_off = take(static_cast<size_t>(p->rows) * sizeof(float));
    ++r.launches;
  }
  if (r.kernel == I8_FEW) {
    r.pad = p->x_quantized && !(x_aligned && p->c_in % 16 == 0 && (p->rows == 1 || sh.ldx % 16 == 0));
    r.ldq = p->x_quantized && !r.pad ? sh.ldx : (p->c_in + 15) / 16 * 16;
    if (!p->x_quantized || r.pad) r.q_off = take(static_cast<size_t>(p->rows) * r.ldq);
    if (r.pad) ++r.launches;
    return r;
  }
  r.ldq = r.ldw = (p->c_in + 63) / 64 * 64;  // whole cache lines
  r.q_off = take(static_cast<size_t>(p->rows) * r.ldq * 2);
  if (p->x_quantized) ++r.launches;
  if (r.kernel == I8_MID) {
    r.mid = int8_mid_plan(static_cast<int>(p->rows), static_cast<int>(p->c_out), static_cast<int>(p->c_in), sm);
    return r;
  }
  r.w_off = take(static_cast<size_t>(p->c_out) * r.ldw * 2);
  r.tc = int8_tc_plan(static_cast<int>(p->rows), static_cast<int>(p->c_out), static_cast<int>(p->c_in), sm);
  r.part_off = take(r.tc.part_bytes);
  r.launches += r.tc.split > 1 ? 2 : 1;
  return r;
}

}  // namespace

extern "C" {

conv_status conv_norm_forward(const conv_norm_problem* p, const void* x, const void* weight, const void* bias, void* y,
                              float* stats, void* stream) {
  NormShape sh;
  conv_status st = validate(p, &sh);
  if (st != CONV_OK) return st;
  if (p->rows == 0) return CONV_OK;
  if (!x || !y || (p->has_weight && !weight) || (p->has_bias && !bias)) return CONV_ERR_NULL;
  if (!p->has_weight) weight = nullptr;
  if (!p->has_bias) bias = nullptr;
  const size_t es = elem_size(p->dtype), width = p->width * es;
  Ranges ranges;
  ranges.add_in(x, p->rows, width, sh.ldx * es);
  ranges.add_in(weight, width);
  ranges.add_in(bias, width);
  ranges.add_out(y, p->rows, width, sh.ldy * es);
  ranges.add_out(stats, static_cast<size_t>(p->rows) * 8);
  if (ranges.clash()) return CONV_ERR_ALIAS;
  if (misplaced(es, {x, weight, bias, y}) || misplaced(8, {stats})) return CONV_ERR_ARG;
  int dev, sm;
  st = current_device(&dev, &sm);
  if (st != CONV_OK) return st;
  NormArgs a = {};
  a.x = x; a.w = weight; a.b = bias; a.y = y; a.stats = stats;
  a.rows = p->rows; a.width = p->width; a.ldx = sh.ldx; a.ldy = sh.ldy;
  a.eps = p->eps;
  CONV_TRY(launch_norm_forward(a, p->dtype, norm_streams(p), sm, static_cast<cudaStream_t>(stream)));
  return CONV_OK;
}

conv_status conv_norm_backward_scratch_bytes(const conv_norm_problem* p, size_t* bytes) {
  if (!bytes) return CONV_ERR_NULL;
  NormShape sh;
  conv_status st = validate(p, &sh);
  int dev, sm;
  if (st == CONV_OK) st = current_device(&dev, &sm);
  if (st == CONV_OK) *bytes = norm_scratch(p, sm);
  return st;
}

conv_status conv_norm_backward(const conv_norm_problem* p, const void* x, const void* weight, const float* stats, const void* dy,
                               void* dx, void* dweight, void* dbias, void* scratch, size_t scratch_bytes, void* stream) {
  NormShape sh;
  conv_status st = validate(p, &sh);
  if (st != CONV_OK) return st;
  const size_t es = elem_size(p->dtype), width = p->width * es;
  const bool sums = dweight || dbias;
  if (!p->has_weight || !dx) weight = nullptr;
  if (p->rows > 0 && (dx || sums) && (!x || !stats || !dy || (dx && p->has_weight && !weight))) return CONV_ERR_NULL;
  Ranges ranges;
  if (p->rows > 0) {
    ranges.add_in(x, p->rows, width, sh.ldx * es);
    ranges.add_in(weight, width);
    ranges.add_in(stats, static_cast<size_t>(p->rows) * 8);
    ranges.add_in(dy, p->rows, width, sh.ldy * es);
  }
  ranges.add_out(dx, p->rows * width);
  ranges.add_out(dweight, width);
  ranges.add_out(dbias, width);
  if (ranges.clash()) return CONV_ERR_ALIAS;
  if (misplaced(es, {x, weight, dy, dx, dweight, dbias}) || misplaced(8, {stats})) return CONV_ERR_ARG;
  int dev, sm;
  st = current_device(&dev, &sm);
  if (st != CONV_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (p->rows == 0) {
    if (dweight) CONV_TRY(cudaMemsetAsync(dweight, 0, width, s));
    if (dbias) CONV_TRY(cudaMemsetAsync(dbias, 0, width, s));
    return CONV_OK;
  }
  const size_t need = sums ? norm_scratch(p, sm) : 0;
  if (scratch_bad(scratch, scratch_bytes, need)) return CONV_ERR_SCRATCH;
  ranges.add_out(need ? scratch : nullptr, need);
  if (ranges.clash()) return CONV_ERR_ALIAS;
  NormArgs a = {};
  a.x = x; a.w = weight; a.dy = dy; a.dx = dx; a.dw = dweight; a.db = dbias;
  a.stats = const_cast<float*>(stats);
  a.part = static_cast<float*>(scratch);
  a.rows = p->rows; a.width = p->width; a.ldx = sh.ldx; a.ldy = sh.ldy;
  a.eps = p->eps;
  CONV_TRY(launch_norm_backward(a, p->dtype, norm_streams(p), sm, s));
  return CONV_OK;
}

conv_status conv_dropout_forward(const conv_dropout_problem* p, const void* x, const void* residual, void* y,
                                 const uint64_t* state, void* stream) {
  DropoutShape sh;
  const conv_status st = validate(p, &sh);
  if (st != CONV_OK) return st;
  return enqueue_dropout(p, x, sh.ldx, residual, sh.ldr, y, sh.ldy, state, stream);
}

conv_status conv_dropout_backward(const conv_dropout_problem* p, const void* dy, void* dx, const uint64_t* state, void* stream) {
  DropoutShape sh;
  const conv_status st = validate(p, &sh);
  if (st != CONV_OK) return st;
  conv_dropout_problem q = *p;
  q.has_residual = 0;
  return enqueue_dropout(&q, dy, sh.ldy, nullptr, 0, dx, sh.ldx, state, stream);
}

conv_status conv_quantize_rows(const conv_quantize_problem* p, const void* x, int8_t* q, float* scale, void* stream) {
  long long ldx, ldq;
  conv_status st = validate(p, &ldx, &ldq);
  if (st != CONV_OK) return st;
  if (p->rows == 0) return CONV_OK;
  if (!x || !q || !scale) return CONV_ERR_NULL;
  const size_t es = elem_size(p->dtype);
  Ranges ranges;
  ranges.add_in(x, p->rows, p->width * es, ldx * es);
  ranges.add_out(q, p->rows, p->width, ldq);
  ranges.add_out(scale, static_cast<size_t>(p->rows) * 4);
  if (ranges.clash()) return CONV_ERR_ALIAS;
  if (misplaced(es, {x}) || misplaced(4, {scale})) return CONV_ERR_ARG;
  int dev, sm;
  st = current_device(&dev, &sm);
  if (st != CONV_OK) return st;
  CONV_TRY(launch_quantize({x, q, scale, p->rows, p->width, ldx, ldq}, p->dtype, false, sm, static_cast<cudaStream_t>(stream)));
  return CONV_OK;
}

conv_status conv_int8_scratch_bytes(const conv_int8_problem* p, size_t* bytes) {
  if (!bytes) return CONV_ERR_NULL;
  Int8Shape sh;
  conv_status st = validate(p, &sh);
  int dev, sm;
  if (st == CONV_OK) st = current_device(&dev, &sm);
  if (st != CONV_OK) return st;
  // (addresses are not known: the most of all.  Weights off 16-byte boundaries may need halves where others do not.)
  *bytes = 0;
  for (int i = 0; i < 4; ++i) *bytes = std::max(*bytes, plan_int8(p, sh, i & 1, i & 2, sm).total);
  return CONV_OK;
}

conv_status conv_int8_describe_plan(const conv_int8_problem* p, int32_t sm_count, char* buf, size_t len) {
  if (!buf || !len) return CONV_ERR_NULL;
  if (sm_count < 1) return CONV_ERR_ARG;
  Int8Shape sh;
  const conv_status st = validate(p, &sh);
  if (st != CONV_OK) return st;
  const Int8Plan r = plan_int8(p, sh, true, true, sm_count);
  if (p->rows == 0) snprintf(buf, len, "nothing launches=0");
  else if (r.kernel == I8_MID)
    snprintf(buf, len, "tcgen05_f16_stream tile=128x%d tiles=%dx%d cluster=%d sums over %lld sms=%d launches=%d", r.mid.nt, r.mid.tiles,
             r.mid.row_tiles, r.mid.split, static_cast<long long>(p->c_in), sm_count, r.launches);
  else if (r.kernel == I8_FEW) snprintf(buf, len, "few_rows sums over %lld sms=%d launches=%d", static_cast<long long>(p->c_in), sm_count, r.launches);
  else
    snprintf(buf, len, "tcgen05_f16 tile=%dx%d sms_per_tile=%d tiles=%d whole=%d split=%d sums over %lld sms=%d launches=%d", 128 * r.tc.cg,
             r.tc.nt, r.tc.cg, r.tc.tiles, r.tc.whole, r.tc.split, static_cast<long long>(p->c_in), sm_count, r.launches);
  return CONV_OK;
}

conv_status conv_int8_forward(const conv_int8_problem* p, const void* x, const float* x_scale, const int8_t* w,
                              const float* w_scale, const void* bias, const void* residual, void* y, void* scratch,
                              size_t scratch_bytes, void* stream) {
  Int8Shape sh;
  conv_status st = validate(p, &sh);
  if (st != CONV_OK) return st;
  if (p->rows == 0) return CONV_OK;
  if (!x || (p->x_quantized && !x_scale) || !w || !w_scale || !y || (p->has_bias && !bias) || (p->has_residual && !residual))
    return CONV_ERR_NULL;
  if (!p->x_quantized) x_scale = nullptr;
  if (!p->has_bias) bias = nullptr;
  if (!p->has_residual) residual = nullptr;
  const size_t es = elem_size(p->dtype), xs = p->x_quantized ? 1 : es;
  Ranges ranges;
  ranges.add_in(x, p->rows, p->c_in * xs, sh.ldx * xs);
  ranges.add_in(x_scale, static_cast<size_t>(p->rows) * 4);
  ranges.add_in(w, p->c_out, p->c_in, sh.ldw);
  ranges.add_in(w_scale, static_cast<size_t>(p->c_out) * 4);
  ranges.add_in(bias, p->c_out * es);
  ranges.add_in(residual, p->rows, p->c_out * es, sh.ldr * es);
  ranges.add_out(y, p->rows, p->c_out * es, sh.ldy * es);
  if (ranges.clash()) return CONV_ERR_ALIAS;
  if (misplaced(xs, {x}) || misplaced(4, {x_scale, w_scale}) || misplaced(es, {bias, residual, y})) return CONV_ERR_ARG;
  int dev, sm;
  st = current_device(&dev, &sm);
  if (st != CONV_OK) return st;
  const Int8Plan r = plan_int8(p, sh, reinterpret_cast<uintptr_t>(w) % 16 == 0, reinterpret_cast<uintptr_t>(x) % 16 == 0, sm);
  if (scratch_bad(scratch, scratch_bytes, r.total)) return CONV_ERR_SCRATCH;
  ranges.add_out(r.total ? scratch : nullptr, r.total);
  if (ranges.clash()) return CONV_ERR_ALIAS;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  char* base = static_cast<char*>(scratch);
  Int8Args g;
  memset(&g, 0, sizeof(g));
  g.w = w; g.w_scale = w_scale;
  g.x = static_cast<const int8_t*>(x);
  g.x_scale = x_scale;
  g.ldx = r.ldq; g.ldw = sh.ldw;
  g.M = static_cast<int>(p->rows); g.N = static_cast<int>(p->c_out); g.K = static_cast<int>(p->c_in);
  DenseEpi& e = g.epi;
  e.mode = EPI_LINEAR;
  e.act = p->act; e.alpha = p->act_alpha; e.beta = p->act_beta;
  e.residual_last = (p->flags & CONV_LINEAR_FLAG_RESIDUAL_LAST) != 0;
  e.bias = bias; e.residual = residual; e.y = y;
  e.ldr = sh.ldr; e.ldy = sh.ldy;
  if (!p->x_quantized) {
    float* scale = reinterpret_cast<float*>(base + r.scale_off);
    CONV_TRY(launch_quantize({x, base + r.q_off, scale, p->rows, p->c_in, sh.ldx, r.ldq}, p->dtype, r.kernel != I8_FEW, sm, s));
    g.x = reinterpret_cast<int8_t*>(base + r.q_off);
    g.x_scale = scale;
  }
  if (r.kernel == I8_FEW) {
    if (r.pad) {
      CONV_TRY(launch_widen({g.x, base + r.q_off, p->rows, p->c_in, sh.ldx, r.ldq}, false, false, sm, s));
      g.x = reinterpret_cast<int8_t*>(base + r.q_off);
    }
    CONV_TRY(launch_int8_few(g, p->dtype, !p->x_quantized || r.pad, sm, s));
    return CONV_OK;
  }
  __half *xh = reinterpret_cast<__half*>(base + r.q_off), *wh = reinterpret_cast<__half*>(base + r.w_off);
  if (p->x_quantized) CONV_TRY(launch_widen({g.x, xh, p->rows, p->c_in, sh.ldx, r.ldq}, true, false, sm, s));
  if (r.kernel == I8_MID) {
    CONV_TRY(launch_int8_mid(r.mid, g, xh, p->dtype, s));
    return CONV_OK;
  }
  CONV_TRY(launch_widen({w, wh, p->c_out, p->c_in, sh.ldw, r.ldw}, true, true, sm, s));
  g.ldw = r.ldw;
  CONV_TRY(launch_int8_tc(r.tc, g, xh, wh, p->dtype, base + r.part_off, s));
  return CONV_OK;
}

}  // extern "C"
