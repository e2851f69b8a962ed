// dense_api.cu -- the C ABI of the dense operators (linear.h): validation,
// planning and dispatch.  Everything here runs on the host; a call only
// enqueues.  A plan is a function of the problem and the SM count (and of
// whether the operands' addresses are 16-byte aligned; where one is not, of the
// scratch given too), so the order of every sum is too.
#include <math.h>
#include <stdio.h>
#include <string.h>

#include <algorithm>
#include <utility>
#include <vector>

#include "dense_internal.h"

using namespace conv;

namespace {

constexpr long long kI32 = 2147483647LL;
constexpr long long kMaxElems = 1LL << 40;   // of one matrix
constexpr uint32_t kFlags = CONV_LINEAR_FLAG_RESIDUAL_LAST | CONV_LINEAR_FLAG_UNALIGNED | CONV_LINEAR_FLAG_FORCE_FFMA |
                            CONV_LINEAR_FLAG_NO_FEW_ROWS;

size_t align256(size_t v) { return (v + 255) / 256 * 256; }
// Row length of the library's own matrices: whole cache lines of 16-bit values, so that a copy of 64 values is one line,
// and blocks of 64 columns exist.
long long round64(long long v) { return (v + 63) / 64 * 64; }
size_t elem_size(int dtype) { return dtype == CONV_F32 ? 4 : 2; }

// Row stride as given (0: dense); false if it is below the width or too large.
bool stride_of(int64_t given, long long width, long long* out) {
  *out = given == 0 ? width : given;
  return *out >= width && *out <= (1LL << 36);
}
// The elements of rows x width at `stride`, if that is in range.
bool elems_ok(long long rows, long long stride) {
  long long n;
  return !__builtin_mul_overflow(rows, stride, &n) && n <= kMaxElems;
}
struct LinearShape {
  long long ldx, ldw, ldr, ldy;
};
conv_status validate(const conv_linear_problem* p, LinearShape* s) {
  if (!p) return CONV_ERR_NULL;
  if (p->dtype < CONV_F32 || p->dtype > CONV_BF16) return CONV_ERR_DTYPE;
  if (p->act < CONV_ACT_IDENTITY || p->act > CONV_ACT_GELU_TANH) return CONV_ERR_ACT;
  if (p->flags & ~kFlags) return CONV_ERR_ARG;
  if (p->rows < 0 || p->c_in < 1 || p->c_out < 1) return CONV_ERR_SHAPE;
  if (p->rows > kI32 - 65536 || p->c_in > kI32 - 65536 || p->c_out > kI32 - 65536) return CONV_ERR_SHAPE;
  if (!stride_of(p->x_stride, p->c_in, &s->ldx) || !stride_of(p->w_stride, p->c_in, &s->ldw) ||
      !stride_of(p->residual_stride, p->c_out, &s->ldr) || !stride_of(p->y_stride, p->c_out, &s->ldy))
    return CONV_ERR_SHAPE;
  if (!elems_ok(p->rows, s->ldx) || !elems_ok(p->c_out, s->ldw) || !elems_ok(p->rows, s->ldy) ||
      (p->has_residual && !elems_ok(p->rows, s->ldr)) || !elems_ok(p->rows, round64(p->c_out)))
    return CONV_ERR_OVERFLOW;
  return CONV_OK;
}

struct GatedShape {
  long long ldx, ldr, ldy, ldh;  // ldh: row length of h, g, u, dg, du as the library keeps them
};
conv_status validate(const conv_gated_problem* p, GatedShape* s) {
  if (!p) return CONV_ERR_NULL;
  if (p->dtype < CONV_F32 || p->dtype > CONV_BF16) return CONV_ERR_DTYPE;
  if (p->act < CONV_ACT_IDENTITY || p->act > CONV_ACT_GELU_TANH) return CONV_ERR_ACT;
  if (p->flags & ~(kFlags & ~CONV_LINEAR_FLAG_RESIDUAL_LAST)) return CONV_ERR_ARG;
  if (p->rows < 0 || p->c_in < 1 || p->hidden < 1 || p->c_out < 1) return CONV_ERR_SHAPE;
  if (p->rows > kI32 - 65536 || p->c_in > kI32 - 65536 || p->hidden > kI32 - 65536 || p->c_out > kI32 - 65536)
    return CONV_ERR_SHAPE;
  if (!stride_of(p->x_stride, p->c_in, &s->ldx) || !stride_of(p->residual_stride, p->c_out, &s->ldr) ||
      !stride_of(p->y_stride, p->c_out, &s->ldy))
    return CONV_ERR_SHAPE;
  s->ldh = round64(p->hidden);
  if (!elems_ok(p->rows, s->ldx) || !elems_ok(p->rows, s->ldy) || (p->has_residual && !elems_ok(p->rows, s->ldr)) ||
      !elems_ok(p->rows, s->ldh) || !elems_ok(round64(p->c_in), s->ldh) || !elems_ok(round64(p->c_out), s->ldh))
    return CONV_ERR_OVERFLOW;
  return CONV_OK;
}

bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }
// Whether an address is no multiple of its element's size (a typed access there would be a fault).
bool misplaced(size_t size, std::initializer_list<const void*> list) {
  uintptr_t all = 0;
  for (const void* p : list) all |= reinterpret_cast<uintptr_t>(p);
  return all % size != 0;
}

// ---- one product: which kernel, and its scratch ------------------------------
// Which kernels a call may run.
struct Mode {
  bool copies;   // every 16-bit operand is copied
  bool tc;       // the tensor-core kernels may run
  bool few;      // the kernel for few rows may run (it takes any alignment)
  bool ranges;   // the CUDA-core kernel may sum in k ranges (it needs scratch then)
};
Mode mode_of(uint32_t flags, int dtype) {
  Mode m;
  m.tc = !(flags & CONV_LINEAR_FLAG_FORCE_FFMA);
  m.copies = m.tc && dtype != CONV_F32 && (flags & CONV_LINEAR_FLAG_UNALIGNED);
  m.few = !(flags & (CONV_LINEAR_FLAG_FORCE_FFMA | CONV_LINEAR_FLAG_NO_FEW_ROWS));
  m.ranges = true;
  return m;
}

enum Variant { V_FFMA = 0, V_TC = 1, V_FEW = 2 };
struct Product {
  Variant variant;
  DenseFfmaPlan ffma;
  DenseTcPlan tc;
  int split;
  size_t part_bytes;   // planes of the k ranges
  int launches, sm;
};

// `g` without addresses.  `few`: the kernel for few rows takes it.
Product plan_product(const DenseGemm& g, int dtype, const Mode& mode, bool few, int sm) {
  Product r = {};
  r.sm = sm;
  if (few) {
    r.variant = V_FEW;
    r.split = 1;
  } else if (mode.tc) {
    r.variant = V_TC;
    r.tc = dense_tc_plan(g, dtype, sm);
    r.split = r.tc.split;
    r.part_bytes = r.tc.part_bytes;
  } else {
    r.variant = V_FFMA;
    r.ffma = dense_ffma_plan(g, sm, mode.ranges);
    r.split = r.ffma.split;
  }
  if (r.variant == V_FFMA && r.split > 1)
    r.part_bytes = static_cast<size_t>(r.split) * dense_products(g) * g.M * g.N * sizeof(float);
  r.launches = r.split > 1 ? 2 : 1;
  return r;
}

// `follows`: the kernel before in the stream is this call's own.
cudaError_t launch_product(const Product& r, DenseGemm g, int dtype, void* part, bool follows, cudaStream_t s) {
  if (r.variant == V_FEW) return launch_dense_few(g, dtype, follows, r.sm, s);
  if (r.variant == V_TC) return launch_dense_tc(r.tc, g, dtype, part, s);
  g.split = r.split;
  g.part = static_cast<float*>(part);
  g.k_per_split = r.ffma.k_per_split;
  const cudaError_t err = launch_dense_ffma(r.ffma, g, dtype, s);
  return err == cudaSuccess && g.split > 1 ? launch_dense_reduce(g, dtype, s) : err;
}

void describe_product(const Product& r, const DenseGemm& g, bool f32, int sm, char* buf, size_t len) {
  const long long k = static_cast<long long>(g.segs) * g.K;
  if (r.variant == V_FEW)
    snprintf(buf, len, "few_rows tile=%dx16 split=1 products=%d sums over %lld sms=%d launches=1", g.M, dense_products(g), k, sm);
  else if (r.variant == V_TC)
    snprintf(buf, len, "%s tile=%dx%d sms_per_tile=%d tiles=%d whole=%d split=%d products=%d sums over %lld sms=%d launches=%d",
             f32 ? "tcgen05_bf16x3" : "tcgen05", 128 * r.tc.cg, r.tc.nt, r.tc.cg, r.tc.tiles, r.tc.whole, r.split, dense_products(g), k, sm, r.launches);
  else
    snprintf(buf, len, "ffma tile=%dx%d split=%d products=%d sums over %lld sms=%d launches=%d", r.ffma.bm, r.ffma.bn,
             r.split, dense_products(g), k, sm, r.launches);
}

// An operand's copy: a 16-bit one's into aligned rows, where its rows need one; the three planes of a float32 one.
struct Copy {
  bool on, planes;
  long long rows, cols, ld_in, ld;
  size_t off, bytes;
};
struct Layout {
  size_t total = 0;
  size_t take(size_t bytes) {
    const size_t at = total;
    total = align256(total + bytes);
    return at;
  }
  // `tc`: for the tensor cores (the other kernels take operands as they are)
  Copy copy(bool tc, int dtype, bool unaligned, long long rows, long long cols, long long ld) {
    Copy c = {};
    c.planes = dtype == CONV_F32;
    c.on = tc && (c.planes || unaligned || ld % 8 != 0) && rows > 0;
    c.rows = rows; c.cols = cols; c.ld_in = ld;
    c.ld = c.on ? round64(cols) : ld;
    if (c.on) {
      c.bytes = static_cast<size_t>(rows) * c.ld * (c.planes ? 6 : 2);
      c.off = take(c.bytes);
    }
    return c;
  }
};
// Operands as the products read them: their copies, or themselves.  add() several, then enqueue() their copies together.
struct Copies {
  CopyJob job[kCopyJobs];
  int count = 0;
  bool planes = false;
  const void* add(const Copy& c, const void* in, char* scratch) {
    if (!c.on) return in;
    planes = c.planes;
    job[count++] = {in, scratch + c.off, c.ld_in, c.ld, c.rows, c.cols};
    return scratch + c.off;
  }
  cudaError_t enqueue(cudaStream_t s) const { return launch_dense_copies(job, count, planes, s); }
};

DenseGemm make_gemm(long long m, long long n, long long k, int a_mn, int b_mn, long long lda, long long ldb) {
  DenseGemm g;
  memset(&g, 0, sizeof(g));
  g.M = static_cast<int>(m); g.N = static_cast<int>(n); g.K = static_cast<int>(k);
  g.a_mn = a_mn; g.b_mn = b_mn;
  g.segs = 1; g.batch = 1;
  g.lda = lda; g.ldb = ldb;
  g.split = 1;
  g.epi.mode = EPI_LINEAR;
  return g;
}

// ---- linear -----------------------------------------------------------------
// Whether the kernel for few rows takes a product: up to 8 rows always, from 9 to 16 (two MMAs a weight piece; 16 sums
// in float32) unless the tensor-core kernel, if it may run, is the quicker one.  Measured, that kernel in brackets:
//   float32 rows that are no whole 16-byte pieces are loaded one by one: 9 rows of 2047 -> 2048 27.5 us (21.1), of
//   4095 -> 12289 193 (159); whole ones 16 of 4096 -> 4096 35.6 (59.6);
//   16-bit products of rows * outputs from 90,000 on: every block reads all of x, and the tensor-core kernel's tiles
//   fill the SMs without k ranges.  16 rows of 4096 -> 12288 25.0 us (21.4), 9 of 4096 -> 16384 29.7 (25.6); below,
//   16 rows of 4096 -> 4096 9.7 (12.3), 9 of 2048 -> 8192 9.7 (10.1).  Not where that kernel would copy the weights.
// `outputs`: of all products over the same x.  `pieces`: every operand's rows are whole 16-byte pieces.
bool few_rows(const Mode& m, long long rows, long long outputs, int dtype, bool pieces) {
  if (!m.few || rows < 1 || rows > kFewRows) return false;
  if (rows <= 8 || !m.tc) return true;
  if (dtype == CONV_F32) return pieces;
  return !pieces || m.copies || rows * outputs < 90000;
}
bool whole_pieces(int dtype, std::initializer_list<long long> sizes) {
  const int per = 16 / static_cast<int>(elem_size(dtype));
  return std::all_of(sizes.begin(), sizes.end(), [&](long long n) { return n % per == 0; });
}

struct LinearPlan {
  Copy x, w, z;
  DenseGemm fwd, dx, dw;
  Product pfwd, pdx, pdw;
  size_t part_off, dz_off, col_off, total;
  long long ldz;
  int col_blocks;
  bool dz, dz_planes;   // dz is written (an activation), as float32 operands' planes; else dy stands for it
};

LinearPlan plan_linear(const conv_linear_problem* p, const LinearShape& sh, const Mode& mode, int sm) {
  LinearPlan r = {};
  Layout l;
  const bool few = few_rows(mode, p->rows, p->c_out, p->dtype, whole_pieces(p->dtype, {p->c_in, sh.ldx, sh.ldw}));
  const bool tc = mode.tc && !few;
  r.x = l.copy(tc, p->dtype, mode.copies, p->rows, p->c_in, sh.ldx);
  r.w = l.copy(tc, p->dtype, mode.copies, p->c_out, p->c_in, sh.ldw);
  r.fwd = make_gemm(p->rows, p->c_out, p->c_in, 0, 0, r.x.ld, r.w.ld);
  DenseEpi& e = r.fwd.epi;
  e.act = p->act; e.alpha = p->act_alpha; e.beta = p->act_beta;
  e.residual_last = (p->flags & CONV_LINEAR_FLAG_RESIDUAL_LAST) != 0;
  e.ldr = sh.ldr; e.ldy = sh.ldy; e.ldp = p->c_out;
  if (p->rows > 0) r.pfwd = plan_product(r.fwd, p->dtype, mode, few, sm);
  r.part_off = l.take(r.pfwd.part_bytes);
  r.total = l.total;
  return r;
}

LinearPlan plan_linear_backward(const conv_linear_problem* p, const LinearShape& sh, const Mode& mode, int sm) {
  LinearPlan r = {};
  Layout l;
  const bool tc = mode.tc;
  r.x = l.copy(tc, p->dtype, mode.copies, p->rows, p->c_in, sh.ldx);
  r.w = l.copy(tc, p->dtype, mode.copies, p->c_out, p->c_in, sh.ldw);
  r.dz = p->act != CONV_ACT_IDENTITY;
  // dz as it is written (or dy, which stands for it), then as the products read it
  r.dz_planes = tc && p->dtype == CONV_F32;
  r.ldz = r.dz ? round64(p->c_out) : sh.ldy;
  if (r.dz) r.dz_off = l.take(static_cast<size_t>(p->rows) * r.ldz * (r.dz_planes ? 6 : elem_size(p->dtype)));
  else r.z = l.copy(tc, p->dtype, mode.copies, p->rows, p->c_out, r.ldz);
  const long long ldz = r.dz ? r.ldz : r.z.ld;
  if (p->rows > 0) {
    r.col_blocks = dense_col_blocks(p->rows, p->c_out, sm);
    r.col_off = l.take(static_cast<size_t>(r.col_blocks) * p->c_out * sizeof(float));
    r.dx = make_gemm(p->rows, p->c_in, p->c_out, 0, 1, ldz, r.w.ld);
    r.dx.b_pad = r.w.on;
    r.dx.epi.ldy = p->c_in;
    r.pdx = plan_product(r.dx, p->dtype, mode, false, sm);
    r.dw = make_gemm(p->c_out, p->c_in, p->rows, 1, 1, ldz, r.x.ld);
    r.dw.a_pad = r.dz || r.z.on;
    r.dw.b_pad = r.x.on;
    r.dw.epi.ldy = p->c_in;
    r.pdw = plan_product(r.dw, p->dtype, mode, false, sm);
  }
  r.part_off = l.take(std::max(r.pdx.part_bytes, r.pdw.part_bytes));
  r.total = l.total;
  return r;
}

// Outputs overlap neither inputs, nor scratch, nor one another.
struct Ranges {
  // rows of `width` bytes, `stride` bytes apart (one row: stride 0)
  struct R { uintptr_t p; size_t width, stride, span; };
  R in[8], out[8];  // the most that a call has
  int ins = 0, outs = 0;
  static R rows_of(const void* p, size_t rows, size_t width, size_t stride) {
    return {reinterpret_cast<uintptr_t>(p), width, rows > 1 ? stride : 0, rows < 1 ? 0 : (rows - 1) * stride + width};
  }
  void add(R* list, int* n, const R& r) { if (r.p && r.span) list[(*n)++] = r; }
  void add_in(const void* p, size_t n) { add(in, &ins, rows_of(p, n ? 1 : 0, n, n)); }
  void add_out(const void* p, size_t n) { add(out, &outs, rows_of(p, n ? 1 : 0, n, n)); }
  void add_in(const void* p, size_t rows, size_t width, size_t stride) { add(in, &ins, rows_of(p, rows, width, stride)); }
  void add_out(const void* p, size_t rows, size_t width, size_t stride) { add(out, &outs, rows_of(p, rows, width, stride)); }
  static bool hit(const R& a, const R& b) {
    if (a.p >= b.p + b.span || b.p >= a.p + a.span) return false;
    if (a.stride && a.stride == b.stride) {  // columns side by side in one wider matrix
      const size_t d = (b.p >= a.p ? b.p - a.p : a.stride - (a.p - b.p) % a.stride) % a.stride;
      if (d >= a.width && d + b.width <= a.stride) return false;
    }
    return true;
  }
  bool clash() const {
    for (int i = 0; i < outs; ++i) {
      for (int j = 0; j < ins; ++j) if (hit(out[i], in[j])) return true;
      for (int j = 0; j < i; ++j) if (hit(out[i], out[j])) return true;
    }
    return false;
  }
};

bool scratch_bad(const void* scratch, size_t have, size_t need) {
  return need > 0 && (!scratch || have < need || reinterpret_cast<uintptr_t>(scratch) % 256 != 0);
}

// The mode for these addresses: where one is unaligned, copies if the scratch
// has room for them, else the CUDA-core kernel, its sums whole where there is no room
// for ranges of them.
template <typename PlanFn>
auto plan_for(uint32_t flags, int dtype, std::initializer_list<const void*> operands, size_t have, PlanFn plan)
    -> decltype(plan(Mode{})) {
  Mode m = mode_of(flags, dtype);
  bool all = true;
  for (const void* p : operands) all = all && aligned16(p);
  if (m.tc && dtype != CONV_F32 && !all && !m.copies) {
    m.copies = true;
    auto r = plan(m);
    if (r.total <= have) return r;
    m.copies = m.tc = false;  // (the kernel for few rows stays)
    r = plan(m);
    if (r.total <= have) return r;
    m.ranges = false;  // what is left is within the scratch that the query asked for without copies
  }
  return plan(m);
}

#define CONV_TRY(call)                                   \
  do {                                                   \
    if ((call) != cudaSuccess) return CONV_ERR_CUDA;     \
  } while (0)

// ---- gated ------------------------------------------------------------------
struct GatedPlan {
  Copy x, wg, wu, wd, dy, h, dg, du;
  DenseGemm up, down;                 // forward
  DenseGemm dh, dx, dwgu, dwd;        // backward
  Product pup, pdown, pdh, pdx, pdwgu, pdw1, pdwd;  // pdw1: one of dWg, dWu alone
  size_t h_off, dg_off, du_off, part_off, total;
};
struct GatedSaved {
  size_t g_off, u_off, h_off, total;
};
GatedSaved gated_saved(const conv_gated_problem* p, const GatedShape& sh) {
  Layout l;
  GatedSaved s;
  const size_t n = static_cast<size_t>(p->rows) * sh.ldh;
  s.g_off = l.take(n * 4);
  s.u_off = l.take(n * 4);
  s.h_off = l.take(n * elem_size(p->dtype));
  s.total = l.total;
  return s;
}

GatedPlan plan_gated(const conv_gated_problem* p, const GatedShape& sh, const Mode& mode, int sm, bool saved) {
  GatedPlan r = {};
  Layout l;
  const bool few = few_rows(mode, p->rows, 2 * p->hidden, p->dtype, whole_pieces(p->dtype, {p->c_in, p->hidden, sh.ldx}));
  const bool tc = mode.tc && !few;
  r.x = l.copy(tc, p->dtype, mode.copies, p->rows, p->c_in, sh.ldx);
  r.wg = l.copy(tc, p->dtype, mode.copies, p->hidden, p->c_in, p->c_in);
  r.wu = l.copy(tc, p->dtype, mode.copies, p->hidden, p->c_in, p->c_in);
  r.wd = l.copy(tc, p->dtype, mode.copies, p->c_out, p->hidden, p->hidden);
  if (!saved) r.h_off = l.take(static_cast<size_t>(p->rows) * sh.ldh * elem_size(p->dtype));
  r.h = l.copy(tc, p->dtype, false, p->rows, p->hidden, sh.ldh);
  if (p->rows > 0) {
    r.up = make_gemm(p->rows, p->hidden, p->c_in, 0, 0, r.x.ld, r.wg.ld);
    r.up.dual = 1;
    r.up.epi.mode = EPI_GATED;
    r.up.epi.act = p->act; r.up.epi.alpha = p->act_alpha; r.up.epi.beta = p->act_beta;
    r.up.epi.ldy = sh.ldh; r.up.epi.ldp = sh.ldh;
    r.pup = plan_product(r.up, p->dtype, mode, few, sm);
    r.down = make_gemm(p->rows, p->c_out, p->hidden, 0, 0, r.h.ld, r.wd.ld);
    r.down.epi.ldr = sh.ldr; r.down.epi.ldy = sh.ldy;
    r.pdown = plan_product(r.down, p->dtype, mode, few, sm);
  }
  r.part_off = l.take(std::max(r.pup.part_bytes, r.pdown.part_bytes));
  r.total = l.total;
  return r;
}

GatedPlan plan_gated_backward(const conv_gated_problem* p, const GatedShape& sh, const Mode& mode, int sm) {
  GatedPlan r = {};
  Layout l;
  const bool tc = mode.tc;
  r.x = l.copy(tc, p->dtype, mode.copies, p->rows, p->c_in, sh.ldx);
  r.wg = l.copy(tc, p->dtype, mode.copies, p->hidden, p->c_in, p->c_in);
  r.wu = l.copy(tc, p->dtype, mode.copies, p->hidden, p->c_in, p->c_in);
  r.wd = l.copy(tc, p->dtype, mode.copies, p->c_out, p->hidden, p->hidden);
  r.dy = l.copy(tc, p->dtype, mode.copies, p->rows, p->c_out, sh.ldy);
  const size_t n = static_cast<size_t>(p->rows) * sh.ldh * elem_size(p->dtype);
  r.dg_off = l.take(n);
  r.du_off = l.take(n);
  r.dg = l.copy(tc, p->dtype, false, p->rows, p->hidden, sh.ldh);
  r.du = l.copy(tc, p->dtype, false, p->rows, p->hidden, sh.ldh);
  r.h = l.copy(tc, p->dtype, false, p->rows, p->hidden, sh.ldh);
  if (p->rows > 0) {
    r.dh = make_gemm(p->rows, p->hidden, p->c_out, 0, 1, r.dy.ld, r.wd.ld);
    r.dh.b_pad = r.wd.on;
    r.dh.epi.mode = EPI_GATED_BWD;
    r.dh.epi.act = p->act; r.dh.epi.alpha = p->act_alpha; r.dh.epi.beta = p->act_beta;
    r.dh.epi.ldy = sh.ldh; r.dh.epi.ldp = sh.ldh;
    r.pdh = plan_product(r.dh, p->dtype, mode, false, sm);
    r.dx = make_gemm(p->rows, p->c_in, p->hidden, 0, 1, r.dg.ld, r.wg.ld);
    r.dx.b_pad = r.wg.on;
    r.dx.segs = 2;
    r.dx.epi.ldy = p->c_in;
    r.pdx = plan_product(r.dx, p->dtype, mode, false, sm);
    r.dwgu = make_gemm(p->hidden, p->c_in, p->rows, 1, 1, r.dg.ld, r.x.ld);
    r.dwgu.a_pad = 1;
    r.dwgu.b_pad = r.x.on;
    r.dwgu.batch = 2;
    r.dwgu.epi.ldy = p->c_in;
    r.pdwgu = plan_product(r.dwgu, p->dtype, mode, false, sm);
    DenseGemm one = r.dwgu;
    one.batch = 1;
    r.pdw1 = plan_product(one, p->dtype, mode, false, sm);
    r.dwd = make_gemm(p->c_out, p->hidden, p->rows, 1, 1, r.dy.ld, r.h.ld);
    r.dwd.a_pad = r.dy.on;
    r.dwd.b_pad = 1;
    r.dwd.epi.ldy = p->hidden;
    r.pdwd = plan_product(r.dwd, p->dtype, mode, false, sm);
  }
  r.part_off = l.take(std::max({r.pdh.part_bytes, r.pdx.part_bytes, r.pdwgu.part_bytes, r.pdw1.part_bytes, r.pdwd.part_bytes}));
  r.total = l.total;
  return r;
}

// The pointer checks of conv_clip_grads.
conv_status clip_check(int64_t count, const void* const* in, void* const* out, const int64_t* sizes,
                       const int32_t* dtypes, const float* norm, const void* scratch, size_t have, size_t need) {
  // ranges by address: an output touches no other range but its own input's, exactly
  struct R { uintptr_t lo, hi; bool out; };
  auto below = [](const R& a, const R& b) { return a.lo < b.lo; };
  std::vector<R> ins, outs, ranges;
  ins.reserve(static_cast<size_t>(count));
  outs.reserve(static_cast<size_t>(count) + 2);
  for (int64_t i = 0; i < count; ++i) {
    if (dtypes[i] < CONV_F32 || dtypes[i] > CONV_BF16) return CONV_ERR_DTYPE;
    if (sizes[i] == 0) continue;
    const size_t es = elem_size(dtypes[i]), n = static_cast<size_t>(sizes[i]) * es;
    const uintptr_t a = reinterpret_cast<uintptr_t>(in[i]), b = out ? reinterpret_cast<uintptr_t>(out[i]) : 0;
    if (!a || (out && !b)) return CONV_ERR_NULL;
    if (a % es || b % es) return CONV_ERR_ARG;
    if (a != b) ins.push_back({a, a + n, false});
    if (b) outs.push_back({b, b + n, true});
  }
  if (scratch_bad(scratch, have, need)) return CONV_ERR_SCRATCH;
  // (buffers mostly come in order already)
  if (!std::is_sorted(ins.begin(), ins.end(), below)) std::sort(ins.begin(), ins.end(), below);
  outs.push_back({reinterpret_cast<uintptr_t>(scratch), reinterpret_cast<uintptr_t>(scratch) + need, true});
  outs.push_back({reinterpret_cast<uintptr_t>(norm), reinterpret_cast<uintptr_t>(norm) + 4, true});
  std::sort(outs.end() - 2, outs.end(), below);
  if (!std::is_sorted(outs.begin(), outs.end() - 2, below)) std::sort(outs.begin(), outs.end() - 2, below);
  std::inplace_merge(outs.begin(), outs.end() - 2, outs.end(), below);
  ranges.resize(ins.size() + outs.size());
  std::merge(ins.begin(), ins.end(), outs.begin(), outs.end(), ranges.begin(), below);
  // the furthest end so far of any range, and of the written ones
  uintptr_t end = 0, end_out = 0;
  for (const R& r : ranges) {
    if (r.lo < end_out || (r.out && r.lo < end)) return CONV_ERR_ALIAS;
    end = std::max(end, r.hi);
    if (r.out) end_out = std::max(end_out, r.hi);
  }
  return CONV_OK;
}

}  // namespace

extern "C" {

conv_status conv_linear_scratch_bytes(const conv_linear_problem* p, size_t* bytes) {
  if (!bytes) return CONV_ERR_NULL;
  LinearShape sh;
  conv_status st = validate(p, &sh);
  int dev, sm;
  if (st == CONV_OK) st = current_device(&dev, &sm);
  if (st == CONV_OK) *bytes = plan_linear(p, sh, mode_of(p->flags, p->dtype), sm).total;
  return st;
}

conv_status conv_linear_backward_scratch_bytes(const conv_linear_problem* p, size_t* bytes) {
  if (!bytes) return CONV_ERR_NULL;
  LinearShape sh;
  conv_status st = validate(p, &sh);
  int dev, sm;
  if (st == CONV_OK) st = current_device(&dev, &sm);
  if (st == CONV_OK) *bytes = plan_linear_backward(p, sh, mode_of(p->flags, p->dtype), sm).total;
  return st;
}

conv_status conv_linear_describe_plan(const conv_linear_problem* p, int32_t pass, int32_t sm_count, char* buf,
                                      size_t len) {
  if (!buf || !len) return CONV_ERR_NULL;
  if (pass < 0 || pass > 2 || sm_count < 1) return CONV_ERR_ARG;
  LinearShape sh;
  const conv_status st = validate(p, &sh);
  if (st != CONV_OK) return st;
  if (p->rows == 0) {
    snprintf(buf, len, "nothing launches=0");
    return CONV_OK;
  }
  const Mode mode = mode_of(p->flags, p->dtype);
  if (pass == 0) {
    const LinearPlan r = plan_linear(p, sh, mode, sm_count);
    describe_product(r.pfwd, r.fwd, p->dtype == CONV_F32, sm_count, buf, len);
  } else {
    const LinearPlan r = plan_linear_backward(p, sh, mode, sm_count);
    describe_product(pass == 1 ? r.pdx : r.pdw, pass == 1 ? r.dx : r.dw, p->dtype == CONV_F32, sm_count, buf, len);
  }
  return CONV_OK;
}

conv_status conv_linear_forward(const conv_linear_problem* p, const void* x, const void* w, const void* bias,
                                const void* residual, void* y, float* pre, void* scratch, size_t scratch_bytes,
                                void* stream) {
  LinearShape sh;
  conv_status st = validate(p, &sh);
  if (st != CONV_OK) return st;
  if (p->rows == 0) return CONV_OK;
  if (!x || !w || !y || (p->has_bias && !bias) || (p->has_residual && !residual)) return CONV_ERR_NULL;
  const size_t es = elem_size(p->dtype);
  Ranges ranges;
  ranges.add_in(x, p->rows, p->c_in * es, sh.ldx * es);
  ranges.add_in(w, p->c_out, p->c_in * es, sh.ldw * es);
  if (p->has_bias) ranges.add_in(bias, p->c_out * es);
  if (p->has_residual) ranges.add_in(residual, p->rows, p->c_out * es, sh.ldr * es);
  ranges.add_out(y, p->rows, p->c_out * es, sh.ldy * es);
  ranges.add_out(pre, static_cast<size_t>(p->rows) * p->c_out * 4);
  if (ranges.clash()) return CONV_ERR_ALIAS;
  if (misplaced(es, {x, w, p->has_bias ? bias : nullptr, p->has_residual ? residual : nullptr, y}) || misplaced(4, {pre}))
    return CONV_ERR_ARG;
  int dev, sm;
  st = current_device(&dev, &sm);
  if (st != CONV_OK) return st;
  const LinearPlan r = plan_for(p->flags, p->dtype, {x, w}, scratch_bytes,
                                [&](const Mode& m) { return plan_linear(p, sh, m, sm); });
  if (scratch_bad(scratch, scratch_bytes, r.total)) return CONV_ERR_SCRATCH;
  ranges.add_out(r.total ? scratch : nullptr, r.total);
  if (ranges.clash()) return CONV_ERR_ALIAS;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  char* base = static_cast<char*>(scratch);
  DenseGemm g = r.fwd;
  Copies copies;
  g.a[0] = copies.add(r.x, x, base);
  g.b[0] = copies.add(r.w, w, base);
  CONV_TRY(copies.enqueue(s));
  g.epi.bias = p->has_bias ? bias : nullptr;
  g.epi.residual = p->has_residual ? residual : nullptr;
  g.epi.y = y;
  g.epi.pre = pre;
  CONV_TRY(launch_product(r.pfwd, g, p->dtype, base + r.part_off, false, s));
  return CONV_OK;
}

conv_status conv_linear_backward(const conv_linear_problem* p, const void* x, const void* w, const float* pre,
                                 const void* dy, void* dx, void* dw, void* dbias, void* dresidual, void* scratch,
                                 size_t scratch_bytes, void* stream) {
  LinearShape sh;
  conv_status st = validate(p, &sh);
  if (st != CONV_OK) return st;
  const size_t es = elem_size(p->dtype);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool act = p->act != CONV_ACT_IDENTITY;
  if (p->rows > 0 && (!dy || (dw && !x) || (dx && !w) || (act && !pre))) return CONV_ERR_NULL;
  Ranges ranges;
  if (p->rows > 0) {
    if (dw) ranges.add_in(x, p->rows, p->c_in * es, sh.ldx * es);
    if (dx) ranges.add_in(w, p->c_out, p->c_in * es, sh.ldw * es);
    if (act) ranges.add_in(pre, static_cast<size_t>(p->rows) * p->c_out * 4);
    ranges.add_in(dy, p->rows, p->c_out * es, sh.ldy * es);
  }
  ranges.add_out(dx, static_cast<size_t>(p->rows) * p->c_in * es);
  ranges.add_out(dw, static_cast<size_t>(p->c_out) * p->c_in * es);
  ranges.add_out(dbias, p->c_out * es);
  ranges.add_out(dresidual, static_cast<size_t>(p->rows) * p->c_out * es);
  if (ranges.clash()) return CONV_ERR_ALIAS;
  if (misplaced(es, {x, w, dy, dx, dw, dbias, dresidual}) || misplaced(4, {pre})) return CONV_ERR_ARG;
  int dev, sm;
  st = current_device(&dev, &sm);
  if (st != CONV_OK) return st;
  if (p->rows == 0) {
    if (dw) CONV_TRY(cudaMemsetAsync(dw, 0, static_cast<size_t>(p->c_out) * p->c_in * es, s));
    if (dbias) CONV_TRY(cudaMemsetAsync(dbias, 0, p->c_out * es, s));
    return CONV_OK;
  }
  // an operand that no wanted output reads does not count
  const LinearPlan r = plan_for(p->flags, p->dtype, {dw ? x : nullptr, dx ? w : nullptr, act || !(dx || dw) ? nullptr : dy},
                                scratch_bytes, [&](const Mode& m) { return plan_linear_backward(p, sh, m, sm); });
  if (scratch_bad(scratch, scratch_bytes, r.total)) return CONV_ERR_SCRATCH;
  ranges.add_out(r.total ? scratch : nullptr, r.total);
  if (ranges.clash()) return CONV_ERR_ALIAS;
  char* base = static_cast<char*>(scratch);
  const bool last = (p->flags & CONV_LINEAR_FLAG_RESIDUAL_LAST) != 0;
  // dz (as the products read it), and its column sums
  const bool products = dx || dw;
  Copies copies;
  const void* z = nullptr;
  if (products) z = r.dz ? base + r.dz_off : copies.add(r.z, dy, base);
  const void* xc = dw ? copies.add(r.x, x, base) : nullptr;
  const void* wc = dx ? copies.add(r.w, w, base) : nullptr;
  CONV_TRY(copies.enqueue(s));
  if ((products && r.dz) || dbias)
    CONV_TRY(launch_dense_dz(dy, sh.ldy, pre, products && r.dz ? base + r.dz_off : nullptr, r.ldz, r.dz_planes, dbias,
                             reinterpret_cast<float*>(base + r.col_off), r.col_blocks, p->rows, p->c_out, p->act,
                             p->act_alpha, p->act_beta, p->dtype, s));
  if (dresidual) {
    if (act && !last)
      CONV_TRY(launch_dense_dz(dy, sh.ldy, pre, dresidual, p->c_out, false, nullptr, nullptr, r.col_blocks, p->rows, p->c_out,
                               p->act, p->act_alpha, p->act_beta, p->dtype, s));
    else
      CONV_TRY(cudaMemcpy2DAsync(dresidual, p->c_out * es, dy, sh.ldy * es, p->c_out * es, p->rows,
                                 cudaMemcpyDeviceToDevice, s));
  }
  if (dx) {
    DenseGemm g = r.dx;
    g.a[0] = z;
    g.b[0] = wc;
    g.epi.y = dx;
    CONV_TRY(launch_product(r.pdx, g, p->dtype, base + r.part_off, false, s));
  }
  if (dw) {
    DenseGemm g = r.dw;
    g.a[0] = z;
    g.b[0] = xc;
    g.epi.y = dw;
    CONV_TRY(launch_product(r.pdw, g, p->dtype, base + r.part_off, false, s));
  }
  return CONV_OK;
}

conv_status conv_gated_scratch_bytes(const conv_gated_problem* p, size_t* bytes) {
  if (!bytes) return CONV_ERR_NULL;
  GatedShape sh;
  conv_status st = validate(p, &sh);
  int dev, sm;
  if (st == CONV_OK) st = current_device(&dev, &sm);
  if (st == CONV_OK) *bytes = plan_gated(p, sh, mode_of(p->flags, p->dtype), sm, false).total;
  return st;
}

conv_status conv_gated_backward_scratch_bytes(const conv_gated_problem* p, size_t* bytes) {
  if (!bytes) return CONV_ERR_NULL;
  GatedShape sh;
  conv_status st = validate(p, &sh);
  int dev, sm;
  if (st == CONV_OK) st = current_device(&dev, &sm);
  if (st == CONV_OK) *bytes = plan_gated_backward(p, sh, mode_of(p->flags, p->dtype), sm).total;
  return st;
}

conv_status conv_gated_saved_bytes(const conv_gated_problem* p, size_t* bytes) {
  if (!bytes) return CONV_ERR_NULL;
  GatedShape sh;
  const conv_status st = validate(p, &sh);
  if (st == CONV_OK) *bytes = gated_saved(p, sh).total;
  return st;
}

conv_status conv_gated_forward(const conv_gated_problem* p, const void* x, const void* w_gate, const void* w_up,
                               const void* w_down, const void* residual, void* y, void* saved, void* scratch,
                               size_t scratch_bytes, void* stream) {
  GatedShape sh;
  conv_status st = validate(p, &sh);
  if (st != CONV_OK) return st;
  if (p->rows == 0) return CONV_OK;
  if (!x || !w_gate || !w_up || !w_down || !y || (p->has_residual && !residual)) return CONV_ERR_NULL;
  if (reinterpret_cast<uintptr_t>(saved) % 256) return CONV_ERR_ARG;
  const size_t es = elem_size(p->dtype);
  const size_t wbytes = static_cast<size_t>(p->hidden) * p->c_in * es;
  const GatedSaved keep = gated_saved(p, sh);
  Ranges ranges;
  ranges.add_in(x, p->rows, p->c_in * es, sh.ldx * es);
  ranges.add_in(w_gate, wbytes);
  ranges.add_in(w_up, wbytes);
  ranges.add_in(w_down, static_cast<size_t>(p->c_out) * p->hidden * es);
  if (p->has_residual) ranges.add_in(residual, p->rows, p->c_out * es, sh.ldr * es);
  ranges.add_out(y, p->rows, p->c_out * es, sh.ldy * es);
  ranges.add_out(saved, keep.total);
  if (ranges.clash()) return CONV_ERR_ALIAS;
  if (misplaced(es, {x, w_gate, w_up, w_down, p->has_residual ? residual : nullptr, y})) return CONV_ERR_ARG;
  int dev, sm;
  st = current_device(&dev, &sm);
  if (st != CONV_OK) return st;
  const GatedPlan r = plan_for(p->flags, p->dtype, {x, w_gate, w_up, w_down}, scratch_bytes,
                               [&](const Mode& m) { return plan_gated(p, sh, m, sm, saved != nullptr); });
  if (scratch_bad(scratch, scratch_bytes, r.total)) return CONV_ERR_SCRATCH;
  ranges.add_out(r.total ? scratch : nullptr, r.total);
  if (ranges.clash()) return CONV_ERR_ALIAS;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  char* base = static_cast<char*>(scratch);
  char* kept = static_cast<char*>(saved);
  void* h = saved ? kept + keep.h_off : base + r.h_off;
  DenseGemm g = r.up;
  Copies copies, hidden;
  g.a[0] = copies.add(r.x, x, base);
  g.b[0] = copies.add(r.wg, w_gate, base);
  g.b[1] = copies.add(r.wu, w_up, base);
  const void* down = copies.add(r.wd, w_down, base);
  CONV_TRY(copies.enqueue(s));
  g.epi.y = h;
  if (saved) {
    g.epi.pre = reinterpret_cast<float*>(kept + keep.g_off);
    g.epi.pre2 = reinterpret_cast<float*>(kept + keep.u_off);
  }
  CONV_TRY(launch_product(r.pup, g, p->dtype, base + r.part_off, false, s));
  g = r.down;
  g.a[0] = hidden.add(r.h, h, base);
  CONV_TRY(hidden.enqueue(s));
  g.b[0] = down;
  g.epi.residual = p->has_residual ? residual : nullptr;
  g.epi.y = y;
  CONV_TRY(launch_product(r.pdown, g, p->dtype, base + r.part_off, true, s));
  return CONV_OK;
}

conv_status conv_gated_backward(const conv_gated_problem* p, const void* x, const void* w_gate, const void* w_up,
                                const void* w_down, const void* saved, const void* dy, void* dx, void* dw_gate,
                                void* dw_up, void* dw_down, void* scratch, size_t scratch_bytes, void* stream) {
  GatedShape sh;
  conv_status st = validate(p, &sh);
  if (st != CONV_OK) return st;
  const size_t es = elem_size(p->dtype);
  const size_t wbytes = static_cast<size_t>(p->hidden) * p->c_in * es;
  const size_t wdbytes = static_cast<size_t>(p->c_out) * p->hidden * es;
  const bool dgu = dx || dw_gate || dw_up;
  if (p->rows > 0 && (!dy || !saved || (dgu && !w_down) || ((dw_gate || dw_up) && !x) || (dx && (!w_gate || !w_up))))
    return CONV_ERR_NULL;
  if (reinterpret_cast<uintptr_t>(saved) % 256) return CONV_ERR_ARG;
  const GatedSaved keep = gated_saved(p, sh);
  Ranges ranges;
  if (p->rows > 0) {
    if (dw_gate || dw_up) ranges.add_in(x, p->rows, p->c_in * es, sh.ldx * es);
    if (dx) {
      ranges.add_in(w_gate, wbytes);
      ranges.add_in(w_up, wbytes);
    }
    if (dgu) ranges.add_in(w_down, wdbytes);
    ranges.add_in(saved, keep.total);
    ranges.add_in(dy, p->rows, p->c_out * es, sh.ldy * es);
  }
  ranges.add_out(dx, static_cast<size_t>(p->rows) * p->c_in * es);
  ranges.add_out(dw_gate, wbytes);
  ranges.add_out(dw_up, wbytes);
  ranges.add_out(dw_down, wdbytes);
  if (ranges.clash()) return CONV_ERR_ALIAS;
  if (misplaced(es, {x, w_gate, w_up, w_down, dy, dx, dw_gate, dw_up, dw_down})) return CONV_ERR_ARG;
  int dev, sm;
  st = current_device(&dev, &sm);
  if (st != CONV_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (p->rows == 0) {
    if (dw_gate) CONV_TRY(cudaMemsetAsync(dw_gate, 0, wbytes, s));
    if (dw_up) CONV_TRY(cudaMemsetAsync(dw_up, 0, wbytes, s));
    if (dw_down) CONV_TRY(cudaMemsetAsync(dw_down, 0, wdbytes, s));
    return CONV_OK;
  }
  const bool dwgu = dw_gate || dw_up;
  const GatedPlan r = plan_for(
      p->flags, p->dtype, {dwgu ? x : nullptr, dx ? w_gate : nullptr, dx ? w_up : nullptr, dgu ? w_down : nullptr, dy},
      scratch_bytes, [&](const Mode& m) { return plan_gated_backward(p, sh, m, sm); });
  if (scratch_bad(scratch, scratch_bytes, r.total)) return CONV_ERR_SCRATCH;
  ranges.add_out(r.total ? scratch : nullptr, r.total);
  if (ranges.clash()) return CONV_ERR_ALIAS;
  char* base = static_cast<char*>(scratch);
  const char* kept = static_cast<const char*>(saved);
  void* part = base + r.part_off;
  Copies copies, grads;
  const void* dyc = copies.add(r.dy, dy, base);
  const void* wdc = dgu ? copies.add(r.wd, w_down, base) : nullptr;
  const void* wgc = dx ? copies.add(r.wg, w_gate, base) : nullptr;
  const void* wuc = dx ? copies.add(r.wu, w_up, base) : nullptr;
  const void* xc = dwgu ? copies.add(r.x, x, base) : nullptr;
  const void* hc = dw_down ? copies.add(r.h, kept + keep.h_off, base) : nullptr;
  CONV_TRY(copies.enqueue(s));
  const void *dg = nullptr, *du = nullptr;
  if (dgu) {
    DenseGemm g = r.dh;
    g.a[0] = dyc;
    g.b[0] = wdc;
    g.epi.pre = reinterpret_cast<float*>(const_cast<char*>(kept + keep.g_off));
    g.epi.pre2 = reinterpret_cast<float*>(const_cast<char*>(kept + keep.u_off));
    g.epi.y = base + r.dg_off;
    g.epi.y2 = base + r.du_off;
    CONV_TRY(launch_product(r.pdh, g, p->dtype, part, false, s));
    dg = grads.add(r.dg, base + r.dg_off, base);
    du = grads.add(r.du, base + r.du_off, base);
    CONV_TRY(grads.enqueue(s));
  }
  if (dx) {
    DenseGemm g = r.dx;
    g.a[0] = dg;
    g.a[1] = du;
    g.b[0] = wgc;
    g.b[1] = wuc;
    g.epi.y = dx;
    CONV_TRY(launch_product(r.pdx, g, p->dtype, part, false, s));
  }
  if (dwgu) {
    DenseGemm g = r.dwgu;
    Product q = r.pdwgu;
    g.b[0] = g.b[1] = xc;
    g.a[0] = dg;
    g.a[1] = du;
    g.epi.y = dw_gate;
    g.epi.y2 = dw_up;
    if (!dw_gate || !dw_up) {
      g.batch = 1;
      q = r.pdw1;
      if (!dw_gate) g.a[0] = g.a[1], g.epi.y = dw_up;
    }
    CONV_TRY(launch_product(q, g, p->dtype, part, false, s));
  }
  if (dw_down) {
    DenseGemm g = r.dwd;
    g.a[0] = dyc;
    g.b[0] = hc;
    g.epi.y = dw_down;
    CONV_TRY(launch_product(r.pdwd, g, p->dtype, part, false, s));
  }
  return CONV_OK;
}

conv_status conv_clip_scratch_bytes(int64_t count, const int64_t* sizes, size_t* bytes) {
  if (!bytes || (count > 0 && !sizes)) return CONV_ERR_NULL;
  if (count < 0 || count > (1 << 24)) return CONV_ERR_SHAPE;
  for (int64_t i = 0; i < count; ++i)
    if (sizes[i] < 0 || sizes[i] > kMaxElems) return CONV_ERR_SHAPE;
  *bytes = clip_scratch_bytes(count, sizes);
  return CONV_OK;
}

conv_status conv_clip_grads(int64_t count, const void* const* in, void* const* out, const int64_t* sizes,
                            const int32_t* dtypes, float max_norm, float eps, float* norm, void* scratch,
                            size_t scratch_bytes, void* stream) {
  if (!norm || (count > 0 && (!in || !sizes || !dtypes))) return CONV_ERR_NULL;
  size_t need;
  conv_status st = conv_clip_scratch_bytes(count, sizes, &need);
  if (st != CONV_OK) return st;
  if (!(max_norm >= 0.0f) || !(eps >= 0.0f) || misplaced(4, {norm})) return CONV_ERR_ARG;
  try {  // the list of ranges is host memory
    st = clip_check(count, in, out, sizes, dtypes, norm, scratch, scratch_bytes, need);
  } catch (...) {
    st = CONV_ERR_OVERFLOW;
  }
  if (st != CONV_OK) return st;
  int dev, sm;
  st = current_device(&dev, &sm);
  if (st != CONV_OK) return st;
  CONV_TRY(launch_clip(count, in, out, sizes, dtypes, max_norm, eps, norm, scratch, sm,
                       static_cast<cudaStream_t>(stream)));
  return CONV_OK;
}

conv_status conv_linear_device_error(uint32_t* word, int32_t reset) {
  if (!word) return CONV_ERR_NULL;
  int dev, sm;
  const conv_status st = current_device(&dev, &sm);
  if (st != CONV_OK) return st;
  CONV_TRY(dense_error_word(word, reset));
  return CONV_OK;
}

}  // extern "C"
