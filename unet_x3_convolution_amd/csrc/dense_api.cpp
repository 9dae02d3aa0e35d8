// Host side of the dense operators' C ABI: argument checks, launch plans,
// workspace layout and the launch sequences.  Nothing here allocates device
// memory, waits for the device or throws.
#include <algorithm>

#include "dense_checks.h"

using namespace oidn;

namespace {

// One product: bytes of the workspace its slices take, and its launch.
struct Product {
  int layout, epi;
  long rows, cols, len;
  int dtype;
  GemmPlan plan;
};
// Whether the sizes alone let a 16-bit product's operands go straight to LDS.
bool direct_sizes(const Product& p) {
  const bool ps = p.layout != kForward, qs = p.layout == kWeightGrad;
  return (qs ? p.rows : p.len) % 8 == 0 && (ps ? p.cols : p.len) % 8 == 0;
}
// Plans products that are to share a launch.
void plan_together(Product* const* p, int count) {
  GemmPlan* plans[kMaxGroup];
  PlanShape shapes[kMaxGroup];
  bool direct = true;
  for (int k = 0; k < count; ++k) {
    plans[k] = &p[k]->plan;
    shapes[k] = {p[k]->rows, p[k]->cols, p[k]->len, p[k]->epi, 0};
    direct = direct && direct_sizes(*p[k]);
  }
  plan_products(plans, shapes, count, p[0]->dtype, direct);
}
Product product(int layout, int epi, long rows, long cols, long len, int dtype) {
  Product p{layout, epi, rows, cols, len, dtype, {}};
  if (layout == kForward && rows <= kFewRows) {
    p.plan = GemmPlan{64, 64, true, false, 1, 0};
  } else {
    Product* one = &p;
    plan_together(&one, 1);
  }
  return p;
}
size_t product_bytes(const Product& p) {
  return p.plan.splits > 1 ? align256((size_t)p.plan.splits * p.rows * p.cols * sizeof(float)) : 0;
}
// Workgroups of a product's launch at most: where operands cannot go straight to
// LDS, the largest tiles give way to the next smaller ones.
long most_blocks(const Product& p) {
  if (p.plan.few) return 0;
  const bool staged = p.dtype != OIDN_F32 && p.plan.tile_r > 128;
  const long r = staged ? 128 : p.plan.tile_r, t = staged ? 128 : p.plan.tile_c, c = p.epi == kEpiGated ? t / 2 : t;
  return gemm_blocks((p.rows + r - 1) / r, (p.cols + c - 1) / c, p.plan.splits);
}
long sum_blocks(const Product& p) {
  return p.plan.splits > 1 ? slice_blocks(p.rows, (int)p.cols, p.plan.splits) : 0;
}
long slope_blocks(long rows, int cols, long chunk) {
  SlopeArgs s{};
  s.rows = rows;
  s.cols = cols;
  s.chunk = chunk;
  s.lanes = slope_lanes(cols);
  return slope_blocks(s);
}
// Whether a 16-bit operand can go straight to LDS in 16-byte units: `extent`
// is what its rows hold of (the summed length, or the output's rows or columns
// of a strided one), `span` the most rows that one tile's 32-bit offsets pass.
bool direct_operand(const void* p, long ld, long extent, long span) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && ld % 8 == 0 && extent % 8 == 0 &&
         span * ld < (1L << 30);
}
GemmArgs gemm_args(Product& p, const void* q, long ldq, const void* pm, long ldp, const EpilogueArgs& e,
                   void* slices) {
  if (p.dtype != OIDN_F32) {
    const bool ps = p.layout != kForward, qs = p.layout == kWeightGrad;
    p.plan.direct = direct_operand(q, ldq, qs ? p.rows : p.len, 256) &&
                    direct_operand(pm, ldp, ps ? p.cols : p.len, (p.epi == kEpiGated ? p.cols : 0) + 256);
  }
  if (!p.plan.direct && p.plan.tile_r > 128) p.plan.tile_r = p.plan.tile_c = 128;
  GemmArgs a{};
  a.q = q;
  a.ldq = ldq;
  a.p = pm;
  a.ldp = ldp;
  a.len = p.len;
  a.splits = p.plan.splits;
  a.per_split = p.plan.per_split;
  a.e = e;
  a.e.rows = p.rows;
  a.e.cols = (int)p.cols;
  a.e.stream = stream_result(p.rows, p.cols);
  if (p.plan.splits > 1) a.e.part = static_cast<float*>(slices);
  return a;
}
void set_tiles(const Product& p, GemmArgs& a) {
  a.tiles_r = (int)((p.rows + p.plan.tile_r - 1) / p.plan.tile_r);
  const long c = p.epi == kEpiGated ? p.plan.tile_c / 2 : p.plan.tile_c;
  a.tiles_c = (int)((p.cols + c - 1) / c);
}
// A forward or gated backward product; `groups` receives the row groups of the
// latter's column sums, and it takes `job` along.
int run_product(Product p, const void* q, long ldq, const void* pm, long ldp, const EpilogueArgs& e,
                void* slices, hipStream_t stream, long* groups = nullptr, const UnpackJob& job = {}) {
  GemmArgs a = gemm_args(p, q, ldq, pm, ldp, e, slices);
  set_tiles(p, a);
  if (groups) *groups = gated_back_groups(p.rows, p.plan.tile_r);
  hipError_t r;
  if (p.plan.few) r = launch_few(a, p.epi, p.dtype, stream);
  else if (p.dtype == OIDN_F32) r = launch_gemm32(a, p.plan, p.epi, job, stream);
  else if (p.epi == kEpiGatedBack) r = launch_gemm16_gated_back(a, p.plan, p.dtype == OIDN_BF16, job, stream);
  else r = launch_gemm16_forward(a, p.plan, p.epi, p.dtype == OIDN_BF16, stream);
  OIDN_TRY(ran(r, "matrix product launch"));
  if (p.plan.splits > 1)
    OIDN_TRY(ran(launch_split_sum(a.e, p.plan.splits, p.dtype, stream), "slice sum launch"));
  return OIDN_OK;
}

// The products that end a backward pass.  They run together in one launch
// where they can share a kernel (same tile, operands alike), and what is left
// to sum after them goes into `finish`.
struct Gradients {
  int dtype;
  int count;
  Product p[kMaxGroup];
  GemmArgs a[kMaxGroup];
  FinishArgs finish;
  bool summing;            // sums is to run (its column sums alone)
  SlopeArgs sums;
  void add(const Product& pr, const void* q, long ldq, const void* pm, long ldp, const EpilogueArgs& e,
           void* slices) {
    p[count] = pr;
    a[count] = gemm_args(p[count], q, ldq, pm, ldp, e, slices);
    ++count;
  }
  void add_slices(const EpilogueArgs& e, int splits) {
    finish.product[finish.products].e = e;
    finish.product[finish.products++].splits = splits;
  }
  void add_columns(const void* part, long groups, int cols, float* out) {
    auto& c = finish.column[finish.columns++];
    c.part = static_cast<const float*>(part);
    c.groups = groups;
    c.cols = cols;
    c.out = out;
  }
  // Column sums of dy (rows x cols) into out, through `part` (chunk by chunk).
  void sum_columns(const void* dy, long lddy, long rows, int cols, long chunk, void* part, float* out) {
    const long chunks = (rows + chunk - 1) / chunk;
    sums = SlopeArgs{};
    sums.dy = dy;
    sums.lddy = lddy;
    sums.part = chunks > 1 ? static_cast<float*>(part) : out;     // one chunk: the sums themselves
    sums.rows = rows;
    sums.cols = cols;
    sums.chunk = chunk;
    sums.lanes = slope_lanes(cols);
    sums.act = OIDN_ACT_NONE;
    summing = true;
    if (chunks > 1) add_columns(part, chunks, cols, out);
  }
  int run(hipStream_t stream) {
    bool done[kMaxGroup] = {};
    for (int first = 0; first < count; ++first) {
      if (done[first]) continue;
      const GemmPlan& plan = p[first].plan;
      GemmGroup g{};
      for (int k = first; k < count; ++k) {
        if (done[k] || p[k].plan.tile_r != plan.tile_r || p[k].plan.direct != plan.direct) continue;
        done[k] = true;
        set_tiles(p[k], a[k]);
        g.start[g.count] = g.blocks;
        g.blocks += (int)gemm_blocks(a[k]);
        g.layout[g.count] = p[k].layout;
        g.a[g.count++] = a[k];
        if (p[k].plan.splits > 1) add_slices(a[k].e, p[k].plan.splits);
      }
      g.sums_start = g.blocks;
      if (summing) {
        g.sums = sums;
        g.blocks += (int)slope_blocks(sums);
        summing = false;
      }
      OIDN_TRY(ran(dtype == OIDN_F32 ? launch_gemm32_group(g, plan, stream)
                                     : launch_gemm16_group(g, plan, dtype == OIDN_BF16, stream),
                   "gradient products launch"));
    }
    if (summing) OIDN_TRY(ran(launch_slope(sums, {}, dtype, stream), "column sum launch"));
    return ran(launch_finish(finish, dtype, stream), "sums launch");
  }
};

// ---------------------------------------------------------------- linear
struct LinearBack {
  bool narrow;             // one pass over the rows (launch_narrow_back)
  Product dx, dw;
  long chunk, chunks;
  void *dz, *x, *sums, *dx_slices, *dw_slices;
  size_t bytes;
};
LinearBack linear_back(long m, int k, int n, int act, int dtype, unsigned flags, void* ws) {
  LinearBack b{};
  if (dtype != OIDN_F32 && flags == 0 && narrow_layer(m, n, k)) {
    b.narrow = true;
    const size_t grid = narrow_grid(m, n, k);
    Regions r{static_cast<char*>(ws), 0};
    b.sums = r.take(align256(grid * n * sizeof(float)));
    b.dw_slices = grid > 1 ? r.take(align256(grid * n * k * sizeof(float))) : nullptr;
    b.bytes = r.used;
    return b;
  }
  b.dx = Product{kInputGrad, kEpiStore, m, k, n, dtype, {}};
  b.dw = Product{kWeightGrad, kEpiStore, n, k, m, dtype, {}};
  Product* const both[] = {&b.dw, &b.dx};
  plan_together(both, 2);
  b.chunk = slope_chunk(m);
  b.chunks = (m + b.chunk - 1) / b.chunk;
  Regions r{static_cast<char*>(ws), 0};
  b.dz = act != OIDN_ACT_NONE ? r.take(bytes_of(m, n, dtype)) : nullptr;
  b.x = flags & OIDN_X_CKPT8 ? r.take(bytes_of(m, k, dtype)) : nullptr;
  b.sums = r.take(align256(b.chunks * (size_t)n * sizeof(float)));
  b.dx_slices = r.take(product_bytes(b.dx));
  b.dw_slices = r.take(product_bytes(b.dw));
  b.bytes = r.used;
  return b;
}

int check_linear(long m, int k, int n, int dtype) {
  OIDN_TRY(check_type(dtype));
  OIDN_TRY(check_size("x", m, k));
  OIDN_TRY(check_size("y", m, n));
  return check_size("w", n, k);
}

// ------------------------------------------------------------------- ffn
struct Ffn {
  Product in, out;
  void *h, *slices;
  size_t bytes;
  long launch;             // workgroups of the largest launch, at most
};
Ffn ffn_plan(long m, int d, int f, int dtype, void* ws) {
  Ffn p{};
  p.in = product(kForward, kEpiGated, m, f, d, dtype);
  p.out = product(kForward, kEpiLinear, m, d, f, dtype);
  Regions r{static_cast<char*>(ws), 0};
  p.h = r.take(bytes_of(m, f, dtype));
  p.slices = r.take(product_bytes(p.out));
  p.bytes = r.used;
  p.launch = std::max({most_blocks(p.in), most_blocks(p.out), sum_blocks(p.out)});
  return p;
}

struct FfnBack {
  Product dh, dx, dw_in, dw_out;
  long groups, chunk, chunks;
  void *h, *dz, *x, *in_sums, *out_sums, *dx_slices, *in_slices, *out_slices;
  size_t bytes;
};
FfnBack ffn_back(long m, int d, int f, int dtype, unsigned flags, void* ws) {
  FfnBack b{};
  b.dh = product(kInputGrad, kEpiGatedBack, m, f, d, dtype);
  b.dx = Product{kInputGrad, kEpiStore, m, d, 2L * f, dtype, {}};
  b.dw_in = Product{kWeightGrad, kEpiStore, 2L * f, d, m, dtype, {}};
  b.dw_out = Product{kWeightGrad, kEpiStore, d, f, m, dtype, {}};
  Product* const all[] = {&b.dw_in, &b.dw_out, &b.dx};
  plan_together(all, 3);
  b.groups = gated_back_groups(m, kMinTile);
  b.chunk = slope_chunk(m);
  b.chunks = (m + b.chunk - 1) / b.chunk;
  Regions r{static_cast<char*>(ws), 0};
  b.h = r.take(bytes_of(m, f, dtype));
  b.dz = r.take(bytes_of(m, 2L * f, dtype));
  b.x = flags & OIDN_X_CKPT8 ? r.take(bytes_of(m, d, dtype)) : nullptr;
  b.in_sums = r.take(align256(b.groups * 2 * (size_t)f * sizeof(float)));
  b.out_sums = r.take(align256(b.chunks * (size_t)d * sizeof(float)));
  b.dx_slices = r.take(product_bytes(b.dx));
  b.in_slices = r.take(product_bytes(b.dw_in));
  b.out_slices = r.take(product_bytes(b.dw_out));
  b.bytes = r.used;
  return b;
}

int check_ffn(long m, int d, int f, int dtype) {
  OIDN_TRY(check_type(dtype));
  OIDN_TRY(check_size("x", m, d));
  if (f < 1 || f > kMaxColumns / 2)
    return fail(f < 1 ? OIDN_E_INVALID : OIDN_E_UNSUPPORTED, "hidden width %d is out of range", f);
  OIDN_TRY(check_size("z", m, 2L * f));
  return check_size("w_in", 2L * f, d);
}

}  // namespace

namespace oidn {

// Launch plans come from what the kernels were measured to take (us, one
// MI355X, 256 compute units; q = tiles per compute unit, kt = staged tiles of
// the summed length; 4096 x 1024 and 4096 x 4096 outputs, kt 1 to 32):
//   64 x 64     3.5 + 0.27 kt at q = 1,  5.0 + 0.76 kt at q = 4,  14 + 2.6 kt at q = 16
//   128 x 128   6.2 + 0.49 kt at q = 1,  15 + 1.6 kt at q = 4
//   256 x 256   16 + 1.4 kt at q = 1,    19 + 2.9 kt at q = 2
// that is, a start, a cost per tile, and per staged tile the larger of a
// workgroup's own pace and its share of the compute unit's.  fp32 tiles (64 x
// 64) hold half as many summed elements and take 0.8 us alone, 0.53 us of a
// full unit; 32 x 64 ones, for a lone plain product, give two workgroups to a unit
// that would hold one.  Summing slices costs a launch and moves their bytes twice.
struct TileCost { long tile; double start, each, own, share; };
constexpr TileCost kCost16[] = {{64, 2.8, 0.7, 0.27, 0.17}, {128, 3.4, 2.9, 0.49, 0.40}, {256, 6.5, 9.0, 1.35, 1.40}};
constexpr TileCost kCostGated = {64, 2.8, 1.3, 0.35, 0.30};      // a gated product's 64 x 128
constexpr TileCost kCost32[] = {{64, 3.5, 1.0, 0.80, 0.53}, {32, 3.0, 0.7, 0.50, 0.30}};
constexpr long kMaxSlices = 256;
constexpr double kCus = 256, kSliceLaunch = 3.0, kSliceBytesPerUs = 4e6;

void plan_products(GemmPlan* const* plans, const PlanShape* shapes, int count, int dtype, bool direct) {
  const long bk = dtype == OIDN_F32 ? kDenseKF32 : kDenseK;
  const TileCost* const table = dtype == OIDN_F32 ? kCost32 : kCost16;
  const int choices = dtype == OIDN_F32 ? (shapes[0].epi == kEpiLinear ? 2 : 1) : direct ? 3 : 2;
  double best = 0;
  for (int c = 0; c < choices; ++c) {
    const TileCost t = shapes[0].epi == kEpiGated && table[c].tile == 64 ? kCostGated : table[c];
    // Smaller tiles' epilogues run beside other workgroups' multiplications: gelu added 0.13 of
    // what it added to a 256 x 256 tile to a 128 x 128 one, 0.025 to a 64 x 64 one.  With these
    // shares themselves 128 x 128 lost to 256 x 256 where it is faster (8-bit, 8192 x 256 -> 4096
    // with silu 49.5 us for 43.0).
    const double each = t.each + shapes[0].extra * (t.tile == 256 ? 1.0 : t.tile == 128 ? 0.16 : 0.05);
    long tiles[kMaxGroup], kt[kMaxGroup], longest = 1;
    for (int k = 0; k < count; ++k) {
      const PlanShape& s = shapes[k];
      // a gated tile holds half its columns of each projection, 64 at least
      const long tc = s.epi == kEpiGated ? (t.tile < 128 ? 64 : t.tile / 2) : t.tile < 64 ? 64 : t.tile;
      tiles[k] = ((s.rows + t.tile - 1) / t.tile) * ((s.cols + tc - 1) / tc);
      kt[k] = (s.len + bk - 1) / bk;
      if (kt[k] > longest) longest = kt[k];
    }
    // slices of at most `cap` staged tiles, from none down to two tiles each
    for (long cap = longest; cap >= 1; cap = cap * 3 / 4) {
      GemmPlan tried[kMaxGroup];
      double work = 0, number = 0, slices = 0, own = 0;
      for (int k = 0; k < count; ++k) {
        const PlanShape& s = shapes[k];
        GemmPlan& p = tried[k];
        p = GemmPlan{(int)t.tile, s.epi == kEpiGated && t.tile < 128 ? 128 : t.tile < 64 ? 64 : (int)t.tile, false, false, 1, kt[k]};
        if ((s.epi == kEpiLinear || s.epi == kEpiStore) && kt[k] > cap && cap >= 2) {
          long n = (kt[k] + cap - 1) / cap;
          if (n > kMaxSlices) n = kMaxSlices;
          p.per_split = (kt[k] + n - 1) / n;
          p.splits = (int)((kt[k] + p.per_split - 1) / p.per_split);
          if (p.splits > 1) slices += (double)p.splits * s.rows * s.cols * 8 / kSliceBytesPerUs;
        }
        number += (double)tiles[k] * p.splits;
        work += (double)tiles[k] * kt[k];
        if (t.own * p.per_split > own) own = t.own * p.per_split;
      }
      // a lone product goes in whole rounds; several fill each other's last one
      double q = number / kCus;
      if (count == 1 || q < 1) {
        const double whole = (double)(long)((number + kCus - 1) / kCus);
        work *= whole / q;
        q = whole;
      }
      const double pace = t.share * work / kCus;
      const double cost = t.start + each * q + (pace > own ? pace : own) + (slices > 0 ? kSliceLaunch + slices : 0);
      if (best == 0 || cost < best) {
        best = cost;
        for (int k = 0; k < count; ++k) *plans[k] = tried[k];
      }
      if (cap < 3) break;
    }
  }
}

}  // namespace oidn

extern "C" {

// ------------------------------------------------------------ checkpoints
int oidn_ckpt_bytes(long m, long n, size_t* bytes) {
  if (!bytes) return fail(OIDN_E_INVALID, "null bytes pointer");
  OIDN_TRY(check_size("checkpoint", m, n));
  *bytes = ckpt_bytes(m, n);
  return clear_error();
}

int oidn_ckpt_pack(const void* x, long ldx, long m, long n, void* ckpt, int dtype, hipStream_t stream) {
  OIDN_TRY(check_type(dtype));
  OIDN_TRY(check_size("x", m, n));
  if (m == 0) return clear_error();
  OIDN_TRY(check_matrix("x", x, ldx, n, dtype, false));
  OIDN_TRY(check_blob("checkpoint", ckpt));
  OIDN_TRY(ran(launch_ckpt_pack(x, ldx, m, n, ckpt, dtype, stream), "checkpoint pack launch"));
  return clear_error();
}

int oidn_ckpt_unpack(const void* ckpt, long m, long n, void* y, long ldy, int dtype, hipStream_t stream) {
  OIDN_TRY(check_type(dtype));
  OIDN_TRY(check_size("y", m, n));
  if (m == 0) return clear_error();
  OIDN_TRY(check_matrix("y", y, ldy, n, dtype, false));
  OIDN_TRY(check_blob("checkpoint", ckpt));
  OIDN_TRY(ran(launch_ckpt_unpack(ckpt, m, n, y, ldy, dtype, stream), "checkpoint unpack launch"));
  return clear_error();
}

// ----------------------------------------------------------------- linear
int oidn_linear_workspace_bytes(long m, int k, int n, int dtype, size_t* bytes) {
  if (!bytes) return fail(OIDN_E_INVALID, "null bytes pointer");
  OIDN_TRY(check_linear(m, k, n, dtype));
  *bytes = 0;
  if (m) {
    const Product p = product(kForward, kEpiLinear, m, n, k, dtype);
    OIDN_TRY(check_launch(std::max(most_blocks(p), sum_blocks(p))));
    *bytes = product_bytes(p);
  }
  return clear_error();
}

int oidn_linear(const void* x, long ldx, const void* w, long ldw, const float* bias,
                const void* residual, long ldr, void* y, long ldy, void* z, long ldz, long m, int k,
                int n, int act, int dtype, unsigned flags, void* workspace, size_t ws_bytes,
                hipStream_t stream) {
  OIDN_TRY(check_linear(m, k, n, dtype));
  OIDN_TRY(check_act(act));
  OIDN_TRY(check_flags(flags, OIDN_Z_CKPT8));
  if (m == 0) return clear_error();
  const bool z8 = flags & OIDN_Z_CKPT8;
  OIDN_TRY(check_matrix("x", x, ldx, k, dtype, false));
  OIDN_TRY(check_matrix("w", w, ldw, k, dtype, false));
  OIDN_TRY(check_aligned("bias", bias, 4));
  OIDN_TRY(check_matrix("residual", residual, ldr, n, dtype, true));
  OIDN_TRY(check_matrix("y", y, ldy, n, dtype, false));
  if (z8) OIDN_TRY(check_blob("z", z));
  else OIDN_TRY(check_matrix("z", z, ldz, n, dtype, true));
  const Product p = product(kForward, kEpiLinear, m, n, k, dtype);
  OIDN_TRY(check_launch(std::max(most_blocks(p), sum_blocks(p))));
  OIDN_TRY(check_workspace(workspace, ws_bytes, product_bytes(p)));
  EpilogueArgs e = store_to(y, ldy, residual, ldr);
  e.bias = bias;
  e.z = z;
  e.ldz = ldz;
  e.z8 = z8;
  e.act = act;
  OIDN_TRY(run_product(p, x, ldx, w, ldw, e, workspace, stream));
  return clear_error();
}

int oidn_linear_backward_workspace_bytes(long m, int k, int n, int act, int dtype, unsigned flags,
                                         size_t* bytes) {
  if (!bytes) return fail(OIDN_E_INVALID, "null bytes pointer");
  OIDN_TRY(check_linear(m, k, n, dtype));
  OIDN_TRY(check_act(act));
  OIDN_TRY(check_flags(flags, OIDN_X_CKPT8 | OIDN_Z_CKPT8));
  *bytes = m ? linear_back(m, k, n, act, dtype, flags, nullptr).bytes : 0;
  return clear_error();
}

int oidn_linear_backward(const void* dy, long lddy, const void* x, long ldx, const void* z, long ldz,
                         const void* w, long ldw, void* dx, long lddx, void* dw, long lddw,
                         float* dbias, long m, int k, int n, int act, int dtype, unsigned flags,
                         void* workspace, size_t ws_bytes, hipStream_t stream) {
  OIDN_TRY(check_linear(m, k, n, dtype));
  OIDN_TRY(check_act(act));
  OIDN_TRY(check_flags(flags, OIDN_X_CKPT8 | OIDN_Z_CKPT8));
  const bool x8 = flags & OIDN_X_CKPT8, z8 = flags & OIDN_Z_CKPT8, slope = act != OIDN_ACT_NONE;
  OIDN_TRY(check_matrix("dw", dw, lddw, k, dtype, true));
  OIDN_TRY(check_aligned("dbias", dbias, 4));
  if (m == 0) {
    // sums over no rows
    const size_t es = esize(dtype);
    if (dw) OIDN_TRY(ran(launch_zero(dw, n, k * es, lddw * es, stream), "zero launch"));
    if (dbias) OIDN_TRY(ran(launch_zero(dbias, 1, n * sizeof(float), 0, stream), "zero launch"));
    return clear_error();
  }
  OIDN_TRY(check_matrix("dy", dy, lddy, n, dtype, false));
  if (dw) {
    if (x8) OIDN_TRY(check_blob("x", x));
    else OIDN_TRY(check_matrix("x", x, ldx, k, dtype, false));
  }
  if (slope) {
    if (z8) OIDN_TRY(check_blob("z", z));
    else OIDN_TRY(check_matrix("z", z, ldz, n, dtype, false));
  }
  if (dx) OIDN_TRY(check_matrix("w", w, ldw, k, dtype, false));
  OIDN_TRY(check_matrix("dx", dx, lddx, k, dtype, true));
  LinearBack b = linear_back(m, k, n, act, dtype, flags, workspace);
  const UnpackJob job = dw && x8 && slope ? unpack_job(x, m, k, b.x) : UnpackJob{};
  if (!b.narrow) {
    const long pass = slope_blocks(m, n, b.chunk);
    OIDN_TRY(check_launch(std::max({job.blocks + pass, (dx ? most_blocks(b.dx) : 0) + (dw ? most_blocks(b.dw) : 0) + pass,
                                    sum_blocks(b.dx) + sum_blocks(b.dw) + column_blocks(b.chunks, n)})));
  }
  OIDN_TRY(check_workspace(workspace, ws_bytes, b.bytes));

  Gradients g{};
  g.dtype = dtype;
  if (b.narrow) {
    const int grid = narrow_grid(m, n, k);
    NarrowArgs a{};
    a.dy = dy;
    a.lddy = lddy;
    a.z = z;
    a.ldz = ldz;
    a.x = x;
    a.ldx = ldx;
    a.w = w;
    a.ldw = ldw;
    a.dx = dx;
    a.lddx = lddx;
    a.dw = dw;
    a.lddw = lddw;
    a.slices = static_cast<float*>(b.dw_slices);
    a.sums = dbias && grid > 1 ? static_cast<float*>(b.sums) : dbias;
    a.rows = m;
    a.n = n;
    a.k = k;
    a.blocks = (int)((m + 63) / 64);
    a.act = act;
    if (dx || dw || dbias) OIDN_TRY(ran(launch_narrow_back(a, grid, dtype == OIDN_BF16, stream), "gradients launch"));
    if (grid > 1) {
      if (dw) {
        EpilogueArgs e = store_to(dw, lddw, nullptr, 0);
        e.part = a.slices;
        e.rows = n;
        e.cols = k;
        g.add_slices(e, grid);
      }
      if (dbias) g.add_columns(b.sums, grid, n, dbias);
      OIDN_TRY(g.run(stream));
    }
    return clear_error();
  }
  if (slope) {
    SlopeArgs s{};
    s.dy = dy;
    s.lddy = lddy;
    s.z = z;
    s.ldz = ldz;
    s.z8 = z8;
    s.dz = b.dz;
    s.part = dbias && b.chunks > 1 ? static_cast<float*>(b.sums) : dbias;   // one chunk: the sums themselves
    s.rows = m;
    s.cols = n;
    s.chunk = b.chunk;
    s.lanes = slope_lanes(n);
    s.act = act;
    OIDN_TRY(ran(launch_slope(s, job, dtype, stream), "slope pass launch"));
    if (dbias && b.chunks > 1) g.add_columns(b.sums, b.chunks, n, dbias);
  } else if (dbias) {
    g.sum_columns(dy, lddy, m, n, b.chunk, b.sums, dbias);
  }
  const void* dz = slope ? b.dz : dy;
  const long lddz = slope ? n : lddy;
  if (dw) {
    if (x8) {
      if (!slope) OIDN_TRY(ran(launch_ckpt_unpack(x, m, k, b.x, k, dtype, stream), "checkpoint unpack launch"));
      x = b.x;
      ldx = k;
    }
    g.add(b.dw, dz, lddz, x, ldx, store_to(dw, lddw, nullptr, 0), b.dw_slices);
  }
  if (dx) g.add(b.dx, dz, lddz, w, ldw, store_to(dx, lddx, nullptr, 0), b.dx_slices);
  OIDN_TRY(g.run(stream));
  return clear_error();
}

// -------------------------------------------------------------------- ffn
int oidn_ffn_workspace_bytes(long m, int d, int f, int dtype, size_t* bytes) {
  if (!bytes) return fail(OIDN_E_INVALID, "null bytes pointer");
  OIDN_TRY(check_ffn(m, d, f, dtype));
  *bytes = 0;
  if (m) {
    const Ffn b = ffn_plan(m, d, f, dtype, nullptr);
    OIDN_TRY(check_launch(b.launch));
    *bytes = b.bytes;
  }
  return clear_error();
}

int oidn_ffn(const void* x, long ldx, const void* w_in, const float* b_in, const void* w_out,
             const float* b_out, const void* residual, long ldr, void* y, long ldy, void* z, long m,
             int d, int f, int act, int dtype, unsigned flags, void* workspace, size_t ws_bytes,
             hipStream_t stream) {
  OIDN_TRY(check_ffn(m, d, f, dtype));
  OIDN_TRY(check_act(act));
  OIDN_TRY(check_flags(flags, OIDN_Z_CKPT8));
  if (m == 0) return clear_error();
  const bool z8 = flags & OIDN_Z_CKPT8;
  OIDN_TRY(check_matrix("x", x, ldx, d, dtype, false));
  OIDN_TRY(check_matrix("w_in", w_in, d, d, dtype, false));
  OIDN_TRY(check_matrix("w_out", w_out, f, f, dtype, false));
  OIDN_TRY(check_aligned("b_in", b_in, 4));
  OIDN_TRY(check_aligned("b_out", b_out, 4));
  OIDN_TRY(check_matrix("residual", residual, ldr, d, dtype, true));
  OIDN_TRY(check_matrix("y", y, ldy, d, dtype, false));
  if (z8) OIDN_TRY(check_blob("z", z));
  else OIDN_TRY(check_matrix("z", z, 2L * f, 2L * f, dtype, true));
  const Ffn p = ffn_plan(m, d, f, dtype, workspace);
  OIDN_TRY(check_launch(p.launch));
  OIDN_TRY(check_workspace(workspace, ws_bytes, p.bytes));

  EpilogueArgs e = store_to(p.h, f, nullptr, 0);
  e.bias = b_in;
  e.z = z;
  e.ldz = 2L * f;
  e.z8 = z8;
  e.act = act;
  OIDN_TRY(run_product(p.in, x, ldx, w_in, d, e, nullptr, stream));
  EpilogueArgs o = store_to(y, ldy, residual, ldr);
  o.bias = b_out;
  OIDN_TRY(run_product(p.out, p.h, f, w_out, f, o, p.slices, stream));
  return clear_error();
}

int oidn_ffn_backward_workspace_bytes(long m, int d, int f, int dtype, unsigned flags, size_t* bytes) {
  if (!bytes) return fail(OIDN_E_INVALID, "null bytes pointer");
  OIDN_TRY(check_ffn(m, d, f, dtype));
  OIDN_TRY(check_flags(flags, OIDN_X_CKPT8 | OIDN_Z_CKPT8));
  *bytes = m ? ffn_back(m, d, f, dtype, flags, nullptr).bytes : 0;
  return clear_error();
}

int oidn_ffn_backward(const void* dy, long lddy, const void* x, long ldx, const void* z,
                      const void* w_in, const void* w_out, const void* add, long ldadd, void* dx,
                      long lddx, void* dw_in, float* db_in, void* dw_out, float* db_out, long m, int d,
                      int f, int act, int dtype, unsigned flags, void* workspace, size_t ws_bytes,
                      hipStream_t stream) {
  OIDN_TRY(check_ffn(m, d, f, dtype));
  OIDN_TRY(check_act(act));
  OIDN_TRY(check_flags(flags, OIDN_X_CKPT8 | OIDN_Z_CKPT8));
  const bool x8 = flags & OIDN_X_CKPT8, z8 = flags & OIDN_Z_CKPT8;
  const size_t es = esize(dtype);
  OIDN_TRY(check_matrix("dw_in", dw_in, d, d, dtype, true));
  OIDN_TRY(check_matrix("dw_out", dw_out, f, f, dtype, true));
  OIDN_TRY(check_aligned("db_in", db_in, 4));
  OIDN_TRY(check_aligned("db_out", db_out, 4));
  if (m == 0) {
    // sums over no rows
    if (dw_in) OIDN_TRY(ran(launch_zero(dw_in, 1, 2 * (size_t)f * d * es, 0, stream), "zero launch"));
    if (dw_out) OIDN_TRY(ran(launch_zero(dw_out, 1, (size_t)f * d * es, 0, stream), "zero launch"));
    if (db_in) OIDN_TRY(ran(launch_zero(db_in, 1, 2 * (size_t)f * sizeof(float), 0, stream), "zero launch"));
    if (db_out) OIDN_TRY(ran(launch_zero(db_out, 1, d * sizeof(float), 0, stream), "zero launch"));
    return clear_error();
  }
  const bool inner = dx || dw_in || db_in || dw_out;     // what needs dh
  OIDN_TRY(check_matrix("dy", dy, lddy, d, dtype, false));
  if (dw_in) {
    if (x8) OIDN_TRY(check_blob("x", x));
    else OIDN_TRY(check_matrix("x", x, ldx, d, dtype, false));
  }
  if (inner) {
    if (z8) OIDN_TRY(check_blob("z", z));
    else OIDN_TRY(check_matrix("z", z, 2L * f, 2L * f, dtype, false));
    OIDN_TRY(check_matrix("w_out", w_out, f, f, dtype, false));
  }
  if (dx) OIDN_TRY(check_matrix("w_in", w_in, d, d, dtype, false));
  OIDN_TRY(check_matrix("dx", dx, lddx, d, dtype, true));
  OIDN_TRY(check_matrix("add", add, ldadd, d, dtype, true));
  const FfnBack b = ffn_back(m, d, f, dtype, flags, workspace);
  const UnpackJob job = dw_in && x8 ? unpack_job(x, m, d, b.x) : UnpackJob{};
  OIDN_TRY(check_launch(std::max({(inner ? most_blocks(b.dh) : 0) + job.blocks,
                                  (dx ? most_blocks(b.dx) : 0) + (dw_in ? most_blocks(b.dw_in) : 0) +
                                      (dw_out ? most_blocks(b.dw_out) : 0) + slope_blocks(m, d, b.chunk),
                                  sum_blocks(b.dx) + sum_blocks(b.dw_in) + sum_blocks(b.dw_out) +
                                      column_blocks(b.groups, 2 * f) + column_blocks(b.chunks, d)})));
  OIDN_TRY(check_workspace(workspace, ws_bytes, b.bytes));

  const long f2 = 2L * f;
  Gradients g{};
  g.dtype = dtype;
  if (inner) {
    EpilogueArgs e{};
    e.y = b.dz;
    e.ldy = f2;
    e.h = b.h;
    e.z = const_cast<void*>(z);
    e.ldz = f2;
    e.z8 = z8;
    e.act = act;
    e.part = db_in ? static_cast<float*>(b.in_sums) : nullptr;
    long groups = 0;
    OIDN_TRY(run_product(b.dh, dy, lddy, w_out, f, e, nullptr, stream, &groups, job));
    if (db_in) g.add_columns(e.part, groups, (int)f2, db_in);
  }
  if (db_out) g.sum_columns(dy, lddy, m, d, b.chunk, b.out_sums, db_out);
  // the longest sums first
  if (dw_in) {
    if (x8) {
      x = b.x;
      ldx = d;
    }
    g.add(b.dw_in, b.dz, f2, x, ldx, store_to(dw_in, d, nullptr, 0), b.in_slices);
  }
  if (dw_out) g.add(b.dw_out, dy, lddy, b.h, f, store_to(dw_out, f, nullptr, 0), b.out_slices);
  if (dx) g.add(b.dx, b.dz, f2, w_in, d, store_to(dx, lddx, add, ldadd), b.dx_slices);
  OIDN_TRY(g.run(stream));
  return clear_error();
}

}  // extern "C"
