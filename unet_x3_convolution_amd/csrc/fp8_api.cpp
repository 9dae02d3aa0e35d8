// Host side of the dense layer in 8-bit floating point: argument checks, launch
// plans, workspace layout and the launch sequences.  Nothing here allocates device
// memory, waits for the device or throws.
#include <algorithm>

#include "dense_checks.h"
#include "fp8.h"

using namespace oidn;

namespace {

// A product sums at most so many elements: a tile's 32-bit offsets pass 256 rows.
constexpr long kMaxSummed = 1L << 23;

int check_packed(const char* name, long m, long n) {
  OIDN_TRY(check_size(name, m, n));
  if (fp8_cols(n) > kMaxElements / (m ? m : 1))
    return fail(OIDN_E_UNSUPPORTED, "%s: %ld x %ld is larger than the kernels index", name, m, n);
  return OIDN_OK;
}
int check_layer(long m, int k, int n, int dtype) {
  OIDN_TRY(check_type(dtype));
  if (dtype == OIDN_F32)
    return fail(OIDN_E_UNSUPPORTED, "8-bit products have 16-bit results: OIDN_F16 or OIDN_BF16");
  OIDN_TRY(check_packed("x", m, k));
  OIDN_TRY(check_packed("y", m, n));
  OIDN_TRY(check_packed("w", n, k));
  OIDN_TRY(check_packed("w's transpose", k, n));
  if (std::max(k, n) > kMaxSummed)
    return fail(OIDN_E_UNSUPPORTED, "a layer of %d -> %d channels is larger than the kernels index", k, n);
  return OIDN_OK;
}

struct Product8 {
  long rows, cols, len;    // len: bytes of a row
  int act;
  GemmPlan plan;
};
// Plans products that share a launch, as 16-bit ones of half the length: a staged
// tile has the bytes and the matrix cycles of one of theirs.
void plan_together(Product8* const* p, int count) {
  GemmPlan* plans[kMaxGroup8];
  PlanShape shapes[kMaxGroup8];
  for (int k = 0; k < count; ++k) {
    plans[k] = &p[k]->plan;
    // A 256 x 256 tile's epilogue stands beside a loop half as long as a 16-bit product's: fitted
    // to 8192 x 512 to 4096 -> 4096 (us, 256 x 256 against 128 x 128, none, relu, silu, gelu: 512
    // 40 and 37, 43 and 37, 47 and 40, 58 and 48; 1024 52 and 51, 56 and 53, 62 and 56, 72 and 64;
    // 2048 75 and 78, 79 and 79, 84 and 83, 94 and 89; 4096 119 and 131, 123 and 132, 129 and 136,
    // 136 and 139).  Of 200 layers (2048 to 32640 rows, 256 to 4096 inputs, 448 to 8192 outputs)
    // four got a tile that is over 3% slower than with 0, 2, 5, 10 (32640 x 4096 -> 448 with gelu 90
    // for 80), 60 a faster one (32640 x 1024 -> 448 28 for 44).
    const double extra[] = {7.5, 11.5, 14, 18.5};      // none, relu, silu, gelu
    shapes[k] = {p[k]->rows, p[k]->cols, p[k]->len / 2, kEpiStore, count == 1 ? extra[p[k]->act] : 0};
  }
  plan_products(plans, shapes, count, OIDN_F16, true);
  for (int k = 0; k < count; ++k) {
    const long tiles = p[k]->len / kFp8Block;
    p[k]->plan.per_split = (p[k]->plan.per_split + 3) / 4 * 4;      // whole words of scales
    p[k]->plan.splits = (int)((tiles + p[k]->plan.per_split - 1) / p[k]->plan.per_split);
  }
}
Product8 product8(long rows, long cols, long len, int act = OIDN_ACT_NONE) {
  return Product8{rows, cols, fp8_cols(len), act, {}};
}
size_t slice_bytes(const Product8& p) {
  return p.plan.splits > 1 ? align256((size_t)p.plan.splits * p.rows * p.cols * sizeof(float)) : 0;
}
long tiles_of(long n, const Product8& p) { return (n + p.plan.tile_r - 1) / p.plan.tile_r; }
long most_blocks(const Product8& p) { return gemm_blocks(tiles_of(p.rows, p), tiles_of(p.cols, p), p.plan.splits); }
long sum_blocks(const Product8& p) {
  return p.plan.splits > 1 ? slice_blocks(p.rows, (int)p.cols, p.plan.splits) : 0;
}
Gemm8Args gemm8_args(const Product8& p, const void* q, const void* pm, const EpilogueArgs& e, void* slices) {
  Gemm8Args a{};
  a.g.q = q;
  a.g.p = pm;
  a.g.ldq = a.g.ldp = a.g.len = p.len / 2;
  a.g.tiles_r = (int)tiles_of(p.rows, p);
  a.g.tiles_c = (int)tiles_of(p.cols, p);
  a.g.splits = p.plan.splits;
  a.g.per_split = p.plan.per_split;
  a.g.e = e;
  a.g.e.rows = p.rows;
  a.g.e.cols = (int)p.cols;
  a.g.e.stream = stream_result(p.rows, p.cols);
  if (p.plan.splits > 1) a.g.e.part = static_cast<float*>(slices);
  a.qs = static_cast<const unsigned char*>(q) + p.rows * p.len;
  a.ps = static_cast<const unsigned char*>(pm) + p.cols * p.len;
  a.qn = a.pn = fp8_scales(p.len);
  return a;
}

struct Forward {
  bool narrow;             // at most kFp8Block inputs, not packed: one launch
  bool few;                // else at most kFewRows rows: the product in one launch
  bool pack;               // x is packed first
  Product8 p;
  void *x8, *slices;
  size_t bytes;
};
Forward forward(long m, int k, int n, int act, unsigned flags, void* ws) {
  Forward f{};
  f.p = product8(m, n, k, act);
  const bool x8 = flags & OIDN_X_FP8;
  f.narrow = !x8 && k <= kFp8Block && m > kCodedRows;
  f.few = !f.narrow && m <= kFewRows;
  f.pack = !x8 && !f.narrow && m > kCodedRows;
  Product8* one = &f.p;
  if (f.narrow) {
    // one staged tile: 128 x 128 where they fill the units and none is half empty (us, 64 x 64
    // and 128 x 128: 16384 x 128 -> 512 with gelu 17.7 and 16.4, 32640 x 96 -> 1024 plain 34.4 and
    // 31.8; 384 tiles, 16384 x 96 -> 384 with gelu 14.7 and 16.0; half empty ones, 65536 x 64 ->
    // 64 11.4 and 15.7, 130560 x 96 -> 160 43 and 55, 65536 x 96 -> 448 53 and 57; from 1500
    // tiles on they are even with an activation, and 0 to 8% ahead without)
    const bool whole = (n + 63l) / 64 % 2 == 0;
    const int tile = whole && ((m + 127) / 128) * ((n + 127l) / 128) >= 512 ? 128 : 64;
    f.p.plan = GemmPlan{tile, tile, false, true, 1, 4};
  } else if (f.few) f.p.plan = GemmPlan{64, 64, true, true, 1, 0};
  else plan_together(&one, 1);
  Regions r{static_cast<char*>(ws), 0};
  f.x8 = f.pack ? r.take(fp8_bytes(m, k)) : nullptr;
  f.slices = r.take(slice_bytes(f.p));
  f.bytes = r.used;
  return f;
}
int check_forward_launch(const Forward& f, long m, int k) {
  return check_launch(std::max({f.few ? 0 : most_blocks(f.p), sum_blocks(f.p), f.pack ? fp8_pack_blocks(m, k) : 0}));
}

struct Backward {
  Product8 dx, dw;
  void *dz, *dzt, *xt, *sums, *dx_slices, *dw_slices;
  size_t bytes;
};
Backward backward(long m, int k, int n, unsigned flags, void* ws) {
  Backward b{};
  b.dx = product8(m, k, n);
  b.dw = product8(n, k, m);
  Product8* const both[] = {&b.dw, &b.dx};
  plan_together(both, 2);
  Regions r{static_cast<char*>(ws), 0};
  b.dz = r.take(fp8_bytes(m, n));
  b.dzt = r.take(fp8_bytes(n, m));
  b.xt = flags & OIDN_X_FP8 ? nullptr : r.take(fp8_bytes(k, m));
  b.sums = r.take(align256((size_t)((m + kFp8Block - 1) / kFp8Block) * n * sizeof(float)));
  b.dx_slices = r.take(slice_bytes(b.dx));
  b.dw_slices = r.take(slice_bytes(b.dw));
  b.bytes = r.used;
  return b;
}

}  // namespace

extern "C" {

int oidn_fp8_bytes(long m, long n, size_t* bytes) {
  if (!bytes) return fail(OIDN_E_INVALID, "null bytes pointer");
  OIDN_TRY(check_packed("packed matrix", m, n));
  *bytes = fp8_bytes(m, n);
  return clear_error();
}

int oidn_fp8_pack(const void* x, long ldx, long m, long n, void* packed, void* packed_t, int dtype, unsigned flags,
                  hipStream_t stream) {
  OIDN_TRY(check_type(dtype));
  OIDN_TRY(check_packed("x", m, n));
  OIDN_TRY(check_flags(flags, OIDN_FP8_SQUARE));
  if (m > kMaxColumns && packed_t)
    return fail(OIDN_E_UNSUPPORTED, "a transpose of %ld columns is larger than the kernels index", m);
  if (m == 0) return clear_error();
  OIDN_TRY(check_matrix("x", x, ldx, n, dtype, false));
  if (!packed && !packed_t) return fail(OIDN_E_INVALID, "null pointer: packed and packed_t");
  OIDN_TRY(check_aligned("packed", packed, 16));
  OIDN_TRY(check_aligned("packed_t", packed_t, 16));
  OIDN_TRY(check_launch(fp8_pack_blocks(m, n)));
  Fp8PackArgs a{};
  a.x = x;
  a.ldx = ldx;
  a.m = m;
  a.n = (int)n;
  a.rows = packed;
  a.turned = packed_t;
  a.square = flags & OIDN_FP8_SQUARE ? 1 : 0;
  OIDN_TRY(ran(launch_fp8_pack(a, {}, dtype, stream), "8-bit pack launch"));
  return clear_error();
}

int oidn_fp8_unpack(const void* packed, long m, long n, void* y, long ldy, int dtype, hipStream_t stream) {
  OIDN_TRY(check_type(dtype));
  OIDN_TRY(check_packed("y", m, n));
  if (m == 0) return clear_error();
  OIDN_TRY(check_matrix("y", y, ldy, n, dtype, false));
  OIDN_TRY(check_blob("packed", packed));
  OIDN_TRY(ran(launch_fp8_unpack(packed, m, n, y, ldy, dtype, stream), "8-bit unpack launch"));
  return clear_error();
}

int oidn_linear_fp8_workspace_bytes(long m, int k, int n, int dtype, unsigned flags, size_t* bytes) {
  if (!bytes) return fail(OIDN_E_INVALID, "null bytes pointer");
  OIDN_TRY(check_layer(m, k, n, dtype));
  OIDN_TRY(check_flags(flags, OIDN_X_FP8 | OIDN_Z_CKPT8));
  *bytes = 0;
  if (m) {
    // the plan goes by the activation too: enough for each
    for (int act = OIDN_ACT_NONE; act <= OIDN_ACT_GELU; ++act) {
      const Forward f = forward(m, k, n, act, flags, nullptr);
      OIDN_TRY(check_forward_launch(f, m, k));
      *bytes = std::max(*bytes, f.bytes);
    }
  }
  return clear_error();
}

int oidn_linear_fp8(const void* x, long ldx, const void* w8, const float* bias, const void* residual, long ldr, void* y,
                    long ldy, void* z, long ldz, long m, int k, int n, int act, int dtype, unsigned flags,
                    void* workspace, size_t ws_bytes, hipStream_t stream) {
  OIDN_TRY(check_layer(m, k, n, dtype));
  OIDN_TRY(check_act(act));
  OIDN_TRY(check_flags(flags, OIDN_X_FP8 | OIDN_Z_CKPT8));
  if (m == 0) return clear_error();
  const bool x8 = flags & OIDN_X_FP8, z8 = flags & OIDN_Z_CKPT8;
  if (x8) OIDN_TRY(check_blob("x", x));
  else OIDN_TRY(check_matrix("x", x, ldx, k, dtype, false));
  OIDN_TRY(check_blob("w8", w8));
  OIDN_TRY(check_aligned("bias", bias, 4));
  OIDN_TRY(check_matrix("residual", residual, ldr, n, dtype, true));
  OIDN_TRY(check_matrix("y", y, ldy, n, dtype, false));
  if (z8) OIDN_TRY(check_blob("z", z));
  else OIDN_TRY(check_matrix("z", z, ldz, n, dtype, true));
  const Forward f = forward(m, k, n, act, flags, workspace);
  OIDN_TRY(check_forward_launch(f, m, k));
  OIDN_TRY(check_workspace(workspace, ws_bytes, f.bytes));
  if (f.pack) {
    Fp8PackArgs a{};
    a.x = x;
    a.ldx = ldx;
    a.m = m;
    a.n = k;
    a.rows = f.x8;
    OIDN_TRY(ran(launch_fp8_pack(a, {}, dtype, stream), "8-bit pack launch"));
    x = f.x8;
  }
  EpilogueArgs e = store_to(y, ldy, residual, ldr);
  e.bias = bias;
  e.z = z;
  e.ldz = ldz;
  e.z8 = z8;
  e.act = act;
  Gemm8Args g = gemm8_args(f.p, x, w8, e, f.slices);
  if (f.narrow) {
    g.g.ldq = ldx;
    OIDN_TRY(ran(launch_narrow8(g, k, f.p.plan.tile_r, dtype == OIDN_BF16, stream), "8-bit product launch"));
    return clear_error();
  }
  if (f.few) {
    const bool packed = x8 || f.pack;
    if (!packed) g.g.ldq = ldx;
    OIDN_TRY(ran(launch_few8(g, k, packed, dtype == OIDN_BF16, stream), "8-bit product launch"));
    return clear_error();
  }
  OIDN_TRY(ran(launch_gemm8(g, f.p.plan.tile_r, dtype == OIDN_BF16, stream), "8-bit product launch"));
  if (f.p.plan.splits > 1)
    OIDN_TRY(ran(launch_split_sum(g.g.e, f.p.plan.splits, dtype, stream), "slice sum launch"));
  return clear_error();
}

int oidn_linear_fp8_backward_workspace_bytes(long m, int k, int n, int act, int dtype, unsigned flags, size_t* bytes) {
  if (!bytes) return fail(OIDN_E_INVALID, "null bytes pointer");
  OIDN_TRY(check_layer(m, k, n, dtype));
  OIDN_TRY(check_act(act));
  OIDN_TRY(check_flags(flags, OIDN_X_FP8 | OIDN_Z_CKPT8));
  if (m > kMaxSummed) return fail(OIDN_E_UNSUPPORTED, "sums over %ld rows are longer than the kernels index", m);
  *bytes = m ? backward(m, k, n, flags, nullptr).bytes : 0;
  return clear_error();
}

int oidn_linear_fp8_backward(const void* dy, long lddy, const void* x, long ldx, const void* z, long ldz,
                             const void* w8t, void* dx, long lddx, void* dw, long lddw, float* dbias, long m, int k,
                             int n, int act, int dtype, unsigned flags, void* workspace, size_t ws_bytes,
                             hipStream_t stream) {
  OIDN_TRY(check_layer(m, k, n, dtype));
  OIDN_TRY(check_act(act));
  OIDN_TRY(check_flags(flags, OIDN_X_FP8 | OIDN_Z_CKPT8));
  if (m > kMaxSummed) return fail(OIDN_E_UNSUPPORTED, "sums over %ld rows are longer than the kernels index", m);
  const bool x8 = flags & OIDN_X_FP8, z8 = flags & OIDN_Z_CKPT8, slope = act != OIDN_ACT_NONE;
  OIDN_TRY(check_matrix("dw", dw, lddw, k, dtype, true));
  OIDN_TRY(check_aligned("dbias", dbias, 4));
  if (m == 0) {
    // sums over no rows
    if (dw) OIDN_TRY(ran(launch_zero(dw, n, k * esize(dtype), lddw * esize(dtype), stream), "zero launch"));
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
  if (dx) OIDN_TRY(check_blob("w8t", w8t));
  OIDN_TRY(check_matrix("dx", dx, lddx, k, dtype, true));
  const Backward b = backward(m, k, n, flags, workspace);
  const long row_blocks = (m + kFp8Block - 1) / kFp8Block;
  OIDN_TRY(check_launch(std::max({fp8_pack_blocks(m, n) + (dw && !x8 ? fp8_pack_blocks(m, k) : 0),
                                  (dx ? most_blocks(b.dx) : 0) + (dw ? most_blocks(b.dw) : 0) + column_blocks(row_blocks, n),
                                  sum_blocks(b.dx) + sum_blocks(b.dw) + column_blocks(row_blocks, n)})));
  OIDN_TRY(check_workspace(workspace, ws_bytes, b.bytes));
  if (!dx && !dw && !dbias) return clear_error();

  Fp8PackArgs d{}, t{};
  d.x = dy;
  d.ldx = lddy;
  d.z = slope ? z : nullptr;
  d.ldz = ldz;
  d.z8 = z8;
  d.act = act;
  d.m = m;
  d.n = n;
  d.rows = dx ? b.dz : nullptr;
  d.turned = dw ? b.dzt : nullptr;
  d.sums = !dbias ? nullptr : row_blocks > 1 ? static_cast<float*>(b.sums) : dbias;     // one block: the sums themselves
  if (dw && !x8) {
    t.x = x;
    t.ldx = ldx;
    t.m = m;
    t.n = k;
    t.turned = b.xt;
  }
  OIDN_TRY(ran(launch_fp8_pack(d, t, dtype, stream), "8-bit pack launch"));

  FinishArgs finish{};
  Gemm8Group g{};
  int blocks = 0;
  auto add = [&](const Product8& p, const void* q, const void* pm, void* out, long ld, void* slices) {
    g.start[g.count] = blocks;
    g.a[g.count] = gemm8_args(p, q, pm, store_to(out, ld, nullptr, 0), slices);
    blocks += (int)gemm_blocks(g.a[g.count].g);
    if (p.plan.splits > 1) {
      finish.product[finish.products].e = g.a[g.count].g.e;
      finish.product[finish.products++].splits = p.plan.splits;
    }
    ++g.count;
  };
  if (dw) add(b.dw, b.dzt, x8 ? x : b.xt, dw, lddw, b.dw_slices);
  if (dx) add(b.dx, b.dz, w8t, dx, lddx, b.dx_slices);
  if (dbias && row_blocks > 1) {
    // with the products where there are some: 2048 x 2048 -> 2048 in 42.8 us, in a launch of
    // their own 45.7
    ColumnJob& c = g.count ? g.column : finish.column[finish.columns++];
    c.part = static_cast<const float*>(b.sums);
    c.groups = row_blocks;
    c.cols = n;
    c.out = dbias;
  }
  if (g.count)
    OIDN_TRY(ran(launch_gemm8_group(g, blocks, b.dx.plan.tile_r, dtype == OIDN_BF16, stream), "8-bit gradients launch"));
  OIDN_TRY(ran(launch_finish(finish, dtype, stream), "sums launch"));
  return clear_error();
}

}  // extern "C"
