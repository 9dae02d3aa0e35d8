// Internal declarations of the dense operators over activation rows: matrix
// products with fused epilogues, the gated feed-forward block, and 8-bit
// activation checkpoints.
#pragma once

#include "internal.h"

namespace oidn {

// ---------------------------------------------------------------------------
// 8-bit checkpoint of an m x n matrix: int8 codes, rows padded to whole blocks
// of 32 columns, then one bf16 scale per row and block.
// ---------------------------------------------------------------------------
constexpr int kCkptBlock = 32;
inline long ckpt_cols(long n) { return (n + kCkptBlock - 1) / kCkptBlock * kCkptBlock; }
inline size_t ckpt_bytes(long m, long n) {
  const size_t codes = (size_t)m * (size_t)ckpt_cols(n);
  return align256(codes + codes / (kCkptBlock / 2));
}

// ---------------------------------------------------------------------------
// Products C[i][j] = sum_l Q(i, l) P(j, l), i < rows, j < cols, l < len.
// An operand is either stored with l fastest (element (i, l) at i * ld + l) or
// "strided" (element (i, l) at l * ld + i):
//   forward  y = x w^T:    Q = x, P = w            both l-fastest
//   input    dx = dz w:    Q = dz, P = w           P strided
//   weight   dw = dz^T x:  Q = dz, P = x           both strided
// ---------------------------------------------------------------------------
enum DenseLayout { kForward = 0, kInputGrad = 1, kWeightGrad = 2 };

// What happens to the sums.
enum DenseEpilogue {
  kEpiLinear = 0,     // bias, saved z, activation, residual, store
  kEpiPartial = 1,    // fp32 sums of one slice of l (any product with splits > 1)
  kEpiGated = 2,      // columns j and f + j of one product: h = act(a) * b
  kEpiGatedBack = 3,  // dh with the saved z: h, da, db and column sums of da, db
  kEpiStore = 4,      // residual, store
};

struct EpilogueArgs {
  const float* bias;       // cols floats (kEpiGated: 2 * cols), may be null
  const void* res;         // rows x cols, row pitch ldr, may be null
  long ldr;
  void* y;                 // rows x cols, row pitch ldy
  long ldy;
  void* z;                 // pre-activation, may be null: row pitch ldz, or checkpoint(s)
  long ldz;
  void* h;                 // kEpiGatedBack: rows x cols, contiguous
  float* part;             // kEpiPartial: [slice][rows][cols]; kEpiGatedBack: column sums or null
  int act;
  int z8;                  // z is held in 8 bits
  int stream;              // kEpiLinear, kEpiStore: stream_result
  long rows;
  int cols;
};
// Whether a 16-bit result goes past the caches.  Two layers one after the other
// (bf16, 32 to 2048 columns, 2 to 160 MB a result; streamed against kept, us): up to
// 18 MB in at most 512 columns 2% slower to 14% faster (64 columns, 16 MB 17.9 and
// 19.6); in 1024 and more, whose rows several tiles read again, 5% faster to 14%
// slower (2048 columns, 2 MB 41 and 36); 20 to 80 MB mostly slower, up to 24% (192
// columns, 64 MB 88 and 71); from 96 MB on 3% slower to 10% faster (1024 columns,
// 112 MB 266 and 278) but for 96 columns (9% slower).  A call by itself may gain by
// it where the next reader loses: 8192 x 4096 -> 4096 231 and 234 alone, 402 and 397
// twice in a row.
inline bool stream_result(long rows, long cols) {
  const long bytes = 2 * rows * cols;
  return (bytes <= 18L << 20 && cols <= 512) || bytes >= 96L << 20;
}

struct GemmArgs {
  const void* q;
  long ldq;
  const void* p;
  long ldp;
  long len;                // summed length
  int tiles_r, tiles_c;    // output tiles
  int splits;              // slices of the summed length
  long per_split;          // K tiles per slice
  EpilogueArgs e;
};

// Tile shape and slices of a launch.
struct GemmPlan {
  int tile_r, tile_c;      // rows and columns of a workgroup's tile
  bool few;                // few rows: launch_few
  bool direct;             // 16-bit: operands go straight from memory to LDS
  int splits;
  long per_split;
};
constexpr int kDenseK = 64;      // summed length of one staged 16-bit tile
constexpr int kDenseKF32 = 32;   // the same in fp32
// Plans `count` (at most kMaxGroup) products that are to share a launch: one
// tile for all, slices for each.  direct: the operands' sizes let them go
// straight to LDS.
struct PlanShape {
  long rows, cols, len;
  int epi;
};
constexpr int kMaxGroup = 3;
void plan_products(GemmPlan* const* plans, const PlanShape* shapes, int count, int dtype, bool direct);
// Row groups of kEpiGatedBack's column sums: one per wave row of every tile.
inline long gated_back_groups(long rows, int tile_r) { return (rows + tile_r - 1) / tile_r * 2; }
constexpr int kMinTile = 64;

// Workgroups of a product: its tiles, rounded up so that every slice starts on
// the first XCD, times its slices.
inline long gemm_blocks(long tiles_r, long tiles_c, int splits) { return (tiles_r * tiles_c + 7) / 8 * 8 * splits; }
inline long gemm_blocks(const GemmArgs& a) { return gemm_blocks(a.tiles_r, a.tiles_c, a.splits); }
// A launch holds less than 2^32 work items, here in workgroups of 256.
constexpr long kMaxWorkgroups = 0xffffffffL / 256;

// dz = dy * act'(z) (dz may be null: column sums alone; act none: z unused)
// and, with part, partial column sums of dz over `chunk` rows: part[r / chunk][n].
struct SlopeArgs {
  const void* dy;
  long lddy;
  const void* z;
  long ldz;
  int z8;
  void* dz;                // contiguous rows x cols
  float* part;
  long rows;
  int cols;
  long chunk;
  int lanes;               // slope_lanes(cols)
  int act;
};

// A checkpoint read back beside another launch's work: blocks workgroups of
// kUnpackRun * 256 units of eight columns each; y is contiguous.
struct UnpackJob {
  const void* ckpt;
  long m;
  int n;
  void* y;
  int blocks;              // 0: none
};
constexpr int kUnpackRun = 4;
inline UnpackJob unpack_job(const void* ckpt, long m, int n, void* y) {
  const long units = m * ((n + 7) / 8), per = kUnpackRun * 256;
  return {ckpt, m, n, y, (int)((units + per - 1) / per)};
}

// Up to three gradients' products in one launch (kEpiStore), the ones with the
// longest tiles first.
struct GemmGroup {
  int count;
  int start[kMaxGroup];      // first workgroup of each
  int layout[kMaxGroup];     // kInputGrad or kWeightGrad
  GemmArgs a[kMaxGroup];
  int sums_start;            // first workgroup of the column sums (the grid's size if there are none)
  int blocks;
  SlopeArgs sums;            // column sums alone
};

// 16-bit: kForward with kEpiLinear or kEpiGated, kInputGrad with kEpiGatedBack.
hipError_t launch_gemm16_forward(const GemmArgs& a, const GemmPlan& p, int epi, bool bf16, hipStream_t stream);
// The latter, and the slope pass, take an unpack job along.
hipError_t launch_gemm16_gated_back(const GemmArgs& a, const GemmPlan& p, bool bf16, const UnpackJob& job,
                                    hipStream_t stream);
// They also run a group's column sums, after its products.
hipError_t launch_gemm16_group(const GemmGroup& g, const GemmPlan& p, bool bf16, hipStream_t stream);
// fp32: the same.
hipError_t launch_gemm32(const GemmArgs& a, const GemmPlan& p, int epi, const UnpackJob& job, hipStream_t stream);
hipError_t launch_gemm32_group(const GemmGroup& g, const GemmPlan& p, hipStream_t stream);
// Forward products (kEpiLinear, kEpiGated) of at most kFewRows rows, in one
// launch without slices.
constexpr int kFewRows = 32;
hipError_t launch_few(const GemmArgs& a, int epi, int dtype, hipStream_t stream);
// Adds a product's slices (e.part) and runs the epilogue (kEpiLinear).
hipError_t launch_split_sum(const EpilogueArgs& e, int splits, int dtype, hipStream_t stream);

// What ends a backward pass, in one launch: sums of products' slices
// (kEpiStore) and of partial column sums, all in a fixed order.
struct FinishArgs {
  int products, columns;
  struct { EpilogueArgs e; int splits; } product[kMaxGroup];
  struct { const float* part; long groups; int cols; float* out; } column[2];
};
hipError_t launch_finish(const FinishArgs& a, int dtype, hipStream_t stream);

// Workgroups that the sum of a product's slices takes, and that of partial columns.
long slice_blocks(long rows, int cols, int splits);
long column_blocks(long groups, int cols);

long slope_chunk(long rows);
int slope_lanes(int cols);
long slope_blocks(const SlopeArgs& a);
hipError_t launch_slope(const SlopeArgs& a, const UnpackJob& job, int dtype, hipStream_t stream);
// All gradients of a narrow 16-bit layer (n, k <= kNarrow) in one pass over its
// rows; `grid` workgroups share the blocks of 64 rows.  dx, dw and sums may be
// null.  With more than one workgroup dw goes to `slices` ([grid][n][k], fp32)
// and the column sums to `sums` ([grid][n]).
constexpr int kNarrow = 128;
struct NarrowArgs {
  const void* dy;
  long lddy;
  const void* z;
  long ldz;
  const void* x;
  long ldx;
  const void* w;
  long ldw;
  void* dx;
  long lddx;
  void* dw;
  long lddw;
  float* slices;
  float* sums;
  long rows;
  int n, k;
  int blocks;              // of 64 rows
  int act;
};
// Whether a layer is narrow.  Where n and k are both over 64 the pass pays from
// 8192 rows on (us, bf16, gelu, 128 x 128: 17 against 14 in separate launches at
// 2040 rows, 20 against 19 at 8160, 26 against 26 at 16320, 55 against 115 at
// 130560); where one is 64 or less it was ahead at every length measured, 64 to
// 130560 rows of 3 -> 32, 8 -> 8, 32 -> 64, 64 -> 16, 64 -> 64, 96 -> 48, 48 -> 96,
// 128 -> 32 and 32 -> 128 (32 -> 64: 10 against 14 at 510 rows, 25 against 61 at
// 130560; the least, 48 -> 96 at 2040 rows, 12.6 against 13.3).
inline bool narrow_layer(long rows, int n, int k) {
  return n <= kNarrow && k <= kNarrow && (n <= 64 || k <= 64 || rows >= 8192);
}
// Workgroups: one per block while units are free for them, then 256 with at
// least two blocks each, for a slice of dw less to write and add (64 x 64, 510
// blocks: 15.9 us against 18.7 with 510), then 512 that hide each other's
// barriers (2040 blocks: 26 against 27, 96 x 48 34 against 44).  128 x 128 takes
// a unit's registers, so there 256 remain (54 against 64).
inline int narrow_grid(long rows, int n, int k) {
  const long b = (rows + 63) / 64;
  return (int)(b <= 256 ? b : b <= 512 || (n > 64 && k > 64) ? 256 : 512);
}
hipError_t launch_narrow_back(const NarrowArgs& a, int grid, bool bf16, hipStream_t stream);

hipError_t launch_ckpt_pack(const void* x, long ldx, long m, long n, void* ckpt, int dtype,
                            hipStream_t stream);
hipError_t launch_ckpt_unpack(const void* ckpt, long m, long n, void* y, long ldy, int dtype,
                              hipStream_t stream);
// Zeros in rows of `width` bytes (a plain store kernel, so that a captured graph
// holds no memset node).
hipError_t launch_zero(void* p, long rows, size_t width, size_t pitch, hipStream_t stream);

}  // namespace oidn
