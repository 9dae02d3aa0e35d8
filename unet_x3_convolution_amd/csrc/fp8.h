// Internal declarations of the dense layer in 8-bit floating point: packed
// matrices and their products.
#pragma once

#include "dense.h"

namespace oidn {

// A packed m x n matrix: e4m3 codes, rows padded with zeros to whole blocks of
// 128 columns, then a byte e + 127 for each row and block, whose codes stand for
// code * 2^e; a row's bytes are padded to whole words of four, as a product reads them.
constexpr int kFp8Block = 128;
inline long fp8_cols(long n) { return (n + kFp8Block - 1) / kFp8Block * kFp8Block; }
inline long fp8_scales(long n) { return (fp8_cols(n) / kFp8Block + 3) / 4 * 4; }
inline size_t fp8_bytes(long m, long n) { return align256((size_t)m * (size_t)(fp8_cols(n) + fp8_scales(n))); }

// Eight-bit forms of x, or of dy act'(z): `rows` (m x n, blocks along a row) and
// `turned` (n x m, blocks along a column) may each be null.
struct Fp8PackArgs {
  const void* x;
  long ldx;
  const void* z;           // null: x itself
  long ldz;
  int z8, act;
  long m;
  int n;
  void* rows;
  void* turned;
  int square;              // a scale for 128 x 128
  float* sums;             // column sums of each 128 rows before coding: [row block][n], may be null
};
long fp8_pack_blocks(long m, long n);      // at most
inline long fp8_tiles(long m, long n) { return ((m + kFp8Block - 1) / kFp8Block) * (fp8_cols(n) / kFp8Block); }
// Packs a and b in one launch (b.x null: a alone).
hipError_t launch_fp8_pack(const Fp8PackArgs& a, const Fp8PackArgs& b, int dtype, hipStream_t stream);
hipError_t launch_fp8_unpack(const void* packed, long m, long n, void* y, long ldy, int dtype, hipStream_t stream);

// C = Q P^T of packed matrices.  g: as for a 16-bit product whose elements are
// pairs of codes (pitches and length half the bytes); e.cols columns, e.rows rows.
struct Gemm8Args {
  GemmArgs g;
  const unsigned char *qs, *ps;    // scales
  long qn, pn;                     // their bytes a row
};
constexpr int kMaxGroup8 = 2;
struct Gemm8Group {
  int count;
  int start[kMaxGroup8];
  Gemm8Args a[kMaxGroup8];
  ColumnJob column;                // sums in workgroups of their own, from `columns` on; out null: none
  int columns;
};
// Forward products of at most kFewRows packed rows, in one launch, or (packed false) of
// at most kCodedRows rows of dtype, k columns at pitch g.ldq, coded on the way.
// In a launch of their own from 5 rows on (us a call, coded on the way against before; bf16
// 4096 -> 4096: 1 row 7.0 and 10.4, 4 rows 8.8 and 10.6, 8 rows 10.8 and 11.0; 8192 ->
// 2048, 8 rows 14.7 and 14.1).
constexpr int kCodedRows = 4;
hipError_t launch_few8(const Gemm8Args& a, int k, bool packed, bool bf16, hipStream_t stream);
// Forward products of k <= kFp8Block inputs: g.q is a matrix of dtype, k columns at pitch
// g.ldq, coded on the way; tile 64 or 128.
hipError_t launch_narrow8(const Gemm8Args& a, int k, int tile, bool bf16, hipStream_t stream);
// kEpiLinear, and kEpiStore for a group; 16-bit results.
hipError_t launch_gemm8(const Gemm8Args& a, int tile, bool bf16, hipStream_t stream);
// `blocks` of the products
hipError_t launch_gemm8_group(Gemm8Group g, int blocks, int tile, bool bf16, hipStream_t stream);

}  // namespace oidn
