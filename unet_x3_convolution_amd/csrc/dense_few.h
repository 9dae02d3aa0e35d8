// Products of a few rows (5 to 32; 3 and 4 where a plain product has 4096 columns or
// more; any where z is saved in 8 bits) with
// l-fastest operands: y = x w^T and the gated projections.
//
// The weights are all there is to read, each once, so the kernel is built
// around keeping their loads in flight.  A workgroup of 8 waves owns 16
// columns (two runs of 16 for a gated product, 32 where an 8-bit block has to
// be whole) and all of the summed length, which its waves share in turns of
// one chunk; every wave loads weight fragments straight into registers, two
// batches of kDepth chunks at once, and multiplies them by the rows' fragments
// with MFMAs (rows past the last read the last).  The waves' sums meet in LDS, are
// added in wave order, and one launch is enough.
//
// A chunk is 128 bytes of every weight row: lane group g of 16 lanes takes
// bytes 32 g .. + 31 in two 16-byte loads, so a pair of loads covers whole
// lines.  MFMA s multiplies the s-th 16 bytes of all lanes: the order of the
// sum is permuted alike in both operands.
//
// Bound by those loads, which touch 16 half lines each: about 31 GB/s per
// compute unit with the waves and depths that were tried.  bf16, weights cold, us
// a call: 4096 -> 4096 8.6 at 3 rows, 9.9 at 8, 11 at 16, 14 at 32, where tiles,
// their slices and the sum take 14, 14, 14 and 18.
#pragma once

#include "dense_gemm16.h"

namespace oidn {
namespace {

template <int DT>
__device__ __forceinline__ floatx4 multiply16(uint4 a, uint4 b, floatx4 c) {
  if constexpr (DT == OIDN_F32) {
    const floatx4 av = __builtin_bit_cast(floatx4, a), bv = __builtin_bit_cast(floatx4, b);
#pragma unroll
    for (int e = 0; e < 4; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(av[e], bv[e], c, 0, 0, 0);
    return c;
  } else {
    return mfma16<DT == OIDN_BF16>(a, b, c);
  }
}

constexpr int kFewWaves = 8, kDepth = 2;

// EPI kEpiLinear or kEpiGated; MF: fragments of 16 rows; NF: fragments of 16
// columns of each projection.
template <int DT, int EPI, int MF, int NF>
__global__ __launch_bounds__(64 * kFewWaves) void dense_few(GemmArgs a) {
  constexpr int kSize = DT == OIDN_F32 ? 4 : 2, kPer = 16 / kSize;   // elements of 16 bytes
  constexpr int kChunk = 128 / kSize;
  constexpr int kSets = EPI == kEpiGated ? 2 : 1, WF = NF * kSets;   // weight fragments
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
  const int j0 = blockIdx.x * 16 * NF;
  const long len = a.len;

  const char* wp[WF];
  const char* xp[MF];
#pragma unroll
  for (int f = 0; f < WF; ++f) {
    int j = j0 + 16 * (f % NF) + r;
    j = j < a.e.cols ? j : a.e.cols - 1;
    wp[f] = static_cast<const char*>(a.p) + kSize * ((long)j + (f / NF) * (long)a.e.cols) * a.ldp;
  }
#pragma unroll
  for (int f = 0; f < MF; ++f) {
    long i = 16 * f + r;
    i = i < a.e.rows ? i : a.e.rows - 1;
    xp[f] = static_cast<const char*>(a.q) + kSize * i * a.ldq;
  }
  floatx4 acc[WF][MF];
#pragma unroll
  for (int f = 0; f < WF; ++f)
#pragma unroll
    for (int m = 0; m < MF; ++m) acc[f][m] = floatx4{0.f, 0.f, 0.f, 0.f};

  const Extent<kSize> all_w(a.p, (long)a.e.cols * kSets, a.ldp, len), all_x(a.q, a.e.rows, a.ldq, len);
  struct Batch {
    uint4 w[kDepth][2][WF], x[kDepth][2][MF];
  };
  // Chunks c, c + kFewWaves, ... of this wave, `depth` of them, all whole.
  auto load = [&](Batch& t, long c, auto depth) {
#pragma unroll
    for (int d = 0; d < decltype(depth)::value; ++d)
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const long l = (c + d * kFewWaves) * kChunk + 2 * kPer * g + kPer * s;
#pragma unroll
        for (int f = 0; f < WF; ++f) t.w[d][s][f] = load16_any(wp[f] + kSize * l);
#pragma unroll
        for (int m = 0; m < MF; ++m) t.x[d][s][m] = load16_any(xp[m] + kSize * l);
      }
  };
  auto multiply = [&](const Batch& t, auto depth) {
#pragma unroll
    for (int d = 0; d < decltype(depth)::value; ++d)
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int f = 0; f < WF; ++f)
#pragma unroll
          for (int m = 0; m < MF; ++m) acc[f][m] = multiply16<DT>(t.w[d][s][f], t.x[d][s][m], acc[f][m]);
  };
  constexpr std::integral_constant<int, kDepth> kAll{};
  constexpr std::integral_constant<int, 1> kOne{};
  const long whole = len / kChunk;
  long c = wave;
  auto there = [&](long from) { return from + (kDepth - 1) * kFewWaves < whole; };
  if (there(c)) {
    // one batch is multiplied while the next one's loads are in flight
    Batch t[2];
    load(t[0], c, kAll);
    for (;;) {
      c += kDepth * kFewWaves;
      const bool more = there(c);
      if (more) load(t[1], c, kAll);
      multiply(t[0], kAll);
      if (!more) break;
      c += kDepth * kFewWaves;
      const bool again = there(c);
      if (again) load(t[0], c, kAll);
      multiply(t[1], kAll);
      if (!again) break;
    }
  }
  for (; c < whole; c += kFewWaves) {
    Batch t;
    load(t, c, kOne);
    multiply(t, kOne);
  }
  if (c == whole && len % kChunk) {        // the last chunk, of which a part exists
    Batch t;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const long l = c * kChunk + 2 * kPer * g + kPer * s;
      all_w.load(t.w[0][s], [&](int f, const char*& p, long& n) { p = wp[f] + kSize * l, n = len - l; });
      all_x.load(t.x[0][s], [&](int m, const char*& p, long& n) { p = xp[m] + kSize * l, n = len - l; });
    }
    multiply(t, kOne);
  }

  // [wave][set][row][column]; a row's pitch is padded by 16 bytes
  constexpr int kCols = 16 * NF, kPitch = kCols + 4;
  __shared__ __attribute__((aligned(16))) float part[kFewWaves][kSets][16 * MF][kPitch];
#pragma unroll
  for (int f = 0; f < WF; ++f)
#pragma unroll
    for (int m = 0; m < MF; ++m)
      *reinterpret_cast<floatx4*>(&part[wave][f / NF][16 * m + r][16 * (f % NF) + 4 * g]) = acc[f][m];
  __syncthreads();
  // eight columns of a row per lane; lanes of a row are neighbours
  constexpr int kLanes = 2 * NF;
  const int t = threadIdx.x, i = t / kLanes, j8 = 8 * (t % kLanes);
  if (t >= 16 * MF * kLanes) return;         // whole groups of kLanes
  Eight v[2] = {};
#pragma unroll
  for (int k = 0; k < kFewWaves; ++k)
#pragma unroll
    for (int s = 0; s < kSets; ++s)
#pragma unroll
      for (int e = 0; e < 8; ++e) v[s].v[e] += part[k][s][i][j8 + e];
  const int j = j0 + j8;
  Fetched bias{}, none;
  RawFetched<DT, false> f;
  bias.a = bias8(a.e.bias, j, a.e.cols - j);
  if constexpr (EPI == kEpiGated) bias.b = bias8(a.e.bias ? a.e.bias + a.e.cols : nullptr, j, a.e.cols - j);
  if (j0 + kCols <= a.e.cols) {
    fetch<DT, EPI, true, false>(a.e, i, j, f);
    finish<DT, EPI, true, false>(a.e, 0, i, j, v[0], v[1], bias, f, none);
  } else {
    fetch<DT, EPI, false, false>(a.e, i, j, f);
    finish<DT, EPI, false, false>(a.e, 0, i, j, v[0], v[1], bias, f, none);
  }
}

}  // namespace
}  // namespace oidn
