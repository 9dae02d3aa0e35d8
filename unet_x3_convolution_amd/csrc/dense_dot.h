// Products of at most four rows with l-fastest operands: y = x w^T and the
// gated projections, as when single pixels or tokens are served.
//
// The weights are all there is to read, each once, so what counts is how their
// loads run: a wave owns a column (a row of w; of a gated product one of each
// projection) and reads 1 KB of it with every load, whole lines in order, four
// chunks in flight.  Loads in a matrix fragment's order (dense_few.h) touch 16
// half lines each and stop at about 31 GB/s per compute unit.  The rows of x
// come along in the same layout, out of the caches, and are multiplied with
// dot instructions; a matrix core would have 16 rows to fill.  The lanes' sums
// are added across the wave at the end, and the workgroup's eight columns leave
// through one epilogue.  One launch is enough.
//
// Measured (bf16, weights cold): one row 4096 -> 4096 6.6 us (fragment order
// 7.6), four rows gated 2048 -> 5632 10.2 us (13.4), 5632 -> 2048 6.5 us (9.6);
// eight rows 19 us (13.4) and 10.5 us (9.6), which is why four is the limit.
// Two columns a wave take 14.0 us instead of 10.2.
#pragma once

#include "dense_gemm16.h"

namespace oidn {
namespace {

// acc + the dot product of 16 bytes of each, in fp32.
template <int DT>
__device__ __forceinline__ float dot16(uint4 a, uint4 b, float acc) {
  const unsigned av[4] = {a.x, a.y, a.z, a.w}, bv[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if constexpr (DT == OIDN_F32) {
      acc = __builtin_fmaf(__uint_as_float(av[k]), __uint_as_float(bv[k]), acc);
    } else if constexpr (DT == OIDN_F16) {
      typedef _Float16 half2v __attribute__((ext_vector_type(2)));
      acc = __builtin_amdgcn_fdot2(__builtin_bit_cast(half2v, av[k]), __builtin_bit_cast(half2v, bv[k]), acc, false);
    } else {
      typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
      acc = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, av[k]), __builtin_bit_cast(bf16x2, bv[k]), acc,
                                            false);
    }
  }
  return acc;
}

// Sums of N (a power of two) values over the wave's 64 lanes, in a fixed order.
// Each step adds the lanes XOR s; while several values are left, a lane keeps
// one half of them and gives the other away, so N + 5 exchanges do for all.
// Lane l ends with the sum of value `wave_sums_index<N>(l)`.
template <int N>
__device__ __forceinline__ float wave_sums(float (&v)[N], int lane) {
  int left = N;
#pragma unroll
  for (int s = 1; s < 64; s *= 2) {
    if (left > 1) {
      left /= 2;
#pragma unroll
      for (int k = 0; k < N / 2; ++k)
        if (k < left) {
          const bool up = lane & s;
          const float give = up ? v[k] : v[k + left];
          v[k] = (up ? v[k + left] : v[k]) + __shfl_xor(give, s);
        }
    } else {
      v[0] += __shfl_xor(v[0], s);
    }
  }
  return v[0];
}
template <int N>
__device__ __forceinline__ int wave_sums_index(int lane) {
  int at = 0;
#pragma unroll
  for (int left = N / 2, s = 1; left >= 1; left /= 2, s *= 2) at += lane & s ? left : 0;
  return at;
}

constexpr int kDotWaves = 8;

// M rows.
template <int DT, int EPI, int M>
__global__ __launch_bounds__(64 * kDotWaves) void dense_dot(GemmArgs a) {
  constexpr int kSize = DT == OIDN_F32 ? 4 : 2, kPer = 16 / kSize, kChunk = 64 * kPer;
  constexpr int kSets = EPI == kEpiGated ? 2 : 1, W = kSets;        // weight rows of a wave
  constexpr int kDepth = 4;                // chunks in flight
  constexpr int kCols = kDotWaves;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int j0 = blockIdx.x * kCols;
  const long len = a.len;

  const char* wp[W];
  const char* xp[M];
#pragma unroll
  for (int c = 0; c < W; ++c) {
    const int j = j0 + wave < a.e.cols ? j0 + wave : a.e.cols - 1;
    wp[c] = static_cast<const char*>(a.p) + kSize * ((j + c * (long)a.e.cols) * a.ldp + kPer * lane);
  }
#pragma unroll
  for (int m = 0; m < M; ++m)
    xp[m] = static_cast<const char*>(a.q) + kSize * ((m < a.e.rows ? m : a.e.rows - 1) * a.ldq + kPer * lane);
  float acc[M][W] = {};

  auto chunks = [&](long l, auto depth) {         // whole chunks from element l on
    constexpr int D = decltype(depth)::value;
    uint4 w[D][W], x[D][M];
#pragma unroll
    for (int d = 0; d < D; ++d) {
#pragma unroll
      for (int c = 0; c < W; ++c) w[d][c] = load16_any(wp[c] + kSize * (l + d * kChunk));
#pragma unroll
      for (int m = 0; m < M; ++m) x[d][m] = load16_any(xp[m] + kSize * (l + d * kChunk));
    }
#pragma unroll
    for (int d = 0; d < D; ++d)
#pragma unroll
      for (int c = 0; c < W; ++c)
#pragma unroll
        for (int m = 0; m < M; ++m) acc[m][c] = dot16<DT>(w[d][c], x[d][m], acc[m][c]);
  };
  long l = 0;
  for (; l + kDepth * kChunk <= len; l += kDepth * kChunk) chunks(l, std::integral_constant<int, kDepth>{});
  for (; l + kChunk <= len; l += kChunk) chunks(l, std::integral_constant<int, 1>{});
  if (l < len) {                                  // a part of a chunk
    const Extent<kSize> all_w(a.p, (long)a.e.cols * kSets, a.ldp, len), all_x(a.q, a.e.rows, a.ldq, len);
    const long n = len - l - kPer * lane;
    uint4 w[W], x[M];
    all_w.load(w, [&](int c, const char*& p, long& k) { p = wp[c] + kSize * l, k = n; });
    all_x.load(x, [&](int m, const char*& p, long& k) { p = xp[m] + kSize * l, k = n; });
#pragma unroll
    for (int c = 0; c < W; ++c)
#pragma unroll
      for (int m = 0; m < M; ++m) acc[m][c] = dot16<DT>(w[c], x[m], acc[m][c]);
  }

  __shared__ float sums[kSets][M][kCols];
  static_assert(M * W <= 64, "one sum per lane");
  float all[M * W];
#pragma unroll
  for (int m = 0; m < M; ++m)
#pragma unroll
    for (int c = 0; c < W; ++c) all[m * W + c] = acc[m][c];
  const float sum = wave_sums<M * W>(all, lane);
  const int at = wave_sums_index<M * W>(lane);
  if (lane < M * W) sums[at % W][at / W][wave] = sum;
  __syncthreads();
  // eight columns of a row per lane
  const int i = threadIdx.x, j = j0;
  if (i >= M) return;
  Eight v[2] = {};
#pragma unroll
  for (int s = 0; s < kSets; ++s)
#pragma unroll
    for (int e = 0; e < 8; ++e) v[s].v[e] = sums[s][i][e];
  Fetched bias{}, none;
  RawFetched<DT, false> f;
  bias.a = bias8(a.e.bias, j, a.e.cols - j);
  if constexpr (EPI == kEpiGated) bias.b = bias8(a.e.bias ? a.e.bias + a.e.cols : nullptr, j, a.e.cols - j);
  fetch<DT, EPI, false, false>(a.e, i, j, f);
  finish<DT, EPI, false, false>(a.e, 0, i, j, v[0], v[1], bias, f, none);
}

}  // namespace
}  // namespace oidn
