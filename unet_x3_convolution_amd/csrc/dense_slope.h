// The pass dz = dy * act'(z) over rows, with column sums (SlopeArgs), and
// checkpoints read back beside other work (UnpackJob).
//
// Bound by memory and by the slope's arithmetic: gelu's over 8192 x 4096 bf16 (201
// MB) in 64 to 68 us, 3.0 to 3.1 TB/s.  Four rows' loads are in
// flight per thread; a chunk is a workgroup's rows, at most 256 chunks, so that
// their column sums stay one short pass.
#pragma once

#include "dense_epilogue.h"

namespace oidn {
namespace {

constexpr int kRowThreads = 256;
constexpr int kSlopeLds = kRowThreads * 9 * 4;

// Workgroup `block` covers `chunk` rows by 8 << lanes columns: 1 << lanes units
// of eight columns, the other threads are row lanes.
template <int DT>
__device__ __forceinline__ void slope_rows(const SlopeArgs& a, int block, float* lds) {
  const int cs = a.lanes, u = threadIdx.x & ((1 << cs) - 1), rl = threadIdx.x >> cs, rows_at_once = kRowThreads >> cs;
  const int across = ((a.cols + 7) / 8 + (1 << cs) - 1) >> cs, chunk = block / across, bc = block - chunk * across;
  const int j = ((bc << cs) + u) * 8;
  const int n = a.cols - j;
  const long r0 = chunk * a.chunk, r1 = r0 + a.chunk < a.rows ? r0 + a.chunk : a.rows;
  Eight sum{};
  if (n > 0) {
    // four rows' reads in flight
    for (long i0 = r0 + rl; i0 < r1; i0 += 4 * rows_at_once) {
      Eight d[4], z[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const long i = i0 + k * rows_at_once;
        if (i >= r1) break;
        d[k] = load8<DT>(a.dy, i * a.lddy + j, n);
        if (a.act != OIDN_ACT_NONE)
          z[k] = a.z8 ? ckpt_load8(ckpt_at(const_cast<void*>(a.z), a.rows, a.cols), i, j)
                      : load8<DT>(a.z, i * a.ldz + j, n);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const long i = i0 + k * rows_at_once;
        if (i >= r1) break;
        if (a.act != OIDN_ACT_NONE) {
          Eight value;
          activate_slope8<DT>(a.act, z[k], value);
#pragma unroll
          for (int m = 0; m < 8; ++m) d[k].v[m] *= z[k].v[m];
        }
        // dz is rounded to what dx's and dw's products read (16-bit operands of the
        // matrix cores); the column sums are of the unrounded values
        if (a.dz) store8<DT>(a.dz, i * (long)a.cols + j, d[k], n);
        add8(sum, d[k]);
      }
    }
  }
  if (!a.part) return;
  // row lanes are added in order through LDS
#pragma unroll
  for (int k = 0; k < 8; ++k) lds[threadIdx.x * 9 + k] = sum.v[k];
  __syncthreads();
  for (int c = threadIdx.x; c < (8 << cs); c += kRowThreads) {
    float s = 0.f;
    for (int r = 0; r < rows_at_once; ++r) s += lds[((r << cs) + c / 8) * 9 + c % 8];
    const int col = (bc << cs) * 8 + c;
    if (col < a.cols) a.part[(long)chunk * a.cols + col] = s;
  }
}

// The values are rounded to DT, as dw's product reads them: in 16 bits a third
// rounding beside dz's and the output's (bf16 0.0029, fp16 0.00036 of dw in all).
template <int DT>
__device__ __forceinline__ void unpack_rows(const UnpackJob& u, int block) {
  const long units = (u.n + 7) / 8, total = u.m * units;
  const CkptAt at = ckpt_at(const_cast<void*>(u.ckpt), u.m, u.n);
  RawCodes got[kUnpackRun];
#pragma unroll
  for (int k = 0; k < kUnpackRun; ++k) {
    const long t = ((long)block * kUnpackRun + k) * kRowThreads + threadIdx.x, i = t / units;
    if (t < total) got[k] = load_codes(at, i, (int)(t - i * units) * 8);
  }
#pragma unroll
  for (int k = 0; k < kUnpackRun; ++k) {
    const long t = ((long)block * kUnpackRun + k) * kRowThreads + threadIdx.x, i = t / units;
    const int j = (int)(t - i * units) * 8;
    if (t < total) store8<DT>(u.y, i * u.n + j, ckpt_stored<DT>(got[k]), u.n - j);
  }
}

}  // namespace
}  // namespace oidn
