// Column sums of partial rows, in the launches that finish sums.
#pragma once

#include "dense.h"

namespace oidn {
namespace {

constexpr int kColumnThreads = 256;      // and as many floats of LDS

// Columns of partial sums, 256 / lanes of them a workgroup: each is shared by
// `lanes` threads, eight reads in flight each, added in order.
__device__ __forceinline__ void sum_columns(const float* __restrict__ part, long groups, int cols,
                                            float* __restrict__ out, int block, int lanes, char* mem) {
  const int across = kColumnThreads / lanes, c = threadIdx.x % across, l = threadIdx.x / across, j = block * across + c;
  float s = 0.f;
  if (j < cols) {
#pragma unroll 8
    for (long g = l; g < groups; g += lanes) s += part[g * cols + j];
  }
  float* const lds = reinterpret_cast<float*>(mem);
  lds[threadIdx.x] = s;
  __syncthreads();
  if (l == 0 && j < cols) {
    for (int k = 1; k < lanes; ++k) s += lds[k * across + c];
    out[j] = s;
  }
}
constexpr int column_lanes(long groups) { return groups > 64 ? 32 : 8; }

}  // namespace
}  // namespace oidn
