// Gradients of the norms before and after a block.
#include "norm_wide.h"

namespace oidn {
namespace {

// Sums of partial rows: kinds 0 .. kNormSums - 1 over all chunks, then a gate
// group's chunks.  A workgroup takes kAcross columns, its threads share the rows,
// whose sums are added in order.
constexpr int kAcross = 16;
__global__ __launch_bounds__(kNormThreads) void norm_finish(NormBackArgs a) {
  __shared__ float lds[kNormThreads];
  const int c = threadIdx.x % kAcross, l = threadIdx.x / kAcross, n = a.n;
  const long j = (long)blockIdx.x * kAcross + c, what = blockIdx.y;
  const float* p;
  float* out;
  long count, step;
  if (what < kNormSums) {
    out = a.sums[what];
    p = a.part + what * n;
    count = a.chunks.count;
    step = (long)kNormSums * n;
  } else {
    const long group = what - kNormSums;
    out = a.dgate && a.chunks.per_group ? a.dgate + group * a.lddg : nullptr;
    p = a.gate_part + group * a.chunks.per_group * n;
    count = a.chunks.per_group;
    step = n;
  }
  if (!out) return;
  float s = 0.f;
  if (j < n) {
#pragma unroll 8
    for (long g = l; g < count; g += kNormThreads / kAcross) s += p[g * step + j];
  }
  lds[threadIdx.x] = s;
  __syncthreads();
  if (l == 0 && j < n) {
    for (int k = 1; k < kNormThreads / kAcross; ++k) s += lds[k * kAcross + c];
    out[j] = s;
  }
}

template <int DT>
hipError_t launch_type(const NormBackArgs& a, hipStream_t stream) {
  const dim3 block(kNormThreads);
  hipLaunchKernelGGL(norm_back_wide<DT>, dim3((unsigned)(a.m < 65536 ? a.m : 65536)), block, 0, stream, a);
  hipError_t e = hipGetLastError();
  bool columns = a.dgate != nullptr;
  for (int k = 0; k < kNormSums; ++k) columns = columns || a.sums[k];
  if (e != hipSuccess || !columns) return e;
  const unsigned across = (unsigned)((a.n + 8l * kNormThreads - 1) / (8 * kNormThreads));
  hipLaunchKernelGGL(norm_columns<DT>, dim3((unsigned)a.chunks.count, across), block, 0, stream, a);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  const long groups = a.dgate && a.chunks.per_group ? a.chunks.count / a.chunks.per_group : 0;
  hipLaunchKernelGGL(norm_finish, dim3((unsigned)((a.n + kAcross - 1l) / kAcross), (unsigned)(kNormSums + groups)), block,
                     0, stream, a);
  return hipGetLastError();
}

}  // namespace

// At most about 1024 chunks, so that the sums over them stay a short pass.
NormChunks norm_chunks(long m, int n, long gate_rows) {
  NormChunks c{};
  (void)n;
  long most = (m + 1023) / 1024;
  if (most < 16) most = 16;
  c.group_rows = gate_rows && gate_rows < m ? gate_rows : m;
  if (c.group_rows <= most) {
    c.rows = most / c.group_rows * c.group_rows;
    c.count = (m + c.rows - 1) / c.rows;
  } else {
    c.per_group = (c.group_rows + most - 1) / most;
    c.rows = (c.group_rows + c.per_group - 1) / c.per_group;
    c.count = (m + c.group_rows - 1) / c.group_rows * c.per_group;
  }
  return c;
}

hipError_t launch_norm_back(const NormBackArgs& a, int dtype, hipStream_t stream) {
  if (dtype == OIDN_F32) return launch_type<OIDN_F32>(a, stream);
  return dtype == OIDN_F16 ? launch_type<OIDN_F16>(a, stream) : launch_type<OIDN_BF16>(a, stream);
}

}  // namespace oidn
