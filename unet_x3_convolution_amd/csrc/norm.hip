// The norms before and after a block, forward, and dropout.
#include "norm_fast.h"
#include "norm_wide.h"

namespace oidn {
namespace {

// y = drop(x) + residual, rounded once.  A thread takes eight columns, the share of one call
// of the generator (norm_rows.h).  Bound by memory: 16384 x 4096 bf16 with a residual
// (403 MB) 68.9 us, without one (268 MB) 48.7, 5.5 TB/s (the end of the last pass's results is
// still in the caches); 32640 x 112 fp16 4.9.
template <int DT>
__global__ __launch_bounds__(kNormThreads) void dropout_rows(const void* x, long ldx, const void* residual, long ldr,
                                                             void* y, long ldy, long m, int n, long units, Dropout d) {
  const Generator random(d);
  const long total = m * units, step = (long)gridDim.x * kNormThreads;
  for (long t = (long)blockIdx.x * kNormThreads + threadIdx.x; t < total; t += step) {
    const long i = t / units;
    const int j = (int)(t - i * units) * 8;
    Eight v = row8<DT>(x, ldx, i, j, m, n);
    if (d.threshold) drop8(v, kept8(random.words(t), d), d);
    if (residual) add8(v, row8<DT>(residual, ldr, i, j, m, n));
    store8<DT>(y, i * ldy + j, v, n - j);
  }
}

template <int DT, int LANES>
hipError_t launch_rows(const NormArgs& a, hipStream_t stream) {
  constexpr int kThreads = norm_threads<LANES>(), kRows = kThreads / LANES;
  const long blocks = (a.m + kRows - 1) / kRows, most = 2048 * 256 / kThreads;
  const dim3 grid((unsigned)(blocks < most ? blocks : most)), block(kThreads);
  if (a.n % 8 == 0) hipLaunchKernelGGL((norm_rows<DT, LANES, true>), grid, block, 0, stream, a);
  else hipLaunchKernelGGL((norm_rows<DT, LANES, false>), grid, block, 0, stream, a);
  return hipGetLastError();
}
template <int DT>
hipError_t launch_type(const NormArgs& a, hipStream_t stream) {
  switch (norm_lanes(a.n)) {
    case 4: return launch_rows<DT, 4>(a, stream);
    case 8: return launch_rows<DT, 8>(a, stream);
    case 16: return launch_rows<DT, 16>(a, stream);
    case 32: return launch_rows<DT, 32>(a, stream);
    case 64: return launch_rows<DT, 64>(a, stream);
    case 128: return launch_rows<DT, 128>(a, stream);
    case 256: return launch_rows<DT, 256>(a, stream);
    case 512: return launch_rows<DT, 512>(a, stream);
    case 1024: return launch_rows<DT, 1024>(a, stream);
  }
  const dim3 grid((unsigned)(a.m < 65536 ? a.m : 65536));
  hipLaunchKernelGGL(norm_wide<DT>, grid, dim3(kNormThreads), 0, stream, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_norm(const NormArgs& a, int dtype, hipStream_t stream) {
  if (dtype == OIDN_F32) return launch_type<OIDN_F32>(a, stream);
  return dtype == OIDN_F16 ? launch_type<OIDN_F16>(a, stream) : launch_type<OIDN_BF16>(a, stream);
}

hipError_t launch_dropout(const void* x, long ldx, const void* residual, long ldr, void* y, long ldy, long m, int n,
                          const Dropout& d, int dtype, hipStream_t stream) {
  const long units = (n + 7l) / 8, blocks = (m * units + kNormThreads - 1) / kNormThreads;
  const dim3 grid((unsigned)(blocks < 65536 ? blocks : 65536)), block(kNormThreads);
  if (dtype == OIDN_F32)
    hipLaunchKernelGGL(dropout_rows<OIDN_F32>, grid, block, 0, stream, x, ldx, residual, ldr, y, ldy, m, n, units, d);
  else if (dtype == OIDN_F16)
    hipLaunchKernelGGL(dropout_rows<OIDN_F16>, grid, block, 0, stream, x, ldx, residual, ldr, y, ldy, m, n, units, d);
  else
    hipLaunchKernelGGL(dropout_rows<OIDN_BF16>, grid, block, 0, stream, x, ldx, residual, ldr, y, ldy, m, n, units, d);
  return hipGetLastError();
}

}  // namespace oidn
