// 16-bit products with operands as in dw = dz^T x.
#include "dense_gemm16_direct.h"

namespace oidn {
namespace {

template <bool BF, int EPI, int TR, int TC>
hipError_t launch(const GemmArgs& a, const GemmPlan& p, hipStream_t stream) {
  const dim3 grid((unsigned)((a.tiles_r * (long)a.tiles_c + kXcds - 1) / kXcds * kXcds), p.splits);
  if (p.direct)
    hipLaunchKernelGGL((dense_gemm16_direct<BF, kWeightGrad, EPI, TR, TC>), grid, dim3(256), 0, stream, a);
  else if constexpr (TR <= 128)
    hipLaunchKernelGGL((dense_gemm16<BF, kWeightGrad, EPI, TR, TC>), grid, dim3(256), 0, stream, a);
  else
    return hipErrorInvalidValue;
  return hipGetLastError();
}

template <bool BF, int EPI>
hipError_t launch_epi(const GemmArgs& a, const GemmPlan& p, hipStream_t stream) {
  if constexpr (EPI != kEpiPartial) {
    if (p.tile_r == 256) return launch<BF, EPI, 256, 256>(a, p, stream);
  }
  if (p.tile_r == 128) return launch<BF, EPI, 128, 128>(a, p, stream);
  if constexpr (EPI == kEpiGated) return launch<BF, EPI, 64, 128>(a, p, stream);
  else return launch<BF, EPI, 64, 64>(a, p, stream);
}

template <bool BF>
hipError_t launch_type(const GemmArgs& a, const GemmPlan& p, int epi, hipStream_t stream) {
  switch (epi) {
    case kEpiLinear: return launch_epi<BF, kEpiLinear>(a, p, stream);
    case kEpiPartial: return launch_epi<BF, kEpiPartial>(a, p, stream);
  }
  return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_gemm16_weight(const GemmArgs& a, const GemmPlan& p, int epi, bool bf16,
                            hipStream_t stream) {
  return bf16 ? launch_type<true>(a, p, epi, stream) : launch_type<false>(a, p, epi, stream);
}

}  // namespace oidn
