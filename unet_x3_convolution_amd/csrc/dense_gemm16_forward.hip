// 16-bit forward products: y = x w^T and the gated projections.
#include "dense_gemm16_direct.h"

namespace oidn {
namespace {

template <bool BF, int EPI, int TR, int TC, Caching WHERE>
hipError_t launch_where(const GemmArgs& a, const GemmPlan& p, hipStream_t stream) {
  const dim3 grid((unsigned)gemm_blocks(a));
  if (p.direct)
    hipLaunchKernelGGL((dense_gemm16<BF, kForward, EPI, TR, TC, true, WHERE>), grid, dim3(256), 0, stream, a);
  else if constexpr (TR <= 128)
    hipLaunchKernelGGL((dense_gemm16<BF, kForward, EPI, TR, TC, false, WHERE>), grid, dim3(256), 0, stream, a);
  else
    return hipErrorInvalidValue;
  return hipGetLastError();
}

// A kernel of its own for results past the caches: a branch between the two
// epilogues cost the shortest launches 0.3 us (8160 x 96 -> 384 8.3 against 8.0).
template <bool BF, int EPI, int TR, int TC>
hipError_t launch(const GemmArgs& a, const GemmPlan& p, hipStream_t stream) {
  if constexpr (EPI == kEpiLinear) {
    if (a.e.stream) return launch_where<BF, EPI, TR, TC, kStreamed>(a, p, stream);
  }
  return launch_where<BF, EPI, TR, TC, kKept>(a, p, stream);
}

template <bool BF, int EPI>
hipError_t launch_epi(const GemmArgs& a, const GemmPlan& p, hipStream_t stream) {
  if (p.tile_r == 256) return launch<BF, EPI, 256, 256>(a, p, stream);
  if (p.tile_r == 128) return launch<BF, EPI, 128, 128>(a, p, stream);
  return launch<BF, EPI, 64, EPI == kEpiGated ? 128 : 64>(a, p, stream);
}

}  // namespace

hipError_t launch_gemm16_forward(const GemmArgs& a, const GemmPlan& p, int epi, bool bf16,
                                 hipStream_t stream) {
  if (epi == kEpiLinear)
    return bf16 ? launch_epi<true, kEpiLinear>(a, p, stream) : launch_epi<false, kEpiLinear>(a, p, stream);
  if (epi == kEpiGated)
    return bf16 ? launch_epi<true, kEpiGated>(a, p, stream) : launch_epi<false, kEpiGated>(a, p, stream);
  return hipErrorInvalidValue;
}

}  // namespace oidn
