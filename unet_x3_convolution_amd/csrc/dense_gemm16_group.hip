// 16-bit gradients' products, dx = dz w and dw = dz^T x, in one launch.
#include "dense_gemm16_direct.h"

namespace oidn {
namespace {

template <bool BF, int T>
hipError_t launch(const GemmGroup& g, const GemmPlan& p, hipStream_t stream) {
  const dim3 grid((unsigned)g.blocks);
  if (p.direct)
    hipLaunchKernelGGL((dense_gemm16_group<BF, T, true>), grid, dim3(256), 0, stream, g);
  else if constexpr (T <= 128)
    hipLaunchKernelGGL((dense_gemm16_group<BF, T, false>), grid, dim3(256), 0, stream, g);
  else
    return hipErrorInvalidValue;
  return hipGetLastError();
}

template <bool BF>
hipError_t launch_tile(const GemmGroup& g, const GemmPlan& p, hipStream_t stream) {
  if (p.tile_r == 256) return launch<BF, 256>(g, p, stream);
  return p.tile_r == 128 ? launch<BF, 128>(g, p, stream) : launch<BF, 64>(g, p, stream);
}

}  // namespace

hipError_t launch_gemm16_group(const GemmGroup& g, const GemmPlan& p, bool bf16, hipStream_t stream) {
  return bf16 ? launch_tile<true>(g, p, stream) : launch_tile<false>(g, p, stream);
}

}  // namespace oidn
