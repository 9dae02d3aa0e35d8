// 16-bit product dh = dy w_out with the gated block's backward epilogue.
#include "dense_gemm16_direct.h"

namespace oidn {
namespace {

template <bool BF, int T>
hipError_t launch(const GemmArgs& a, const GemmPlan& p, const UnpackJob& u, hipStream_t stream) {
  const dim3 grid((unsigned)(gemm_blocks(a) + u.blocks));
  if (p.direct)
    hipLaunchKernelGGL((dense_gemm16_gated_back<BF, T, true>), grid, dim3(256), 0, stream, a, u);
  else if constexpr (T <= 128)
    hipLaunchKernelGGL((dense_gemm16_gated_back<BF, T, false>), grid, dim3(256), 0, stream, a, u);
  else
    return hipErrorInvalidValue;
  return hipGetLastError();
}

template <bool BF>
hipError_t launch_tile(const GemmArgs& a, const GemmPlan& p, const UnpackJob& u, hipStream_t stream) {
  if (p.tile_r == 256) return launch<BF, 256>(a, p, u, stream);
  return p.tile_r == 128 ? launch<BF, 128>(a, p, u, stream) : launch<BF, 64>(a, p, u, stream);
}

}  // namespace

hipError_t launch_gemm16_gated_back(const GemmArgs& a, const GemmPlan& p, bool bf16, const UnpackJob& u,
                                    hipStream_t stream) {
  return bf16 ? launch_tile<true>(a, p, u, stream) : launch_tile<false>(a, p, u, stream);
}

}  // namespace oidn
