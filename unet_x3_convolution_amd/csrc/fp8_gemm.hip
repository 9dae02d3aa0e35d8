// Launches of the packed matrices' products (fp8_gemm.h).
#include "fp8_gemm.h"

namespace oidn {
namespace {

template <bool BF, int T>
void launch(const Gemm8Args& a, hipStream_t stream) {
  const dim3 grid((unsigned)gemm_blocks(a.g));
  if (a.g.e.stream) hipLaunchKernelGGL((dense_gemm8<BF, T, kStreamed>), grid, dim3(256), 0, stream, a);
  else hipLaunchKernelGGL((dense_gemm8<BF, T, kKept>), grid, dim3(256), 0, stream, a);
}
template <bool BF>
void launch_tile(const Gemm8Args& a, int tile, hipStream_t stream) {
  if (tile == 256) launch<BF, 256>(a, stream);
  else if (tile == 128) launch<BF, 128>(a, stream);
  else launch<BF, 64>(a, stream);
}
template <bool BF>
void launch_group(const Gemm8Group& g, int blocks, int tile, hipStream_t stream) {
  const dim3 grid((unsigned)blocks), block(256);
  if (tile == 256) hipLaunchKernelGGL((dense_gemm8_group<BF, 256>), grid, block, 0, stream, g);
  else if (tile == 128) hipLaunchKernelGGL((dense_gemm8_group<BF, 128>), grid, block, 0, stream, g);
  else hipLaunchKernelGGL((dense_gemm8_group<BF, 64>), grid, block, 0, stream, g);
}

}  // namespace

hipError_t launch_gemm8(const Gemm8Args& a, int tile, bool bf16, hipStream_t stream) {
  if (bf16) launch_tile<true>(a, tile, stream);
  else launch_tile<false>(a, tile, stream);
  return hipGetLastError();
}
hipError_t launch_gemm8_group(Gemm8Group g, int blocks, int tile, bool bf16, hipStream_t stream) {
  g.columns = blocks;
  if (g.column.out) blocks += (int)column_blocks(g.column.groups, g.column.cols);
  if (bf16) launch_group<true>(g, blocks, tile, stream);
  else launch_group<false>(g, blocks, tile, stream);
  return hipGetLastError();
}

}  // namespace oidn
