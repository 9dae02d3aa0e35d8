// Launches of the products of a few rows (dense_few.h).
#include "dense_dot.h"
#include "dense_few.h"

namespace oidn {
namespace {

template <int DT, int EPI, int NF>
hipError_t launch_rows(const GemmArgs& a, hipStream_t stream) {
  const dim3 grid((unsigned)((a.e.cols + 16 * NF - 1) / (16 * NF))), block(64 * kFewWaves);
  if (a.e.rows <= 16)
    hipLaunchKernelGGL((dense_few<DT, EPI, 1, NF>), grid, block, 0, stream, a);
  else
    hipLaunchKernelGGL((dense_few<DT, EPI, 2, NF>), grid, block, 0, stream, a);
  return hipGetLastError();
}

template <int DT, int EPI>
hipError_t launch_dot(const GemmArgs& a, hipStream_t stream) {
  const dim3 grid((unsigned)((a.e.cols + kDotWaves - 1) / kDotWaves)), block(64 * kDotWaves);
  if (a.e.rows == 1) hipLaunchKernelGGL((dense_dot<DT, EPI, 1>), grid, block, 0, stream, a);
  else if (a.e.rows == 2) hipLaunchKernelGGL((dense_dot<DT, EPI, 2>), grid, block, 0, stream, a);
  else hipLaunchKernelGGL((dense_dot<DT, EPI, 4>), grid, block, 0, stream, a);
  return hipGetLastError();
}

template <int DT>
hipError_t launch_type(const GemmArgs& a, int epi, hipStream_t stream) {
  // 16 columns a workgroup, unless an 8-bit block of 32 has to be in one
  const bool block32 = a.e.z && a.e.z8;
  // Dot instructions, or matrix fragments (us a call, weights cold).  One and two
  // rows: dots (bf16 4096 -> 4096 7.6 against 8.4).  Three and four: a plain
  // product's dots read four rows of x for one of w, and where the fragments'
  // workgroups of 16 columns fill the 256 units they are ahead (bf16 4096 -> 4096
  // 8.8 against 11.5, fp32 2048 -> 8192 15.1 against 20.6), else not (bf16 5632 ->
  // 2048 10.7 against 8.6).  A gated product reads two rows of w with them: dots
  // (block of 2048 x 5632 21.5 against 25.6).
  const bool wide = epi == kEpiLinear && a.e.cols >= 16 * 256;
  if (a.e.rows <= (wide ? 2 : 4) && !block32) {
    if (epi == kEpiLinear) return launch_dot<DT, kEpiLinear>(a, stream);
    if (epi == kEpiGated) return launch_dot<DT, kEpiGated>(a, stream);
  }
  if (epi == kEpiLinear)
    return block32 ? launch_rows<DT, kEpiLinear, 2>(a, stream) : launch_rows<DT, kEpiLinear, 1>(a, stream);
  if (epi == kEpiGated)
    return block32 ? launch_rows<DT, kEpiGated, 2>(a, stream) : launch_rows<DT, kEpiGated, 1>(a, stream);
  return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_few(const GemmArgs& a, int epi, int dtype, hipStream_t stream) {
  if (a.e.rows > kFewRows) return hipErrorInvalidValue;
  if (dtype == OIDN_F32) return launch_type<OIDN_F32>(a, epi, stream);
  return dtype == OIDN_F16 ? launch_type<OIDN_F16>(a, epi, stream) : launch_type<OIDN_BF16>(a, epi, stream);
}

}  // namespace oidn
