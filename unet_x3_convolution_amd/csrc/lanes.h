// Sums and maxima over neighbouring lanes of a wave, in registers: no LDS, which a
// shuffle goes through (a sum over 64 lanes takes 6 vector instructions here, and
// 6 LDS round trips with shuffles).
#pragma once

#include <hip/hip_runtime.h>

namespace oidn {
namespace {

// combine(a, b) of the two groups of S lanes that make up 2 S neighbouring lanes, where
// the lanes of each hold the same value.
template <int S, typename Combine>
__device__ __forceinline__ unsigned combine_lanes(unsigned v, Combine combine) {
  if constexpr (S == 1) return combine(v, (unsigned)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, false));        // quad [1 0 3 2]
  else if constexpr (S == 2) return combine(v, (unsigned)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, false));   // quad [2 3 0 1]
  else if constexpr (S == 4) return combine(v, (unsigned)__builtin_amdgcn_mov_dpp((int)v, 0x141, 0xF, 0xF, false));  // mirrored in 8
  else if constexpr (S == 8) return combine(v, (unsigned)__builtin_amdgcn_mov_dpp((int)v, 0x140, 0xF, 0xF, false));  // mirrored in 16
  else {
    // the other 16 (32) lanes' value, and one's own
    const auto both = S == 16 ? __builtin_amdgcn_permlane16_swap(v, v, false, false)
                              : __builtin_amdgcn_permlane32_swap(v, v, false, false);
    return combine((unsigned)both[0], (unsigned)both[1]);
  }
}
// Over N neighbouring lanes, from groups of FROM whose lanes agree already.
template <int N, int FROM = 1>
__device__ __forceinline__ float lanes_sum(float v) {
  if constexpr (FROM < N) {
    const unsigned r = combine_lanes<FROM>(__float_as_uint(v), [](unsigned a, unsigned b) {
      return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
    });
    return lanes_sum<N, 2 * FROM>(__uint_as_float(r));
  } else {
    return v;
  }
}
// Over the lanes of a wave that are a multiple of N apart, N from 4 to 64.
template <int N>
__device__ __forceinline__ float strided_sum(float v) {
  // rotated by 8, by 4 in 16 lanes
  if constexpr (N <= 8) v += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0x128, 0xF, 0xF, false));
  if constexpr (N <= 4) v += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0x124, 0xF, 0xF, false));
  const auto add = [](unsigned a, unsigned b) { return __float_as_uint(__uint_as_float(a) + __uint_as_float(b)); };
  if constexpr (N <= 16) v = __uint_as_float(combine_lanes<16>(__float_as_uint(v), add));
  if constexpr (N <= 32) v = __uint_as_float(combine_lanes<32>(__float_as_uint(v), add));
  return v;
}
template <int N, int FROM = 1>
__device__ __forceinline__ unsigned lanes_max(unsigned v) {
  if constexpr (FROM < N)
    return lanes_max<N, 2 * FROM>(combine_lanes<FROM>(v, [](unsigned a, unsigned b) { return a > b ? a : b; }));
  else
    return v;
}

}  // namespace
}  // namespace oidn
