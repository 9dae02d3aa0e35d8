// Device code of the 8-bit floating-point form (fp8.h).
//
// A block's scale is the least power of two 2^e with max|x| <= 448 2^e (448 is
// e4m3's largest value), e held in [-120, 120].  Being a power of two it changes no
// mantissa: a value is rounded once, to the four significant bits of e4m3 (2^-4 of
// it; below 2^-6 of the scale to steps of 2^-9), and the matrix cores take the
// exponent as an operand of their own, so that blocks cost a product nothing.
// Infinities and NaN are coded NaN; the scale is that of the finite values.
#pragma once

#include "dense_epilogue.h"
#include "fp8.h"

namespace oidn {
namespace {

struct Fp8At {
  unsigned char* codes;
  unsigned char* scales;
  long pitch, words;       // bytes of a row: codes, scales
};
__device__ __forceinline__ Fp8At fp8_at(void* packed, long m, long n) {
  const long pitch = (n + kFp8Block - 1) / kFp8Block * kFp8Block, words = (pitch / kFp8Block + 3) / 4 * 4;
  unsigned char* const p = static_cast<unsigned char*>(packed);
  return {p, p + m * pitch, pitch, words};
}
// Bits of the magnitude; of infinities and NaN: 0x7f800000 and more.
__device__ __forceinline__ unsigned magnitude_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }
// The same, 0 for what is not finite.
__device__ __forceinline__ unsigned finite_bits(float v) {
  const unsigned b = magnitude_bits(v);
  return b < 0x7f800000u ? b : 0u;
}
// The largest finite magnitude of eight values: infinities and NaN are rare, so they are
// left out only where the plain maximum shows one.
__device__ __forceinline__ unsigned finite_top(const Eight& x) {
  unsigned t = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) t = max(t, magnitude_bits(x.v[e]));
  if (t >= 0x7f800000u) {
    t = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) t = max(t, finite_bits(x.v[e]));
  }
  return t;
}
// e of a block from the bits of its largest magnitude; 448 = 1.75 * 2^8.
__device__ __forceinline__ int fp8_power(unsigned top) {
  if (top == 0) return 0;
  const int e = (int)(top >> 23) - 127 - 8 + ((top & 0x7fffffu) > 0x600000u ? 1 : 0);
  return e < -120 ? -120 : e > 120 ? 120 : e;
}
__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float((unsigned)(e + 127) << 23); }
// Codes of x 2^-e, nearest even; `inverse` is 2^-e.  The conversion gives NaN for infinities
// and NaN; finite values do not pass its range.
__device__ __forceinline__ unsigned fp8_codes4(const float* x, float inverse) {
  const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(x[0] * inverse, x[1] * inverse, 0, false);
  return (unsigned)__builtin_amdgcn_cvt_pk_fp8_f32(x[2] * inverse, x[3] * inverse, lo, true);
}
__device__ __forceinline__ uint2 fp8_codes(const float (&x)[8], float inverse) {
  return make_uint2(fp8_codes4(x, inverse), fp8_codes4(x + 4, inverse));
}
__device__ __forceinline__ Eight fp8_values(uint2 c, float scale) {
  typedef float floatx2 __attribute__((ext_vector_type(2)));
  const floatx2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)c.x, false), b = __builtin_amdgcn_cvt_pk_f32_fp8((int)c.x, true),
                d = __builtin_amdgcn_cvt_pk_f32_fp8((int)c.y, false), f = __builtin_amdgcn_cvt_pk_f32_fp8((int)c.y, true);
  return {{a[0] * scale, a[1] * scale, b[0] * scale, b[1] * scale, d[0] * scale, d[1] * scale, f[0] * scale, f[1] * scale}};
}

}  // namespace
}  // namespace oidn
