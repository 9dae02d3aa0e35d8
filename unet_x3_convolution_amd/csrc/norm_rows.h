// Device code shared by the norms around a block and dropout: the
// counter-based generator, row loads and row statistics.
#pragma once

#include "dense_epilogue.h"
#include "norm.h"

namespace oidn {
namespace {

constexpr int kNormThreads = 256;

// ------------------------------------------------------------------ dropout
// Philox4x32-10 (Salmon, Moraes, Dror, Shaw: Parallel random numbers: as easy
// as 1, 2, 3; 2011).  The eight columns j .. j + 7 (j a multiple of 8) of row i
// take one call: counter (i * ceil(n / 8) + j / 8, offset), key seed, and 16
// bits of its 128 each, the low half of word 0 first.  So an element's fate is a
// function of its place in the logical matrix, whatever the pitch, the type and
// the kernel, and a backward pass forms it again.  16 bits make a probability
// exact to 2^-16 and cost 2.5 wide multiplications an element; 32 would be 5,
// more than the memory's pace leaves.
struct Generator {
  unsigned k0, k1, o0, o1;
  __device__ __forceinline__ explicit Generator(const Dropout& d) {
    const unsigned long long s = d.threshold ? d.rng[0] : 0, o = d.threshold ? d.rng[1] : 0;
    k0 = (unsigned)s, k1 = (unsigned)(s >> 32), o0 = (unsigned)o, o1 = (unsigned)(o >> 32);
  }
  __device__ __forceinline__ uint4 words(unsigned long long at) const {
    unsigned a = (unsigned)at, b = (unsigned)(at >> 32), c = o0, d = o1, k = k0, l = k1;
#pragma unroll
    for (int r = 0; r < 10; ++r) {
      const unsigned long long p = (unsigned long long)a * 0xD2511F53u, q = (unsigned long long)c * 0xCD9E8D57u;
      a = (unsigned)(q >> 32) ^ b ^ k;
      b = (unsigned)q;
      c = (unsigned)(p >> 32) ^ d ^ l;
      d = (unsigned)p;
      k += 0x9E3779B9u;
      l += 0xBB67AE85u;
    }
    return make_uint4(a, b, c, d);
  }
};
// Bit k: column k of the eight is kept.
__device__ __forceinline__ unsigned kept8(const uint4& w, const Dropout& d) {
  const unsigned v[4] = {w.x, w.y, w.z, w.w};
  unsigned keep = 0;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const unsigned bits = k % 2 ? v[k / 2] >> 16 : v[k / 2] & 0xffffu;
    keep |= bits >= d.threshold ? 1u << k : 0u;
  }
  return keep;
}
// Dropped elements become 0 whatever they hold, the others times the gain.
__device__ __forceinline__ void drop8(Eight& x, unsigned keep, const Dropout& d) {
#pragma unroll
  for (int k = 0; k < 8; ++k) x.v[k] = keep >> k & 1u ? x.v[k] * d.gain : 0.f;
}

// --------------------------------------------------------------------- rows
// Columns j .. j + 7 of row i of an m x n matrix, zeros past its columns.
template <int DT>
__device__ __forceinline__ Eight row8(const void* p, long ld, long i, int j, long m, int n) {
  Eight r = load_raw<DT>(p, i * ld + j, n - j, (m - 1 - i) * ld + n - j).value();
  if (n - j < 8) clear_tail(n - j, r);
  return r;
}
// Columns of a vector, `other` where there is none.
__device__ __forceinline__ Eight vector8(const float* p, int j, int n, float other) {
  Eight r;
  if (p && n - j >= 8) {
    __builtin_memcpy(r.v, p + j, 32);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) r.v[k] = p ? (k < n - j ? p[j + k] : 0.f) : other;
  }
  return r;
}
template <int DT>
__device__ __forceinline__ float rounded(float v) { return (float)(typename Storage<DT>::T)v; }

// A normalised row is (x - mean) r.
struct Stat { float mean, r; };

}  // namespace
}  // namespace oidn
