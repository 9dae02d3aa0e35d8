// Device code shared by the dense operators: storage types, activations and
// their slopes, 8-bit checkpoint blocks, and the epilogues that the tile
// kernels and the slice sum run on eight neighbouring columns of one row.
#pragma once

#include <type_traits>

#include "dense.h"
#include "mfma_common.h"

namespace oidn {
namespace {

typedef float floatx8 __attribute__((ext_vector_type(8)));
typedef _Float16 halfx8 __attribute__((ext_vector_type(8)));

// Tile and slice of workgroup `block` (gemm_blocks); false for a padding one.
__device__ __forceinline__ bool tile_and_slice(const GemmArgs& a, int block, int& tc, int& tr, int& slice) {
  const int per = (a.tiles_r * a.tiles_c + kXcds - 1) / kXcds * kXcds;
  slice = block / per;
  return tile_of_block(block - slice * per, a.tiles_c, a.tiles_r, tc, tr);
}

// ------------------------------------------------------------ storage types
// DT is OIDN_F32, OIDN_F16 or OIDN_BF16.  Values are computed in fp32 and
// rounded to nearest even once, where they are stored.
template <int DT> struct Storage;
template <> struct Storage<OIDN_F32> { typedef float T; };
template <> struct Storage<OIDN_F16> { typedef _Float16 T; };
template <> struct Storage<OIDN_BF16> { typedef __bf16 T; };

struct Eight { float v[8]; };

template <int DT>
__device__ __forceinline__ float load1(const void* p, long i) {
  return (float)static_cast<const typename Storage<DT>::T*>(p)[i];
}
template <int DT>
__device__ __forceinline__ void store1(void* p, long i, float v) {
  static_cast<typename Storage<DT>::T*>(p)[i] = (typename Storage<DT>::T)v;
}

// Eight elements from element offset i, of which n (if less than eight) exist;
// 0 in place of the others.  Accesses are 16 bytes wide at any element
// alignment (unaligned access is enabled on this target).
template <int DT>
__device__ __forceinline__ Eight load8(const void* p, long i, int n) {
  typedef typename Storage<DT>::T T;
  const T* s = static_cast<const T*>(p) + i;
  Eight r;
  if (n >= 8) {
    if constexpr (DT == OIDN_F32) {
      __builtin_memcpy(r.v, s, 32);
    } else {
      typedef T T8 __attribute__((ext_vector_type(8)));
      T8 t;
      __builtin_memcpy(&t, s, 16);
#pragma unroll
      for (int k = 0; k < 8; ++k) r.v[k] = (float)t[k];
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) r.v[k] = k < n ? (float)s[k] : 0.f;
  }
  return r;
}

// STREAM: whole units are not kept in the caches (stream_result).
template <int DT, bool STREAM = false>
__device__ __forceinline__ void store8(void* p, long i, const Eight& r, int n) {
  typedef typename Storage<DT>::T T;
  T* s = static_cast<T*>(p) + i;
  if (n >= 8) {
    if constexpr (DT == OIDN_F32) {
      __builtin_memcpy(s, r.v, 32);
    } else {
      typedef T T8 __attribute__((ext_vector_type(8)));
      T8 t;
#pragma unroll
      for (int k = 0; k < 8; ++k) t[k] = (T)r.v[k];
      if constexpr (STREAM) {
        typedef unsigned int u32x4 __attribute__((ext_vector_type(4), aligned(2)));
        __builtin_nontemporal_store(__builtin_bit_cast(u32x4, t), reinterpret_cast<u32x4*>(s));
      } else {
        __builtin_memcpy(s, &t, 16);
      }
    }
  } else {
    // runs of four, two and one
    T t[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) t[k] = (T)r.v[k];
    const bool four = n & 4, two = n & 2;
    if (four) __builtin_memcpy(s, t, 4 * sizeof(T));
    if (two) {
      const T p[2] = {four ? t[4] : t[0], four ? t[5] : t[1]};
      __builtin_memcpy(s + (n & 4), p, 2 * sizeof(T));
    }
    if (n & 1) s[n - 1] = four ? (two ? t[6] : t[4]) : (two ? t[2] : t[0]);
  }
}

// -------------------------------------------------------------- activations
// silu(z) = z p with p = 1 / (1 + e^-z); gelu(z) = z Phi(z), Phi the normal
// distribution function.  Phi is formed from Phi(-|z|), which is small where z is
// negative, so gelu keeps its relative accuracy there: (1 + erf) / 2 would leave
// what two numbers near 1/2 differ by (18% off at z = -5.25).  Phi(-|z|) is
// e^(-z^2 / 2) P(t), t = 1 / (1 + c |z|), with a P fitted to it by minimax of the
// relative error up to |z| = 13.5, where fp32 ends.  fp32: c = 0.35, degree 9, to 3e-8
// (3e-7 with the roundings of fp32, which the exponential's argument adds z^2 6e-8
// to); erfcf took 5% longer on a whole block's gradients.  16 bits: c = 0.29, degree
// 6, to 5e-8 absolute and 2e-5 of the value up to |z| = 5.8 (where fp16 ends; half its
// step is 4.9e-4), 3.3e-4 of it beyond (half a step of bf16 is 3.9e-3).
__device__ __forceinline__ float logistic(float z) {
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-1.44269504f * z));
}
// Phi(z) and e = exp(-z^2 / 2).
template <int DT>
__device__ __forceinline__ float normal_cdf(float z, float& e) {
  e = __builtin_amdgcn_exp2f(-0.72134752f * z * z);
  const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(DT == OIDN_F32 ? 0.35f : 0.29f, __builtin_fabsf(z), 1.f));
  float p;
  if constexpr (DT == OIDN_F32) {
    p = 0.139621571f + t * (0.13985908f + t * (0.119852439f + t * (0.105432935f + t * (-0.0229371302f +
        t * (0.158929259f + t * (-0.255504519f + t * (0.143872216f + t * -0.02912586f)))))));
  } else {
    p = 0.117000229f + t * (0.0996669881f + t * (0.182742287f + t * (-0.097846044f + t * (0.288142841f +
        t * -0.0897063499f))));
  }
  const float q = e * (t * p);
  return z < 0.f ? q : 1.f - q;
}

// Past |z| = 100 (silu) and 30 (gelu) the functions have reached 0, z and the
// slopes 0, 1 in fp32; holding the factor z there keeps infinities from giving
// 0 * inf.  NaN stays NaN through the other factor.
template <int DT>
__device__ __forceinline__ float activate(int act, float z) {
  if (act == OIDN_ACT_RELU) return z < 0.f ? 0.f : z;
  if (act == OIDN_ACT_SILU) return fmaxf(z, -100.f) * logistic(z);
  if (act == OIDN_ACT_GELU) {
    float e;
    return fmaxf(z, -30.f) * normal_cdf<DT>(z, e);
  }
  return z;
}
// act(z) and act'(z); relu'(0) = 0.
template <int DT>
__device__ __forceinline__ void activate_slope(int act, float z, float& a, float& s) {
  if (act == OIDN_ACT_RELU) {
    a = z < 0.f ? 0.f : z;
    s = z > 0.f ? 1.f : z - z;                       // NaN where z is
    s = z < 0.f ? 0.f : s;
  } else if (act == OIDN_ACT_SILU) {
    const float p = logistic(z), c = fminf(fmaxf(z, -100.f), 100.f);
    a = fmaxf(z, -100.f) * p;
    s = p + c * p * (1.f - p);
  } else if (act == OIDN_ACT_GELU) {
    float e;
    const float p = normal_cdf<DT>(z, e), c = fminf(fmaxf(z, -30.f), 30.f);
    a = fmaxf(z, -30.f) * p;
    s = p + c * e * 0.39894228f;
  } else {
    a = z;
    s = 1.f;
  }
}

// ------------------------------------------------------ 8-bit checkpoints
// A block is 32 columns of a row: s = bf16(max|x| / 127), q = rint(x / s).  The
// error is at most half a step of s: the rounding of s leaves max|x| / s at most
// 127.5, so the clamp to 127 costs no more.  Blocks whose scale falls below
// 2^-120 are stored as zeros; a block with an infinity or a NaN gets the scale
// NaN, so all of it reads back as NaN and the gradients it enters show it.
__device__ __forceinline__ float bf16_round(float v) { return (float)(__bf16)v; }

struct CkptAt {
  signed char* codes;
  __bf16* scales;
  long pitch;              // codes per row
};
__device__ __forceinline__ CkptAt ckpt_at(void* blob, long rows, long cols) {
  const long pitch = (cols + kCkptBlock - 1) / kCkptBlock * kCkptBlock;
  return {static_cast<signed char*>(blob),
          reinterpret_cast<__bf16*>(static_cast<char*>(blob) + rows * pitch), pitch};
}
__device__ __forceinline__ long ckpt_size(long rows, long cols) {
  const long codes = rows * ((cols + kCkptBlock - 1) / kCkptBlock * kCkptBlock);
  return (codes + codes / (kCkptBlock / 2) + 255) / 256 * 256;
}

// Scale of a block from the bits of its largest magnitude (infinities and NaN
// are the largest bit patterns).  The division by 127 is a multiplication and
// one correction step, which rounds it correctly.
__device__ __forceinline__ float ckpt_scale(unsigned top) {
  if (top >= 0x7f800000u) return __builtin_nanf("");
  const float t = __uint_as_float(top), r = 1.f / 127.f, q = t * r;
  const float s = bf16_round(__builtin_fmaf(__builtin_fmaf(-q, 127.f, t), r, q));
  return s < 7.52316385e-37f ? 0.f : s;
}
// The quotient takes one correction step, so that ties are ties (common where x
// has few bits); adding 1.5 * 2^23 rounds to a whole number, nearest even, and
// leaves its two's complement in the low byte.
__device__ __forceinline__ uint2 ckpt_codes(const Eight& x, float s) {
  const float inv = s > 0.f ? __builtin_amdgcn_rcpf(s) : 0.f, magic = 12582912.f;
  unsigned q[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float t = x.v[k] * inv, exact = __builtin_fmaf(__builtin_fmaf(-t, s, x.v[k]), inv, t);
    q[k] = __float_as_uint(__builtin_amdgcn_fmed3f(exact + magic, magic - 127.f, magic + 127.f));
  }
  auto four = [&](const unsigned* p) {        // low bytes of four values
    return __builtin_amdgcn_perm(__builtin_amdgcn_perm(p[3], p[2], 0x0c0c0400),
                                 __builtin_amdgcn_perm(p[1], p[0], 0x0c0c0400), 0x05040100);
  };
  return make_uint2(four(q), four(q + 4));
}
__device__ __forceinline__ unsigned top_of(const Eight& x) {
  unsigned t = 0;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const unsigned a = __float_as_uint(x.v[k]) & 0x7fffffffu;
    t = a > t ? a : t;
  }
  return t;
}
// The largest over the lanes XOR 1 and XOR 2 (in the lane's quad).
__device__ __forceinline__ unsigned top_of_quad(unsigned t) {
  unsigned o = __builtin_amdgcn_mov_dpp(t, 0xB1, 0xF, 0xF, false);
  t = o > t ? o : t;
  o = __builtin_amdgcn_mov_dpp(t, 0x4E, 0xF, 0xF, false);
  return o > t ? o : t;
}
// Stores eight columns of a row.  The four neighbouring lanes that hold a block
// call it together; columns past `cols` must hold 0.
__device__ __forceinline__ void ckpt_store8(const CkptAt& c, long i, int j, const Eight& x,
                                            bool row_ok) {
  const float s = ckpt_scale(top_of_quad(top_of(x)));
  if (row_ok && j < c.pitch) {
    *reinterpret_cast<uint2*>(c.codes + i * c.pitch + j) = ckpt_codes(x, s);
    if (j % kCkptBlock == 0) c.scales[(i * c.pitch + j) / kCkptBlock] = (__bf16)s;
  }
}
// ---------------------------------------------------------------- epilogues
// Eight columns j .. j + 7 (j a multiple of 8) of row i.  fetch() reads what
// the epilogue needs from memory, finish() computes and stores; apart, so that
// several rows' reads are in flight together.  All lanes call finish(): the
// 8-bit stores exchange maxima between the four lanes of a block.
// WHOLE: all eight columns exist, so no element is looked at by itself.
__device__ __forceinline__ Eight bias8(const float* bias, int j, int n) {
  Eight b{};
  if (bias) {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < n) b.v[k] = bias[j + k];
  }
  return b;
}
__device__ __forceinline__ void add8(Eight& x, const Eight& b) {
#pragma unroll
  for (int k = 0; k < 8; ++k) x.v[k] += b.v[k];
}
__device__ __forceinline__ void clear_tail(int n, Eight& x) {
#pragma unroll
  for (int k = 0; k < 8; ++k)
    if (k >= n) x.v[k] = 0.f;
}
// The activation is the same for the whole launch: one branch for eight values.
template <int DT>
__device__ __forceinline__ void activate8(int act, Eight& x) {
  if (act == OIDN_ACT_RELU) {
#pragma unroll
    for (int k = 0; k < 8; ++k) x.v[k] = activate<DT>(OIDN_ACT_RELU, x.v[k]);
  } else if (act == OIDN_ACT_SILU) {
#pragma unroll
    for (int k = 0; k < 8; ++k) x.v[k] = activate<DT>(OIDN_ACT_SILU, x.v[k]);
  } else if (act == OIDN_ACT_GELU) {
#pragma unroll
    for (int k = 0; k < 8; ++k) x.v[k] = activate<DT>(OIDN_ACT_GELU, x.v[k]);
  }
}
// g = act(z), z becomes act'(z).
template <int DT>
__device__ __forceinline__ void activate_slope8(int act, Eight& z, Eight& g) {
  if (act == OIDN_ACT_RELU) {
#pragma unroll
    for (int k = 0; k < 8; ++k) activate_slope<DT>(OIDN_ACT_RELU, z.v[k], g.v[k], z.v[k]);
  } else if (act == OIDN_ACT_SILU) {
#pragma unroll
    for (int k = 0; k < 8; ++k) activate_slope<DT>(OIDN_ACT_SILU, z.v[k], g.v[k], z.v[k]);
  } else if (act == OIDN_ACT_GELU) {
#pragma unroll
    for (int k = 0; k < 8; ++k) activate_slope<DT>(OIDN_ACT_GELU, z.v[k], g.v[k], z.v[k]);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      g.v[k] = z.v[k];
      z.v[k] = 1.f;
    }
  }
}

struct Fetched { Eight a, b; };

// What fetch() has read, as it is stored: eight elements, or eight codes and a
// scale (fewer registers than their values, so more of them can be in flight).
template <int DT>
struct Raw {
  typedef typename Storage<DT>::T T;
  typedef T T8 __attribute__((ext_vector_type(8)));
  T8 e;
  __device__ __forceinline__ Eight value() const {
    Eight r;
#pragma unroll
    for (int k = 0; k < 8; ++k) r.v[k] = (float)e[k];
    return r;
  }
};
struct RawCodes {
  uint2 q;
  __bf16 s;
  __device__ __forceinline__ Eight value() const {
    Eight r;
#pragma unroll
    for (int k = 0; k < 8; ++k)
      r.v[k] = (float)s * (float)(int)(signed char)((k < 4 ? q.x : q.y) >> (8 * (k % 4)));
    return r;
  }
};
// Z8: the saved z of kEpiGatedBack is held in 8 bits.
template <int DT, bool Z8> struct RawFetched { Raw<DT> a, b; };
template <int DT> struct RawFetched<DT, true> { RawCodes a, b; };

// n of the elements are wanted; the rest may be anything, so that only where the
// matrix ends within eight elements (`left` from here on) single ones are read.
template <int DT>
__device__ __forceinline__ Raw<DT> load_raw(const void* p, long i, int n, long left) {
  typedef typename Storage<DT>::T T;
  const T* s = static_cast<const T*>(p) + i;
  Raw<DT> r;
  if (left >= 8) {
    __builtin_memcpy(&r.e, s, sizeof(r.e));
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) r.e[k] = k < n ? s[k] : (T)0.f;
  }
  return r;
}
__device__ __forceinline__ RawCodes load_codes(const CkptAt& c, long i, int j) {
  return {*reinterpret_cast<const uint2*>(c.codes + i * c.pitch + j), c.scales[(i * c.pitch + j) / kCkptBlock]};
}

__device__ __forceinline__ Eight ckpt_load8(const CkptAt& c, long i, int j) { return load_codes(c, i, j).value(); }

// Values that go back to type DT.  The rounding of a block's scale can carry its
// largest value past the type's range (fp16: 127 x 516 = 65532); up to the scale
// that the type's largest value gets, such a value is that largest one, beyond
// (sums that were kept in 8 bits) it is infinite.  NaN, the scale of a block with
// no finite maximum, stays.  In fp32 127 times the largest scale is finite.
template <int DT>
__device__ __forceinline__ Eight ckpt_stored(const RawCodes& c) {
  Eight r = c.value();
  if constexpr (DT != OIDN_F32) {
    const float top = DT == OIDN_F16 ? 0x1.02p9f : 0x1.02p121f, most = DT == OIDN_F16 ? 65504.f : 0x1.fep127f;
    const float s = (float)c.s, limit = s <= top ? most : s * __builtin_inff();
#pragma unroll
    for (int k = 0; k < 8; ++k) r.v[k] = __builtin_amdgcn_fmed3f(r.v[k], -limit, limit);
  }
  return r;
}

template <int DT, int EPI, bool WHOLE, bool Z8>
__device__ __forceinline__ void fetch(const EpilogueArgs& e, long i, int j, RawFetched<DT, Z8>& f) {
  if constexpr (EPI == kEpiPartial || EPI == kEpiGated) return;
  const int n = e.cols - j;                 // columns that exist from j on
  if (!WHOLE && n <= 0) return;
  i = i < e.rows ? i : e.rows - 1;
  const long below = e.rows - 1 - i;        // rows after this one
  if constexpr (EPI == kEpiLinear || EPI == kEpiStore) {
    if (e.res) f.a = load_raw<DT>(e.res, i * e.ldr + j, n, WHOLE ? 8 : below * e.ldr + n);
  }
  if constexpr (EPI == kEpiGatedBack) {
    if constexpr (Z8) {
      f.a = load_codes(ckpt_at(e.z, e.rows, e.cols), i, j);
      f.b = load_codes(ckpt_at(static_cast<char*>(e.z) + ckpt_size(e.rows, e.cols), e.rows, e.cols), i, j);
    } else {
      f.a = load_raw<DT>(e.z, i * e.ldz + j, n, WHOLE ? 8 : below * e.ldz + e.cols + n);
      f.b = load_raw<DT>(e.z, i * e.ldz + e.cols + j, n, WHOLE ? 8 : below * e.ldz + n);
    }
  }
}

// x: the sums (kEpiGated: the gate's, u the up projection's); bias: that of
// the same columns, zeros if there is none.  kEpiGatedBack adds da and db to
// sums.
template <int DT, int EPI, bool WHOLE, bool Z8, bool STREAM = false>
__device__ __forceinline__ void finish(const EpilogueArgs& e, int slice, long i, int j, Eight x, Eight u,
                                       const Fetched& bias, const RawFetched<DT, Z8>& f, Fetched& sums) {
  const int n = WHOLE ? 8 : e.cols - j;
  const bool row_ok = i < e.rows, ok = row_ok && n > 0;
  if constexpr (EPI == kEpiPartial) {       // fp32 sums of one slice
    if (ok)
      store8<OIDN_F32>(e.part, ((long)slice * e.rows + i) * e.cols + j, x, n);
  } else if constexpr (EPI == kEpiStore) {
    if (e.res) add8(x, f.a.value());
    if (ok) store8<DT, WHOLE && STREAM>(e.y, i * e.ldy + j, x, n);
  } else if constexpr (EPI == kEpiLinear) {
    add8(x, bias.a);
    if (e.z) {
      if (e.z8) {
        if constexpr (!WHOLE) clear_tail(n, x);
        ckpt_store8(ckpt_at(e.z, e.rows, e.cols), i, j, x, row_ok);
      } else if (ok) {
        store8<DT>(e.z, i * e.ldz + j, x, n);
      }
    }
    activate8<DT>(e.act, x);
    if (e.res) add8(x, f.a.value());
    if (ok) store8<DT, WHOLE && STREAM>(e.y, i * e.ldy + j, x, n);
  } else if constexpr (EPI == kEpiGated) {
    add8(x, bias.a);
    add8(u, bias.b);
    if (e.z) {
      if (e.z8) {
        if constexpr (!WHOLE) {
          clear_tail(n, x);
          clear_tail(n, u);
        }
        ckpt_store8(ckpt_at(e.z, e.rows, e.cols), i, j, x, row_ok);
        ckpt_store8(ckpt_at(static_cast<char*>(e.z) + ckpt_size(e.rows, e.cols), e.rows, e.cols),
                          i, j, u, row_ok);
      } else if (ok) {
        store8<DT>(e.z, i * e.ldz + j, x, n);
        store8<DT>(e.z, i * e.ldz + e.cols + j, u, n);
      }
    }
    activate8<DT>(e.act, x);
    // h is rounded to the storage type, as the second product's matrix cores take it
    // (y of a block is off by 0.0019 in bf16 and 0.00023 in fp16, where an fp32 h
    // would leave 0.0017 and 0.00021, its own rounding)
#pragma unroll
    for (int k = 0; k < 8; ++k) x.v[k] *= u.v[k];
    if (ok) store8<DT>(e.y, i * e.ldy + j, x, n);
  } else {                                  // x is dh: h and [da | db]
    Eight a = f.a.value(), g, h, da, db;
    const Eight b = f.b.value();
    activate_slope8<DT>(e.act, a, g);
    if (!ok) return;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      h.v[k] = g.v[k] * b.v[k];
      da.v[k] = x.v[k] * b.v[k] * a.v[k];
      db.v[k] = x.v[k] * g.v[k];
      if (k < n) {
        sums.a.v[k] += da.v[k];
        sums.b.v[k] += db.v[k];
      }
    }
    // rounded to what the gradients' products read, 16-bit operands of the matrix
    // cores: dx and both dw then carry two roundings, sqrt 2 of the output's own; the
    // column sums above are of the unrounded values
    store8<DT>(e.h, i * (long)e.cols + j, h, n);
    store8<DT>(e.y, i * e.ldy + j, da, n);
    store8<DT>(e.y, i * e.ldy + e.cols + j, db, n);
  }
}

// The epilogue of a wave's 16 FR x 16 FC quarter of a tile, whose accumulators
// are in pairs of column fragments: lane l holds row l % 16 of row fragment r
// and columns 8 (l / 16) + 4 q .. + 3 of a pair's 32 in fragment q.  They pass
// through the wave's own part of LDS, so that a row's columns leave in one
// contiguous run and one copy of the epilogue's code serves all of them:
// 16-byte unit u of row r sits at u ^ (r % 16), which keeps both the writes
// (16 rows of a unit) and the reads (neighbouring units of a row) on distinct
// banks.  kEpiGated: the first half of the columns is the gate's.
// lds: epilogue_bytes of this wave; i0, j0: its first row and column; slice:
// -1 for a whole sum, else the slice that kEpiPartial stores; group: its row
// of the partial column sums.
template <int FR, int FC>
constexpr int epilogue_rows() { return FR * FC > 32 ? 8 * FR : 16 * FR; }
template <int FR, int FC>
constexpr int epilogue_bytes() { return epilogue_rows<FR, FC>() * 64 * FC; }

// Results kept in the caches, past them, or as e.stream has it.
enum Caching { kKept, kStreamed, kEither };

template <int DT, int EPI, int FR, int FC, bool Z8 = false, Caching WHERE = kKept>
__device__ __forceinline__ void tile_epilogue(const EpilogueArgs& e, const floatx4 (&acc)[FC][FR], char* lds,
                                              long i0, int j0, int slice, long group) {
  if constexpr (EPI == kEpiLinear || EPI == kEpiStore) {
    if (slice >= 0) return tile_epilogue<DT, kEpiPartial, FR, FC>(e, acc, lds, i0, j0, slice, group);
    if constexpr (WHERE == kEither) {
      if (e.stream) return tile_epilogue<DT, EPI, FR, FC, Z8, kStreamed>(e, acc, lds, i0, j0, slice, group);
      return tile_epilogue<DT, EPI, FR, FC, Z8, kKept>(e, acc, lds, i0, j0, slice, group);
    }
  }
  if constexpr (EPI == kEpiGatedBack && !Z8) {
    if (e.z8) return tile_epilogue<DT, EPI, FR, FC, true>(e, acc, lds, i0, j0, slice, group);
  }
  constexpr int kRows = epilogue_rows<FR, FC>();       // rows per round
  constexpr int kUnits = 4 * FC;                       // 16-byte units of a row
  constexpr int kMask = kUnits < 16 ? kUnits - 1 : 15;
  constexpr bool kGated = EPI == kEpiGated;
  constexpr int kLanes = kGated ? FC : 2 * FC;         // lanes per row, eight columns each
  constexpr int kAtOnce = 64 / kLanes;                 // rows per step
  constexpr int kSteps = kRows / kAtOnce;
  const int lane = threadIdx.x & 63, g = lane >> 4;
  const int c = lane % kLanes, j = j0 + 8 * c;
  auto unit = [&](int row, int u) -> floatx4& {
    return *reinterpret_cast<floatx4*>(lds + (row * kUnits + (u ^ (row & kMask))) * 16);
  };
  Fetched bias{}, sums{};
  if constexpr (EPI == kEpiLinear || kGated) {
    bias.a = bias8(e.bias, j, e.cols - j);
    if constexpr (kGated) bias.b = bias8(e.bias ? e.bias + e.cols : nullptr, j, e.cols - j);
  }
  // steps whose reads are in flight together; the first ones' are issued before
  // the accumulators go to LDS
  constexpr bool kReads = EPI != kEpiPartial && EPI != kEpiGated;
  constexpr int kTogether = kSteps < 8 ? kSteps : kReads ? 8 : 4;
  RawFetched<DT, Z8> got[kReads ? kTogether : 1];
  const bool whole = j0 + 8 * kLanes <= e.cols;
  auto read = [&](long ir, int s) {
    if constexpr (kReads) {
      if (whole) {
#pragma unroll
        for (int k = 0; k < kTogether; ++k) fetch<DT, EPI, true, Z8>(e, ir + (s + k) * kAtOnce, j, got[k]);
      } else {
#pragma unroll
        for (int k = 0; k < kTogether; ++k) fetch<DT, EPI, false, Z8>(e, ir + (s + k) * kAtOnce, j, got[k]);
      }
    }
  };
  auto step = [&](auto is_whole, long ir, int s, RawFetched<DT, Z8>& f) {
    constexpr bool kWhole = decltype(is_whole)::value;
    const int row = s * kAtOnce + lane / kLanes;
    Eight x, u{};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const floatx4 v = unit(row, 2 * c + h);
#pragma unroll
      for (int m = 0; m < 4; ++m) x.v[4 * h + m] = v[m];
      if constexpr (kGated) {
        const floatx4 w = unit(row, kUnits / 2 + 2 * c + h);
#pragma unroll
        for (int m = 0; m < 4; ++m) u.v[4 * h + m] = w[m];
      }
    }
    finish<DT, EPI, kWhole, Z8, WHERE == kStreamed>(e, slice, ir + s * kAtOnce, j, x, u, bias, f, sums);
  };
  constexpr int kRounds = 16 * FR / kRows;
#pragma unroll 1
  for (int round = 0; round < kRounds; ++round) {
    const long ir = i0 + round * kRows + lane / kLanes;
    read(ir, 0);
#pragma unroll
    for (int k = 0; k < kRounds; ++k)
      if (round == k) {
#pragma unroll
        for (int f = 0; f < FC; ++f)
#pragma unroll
          for (int r = 0; r < kRows / 16; ++r)
            unit(16 * r + (lane & 15), 8 * (f / 2) + 2 * g + f % 2) = acc[f][k * (kRows / 16) + r];
      }
    // the wave's own writes, back in order
    __builtin_amdgcn_wave_barrier();
#pragma unroll 1
    for (int s = 0; s < kSteps; s += kTogether) {
      if (s) read(ir, s);
      if (whole) {
#pragma unroll
        for (int k = 0; k < kTogether; ++k) step(std::true_type{}, ir, s + k, got[kReads ? k : 0]);
      } else {
#pragma unroll
        for (int k = 0; k < kTogether; ++k) step(std::false_type{}, ir, s + k, got[kReads ? k : 0]);
      }
    }
    __builtin_amdgcn_wave_barrier();
  }
  if constexpr (EPI == kEpiGatedBack) {
    if (!e.part) return;
    // rows of the other lanes with the same columns
#pragma unroll
    for (int s = kLanes; s < 64; s *= 2)
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        sums.a.v[k] += __shfl_xor(sums.a.v[k], s);
        sums.b.v[k] += __shfl_xor(sums.b.v[k], s);
      }
    if (lane >= kLanes) return;
    float* const row = e.part + group * 2 * e.cols;
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (j + k < e.cols) {
        row[j + k] = sums.a.v[k];
        row[e.cols + j + k] = sums.b.v[k];
      }
  }
}

}  // namespace
}  // namespace oidn
