// Device code shared by the dense operators: storage types, activations and
// their slopes, 8-bit checkpoint blocks, and the epilogues that the tile
// kernels and the slice sum run on eight neighbouring columns of one row.
#pragma once

#include "dense.h"
#include "mfma_common.h"

namespace oidn {
namespace {

typedef float floatx8 __attribute__((ext_vector_type(8)));
typedef _Float16 halfx8 __attribute__((ext_vector_type(8)));

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

// Eight elements from element offset i; `vec`: the address is a multiple of
// 16 bytes and all eight exist, else only the first n are read (0 after).
template <int DT>
__device__ __forceinline__ Eight load8(const void* p, long i, bool vec, int n) {
  typedef typename Storage<DT>::T T;
  const T* s = static_cast<const T*>(p) + i;
  Eight r;
  if (vec) {
    if constexpr (DT == OIDN_F32) {
      const float4 a = reinterpret_cast<const float4*>(s)[0], b = reinterpret_cast<const float4*>(s)[1];
      r.v[0] = a.x; r.v[1] = a.y; r.v[2] = a.z; r.v[3] = a.w;
      r.v[4] = b.x; r.v[5] = b.y; r.v[6] = b.z; r.v[7] = b.w;
    } else {
      const uint4 u = *reinterpret_cast<const uint4*>(s);
      typedef T T8 __attribute__((ext_vector_type(8)));
      const T8 t = __builtin_bit_cast(T8, u);
#pragma unroll
      for (int k = 0; k < 8; ++k) r.v[k] = (float)t[k];
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) r.v[k] = k < n ? (float)s[k] : 0.f;
  }
  return r;
}

template <int DT>
__device__ __forceinline__ void store8(void* p, long i, const Eight& r, bool vec, int n) {
  typedef typename Storage<DT>::T T;
  T* s = static_cast<T*>(p) + i;
  if (vec) {
    if constexpr (DT == OIDN_F32) {
      reinterpret_cast<float4*>(s)[0] = make_float4(r.v[0], r.v[1], r.v[2], r.v[3]);
      reinterpret_cast<float4*>(s)[1] = make_float4(r.v[4], r.v[5], r.v[6], r.v[7]);
    } else {
      typedef T T8 __attribute__((ext_vector_type(8)));
      T8 t;
#pragma unroll
      for (int k = 0; k < 8; ++k) t[k] = (T)r.v[k];
      *reinterpret_cast<uint4*>(s) = __builtin_bit_cast(uint4, t);
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < n) s[k] = (T)r.v[k];
  }
}

// -------------------------------------------------------------- activations
// silu(z) = z p with p = 1 / (1 + e^-z); gelu(z) = z Phi(z), Phi the normal
// distribution function (erf form).  fp32 uses erff; the 16-bit types use
// formula 7.1.26 of Abramowitz and Stegun, Handbook of Mathematical Functions
// (|error| <= 1.5e-7, far below half a step of fp16), about a third of the
// instructions.
__device__ __forceinline__ float logistic(float z) {
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-1.44269504f * z));
}
// Phi(z) and e = exp(-z^2 / 2).
template <int DT>
__device__ __forceinline__ float normal_cdf(float z, float& e) {
  e = __builtin_amdgcn_exp2f(-0.72134752f * z * z);
  if constexpr (DT == OIDN_F32) {
    return 0.5f * (1.f + erff(0.70710678f * z));
  } else {
    const float t = __builtin_amdgcn_rcpf(1.f + 0.3275911f * 0.70710678f * __builtin_fabsf(z));
    const float poly = t * (0.254829592f + t * (-0.284496736f +
                       t * (1.421413741f + t * (-1.453152027f + t * 1.061405429f))));
    const float tail = 0.5f * poly * e;        // Phi(-|z|)
    return z >= 0.f ? 1.f - tail : tail;
  }
}

// Past |z| = 100 (silu) and 30 (gelu) the functions have reached 0, z and the
// slopes 0, 1 in fp32; taking them there keeps infinities from giving 0 * inf.
// NaN stays NaN.
template <int DT>
__device__ __forceinline__ float activate(int act, float z) {
  if (act == OIDN_ACT_RELU) return z < 0.f ? 0.f : z;
  if (act == OIDN_ACT_SILU) return z < -100.f ? 0.f : z * logistic(z);
  if (act == OIDN_ACT_GELU) {
    float e;
    return z < -30.f ? 0.f : z * normal_cdf<DT>(z, e);
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
    a = z < -100.f ? 0.f : z * p;
    s = p + c * p * (1.f - p);
  } else if (act == OIDN_ACT_GELU) {
    float e;
    const float p = normal_cdf<DT>(z, e), c = fminf(fmaxf(z, -30.f), 30.f);
    a = z < -30.f ? 0.f : z * p;
    s = p + c * e * 0.39894228f;
  } else {
    a = z;
    s = 1.f;
  }
}

// ------------------------------------------------------ 8-bit checkpoints
// A block is 32 columns of a row: s = bf16(max|x| / 127), q = rint(x / s).
// Taken as x * (1 / s): the code differs from rint(x / s) only where x / s is
// within 2^-16 of a tie.  The error is at most half a step of s: the rounding
// of s leaves max|x| / s at most 127.5, so the clamp to 127 costs no more.
// Blocks whose scale falls below 2^-120 are stored as zeros; a block with an
// infinity or a NaN gets the scale NaN, so all of it reads back as NaN and
// the gradients it enters show it.
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

// Scale of a block from its largest magnitude (NaN if any value is not finite).
__device__ __forceinline__ float ckpt_scale(float top) {
  if (!(top <= 3.4028234e38f)) return __builtin_nanf("");
  const float s = bf16_round(top / 127.f);
  return s < 7.52316385e-37f ? 0.f : s;
}
__device__ __forceinline__ uint2 ckpt_codes(const Eight& x, float s) {
  const float inv = s > 0.f ? 1.f / s : 0.f;
  unsigned w[2] = {0u, 0u};
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float q = fminf(fmaxf(__builtin_rintf(x.v[k] * inv), -127.f), 127.f);
    w[k / 4] |= ((unsigned)(int)q & 255u) << (8 * (k % 4));
  }
  return make_uint2(w[0], w[1]);
}
// Largest magnitude of eight values; a NaN or infinity gives infinity.
__device__ __forceinline__ float top_of(const Eight& x) {
  float t = 0.f;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float a = __builtin_fabsf(x.v[k]);
    t = a <= t ? t : (a == a ? a : __builtin_inff());
  }
  return t;
}
// Stores eight columns of a row.  The four lanes that hold a block (lane XOR
// A, lane XOR B) call it together; columns past `cols` must hold 0.
template <int A, int B>
__device__ __forceinline__ void ckpt_store8(const CkptAt& c, long i, int j, const Eight& x,
                                            bool row_ok) {
  float t = top_of(x);
  t = fmaxf(t, __shfl_xor(t, A));
  t = fmaxf(t, __shfl_xor(t, B));
  const float s = ckpt_scale(t);
  if (row_ok && j < c.pitch) {
    *reinterpret_cast<uint2*>(c.codes + i * c.pitch + j) = ckpt_codes(x, s);
    if (j % kCkptBlock == 0) c.scales[(i * c.pitch + j) / kCkptBlock] = (__bf16)s;
  }
}
__device__ __forceinline__ Eight ckpt_load8(const CkptAt& c, long i, int j) {
  Eight r;
  const uint2 w = *reinterpret_cast<const uint2*>(c.codes + i * c.pitch + j);
  const float s = (float)c.scales[(i * c.pitch + j) / kCkptBlock];
#pragma unroll
  for (int k = 0; k < 8; ++k)
    r.v[k] = s * (float)(int)(signed char)((k < 4 ? w.x : w.y) >> (8 * (k % 4)));
  return r;
}

// ---------------------------------------------------------------- epilogues
// Eight columns j .. j + 7 (j a multiple of 8) of row i; row_ok: the row
// exists.  All lanes call them (the 8-bit stores exchange maxima between the
// lanes XOR A and XOR B).
__device__ __forceinline__ void add_bias(const float* bias, int j, int n, Eight& x) {
#pragma unroll
  for (int k = 0; k < 8; ++k)
    if (k < n) x.v[k] += bias[j + k];
}
__device__ __forceinline__ void clear_tail(int n, Eight& x) {
#pragma unroll
  for (int k = 0; k < 8; ++k)
    if (k >= n) x.v[k] = 0.f;
}

template <int DT, int A, int B>
__device__ __forceinline__ void epilogue_linear(const EpilogueArgs& e, long i, int j, Eight x,
                                                bool row_ok) {
  const int n = e.cols - j;                 // columns that exist from j on
  const bool full = n >= 8;
  if (e.bias) add_bias(e.bias, j, n, x);
  if (e.z) {
    if (e.z8) {
      clear_tail(n, x);
      ckpt_store8<A, B>(ckpt_at(e.z, e.rows, e.cols), i, j, x, row_ok);
    } else if (row_ok && n > 0) {
      store8<DT>(e.z, i * e.ldz + j, x, full && (e.vec & kVecZ), n);
    }
  }
  if (!row_ok || n <= 0) return;
  if (e.act != OIDN_ACT_NONE) {
#pragma unroll
    for (int k = 0; k < 8; ++k) x.v[k] = activate<DT>(e.act, x.v[k]);
  }
  if (e.res) {
    const Eight r = load8<DT>(e.res, i * e.ldr + j, full && (e.vec & kVecRes), n);
#pragma unroll
    for (int k = 0; k < 8; ++k) x.v[k] += r.v[k];
  }
  store8<DT>(e.y, i * e.ldy + j, x, full && (e.vec & kVecY), n);
}

// fp32 sums of one slice.
__device__ __forceinline__ void epilogue_partial(const EpilogueArgs& e, int slice, long i, int j,
                                                 const Eight& x, bool row_ok) {
  const int n = e.cols - j;
  if (!row_ok || n <= 0) return;
  store8<OIDN_F32>(e.part, ((long)slice * e.rows + i) * e.cols + j, x,
                   n >= 8 && (e.cols & 3) == 0, n);
}

// a, b: columns j of the gate and of the up projection.
template <int DT, int A, int B>
__device__ __forceinline__ void epilogue_gated(const EpilogueArgs& e, long i, int j, Eight a,
                                               Eight b, bool row_ok) {
  const int n = e.cols - j;
  const bool full = n >= 8;
  if (e.bias) {
    add_bias(e.bias, j, n, a);
    add_bias(e.bias + e.cols, j, n, b);
  }
  if (e.z) {
    if (e.z8) {
      clear_tail(n, a);
      clear_tail(n, b);
      ckpt_store8<A, B>(ckpt_at(e.z, e.rows, e.cols), i, j, a, row_ok);
      ckpt_store8<A, B>(ckpt_at(static_cast<char*>(e.z) + ckpt_size(e.rows, e.cols), e.rows, e.cols),
                        i, j, b, row_ok);
    } else if (row_ok && n > 0) {
      store8<DT>(e.z, i * e.ldz + j, a, full && (e.vec & kVecZ), n);
      store8<DT>(e.z, i * e.ldz + e.cols + j, b, full && (e.vec & kVecZ), n);
    }
  }
  if (!row_ok || n <= 0) return;
#pragma unroll
  for (int k = 0; k < 8; ++k) a.v[k] = activate<DT>(e.act, a.v[k]) * b.v[k];
  store8<DT>(e.y, i * e.ldy + j, a, full && (e.vec & kVecY), n);
}

// dh: columns j of dy w_out.  Writes h and [da | db] and adds da, db to sa, sb
// (0 where nothing exists).
template <int DT>
__device__ __forceinline__ void epilogue_gated_back(const EpilogueArgs& e, long i, int j, Eight dh,
                                                    bool row_ok, Eight& sa, Eight& sb) {
  const int n = e.cols - j;
  const bool full = n >= 8;
  if (!row_ok || n <= 0) return;
  Eight a, b, h;
  if (e.z8) {
    void* z = e.z;
    a = ckpt_load8(ckpt_at(z, e.rows, e.cols), i, j);
    b = ckpt_load8(ckpt_at(static_cast<char*>(z) + ckpt_size(e.rows, e.cols), e.rows, e.cols), i, j);
  } else {
    a = load8<DT>(e.z, i * e.ldz + j, full && (e.vec & kVecZ), n);
    b = load8<DT>(e.z, i * e.ldz + e.cols + j, full && (e.vec & kVecZ), n);
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    float g, s;
    activate_slope<DT>(e.act, a.v[k], g, s);
    h.v[k] = g * b.v[k];
    a.v[k] = dh.v[k] * b.v[k] * s;
    b.v[k] = dh.v[k] * g;
    if (k < n) {
      sa.v[k] += a.v[k];
      sb.v[k] += b.v[k];
    }
  }
  store8<DT>(e.h, i * (long)e.cols + j, h, full && (e.vec & kVecH), n);
  store8<DT>(e.y, i * e.ldy + j, a, full && (e.vec & kVecY), n);
  store8<DT>(e.y, i * e.ldy + e.cols + j, b, full && (e.vec & kVecY), n);
}

// Column sums of a wave's rows: adds over the 16 lanes of a row fragment and
// stores them as row `group` of the partial sums (2 * cols wide, da then db).
__device__ __forceinline__ void store_column_sums(const EpilogueArgs& e, long group, int j,
                                                  Eight sa, Eight sb) {
#pragma unroll
  for (int s = 1; s < 16; s *= 2)
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      sa.v[k] += __shfl_xor(sa.v[k], s);
      sb.v[k] += __shfl_xor(sb.v[k], s);
    }
  if (threadIdx.x & 15) return;
  float* const row = e.part + group * 2 * e.cols;
#pragma unroll
  for (int k = 0; k < 8; ++k)
    if (j + k < e.cols) {
      row[j + k] = sa.v[k];
      row[e.cols + j + k] = sb.v[k];
    }
}

}  // namespace
}  // namespace oidn
