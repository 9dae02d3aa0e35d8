// 16-bit matrix products on the matrix cores, C[i][j] = sum_l Q(i, l) P(j, l)
// (see dense.h for the operands' layouts).
//
// A workgroup of 2 x 2 waves computes a TR x TC tile of C, each wave a
// quarter of it in 16 x 16 fragments of v_mfma_f32_16x16x32.  P is the MFMA's A
// operand (its rows are C's columns), so a lane's accumulator holds
// neighbouring columns of one row: fragments go in pairs whose rows are dealt
// so that lane group g of a pair owns the 8 columns 32 p + 8 g .. + 7.
//
// kDenseK = 64 summed elements are staged at a time, through registers into
// one of two LDS buffers: the loads of the next two or three tiles are in
// flight while the current one is multiplied.  An l-fastest operand keeps rows of 64 elements
// (128 B); its 16-byte slot s of row r sits at s ^ (r / 2 % 8), which spreads
// the 16 rows that a fragment read touches over all banks.  A strided operand
// keeps rows of T elements, one per l, and is read with the transposing
// ds_read_b64_tr_b16: four rows of l by 16 columns per 16 lanes; slot s of
// row l sits at s ^ 4 (l % 4) (T = 64: s ^ 4 (l / 2 % 2)), which puts those
// four rows on different banks.
//
// Rows and columns past the matrix are read from its last row or as zeros and
// never stored; elements past the summed length are zeros in both operands.
// Loads are 16 bytes wide at any 2-byte alignment.  This form is for operands
// that the direct one (dense_gemm16_direct.h) does not take: odd pitches, bases
// and sizes.  4096 x 4096 x 2048 takes 82 to 91 us (838 to 758 TFLOP/s; direct 57 to
// 67, by the card), with odd pitches, whose loads straddle lines, 100 to 105.
#pragma once

#include "dense_epilogue.h"
#include "dense_load.h"

namespace oidn {
namespace {

typedef short shortx4 __attribute__((ext_vector_type(4)));

// One operand's tile in LDS: T rows of the output side x 64 of l.
template <int T, bool STRIDED, int THREADS_>
struct Stage16 {
  static constexpr int kUnits = T * kDenseK / 8 / THREADS_;   // 16-byte units per thread
  static constexpr int kBytes = T * kDenseK * 2;

  static __device__ __forceinline__ int slot(int row, int s) {
    if constexpr (!STRIDED) return row * 8 + (s ^ ((row >> 1) & 7));
    else if constexpr (T >= 128) return row * (T / 8) + (s ^ ((row & 3) << 2));
    else return row * (T / 8) + (s ^ ((row & 2) << 1));
  }

  static __device__ __forceinline__ void store(const uint4 (&u)[kUnits], char* lds) {
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
      const int t = threadIdx.x + k * THREADS_;
      const int at = STRIDED ? slot(t / (T / 8), t % (T / 8)) : slot(t >> 3, t & 7);
      *reinterpret_cast<uint4*>(lds + 16 * at) = u[k];
    }
  }

  // Fragment of 16 output rows for summed elements 32 kk .. + 31: lane l holds
  // its row's elements 32 kk + 8 (l / 16) .. + 7.  PAIR: row r of fragment q
  // is tile row base + 8 (r / 4) + 4 q + r % 4; else base + 16 q + r.
  template <bool PAIR>
  static __device__ __forceinline__ uint4 fragment(const char* lds, int base, int q, int kk) {
    const int lane = threadIdx.x & 63, g = lane >> 4, r = lane & 15;
    if constexpr (!STRIDED) {
      const int row = base + (PAIR ? 8 * (r >> 2) + 4 * q + (r & 3) : 16 * q + r);
      return *reinterpret_cast<const uint4*>(lds + 16 * slot(row, 4 * kk + g));
    } else {
      const int c = r & 3;       // 4-column chunk of the 16 that this lane reads
      const int col = base + (PAIR ? 8 * c + 4 * q : 16 * q + 4 * c);
      typedef __attribute__((address_space(3))) shortx4* lds4;
      uint2 h[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int l = 32 * kk + 8 * g + 4 * e + (r >> 2);
        const char* p = lds + 16 * slot(l, col >> 3) + 2 * (col & 7);
        h[e] = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)p));
      }
      return make_uint4(h[0].x, h[0].y, h[1].x, h[1].y);
    }
  }
};

template <int TR, int TC>
constexpr int gemm16_lds() { return 2 * (TR + TC) * kDenseK * 2; }

// Workgroup `block` of the product; lds: gemm16_lds<TR, TC>() bytes.
template <bool BF, int LAYOUT, int EPI, int TR, int TC, Caching WHERE>
__device__ __forceinline__ void gemm16_staged(const GemmArgs& a, int block, char* lds) {
  constexpr int DT = BF ? OIDN_BF16 : OIDN_F16;
  constexpr bool PS = LAYOUT != kForward, QS = LAYOUT == kWeightGrad;
  constexpr int FR = TR / 32, FC = TC / 32;      // 16-wide fragments per wave
  static_assert(EPI != kEpiGated || FC % 4 == 0, "a wave holds pairs of both projections");
  typedef Stage16<TC, PS, 256> P;
  typedef Stage16<TR, QS, 256> Q;

  int tc, tr;
  int slice;
  if (!tile_and_slice(a, block, tc, tr, slice)) return;
  const long i0 = (long)tr * TR;
  // a gated tile covers TC / 2 columns of both projections
  constexpr int C = EPI == kEpiGated ? TC / 2 : TC;
  const long j0 = (long)tc * C;
  const long half = EPI == kEpiGated ? a.e.cols : 0;
  const int wave = threadIdx.x >> 6, wr = wave >> 1, wc = wave & 1;
  const long t0 = (long)slice * a.per_split;
  const long nt = (a.len + kDenseK - 1) / kDenseK;
  const long t1 = t0 + a.per_split < nt ? t0 + a.per_split : nt;

  floatx4 acc[FC][FR];
#pragma unroll
  for (int c = 0; c < FC; ++c)
#pragma unroll
    for (int r = 0; r < FR; ++r) acc[c][r] = floatx4{0.f, 0.f, 0.f, 0.f};

  // Tiles in flight in registers; tile t waits in set (t - t0) % kAhead.
  constexpr int kAhead = TR * TC > 64 * 128 ? 2 : 3;
  Loader<2, TC, kDenseK, PS> from_p(a.p, a.ldp, j0, a.e.cols, t0 * kDenseK, a.len, half);
  Loader<2, TR, kDenseK, QS> from_q(a.q, a.ldq, i0, a.e.rows, t0 * kDenseK, a.len, 0);
  uint4 up[kAhead][P::kUnits], uq[kAhead][Q::kUnits];
  auto load = [&](long t, int set) {
    from_p.load(up[set], t * kDenseK);
    from_q.load(uq[set], t * kDenseK);
  };
#pragma unroll
  for (int s = 0; s < kAhead; ++s)
    if (t0 + s < t1) load(t0 + s, s);
  for (long tt = t0; tt < t1; tt += kAhead) {
#pragma unroll
    for (int s = 0; s < kAhead; ++s) {
      const long t = tt + s;
      if (t >= t1) break;
      char* const lp = lds + ((t - t0) & 1) * (P::kBytes + Q::kBytes);
      char* const lq = lp + P::kBytes;
      // this buffer was last read two tiles ago, before the previous barrier
      P::store(up[s], lp);
      Q::store(uq[s], lq);
      __syncthreads();
      if (t + kAhead < t1) load(t + kAhead, s);
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) {
        uint4 fp[FC], fq[FR];
#pragma unroll
        for (int c = 0; c < FC; ++c) {
          // pair c / 2 of the wave: a gated wave's second half is the up side
          const int pair = c / 2;
          const int base = EPI == kEpiGated
                               ? (pair < FC / 4 ? wc * (TC / 4) + 32 * pair
                                                : TC / 2 + wc * (TC / 4) + 32 * (pair - FC / 4))
                               : wc * (TC / 2) + 32 * pair;
          fp[c] = P::template fragment<true>(lp, base, c & 1, kk);
        }
#pragma unroll
        for (int r = 0; r < FR; ++r) fq[r] = Q::template fragment<false>(lq, wr * (TR / 2), r, kk);
#pragma unroll
        for (int c = 0; c < FC; ++c)
#pragma unroll
          for (int r = 0; r < FR; ++r) acc[c][r] = mfma16<BF>(fp[c], fq[r], acc[c][r]);
      }
    }
  }
  __syncthreads();                       // every wave has read its last fragments
  tile_epilogue<DT, EPI, FR, FC, false, WHERE>(a.e, acc, lds + wave * epilogue_bytes<FR, FC>(), i0 + wr * (TR / 2),
                                 (int)j0 + wc * (C / 2), a.splits > 1 ? slice : -1, (long)tr * 2 + wr);
}

}  // namespace
}  // namespace oidn
