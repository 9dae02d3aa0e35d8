// Products of packed matrices on the matrix cores, C[i][j] = sum_l Q(i, l) P(j, l).
//
// v_mfma_scale_f32_16x16x128_f8f6f4 multiplies 128 codes of 16 rows by 16 and
// takes the exponent of each row's block of 128 as an operand, so blocks need no
// work of their own.  A row of 128 codes has the bytes of 64 16-bit elements: tiles,
// their copies to LDS, slots and epilogues are those of the 16-bit products
// (dense_gemm16_direct.h), and a fragment is both 16-byte halves of a row that a lane
// reads (the order of the sum is permuted alike in both operands).
//
// The instruction adds eight products with the last bit at 2^-13 of the largest
// one's power of two, what is beyond cut off, and sums of eight in fp32: 1.5e-5 of the
// result at normal data, 3.6e-5 where channels differ e-fold (measured over 4096 summed
// elements), a tenth and less of a 16-bit result's rounding.  The 8-bit
// instructions without scales do the same.
#pragma once

#include "dense_gemm16_direct.h"
#include "fp8.h"

namespace oidn {
namespace {

typedef int intx8 __attribute__((ext_vector_type(8)));

// c += a b in place, scales in byte BYTE of sa and sb.  As an instruction of its own:
// the builtin's result may be given the registers of an operand (seen with the
// scale's, and wrong sums with it).  The waits are dense_gemm16_direct.h's settle().
template <int BYTE>
__device__ __forceinline__ void mfma8_acc(floatx4& c, const intx8& a, const intx8& b, unsigned sa, unsigned sb) {
  if constexpr (BYTE == 0)
    asm("v_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel:[0,0,0] op_sel_hi:[0,0,0]"
        : "+a"(c) : "v"(a), "v"(b), "v"(sa), "v"(sb));
  else if constexpr (BYTE == 1)
    asm("v_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel:[1,1,0] op_sel_hi:[0,0,0]"
        : "+a"(c) : "v"(a), "v"(b), "v"(sa), "v"(sb));
  else if constexpr (BYTE == 2)
    asm("v_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel:[0,0,0] op_sel_hi:[1,1,0]"
        : "+a"(c) : "v"(a), "v"(b), "v"(sa), "v"(sb));
  else
    asm("v_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel:[1,1,0] op_sel_hi:[1,1,0]"
        : "+a"(c) : "v"(a), "v"(b), "v"(sa), "v"(sb));
}

// Workgroup `block` of the product; lds: gemm16_lds<T, T>() bytes, two buffers of a P
// and a Q tile.  Slices begin at multiples of four staged tiles, whose scales are a
// word.
template <bool BF, int EPI, int T, Caching WHERE>
__device__ __forceinline__ void gemm8(const Gemm8Args& a8, int block, char* lds) {
  const GemmArgs& a = a8.g;
  constexpr int DT = BF ? OIDN_BF16 : OIDN_F16;
  constexpr int F = T / 32;                      // 16-wide fragments per wave, each way
  typedef Direct16<T, false> D;
  typedef typename D::S S;
  constexpr unsigned kBuf = 2 * S::kBytes;

  int tc, tr, slice;
  if (!tile_and_slice(a, block, tc, tr, slice)) return;
  const long i0 = (long)tr * T, j0 = (long)tc * T;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, wr = wave >> 1, wc = wave & 1, r = lane & 15;
  const long t0 = (long)slice * a.per_split, nt = a.len / kDenseK;
  const long t1 = t0 + a.per_split < nt ? t0 + a.per_split : nt;

  const unsigned lds_at = (unsigned)(unsigned long)(__attribute__((address_space(3))) void*)lds;
  D p, q;
  p.init(a.p, a.ldp, j0, a.e.cols, t0 * kDenseK, 0, lds_at);
  q.init(a.q, a.ldq, i0, a.e.rows, t0 * kDenseK, 0, lds_at + S::kBytes);

  // this lane's rows' scales, four staged tiles a word
  const unsigned char *sp[F], *sq[F];
#pragma unroll
  for (int f = 0; f < F; ++f) {
    const long j = j0 + wc * (T / 2) + 32 * (f / 2) + 8 * (r >> 2) + 4 * (f & 1) + (r & 3), last = a.e.cols - 1l;
    sp[f] = a8.ps + (j < last ? j : last) * a8.pn;
    const long i = i0 + wr * (T / 2) + 16 * f + r;
    sq[f] = a8.qs + (i < a.e.rows - 1 ? i : a.e.rows - 1) * a8.qn;
  }
  unsigned up[F], uq[F];

  floatx4 acc[F][F];
#pragma unroll
  for (int c = 0; c < F; ++c)
#pragma unroll
    for (int k = 0; k < F; ++k) acc[c][k] = floatx4{0.f, 0.f, 0.f, 0.f};

  auto stage = [&](unsigned buf) {
#pragma unroll
    for (int n = 0; n < D::kCopies; ++n) {
      p.copy(n, buf);
      q.copy(n, buf);
    }
    p.advance();
    q.advance();
  };
  auto both = [](uint4 lo, uint4 hi) {
    return intx8{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
  };
  auto wait_all = [&] {
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
  };
  auto multiply = [&](auto byte, unsigned buf) {
    constexpr int kByte = decltype(byte)::value;
    const char* const l = lds + buf;
    intx8 fq[F];
#pragma unroll
    for (int k = 0; k < F; ++k)
      fq[k] = both(S::template fragment<false>(l + S::kBytes, wr * (T / 2), k, 0),
                   S::template fragment<false>(l + S::kBytes, wr * (T / 2), k, 1));
#pragma unroll
    for (int c = 0; c < F; ++c) {
      const int base = wc * (T / 2) + 32 * (c / 2);
      const intx8 fp = both(S::template fragment<true>(l, base, c & 1, 0), S::template fragment<true>(l, base, c & 1, 1));
#pragma unroll
      for (int k = 0; k < F; ++k) mfma8_acc<kByte>(acc[c][k], fp, fq[k], up[c], uq[k]);
    }
  };

  stage(0);
  unsigned cur = 0;
  for (long t = t0; t < t1; ++t) {
    wait_all();                                  // tile t is there, and every wave has read tile t - 1
    if (((t - t0) & 3) == 0) {
#pragma unroll
      for (int f = 0; f < F; ++f) {
        up[f] = *reinterpret_cast<const unsigned*>(sp[f] + t);
        uq[f] = *reinterpret_cast<const unsigned*>(sq[f] + t);
      }
    }
    if (t + 1 < t1) stage(kBuf - cur);
    switch ((int)(t - t0) & 3) {
      case 0: multiply(std::integral_constant<int, 0>{}, cur); break;
      case 1: multiply(std::integral_constant<int, 1>{}, cur); break;
      case 2: multiply(std::integral_constant<int, 2>{}, cur); break;
      default: multiply(std::integral_constant<int, 3>{}, cur);
    }
    cur = kBuf - cur;
  }
#pragma unroll
  for (int c = 0; c < F; c += 2)
#pragma unroll
    for (int k = 0; k < F; k += 2) settle(acc[c][k], acc[c][k + 1], acc[c + 1][k], acc[c + 1][k + 1]);
  __syncthreads();
  tile_epilogue<DT, EPI, F, F, false, WHERE>(a.e, acc, lds + wave * epilogue_bytes<F, F>(), i0 + wr * (T / 2),
                                             (int)j0 + wc * (T / 2), a.splits > 1 ? slice : -1, (long)tr * 2 + wr);
}

template <bool BF, int T, Caching WHERE>
__global__ __launch_bounds__(256, workgroups_per_cu(T, T)) void dense_gemm8(Gemm8Args a) {
  __shared__ __attribute__((aligned(1024))) char lds[gemm16_lds<T, T>()];
  gemm8<BF, kEpiLinear, T, WHERE>(a, blockIdx.x, lds);
}
template <bool BF, int T>
__global__ __launch_bounds__(256, workgroups_per_cu(T, T)) void dense_gemm8_group(Gemm8Group g) {
  __shared__ __attribute__((aligned(1024))) char lds[gemm16_lds<T, T>()];
  const int k = g.count > 1 && (int)blockIdx.x >= g.start[1] ? 1 : 0;
  gemm8<BF, kEpiStore, T, kEither>(g.a[k], blockIdx.x - g.start[k], lds);
}

}  // namespace
}  // namespace oidn
