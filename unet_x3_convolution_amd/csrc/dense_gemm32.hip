// fp32 matrix products on the matrix cores (v_mfma_f32_16x16x4), the same
// products, tiles of C and epilogues as the 16-bit form (dense_gemm16.h).
//
// Tiles of C are 64 x 64 (gated: 64 x 128), several to a compute unit: 4096 x
// 4096 x 1024 runs at 120 TFLOP/s, 128 x 128 tiles at 105, one or two to a unit
// with their registers full.  Plain forward products of few tiles take 32 x 64,
// whose second workgroup on a unit works while the first one waits (us a call,
// gelu and residual, 64 x 64 against 32 x 64): 2040 x 112 -> 96 7.8 and 6.0, 510
// x 128 -> 512 7.3 and 5.7, 1021 x 515 -> 771 18.8 and 18.3; with many tiles the
// larger ones' fewer loads win: 4096 x 1024 -> 4096 298 and 325.
//
// 32 summed elements are staged at a time through registers into one of two
// LDS buffers, two or three tiles ahead, as rows of 32 + 4 floats: the pad puts
// the 16 rows of a fragment's 16-byte reads on distinct banks.  A lane's 16 bytes are elements
// 4 g .. 4 g + 3 (g = lane / 16) of 16; MFMA e takes element e of every lane,
// in both operands, so the order of the sum is permuted within 16 elements
// and nothing is shuffled.  Strided operands keep rows of T + 4 floats, one per
// summed element, and are read float by float: the pad puts the rows of the
// four lane groups on distinct banks.
#include "dense_gemm16.h"
#include "dense_slope.h"

namespace oidn {
namespace {

constexpr int kPad32 = kDenseKF32 + 4;

template <int T, bool STRIDED>
struct Stage32 {
  typedef Loader<4, T, kDenseKF32, STRIDED> From;
  static constexpr int kUnits = From::kUnits;
  static constexpr int kPitch = STRIDED ? T + 4 : kPad32;
  static constexpr int kFloats = (STRIDED ? kDenseKF32 : T) * kPitch;

  static __device__ __forceinline__ void store(const uint4 (&u)[kUnits], float* lds) {
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
      int r, s;
      From::place(k, r, s);
      *reinterpret_cast<uint4*>(lds + r * kPitch + 4 * s) = u[k];
    }
  }
  template <bool PAIR>
  static __device__ __forceinline__ floatx4 fragment(const float* lds, int base, int q, int kk) {
    const int lane = threadIdx.x & 63, g = lane >> 4, r = lane & 15;
    const int row = base + (PAIR ? 8 * (r >> 2) + 4 * q + (r & 3) : 16 * q + r);
    if constexpr (!STRIDED) {
      return *reinterpret_cast<const floatx4*>(lds + row * kPitch + 16 * kk + 4 * g);
    } else {
      floatx4 v;
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = lds[(16 * kk + 4 * g + e) * kPitch + row];
      return v;
    }
  }
};

template <int TR, int TC>
constexpr int gemm32_lds() { return 2 * (TR + TC) * kPad32 * 4; }    // strided tiles take less

template <int LAYOUT, int EPI, int TR, int TC>
__device__ __forceinline__ void gemm32(const GemmArgs& a, int block, float* lds) {
  constexpr int DT = OIDN_F32;
  constexpr bool PS = LAYOUT != kForward, QS = LAYOUT == kWeightGrad;
  constexpr int FR = TR / 32, FC = TC / 32;
  static_assert(EPI != kEpiGated || FC % 4 == 0, "a wave holds pairs of both projections");
  typedef Stage32<TC, PS> P;
  typedef Stage32<TR, QS> Q;

  int tc, tr;
  int slice;
  if (!tile_and_slice(a, block, tc, tr, slice)) return;
  const long i0 = (long)tr * TR;
  constexpr int C = EPI == kEpiGated ? TC / 2 : TC;
  const long j0 = (long)tc * C;
  const long half = EPI == kEpiGated ? a.e.cols : 0;
  const int wave = threadIdx.x >> 6, wr = wave >> 1, wc = wave & 1;
  const long t0 = (long)slice * a.per_split;
  const long nt = (a.len + kDenseKF32 - 1) / kDenseKF32;
  const long t1 = t0 + a.per_split < nt ? t0 + a.per_split : nt;

  floatx4 acc[FC][FR];
#pragma unroll
  for (int c = 0; c < FC; ++c)
#pragma unroll
    for (int r = 0; r < FR; ++r) acc[c][r] = floatx4{0.f, 0.f, 0.f, 0.f};

  // Tile t is multiplied out of LDS buffer (t - t0) % 2 while tile t + 1 goes
  // into the other one from register set (t + 1 - t0) % 2 and the loads of tile
  // t + 3 leave for that set: the LDS writes and the second half's reads are
  // issued between the MFMAs, which take 32 cycles each.
  typename P::From from_p(a.p, a.ldp, j0, a.e.cols, t0 * kDenseKF32, a.len, half);
  typename Q::From from_q(a.q, a.ldq, i0, a.e.rows, t0 * kDenseKF32, a.len, 0);
  uint4 up[2][P::kUnits], uq[2][Q::kUnits];
  auto load = [&](long t, int set) {
    if (t >= t1) return;
    from_p.load(up[set], t * kDenseKF32);
    from_q.load(uq[set], t * kDenseKF32);
  };
  auto store = [&](long t, int set) {
    if (t >= t1) return;
    float* const l = lds + set * (P::kFloats + Q::kFloats);
    P::store(up[set], l);
    Q::store(uq[set], l + P::kFloats);
  };
  floatx4 fp[2][FC], fq[2][FR];          // [half of the tile][fragment]
  auto read = [&](int set, int kk) {
    const float* const lp = lds + set * (P::kFloats + Q::kFloats);
#pragma unroll
    for (int c = 0; c < FC; ++c) {
      const int pair = c / 2;
      const int base = EPI == kEpiGated
                           ? (pair < FC / 4 ? wc * (TC / 4) + 32 * pair
                                            : TC / 2 + wc * (TC / 4) + 32 * (pair - FC / 4))
                           : wc * (TC / 2) + 32 * pair;
      fp[kk][c] = P::template fragment<true>(lp, base, c & 1, kk);
    }
#pragma unroll
    for (int r = 0; r < FR; ++r)
      fq[kk][r] = Q::template fragment<false>(lp + P::kFloats, wr * (TR / 2), r, kk);
  };
  auto multiply = [&](int kk, int e0, int e1) {
#pragma unroll
    for (int e = e0; e < e1; ++e)
#pragma unroll
      for (int c = 0; c < FC; ++c)
#pragma unroll
        for (int r = 0; r < FR; ++r)
          acc[c][r] = __builtin_amdgcn_mfma_f32_16x16x4f32(fp[kk][c][e], fq[kk][r][e], acc[c][r], 0, 0, 0);
  };
  load(t0, 0);
  load(t0 + 1, 1);
  store(t0, 0);
  load(t0 + 2, 0);
  for (long tt = t0; tt < t1; tt += 2) {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const long t = tt + s;
      if (t >= t1) break;
      __syncthreads();                   // tile t is written, tile t - 1 has been read
      read(s, 0);
      read(s, 1);
      multiply(0, 0, 2);
      __builtin_amdgcn_sched_barrier(0);
      store(t + 1, 1 - s);
      __builtin_amdgcn_sched_barrier(0);
      multiply(0, 2, 4);
      __builtin_amdgcn_sched_barrier(0);
      load(t + 3, 1 - s);
      __builtin_amdgcn_sched_barrier(0);
      multiply(1, 0, 4);
    }
  }
  __syncthreads();                       // every wave has read its last fragments
  tile_epilogue<DT, EPI, FR, FC>(a.e, acc, reinterpret_cast<char*>(lds) + wave * epilogue_bytes<FR, FC>(),
                                 i0 + wr * (TR / 2), (int)j0 + wc * (C / 2), a.splits > 1 ? slice : -1,
                                 (long)tr * 2 + wr);
}

template <int LAYOUT, int EPI, int TR, int TC>
__global__ __launch_bounds__(256, 2) void dense_gemm32(GemmArgs a, UnpackJob u) {
  __shared__ __attribute__((aligned(16))) float lds[gemm32_lds<TR, TC>() / 4];
  if constexpr (EPI == kEpiGatedBack) {
    if ((int)blockIdx.x < u.blocks) return unpack_rows<OIDN_F32>(u, blockIdx.x);
  }
  gemm32<LAYOUT, EPI, TR, TC>(a, blockIdx.x - (EPI == kEpiGatedBack ? u.blocks : 0), lds);
}

// Several gradients' products in one launch.
template <int T>
__global__ __launch_bounds__(256, 2) void dense_gemm32_group(GemmGroup g) {
  __shared__ __attribute__((aligned(16))) float lds[gemm32_lds<T, T>() / 4];
  if ((int)blockIdx.x >= g.sums_start) return slope_rows<OIDN_F32>(g.sums, blockIdx.x - g.sums_start, lds);
  int k = 0;
  while (k + 1 < g.count && (int)blockIdx.x >= g.start[k + 1]) ++k;
  const int block = blockIdx.x - g.start[k];
  if (g.layout[k] == kInputGrad) gemm32<kInputGrad, kEpiStore, T, T>(g.a[k], block, lds);
  else gemm32<kWeightGrad, kEpiStore, T, T>(g.a[k], block, lds);
}

template <int LAYOUT, int EPI>
hipError_t launch_epi(const GemmArgs& a, const GemmPlan& p, const UnpackJob& u, hipStream_t stream) {
  const dim3 grid((unsigned)(gemm_blocks(a) + u.blocks)), block(256);
  constexpr int SC = EPI == kEpiGated ? 128 : 64;
  if constexpr (EPI == kEpiLinear) {
    if (p.tile_r == 32 && p.tile_c == 64) {
      hipLaunchKernelGGL((dense_gemm32<LAYOUT, EPI, 32, 64>), grid, block, 0, stream, a, u);
      return hipGetLastError();
    }
  }
  if (p.tile_r != 64 || p.tile_c != SC) return hipErrorInvalidValue;
  hipLaunchKernelGGL((dense_gemm32<LAYOUT, EPI, 64, SC>), grid, block, 0, stream, a, u);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_gemm32(const GemmArgs& a, const GemmPlan& p, int epi, const UnpackJob& u, hipStream_t stream) {
  if (epi == kEpiLinear) return launch_epi<kForward, kEpiLinear>(a, p, u, stream);
  if (epi == kEpiGated) return launch_epi<kForward, kEpiGated>(a, p, u, stream);
  if (epi == kEpiGatedBack) return launch_epi<kInputGrad, kEpiGatedBack>(a, p, u, stream);
  return hipErrorInvalidValue;
}

hipError_t launch_gemm32_group(const GemmGroup& g, const GemmPlan& p, hipStream_t stream) {
  const dim3 grid((unsigned)g.blocks), block(256);
  if (p.tile_r != 64) return hipErrorInvalidValue;
  hipLaunchKernelGGL(dense_gemm32_group<64>, grid, block, 0, stream, g);
  return hipGetLastError();
}

}  // namespace oidn
