// Forward products of at most 32 rows by packed weights, in one launch.
//
// The weights are all there is to read, each once.  A workgroup of 8 waves owns 16
// columns (32 where an 8-bit block of z has to be whole) and all of the summed length,
// which its waves share in turns of one block of 128; every wave loads weight codes
// straight into registers, kDepth blocks at once, and multiplies them by the rows' with
// v_mfma_scale_f32_16x16x128_f8f6f4 (rows past the last read the last).  Rows that come
// in 16 bits are coded on the way, by every workgroup for itself: a lane holds 32 of
// a row's 128 values, four lanes a block.  That costs about 150 vector instructions a
// block, less than the launch that would code them once.  The waves' sums meet in LDS
// and are added in wave order.
#include "dense_few.h"
#include "fp8_code.h"
#include "fp8_gemm.h"
#include "lanes.h"

namespace oidn {
namespace {

constexpr int kDepth8 = 4;

// 32 values of a row as codes, and their block's scale byte.  The four lanes that hold
// a block (16 apart) call it together.
template <int DT>
__device__ __forceinline__ intx8 code32(const Raw<DT> (&x)[4], unsigned& scale) {
  Eight v[4];
  unsigned top = 0;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    v[q] = x[q].value();
#pragma unroll
    for (int e = 0; e < 8; ++e) top = max(top, finite_bits(v[q].v[e]));
  }
  top = lanes_max<64, 16>(top);
  const int p = fp8_power(top);
  scale = (unsigned)(p + 127);
  intx8 r;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const uint2 c = fp8_codes(v[q].v, power_of_two(-p));
    r[2 * q] = (int)c.x;
    r[2 * q + 1] = (int)c.y;
  }
  return r;
}

// One block's product.  The compiler knows neither what the instruction reads nor when
// its result is there: the waits are for operands that vector instructions have just
// written, and for the next product, which adds to the same registers (12 wait states
// cover an 8-pass instruction).
__device__ __forceinline__ void mfma8_now(floatx4& c, const intx8& a, const intx8& b, unsigned sa, unsigned sb) {
  asm("s_nop 1\n\tv_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel:[0,0,0] op_sel_hi:[0,0,0]\n\ts_nop 11"
      : "+a"(c) : "v"(a), "v"(b), "v"(sa), "v"(sb));
}

// x of dtype (PACKED false: a.g.q elements at pitch a.g.ldq) or packed.  MF: fragments
// of 16 rows; NF: of 16 columns.
template <int DT, bool PACKED, int MF, int NF>
__global__ __launch_bounds__(64 * kFewWaves) void dense_few8(Gemm8Args a, int k) {
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
  const int j0 = blockIdx.x * 16 * NF;
  const long pitch = 2 * a.g.ldp, blocks = pitch / kFp8Block;      // bytes of a row of codes
  const EpilogueArgs& e = a.g.e;

  const unsigned char *wp[NF], *ws[NF], *xp[MF], *xs[MF];
#pragma unroll
  for (int f = 0; f < NF; ++f) {
    long j = j0 + 16 * f + r;
    j = j < e.cols ? j : e.cols - 1;
    wp[f] = static_cast<const unsigned char*>(a.g.p) + j * pitch + 32 * g;
    ws[f] = a.ps + j * a.pn;
  }
  long row[MF];
#pragma unroll
  for (int f = 0; f < MF; ++f) {
    row[f] = 16 * f + r < e.rows ? 16 * f + r : e.rows - 1;
    if constexpr (PACKED) {
      xp[f] = static_cast<const unsigned char*>(a.g.q) + row[f] * pitch + 32 * g;
      xs[f] = a.qs + row[f] * a.qn;
    }
  }
  floatx4 acc[NF][MF];
#pragma unroll
  for (int f = 0; f < NF; ++f)
#pragma unroll
    for (int m = 0; m < MF; ++m) acc[f][m] = floatx4{0.f, 0.f, 0.f, 0.f};

  auto block = [&](long b, auto depth) {       // blocks b, b + kFewWaves, ... of this wave
    constexpr int kN = decltype(depth)::value;
    intx8 w[kN][NF], xc[kN][MF];
    unsigned sw[kN][NF], sx[kN][MF];
    Raw<DT> raw[kN][MF][4];
#pragma unroll
    for (int d = 0; d < kN; ++d) {
      const long at = b + d * kFewWaves;
#pragma unroll
      for (int f = 0; f < NF; ++f) {
        __builtin_memcpy(&w[d][f], wp[f] + at * kFp8Block, 32);
        sw[d][f] = ws[f][at];
      }
#pragma unroll
      for (int m = 0; m < MF; ++m) {
        if constexpr (PACKED) {
          __builtin_memcpy(&xc[d][m], xp[m] + at * kFp8Block, 32);
          sx[d][m] = xs[m][at];
        } else {
          const long j = at * kFp8Block + 32 * g;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const long n = k - (j + 8 * q), left = (e.rows - 1 - row[m]) * a.g.ldq + n;
            raw[d][m][q] = load_raw<DT>(a.g.q, row[m] * a.g.ldq + j + 8 * q, n < 8 ? (int)(n < 0 ? 0 : n) : 8, left);
            if (n < 8) {
#pragma unroll
              for (int t = 0; t < 8; ++t)
                if (t >= n) raw[d][m][q].e[t] = (typename Raw<DT>::T)0.f;
            }
          }
        }
      }
    }
#pragma unroll
    for (int d = 0; d < kN; ++d) {
      if constexpr (!PACKED) {
#pragma unroll
        for (int m = 0; m < MF; ++m) xc[d][m] = code32<DT>(raw[d][m], sx[d][m]);
      }
#pragma unroll
      for (int f = 0; f < NF; ++f)
#pragma unroll
        for (int m = 0; m < MF; ++m) mfma8_now(acc[f][m], w[d][f], xc[d][m], sw[d][f], sx[d][m]);
    }
  };
  constexpr int kAtOnce = MF == 1 ? kDepth8 : 2;
  long b = wave;
  for (; b + (kAtOnce - 1) * kFewWaves < blocks; b += kAtOnce * kFewWaves)
    block(b, std::integral_constant<int, kAtOnce>{});
  for (; b < blocks; b += kFewWaves) block(b, std::integral_constant<int, 1>{});
#pragma unroll
  for (int f = 0; f < NF; ++f)
#pragma unroll
    for (int m = 0; m < MF; ++m) asm volatile("s_nop 15" : "+a"(acc[f][m]));

  // [wave][row][column]; a row's pitch is padded by 16 bytes
  constexpr int kCols = 16 * NF, kPitch = kCols + 4;
  __shared__ __attribute__((aligned(16))) float part[kFewWaves][16 * MF][kPitch];
#pragma unroll
  for (int f = 0; f < NF; ++f)
#pragma unroll
    for (int m = 0; m < MF; ++m) *reinterpret_cast<floatx4*>(&part[wave][16 * m + r][16 * f + 4 * g]) = acc[f][m];
  __syncthreads();
  // eight columns of a row per lane; lanes of a row are neighbours
  constexpr int kLanes = 2 * NF;
  const int t = threadIdx.x, i = t / kLanes, j8 = 8 * (t % kLanes);
  if (t >= 16 * MF * kLanes) return;         // whole groups of kLanes
  Eight v{};
#pragma unroll
  for (int w = 0; w < kFewWaves; ++w)
#pragma unroll
    for (int c = 0; c < 8; ++c) v.v[c] += part[w][i][j8 + c];
  const int j = j0 + j8;
  Fetched bias{}, none;
  RawFetched<DT, false> f;
  bias.a = bias8(e.bias, j, e.cols - j);
  if (j0 + kCols <= e.cols) {
    fetch<DT, kEpiLinear, true, false>(e, i, j, f);
    finish<DT, kEpiLinear, true, false>(e, 0, i, j, v, v, bias, f, none);
  } else {
    fetch<DT, kEpiLinear, false, false>(e, i, j, f);
    finish<DT, kEpiLinear, false, false>(e, 0, i, j, v, v, bias, f, none);
  }
}

template <int DT, bool PACKED, int NF>
void launch_rows(const Gemm8Args& a, int k, hipStream_t stream) {
  const dim3 grid((unsigned)((a.g.e.cols + 16 * NF - 1) / (16 * NF))), block(64 * kFewWaves);
  if (a.g.e.rows <= 16) hipLaunchKernelGGL((dense_few8<DT, PACKED, 1, NF>), grid, block, 0, stream, a, k);
  else hipLaunchKernelGGL((dense_few8<DT, PACKED, 2, NF>), grid, block, 0, stream, a, k);
}
template <int DT>
void launch_type(const Gemm8Args& a, int k, bool packed, hipStream_t stream) {
  const bool block32 = a.g.e.z && a.g.e.z8;
  if (packed) {
    if (block32) launch_rows<DT, true, 2>(a, k, stream);
    else launch_rows<DT, true, 1>(a, k, stream);
  } else {
    if (block32) launch_rows<DT, false, 2>(a, k, stream);
    else launch_rows<DT, false, 1>(a, k, stream);
  }
}

}  // namespace

hipError_t launch_few8(const Gemm8Args& a, int k, bool packed, bool bf16, hipStream_t stream) {
  if (a.g.e.rows > kFewRows) return hipErrorInvalidValue;
  if (bf16) launch_type<OIDN_BF16>(a, k, packed, stream);
  else launch_type<OIDN_F16>(a, k, packed, stream);
  return hipGetLastError();
}

}  // namespace oidn
