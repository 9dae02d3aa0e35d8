// Forward products of at most 32 rows by packed weights, in one launch.
//
// The weights are all there is to read, each once.  A workgroup of 8 waves owns 16
// columns (32 where an 8-bit block of z has to be whole) and all of the summed length,
// in segments of 32 blocks of 128: a wave loads the weight codes of four neighbouring
// blocks and their word of scales straight into registers and multiplies them by the
// rows' with v_mfma_scale_f32_16x16x128_f8f6f4 (rows past the last read the last).  Rows
// that come in 16 bits, kCodedRows at most, are coded on the way, by every workgroup for
// itself, while the weights' loads are in flight: a thread codes eight values of each row's segment, which
// the waves read from LDS.  The waves' sums meet in LDS and are added in wave order.
//
// Bound by the weights' bytes and a launch's latency: bf16 4096 -> 4096 (17 MB, 3.3 us at a
// copy's rate) 7.0 us for one row, 8.4 to 8.8 for 2 to 4, 11.0 for 8 and 14.2 for 32 with
// their packing; 8192 -> 8192 (67 MB) 17 us, 3.9 TB/s.  16-bit weights take 7.0, 8.2 (4 rows),
// 9.3 (8), 13.9 (32) and 24.8: 4096 -> 4096 gains only where x is packed already (8 rows 8.2, 32
// 10.0 to 11.0), smaller layers nothing (1024 -> 1024, one row 5.6 for 3.1).
#include "dense_few.h"
#include "fp8_code.h"
#include "fp8_gemm.h"
#include "lanes.h"

namespace oidn {
namespace {

constexpr int kSegment = 4 * kFewWaves;      // blocks

// x of dtype (PACKED false: k columns at pitch a.g.ldq) or packed.  ROWS: rows at most;
// NF: fragments of 16 columns.
template <int DT, bool PACKED, int ROWS, int NF>
__global__ __launch_bounds__(64 * kFewWaves) void dense_few8(Gemm8Args a, int k) {
  constexpr int MF = ROWS > 16 ? 2 : 1;        // fragments of 16 rows
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
  const int j0 = blockIdx.x * 16 * NF;
  const long pitch = 2 * a.g.ldp, blocks = pitch / kFp8Block;      // bytes of a row of codes
  const EpilogueArgs& e = a.g.e;
  // a segment's codes, rows 32 bytes apart in the banks, and its scales
  constexpr int kRowBytes = kSegment * kFp8Block + 32;
  constexpr int kCols = 16 * NF, kPitch = kCols + 4;         // a row of sums is padded by 16 bytes
  constexpr int kCodes = PACKED ? 0 : ROWS * (kRowBytes + kSegment), kSums = kFewWaves * 16 * MF * kPitch * 4;
  __shared__ __attribute__((aligned(16))) unsigned char lds[kCodes > kSums ? kCodes : kSums];
  unsigned char* const codes = lds;
  unsigned char* const scales = lds + ROWS * kRowBytes;
  typedef float Sums[16 * MF][kPitch];
  Sums* const part = reinterpret_cast<Sums*>(lds);           // [wave][row][column], after the codes

  const unsigned char *wp[NF], *ws[NF];
#pragma unroll
  for (int f = 0; f < NF; ++f) {
    long j = j0 + 16 * f + r;
    j = j < e.cols ? j : e.cols - 1;
    wp[f] = static_cast<const unsigned char*>(a.g.p) + j * pitch + 32 * g;
    ws[f] = a.ps + j * a.pn;
  }
  int row[MF];
#pragma unroll
  for (int f = 0; f < MF; ++f) row[f] = 16 * f + r < e.rows ? 16 * f + r : (int)e.rows - 1;
  floatx4 acc[NF][MF];
#pragma unroll
  for (int f = 0; f < NF; ++f)
#pragma unroll
    for (int m = 0; m < MF; ++m) acc[f][m] = floatx4{0.f, 0.f, 0.f, 0.f};

  for (long from = 0; from < blocks; from += kSegment) {
    // blocks past the last are loaded from the last and not multiplied
    const long b0 = from + 4 * wave;
    const int exist = __builtin_amdgcn_readfirstlane((int)(blocks - b0 < 4 ? blocks - b0 : 4));
    intx8 w[4][NF];
    unsigned sw[NF];
#pragma unroll
    for (int f = 0; f < NF; ++f) {
#pragma unroll
      for (int d = 0; d < 4; ++d)
        __builtin_memcpy(&w[d][f], wp[f] + (b0 + d < blocks ? b0 + d : blocks - 1) * kFp8Block, 32);
      sw[f] = *reinterpret_cast<const unsigned*>(ws[f] + (b0 < blocks ? b0 : 0));
    }
    intx8 x[4][MF];
    unsigned sx[MF];
    if constexpr (PACKED) {
      const unsigned char* const q = static_cast<const unsigned char*>(a.g.q);
#pragma unroll
      for (int m = 0; m < MF; ++m) {
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          __builtin_memcpy(&x[d][m], q + row[m] * pitch + (b0 + d < blocks ? b0 + d : blocks - 1) * kFp8Block + 32 * g, 32);
        }
        sx[m] = *reinterpret_cast<const unsigned*>(a.qs + row[m] * a.qn + (b0 < blocks ? b0 : 0));
      }
    } else {
      // thread t: values 8 t .. + 7 of the segment, of every row; 16 lanes hold a block
      typedef typename Raw<DT>::T T;
      const long j = from * kFp8Block + 8 * threadIdx.x, left = k - j;
      constexpr int kAtOnce = ROWS < 4 ? ROWS : 4;
      for (int i = 0; i < e.rows; i += kAtOnce) {
        Raw<DT> raw[kAtOnce];
#pragma unroll
        for (int n = 0; n < kAtOnce; ++n) {
          const T* const p = static_cast<const T*>(a.g.q) + (i + n < e.rows ? i + n : e.rows - 1) * a.g.ldq;
          if (left >= 8) {
            __builtin_memcpy(&raw[n].e, p + j, 16);
          } else {
#pragma unroll
            for (int c = 0; c < 8; ++c) raw[n].e[c] = c < left ? p[j + c] : (T)0.f;
          }
        }
#pragma unroll
        for (int n = 0; n < kAtOnce; ++n) {
          const Eight v = raw[n].value();
          const int power = fp8_power(lanes_max<16>(finite_top(v)));
          if (i + n < e.rows) {
            *reinterpret_cast<uint2*>(codes + (i + n) * kRowBytes + 8 * threadIdx.x) = fp8_codes(v.v, power_of_two(-power));
            if (threadIdx.x % 16 == 0) scales[(i + n) * kSegment + threadIdx.x / 16] = (unsigned char)(power + 127);
          }
        }
      }
      __syncthreads();
#pragma unroll
      for (int m = 0; m < MF; ++m) {
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          const uint4* const p = reinterpret_cast<const uint4*>(codes + row[m] * kRowBytes + (4 * wave + d) * kFp8Block + 32 * g);
          const uint4 lo = p[0], hi = p[1];
          x[d][m] = intx8{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
        }
        sx[m] = *reinterpret_cast<const unsigned*>(scales + row[m] * kSegment + 4 * wave);
      }
    }
    auto multiply = [&](auto byte) {
      constexpr int kByte = decltype(byte)::value;
      if (kByte < exist) {
#pragma unroll
        for (int f = 0; f < NF; ++f)
#pragma unroll
          for (int m = 0; m < MF; ++m) mfma8_acc<kByte, true>(acc[f][m], w[kByte][f], x[kByte][m], sw[f], sx[m]);
      }
    };
    multiply(std::integral_constant<int, 0>{});
    multiply(std::integral_constant<int, 1>{});
    multiply(std::integral_constant<int, 2>{});
    multiply(std::integral_constant<int, 3>{});
    if (!PACKED) __syncthreads();      // the codes have been read
  }
#pragma unroll
  for (int f = 0; f < NF; ++f)
#pragma unroll
    for (int m = 0; m < MF; ++m) asm volatile("s_nop 15" : "+a"(acc[f][m]));

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
  const long m = a.g.e.rows;
  if constexpr (PACKED) {
    if (m <= 16) hipLaunchKernelGGL((dense_few8<DT, true, 16, NF>), grid, block, 0, stream, a, k);
    else hipLaunchKernelGGL((dense_few8<DT, true, kFewRows, NF>), grid, block, 0, stream, a, k);
  } else {
    if (m == 1) hipLaunchKernelGGL((dense_few8<DT, false, 1, NF>), grid, block, 0, stream, a, k);
    else hipLaunchKernelGGL((dense_few8<DT, false, kCodedRows, NF>), grid, block, 0, stream, a, k);
  }
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
  if (a.g.e.rows > (packed ? kFewRows : kCodedRows)) return hipErrorInvalidValue;
  if (bf16) launch_type<OIDN_BF16>(a, k, packed, stream);
  else launch_type<OIDN_F16>(a, k, packed, stream);
  return hipGetLastError();
}

}  // namespace oidn
