// Matrices to 8-bit floating point and back.
#include "fp8_code.h"

namespace oidn {
namespace {

constexpr int kPackThreads = 256;

// Columns j .. j + 7 of row i, zeros past the matrix.
template <int DT>
__device__ __forceinline__ Eight cell8(const void* p, long ld, long i, int j, long m, int n) {
  Eight r{};
  if (i < m) {
    r = load_raw<DT>(p, i * ld + j, n - j, (m - 1 - i) * ld + n - j).value();
    if (n - j < 8) clear_tail(n - j, r);
  }
  return r;
}
__device__ __forceinline__ unsigned top_over(unsigned t, int lanes) {
  const unsigned o = __shfl_xor(t, lanes);
  return o > t ? o : t;
}

// A workgroup takes 128 x 128 elements, a thread eight columns of eight rows that
// follow each other, so that it holds eight codes in a row of either form.  A row's
// block lies in 16 lanes; a column's in all waves.
struct PackLds {
  unsigned top[4][kFp8Block];
  float sum[4][kFp8Block];
  uint2 codes[kFp8Block][16];      // turned: [column][eight rows], unit u at u ^ (column / 8)
};
template <int DT>
__device__ __forceinline__ void pack_tile(const Fp8PackArgs& a, long block, PackLds& lds) {
  const long across = (a.n + kFp8Block - 1) / kFp8Block, tile_r = block / across;
  const int tile_c = (int)(block - tile_r * across);
  const int t = threadIdx.x, c = t & 15, g = t >> 4, wave = t >> 6;
  const long i0 = tile_r * kFp8Block + 8 * g;
  const int j = tile_c * kFp8Block + 8 * c;
  Eight v[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) v[k] = cell8<DT>(a.x, a.ldx, i0 + k, j, a.m, a.n);
  if (a.z) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      Eight z{}, value;
      if (a.z8) {
        if (i0 + k < a.m && j < a.n) z = ckpt_load8(ckpt_at(const_cast<void*>(a.z), a.m, a.n), i0 + k, j);
      } else {
        z = cell8<DT>(a.z, a.ldz, i0 + k, j, a.m, a.n);
      }
      // the slope's fp32 form: a dz next to a border of two codes should fall as the formula's does
      activate_slope8<OIDN_F32>(a.act, z, value);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[k].v[e] *= z.v[e];
    }
  }
  unsigned row_top[8], col_top[8] = {};
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    row_top[k] = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const unsigned b = finite_bits(v[k].v[e]);
      row_top[k] = b > row_top[k] ? b : row_top[k];
      col_top[e] = b > col_top[e] ? b : col_top[e];
    }
  }
  if (a.sums) {
    Eight s{};
#pragma unroll
    for (int k = 0; k < 8; ++k) add8(s, v[k]);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      s.v[e] += __shfl_xor(s.v[e], 16);
      s.v[e] += __shfl_xor(s.v[e], 32);
      if ((t & 63) < 16) lds.sum[wave][8 * c + e] = s.v[e];
    }
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    col_top[e] = top_over(top_over(col_top[e], 16), 32);
    if ((t & 63) < 16) lds.top[wave][8 * c + e] = col_top[e];
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) row_top[k] = top_over(top_over(top_over(top_over(row_top[k], 1), 2), 4), 8);
  __syncthreads();
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    col_top[e] = 0;
#pragma unroll
    for (int w = 0; w < 4; ++w) col_top[e] = max(col_top[e], lds.top[w][8 * c + e]);
  }
  if (a.square) {
    unsigned all = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) all = max(all, col_top[e]);
    all = top_over(top_over(top_over(top_over(all, 1), 2), 4), 8);
#pragma unroll
    for (int k = 0; k < 8; ++k) row_top[k] = col_top[k] = all;
  }
  if (a.sums && t < kFp8Block && tile_c * kFp8Block + t < a.n)
    a.sums[tile_r * a.n + tile_c * kFp8Block + t] = lds.sum[0][t] + lds.sum[1][t] + lds.sum[2][t] + lds.sum[3][t];
  if (a.rows) {
    const Fp8At at = fp8_at(a.rows, a.m, a.n);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const long i = i0 + k;
      if (i >= a.m) break;
      const int e = fp8_power(row_top[k]);
      *reinterpret_cast<uint2*>(at.codes + i * at.pitch + j) = fp8_codes(v[k].v, power_of_two(-e));
      if (c == 0) at.scales[i * at.words + tile_c] = (unsigned char)(e + 127);
    }
  }
  if (a.turned) {
    const Fp8At at = fp8_at(a.turned, a.n, a.m);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int p = fp8_power(col_top[e]);
      float col[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) col[k] = v[k].v[e];
      lds.codes[8 * c + e][g ^ c] = fp8_codes(col, power_of_two(-p));
      if (g == 0 && j + e < a.n) at.scales[(j + e) * at.words + tile_r] = (unsigned char)(p + 127);
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int u = t + k * kPackThreads, column = u >> 3, q = u & 7, x = column >> 3;
      const int col = tile_c * kFp8Block + column;
      if (col >= a.n) break;
      const uint2 first = lds.codes[column][(2 * q) ^ x], second = lds.codes[column][(2 * q + 1) ^ x];
      *reinterpret_cast<uint4*>(at.codes + col * at.pitch + tile_r * kFp8Block + 16 * q) =
          make_uint4(first.x, first.y, second.x, second.y);
    }
  }
}

template <int DT>
__global__ __launch_bounds__(kPackThreads) void fp8_pack(Fp8PackArgs a, Fp8PackArgs b, int first) {
  __shared__ __attribute__((aligned(16))) PackLds lds;
  if ((int)blockIdx.x < first) pack_tile<DT>(a, blockIdx.x, lds);
  else pack_tile<DT>(b, (int)blockIdx.x - first, lds);
}

// A thread takes eight columns.  A finite value whose rounding passes the type's
// range becomes the largest one.
template <int DT>
__global__ __launch_bounds__(kPackThreads) void fp8_unpack(void* packed, long m, int n, void* y, long ldy, long units) {
  const Fp8At at = fp8_at(packed, m, n);
  const long total = m * units, step = (long)gridDim.x * kPackThreads;
  for (long t = (long)blockIdx.x * kPackThreads + threadIdx.x; t < total; t += step) {
    const long i = t / units;
    const int j = (int)(t - i * units) * 8;
    const int e = (int)at.scales[i * at.words + j / kFp8Block] - 127;
    Eight v = fp8_values(*reinterpret_cast<const uint2*>(at.codes + i * at.pitch + j), power_of_two(e));
    const float most = DT == OIDN_F16 ? 65504.f : DT == OIDN_BF16 ? 0x1.fep127f : 0x1.fffffep127f;
#pragma unroll
    for (int k = 0; k < 8; ++k)
      v.v[k] = v.v[k] == v.v[k] ? __builtin_amdgcn_fmed3f(v.v[k], -most, most) : v.v[k];
    store8<DT>(y, i * ldy + j, v, n - j);
  }
}

template <int DT>
void launch(const Fp8PackArgs& a, const Fp8PackArgs& b, hipStream_t stream) {
  const long first = fp8_pack_blocks(a.m, a.n), second = b.x ? fp8_pack_blocks(b.m, b.n) : 0;
  hipLaunchKernelGGL(fp8_pack<DT>, dim3((unsigned)(first + second)), dim3(kPackThreads), 0, stream, a, b, (int)first);
}

}  // namespace

long fp8_pack_blocks(long m, long n) { return ((m + kFp8Block - 1) / kFp8Block) * (fp8_cols(n) / kFp8Block); }

hipError_t launch_fp8_pack(const Fp8PackArgs& a, const Fp8PackArgs& b, int dtype, hipStream_t stream) {
  if (dtype == OIDN_F32) launch<OIDN_F32>(a, b, stream);
  else if (dtype == OIDN_F16) launch<OIDN_F16>(a, b, stream);
  else launch<OIDN_BF16>(a, b, stream);
  return hipGetLastError();
}

hipError_t launch_fp8_unpack(const void* packed, long m, long n, void* y, long ldy, int dtype, hipStream_t stream) {
  const long units = (n + 7) / 8, blocks = (m * units + kPackThreads - 1) / kPackThreads;
  const dim3 grid((unsigned)(blocks < 65536 ? blocks : 65536)), block(kPackThreads);
  void* const p = const_cast<void*>(packed);
  if (dtype == OIDN_F32) hipLaunchKernelGGL(fp8_unpack<OIDN_F32>, grid, block, 0, stream, p, m, (int)n, y, ldy, units);
  else if (dtype == OIDN_F16) hipLaunchKernelGGL(fp8_unpack<OIDN_F16>, grid, block, 0, stream, p, m, (int)n, y, ldy, units);
  else hipLaunchKernelGGL(fp8_unpack<OIDN_BF16>, grid, block, 0, stream, p, m, (int)n, y, ldy, units);
  return hipGetLastError();
}

}  // namespace oidn
