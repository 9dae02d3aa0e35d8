// Matrices to 8-bit floating point and back.
#include "fp8_code.h"
#include "lanes.h"

namespace oidn {
namespace {

constexpr int kPackThreads = 256;

// Columns j .. j + 7 of row i, zeros past the matrix.  The load is always made, from the
// last row past the end, so that a thread's loads are in flight together.
template <int DT>
struct Cell {
  Raw<DT> raw;
  int n;                   // columns that exist, 0 past the rows
  __device__ __forceinline__ void load(const void* p, long ld, long i, int j, long m, int cols) {
    const long at = i < m ? i : m - 1;
    raw = load_raw<DT>(p, at * ld + j, cols - j, (m - 1 - at) * ld + cols - j);
    n = i < m ? cols - j : 0;
  }
  __device__ __forceinline__ Eight value() const {
    Eight r = raw.value();
    if (n < 8) clear_tail(n, r);
    return r;
  }
};
// x alone, blocks along the rows.  1 << lg lanes (16 to 64) take a row's one to four
// blocks, so that a word of scales is theirs; a wave's loads are of kPackRows rows
// each.  Bound by memory: 8192 x 4096 bf16 (101 MB) 18.1 us, 5.6 TB/s.
constexpr int kPackRows = 4;
template <int DT>
__global__ __launch_bounds__(kPackThreads) void fp8_pack_rows(Fp8PackArgs a, int lg, int words) {
  const int lane = threadIdx.x & 63, part = lane & ((1 << lg) - 1), rows = kPackThreads >> lg;
  const long chunk = blockIdx.x / words;
  const int word = (int)(blockIdx.x - chunk * words), j = word * 4 * kFp8Block + 8 * part;
  const long i0 = chunk * rows * kPackRows + (threadIdx.x >> lg);
  const Fp8At at = fp8_at(a.rows, a.m, a.n);
  Cell<DT> cell[kPackRows];
#pragma unroll
  for (int k = 0; k < kPackRows; ++k) cell[k].load(a.x, a.ldx, i0 + k * rows, j, a.m, a.n);
#pragma unroll
  for (int k = 0; k < kPackRows; ++k) {
    const long i = i0 + k * rows;
    const Eight v = cell[k].value();
    const int p = fp8_power(lanes_max<16>(finite_top(v)));
    // each block's byte in its place of the word, brought together in the row's first lane
    unsigned s = (unsigned)(p + 127) << (part / 16 * 8);
    if (lg > 4) s |= __shfl_xor(s, 16);
    if (lg > 5) s |= __shfl_xor(s, 32);
    if (i < a.m) {
      if (j < at.pitch) *reinterpret_cast<uint2*>(at.codes + i * at.pitch + j) = fp8_codes(v.v, power_of_two(-p));
      if (part == 0) *reinterpret_cast<unsigned*>(at.scales + i * at.words + 4 * word) = s;
    }
  }
}

// Both forms, or with a slope, a square's scale or column sums.  A workgroup takes 128 x
// 128 elements, a thread eight columns of four rows that follow each other, so that it
// holds four codes in a row of the turned form.  A row's block lies in 16 lanes; a
// column's in all waves.  The turned codes pass through LDS, from where whole lines
// leave: 16-byte unit u of column 8 c + e sits at u ^ c % 8, and every second half of
// the columns in the neighbouring row, so that a wave's writes go to 64 banks.
// 8192 x 4096 bf16: turned (101 MB) 20.0 us, both forms (135 MB) 26.9, 5.0 TB/s; with the slope
// of gelu and column sums (202 MB) 52 to 58, bound by the activation's instructions.  Few
// tiles take one tile's time on one unit, some 1000 to 2500 instructions of two waves a SIMD:
// 5 us, with a slope, sums and both forms 8.
constexpr int kTileThreads = 512, kTileWaves = kTileThreads / 64, kTileRows = 4;
struct PackLds {
  unsigned top[kTileWaves][kFp8Block];
  float sum[kTileWaves][kFp8Block];
  unsigned codes[kFp8Block][kFp8Block / 4];
};
__device__ __forceinline__ int turned_row(int column) { return column ^ (column >> 6 & 1); }
__device__ __forceinline__ int turned_unit(int column, int unit) { return unit ^ (column >> 3 & 7); }

// INSIDE: all of the tile lies in the matrix.  ACT: that of z, where there is a z; a
// kernel for each, as the code of all of them takes longer to fetch than to run.
template <int DT, bool INSIDE, int ACT>
__device__ __forceinline__ void pack_tile(const Fp8PackArgs& a, long tile_r, int tile_c, PackLds& lds) {
  const int t = threadIdx.x, c = t & 15, g = t >> 4, wave = t >> 6;
  const long i0 = tile_r * kFp8Block + kTileRows * g;
  const int j = tile_c * kFp8Block + 8 * c;
  typedef typename Storage<DT>::T E;
  Cell<DT> cell[kTileRows], slope[kTileRows];
  RawCodes slope8[kTileRows];
  auto load = [&](Cell<DT> (&to)[kTileRows], const void* p, long ld) __attribute__((always_inline)) {
    const E* at = static_cast<const E*>(p) + i0 * ld + j;
#pragma unroll
    for (int k = 0; k < kTileRows; ++k) {
      if constexpr (INSIDE) {
        __builtin_memcpy(&to[k].raw.e, at, sizeof(to[k].raw.e));
        at += ld;
      } else {
        to[k].load(p, ld, i0 + k, j, a.m, a.n);
      }
    }
  };
  load(cell, a.x, a.ldx);
  if (ACT != OIDN_ACT_NONE && a.z && !a.z8) {
    load(slope, a.z, a.ldz);
  } else if (ACT != OIDN_ACT_NONE && a.z) {
#pragma unroll
    for (int k = 0; k < kTileRows; ++k)
      slope8[k] = load_codes(ckpt_at(const_cast<void*>(a.z), a.m, a.n), i0 + k < a.m ? i0 + k : a.m - 1,
                             j < a.n ? j : 0);
  }
  Eight v[kTileRows];
#pragma unroll
  for (int k = 0; k < kTileRows; ++k) {
    v[k] = INSIDE ? cell[k].raw.value() : cell[k].value();
    if (ACT != OIDN_ACT_NONE && a.z) {
      Eight z = a.z8 ? slope8[k].value() : INSIDE ? slope[k].raw.value() : slope[k].value(), value;
      activate_slope8<DT>(ACT, z, value);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (INSIDE || e < cell[k].n) v[k].v[e] *= z.v[e];
    }
  }
  unsigned row_top[kTileRows], col_top[8] = {}, top = 0;
  auto tops = [&](auto bits) {
#pragma unroll
    for (int e = 0; e < 8; ++e) col_top[e] = 0;
#pragma unroll
    for (int k = 0; k < kTileRows; ++k) {
      row_top[k] = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const unsigned b = bits(v[k].v[e]);
        row_top[k] = max(row_top[k], b);
        col_top[e] = max(col_top[e], b);
      }
      top = max(top, row_top[k]);
    }
  };
  tops([](float f) { return magnitude_bits(f); });
  if (top >= 0x7f800000u) tops([](float f) { return finite_bits(f); });      // rare
  if (a.sums) {
    Eight s = v[0];
#pragma unroll
    for (int k = 1; k < kTileRows; ++k) add8(s, v[k]);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      s.v[e] = lanes_sum<64, 16>(s.v[e]);
      if ((t & 63) < 16) lds.sum[wave][8 * c + e] = s.v[e];
    }
  }
  if (a.turned || a.square) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      col_top[e] = lanes_max<64, 16>(col_top[e]);
      if ((t & 63) < 16) lds.top[wave][8 * c + e] = col_top[e];
    }
  }
  __syncthreads();
  if (a.turned || a.square) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      col_top[e] = 0;
#pragma unroll
      for (int w = 0; w < kTileWaves; ++w) col_top[e] = max(col_top[e], lds.top[w][8 * c + e]);
    }
  }
  if (a.square) {
    unsigned all = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) all = max(all, col_top[e]);
    all = lanes_max<16>(all);
#pragma unroll
    for (int e = 0; e < 8; ++e) col_top[e] = all;
#pragma unroll
    for (int k = 0; k < kTileRows; ++k) row_top[k] = all;
  }
  if (a.sums && t < kFp8Block && tile_c * kFp8Block + t < a.n) {
    float s = lds.sum[0][t];
#pragma unroll
    for (int w = 1; w < kTileWaves; ++w) s += lds.sum[w][t];
    a.sums[tile_r * a.n + tile_c * kFp8Block + t] = s;
  }
  if (a.rows) {
    const Fp8At at = fp8_at(a.rows, a.m, a.n);
#pragma unroll
    for (int k = 0; k < kTileRows; ++k) {
      const long i = i0 + k;
      const int p = fp8_power(a.square ? row_top[k] : lanes_max<16>(row_top[k]));
      if (!INSIDE && i >= a.m) continue;
      *reinterpret_cast<uint2*>(at.codes + i * at.pitch + j) = fp8_codes(v[k].v, power_of_two(-p));
      if (c == 0) at.scales[i * at.words + tile_c] = (unsigned char)(p + 127);
    }
  }
  if (a.turned) {
    const Fp8At at = fp8_at(a.turned, a.n, a.m);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int p = fp8_power(col_top[e]), column = 8 * c + e;
      const float inverse = power_of_two(-p);
      float f[kTileRows];
#pragma unroll
      for (int k = 0; k < kTileRows; ++k) f[k] = v[k].v[e];
      lds.codes[turned_row(column)][4 * turned_unit(column, g >> 2) + (g & 3)] = fp8_codes4(f, inverse);
      if (g == 0 && (INSIDE || j + e < a.n)) at.scales[(j + e) * at.words + tile_r] = (unsigned char)(p + 127);
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kFp8Block * kFp8Block / 16 / kTileThreads; ++k) {
      const int u = t + k * kTileThreads, column = u >> 3, unit = u & 7;
      const long col = tile_c * (long)kFp8Block + column;
      if (INSIDE || col < a.n)
        *reinterpret_cast<uint4*>(at.codes + col * at.pitch + tile_r * kFp8Block + 16 * unit) =
            *reinterpret_cast<const uint4*>(&lds.codes[turned_row(column)][4 * turned_unit(column, unit)]);
    }
  }
}

template <int DT, int ACT>
__global__ __launch_bounds__(kTileThreads) void fp8_pack_tiles(Fp8PackArgs a, Fp8PackArgs b, int first) {
  __shared__ __attribute__((aligned(16))) PackLds lds;
  const bool second = (int)blockIdx.x >= first;
  const Fp8PackArgs& p = second ? b : a;
  const unsigned block = blockIdx.x - (second ? first : 0), across = ((unsigned)p.n + kFp8Block - 1) / kFp8Block;
  const long tile_r = block / across;
  const int tile_c = (int)(block % across);
  if ((tile_r + 1) * kFp8Block <= p.m && (tile_c + 1) * kFp8Block <= p.n) pack_tile<DT, true, ACT>(p, tile_r, tile_c, lds);
  else pack_tile<DT, false, ACT>(p, tile_r, tile_c, lds);
}

// A thread takes eight columns.  A finite value whose rounding passes the type's
// range becomes the largest one.  Bound by memory:
// 8192 x 4096 bf16 (101 MB) 21.9 us, 4.6 TB/s; 32640 x 112 fp16 5.3.
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

bool rows_alone(const Fp8PackArgs& a) { return !a.turned && !a.z && !a.square && !a.sums; }
// Lanes of a row in fp8_pack_rows.
int row_lanes(long n) {
  const long blocks = fp8_cols(n) / kFp8Block;
  return blocks == 1 ? 4 : blocks == 2 ? 5 : 6;
}
long row_chunks(long m, long n) {
  const long rows = (kPackThreads >> row_lanes(n)) * kPackRows;
  return (m + rows - 1) / rows;
}

template <int DT>
void launch(const Fp8PackArgs& a, const Fp8PackArgs& b, hipStream_t stream) {
  if (rows_alone(a) && !b.x) {
    const int words = (int)(fp8_scales(a.n) / 4);
    hipLaunchKernelGGL(fp8_pack_rows<DT>, dim3((unsigned)(row_chunks(a.m, a.n) * words)), dim3(kPackThreads), 0, stream, a,
                       row_lanes(a.n), words);
    return;
  }
  const long first = fp8_tiles(a.m, a.n), second = b.x ? fp8_tiles(b.m, b.n) : 0;
  const dim3 grid((unsigned)(first + second)), block(kTileThreads);
  const int act = a.z ? a.act : OIDN_ACT_NONE;
  if (act == OIDN_ACT_NONE) hipLaunchKernelGGL((fp8_pack_tiles<DT, OIDN_ACT_NONE>), grid, block, 0, stream, a, b, (int)first);
  else if (act == OIDN_ACT_RELU) hipLaunchKernelGGL((fp8_pack_tiles<DT, OIDN_ACT_RELU>), grid, block, 0, stream, a, b, (int)first);
  else if (act == OIDN_ACT_SILU) hipLaunchKernelGGL((fp8_pack_tiles<DT, OIDN_ACT_SILU>), grid, block, 0, stream, a, b, (int)first);
  else hipLaunchKernelGGL((fp8_pack_tiles<DT, OIDN_ACT_GELU>), grid, block, 0, stream, a, b, (int)first);
}

}  // namespace

// In workgroups of 256: a tile is twice that.
long fp8_pack_blocks(long m, long n) {
  const long rows = row_chunks(m, n) * (fp8_scales(n) / 4), tiles = 2 * fp8_tiles(m, n);
  return rows > tiles ? rows : tiles;
}

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
