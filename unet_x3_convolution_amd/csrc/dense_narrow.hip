// Gradients of a narrow 16-bit dense layer (at most 128 inputs and outputs, as
// the network's own activations have) in one pass over the rows.
//
// dz = dy act'(z) is needed twice, for dx = dz w and for dw = dz^T x, and in a
// layer this narrow it costs more to move than to compute.  A workgroup takes
// blocks of 64 rows: it reads dy, z and x once, keeps dz and x in LDS in one
// layout that serves both products (rows of 64 elements, 16-byte slot s of row r
// at s ^ (r / 2 % 8); dw reads them transposed), holds w in LDS and its share of
// dw (and the bias's column sums) in registers over all its blocks, and writes
// dx.  The next block's loads are in flight while this one is multiplied.  Each
// workgroup leaves one fp32 slice of dw, which the finishing sums add in order.
//
// Bound by memory: 130560 rows, 32 -> 64 fp16 move 50 MB in 17 us (2.9 TB/s), and
// the sums of 512 slices take 7 us after it; as separate passes (slope, products,
// sums) the same took 60.  The number of workgroups: narrow_grid.
#include "dense_gemm16.h"

namespace oidn {
namespace {

// ROWS rows of 64 * CHUNKS elements, in chunks of 64 columns.
template <int ROWS>
struct Rows16 {
  static __device__ __forceinline__ int at(int row, int col) {
    return (((col >> 6) * ROWS + row) * 8 + (((col >> 3) & 7) ^ ((row >> 1) & 7))) * 16 + 2 * (col & 7);
  }
  // Fragment of 16 rows for the 32 summed columns from l on.
  static __device__ __forceinline__ uint4 along(const char* lds, int row0, int l) {
    const int lane = threadIdx.x & 63;
    return *reinterpret_cast<const uint4*>(lds + at(row0 + (lane & 15), l + 8 * (lane >> 4)));
  }
  // Fragment of 16 columns for the 32 summed rows from l on.  PAIR: row r of
  // fragment q is column col0 + 8 (r / 4) + 4 q + r % 4; else col0 + 16 q + r.
  template <bool PAIR>
  static __device__ __forceinline__ uint4 across(const char* lds, int col0, int q, int l) {
    const int lane = threadIdx.x & 63, g = lane >> 4, r = lane & 15, c = r & 3;
    const int col = col0 + (PAIR ? 8 * c + 4 * q : 16 * q + 4 * c);
    typedef __attribute__((address_space(3))) shortx4* lds4;
    uint2 h[2];
#pragma unroll
    for (int e = 0; e < 2; ++e)
      h[e] = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                           (lds4)(lds + at(l + 8 * g + 4 * e + (r >> 2), col))));
    return make_uint4(h[0].x, h[0].y, h[1].x, h[1].y);
  }
};

// 128 x 128 needs more than the 256 registers that two workgroups a unit would
// leave each thread: within them it spilled and took 98 us at 130560 rows, now 54.
template <bool BF, int NP, int KP>
__global__ __launch_bounds__(256, NP * KP == 128 * 128 ? 1 : NP * KP > 64 * 64 ? 2 : 3)
void narrow_back(NarrowArgs a) {
  constexpr int DT = BF ? OIDN_BF16 : OIDN_F16;
  constexpr int FC = KP / 32;              // column fragments of a wave, of dx and of dw
  constexpr int FN = NP / 32;              // row fragments of a wave's dw
  typedef Loader<2, NP, 64, true> FromN;
  typedef Loader<2, KP, 64, true> FromK;
  __shared__ __attribute__((aligned(16))) char dz_lds[64 * NP * 2], x_lds[64 * KP * 2], w_lds[NP * KP * 2];
  const int wave = threadIdx.x >> 6, wr = wave >> 1, wc = wave & 1;
  const int lane = threadIdx.x & 63, g = lane >> 4;
  const bool slope = a.act != OIDN_ACT_NONE;

  if (a.dx) {                              // w, row by row; zeros past its rows and columns
    const Extent<2> all(a.w, a.n, a.ldw, a.k);
    for (int t = threadIdx.x; t < NP * KP / 8; t += 256) {
      const int r = t / (KP / 8), c = t % (KP / 8) * 8;
      uint4 u[1];
      all.load(u, [&](int, const char*& p, long& n) {
        p = all.first + 2 * (r * a.ldw + c);
        n = r < a.n ? a.k - c : 0;
      });
      *reinterpret_cast<uint4*>(w_lds + Rows16<NP>::at(r, c)) = u[0];
    }
  }

  FromN from_dy(a.dy, a.lddy, 0, a.n, 64L * blockIdx.x, a.rows, 0);
  FromN from_z(slope ? a.z : a.dy, slope ? a.ldz : a.lddy, 0, a.n, 64L * blockIdx.x, a.rows, 0);
  FromK from_x(a.dw ? a.x : a.dy, a.dw ? a.ldx : a.lddy, 0, a.dw ? a.k : a.n, 64L * blockIdx.x, a.rows, 0);
  from_dy.step *= gridDim.x;
  from_z.step *= gridDim.x;
  from_x.step *= gridDim.x;
  uint4 dy[FromN::kUnits], z[FromN::kUnits], x[FromK::kUnits];
  auto load = [&](int b) {
    if (b >= a.blocks) return;
    from_dy.load(dy, 64L * b);
    if (slope) from_z.load(z, 64L * b);
    if (a.dw) from_x.load(x, 64L * b);
  };

  floatx4 dw[FC][FN];
#pragma unroll
  for (int c = 0; c < FC; ++c)
#pragma unroll
    for (int r = 0; r < FN; ++r) dw[c][r] = floatx4{0.f, 0.f, 0.f, 0.f};
  Eight sum{};                             // of the thread's eight columns (the same for all its units)
  static_assert(256 % (NP / 8) == 0, "a thread's units share their columns");

  load(blockIdx.x);
  for (int b = blockIdx.x; b < a.blocks; b += gridDim.x) {
    __syncthreads();                       // the block before this one has been read (and w is written)
    typedef typename Storage<DT>::T T;
    typedef T T8 __attribute__((ext_vector_type(8)));
#pragma unroll
    for (int u = 0; u < FromN::kUnits; ++u) {
      const T8 d = __builtin_bit_cast(T8, dy[u]);
      Eight v;
#pragma unroll
      for (int k = 0; k < 8; ++k) v.v[k] = (float)d[k];
      uint4 kept = dy[u];
      if (slope) {
        const T8 zz = __builtin_bit_cast(T8, z[u]);
        Eight s, value;
#pragma unroll
        for (int k = 0; k < 8; ++k) s.v[k] = (float)zz[k];
        activate_slope8<DT>(a.act, s, value);
        T8 r;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          v.v[k] *= s.v[k];
          r[k] = (T)v.v[k];                // rounded as the products read it; the sums are not
        }
        kept = __builtin_bit_cast(uint4, r);
      }
      add8(sum, v);                        // rows and columns that do not exist are zeros
      int r, s;
      FromN::place(u, r, s);
      *reinterpret_cast<uint4*>(dz_lds + Rows16<64>::at(r, 8 * s)) = kept;
    }
    if (a.dw) {
#pragma unroll
      for (int u = 0; u < FromK::kUnits; ++u) {
        int r, s;
        FromK::place(u, r, s);
        *reinterpret_cast<uint4*>(x_lds + Rows16<64>::at(r, 8 * s)) = x[u];
      }
    }
    __syncthreads();
    load(b + gridDim.x);
    if (a.dx) {
      floatx4 dx[FC][2];
#pragma unroll
      for (int c = 0; c < FC; ++c)
#pragma unroll
        for (int r = 0; r < 2; ++r) dx[c][r] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int l = 0; l < NP; l += 32) {
        uint4 fq[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) fq[r] = Rows16<64>::along(dz_lds, 32 * wr + 16 * r, l);
#pragma unroll
        for (int c = 0; c < FC; ++c) {
          const uint4 fp = Rows16<NP>::template across<true>(w_lds, wc * (KP / 2) + 32 * (c / 2), c & 1, l);
#pragma unroll
          for (int r = 0; r < 2; ++r) dx[c][r] = mfma16<BF>(fp, fq[r], dx[c][r]);
        }
      }
      // lane l: row l % 16 of a row fragment, columns 8 (l / 16) .. + 7 of a pair
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const long i = 64L * b + 32 * wr + 16 * r + (lane & 15);
#pragma unroll
        for (int pair = 0; pair < FC / 2; ++pair) {
          const int j = wc * (KP / 2) + 32 * pair + 8 * g, n = a.k - j;
          Eight v;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            v.v[k] = dx[2 * pair][r][k];
            v.v[4 + k] = dx[2 * pair + 1][r][k];
          }
          if (i < a.rows && n > 0) store8<DT>(a.dx, i * a.lddx + j, v, n);
        }
      }
    }
    if (a.dw) {
#pragma unroll
      for (int l = 0; l < 64; l += 32) {
        uint4 fq[FN];
#pragma unroll
        for (int r = 0; r < FN; ++r) fq[r] = Rows16<64>::template across<false>(dz_lds, wr * (NP / 2), r, l);
#pragma unroll
        for (int c = 0; c < FC; ++c) {
          const uint4 fp = Rows16<64>::template across<true>(x_lds, wc * (KP / 2) + 32 * (c / 2), c & 1, l);
#pragma unroll
          for (int r = 0; r < FN; ++r) dw[c][r] = mfma16<BF>(fp, fq[r], dw[c][r]);
        }
      }
    }
  }

  if (a.dw) {
#pragma unroll
    for (int r = 0; r < FN; ++r) {
      const long i = wr * (NP / 2) + 16 * r + (lane & 15);
#pragma unroll
      for (int pair = 0; pair < FC / 2; ++pair) {
        const int j = wc * (KP / 2) + 32 * pair + 8 * g, n = a.k - j;
        Eight v;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          v.v[k] = dw[2 * pair][r][k];
          v.v[4 + k] = dw[2 * pair + 1][r][k];
        }
        if (i >= a.n || n <= 0) continue;
        if (gridDim.x > 1) store8<OIDN_F32>(a.slices, (blockIdx.x * (long)a.n + i) * a.k + j, v, n);
        else store8<DT>(a.dw, i * a.lddw + j, v, n);
      }
    }
  }
  if (a.sums) {
    // the row lanes of a unit are added in order; LDS is free after the last block
    constexpr int kUnits = NP / 8, kLanes = 256 / kUnits;
    float* const lds = reinterpret_cast<float*>(w_lds);
    static_assert(sizeof(w_lds) >= 64 * 64 * 2, "room for 256 x 8 floats");
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 8; ++k) lds[threadIdx.x * 8 + k] = sum.v[k];
    __syncthreads();
    if ((int)threadIdx.x < a.n) {
      const int u = threadIdx.x / 8, k = threadIdx.x % 8;
      float s = 0.f;
      for (int r = 0; r < kLanes; ++r) s += lds[(r * kUnits + u) * 8 + k];
      a.sums[blockIdx.x * (long)a.n + threadIdx.x] = s;
    }
  }
}

template <bool BF>
hipError_t launch_type(const NarrowArgs& a, int grid, hipStream_t stream) {
  const dim3 g((unsigned)grid), block(256);
  if (a.n <= 64 && a.k <= 64) hipLaunchKernelGGL((narrow_back<BF, 64, 64>), g, block, 0, stream, a);
  else if (a.n <= 64) hipLaunchKernelGGL((narrow_back<BF, 64, 128>), g, block, 0, stream, a);
  else if (a.k <= 64) hipLaunchKernelGGL((narrow_back<BF, 128, 64>), g, block, 0, stream, a);
  else hipLaunchKernelGGL((narrow_back<BF, 128, 128>), g, block, 0, stream, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_narrow_back(const NarrowArgs& a, int grid, bool bf16, hipStream_t stream) {
  return bf16 ? launch_type<true>(a, grid, stream) : launch_type<false>(a, grid, stream);
}

}  // namespace oidn
