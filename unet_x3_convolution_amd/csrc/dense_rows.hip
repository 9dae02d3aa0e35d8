// Memory-bound passes of the dense operators: the sum of a product's slices,
// the slope pass dz = dy * act'(z) with column sums, column sums of partial
// rows, 8-bit checkpoints of whole matrices, and zeros.
//
// Small ones take a launch's 2 to 3 us; 32640 x 112 fp16 goes to 8 bits in 5.2 us
// and back in 4.0, 16384 x 2048 bf16 (103 MB) in 22.6 us (4.6 TB/s), there and back
// in 40.
#include "dense_slope.h"

namespace oidn {
namespace {

// Sums of a product's slices: a workgroup takes 256 >> lg units of eight
// columns, 1 << lg of its threads share a unit's slices, several reads in
// flight each, and their sums are added in order, so the result does not
// depend on timing.  Units of a row are padded to whole 32-column blocks: four
// neighbouring threads hold one.
template <int DT, int EPI>
__device__ __forceinline__ void sum_slices(const EpilogueArgs& e, int splits, int lg, long block, char* lds) {
  const int at_once = kRowThreads >> lg, u = threadIdx.x & (at_once - 1), lane = threadIdx.x >> (8 - lg);
  const long units = (e.cols + 31) / 32 * 4, total = e.rows * units;
  const long t = block * at_once + u, i = t / units;
  const int j = (int)(t - i * units) * 8, n = e.cols - j;
  Eight x{};
  if (t < total && n > 0) {
    const long step = e.rows * (long)e.cols;
    const float* p = e.part + i * e.cols + j;
#pragma unroll 4
    for (int s = lane; s < splits; s += 1 << lg) add8(x, load8<OIDN_F32>(p, s * step, n));
  }
  if (lg) {
    Eight* const sums = reinterpret_cast<Eight*>(lds);
    if (lane) sums[threadIdx.x - at_once] = x;
    __syncthreads();
    if (lane) return;
    for (int s = 1; s < 1 << lg; ++s) add8(x, sums[(s - 1) * at_once + u]);
  }
  Fetched none, bias{};
  RawFetched<DT, false> f;
  if constexpr (EPI == kEpiLinear) bias.a = bias8(e.bias, j, n);
  fetch<DT, EPI, false, false>(e, i, j, f);
  finish<DT, EPI, false, false>(e, 0, i, j, x, x, bias, f, none);
}
constexpr int kSumLds = kRowThreads * 32;

// Threads that share a unit: as many as have four slices each, at most 32.
int slice_lanes(int splits) {
  int lg = 0;
  while (lg < 5 && (8 << lg) <= splits) ++lg;
  return lg;
}

template <int DT>
__global__ __launch_bounds__(kRowThreads) void split_sum(EpilogueArgs e, int splits, int lg) {
  __shared__ __attribute__((aligned(16))) char lds[kSumLds];
  sum_slices<DT, kEpiLinear>(e, splits, lg, blockIdx.x, lds);
}

// Columns of partial sums, 256 / lanes of them a workgroup: each is shared by
// `lanes` threads, eight reads in flight each, added in order.
__device__ __forceinline__ void sum_columns(const float* __restrict__ part, long groups, int cols,
                                            float* __restrict__ out, int block, int lanes, char* mem) {
  const int across = kRowThreads / lanes, c = threadIdx.x % across, l = threadIdx.x / across, j = block * across + c;
  float s = 0.f;
  if (j < cols) {
#pragma unroll 8
    for (long g = l; g < groups; g += lanes) s += part[g * cols + j];
  }
  float* const lds = reinterpret_cast<float*>(mem);
  lds[threadIdx.x] = s;
  __syncthreads();
  if (l == 0 && j < cols) {
    for (int k = 1; k < lanes; ++k) s += lds[k * across + c];
    out[j] = s;
  }
}
int column_lanes(long groups) { return groups > 64 ? 32 : 8; }

struct FinishPlan {
  int start[kMaxGroup + 2 + 1];     // first workgroup of each job, products first
  int lg[kMaxGroup];
  int lanes[2];
};
template <int DT>
__global__ __launch_bounds__(kRowThreads) void finish_sums(FinishArgs a, FinishPlan p) {
  __shared__ __attribute__((aligned(16))) char lds[kSumLds];
  int k = 0;
  while ((int)blockIdx.x >= p.start[k + 1]) ++k;
  const int block = blockIdx.x - p.start[k];
  if (k < a.products) {
    sum_slices<DT, kEpiStore>(a.product[k].e, a.product[k].splits, p.lg[k], block, lds);
  } else {
    const auto& c = a.column[k - a.products];
    sum_columns(c.part, c.groups, c.cols, c.out, block, p.lanes[k - a.products], lds);
  }
}

template <int DT>
__global__ __launch_bounds__(kRowThreads) void slope_pass(SlopeArgs a, UnpackJob u) {
  __shared__ float lds[kSlopeLds / 4];
  if ((int)blockIdx.x < u.blocks) unpack_rows<DT>(u, blockIdx.x);
  else slope_rows<DT>(a, blockIdx.x - u.blocks, lds);
}

// Thread of a launch over `row_grid`: one dimension, or two where a matrix has more
// units than the work items that one holds.
__device__ __forceinline__ long unit_index() {
  return ((long)blockIdx.y * gridDim.x + blockIdx.x) * kRowThreads + threadIdx.x;
}
dim3 row_grid(long units) {
  const long blocks = (units + kRowThreads - 1) / kRowThreads, most = 1L << 23;
  return blocks <= most ? dim3((unsigned)blocks) : dim3((unsigned)most, (unsigned)((blocks + most - 1) / most));
}

// A thread codes eight columns; four neighbouring lanes hold a block.
template <int DT>
__global__ __launch_bounds__(kRowThreads) void ckpt_pack(const void* __restrict__ x, long ldx, long m,
                                                         long n, void* ckpt, long units, long total) {
  const long t = unit_index();
  const long i = t / units, j = (t - i * units) * 8;
  Eight v{};
  const int left = n - j < 8 ? (int)(n - j) : 8;
  if (t < total && left > 0) v = load8<DT>(x, i * ldx + j, left);
  ckpt_store8(ckpt_at(ckpt, m, n), i, (int)j, v, t < total);
}

template <int DT>
__global__ __launch_bounds__(kRowThreads) void ckpt_unpack(void* ckpt, long m, long n, void* __restrict__ y,
                                                           long ldy, long units, long total) {
  const long t = unit_index();
  const long i = t / units, j = (t - i * units) * 8;
  const int left = n - j < 8 ? (int)(n - j) : 8;
  if (t >= total || left <= 0) return;
  store8<DT>(y, i * ldy + j, ckpt_stored<DT>(load_codes(ckpt_at(ckpt, m, n), i, (int)j)), left);
}

__global__ __launch_bounds__(kRowThreads) void zero_rows(unsigned char* p, size_t width, size_t pitch, size_t total) {
  const size_t step = (size_t)gridDim.x * kRowThreads;
  for (size_t i = (size_t)blockIdx.x * kRowThreads + threadIdx.x; i < total; i += step)
    p[i / width * pitch + i % width] = 0;
}

}  // namespace

long slice_blocks(long rows, int cols, int splits) {
  const long per = kRowThreads >> slice_lanes(splits);
  return (rows * ((cols + 31) / 32 * 4) + per - 1) / per;
}
long column_blocks(long groups, int cols) {
  const int across = kRowThreads / column_lanes(groups);
  return (cols + across - 1) / across;
}

hipError_t launch_split_sum(const EpilogueArgs& e, int splits, int dtype, hipStream_t stream) {
  const int lg = slice_lanes(splits);
  const dim3 grid((unsigned)slice_blocks(e.rows, e.cols, splits)), block(kRowThreads);
  if (dtype == OIDN_F32) hipLaunchKernelGGL(split_sum<OIDN_F32>, grid, block, 0, stream, e, splits, lg);
  else if (dtype == OIDN_F16) hipLaunchKernelGGL(split_sum<OIDN_F16>, grid, block, 0, stream, e, splits, lg);
  else hipLaunchKernelGGL(split_sum<OIDN_BF16>, grid, block, 0, stream, e, splits, lg);
  return hipGetLastError();
}

hipError_t launch_finish(const FinishArgs& a, int dtype, hipStream_t stream) {
  FinishPlan p{};
  int k = 0;
  for (; k < a.products; ++k) {
    const auto& s = a.product[k];
    p.lg[k] = slice_lanes(s.splits);
    p.start[k + 1] = p.start[k] + (int)slice_blocks(s.e.rows, s.e.cols, s.splits);
  }
  for (int c = 0; c < a.columns; ++c, ++k) {
    p.lanes[c] = column_lanes(a.column[c].groups);
    p.start[k + 1] = p.start[k] + (int)column_blocks(a.column[c].groups, a.column[c].cols);
  }
  if (k == 0) return hipSuccess;
  const dim3 grid((unsigned)p.start[k]), block(kRowThreads);
  if (dtype == OIDN_F32) hipLaunchKernelGGL(finish_sums<OIDN_F32>, grid, block, 0, stream, a, p);
  else if (dtype == OIDN_F16) hipLaunchKernelGGL(finish_sums<OIDN_F16>, grid, block, 0, stream, a, p);
  else hipLaunchKernelGGL(finish_sums<OIDN_BF16>, grid, block, 0, stream, a, p);
  return hipGetLastError();
}

long slope_chunk(long rows) {
  // at most 256 chunks, so that the column sums stay a short second pass; at
  // least 32 rows, so that a workgroup's lanes have work
  const long c = (rows + 255) / 256;
  return c < 32 ? 32 : c;
}

int slope_lanes(int cols) {
  const int units = (cols + 7) / 8;
  int cs = 0;
  while (cs < 5 && (1 << cs) < units) ++cs;
  return cs;
}
long slope_blocks(const SlopeArgs& a) {
  return ((a.rows + a.chunk - 1) / a.chunk) * (((a.cols + 7) / 8 + (1 << a.lanes) - 1) >> a.lanes);
}

hipError_t launch_slope(const SlopeArgs& a, const UnpackJob& u, int dtype, hipStream_t stream) {
  const dim3 grid((unsigned)(slope_blocks(a) + u.blocks)), block(kRowThreads);
  if (dtype == OIDN_F32) hipLaunchKernelGGL(slope_pass<OIDN_F32>, grid, block, 0, stream, a, u);
  else if (dtype == OIDN_F16) hipLaunchKernelGGL(slope_pass<OIDN_F16>, grid, block, 0, stream, a, u);
  else hipLaunchKernelGGL(slope_pass<OIDN_BF16>, grid, block, 0, stream, a, u);
  return hipGetLastError();
}

hipError_t launch_ckpt_pack(const void* x, long ldx, long m, long n, void* ckpt, int dtype,
                            hipStream_t stream) {
  const long units = ckpt_cols(n) / 8, total = m * units;
  const dim3 grid = row_grid(total), block(kRowThreads);
  if (dtype == OIDN_F32)
    hipLaunchKernelGGL(ckpt_pack<OIDN_F32>, grid, block, 0, stream, x, ldx, m, n, ckpt, units, total);
  else if (dtype == OIDN_F16)
    hipLaunchKernelGGL(ckpt_pack<OIDN_F16>, grid, block, 0, stream, x, ldx, m, n, ckpt, units, total);
  else
    hipLaunchKernelGGL(ckpt_pack<OIDN_BF16>, grid, block, 0, stream, x, ldx, m, n, ckpt, units, total);
  return hipGetLastError();
}

hipError_t launch_ckpt_unpack(const void* ckpt, long m, long n, void* y, long ldy, int dtype,
                              hipStream_t stream) {
  void* const c = const_cast<void*>(ckpt);
  const long units = (n + 7) / 8, total = m * units;
  const dim3 grid = row_grid(total), block(kRowThreads);
  if (dtype == OIDN_F32)
    hipLaunchKernelGGL(ckpt_unpack<OIDN_F32>, grid, block, 0, stream, c, m, n, y, ldy, units, total);
  else if (dtype == OIDN_F16)
    hipLaunchKernelGGL(ckpt_unpack<OIDN_F16>, grid, block, 0, stream, c, m, n, y, ldy, units, total);
  else
    hipLaunchKernelGGL(ckpt_unpack<OIDN_BF16>, grid, block, 0, stream, c, m, n, y, ldy, units, total);
  return hipGetLastError();
}

hipError_t launch_zero(void* p, long rows, size_t width, size_t pitch, hipStream_t stream) {
  const size_t total = rows * width, b = (total + kRowThreads - 1) / kRowThreads;
  hipLaunchKernelGGL(zero_rows, dim3((unsigned)(b < 2048 ? b : 2048)), dim3(kRowThreads), 0, stream,
                     static_cast<unsigned char*>(p), width, pitch, total);
  return hipGetLastError();
}

}  // namespace oidn
