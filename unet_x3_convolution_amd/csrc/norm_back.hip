// Gradients of the norms before and after a block.
#include "norm_fast.h"
#include "norm_wide.h"

namespace oidn {
namespace {

// Sums of partial rows: kinds 0 .. kNormSums - 1 over all chunks, then a gate
// group's chunks.  A workgroup takes ACROSS columns, its threads share the rows,
// whose sums are added in order.  Wide rows are bound by memory, narrow ones by the latency
// of a thread's loads, which are made sixteen at a time (us a call, 16 and 32 columns: 16384 x
// 4096 188 and 185, 4096 x 8192 149 and 143; 8160 x 96 fp32 14.4 and 15.3, 16384 x 128 19.6 and
// 21.1; in turn past the last sixteen, 8160 x 96 took 18.2).
constexpr int kFinishThreads = 512;
inline int finish_columns(int n) { return n >= 1024 ? 32 : 16; }
template <int ACROSS>
__global__ __launch_bounds__(kFinishThreads) void norm_finish(NormBackArgs a) {
  constexpr int kLines = kFinishThreads / ACROSS;
  __shared__ float lds[kFinishThreads];
  const int c = threadIdx.x % ACROSS, l = threadIdx.x / ACROSS, n = a.n;
  const long j = (long)blockIdx.x * ACROSS + c, what = blockIdx.y;
  const float* p;
  float* out;
  long count, step;
  if (what < kNormSums) {
    out = a.chunks.count > 1 ? a.sums[what] : nullptr;
    p = a.part + what * n;
    count = a.chunks.count;
    step = (long)kNormSums * n;
  } else {
    const long group = what - kNormSums;
    out = a.dgate + group * a.lddg;
    p = a.gate_part + group * a.chunks.per_group * n;
    count = a.chunks.per_group;
    step = n;
  }
  if (!out) return;
  float s = 0.f;
  if (j < n) {
    // sixteen reads at a time, the last row in place of those past it
    for (long g = l; g < count; g += 16 * kLines) {
      float t[16];
#pragma unroll
      for (int k = 0; k < 16; ++k) t[k] = p[(g + k * kLines < count ? g + k * kLines : count - 1) * step + j];
#pragma unroll
      for (int k = 0; k < 16; ++k) s += g + k * kLines < count ? t[k] : 0.f;
    }
  }
  lds[threadIdx.x] = s;
  __syncthreads();
  if (l == 0 && j < n) {
#pragma unroll
    for (int k = 1; k < kLines; ++k) s += lds[k * ACROSS + c];
    out[j] = s;
  }
}

template <int DT, int LANES, bool BRANCH, bool WHOLE, bool SHIFTS>
void launch_kernel(const NormBackArgs& a, hipStream_t stream) {
  hipLaunchKernelGGL((norm_back_rows<DT, LANES, BRANCH, WHOLE, SHIFTS>), dim3((unsigned)a.chunks.count),
                     dim3(norm_threads<LANES>()), 0, stream, a);
}
template <int DT, int LANES>
void launch_rows(const NormBackArgs& a, hipStream_t stream) {
  const bool whole = a.n % 8 == 0;
  if (!a.o && whole) launch_kernel<DT, LANES, false, true, true>(a, stream);
  else if (!a.o) launch_kernel<DT, LANES, false, false, true>(a, stream);
  else if (!whole) launch_kernel<DT, LANES, true, false, true>(a, stream);
  else if (a.sums[1] || a.sums[3]) launch_kernel<DT, LANES, true, true, true>(a, stream);
  else launch_kernel<DT, LANES, true, true, false>(a, stream);
}
template <int DT>
hipError_t launch_type(const NormBackArgs& a, hipStream_t stream) {
  bool columns = a.dgate != nullptr;
  for (int k = 0; k < kNormSums; ++k) columns = columns || a.sums[k];
  switch (norm_lanes(a.n)) {
    case 4: launch_rows<DT, 4>(a, stream); break;
    case 8: launch_rows<DT, 8>(a, stream); break;
    case 16: launch_rows<DT, 16>(a, stream); break;
    case 32: launch_rows<DT, 32>(a, stream); break;
    case 64: launch_rows<DT, 64>(a, stream); break;
    case 128: launch_rows<DT, 128>(a, stream); break;
    case 256: launch_rows<DT, 256>(a, stream); break;
    case 512: launch_rows<DT, 512>(a, stream); break;
    case 1024: launch_rows<DT, 1024>(a, stream); break;
    default: {
      const dim3 block(kNormThreads);
      hipLaunchKernelGGL(norm_back_wide<DT>, dim3((unsigned)(a.m < 65536 ? a.m : 65536)), block, 0, stream, a);
      const unsigned across = (unsigned)((a.n + 8l * kNormThreads - 1) / (8 * kNormThreads));
      if (columns) hipLaunchKernelGGL(norm_columns<DT>, dim3((unsigned)a.chunks.count, across), block, 0, stream, a);
    }
  }
  const hipError_t e = hipGetLastError();
  const long groups = a.dgate && a.chunks.per_group ? a.chunks.count / a.chunks.per_group : 0;
  if (e != hipSuccess || !columns || (a.chunks.count == 1 && !groups)) return e;
  const int across = finish_columns(a.n);
  const dim3 grid((unsigned)((a.n + across - 1l) / across), (unsigned)(kNormSums + groups)), block(kFinishThreads);
  if (across == 32) hipLaunchKernelGGL(norm_finish<32>, grid, block, 0, stream, a);
  else hipLaunchKernelGGL(norm_finish<16>, grid, block, 0, stream, a);
  return hipGetLastError();
}

}  // namespace

// Chunks enough to fill the device once, and few enough that the sums over them stay a
// short pass.  us, both norms, gate and dropout, at 512, 768 and 1024 chunks: 65536 rows of
// 400 fp16 columns 98, 90 and 103 (so 768 up to 512 columns), 16384 bf16 rows of 1024 84, 64 and
// 59 (1024 up to there), of 2048 95, 97 and 96, of 4096 183, 186 and 198 (512 from there on;
// 1032 columns alone would gain by more, 86, 79 and 75).
//
// A gate's groups of more rows than such a chunk are parted only while all their chunks
// fit the device together (1.5 times as many of 128 and 256 lanes), as one that runs after the
// others costs a chunk's whole time, and parts' sums a workgroup for every group and 16
// or 32 columns.  us, in one part and in as many as the rows ask for: 65536 rows of 32 fp16
// columns, groups of 65 24.6 and 29.7; 16384 x 4096, of 33 186 and 295, of 200 in 3 parts and 7
// 203 and 249; 16384 x 600, of 40 in 2 parts and 3 98 and 82; 16384 x 2048, of 48 149 and 135.
// Groups of fewer rows come several to a chunk, as many as it holds: less than twice the
// chunks named.
NormChunks norm_chunks(long m, int n, long gate_rows) {
  NormChunks c{};
  const int lanes = norm_lanes(n);
  const long step = norm_chunk_step(n), target = lanes && lanes <= 64 ? 768 : lanes == 128 ? 1024 : 512,
             together = lanes == 128 || lanes == 256 ? target * 3 / 2 : target;
  long most = (m + target - 1) / target;
  if (most < step) most = step;
  c.group_rows = gate_rows && gate_rows < m ? gate_rows : m;
  const long groups = (m + c.group_rows - 1) / c.group_rows, asked = (c.group_rows + most - 1) / most;
  const long parts = asked * groups <= together ? asked : together / groups;
  if (parts > 1) {
    c.rows = ((c.group_rows + parts - 1) / parts + step - 1) / step * step;
    c.per_group = (c.group_rows + c.rows - 1) / c.rows;
    c.count = groups * c.per_group;
    return c;
  }
  // A group of so few rows leaves most of a workgroup's row lanes without one.  Either row
  // lanes take a group each, whose rows they add one after another (about 7 us and 1.6 for
  // each row), or a workgroup takes one (6 us and one for each 100 groups).  us, lanes and
  // workgroups, 32 fp16 columns: 1 row, 256 groups 8.8 and 9.7; 2 rows, 256 groups 10.3 and 9.6,
  // 512 10.4 and 10.9; 4 rows, 768 groups 13.8 and 13.5, 1024 13.7 and 16.4; 8 rows, 1024 groups
  // 21.7 and 19.1, 1536 22.1 and 23.8; 16 rows, 1024 groups 35.2 and 19.4.  96 columns: 4 rows,
  // 768 groups 15.7 and 14.9, 1024 15.8 and 18.8.
  const bool few_rows = c.group_rows * 4 <= step;
  c.lane_groups = few_rows && groups > 160 * (c.group_rows + 1);
  long held = few_rows && !c.lane_groups ? 1 : most / c.group_rows;
  if (c.lane_groups && held < step) held = step;
  if (held < 1) held = 1;
  c.rows = held * c.group_rows;
  c.count = (m + c.rows - 1) / c.rows;
  return c;
}

hipError_t launch_norm_back(const NormBackArgs& a, int dtype, hipStream_t stream) {
  if (dtype == OIDN_F32) return launch_type<OIDN_F32>(a, stream);
  return dtype == OIDN_F16 ? launch_type<OIDN_F16>(a, stream) : launch_type<OIDN_BF16>(a, stream);
}

}  // namespace oidn
