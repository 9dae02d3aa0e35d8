// Forward products of layers with at most 128 inputs: the rows are coded on the way to
// LDS, so that the layer is one launch.
//
// All of the summed length is one block: a workgroup copies a tile of weight codes to
// LDS, codes its rows beside them (a thread eight values, 16 lanes a row), multiplies
// once and runs the epilogue.  Every column tile codes its rows again, which costs less
// than the launch that would code them once: 8160 x 96 -> 384 fp16, gelu, z kept:
// 9.0 us, in two launches 11.5.  What it reads and writes (14 MB) would take 2.7: the rest is
// the launch, one chain of loads, coding and epilogue, and the activation.  A 16-bit layer of
// so few inputs is faster still, having nothing to code (7.3 to 8.5; 130560 x 32 -> 128 25 for 29).
#include "fp8_code.h"
#include "fp8_gemm.h"
#include "lanes.h"

namespace oidn {
namespace {

template <bool BF, int T, Caching WHERE>
__global__ __launch_bounds__(256, 2) void dense_narrow8(Gemm8Args a8, int k) {
  const GemmArgs& a = a8.g;
  constexpr int DT = BF ? OIDN_BF16 : OIDN_F16;
  constexpr int F = T / 32;
  typedef Direct16<T, false> D;
  typedef typename D::S S;
  constexpr int kTiles = 2 * S::kBytes + 2 * T, kEpilogue = 4 * epilogue_bytes<F, F>();
  __shared__ __attribute__((aligned(1024))) char lds[kTiles > kEpilogue ? kTiles : kEpilogue];
  char* const q_lds = lds + S::kBytes;
  unsigned char* const scales = reinterpret_cast<unsigned char*>(lds + 2 * S::kBytes);     // of P's rows, then Q's

  int tc, tr, slice;
  if (!tile_and_slice(a, blockIdx.x, tc, tr, slice)) return;
  const long i0 = (long)tr * T, j0 = (long)tc * T;
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6, wr = wave >> 1, wc = wave & 1, r = lane & 15;

  // rows in flight first, then the weights' copies
  constexpr int kRows = T / 16;                  // of a thread
  const int c = t & 15, left = k - 8 * c;        // its columns 8 c .. + 7
  Raw<DT> raw[kRows];
#pragma unroll
  for (int n = 0; n < kRows; ++n) {
    const long i = i0 + 16 * n + (t >> 4), at = i < a.e.rows ? i : a.e.rows - 1;
    const int j = left > 0 ? 8 * c : 0;
    raw[n] = load_raw<DT>(a.q, at * a.ldq + j, k - j, (a.e.rows - 1 - at) * a.ldq + k - j);
  }
  const unsigned lds_at = (unsigned)(unsigned long)(__attribute__((address_space(3))) void*)lds;
  D p;
  p.init(a.p, a.ldp, j0, a.e.cols, 0, 0, lds_at);
#pragma unroll
  for (int n = 0; n < D::kCopies; ++n) p.copy(n, 0);
  if (t < T) {
    const long j = j0 + t;
    scales[t] = a8.ps[(j < a.e.cols ? j : a.e.cols - 1) * a8.pn];
  }
#pragma unroll
  for (int n = 0; n < kRows; ++n) {
    Eight v = raw[n].value();
    clear_tail(left, v);
    const int e = fp8_power(lanes_max<16>(finite_top(v))), row = 16 * n + (t >> 4);
    *reinterpret_cast<uint2*>(q_lds + 16 * S::slot(row, c >> 1) + 8 * (c & 1)) = fp8_codes(v.v, power_of_two(-e));
    if (c == 0) scales[T + row] = (unsigned char)(e + 127);
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();

  intx8 fp[F], fq[F];
  unsigned up[F], uq[F];
  auto both = [](uint4 lo, uint4 hi) {
    return intx8{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
  };
#pragma unroll
  for (int f = 0; f < F; ++f) {
    const int base = wc * (T / 2) + 32 * (f / 2), i = wr * (T / 2) + 16 * f + r;
    fp[f] = both(S::template fragment<true>(lds, base, f & 1, 0), S::template fragment<true>(lds, base, f & 1, 1));
    fq[f] = both(S::template fragment<false>(q_lds, wr * (T / 2), f, 0), S::template fragment<false>(q_lds, wr * (T / 2), f, 1));
    up[f] = scales[base + 8 * (r >> 2) + 4 * (f & 1) + (r & 3)];
    uq[f] = scales[T + i];
  }
  floatx4 acc[F][F];
#pragma unroll
  for (int x = 0; x < F; ++x)
#pragma unroll
    for (int y = 0; y < F; ++y) acc[x][y] = floatx4{0.f, 0.f, 0.f, 0.f};
  // between the zeros' writes and the instructions that read them
  asm volatile("s_nop 3");
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int x = 0; x < F; ++x)
#pragma unroll
    for (int y = 0; y < F; ++y) mfma8_acc<0>(acc[x][y], fp[x], fq[y], up[x], uq[y]);
#pragma unroll
  for (int x = 0; x < F; x += 2)
#pragma unroll
    for (int y = 0; y < F; y += 2) settle(acc[x][y], acc[x][y + 1], acc[x + 1][y], acc[x + 1][y + 1]);
  __syncthreads();                       // every wave has read its fragments
  tile_epilogue<DT, kEpiLinear, F, F, false, WHERE>(a.e, acc, lds + wave * epilogue_bytes<F, F>(), i0 + wr * (T / 2),
                                                    (int)j0 + wc * (T / 2), -1, (long)tr * 2 + wr);
}

template <bool BF, int T>
void launch(const Gemm8Args& a, int k, hipStream_t stream) {
  const dim3 grid((unsigned)gemm_blocks(a.g)), block(256);
  if (a.g.e.stream) hipLaunchKernelGGL((dense_narrow8<BF, T, kStreamed>), grid, block, 0, stream, a, k);
  else hipLaunchKernelGGL((dense_narrow8<BF, T, kKept>), grid, block, 0, stream, a, k);
}

}  // namespace

hipError_t launch_narrow8(const Gemm8Args& a, int k, int tile, bool bf16, hipStream_t stream) {
  if (k > kFp8Block) return hipErrorInvalidValue;
  if (tile == 128) {
    if (bf16) launch<true, 128>(a, k, stream);
    else launch<false, 128>(a, k, stream);
  } else {
    if (bf16) launch<true, 64>(a, k, stream);
    else launch<false, 64>(a, k, stream);
  }
  return hipGetLastError();
}

}  // namespace oidn
