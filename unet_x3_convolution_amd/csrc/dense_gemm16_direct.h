// 16-bit matrix products whose operands go straight from memory to LDS.
//
// Same products, fragments, LDS layouts and epilogues as dense_gemm16.h, for
// operands whose 16-byte units are aligned and whole (the host checks: 16-byte
// bases and pitches; the summed length of an l-fastest operand and the
// outputs' extent of a strided one multiples of 8).  What changes is how the
// matrix cores are kept fed:
//
//   - Tiles are copied global -> LDS by global_load_lds (no registers, no LDS
//     write instructions); the slot permutation is applied to the address each
//     lane reads from.
//   - The fragments of one half tile (32 of the 64 summed elements) are read
//     while the other half is multiplied, so an MFMA never waits for the LDS
//     read issued just before it:
//       A: read half 1 of tile t;   multiply half 0 of tile t
//       B: wait for the copies of tile t + 1, barrier
//       C: copy tile t + 2 over tile t, read half 0 of tile t + 1;
//          multiply half 1 of tile t
//     After B every wave holds both halves of tile t, so its buffer is free,
//     and a copy has a whole tile's multiplications to arrive.
//   - Within A and C the order is fixed step by step (sched_barrier): two
//     fragment reads or two copies, then four MFMAs.  Reads come first so that
//     they are back before the next phase needs them.
//
// A wave computes TR / 2 x TC / 2.  256 x 256 tiles: 128 x 128 a wave, 256
// accumulator registers, one workgroup per compute unit; a staged tile takes
// 2048 cycles of MFMAs and 1024 of LDS reads.  128 x 128: 512 of MFMAs and 512
// of reads, two workgroups to a unit; 64 x 64: launches that would leave units
// idle otherwise.
//
// Measured (bf16, one MI355X): 8192 x 4096 x 4096 in 205 us (1340 TFLOP/s), a call
// among others 212, through registers 331; 8192^3 at 1351, 1349 and 1324 TFLOP/s in
// the three layouts.  Power bounds it: the same instructions on zeros ran at 1835.  A
// 256 x 256 tile costs 9 us besides its loop and its launch's start, as fitted over sizes.
#pragma once

#include "dense_gemm16.h"
#include "dense_slope.h"

namespace oidn {
namespace {

// 16 bytes per lane to LDS byte address `lds` + 16 * lane from base + off.
// The caller waits (vmcnt) before anything reads it.
__device__ __forceinline__ void copy16(const char* base, unsigned off, unsigned lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(lds), "v"(off),
               "s"(base)
               : "memory");
}
__device__ __forceinline__ void copy16_from(const char* p, unsigned lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(lds), "v"(p)
               : "memory");
}

// c += a b in place.  As an instruction of its own: left to allocate 64 such
// accumulators, the compiler writes each product to other registers and copies
// it back (over 400 copies per tile at 256 x 256).  It knows no latency for it,
// so settle() stands between the last of them and the first read of c.
template <bool BF>
__device__ __forceinline__ void mfma16_acc(floatx4& c, uint4 a, uint4 b) {
  typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
  const u32x4 av = {a.x, a.y, a.z, a.w}, bv = {b.x, b.y, b.z, b.w};
  if constexpr (BF) asm("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(c) : "v"(av), "v"(bv));
  else asm("v_mfma_f32_16x16x32_f16 %0, %1, %2, %0" : "+a"(c) : "v"(av), "v"(bv));
}
// 16 wait states, more than a 4-pass MFMA's result takes to be readable, for
// each four accumulators.
__device__ __forceinline__ void settle(floatx4& a, floatx4& b, floatx4& c, floatx4& d) {
  asm volatile("s_nop 15" : "+a"(a), "+a"(b), "+a"(c), "+a"(d));
}

// Copies of one operand's T x 64 tile by 4 waves.
template <int T, bool STRIDED>
struct Direct16 {
  typedef Stage16<T, STRIDED, 256> S;
  static constexpr int kCopies = S::kBytes / 1024 / 4;    // per wave
  static constexpr int kSlotsPerRow = STRIDED ? T / 8 : 8;

  const char* base;          // the tile's first element
  long step;                 // bytes to the next tile
  unsigned off[kCopies];     // this lane's unit in each copy
  unsigned lds0;             // LDS byte address of the wave's first copy

  // unit u of the tile: its LDS row and the unit of that row it holds
  static __device__ __forceinline__ void place(int u, int& row, int& s) {
    row = u / kSlotsPerRow;
    const int slot = u % kSlotsPerRow;
    if constexpr (!STRIDED) s = slot ^ ((row >> 1) & 7);
    else if constexpr (T >= 128) s = slot ^ ((row & 3) << 2);
    else s = slot ^ ((row & 2) << 1);
  }
  __device__ __forceinline__ static int unit(int k) {
    return ((int)(threadIdx.x >> 6) * kCopies + k) * 64 + (int)(threadIdx.x & 63);
  }
  __device__ __forceinline__ void init(const void* p, long ld, long i0, long rows, long l0, long half,
                                       unsigned lds) {
    base = static_cast<const char*>(p) + 2 * (STRIDED ? l0 * ld + i0 : i0 * ld + l0);
    step = 2 * (STRIDED ? kDenseK * ld : kDenseK);
    lds0 = __builtin_amdgcn_readfirstlane(lds + (threadIdx.x >> 6) * kCopies * 1024);
#pragma unroll
    for (int k = 0; k < kCopies; ++k) {
      int row, s;
      place(unit(k), row, s);
      if constexpr (!STRIDED) {
        int r = half ? row & (T / 2 - 1) : row;
        const long last = rows - 1 - i0;
        const long i = (r < last ? r : last) + (half && row >= T / 2 ? half : 0);
        off[k] = (unsigned)(2 * (i * ld + 8 * s));
      } else {
        const long last = rows - 8 - i0;
        off[k] = (unsigned)(2 * (row * ld + (8 * s < last ? 8 * s : last)));
      }
    }
  }
  // One copy of the next tile, into buffer offset `buf`.
  __device__ __forceinline__ void copy(int k, unsigned buf) const {
    copy16(base, off[k], lds0 + buf + k * 1024);
  }
  __device__ __forceinline__ void advance() { base += step; }
  // The same for a tile of which only `left` (< 64) summed elements exist:
  // units past them come from a block of zeros.
  __device__ __forceinline__ void copy_tail(long left, unsigned buf) const {
#pragma unroll
    for (int k = 0; k < kCopies; ++k) {
      int row, s;
      place(unit(k), row, s);
      const bool in = (STRIDED ? row : 8 * s) < left;
      copy16_from(in ? base + off[k] : reinterpret_cast<const char*>(g_zero16), lds0 + buf + k * 1024);
    }
  }
};

// Workgroup `block` of the product; lds: gemm16_lds<TR, TC>() bytes, two
// buffers of a P and a Q tile.
template <bool BF, int LAYOUT, int EPI, int TR, int TC, Caching WHERE>
__device__ __forceinline__ void gemm16_direct(const GemmArgs& a, int block, char* lds) {
  constexpr int DT = BF ? OIDN_BF16 : OIDN_F16;
  constexpr bool PS = LAYOUT != kForward, QS = LAYOUT == kWeightGrad;
  constexpr int FR = TR / 32, FC = TC / 32;
  static_assert(EPI != kEpiGated || FC % 4 == 0, "a wave holds pairs of both projections");
  typedef Direct16<TC, PS> PD;
  typedef Direct16<TR, QS> QD;
  typedef typename PD::S P;
  typedef typename QD::S Q;
  constexpr unsigned kBuf = P::kBytes + Q::kBytes;

  int tc, tr;
  int slice;
  if (!tile_and_slice(a, block, tc, tr, slice)) return;
  const long i0 = (long)tr * TR;
  constexpr int C = EPI == kEpiGated ? TC / 2 : TC;
  const long j0 = (long)tc * C;
  const long half = EPI == kEpiGated ? a.e.cols : 0;
  const int wave = threadIdx.x >> 6, wr = wave >> 1, wc = wave & 1;
  const long t0 = (long)slice * a.per_split;
  const long nt = (a.len + kDenseK - 1) / kDenseK;
  const long t1 = t0 + a.per_split < nt ? t0 + a.per_split : nt;
  const long whole = a.len / kDenseK < t1 ? a.len / kDenseK : t1;   // tiles before it are complete

  const unsigned lds_at = (unsigned)(unsigned long)(__attribute__((address_space(3))) void*)lds;
  PD p;
  QD q;
  p.init(a.p, a.ldp, j0, a.e.cols, t0 * kDenseK, half, lds_at);
  q.init(a.q, a.ldq, i0, a.e.rows, t0 * kDenseK, 0, lds_at + P::kBytes);

  floatx4 acc[FC][FR];
#pragma unroll
  for (int c = 0; c < FC; ++c)
#pragma unroll
    for (int r = 0; r < FR; ++r) acc[c][r] = floatx4{0.f, 0.f, 0.f, 0.f};

  uint4 fp[2][FC], fq[2][FR];            // [half][fragment]
  auto read = [&](int n, int kk, unsigned buf) {
    const char* const l = lds + buf;
    if (n < FC) {
      const int pair = n / 2;
      const int base = EPI == kEpiGated
                           ? (pair < FC / 4 ? wc * (TC / 4) + 32 * pair
                                            : TC / 2 + wc * (TC / 4) + 32 * (pair - FC / 4))
                           : wc * (TC / 2) + 32 * pair;
      fp[kk][n] = P::template fragment<true>(l, base, n & 1, kk);
    } else {
      fq[kk][n - FC] = Q::template fragment<false>(l + P::kBytes, wr * (TR / 2), n - FC, kk);
    }
  };
  constexpr int kReads = FC + FR, kCopies = PD::kCopies + QD::kCopies, kSteps = FC * FR / 4;
  auto copy = [&](int n, unsigned buf) {
    if (n < PD::kCopies) p.copy(n, buf);
    else q.copy(n - PD::kCopies, buf);
  };
  auto stage = [&](long t, unsigned buf) {       // tile t < t1, not in step with MFMAs
    if (t < whole) {
#pragma unroll
      for (int n = 0; n < kCopies; ++n) copy(n, buf);
    } else {
      p.copy_tail(a.len - t * kDenseK, buf);
      q.copy_tail(a.len - t * kDenseK, buf);
    }
    p.advance();
    q.advance();
  };
  auto multiply4 = [&](int s, int kk) {
#pragma unroll
    for (int n = 4 * s; n < 4 * s + 4; ++n)
      mfma16_acc<BF>(acc[n / FR][n % FR], fp[kk][n / FR], fq[kk][n % FR]);
  };
  constexpr int kPer = kReads > 2 * kSteps ? (kReads + kSteps - 1) / kSteps : 2;   // reads per step
  auto wait_all = [&] {
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
  };

  stage(t0, 0);
  if (t0 + 1 < t1) stage(t0 + 1, kBuf);
  wait_all();
#pragma unroll
  for (int n = 0; n < kReads; ++n) read(n, 0, 0);
  unsigned cur = 0;
  long t = t0;
  for (; t + 2 < whole; ++t) {
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
#pragma unroll
      for (int n = s * kPer; n < (s + 1) * kPer && n < kReads; ++n) read(n, 1, cur);
      multiply4(s, 0);
      __builtin_amdgcn_sched_barrier(0);
    }
    wait_all();
    const unsigned next = kBuf - cur;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
#pragma unroll
      for (int n = s * kPer; n < (s + 1) * kPer && n < kReads; ++n) read(n, 0, next);
      constexpr int kc = (kCopies + kSteps - 1) / kSteps;
#pragma unroll
      for (int n = s * kc; n < (s + 1) * kc && n < kCopies; ++n) copy(n, cur);
      multiply4(s, 1);
      __builtin_amdgcn_sched_barrier(0);
    }
    p.advance();
    q.advance();
    cur = next;
  }
  // the last tiles: the same phases, copies where there is a tile to copy
  for (; t < t1; ++t) {
#pragma unroll
    for (int n = 0; n < kReads; ++n) read(n, 1, cur);
#pragma unroll
    for (int s = 0; s < kSteps; ++s) multiply4(s, 0);
    wait_all();
    const unsigned next = kBuf - cur;
    if (t + 2 < t1) stage(t + 2, cur);
    if (t + 1 < t1) {
#pragma unroll
      for (int n = 0; n < kReads; ++n) read(n, 0, next);
    }
#pragma unroll
    for (int s = 0; s < kSteps; ++s) multiply4(s, 1);
    cur = next;
  }

#pragma unroll
  for (int s = 0; s < kSteps; ++s) {
    const int n = 4 * s;
    settle(acc[n / FR][n % FR], acc[(n + 1) / FR][(n + 1) % FR], acc[(n + 2) / FR][(n + 2) % FR],
           acc[(n + 3) / FR][(n + 3) % FR]);
  }
  __syncthreads();                       // every wave has read its last fragments
  tile_epilogue<DT, EPI, FR, FC, false, WHERE>(a.e, acc, lds + wave * epilogue_bytes<FR, FC>(), i0 + wr * (TR / 2),
                                 (int)j0 + wc * (C / 2), a.splits > 1 ? slice : -1, (long)tr * 2 + wr);
}

// The kernels.  DIRECT: operands go straight to LDS, else through registers.
template <bool BF, int LAYOUT, int EPI, int TR, int TC, bool DIRECT, Caching WHERE = kKept>
__device__ __forceinline__ void gemm16(const GemmArgs& a, int block, char* lds) {
  if constexpr (DIRECT) gemm16_direct<BF, LAYOUT, EPI, TR, TC, WHERE>(a, block, lds);
  else gemm16_staged<BF, LAYOUT, EPI, TR, TC, WHERE>(a, block, lds);
}
constexpr int workgroups_per_cu(int tr, int tc) { return tr * tc >= 256 * 256 ? 1 : 2; }

template <bool BF, int LAYOUT, int EPI, int TR, int TC, bool DIRECT, Caching WHERE>
__global__ __launch_bounds__(256, workgroups_per_cu(TR, TC)) void dense_gemm16(GemmArgs a) {
  __shared__ __attribute__((aligned(1024))) char lds[gemm16_lds<TR, TC>()];
  gemm16<BF, LAYOUT, EPI, TR, TC, DIRECT, WHERE>(a, blockIdx.x, lds);
}

// The gated block's dh with its epilogue; the first workgroups read a
// checkpoint back for the products that follow.
template <bool BF, int T, bool DIRECT>
__global__ __launch_bounds__(256, workgroups_per_cu(T, T)) void dense_gemm16_gated_back(GemmArgs a, UnpackJob u) {
  __shared__ __attribute__((aligned(1024))) char lds[gemm16_lds<T, T>()];
  if ((int)blockIdx.x < u.blocks) return unpack_rows<BF ? OIDN_BF16 : OIDN_F16>(u, blockIdx.x);
  gemm16<BF, kInputGrad, kEpiGatedBack, T, T, DIRECT>(a, blockIdx.x - u.blocks, lds);
}

// Several gradients' products in one launch: they fill the device together,
// and the last tiles of one run beside the first of the next.
template <bool BF, int T, bool DIRECT>
__global__ __launch_bounds__(256, workgroups_per_cu(T, T)) void dense_gemm16_group(GemmGroup g) {
  __shared__ __attribute__((aligned(1024))) char lds[gemm16_lds<T, T>()];
  if ((int)blockIdx.x >= g.sums_start)
    return slope_rows<BF ? OIDN_BF16 : OIDN_F16>(g.sums, blockIdx.x - g.sums_start, reinterpret_cast<float*>(lds));
  int k = 0;
  while (k + 1 < g.count && (int)blockIdx.x >= g.start[k + 1]) ++k;
  const int block = blockIdx.x - g.start[k];
  if (g.layout[k] == kInputGrad) gemm16<BF, kInputGrad, kEpiStore, T, T, DIRECT, kEither>(g.a[k], block, lds);
  else gemm16<BF, kWeightGrad, kEpiStore, T, T, DIRECT, kEither>(g.a[k], block, lds);
}

}  // namespace
}  // namespace oidn
