// Products of packed matrices on the matrix cores, C[i][j] = sum_l Q(i, l) P(j, l).
//
// v_mfma_scale_f32_16x16x128_f8f6f4 multiplies 128 codes of 16 rows by 16 and
// takes the exponent of each row's block of 128 as an operand, so blocks need no
// work of their own.  A row of 128 codes has the bytes of 64 16-bit elements: tiles,
// their copies to LDS, slots and epilogues are those of the 16-bit products
// (dense_gemm16_direct.h), and a fragment is both 16-byte halves of a row that a lane
// reads (the order of the sum is permuted alike in both operands).
//
// The instruction adds eight products with the last bit at 2^-13 of the largest
// one's power of two, what is beyond cut off (less than 7 2^-13 of the largest product, as it
// needs no cut itself), and sums of eight in fp32: 1.5e-5 of the result at normal data,
// 3.6e-5 where channels differ e-fold (measured over 4096 summed elements), a tenth and
// less of a 16-bit result's rounding.  Where the large products of an eight cancel, what is
// cut may be all of the rest.  The 8-bit instructions without scales do the same; codes
// widened to 16 bits would be added in fp32, at half the rate.
#pragma once

#include "dense_columns.h"
#include "dense_gemm16_direct.h"
#include "fp8.h"

namespace oidn {
namespace {

typedef int intx8 __attribute__((ext_vector_type(8)));

// c += a b in place, scales in byte BYTE of sa and sb.  As an instruction of its own:
// the builtin's result may be given the registers of an operand (seen with the
// scale's, and wrong sums with it).  The compiler knows neither what it reads nor when
// its result is there.  WAITS false: operands come from loads, the same c follows 4
// such instructions later or more, and dense_gemm16_direct.h's settle() stands before
// its first read.  WAITS true: after vector instructions that wrote an operand, and
// before the next product into the same c (12 wait states cover its 8 passes; without
// them sums were wrong).
template <int BYTE, bool WAITS = false>
__device__ __forceinline__ void mfma8_acc(floatx4& c, const intx8& a, const intx8& b, unsigned sa, unsigned sb) {
#define OIDN_MFMA8(before, sel, after)                                                                      \
  asm(before "v_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, %0, %3, %4 " sel after                          \
      : "+a"(c) : "v"(a), "v"(b), "v"(sa), "v"(sb))
#define OIDN_MFMA8_BYTE(sel)                                                 \
  do {                                                                       \
    if constexpr (WAITS) OIDN_MFMA8("s_nop 1\n\t", sel, "\n\ts_nop 11");    \
    else OIDN_MFMA8("", sel, "");                                            \
  } while (0)
  if constexpr (BYTE == 0) OIDN_MFMA8_BYTE("op_sel:[0,0,0] op_sel_hi:[0,0,0]");
  else if constexpr (BYTE == 1) OIDN_MFMA8_BYTE("op_sel:[1,1,0] op_sel_hi:[0,0,0]");
  else if constexpr (BYTE == 2) OIDN_MFMA8_BYTE("op_sel:[0,0,0] op_sel_hi:[1,1,0]");
  else OIDN_MFMA8_BYTE("op_sel:[1,1,0] op_sel_hi:[1,1,0]");
#undef OIDN_MFMA8_BYTE
#undef OIDN_MFMA8
}

// LDS: two buffers of a P tile, two of a Q tile, then two of the rows' scales, a word
// of each for four staged tiles.  (In this order a fragment's place in either buffer
// is an immediate offset of one address.)
template <int T>
constexpr int gemm8_lds() { return 4 * T * kFp8Block + 2 * 2 * T * 4; }

// 4 bytes per lane to LDS byte address `lds` + 4 * lane from base + off; as copy16.
__device__ __forceinline__ void copy4(const void* base, unsigned off, unsigned lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, %2" ::"s"(lds), "v"(off), "s"(base)
               : "memory");
}

// Workgroup `block` of the product; lds: gemm8_lds<T>() bytes.  Slices begin at
// multiples of four staged tiles.
//
// A wave's F x F fragments are multiplied in four quarters, P's halves by Q's, such
// that what a quarter needs is read from LDS a quarter earlier and only F + F
// fragments' registers are held:
//   A  P0 Q0   reads Q1 and P1; then a wait for the copies of tile t + 1 and a barrier:
//              all of tile t is in registers
//   B  P0 Q1   copies of tile t + 2 over tile t
//   C  P1 Q1   reads P0 of tile t + 1
//   D  P1 Q0   reads Q0 of tile t + 1 in Q1's place
// (every fourth tile C and D read the next word of scales too)
// so that Q's halves change places from tile to tile, and a copy has a whole tile's
// multiplications to arrive.  Within a quarter the order is fixed (sched_barrier): a
// read or a copy, then a multiplication, under whose 32 cycles the next one issues.
//
// Bound by the matrix cores (64% of the cycles busy, at the clock that random data leaves):
// bf16, by card and pace 8192 cubed 2430 to 2690 TFLOP/s (a library product with one scale a
// matrix 3200 beside the last), 8192 x 4096 -> 4096 112 to 127 us (94 to 108); gelu adds 18 us to
// that, a residual 10, both 25, as 256 x 256 tiles leave one wave a SIMD and the epilogue stands
// alone.  All of a tile's fragments held in registers spilled (1030 us against 186 for the
// layer with both and packing); reads and copies grouped instead of spread reached 2440
// TFLOP/s where these reached 2520.
template <bool BF, int EPI, int T, Caching WHERE>
__device__ __forceinline__ void gemm8(const Gemm8Args& a8, int block, char* lds) {
  const GemmArgs& a = a8.g;
  constexpr int DT = BF ? OIDN_BF16 : OIDN_F16;
  constexpr int F = T / 32, H = F / 2;           // 16-wide fragments per wave each way, half of them
  typedef Direct16<T, false> D;
  typedef typename D::S S;
  constexpr unsigned kBuf = S::kBytes;           // from one buffer of an operand to the other
  constexpr unsigned kScales = 4 * S::kBytes, kScaleBuf = 2 * T * 4;

  int tc, tr, slice;
  if (!tile_and_slice(a, block, tc, tr, slice)) return;
  const long i0 = (long)tr * T, j0 = (long)tc * T;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, wr = wave >> 1, wc = wave & 1, r = lane & 15;
  const long t0 = (long)slice * a.per_split, nt = a.len / kDenseK;
  const long t1 = t0 + a.per_split < nt ? t0 + a.per_split : nt;

  const unsigned lds_at = (unsigned)(unsigned long)(__attribute__((address_space(3))) void*)lds;
  D p, q;
  p.init(a.p, a.ldp, j0, a.e.cols, t0 * kDenseK, 0, lds_at);
  q.init(a.q, a.ldq, i0, a.e.rows, t0 * kDenseK, 0, lds_at + 2 * S::kBytes);

  // The scales' copies: 64 rows of an operand each, shared by the waves.
  constexpr int kScaleCopies = 2 * T / 64, kScaleTurns = (kScaleCopies + 3) / 4;
  unsigned scale_off[kScaleTurns];
#pragma unroll
  for (int k = 0; k < kScaleTurns; ++k) {
    const int c = wave + 4 * k, row = 64 * (c % (T / 64)) + lane;
    const bool of_p = c < T / 64;
    const long last = of_p ? a.e.cols - 1 - j0 : a.e.rows - 1 - i0;
    scale_off[k] = (unsigned)((row < last ? row : last) * (of_p ? a8.pn : a8.qn));
  }
  const unsigned char* const ps = a8.ps + j0 * a8.pn;
  const unsigned char* const qs = a8.qs + i0 * a8.qn;
  // the word of tiles t .. t + 3 (t a multiple of 4)
  auto copy_scales = [&](long t, unsigned buf) {
#pragma unroll
    for (int k = 0; k < kScaleTurns; ++k) {
      const int c = __builtin_amdgcn_readfirstlane(wave + 4 * k);
      if (c < kScaleCopies) copy4((c < T / 64 ? ps : qs) + t, scale_off[k], lds_at + kScales + buf + 256 * c);
    }
  };
  unsigned up[F], uq[F];
  auto read_up = [&](int f, unsigned buf) {
    up[f] = *reinterpret_cast<const unsigned*>(lds + kScales + buf + 4 * (wc * (T / 2) + 32 * (f / 2) + 8 * (r >> 2) +
                                                                       4 * (f & 1) + (r & 3)));
  };
  auto read_uq = [&](int f, unsigned buf) {
    uq[f] = *reinterpret_cast<const unsigned*>(lds + kScales + buf + 4 * T + 4 * (wr * (T / 2) + 16 * f + r));
  };

  floatx4 acc[F][F];
#pragma unroll
  for (int c = 0; c < F; ++c)
#pragma unroll
    for (int k = 0; k < F; ++k) acc[c][k] = floatx4{0.f, 0.f, 0.f, 0.f};

  intx8 fp[F], fq[F];
  // half h of a fragment: 16 bytes a lane
  auto put = [](intx8& f, int h, uint4 v) {
    f[4 * h] = (int)v.x, f[4 * h + 1] = (int)v.y, f[4 * h + 2] = (int)v.z, f[4 * h + 3] = (int)v.w;
  };
  auto read_p = [&](int c, int h, unsigned buf) {
    put(fp[c], h, S::template fragment<true>(lds + buf, wc * (T / 2) + 32 * (c / 2), c & 1, h));
  };
  auto read_q = [&](int place, int k, int h, unsigned buf) {
    put(fq[place], h, S::template fragment<false>(lds + buf + 2 * S::kBytes, wr * (T / 2), k, h));
  };
  auto wait_all = [&] {
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
  };
  // Tile t of a word's four: its scales are in byte `byte`, Q's first half in
  // fq[byte % 2 * H ..].  full: tiles t + 1 and t + 2 exist; cur, scales: their buffers.
  auto tile = [&](auto byte, auto full, long t, unsigned cur, unsigned scales) {
    constexpr int kByte = decltype(byte)::value, X = kByte % 2 * H, Y = H - X;
    constexpr bool kFull = decltype(full)::value;
    const bool one_more = kFull || t + 1 < t1, two_more = kFull || t + 2 < t1;
    const unsigned next = kBuf - cur;
    // A quarter's H x H multiplications, P's half from c0 on by Q's at `place`, and one
    // other instruction before each: op(0) .. op(H * H - 1).
    auto quarter = [&](int c0, int place, int k0, auto op) {
#pragma unroll
      for (int n = 0; n < H * H; ++n) {
        op(n);
        mfma8_acc<kByte>(acc[c0 + n / H][k0 + n % H], fp[c0 + n / H], fq[place + n % H], up[c0 + n / H], uq[k0 + n % H]);
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    // spread(n, count, f): f of the step-n share of `count` things
    auto spread = [](int n, int count, auto f) {
#pragma unroll
      for (int i = n * count / (H * H); i < (n + 1) * count / (H * H); ++i) f(i);
    };
    __builtin_amdgcn_sched_barrier(0);
    quarter(0, X, 0, [&](int n) {
      spread(n, 4 * H, [&](int i) {
        if (i < 2 * H) read_q(Y + i / 2, H + i / 2, i % 2, cur);
        else read_p(i / 2, i % 2, cur);
      });
    });
    wait_all();
    if constexpr (kByte == 0) {
      // read three tiles on; what it overwrites was read at the end of the last word
      if (t + 4 < t1) copy_scales(t + 4, kScaleBuf - scales);
    }
    quarter(0, Y, H, [&](int n) {
      if (two_more)
        spread(n, 2 * D::kCopies, [&](int i) {
          if (i % 2 == 0) p.copy(i / 2, cur);
          else q.copy(i / 2, cur);
        });
    });
    quarter(H, Y, H, [&](int n) {
      if (one_more) {
        spread(n, 2 * H, [&](int i) { read_p(i / 2, i % 2, next); });
        if constexpr (kByte == 3) spread(n, H, [&](int i) { read_up(i, kScaleBuf - scales); });
      }
    });
    quarter(H, X, 0, [&](int n) {
      if (one_more) {
        spread(n, 2 * H, [&](int i) { read_q(Y + i / 2, i / 2, i % 2, next); });
        if constexpr (kByte == 3) spread(n, H, [&](int i) { read_uq(H + i, kScaleBuf - scales); });
      }
    });
    p.advance();
    q.advance();
    if constexpr (kByte == 3) {
      // their old values were in use until here
#pragma unroll
      for (int f = 0; f < H; ++f) {
        read_up(H + f, kScaleBuf - scales);
        read_uq(f, kScaleBuf - scales);
      }
    }
  };
  auto stage = [&](unsigned buf) {
#pragma unroll
    for (int n = 0; n < D::kCopies; ++n) {
      p.copy(n, buf);
      q.copy(n, buf);
    }
    p.advance();
    q.advance();
  };

  copy_scales(t0, 0);
  stage(0);
  if (t0 + 1 < t1) stage(kBuf);
  wait_all();
#pragma unroll
  for (int f = 0; f < F; ++f) {
    read_up(f, 0);
    read_uq(f, 0);
  }
#pragma unroll
  for (int f = 0; f < H; ++f) {
    read_p(f, 0, 0);
    read_p(f, 1, 0);
    read_q(f, f, 0, 0);
    read_q(f, f, 1, 0);
  }
  constexpr std::integral_constant<int, 0> kB0{};
  constexpr std::integral_constant<int, 1> kB1{};
  constexpr std::integral_constant<int, 2> kB2{};
  constexpr std::integral_constant<int, 3> kB3{};
  long t = t0;
  unsigned scales = 0;
  for (; t + 5 < t1; t += 4) {
    tile(kB0, std::true_type{}, t, 0, scales);
    tile(kB1, std::true_type{}, t + 1, kBuf, scales);
    tile(kB2, std::true_type{}, t + 2, 0, scales);
    tile(kB3, std::true_type{}, t + 3, kBuf, scales);
    scales = kScaleBuf - scales;
  }
  for (; t < t1; t += 4) {
    tile(kB0, std::false_type{}, t, 0, scales);
    if (t + 1 < t1) tile(kB1, std::false_type{}, t + 1, kBuf, scales);
    if (t + 2 < t1) tile(kB2, std::false_type{}, t + 2, 0, scales);
    if (t + 3 < t1) tile(kB3, std::false_type{}, t + 3, kBuf, scales);
    scales = kScaleBuf - scales;
  }
#pragma unroll
  for (int c = 0; c < F; c += 2)
#pragma unroll
    for (int k = 0; k < F; k += 2) settle(acc[c][k], acc[c][k + 1], acc[c + 1][k], acc[c + 1][k + 1]);
  __syncthreads();                       // every wave has read its last fragments
  tile_epilogue<DT, EPI, F, F, false, WHERE>(a.e, acc, lds + wave * epilogue_bytes<F, F>(), i0 + wr * (T / 2),
                                             (int)j0 + wc * (T / 2), a.splits > 1 ? slice : -1, (long)tr * 2 + wr);
}

template <bool BF, int T, Caching WHERE>
__global__ __launch_bounds__(256, workgroups_per_cu(T, T)) void dense_gemm8(Gemm8Args a) {
  __shared__ __attribute__((aligned(1024))) char lds[gemm8_lds<T>()];
  gemm8<BF, kEpiLinear, T, WHERE>(a, blockIdx.x, lds);
}
// Products that do not depend on each other, and column sums of the pass before them.
template <bool BF, int T>
__global__ __launch_bounds__(256, workgroups_per_cu(T, T)) void dense_gemm8_group(Gemm8Group g) {
  __shared__ __attribute__((aligned(1024))) char lds[gemm8_lds<T>()];
  if ((int)blockIdx.x >= g.columns) {
    const ColumnJob& c = g.column;
    sum_columns(c.part, c.groups, c.cols, c.out, blockIdx.x - g.columns, column_lanes(c.groups), lds);
    return;
  }
  const int k = g.count > 1 && (int)blockIdx.x >= g.start[1] ? 1 : 0;
  gemm8<BF, kEpiStore, T, kEither>(g.a[k], blockIdx.x - g.start[k], lds);
}

}  // namespace
}  // namespace oidn
