// Rows that a workgroup holds in registers: each element is read once.
//
//   b = drop((o - mean) r weight + shift),  u = scale x + gate b,
//   v = (u - mean') r' next_weight + next_shift
//
// with mean 0 in the RMS norm, r = (mean of squares + eps)^-1/2.  Elements, statistics and
// sums are fp32 in registers.  u is rounded once to the matrices' type, and the next norm is
// that of the rounded u, which is what a call of its own would read.  The layer norm's
// squares are of deviations from the mean, formed in a second round over the registers:
// the mean of squares less the mean's square would lose it where the mean is large.
//
// LANES lanes take a row, a lane eight columns.  Up to 64 lanes lie in a wave, which takes
// 64 / LANES rows at once and exchanges sums in registers; more are a workgroup's waves,
// which exchange them through LDS.  The next row's loads are in flight while one is worked
// on.  Bound by memory where rows are many: 16384 x 4096 bf16, both norms, gate and dropout
// (537 MB) 104 us, 5.2 TB/s, which is a large copy's rate; 98.9 without dropout and gate; a
// workgroup that goes over each row again (norm_wide.h) took 218.  Few rows are bound by
// latency: one row of 4096 2.6 us, 130560 x 32 fp16 (17 MB) 5.2.
#pragma once

#include "lanes.h"
#include "norm_rows.h"

namespace oidn {
namespace {

template <int LANES>
constexpr int norm_threads() { return LANES > 64 ? LANES : 256; }

// Sums of a pair over a row's lanes.  `turn` alternates the LDS that waves meet in, so
// that one barrier is enough.
template <int LANES>
struct RowSum {
  static constexpr int kWaves = LANES > 64 ? LANES / 64 : 1;
  float2 (*const lds)[kWaves];       // [2][waves]
  int turn;
  __device__ __forceinline__ explicit RowSum(float2 (*at)[kWaves]) : lds(at), turn(0) {}
  __device__ __forceinline__ float2 operator()(float x, float y) {
    constexpr int kIn = LANES > 64 ? 64 : LANES;
    x = lanes_sum<kIn>(x);
    y = lanes_sum<kIn>(y);
    if constexpr (LANES > 64) {
      float2* const at = lds[turn];
      turn ^= 1;
      if ((threadIdx.x & 63) == 0) at[threadIdx.x >> 6] = {x, y};
      __syncthreads();
      x = y = 0.f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        x += at[w].x;
        y += at[w].y;
      }
    }
    return {x, y};
  }
};

// The statistics of two rows at once (or of one: kind OIDN_NORM_NONE), so that they share
// their rounds of sums; a lane's columns past its `left` do not count.
template <int LANES, bool WHOLE>
__device__ __forceinline__ void row_stats(int kind_x, const Eight& x, Stat& sx, int kind_y, const Eight& y, Stat& sy,
                                          int left, float each, float eps, RowSum<LANES>& sum) {
  sx = sy = {0.f, 1.f};
  const bool layer_x = kind_x == OIDN_NORM_LAYER, layer_y = kind_y == OIDN_NORM_LAYER;
  if (layer_x || layer_y) {
    float t = 0.f, u = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (layer_x) t += x.v[e];
      if (layer_y) u += y.v[e];
    }
    const float2 both = sum(t, u);
    sx.mean = both.x * each;
    sy.mean = both.y * each;
  }
  if (kind_x == OIDN_NORM_NONE && kind_y == OIDN_NORM_NONE) return;
  float t = 0.f, u = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float d = x.v[e] - sx.mean, f = y.v[e] - sy.mean;
    if (WHOLE || e < left) {
      if (kind_x != OIDN_NORM_NONE) t += d * d;
      if (kind_y != OIDN_NORM_NONE) u += f * f;
    }
  }
  if (WHOLE && left <= 0) t = u = 0.f;
  const float2 both = sum(t, u);
  if (kind_x != OIDN_NORM_NONE) sx.r = rsqrtf(both.x * each + eps);
  if (kind_y != OIDN_NORM_NONE) sy.r = rsqrtf(both.y * each + eps);
}
template <int LANES, bool WHOLE>
__device__ __forceinline__ Stat row_stat(int kind, const Eight& x, int left, float each, float eps, RowSum<LANES>& sum) {
  Stat s, none;
  row_stats<LANES, WHOLE>(kind, x, s, OIDN_NORM_NONE, x, none, left, each, eps, sum);
  return s;
}

// A lane's eight columns: their first, and how many exist (WHOLE: eight or none).
// Loads are made whether they or the row exist or not, from others in their place.
template <int DT, bool WHOLE>
struct Unit {
  Raw<DT> raw;
  __device__ __forceinline__ void load(const void* p, long ld, long i, int j, long m, int n) {
    const long at = i < m ? i : m - 1;
    const int c = j < n ? j : 0;
    if constexpr (WHOLE) __builtin_memcpy(&raw.e, static_cast<const typename Raw<DT>::T*>(p) + at * ld + c, sizeof(raw.e));
    else raw = load_raw<DT>(p, at * ld + c, n - c, (m - 1 - at) * ld + n - c);
  }
  __device__ __forceinline__ Eight value(int left) const {
    Eight x = raw.value();
    if constexpr (WHOLE) {
      if (left <= 0) x = Eight{};
    } else {
      clear_tail(left, x);
    }
    return x;
  }
};
template <int DT, bool WHOLE>
__device__ __forceinline__ void put8(void* p, long i, const Eight& x, int left) {
  if (left > 0) store8<DT>(p, i, x, WHOLE ? 8 : left);
}
template <bool WHOLE>
__device__ __forceinline__ Eight unit_of(const float* p, int j, int n, float other) {
  if constexpr (WHOLE) {
    Eight r;
    if (p) {
      __builtin_memcpy(r.v, p + (j < n ? j : 0), 32);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) r.v[e] = other;
    }
    return r;
  } else {
    return vector8(p, j < n ? j : 0, n, other);
  }
}

// WHOLE: n is a multiple of 8, so that no single columns are looked at.
template <int DT, int LANES, bool WHOLE>
__global__ __launch_bounds__(norm_threads<LANES>()) void norm_rows(NormArgs a) {
  constexpr int kThreads = norm_threads<LANES>(), kRows = kThreads / LANES;
  __shared__ float2 lds[2][RowSum<LANES>::kWaves];
  const Generator random(a.drop);
  const int part = threadIdx.x % LANES, n = a.n, j = 8 * part, left = n - j;
  const float each = 1.f / n;
  const long units = (n + 7l) / 8, step = (long)gridDim.x * kRows;
  RowSum<LANES> sum(lds);
  Eight w, s, next_w, next_s;
  if (a.o) {
    w = unit_of<WHOLE>(a.weight, j, n, 1.f);
    s = unit_of<WHOLE>(a.shift, j, n, 0.f);
  }
  if (a.v) {
    next_w = unit_of<WHOLE>(a.next_weight, j, n, 1.f);
    next_s = unit_of<WHOLE>(a.next_shift, j, n, 0.f);
  }
  // a row's loads are made before the row in front of it is worked on
  Unit<DT, WHOLE> raw_o, raw_x;
  long i = (long)blockIdx.x * kRows + (kRows == 1 ? 0 : threadIdx.x / LANES);
  raw_x.load(a.x, a.ldx, i, j, a.m, n);
  if (a.o) raw_o.load(a.o, a.ldo, i, j, a.m, n);
  for (long first = (long)blockIdx.x * kRows; first < a.m; first += step, i += step) {
    const bool ok = i < a.m;
    Eight u = raw_x.value(left), b;
    if (a.o) b = raw_o.value(left);
    if (first + step < a.m) {
      raw_x.load(a.x, a.ldx, i + step, j, a.m, n);
      if (a.o) raw_o.load(a.o, a.ldo, i + step, j, a.m, n);
    }
    if (a.o) {
      const Stat t = row_stat<LANES, WHOLE>(a.norm, b, left, each, a.eps, sum);
#pragma unroll
      for (int e = 0; e < 8; ++e) b.v[e] = (b.v[e] - t.mean) * t.r * w.v[e] + s.v[e];
      if (a.drop.threshold) drop8(b, kept8(random.words(i * units + part), a.drop), a.drop);
      if (a.gate) {
        const Eight g = unit_of<WHOLE>(a.gate + (ok ? i : a.m - 1) / a.gate_rows * a.ldg, j, n, 1.f);
#pragma unroll
        for (int e = 0; e < 8; ++e) b.v[e] *= g.v[e];
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) u.v[e] = rounded<DT>(a.scale * u.v[e] + b.v[e]);
      if (ok) put8<DT, WHOLE>(a.u, i * a.ldu + j, u, left);
      if (left < 8) clear_tail(left, u);
    }
    if (!a.v) continue;
    const Stat t = row_stat<LANES, WHOLE>(a.next_norm, u, left, each, a.eps, sum);
#pragma unroll
    for (int e = 0; e < 8; ++e) u.v[e] = (u.v[e] - t.mean) * t.r * next_w.v[e] + next_s.v[e];
    if (ok) put8<DT, WHOLE>(a.v, i * a.ldv + j, u, left);
  }
}

// ------------------------------------------------------------------ gradients
//   D = du + r' (g - [layer: mean g] - uh mean(g uh)),  g = dv next_weight,  uh = (u - mean') r'
//   dx = scale D,  dgate = sum of D b over a gate's rows,  h = drop(gate D)
//   do = r (f - [layer: mean f] - oh mean(f oh)),  f = h weight
//   dnext_weight = sum dv uh,  dnext_shift = sum dv,  dweight = sum h oh,  dshift = sum h
//
// Statistics, dropout's pattern and b are formed again from o, u and the generator: nothing
// but what the forward pass returns is kept.  16384 x 4096 bf16, both norms, gate and
// dropout (805 MB): 185 us, 4.4 TB/s, of which the sums over chunks take 10 (norm_finish).
// The registers decide: five column sums, three of a row's matrices and the next row's
// loads.  Weights from LDS instead of registers 254 -> 197 us.  Without the shifts' sums rows of
// more than a wave are held to 128 registers, four waves a unit, 199 -> 187, though 8 spill (fp32
// 17); with them that spills more than it gains (236 us), except that a workgroup of 1024
// threads has no more registers: there 41 and 66 spill, 53 and 143 at odd widths (4000 x 6091
// fp32 376 us).  All sums are added in a fixed order: results do not depend on timing.
//
// A norm's gradients by themselves, without a branch: 16384 x 4096 bf16 91 us (403 MB, 4.4 TB/s),
// with another gradient added 120 (537 MB, 4.5); 4096 x 8192 58, 4000 x 6091 59 (fp32 76); few
// rows by latency, 130560 x 32 fp16 13, 8160 x 96 fp32 8.2, one row of 4096 4.1.
//
// A row lane is the LANES threads of a row.  Column sums stay in registers over a
// chunk's rows and are added over the row lanes at its end; a gate's, where chunks hold
// whole groups, at the group's end: groups of few rows are a row lane's each, others
// the whole workgroup's.
// Column sums of a workgroup's COUNT kinds, in LDS: a kind's sums over each wave's rows,
// which the threads then add, every column by one of them.
template <int LANES, int COUNT>
struct ColumnSums {
  static constexpr int kThreads = norm_threads<LANES>(), kWaves = LANES > 64 ? 1 : kThreads / 64, kColumns = 8 * LANES;
  typedef float Lds[LANES > 64 ? 1 : COUNT][kWaves][LANES > 64 ? 1 : kColumns];
  // Puts a kind's; where a row is more than a wave there is nothing to add.
  static __device__ __forceinline__ void put(Eight& x, int kind, Lds& lds) {
    if constexpr (LANES <= 64) {
      const int lane = threadIdx.x & 63;
#pragma unroll
      for (int e = 0; e < 8; ++e) x.v[e] = strided_sum<LANES>(x.v[e]);
      if (lane < LANES) __builtin_memcpy(&lds[kind][threadIdx.x >> 6][8 * lane], x.v, 32);
    }
  }
  // Columns' sums to `out`, all of the workgroup's threads calling; between barriers.
  static __device__ __forceinline__ void get(int kind, const Lds& lds, float* out, int n) {
    for (int j = threadIdx.x; j < n; j += kThreads) {
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) s += lds[kind][w][j];
      out[j] = s;
    }
  }
};

// SHIFTS: the shifts' gradients are wanted too.
template <int DT, int LANES, bool BRANCH, bool WHOLE, bool SHIFTS>
__global__ __launch_bounds__(norm_threads<LANES>(), LANES >= 128 && !SHIFTS ? 4 : 1) void norm_back_rows(NormBackArgs a) {
  constexpr int kThreads = norm_threads<LANES>(), kRowLanes = kThreads / LANES;
  constexpr int kSums = SHIFTS ? 4 : 2;
  typedef ColumnSums<LANES, BRANCH ? kSums : kSums / 2> Columns;
  __shared__ float2 lds[2][RowSum<LANES>::kWaves];
  __shared__ __attribute__((aligned(16))) typename Columns::Lds column_lds;
  // the norms' weights, read again for every row: held in registers they leave a unit half
  // as many waves
  __shared__ __attribute__((aligned(16))) float vectors[3][8 * LANES];
  const Generator random(a.drop);
  const int part = threadIdx.x % LANES, lane = kRowLanes == 1 ? 0 : threadIdx.x / LANES, n = a.n, j = 8 * part, left = n - j;
  const float each = 1.f / n;
  const long units = (n + 7l) / 8;
  const NormChunks& c = a.chunks;
  RowSum<LANES> sum(lds);
  Eight along{}, total{}, next_along{}, next_total{}, gate_sum{};
  auto hold_all = [&]() __attribute__((always_inline)) {
    auto hold = [&](int which, const Eight& v) __attribute__((always_inline)) { __builtin_memcpy(&vectors[which][j], v.v, 32); };
    if constexpr (BRANCH) {
      hold(0, unit_of<WHOLE>(a.weight, j, n, 1.f));
      hold(1, unit_of<WHOLE>(a.shift, j, n, 0.f));
    }
    if (a.dv) hold(2, unit_of<WHOLE>(a.next_weight, j, n, 1.f));
  };
  auto held = [&](int which) __attribute__((always_inline)) {
    Eight v;
    __builtin_memcpy(v.v, &vectors[which][j], 32);
    return v;
  };

  Unit<DT, WHOLE> raw_du, raw_dv, raw_u, raw_o;
  // (every lambda here is inlined: left to itself the compiler calls them and keeps the
  // arrays in memory)
  auto load = [&](long i) __attribute__((always_inline)) {
    if (a.du) raw_du.load(a.du, a.lddu, i, j, a.m, n);
    if (a.dv) {
      raw_dv.load(a.dv, a.lddv, i, j, a.m, n);
      raw_u.load(a.u, a.ldu, i, j, a.m, n);
    }
    if constexpr (BRANCH) raw_o.load(a.o, a.ldo, i, j, a.m, n);
  };
  // Row i, whose elements are loaded; ok: it exists.  `next`: the row to load meanwhile.
  auto row = [&](long i, bool ok, long next) __attribute__((always_inline)) {
    Eight d{}, dv{}, u{}, o{};
    if (a.du) d = raw_du.value(left);
    if (a.dv) {
      dv = raw_dv.value(left);
      u = raw_u.value(left);
    }
    if constexpr (BRANCH) o = raw_o.value(left);
    if (next >= 0) load(next);
    Stat of_u, of_o;
    row_stats<LANES, WHOLE>(a.dv ? a.next_norm : OIDN_NORM_NONE, u, of_u, BRANCH ? a.norm : OIDN_NORM_NONE, o, of_o, left,
                            each, a.eps, sum);
    if (a.dv) {
      const Eight next_w = held(2);
      float c0 = 0.f, c1 = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        u.v[e] = (u.v[e] - of_u.mean) * of_u.r;
        if (ok) {
          next_along.v[e] += dv.v[e] * u.v[e];
          if constexpr (SHIFTS) next_total.v[e] += dv.v[e];
        }
        dv.v[e] *= next_w.v[e];
        c0 += dv.v[e];
        c1 += dv.v[e] * u.v[e];
      }
      const float2 both = sum(c0, c1);
      c0 = a.next_norm == OIDN_NORM_LAYER ? both.x * each : 0.f;
      c1 = both.y * each;
#pragma unroll
      for (int e = 0; e < 8; ++e) d.v[e] += of_u.r * (dv.v[e] - c0 - u.v[e] * c1);
    }
    if (a.dx && ok) {
      Eight x;
#pragma unroll
      for (int e = 0; e < 8; ++e) x.v[e] = a.scale * d.v[e];
      put8<DT, WHOLE>(a.dx, i * a.lddx + j, x, left);
    }
    if constexpr (BRANCH) {
      __builtin_amdgcn_sched_barrier(0);       // d alone is left of what is above
      unsigned keep = 0;
      if (a.drop.threshold) keep = kept8(random.words(i * units + part), a.drop);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int e = 0; e < 8; ++e) o.v[e] = (o.v[e] - of_o.mean) * of_o.r;
      const Eight w = held(0);
      if (a.dgate) {
        const Eight s = held(1);
        Eight b;
#pragma unroll
        for (int e = 0; e < 8; ++e) b.v[e] = o.v[e] * w.v[e] + s.v[e];
        if (a.drop.threshold) drop8(b, keep, a.drop);
        if (ok) {
#pragma unroll
          for (int e = 0; e < 8; ++e) gate_sum.v[e] += d.v[e] * b.v[e];
        }
      }
      __builtin_amdgcn_sched_barrier(0);
      if (a.gate) {
        const Eight g = unit_of<WHOLE>(a.gate + (ok ? i : a.m - 1) / c.group_rows * a.ldg, j, n, 1.f);
#pragma unroll
        for (int e = 0; e < 8; ++e) d.v[e] *= g.v[e];
      }
      // h, and h hat(o), which is 0 in dropped places whatever o holds
      Eight weighted;
#pragma unroll
      for (int e = 0; e < 8; ++e) weighted.v[e] = d.v[e] * o.v[e];
      if (a.drop.threshold) {
        drop8(d, keep, a.drop);
        drop8(weighted, keep, a.drop);
      }
      float c0 = 0.f, c1 = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (ok) {
          along.v[e] += weighted.v[e];
          if constexpr (SHIFTS) total.v[e] += d.v[e];
        }
        d.v[e] *= w.v[e];
        if (WHOLE || e < left) {
          c0 += d.v[e];
          c1 += weighted.v[e] * w.v[e];
        }
      }
      if (WHOLE && left <= 0) c0 = c1 = 0.f;
      if (a.d_o) {
        if (a.norm != OIDN_NORM_NONE) {
          const float2 both = sum(c0, c1);
          c0 = a.norm == OIDN_NORM_LAYER ? both.x * each : 0.f;
          c1 = both.y * each;
#pragma unroll
          for (int e = 0; e < 8; ++e) d.v[e] = of_o.r * (d.v[e] - c0 - o.v[e] * c1);
        }
        if (ok) put8<DT, WHOLE>(a.d_o, i * a.lddo + j, d, left);
      }
    }
  };
  const long chunk = blockIdx.x, group = c.per_group ? chunk / c.per_group : 0;
  const bool alone = c.lane_groups && LANES <= 64;       // a row lane's groups are its own
  long first = chunk * c.rows, last = first + c.rows, span = c.group_rows;
  if (c.per_group) {                                     // a part of one group
    first = group * c.group_rows + (chunk - group * c.per_group) * c.rows;
    span = c.rows;
    last = first + span < (group + 1) * c.group_rows ? first + span : (group + 1) * c.group_rows;
  }
  last = last < a.m ? last : a.m;
  const int lanes = alone ? 1 : kRowLanes;
  long g = first;
  do {       // once for a part, which may be empty
    const long begin = g + (alone ? lane * span : 0), end = begin + span < last ? begin + span : last;
    long i = begin + (alone ? 0 : lane);
    load(i);
    if (g == first) {                                    // behind the first row's loads
      if (lane == 0) hold_all();
      __syncthreads();
    }
    for (long r = begin; r < end; r += lanes, i += lanes) row(i, i < end, r + lanes < end ? i + lanes : -1);
    if (BRANCH && a.dgate) {
      float* const out = c.per_group ? a.gate_part + chunk * n : a.dgate + begin / c.group_rows * a.lddg;
      if (alone || LANES > 64) {
        if (begin < end || !alone) put8<OIDN_F32, WHOLE>(out, j, gate_sum, left);
      } else {
        Columns::put(gate_sum, 0, column_lds);
        __syncthreads();
        Columns::get(0, column_lds, out, n);
        __syncthreads();
      }
      gate_sum = Eight{};
    }
    g += alone ? span * kRowLanes : span;
  } while (g < last);
  auto each_kind = [&](auto take) __attribute__((always_inline)) {
    if constexpr (BRANCH) {
      if (a.sums[0]) take(0, 0, along);
      if constexpr (SHIFTS) if (a.sums[1]) take(1, 1, total);
    }
    constexpr int kFirst = BRANCH ? kSums / 2 : 0;
    if (a.sums[2]) take(2, kFirst, next_along);
    if constexpr (SHIFTS) if (a.sums[3]) take(3, kFirst + 1, next_total);
  };
  auto out_of = [&](int which) __attribute__((always_inline)) {
    return c.count > 1 ? a.part + (chunk * kNormSums + which) * n : a.sums[which];
  };
  if constexpr (LANES > 64) {
    each_kind([&](int which, int, Eight& x) __attribute__((always_inline)) { put8<OIDN_F32, WHOLE>(out_of(which), j, x, left); });
  } else {
    each_kind([&](int, int at, Eight& x) __attribute__((always_inline)) { Columns::put(x, at, column_lds); });
    __syncthreads();
    each_kind([&](int which, int at, Eight&) __attribute__((always_inline)) { Columns::get(at, column_lds, out_of(which), n); });
  }
}

}  // namespace
}  // namespace oidn
