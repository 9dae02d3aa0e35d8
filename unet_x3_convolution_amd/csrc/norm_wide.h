// Rows of any width (here: more than 8192 columns): a workgroup takes a row and goes over
// it again for each statistic (the row stays in the caches); column sums take a launch of
// their own, from what the first left of every row.  The mathematics and roundings are
// norm_fast.h's.  Bound by the passes' reads from the caches: 4096 x 16384 bf16 forward
// (537 MB from memory) 190 us, 2.8 TB/s; gradients (805 MB) 561 us, 1.4 TB/s.  8192 columns
// in this form instead of registers: gradients 346 us for 234 (4000 rows, bf16).
#pragma once

#include "lanes.h"
#include "norm_rows.h"

namespace oidn {
namespace {

// Sums of a pair over the workgroup; lds: kNormThreads / 64 pairs.
__device__ __forceinline__ float2 sum_of_group(float2 v, float2* lds) {
  v.x = lanes_sum<64>(v.x);
  v.y = lanes_sum<64>(v.y);
  __syncthreads();                       // what was summed before has been read
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  float2 t = lds[0];
#pragma unroll
  for (int k = 1; k < kNormThreads / 64; ++k) {
    t.x += lds[k].x;
    t.y += lds[k].y;
  }
  return t;
}

// The statistics of a row that load(j) gives eight columns of.
template <typename Load>
__device__ __forceinline__ Stat wide_stat(int kind, int n, float eps, float2* lds, Load load) {
  if (kind == OIDN_NORM_NONE) return {0.f, 1.f};
  Stat s{0.f, 0.f};
  const float each = 1.f / n;
  if (kind == OIDN_NORM_LAYER) {
    float t = 0.f;
    for (int j = 8 * threadIdx.x; j < n; j += 8 * kNormThreads) {
      const Eight x = load(j);
#pragma unroll
      for (int k = 0; k < 8; ++k) t += x.v[k];
    }
    s.mean = sum_of_group({t, 0.f}, lds).x * each;
  }
  float t = 0.f;
  for (int j = 8 * threadIdx.x; j < n; j += 8 * kNormThreads) {
    const Eight x = load(j);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float d = k < n - j ? x.v[k] - s.mean : 0.f;
      t += d * d;
    }
  }
  s.r = rsqrtf(sum_of_group({t, 0.f}, lds).x * each + eps);
  return s;
}

template <int DT>
__global__ __launch_bounds__(kNormThreads) void norm_wide(NormArgs a) {
  __shared__ float2 lds[kNormThreads / 64];
  const Generator random(a.drop);
  const int n = a.n;
  for (long i = blockIdx.x; i < a.m; i += gridDim.x) {
    auto load_x = [&](int j) { return row8<DT>(a.x, a.ldx, i, j, a.m, n); };
    if (a.o) {
      auto load_o = [&](int j) { return row8<DT>(a.o, a.ldo, i, j, a.m, n); };
      const Stat s = wide_stat(a.norm, n, a.eps, lds, load_o);
      const float* const gate = a.gate ? a.gate + i / a.gate_rows * a.ldg : nullptr;
      for (int j = 8 * threadIdx.x; j < n; j += 8 * kNormThreads) {
        Eight b = load_o(j);
        const Eight x = load_x(j), w = vector8(a.weight, j, n, 1.f), t = vector8(a.shift, j, n, 0.f),
                    g = vector8(gate, j, n, 1.f);
#pragma unroll
        for (int k = 0; k < 8; ++k) b.v[k] = (b.v[k] - s.mean) * s.r * w.v[k] + t.v[k];
        if (a.drop.threshold) drop8(b, kept8(random.words(i * ((n + 7l) / 8) + j / 8), a.drop), a.drop);
#pragma unroll
        for (int k = 0; k < 8; ++k) b.v[k] = a.scale * x.v[k] + g.v[k] * b.v[k];
        store8<DT>(a.u, i * a.ldu + j, b, n - j);
      }
    }
    if (!a.v) continue;
    // each thread reads back the columns that it stored itself
    auto load_u = [&](int j) { return a.o ? row8<DT>(a.u, a.ldu, i, j, a.m, n) : load_x(j); };
    const Stat s = wide_stat(a.next_norm, n, a.eps, lds, load_u);
    for (int j = 8 * threadIdx.x; j < n; j += 8 * kNormThreads) {
      Eight u = load_u(j);
      const Eight w = vector8(a.next_weight, j, n, 1.f), t = vector8(a.next_shift, j, n, 0.f);
#pragma unroll
      for (int k = 0; k < 8; ++k) u.v[k] = (u.v[k] - s.mean) * s.r * w.v[k] + t.v[k];
      store8<DT>(a.v, i * a.ldv + j, u, n - j);
    }
  }
}

// What a row's gradients need besides its elements: with hat(u) = (u - mean) r and
// g = dv next_weight, next_norm'(dv) = r (g - c0 - hat c1).
struct BackRow { Stat u, o; float c0, c1; };

// D of eight columns; hat(u) in `hat`, dv in `dv`.
template <int DT>
__device__ __forceinline__ Eight gradient_of_u(const NormBackArgs& a, const BackRow& r, long i, int j, Eight& hat,
                                               Eight& dv) {
  Eight d{};
  if (a.du) d = row8<DT>(a.du, a.lddu, i, j, a.m, a.n);
  if (a.dv) {
    dv = row8<DT>(a.dv, a.lddv, i, j, a.m, a.n);
    hat = row8<DT>(a.u, a.ldu, i, j, a.m, a.n);
    const Eight w = vector8(a.next_weight, j, a.n, 1.f);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      hat.v[k] = (hat.v[k] - r.u.mean) * r.u.r;
      d.v[k] += r.u.r * (dv.v[k] * w.v[k] - r.c0 - hat.v[k] * r.c1);
    }
  }
  return d;
}

// Gradients of every row, and what norm_columns needs of it.
template <int DT>
__global__ __launch_bounds__(kNormThreads) void norm_back_wide(NormBackArgs a) {
  __shared__ float2 lds[kNormThreads / 64];
  const Generator random(a.drop);
  const int n = a.n;
  const float each = 1.f / n;
  for (long i = blockIdx.x; i < a.m; i += gridDim.x) {
    BackRow r{{0.f, 1.f}, {0.f, 1.f}, 0.f, 0.f};
    if (a.dv) {
      r.u = wide_stat(a.next_norm, n, a.eps, lds, [&](int j) { return row8<DT>(a.u, a.ldu, i, j, a.m, n); });
      float2 t = {0.f, 0.f};
      for (int j = 8 * threadIdx.x; j < n; j += 8 * kNormThreads) {
        const Eight u = row8<DT>(a.u, a.ldu, i, j, a.m, n), dv = row8<DT>(a.dv, a.lddv, i, j, a.m, n),
                    w = vector8(a.next_weight, j, n, 1.f);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float g = dv.v[k] * w.v[k];
          t.x += g;
          t.y += g * (u.v[k] - r.u.mean) * r.u.r;
        }
      }
      t = sum_of_group(t, lds);
      r.c0 = a.next_norm == OIDN_NORM_LAYER ? t.x * each : 0.f;
      r.c1 = t.y * each;
    }
    const float* const gate = a.gate ? a.gate + i / a.chunks.group_rows * a.ldg : nullptr;
    if (a.o) r.o = wide_stat(a.norm, n, a.eps, lds, [&](int j) { return row8<DT>(a.o, a.ldo, i, j, a.m, n); });
    // hat(o), and the gradient of norm(o)
    auto branch = [&](const Eight& d, int j, Eight& hat) {
      hat = row8<DT>(a.o, a.ldo, i, j, a.m, n);
      const Eight w = vector8(a.weight, j, n, 1.f), g = vector8(gate, j, n, 1.f);
      Eight h;
#pragma unroll
      for (int k = 0; k < 8; ++k) h.v[k] = d.v[k] * g.v[k];
      if (a.drop.threshold) drop8(h, kept8(random.words(i * ((n + 7l) / 8) + j / 8), a.drop), a.drop);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        hat.v[k] = (hat.v[k] - r.o.mean) * r.o.r;
        h.v[k] *= w.v[k];
      }
      return h;
    };
    float2 t = {0.f, 0.f};
    for (int j = 8 * threadIdx.x; j < n; j += 8 * kNormThreads) {
      Eight hat, dv, d = gradient_of_u<DT>(a, r, i, j, hat, dv);
      if (a.o && a.norm != OIDN_NORM_NONE) {
        const Eight h = branch(d, j, hat);
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (k < n - j) {
            t.x += h.v[k];
            t.y += h.v[k] * hat.v[k];
          }
      }
      if (a.dx) {
#pragma unroll
        for (int k = 0; k < 8; ++k) d.v[k] *= a.scale;
        store8<DT>(a.dx, i * a.lddx + j, d, n - j);
      }
    }
    if (a.d_o) {
      if (a.norm != OIDN_NORM_NONE) t = sum_of_group(t, lds);
      const float c0 = a.norm == OIDN_NORM_LAYER ? t.x * each : 0.f, c1 = t.y * each;
      for (int j = 8 * threadIdx.x; j < n; j += 8 * kNormThreads) {
        Eight hat, dv, d = gradient_of_u<DT>(a, r, i, j, hat, dv), h = branch(d, j, hat);
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (a.norm != OIDN_NORM_NONE) h.v[k] = r.o.r * (h.v[k] - c0 - hat.v[k] * c1);
        store8<DT>(a.d_o, i * a.lddo + j, h, n - j);
      }
    }
    if (threadIdx.x == 0 && a.rows) {
      float* const s = a.rows + kRowFloats * i;
      s[0] = r.u.mean, s[1] = r.u.r, s[2] = r.c0, s[3] = r.c1, s[4] = r.o.mean, s[5] = r.o.r;
    }
  }
}

// Column sums of chunk blockIdx.x: a thread takes eight columns and the chunk's
// rows in order.
template <int DT>
__global__ __launch_bounds__(kNormThreads) void norm_columns(NormBackArgs a) {
  const Generator random(a.drop);
  const int n = a.n, j = 8 * (blockIdx.y * kNormThreads + threadIdx.x);
  if (j >= n) return;
  const NormChunks& c = a.chunks;
  const long chunk = blockIdx.x;
  long first = chunk * c.rows, last = first + c.rows;
  if (c.per_group) {
    const long group = chunk / c.per_group, end = (group + 1) * c.group_rows;
    first = group * c.group_rows + (chunk - group * c.per_group) * c.rows;
    last = first + c.rows < end ? first + c.rows : end;
  }
  last = last < a.m ? last : a.m;
  Eight sums[kNormSums] = {}, gate_sum{};
  const Eight w = vector8(a.weight, j, n, 1.f), s = vector8(a.shift, j, n, 0.f);
  for (long i = first; i < last; ++i) {
    const float* const f = a.rows + kRowFloats * i;
    const BackRow r{{f[0], f[1]}, {f[4], f[5]}, f[2], f[3]};
    Eight hat, dv;
    const Eight d = gradient_of_u<DT>(a, r, i, j, hat, dv);
    if (a.dv) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        sums[2].v[k] += dv.v[k] * hat.v[k];
        sums[3].v[k] += dv.v[k];
      }
    }
    if (!a.o) continue;
    hat = row8<DT>(a.o, a.ldo, i, j, a.m, n);
    const long group = i / c.group_rows;
    const Eight g = vector8(a.gate ? a.gate + group * a.ldg : nullptr, j, n, 1.f);
    Eight b, h, along;           // along: h hat, 0 in dropped places whatever they hold
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      hat.v[k] = (hat.v[k] - r.o.mean) * r.o.r;
      b.v[k] = hat.v[k] * w.v[k] + s.v[k];
      h.v[k] = d.v[k] * g.v[k];
      along.v[k] = h.v[k] * hat.v[k];
    }
    if (a.drop.threshold) {
      const unsigned keep = kept8(random.words(i * ((n + 7l) / 8) + j / 8), a.drop);
      drop8(b, keep, a.drop);
      drop8(h, keep, a.drop);
      drop8(along, keep, a.drop);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      sums[0].v[k] += along.v[k];
      sums[1].v[k] += h.v[k];
      gate_sum.v[k] += d.v[k] * b.v[k];
    }
    // the end of a group inside the chunk
    if (a.dgate && !c.per_group && (i + 1 == last || (i + 1) % c.group_rows == 0)) {
      store8<OIDN_F32>(a.dgate, group * a.lddg + j, gate_sum, n - j);
      gate_sum = Eight{};
    }
  }
#pragma unroll
  for (int k = 0; k < kNormSums; ++k)
    if (a.sums[k]) store8<OIDN_F32>(c.count > 1 ? a.part + (chunk * kNormSums + k) * n : a.sums[k], j, sums[k], n - j);
  if (a.dgate && c.per_group) store8<OIDN_F32>(a.gate_part + chunk * n, j, gate_sum, n - j);
}

}  // namespace
}  // namespace oidn
