// Internal declarations of what stands around a block over activation rows:
// the norms before and after it with its gate and residual scale, and dropout.
#pragma once

#include "internal.h"

namespace oidn {

// Dropout: which elements are kept follows from the generator's state alone
// (norm_rows.h).  threshold 0: nothing is dropped, the state is not read.
struct Dropout {
  unsigned threshold;              // of 65536: an element is kept where its 16 bits are not below
  float gain;                      // of a kept element
  const unsigned long long* rng;   // seed, offset
};

// u = scale x + gate drop(norm(o) weight + shift),  v = next_norm(u) next_weight + next_shift
struct NormArgs {
  const void* o;                   // null: u is x and is not stored
  long ldo;
  const float *weight, *shift;     // may be null
  const float* gate;               // a row for every gate_rows rows, may be null
  long ldg, gate_rows;
  const void* x;
  long ldx;
  float scale;
  Dropout drop;
  void* u;
  long ldu;
  const float *next_weight, *next_shift;
  void* v;                         // null: next_norm is OIDN_NORM_NONE
  long ldv;
  long m;
  int n;
  int norm, next_norm;
  float eps;
};

// Rows in chunks that a workgroup goes through, such that a chunk either holds
// whole gate groups or lies in one.
struct NormChunks {
  long rows;               // of a chunk
  long per_group;          // chunks of a gate group, two at least; 0: a chunk holds whole groups
  long group_rows;         // rows that share a gate, all of them without one
  int lane_groups;         // a chunk's groups are its row lanes' (norm_fast.h), else the workgroup's
  long count;
};
// Lanes that hold a row, eight columns each (norm_fast.h): 0 if it is too wide for them
// (norm_wide.h).
inline int norm_lanes(int n) {
  int lanes = 4;
  while (8 * lanes < n) lanes *= 2;
  return lanes <= 1024 ? lanes : 0;
}
// A chunk's rows come in multiples of this: what a workgroup takes at once, and two where
// 128 threads take one (1000 x 1000 bf16 gradients 15.2 us, in chunks of one row 17.5).
inline int norm_chunk_step(int n) {
  const int lanes = norm_lanes(n);
  return lanes && lanes < 256 ? 256 / lanes : 1;
}
constexpr int kNormSums = 4;       // dweight, dshift, dnext_weight, dnext_shift
// D = du + next_norm'(dv; u),  dx = scale D, and the branch's gradients
struct NormBackArgs {
  const void* du;                  // may be null
  long lddu;
  const void* dv;                  // null: next_norm is OIDN_NORM_NONE
  long lddv;
  const void* o;                   // null: no branch
  long ldo;
  const float *weight, *shift, *gate;
  long ldg;
  const void* u;                   // read where dv is
  long ldu;
  float scale;
  Dropout drop;
  const float* next_weight;
  void* dx;                        // may be null, as the other results
  long lddx;
  void* d_o;
  long lddo;
  float* dgate;
  long lddg;
  float* sums[kNormSums];
  float* rows;                     // workspace: kRowFloats of every row (wide rows)
  float* part;                     // workspace, with more than one chunk: [chunk][kNormSums][n]
  float* gate_part;                // workspace, where a group has more than one: [chunk][n]
  NormChunks chunks;
  long m;
  int n;
  int norm, next_norm;
  float eps;
};
constexpr int kRowFloats = 8;

NormChunks norm_chunks(long m, int n, long gate_rows);
hipError_t launch_norm(const NormArgs& a, int dtype, hipStream_t stream);
hipError_t launch_norm_back(const NormBackArgs& a, int dtype, hipStream_t stream);
// y = drop(x) + residual
hipError_t launch_dropout(const void* x, long ldx, const void* residual, long ldr, void* y, long ldy, long m, int n,
                          const Dropout& d, int dtype, hipStream_t stream);

}  // namespace oidn
