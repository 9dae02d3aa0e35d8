// Host side of the norms around a block and of dropout: argument checks,
// workspace layout and launches.  Nothing here allocates device memory, waits
// for the device or throws.
#include <cmath>

#include "dense_checks.h"
#include "norm.h"

using namespace oidn;

namespace {

int check_norm(const char* name, int norm, int least) {
  if (norm >= least && norm <= OIDN_NORM_LAYER) return OIDN_OK;
  return fail(OIDN_E_INVALID, "%s: %d is not a norm here", name, norm);
}
int check_eps(float eps) {
  if (eps >= 0.f && std::isfinite(eps)) return OIDN_OK;
  return fail(OIDN_E_INVALID, "eps must be a finite number >= 0");
}
int check_dropout(float p, const unsigned long long* rng, Dropout& d) {
  if (!(p >= 0.f && p <= 1.f)) return fail(OIDN_E_INVALID, "dropout probability %g is not in [0, 1]", (double)p);
  d.threshold = (unsigned)std::rint(p * 65536.f);
  d.gain = d.threshold < 65536u ? 65536.f / (float)(65536u - d.threshold) : 0.f;
  d.rng = rng;
  if (!d.threshold) return OIDN_OK;
  if (!rng) return fail(OIDN_E_INVALID, "null pointer: rng");
  return check_aligned("rng", rng, 8);
}
int check_vectors(std::initializer_list<const float*> all) {
  for (const float* v : all) OIDN_TRY(check_aligned("a vector of float32", v, 4));
  return OIDN_OK;
}
// A gate's rows of n columns, each for gate_rows rows.
int check_gate(const char* name, const float* gate, long ld, int n, long gate_rows) {
  if (!gate) return OIDN_OK;
  if (gate_rows < 1) return fail(OIDN_E_INVALID, "gate_rows must be at least 1, got %ld", gate_rows);
  return check_matrix(name, gate, ld, n, OIDN_F32, false);
}

struct BackSpace {
  NormChunks chunks;
  float *rows, *part, *gate_part;
  size_t bytes;
};
BackSpace back_space(long m, int n, long gate_rows, void* ws) {
  BackSpace b{};
  b.chunks = norm_chunks(m, n, gate_rows);
  Regions r{static_cast<char*>(ws), 0};
  auto floats = [&](size_t count) { return static_cast<float*>(r.take(align256(count * sizeof(float)))); };
  if (!norm_lanes(n)) b.rows = floats((size_t)m * kRowFloats);
  if (b.chunks.count > 1) b.part = floats((size_t)b.chunks.count * kNormSums * n);
  if (gate_rows && b.chunks.per_group) b.gate_part = floats((size_t)b.chunks.count * n);
  b.bytes = r.used;
  return b;
}
// Sums over no rows.
int zero_sums(float* const* sums, int n, hipStream_t stream) {
  for (int k = 0; k < kNormSums; ++k)
    if (sums[k]) OIDN_TRY(ran(launch_zero(sums[k], 1, n * sizeof(float), 0, stream), "zero launch"));
  return OIDN_OK;
}
int run_back(NormBackArgs& a, long gate_rows, int dtype, void* workspace, size_t ws_bytes, hipStream_t stream) {
  const BackSpace b = back_space(a.m, a.n, gate_rows, workspace);
  OIDN_TRY(check_workspace(workspace, ws_bytes, b.bytes));
  a.chunks = b.chunks;
  a.rows = b.rows;
  a.part = b.part;
  a.gate_part = b.gate_part;
  return ran(launch_norm_back(a, dtype, stream), "norm gradients launch");
}

}  // namespace

extern "C" {

int oidn_norm(const void* x, long ldx, const float* weight, const float* shift, void* y, long ldy, long m, int n,
              int norm, float eps, int dtype, hipStream_t stream) {
  OIDN_TRY(check_type(dtype));
  OIDN_TRY(check_size("x", m, n));
  OIDN_TRY(check_norm("norm", norm, OIDN_NORM_RMS));
  OIDN_TRY(check_eps(eps));
  if (m == 0) return clear_error();
  OIDN_TRY(check_matrix("x", x, ldx, n, dtype, false));
  OIDN_TRY(check_vectors({weight, shift}));
  OIDN_TRY(check_matrix("y", y, ldy, n, dtype, false));
  NormArgs a{};
  a.x = x;
  a.ldx = ldx;
  a.next_weight = weight;
  a.next_shift = shift;
  a.v = y;
  a.ldv = ldy;
  a.m = m;
  a.n = n;
  a.next_norm = norm;
  a.eps = eps;
  OIDN_TRY(ran(launch_norm(a, dtype, stream), "norm launch"));
  return clear_error();
}

int oidn_norm_backward_workspace_bytes(long m, int n, int dtype, size_t* bytes) {
  if (!bytes) return fail(OIDN_E_INVALID, "null bytes pointer");
  OIDN_TRY(check_type(dtype));
  OIDN_TRY(check_size("x", m, n));
  *bytes = m ? back_space(m, n, 0, nullptr).bytes : 0;
  return clear_error();
}

int oidn_norm_backward(const void* dy, long lddy, const void* x, long ldx, const float* weight, const void* add,
                       long ldadd, void* dx, long lddx, float* dweight, float* dshift, long m, int n, int norm,
                       float eps, int dtype, void* workspace, size_t ws_bytes, hipStream_t stream) {
  OIDN_TRY(check_type(dtype));
  OIDN_TRY(check_size("x", m, n));
  OIDN_TRY(check_norm("norm", norm, OIDN_NORM_RMS));
  OIDN_TRY(check_eps(eps));
  OIDN_TRY(check_vectors({weight, dweight, dshift}));
  NormBackArgs a{};
  a.sums[2] = dweight;
  a.sums[3] = dshift;
  if (m == 0) {
    OIDN_TRY(zero_sums(a.sums, n, stream));
    return clear_error();
  }
  OIDN_TRY(check_matrix("dy", dy, lddy, n, dtype, false));
  OIDN_TRY(check_matrix("x", x, ldx, n, dtype, false));
  OIDN_TRY(check_matrix("add", add, ldadd, n, dtype, true));
  OIDN_TRY(check_matrix("dx", dx, lddx, n, dtype, true));
  a.du = add;
  a.lddu = ldadd;
  a.dv = dy;
  a.lddv = lddy;
  a.u = x;
  a.ldu = ldx;
  a.scale = 1.f;
  a.next_weight = weight;
  a.dx = dx;
  a.lddx = lddx;
  a.m = m;
  a.n = n;
  a.next_norm = norm;
  a.eps = eps;
  OIDN_TRY(run_back(a, 0, dtype, workspace, ws_bytes, stream));
  return clear_error();
}

int oidn_norm_residual(const void* o, long ldo, const float* weight, const float* shift, const float* gate, long ldg,
                       long gate_rows, const void* x, long ldx, float scale, float p, const unsigned long long* rng,
                       void* u, long ldu, const float* next_weight, const float* next_shift, void* v, long ldv, long m,
                       int n, int norm, int next_norm, float eps, int dtype, hipStream_t stream) {
  OIDN_TRY(check_type(dtype));
  OIDN_TRY(check_size("x", m, n));
  OIDN_TRY(check_norm("norm", norm, OIDN_NORM_NONE));
  OIDN_TRY(check_norm("next_norm", next_norm, OIDN_NORM_NONE));
  OIDN_TRY(check_eps(eps));
  NormArgs a{};
  OIDN_TRY(check_dropout(p, rng, a.drop));
  OIDN_TRY(check_gate("gate", gate, ldg, n, gate_rows));
  if (m == 0) return clear_error();
  OIDN_TRY(check_matrix("o", o, ldo, n, dtype, false));
  OIDN_TRY(check_vectors({weight, shift, next_weight, next_shift}));
  OIDN_TRY(check_matrix("x", x, ldx, n, dtype, false));
  OIDN_TRY(check_matrix("u", u, ldu, n, dtype, false));
  if (next_norm == OIDN_NORM_NONE && v) return fail(OIDN_E_INVALID, "v without next_norm");
  OIDN_TRY(check_matrix("v", v, ldv, n, dtype, next_norm == OIDN_NORM_NONE));
  a.o = o;
  a.ldo = ldo;
  a.weight = weight;
  a.shift = shift;
  a.gate = gate;
  a.ldg = ldg;
  a.gate_rows = gate_rows;
  a.x = x;
  a.ldx = ldx;
  a.scale = scale;
  a.u = u;
  a.ldu = ldu;
  a.next_weight = next_weight;
  a.next_shift = next_shift;
  a.v = v;
  a.ldv = ldv;
  a.m = m;
  a.n = n;
  a.norm = norm;
  a.next_norm = next_norm;
  a.eps = eps;
  OIDN_TRY(ran(launch_norm(a, dtype, stream), "norm launch"));
  return clear_error();
}

int oidn_norm_residual_backward_workspace_bytes(long m, int n, long gate_rows, int dtype, size_t* bytes) {
  if (!bytes) return fail(OIDN_E_INVALID, "null bytes pointer");
  OIDN_TRY(check_type(dtype));
  OIDN_TRY(check_size("x", m, n));
  if (gate_rows < 0) return fail(OIDN_E_INVALID, "gate_rows must not be negative, got %ld", gate_rows);
  *bytes = m ? back_space(m, n, gate_rows, nullptr).bytes : 0;
  return clear_error();
}

int oidn_norm_residual_backward(const void* du, long lddu, const void* dv, long lddv, const void* o, long ldo,
                                const float* weight, const float* shift, const float* gate, long ldg, long gate_rows,
                                const void* u, long ldu, float scale, float p, const unsigned long long* rng,
                                const float* next_weight, void* dx, long lddx, void* d_o, long lddo, float* dgate,
                                long lddg, float* dweight, float* dshift, float* dnext_weight, float* dnext_shift,
                                long m, int n, int norm, int next_norm, float eps, int dtype, void* workspace,
                                size_t ws_bytes, hipStream_t stream) {
  OIDN_TRY(check_type(dtype));
  OIDN_TRY(check_size("x", m, n));
  OIDN_TRY(check_norm("norm", norm, OIDN_NORM_NONE));
  OIDN_TRY(check_norm("next_norm", next_norm, OIDN_NORM_NONE));
  OIDN_TRY(check_eps(eps));
  NormBackArgs a{};
  OIDN_TRY(check_dropout(p, rng, a.drop));
  OIDN_TRY(check_gate("gate", gate, ldg, n, gate_rows));
  if (dgate && !gate) return fail(OIDN_E_INVALID, "dgate without gate");
  OIDN_TRY(check_gate("dgate", dgate, lddg, n, gate_rows));
  OIDN_TRY(check_vectors({weight, shift, next_weight, dweight, dshift, dnext_weight, dnext_shift}));
  const bool next = next_norm != OIDN_NORM_NONE;
  if (!next && (dv || dnext_weight || dnext_shift))
    return fail(OIDN_E_INVALID, "dv, dnext_weight or dnext_shift without next_norm");
  a.sums[0] = dweight;
  a.sums[1] = dshift;
  a.sums[2] = dnext_weight;
  a.sums[3] = dnext_shift;
  if (m == 0) {
    OIDN_TRY(zero_sums(a.sums, n, stream));
    return clear_error();
  }
  OIDN_TRY(check_matrix("du", du, lddu, n, dtype, next));
  OIDN_TRY(check_matrix("dv", dv, lddv, n, dtype, !next));
  OIDN_TRY(check_matrix("o", o, ldo, n, dtype, false));
  if (next) OIDN_TRY(check_matrix("u", u, ldu, n, dtype, false));
  OIDN_TRY(check_matrix("dx", dx, lddx, n, dtype, true));
  OIDN_TRY(check_matrix("d_o", d_o, lddo, n, dtype, true));
  a.du = du;
  a.lddu = lddu;
  a.dv = dv;
  a.lddv = lddv;
  a.o = o;
  a.ldo = ldo;
  a.weight = weight;
  a.shift = shift;
  a.gate = gate;
  a.ldg = ldg;
  a.u = u;
  a.ldu = ldu;
  a.scale = scale;
  a.next_weight = next_weight;
  a.dx = dx;
  a.lddx = lddx;
  a.d_o = d_o;
  a.lddo = lddo;
  a.dgate = dgate;
  a.lddg = lddg;
  a.m = m;
  a.n = n;
  a.norm = norm;
  a.next_norm = next_norm;
  a.eps = eps;
  OIDN_TRY(run_back(a, gate ? gate_rows : 0, dtype, workspace, ws_bytes, stream));
  return clear_error();
}

int oidn_dropout(const void* x, long ldx, const void* residual, long ldr, void* y, long ldy, long m, int n, float p,
                 const unsigned long long* rng, int dtype, hipStream_t stream) {
  OIDN_TRY(check_type(dtype));
  OIDN_TRY(check_size("x", m, n));
  Dropout d{};
  OIDN_TRY(check_dropout(p, rng, d));
  if (m == 0) return clear_error();
  OIDN_TRY(check_matrix("x", x, ldx, n, dtype, false));
  OIDN_TRY(check_matrix("residual", residual, ldr, n, dtype, true));
  OIDN_TRY(check_matrix("y", y, ldy, n, dtype, false));
  OIDN_TRY(ran(launch_dropout(x, ldx, residual, ldr, y, ldy, m, n, d, dtype, stream), "dropout launch"));
  return clear_error();
}

}  // extern "C"
