// What the host sides of the operators over activation rows share: argument
// checks, status and workspace regions.  Nothing here throws.
#pragma once

#include <cstdarg>
#include <cstdio>

#include "../../include/oidn_mi355x.h"
#include "dense.h"

namespace oidn {
namespace {

inline int fail(int code, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  return set_error(code, buf);
}
inline int ran(hipError_t e, const char* what) {
  return e == hipSuccess ? OIDN_OK : fail(OIDN_E_HIP, "%s: %s", what, hipGetErrorString(e));
}

// Limits: columns index with 32-bit ints, rows count with them where tiles do.
// Whether a call's products fit a launch's grid is a matter of its plan
// (check_launch).
constexpr long kMaxColumns = 1L << 24;
constexpr long kMaxRows = (1L << 31) - 1;
constexpr long kMaxElements = 1L << 38;

inline size_t esize(int dtype) { return dtype == OIDN_F32 ? 4 : 2; }
inline size_t bytes_of(long rows, long cols, int dtype) {
  return align256((size_t)rows * (size_t)cols * esize(dtype));
}

inline int check_type(int dtype) {
  if (dtype == OIDN_F32 || dtype == OIDN_F16 || dtype == OIDN_BF16) return OIDN_OK;
  return fail(OIDN_E_INVALID, "unknown dtype %d", dtype);
}
inline int check_size(const char* name, long rows, long cols) {
  if (rows < 0 || cols < 1) return fail(OIDN_E_INVALID, "%s: %ld x %ld is not a size", name, rows, cols);
  if (rows > kMaxRows || cols > kMaxColumns || rows > kMaxElements / cols)
    return fail(OIDN_E_UNSUPPORTED, "%s: %ld x %ld is larger than the kernels index", name, rows, cols);
  return OIDN_OK;
}
inline int check_act(int act) {
  if (act >= OIDN_ACT_NONE && act <= OIDN_ACT_GELU) return OIDN_OK;
  return fail(OIDN_E_INVALID, "unknown activation %d", act);
}
inline int check_flags(unsigned flags, unsigned known) {
  if ((flags & ~known) == 0) return OIDN_OK;
  return fail(OIDN_E_INVALID, "unknown flags 0x%x", flags & ~known);
}
inline int check_aligned(const char* name, const void* p, size_t to) {
  if (reinterpret_cast<uintptr_t>(p) % to == 0) return OIDN_OK;
  return fail(OIDN_E_INVALID, "%s must be aligned to %zu bytes", name, to);
}
// A matrix of `cols` columns at row pitch ld; may_be_null: absent is fine.
inline int check_matrix(const char* name, const void* p, long ld, long cols, int dtype, bool may_be_null) {
  if (!p) return may_be_null ? OIDN_OK : fail(OIDN_E_INVALID, "null pointer: %s", name);
  if (ld < cols) return fail(OIDN_E_INVALID, "row pitch %ld of %s is less than its %ld columns", ld, name, cols);
  if (ld > (1L << 32)) return fail(OIDN_E_UNSUPPORTED, "row pitch %ld of %s is above 2^32", ld, name);
  return check_aligned(name, p, esize(dtype));
}
inline int check_blob(const char* name, const void* p) {
  if (!p) return fail(OIDN_E_INVALID, "null pointer: %s", name);
  return check_aligned(name, p, 16);
}
inline int check_workspace(const void* ws, size_t have, size_t need) {
  if (need == 0) return OIDN_OK;
  if (!ws) return fail(OIDN_E_INVALID, "null pointer: workspace");
  const int rc = check_aligned("workspace", ws, 16);
  if (rc) return rc;
  if (have < need)
    return fail(OIDN_E_WORKSPACE, "workspace of %zu bytes is smaller than the %zu needed", have, need);
  return OIDN_OK;
}
#define OIDN_TRY(expr)        \
  do {                        \
    const int rc_ = (expr);   \
    if (rc_) return rc_;      \
  } while (0)

// `blocks`: of the largest launch of a call.
inline int check_launch(long blocks) {
  if (blocks <= kMaxWorkgroups) return OIDN_OK;
  return fail(OIDN_E_UNSUPPORTED, "%ld workgroups are more than the %ld of a launch", blocks, kMaxWorkgroups);
}
// The plain epilogue: store, with `add` (may be null) added.
inline EpilogueArgs store_to(void* y, long ldy, const void* add, long ldadd) {
  EpilogueArgs e{};
  e.y = y;
  e.ldy = ldy;
  e.res = add;
  e.ldr = ldadd;
  return e;
}

// Workspace regions, handed out in order.
struct Regions {
  char* base;
  size_t used;
  void* take(size_t bytes) {
    void* p = base ? base + used : nullptr;
    used += bytes;
    return p;
  }
};

}  // namespace
}  // namespace oidn
