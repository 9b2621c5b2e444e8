// Argument checks shared by the host layers of the training operators (each file has its own copy of
// these small functions: an unnamed namespace).
#pragma once
#include <hip/hip_runtime.h>
#include <stdarg.h>
#include <stdint.h>
#include <stdio.h>

#include "moe.h"
#include "moe_internal.h"

namespace {

moe_status_t fail(moe_status_t st, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  moe::set_last_error(buf);
  return st;
}

moe_status_t done(hipError_t e, const char* what) {
  return e == hipSuccess ? MOE_OK : fail(MOE_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

#define MOE_TRY(expr)                        \
  do {                                       \
    const moe_status_t st_ = (expr);         \
    if (st_ != MOE_OK) return st_;           \
  } while (0)

moe_status_t need(const void* p, const char* name, uintptr_t align = 16) {
  if (!p) return fail(MOE_ERR_INVALID_ARG, "%s must not be NULL", name);
  if (!aligned(p, align)) return fail(MOE_ERR_ALIGNMENT, "%s is not %d-byte aligned", name, (int)align);
  return MOE_OK;
}

moe_status_t need_opt(const void* p, const char* name, uintptr_t align) {
  return p ? need(p, name, align) : MOE_OK;
}

constexpr int64_t MAX_ROWS = ((int64_t)1 << 31) - 1;

// a row-major matrix in memory: its address range, the bytes of a row and between rows
struct Span {
  uintptr_t lo, hi, row, stride;
  const char* name;
};
Span span(const void* p, int64_t rows, int64_t ld, int64_t cols, int64_t size, const char* name) {
  const uintptr_t b = (uintptr_t)p;
  return {b, rows > 0 ? b + (uintptr_t)(((rows - 1) * ld + cols) * size) : b, (uintptr_t)(cols * size), (uintptr_t)(ld * size), name};
}
Span span(const void* p, int64_t n, int64_t size, const char* name) { return span(p, 1, n, n, size, name); }
// Whether an output shares no byte with another array.  Side by side in the rows of one buffer (equal
// strides, or a single row between the rows of the other) is apart.
moe_status_t apart(const Span& out, const Span& in) {
  if (out.lo >= in.hi || in.lo >= out.hi || out.lo == out.hi || in.lo == in.hi) return MOE_OK;
  const bool out_row = out.hi - out.lo == out.row, in_row = in.hi - in.lo == in.row;
  if (out.stride == in.stride || out_row || in_row) {
    const uintptr_t s = out_row ? in.stride : out.stride, d = (out.lo % s + s - in.lo % s) % s;  // out's place in in's rows
    if (d >= in.row && d + out.row <= s) return MOE_OK;
  }
  return fail(MOE_ERR_INVALID_ARG, "%s overlaps %s", out.name, in.name);
}

inline int64_t dsize(int32_t dtype) { return dtype == MOE_DTYPE_FP32 ? 4 : 2; }

}  // namespace
