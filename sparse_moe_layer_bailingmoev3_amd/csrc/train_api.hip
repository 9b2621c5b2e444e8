// C-ABI host layer of the training operators: the products grouped by expert, SwiGLU with routing
// weights, and the AdamW step.  Arguments are checked here, before any HIP call; the declarations
// and contracts are in include/moe.h.
#include <stdarg.h>
#include <stdio.h>
#include <string.h>

#include <algorithm>
#include <cmath>
#include <new>
#include <vector>

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
constexpr int64_t MAX_LD = (int64_t)1 << 22;  // a tile's rows stay within a 32-bit offset
constexpr int32_t MAX_FEATURES = 65536, MAX_GROUPS = 1025;

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

moe_status_t check_ld(int64_t ld, int64_t cols, const char* name) {
  if (ld < cols) return fail(MOE_ERR_INVALID_ARG, "%s: row stride %lld is below the %lld columns", name, (long long)ld, (long long)cols);
  if (ld % 8) return fail(MOE_ERR_UNSUPPORTED, "%s: row stride %lld is not a multiple of 8", name, (long long)ld);
  if (ld > MAX_LD) return fail(MOE_ERR_UNSUPPORTED, "%s: row stride %lld is too large", name, (long long)ld);
  return MOE_OK;
}

moe_status_t check_groups(const moe_groups_t* g) {
  if (!g) return fail(MOE_ERR_INVALID_ARG, "groups must not be NULL");
  if (g->groups < 1) return fail(MOE_ERR_INVALID_ARG, "groups %d must be >= 1", g->groups);
  if (g->groups > MAX_GROUPS) return fail(MOE_ERR_UNSUPPORTED, "groups %d is above %d", g->groups, MAX_GROUPS);
  if (g->out_features < 1 || g->in_features < 1)
    return fail(MOE_ERR_INVALID_ARG, "out_features %d and in_features %d must be >= 1", g->out_features, g->in_features);
  if (g->out_features % 8 || g->in_features % 8)
    return fail(MOE_ERR_UNSUPPORTED, "out_features %d and in_features %d must be multiples of 8", g->out_features, g->in_features);
  if (g->out_features > MAX_FEATURES || g->in_features > MAX_FEATURES)
    return fail(MOE_ERR_UNSUPPORTED, "out_features %d or in_features %d is above %d", g->out_features, g->in_features, MAX_FEATURES);
  if ((int64_t)g->out_features * g->in_features >= (int64_t)0x7FFFFF80)
    return fail(MOE_ERR_UNSUPPORTED, "weights of %d x %d values are above 4 GiB a group", g->out_features, g->in_features);
  if (g->rows < 0) return fail(MOE_ERR_INVALID_ARG, "rows = %lld must be >= 0", (long long)g->rows);
  // the tiles of a partial last row may step past the last position
  if (g->rows > MAX_ROWS - 4096) return fail(MOE_ERR_UNSUPPORTED, "rows = %lld is too large for 32-bit positions", (long long)g->rows);
  return need(g->offsets, "offsets", 4);
}

moe_status_t check_rows(const moe_groups_t* g, const moe_rows_t* r, int64_t cols, const char* name) {
  if (!r) return fail(MOE_ERR_INVALID_ARG, "%s must not be NULL", name);
  if (r->rows < 0) return fail(MOE_ERR_INVALID_ARG, "%s: rows = %lld must be >= 0", name, (long long)r->rows);
  if (r->rows > MAX_ROWS) return fail(MOE_ERR_UNSUPPORTED, "%s: rows = %lld is too large", name, (long long)r->rows);
  if (!r->row_map && r->rows < g->rows)
    return fail(MOE_ERR_INVALID_ARG, "%s: %lld rows for %lld positions without a row map", name, (long long)r->rows, (long long)g->rows);
  MOE_TRY(check_ld(r->ld, cols, name));
  MOE_TRY(need_opt(r->row_map, "row_map", 4));
  if (r->rows > 0) MOE_TRY(need(r->data, name));
  return MOE_OK;
}

moe_status_t check_out(int32_t dtype, int32_t accumulate, const void* p, const char* name) {
  if (dtype != MOE_DTYPE_BF16 && dtype != MOE_DTYPE_FP32) return fail(MOE_ERR_INVALID_ARG, "%s: dtype %d is unknown", name, dtype);
  if (accumulate && dtype != MOE_DTYPE_FP32)
    return fail(MOE_ERR_UNSUPPORTED, "%s: accumulation needs fp32 (a bf16 sum would round at every call)", name);
  return need(p, name);
}

moe::RowsArg rows_arg(const moe_rows_t* r) {
  return {(const uint16_t*)r->data, (int32_t)r->rows, r->ld, r->row_map};
}
int64_t dsize(int32_t dtype) { return dtype == MOE_DTYPE_FP32 ? 4 : 2; }

// forward (dgrad == false: x, w -> y) and input gradient (dy, w [, dy2, w2] -> dx)
moe_status_t grouped_rows(bool dgrad, const moe_groups_t* g, const moe_rows_t* x, const void* w, const moe_rows_t* x2,
                          const void* w2, void* out, int64_t ldo, int32_t dtype, int32_t accumulate, void* stream) {
  MOE_TRY(check_groups(g));
  const char *xn = dgrad ? "dy" : "x", *on = dgrad ? "dx" : "y";
  const int32_t red = dgrad ? g->out_features : g->in_features, cols = dgrad ? g->in_features : g->out_features;
  if (!x2 != !w2) return fail(MOE_ERR_INVALID_ARG, "dy2 and w2 must be given together");
  if (g->rows == 0) return MOE_OK;
  MOE_TRY(check_rows(g, x, red, xn));
  MOE_TRY(need(w, "w"));
  if (x2) {
    MOE_TRY(check_rows(g, x2, red, "dy2"));
    if (x2->row_map != x->row_map || x2->rows != x->rows || x2->ld != x->ld)
      return fail(MOE_ERR_INVALID_ARG, "dy and dy2 must have the same rows, row stride and row map");
    MOE_TRY(need(w2, "w2"));
  }
  MOE_TRY(check_out(dtype, accumulate, out, on));
  MOE_TRY(check_ld(ldo, cols, on));
  const int64_t wrows = (int64_t)g->groups * g->out_features;
  const Span o = span(out, g->rows, ldo, cols, dsize(dtype), on);
  MOE_TRY(apart(o, span(x->data, x->rows, x->ld, red, 2, xn)));
  MOE_TRY(apart(o, span(w, wrows, g->in_features, g->in_features, 2, "w")));
  if (x2) {
    MOE_TRY(apart(o, span(x2->data, x2->rows, x2->ld, red, 2, "dy2")));
    MOE_TRY(apart(o, span(w2, wrows, g->in_features, g->in_features, 2, "w2")));
  }
  MOE_TRY(apart(o, span(g->offsets, g->groups + 1, 4, "offsets")));
  if (x->row_map) MOE_TRY(apart(o, span(x->row_map, g->rows, 4, "row_map")));
  moe::GroupedArgs a{};
  a.offsets = g->offsets;
  a.groups = g->groups;
  a.rows = (int)g->rows;
  a.N = g->out_features;
  a.K = g->in_features;
  a.x0 = rows_arg(x);
  a.w0 = (const uint16_t*)w;
  if (x2) {
    a.x1 = rows_arg(x2);
    a.w1 = (const uint16_t*)w2;
  }
  a.out = out;
  a.ldo = ldo;
  a.out_f32 = dtype == MOE_DTYPE_FP32;
  a.accumulate = accumulate != 0;
  return done(moe::launch_grouped_rows(a, dgrad, (hipStream_t)stream), "grouped product launch");
}

moe_status_t swiglu_args(int64_t n, int64_t mat_rows, int32_t cols, float limit, const void* gate, const void* up,
                         int64_t ld, const float* row_w, const int32_t* pos) {
  if (n < 0 || mat_rows < 0) return fail(MOE_ERR_INVALID_ARG, "n = %lld and mat_rows = %lld must be >= 0", (long long)n, (long long)mat_rows);
  if (n > MAX_ROWS || mat_rows > MAX_ROWS) return fail(MOE_ERR_UNSUPPORTED, "n or mat_rows is too large for 32-bit positions");
  if (cols < 1) return fail(MOE_ERR_INVALID_ARG, "cols %d must be >= 1", cols);
  if (cols % 8) return fail(MOE_ERR_UNSUPPORTED, "cols %d is not a multiple of 8", cols);
  if (std::isnan(limit)) return fail(MOE_ERR_INVALID_ARG, "limit must not be NaN");
  if (!pos && n > mat_rows) return fail(MOE_ERR_INVALID_ARG, "n = %lld rows of %lld without positions", (long long)n, (long long)mat_rows);
  MOE_TRY(check_ld(ld, cols, "gate and up"));
  MOE_TRY(need_opt(row_w, "row_w", 4));
  MOE_TRY(need_opt(pos, "pos", 4));
  if (n == 0 || mat_rows == 0) return MOE_OK;
  MOE_TRY(need(gate, "gate"));
  return need(up, "up");
}

}  // namespace

extern "C" {

moe_status_t moe_grouped_gemm(const moe_groups_t* groups, const moe_rows_t* x, const void* w, void* y, int64_t ldy,
                              int32_t y_dtype, int32_t accumulate, void* stream) {
  moe::set_last_error("");
  return grouped_rows(false, groups, x, w, nullptr, nullptr, y, ldy, y_dtype, accumulate, stream);
}

moe_status_t moe_grouped_gemm_dgrad(const moe_groups_t* groups, const moe_rows_t* dy, const void* w, const moe_rows_t* dy2,
                                    const void* w2, void* dx, int64_t lddx, int32_t dx_dtype, int32_t accumulate,
                                    void* stream) {
  moe::set_last_error("");
  return grouped_rows(true, groups, dy, w, dy2, w2, dx, lddx, dx_dtype, accumulate, stream);
}

moe_status_t moe_grouped_gemm_wgrad(const moe_groups_t* g, const moe_rows_t* dy, const moe_rows_t* x, void* dw,
                                    int32_t dw_dtype, int32_t accumulate, void* stream) {
  moe::set_last_error("");
  MOE_TRY(check_groups(g));
  MOE_TRY(check_rows(g, dy, g->out_features, "dy"));
  MOE_TRY(check_rows(g, x, g->in_features, "x"));
  MOE_TRY(check_out(dw_dtype, accumulate, dw, "dw"));
  const Span o = span(dw, (int64_t)g->groups * g->out_features, g->in_features, g->in_features, dsize(dw_dtype), "dw");
  MOE_TRY(apart(o, span(dy->data, dy->rows, dy->ld, g->out_features, 2, "dy")));
  MOE_TRY(apart(o, span(x->data, x->rows, x->ld, g->in_features, 2, "x")));
  MOE_TRY(apart(o, span(g->offsets, g->groups + 1, 4, "offsets")));
  if (dy->row_map) MOE_TRY(apart(o, span(dy->row_map, g->rows, 4, "the row map of dy")));
  if (x->row_map) MOE_TRY(apart(o, span(x->row_map, g->rows, 4, "the row map of x")));
  moe::GroupedArgs a{};
  a.offsets = g->offsets;
  a.groups = g->groups;
  a.rows = (int)g->rows;
  a.N = g->out_features;
  a.K = g->in_features;
  a.x0 = rows_arg(dy);
  a.x1 = rows_arg(x);
  a.out = dw;
  a.out_f32 = dw_dtype == MOE_DTYPE_FP32;
  a.accumulate = accumulate != 0;
  return done(moe::launch_grouped_wgrad(a, (hipStream_t)stream), "grouped weight gradient launch");
}

moe_status_t moe_swiglu(int64_t n, int64_t mat_rows, int32_t cols, float limit, const void* gate, const void* up, int64_t ld,
                        const float* row_w, const int32_t* pos, void* h, int64_t ldh, void* stream) {
  moe::set_last_error("");
  MOE_TRY(swiglu_args(n, mat_rows, cols, limit, gate, up, ld, row_w, pos));
  MOE_TRY(check_ld(ldh, cols, "h"));
  if (n == 0 || mat_rows == 0) return MOE_OK;
  MOE_TRY(need(h, "h"));
  const Span o = span(h, mat_rows, ldh, cols, 2, "h");
  MOE_TRY(apart(o, span(gate, mat_rows, ld, cols, 2, "gate")));
  MOE_TRY(apart(o, span(up, mat_rows, ld, cols, 2, "up")));
  if (row_w) MOE_TRY(apart(o, span(row_w, n, 4, "row_w")));
  if (pos) MOE_TRY(apart(o, span(pos, n, 4, "pos")));
  moe::SwigluArgs a{};
  a.n = n;
  a.mat_rows = mat_rows;
  a.cols = cols;
  a.limit = std::isfinite(limit) && limit > 0 ? limit : 0.f;
  a.gate = (const uint16_t*)gate;
  a.up = (const uint16_t*)up;
  a.ld = ld;
  a.row_w = row_w;
  a.pos = pos;
  a.h = (uint16_t*)h;
  a.ldh = ldh;
  return done(moe::launch_swiglu(a, false, (hipStream_t)stream), "SwiGLU launch");
}

moe_status_t moe_swiglu_backward(int64_t n, int64_t mat_rows, int32_t cols, float limit, const void* gate, const void* up,
                                 int64_t ld, const void* dh, int64_t lddh, const float* row_w, const int32_t* pos, void* dgate,
                                 void* dup, int64_t ldd, float* drow_w, void* stream) {
  moe::set_last_error("");
  MOE_TRY(swiglu_args(n, mat_rows, cols, limit, gate, up, ld, row_w, pos));
  MOE_TRY(check_ld(lddh, cols, "dh"));
  MOE_TRY(check_ld(ldd, cols, "dgate and dup"));
  MOE_TRY(need_opt(drow_w, "drow_w", 4));
  if (n == 0) return MOE_OK;
  const Span w = span(row_w, row_w ? n : 0, 4, "row_w"), at = span(pos, pos ? n : 0, 4, "pos");
  const Span dw = span(drow_w, drow_w ? n : 0, 4, "drow_w");
  MOE_TRY(apart(dw, w));
  MOE_TRY(apart(dw, at));
  if (mat_rows > 0) {
    MOE_TRY(need(dh, "dh"));
    MOE_TRY(need(dgate, "dgate"));
    MOE_TRY(need(dup, "dup"));
    const Span in[3] = {span(gate, mat_rows, ld, cols, 2, "gate"), span(up, mat_rows, ld, cols, 2, "up"),
                        span(dh, mat_rows, lddh, cols, 2, "dh")};
    const Span og = span(dgate, mat_rows, ldd, cols, 2, "dgate"), ou = span(dup, mat_rows, ldd, cols, 2, "dup");
    for (const Span& i : in) {
      MOE_TRY(apart(og, i));
      MOE_TRY(apart(ou, i));
      MOE_TRY(apart(dw, i));
    }
    MOE_TRY(apart(og, ou));
    for (const Span& o : {og, ou}) {
      MOE_TRY(apart(o, w));
      MOE_TRY(apart(o, at));
      MOE_TRY(apart(dw, o));
    }
  }
  moe::SwigluArgs a{};
  a.n = n;
  a.mat_rows = mat_rows;
  a.cols = cols;
  a.limit = std::isfinite(limit) && limit > 0 ? limit : 0.f;
  a.gate = (const uint16_t*)gate;
  a.up = (const uint16_t*)up;
  a.ld = ld;
  a.row_w = row_w;
  a.pos = pos;
  a.dh = (const uint16_t*)dh;
  a.ldh = lddh;
  a.dgate = (uint16_t*)dgate;
  a.dup = (uint16_t*)dup;
  a.ldd = ldd;
  a.drow_w = drow_w;
  return done(moe::launch_swiglu(a, true, (hipStream_t)stream), "SwiGLU backward launch");
}

moe_status_t moe_adamw_plan(int64_t n_tensors, const moe_adamw_tensor_t* tensors, int32_t param_dtype, int32_t grad_dtype,
                            int32_t state_format, moe_adamw_plan_t* plan, void* image, size_t image_bytes) {
  moe::set_last_error("");
  if (!plan) return fail(MOE_ERR_INVALID_ARG, "plan must not be NULL");
  if (n_tensors < 0) return fail(MOE_ERR_INVALID_ARG, "n_tensors = %lld must be >= 0", (long long)n_tensors);
  if (n_tensors > MAX_ROWS) return fail(MOE_ERR_UNSUPPORTED, "n_tensors = %lld is too large", (long long)n_tensors);
  if (n_tensors && !tensors) return fail(MOE_ERR_INVALID_ARG, "tensors must not be NULL");
  for (int32_t d : {param_dtype, grad_dtype})
    if (d != MOE_DTYPE_BF16 && d != MOE_DTYPE_FP32) return fail(MOE_ERR_INVALID_ARG, "dtype %d is unknown", d);
  if (state_format != MOE_STATE_FP32 && state_format != MOE_STATE_8BIT)
    return fail(MOE_ERR_INVALID_ARG, "state_format %d is unknown", state_format);
  const bool eight = state_format == MOE_STATE_8BIT;
  // said by the first tensor that holds values (an empty one's arrays may have no address)
  bool master = false;
  for (int64_t i = 0; i < n_tensors; ++i)
    if (tensors[i].numel > 0) {
      master = tensors[i].master != nullptr;
      break;
    }
  if (master && param_dtype == MOE_DTYPE_FP32)
    return fail(MOE_ERR_INVALID_ARG, "master weights belong to bf16 parameters");
  const int64_t psize = dsize(param_dtype), gsize = dsize(grad_dtype), ssize = eight ? 1 : 4;
  int64_t chunks = 0;
  for (int64_t i = 0; i < n_tensors; ++i) {
    const moe_adamw_tensor_t& t = tensors[i];
    if (t.numel < 0) return fail(MOE_ERR_INVALID_ARG, "tensor %lld: numel = %lld must be >= 0", (long long)i, (long long)t.numel);
    if (t.numel > ((int64_t)1 << 40)) return fail(MOE_ERR_UNSUPPORTED, "tensor %lld: numel = %lld is too large", (long long)i, (long long)t.numel);
    if (!std::isfinite(t.weight_decay)) return fail(MOE_ERR_INVALID_ARG, "tensor %lld: weight_decay is not finite", (long long)i);
    if (t.numel == 0) continue;
    char name[64];
    const struct { const void* p; const char* n; uintptr_t al; } ptrs[] = {
        {t.param, "param", 16}, {t.grad, "grad", 16}, {t.exp_avg, "exp_avg", 16}, {t.exp_avg_sq, "exp_avg_sq", 16}};
    for (const auto& p : ptrs) {
      snprintf(name, sizeof(name), "tensor %lld: %s", (long long)i, p.n);
      MOE_TRY(need(p.p, name, p.al));
    }
    if (master != (t.master != nullptr))
      return fail(MOE_ERR_INVALID_ARG, "tensor %lld: master weights must be given for all tensors or for none", (long long)i);
    if (t.master && !aligned(t.master, 16)) return fail(MOE_ERR_ALIGNMENT, "tensor %lld: master is not 16-byte aligned", (long long)i);
    if (eight) {
      snprintf(name, sizeof(name), "tensor %lld: exp_avg_scale", (long long)i);
      MOE_TRY(need(t.exp_avg_scale, name, 4));
      snprintf(name, sizeof(name), "tensor %lld: exp_avg_sq_scale", (long long)i);
      MOE_TRY(need(t.exp_avg_sq_scale, name, 4));
    }
    chunks += (t.numel + moe::ADAMW_CHUNK - 1) / moe::ADAMW_CHUNK;
  }
  if (chunks > MAX_ROWS) return fail(MOE_ERR_UNSUPPORTED, "%lld values are too many for one plan", (long long)(chunks * moe::ADAMW_CHUNK));
  plan->n_tensors = n_tensors;
  plan->n_chunks = chunks;
  plan->flags = (param_dtype == MOE_DTYPE_FP32 ? moe::ADAMW_PARAM_F32 : 0) | (grad_dtype == MOE_DTYPE_FP32 ? moe::ADAMW_GRAD_F32 : 0) |
                (eight ? moe::ADAMW_EIGHT : 0) | (master ? moe::ADAMW_MASTER : 0);
  plan->image_bytes = sizeof(moe::AdamWHeader) + (size_t)n_tensors * sizeof(moe::AdamWTensor) + (size_t)chunks * sizeof(moe::AdamWChunk);
  if (!image) return MOE_OK;
  if (image_bytes < plan->image_bytes)
    return fail(MOE_ERR_WORKSPACE, "plan image has %zu bytes, %zu needed", image_bytes, plan->image_bytes);

  // what the step writes must be apart from everything else it touches
  try {
    struct Range { uintptr_t lo, hi; int64_t tensor; bool written; };
    std::vector<Range> all;
    for (int64_t i = 0; i < n_tensors; ++i) {
      const moe_adamw_tensor_t& t = tensors[i];
      auto add = [&](const void* p, int64_t bytes, bool wr) {
        if (p && bytes) all.push_back({(uintptr_t)p, (uintptr_t)p + (uintptr_t)bytes, i, wr});
      };
      const int64_t blocks = (t.numel + moe::ADAMW_BLOCK - 1) / moe::ADAMW_BLOCK;
      add(t.param, t.numel * psize, true);
      add(t.master, t.numel * 4, true);
      add(t.grad, t.numel * gsize, false);
      add(t.exp_avg, t.numel * ssize, true);
      add(t.exp_avg_sq, t.numel * ssize, true);
      if (eight) {
        add(t.exp_avg_scale, blocks * 4, true);
        add(t.exp_avg_sq_scale, blocks * 4, true);
      }
    }
    std::sort(all.begin(), all.end(), [](const Range& a, const Range& b) { return a.lo < b.lo; });
    uintptr_t end_any = 0, end_written = 0;
    for (const Range& r : all) {
      if (r.lo < end_written || (r.written && r.lo < end_any))
        return fail(MOE_ERR_INVALID_ARG, "tensor %lld: an array that the step writes overlaps another", (long long)r.tensor);
      end_any = std::max(end_any, r.hi);
      if (r.written) end_written = std::max(end_written, r.hi);
    }
  } catch (const std::bad_alloc&) {
    return fail(MOE_ERR_INVALID_ARG, "no host memory for %lld tensors", (long long)n_tensors);
  }

  uint8_t* at = (uint8_t*)image;
  const moe::AdamWHeader hd{moe::ADAMW_MAGIC, n_tensors, chunks, plan->flags};
  memcpy(at, &hd, sizeof(hd));
  at += sizeof(hd);
  for (int64_t i = 0; i < n_tensors; ++i) {
    const moe_adamw_tensor_t& t = tensors[i];
    const moe::AdamWTensor d{t.param, t.master, t.grad, t.exp_avg, t.exp_avg_sq, t.exp_avg_scale, t.exp_avg_sq_scale,
                             t.numel, t.weight_decay, 0};
    memcpy(at, &d, sizeof(d));
    at += sizeof(d);
  }
  for (int64_t i = 0; i < n_tensors; ++i)
    for (int64_t c = 0; c * moe::ADAMW_CHUNK < tensors[i].numel; ++c) {
      const moe::AdamWChunk k{(int32_t)i, (int32_t)c};
      memcpy(at, &k, sizeof(k));
      at += sizeof(k);
    }
  return MOE_OK;
}

moe_status_t moe_adamw_step(const moe_adamw_config_t* cfg, const moe_adamw_plan_t* plan, const void* image, void* stream) {
  moe::set_last_error("");
  if (!cfg || !plan) return fail(MOE_ERR_INVALID_ARG, "cfg and plan must not be NULL");
  if (!(cfg->beta1 >= 0 && cfg->beta1 < 1) || !(cfg->beta2 >= 0 && cfg->beta2 < 1))
    return fail(MOE_ERR_INVALID_ARG, "beta1 %g and beta2 %g must be in [0, 1)", cfg->beta1, cfg->beta2);
  if (!(cfg->eps >= 0) || !std::isfinite(cfg->eps)) return fail(MOE_ERR_INVALID_ARG, "eps %g must be finite and >= 0", cfg->eps);
  if (!cfg->lr_ptr && !std::isfinite(cfg->lr)) return fail(MOE_ERR_INVALID_ARG, "lr is not finite");
  if (!cfg->step_ptr && cfg->step < 1) return fail(MOE_ERR_INVALID_ARG, "step = %lld must be >= 1", (long long)cfg->step);
  MOE_TRY(need_opt(cfg->lr_ptr, "lr_ptr", 4));
  MOE_TRY(need_opt(cfg->step_ptr, "step_ptr", 8));
  MOE_TRY(need_opt(cfg->grad_scale, "grad_scale", 4));
  if (plan->n_tensors < 0 || plan->n_chunks < 0 || plan->n_chunks > MAX_ROWS)
    return fail(MOE_ERR_INVALID_ARG, "plan was not filled by moe_adamw_plan");
  if (plan->n_chunks == 0) return MOE_OK;
  MOE_TRY(need(image, "image"));
  moe::AdamWArgs a{};
  a.image = (const uint8_t*)image;
  a.n_tensors = plan->n_tensors;
  a.n_chunks = plan->n_chunks;
  a.flags = plan->flags;
  a.lr = (float)cfg->lr;
  a.b1 = (float)cfg->beta1;
  a.omb1 = (float)(1.0 - cfg->beta1);
  a.b2 = (float)cfg->beta2;
  a.omb2 = (float)(1.0 - cfg->beta2);
  a.eps = (float)cfg->eps;
  a.beta1 = cfg->beta1;
  a.beta2 = cfg->beta2;
  if (!cfg->step_ptr) {
    a.inv_c1 = (float)(1.0 / (1.0 - std::pow(cfg->beta1, (double)cfg->step)));
    a.inv_c2 = (float)(1.0 / (1.0 - std::pow(cfg->beta2, (double)cfg->step)));
    a.step = (uint32_t)cfg->step;
  }
  a.seed = cfg->seed;
  a.lr_ptr = cfg->lr_ptr;
  a.step_ptr = cfg->step_ptr;
  a.grad_scale = cfg->grad_scale;
  return done(moe::launch_adamw(a, (hipStream_t)stream), "AdamW launch");
}

moe_status_t moe_adamw_dequantise(const uint8_t* codes, const float* scales, int64_t numel, int32_t is_signed, float* out,
                                  void* stream) {
  moe::set_last_error("");
  if (numel < 0) return fail(MOE_ERR_INVALID_ARG, "numel = %lld must be >= 0", (long long)numel);
  if (numel == 0) return MOE_OK;
  MOE_TRY(need(codes, "codes"));
  MOE_TRY(need(scales, "scales", 4));
  MOE_TRY(need(out, "out"));
  const int64_t blocks = (numel + moe::ADAMW_BLOCK - 1) / moe::ADAMW_BLOCK;
  const Span o = span(out, 1, numel, numel, 4, "out");
  MOE_TRY(apart(o, span(codes, 1, numel, numel, 1, "codes")));
  MOE_TRY(apart(o, span(scales, 1, blocks, blocks, 4, "scales")));
  return done(moe::launch_adamw_dequantise(codes, scales, numel, is_signed != 0, out, (hipStream_t)stream), "dequantise launch");
}

}  // extern "C"
