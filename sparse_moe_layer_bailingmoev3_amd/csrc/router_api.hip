// C-ABI host layer of the operators that train the router (balance loss, backward pass) and of the
// gradient norm with clipping.  Arguments are checked here, before any HIP call; the declarations and
// contracts are in include/moe.h.
#include <string.h>

#include <algorithm>
#include <cmath>
#include <new>
#include <vector>

#include "host_checks.h"

namespace {

constexpr int32_t MAX_SEQ = 65536;
constexpr int32_t MAX_HIDDEN = 65536;  // of the products: 32 rows of a tile within 32-bit offsets, tiles counted in 32 bits

size_t align256(size_t v) { return (v + 255) & ~(size_t)255; }

// one sequence of all tokens where none are given
moe_status_t check_sequences(int64_t T, const moe_sequences_t* q, moe::SeqArgs* out) {
  out->offsets = out->lens = nullptr;
  out->n = 1;
  out->T = (int)T;
  if (!q) return MOE_OK;
  if (q->n_seq < 1) return fail(MOE_ERR_INVALID_ARG, "n_seq %d must be >= 1", q->n_seq);
  if (q->n_seq > MAX_SEQ) return fail(MOE_ERR_UNSUPPORTED, "n_seq %d is above %d", q->n_seq, MAX_SEQ);
  if (!q->offsets && q->n_seq != 1) return fail(MOE_ERR_INVALID_ARG, "%d sequences need offsets", q->n_seq);
  MOE_TRY(need_opt(q->offsets, "sequence offsets", 4));
  MOE_TRY(need_opt(q->lens, "sequence lens", 4));
  out->offsets = q->offsets;
  out->lens = q->lens;
  out->n = q->n_seq;
  return MOE_OK;
}

struct Layout {
  size_t done, parts, psum, pcnt, balance;  // balance loss
  size_t bf, live, hf, wt, hexp, wexp, part, backward;  // backward pass
};
// chunks: of the balance loss; parts: of the weight gradient (1: not split)
Layout layout(const moe_config_t* c, int64_t T, int n_seq, int64_t chunks, int parts) {
  const size_t E = c->num_experts, slots = (size_t)chunks + n_seq;
  Layout L{};
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off += align256(bytes);
    return o;
  };
  L.done = take(4);
  L.parts = take((size_t)n_seq * (E / 64) * 8);
  L.psum = take(slots * E * 4);
  L.pcnt = take(slots * E * 4);
  L.balance = off;
  off = 0;
  const size_t H = c->hidden_size, end = moe::ROUTER_TILE_MAX;
  L.bf = take((size_t)T * E * 6);
  L.live = take(T + 32);  // (read in words to the end of a step)
  L.hf = take(2 * (size_t)moe::plane_size(T, (int)E) * 2);
  L.wt = take(2 * (size_t)moe::plane_size(H, (int)E) * 2);
  L.hexp = take((T + end) * 4);
  L.wexp = take((H + end) * 4);
  L.part = take((parts > 1 ? parts : 0) * E * H * 4);
  L.backward = off;
  return L;
}

moe_status_t check_ws(const void* ws, size_t have, size_t want) {
  if (!ws) return fail(MOE_ERR_WORKSPACE, "workspace must not be NULL");
  if (!aligned(ws, 256)) return fail(MOE_ERR_ALIGNMENT, "workspace is not 256-byte aligned");
  if (have < want) return fail(MOE_ERR_WORKSPACE, "workspace has %zu bytes, %zu needed", have, want);
  return MOE_OK;
}

struct Spans {
  Span v[12];
  int n = 0;
  void add(const void* p, int64_t count, int64_t size, const char* name) {
    if (p && count > 0) v[n++] = span(p, count, size, name);
  }
};
// every output is apart from every input and from the other outputs
moe_status_t all_apart(const Spans& out, const Spans& in) {
  for (int i = 0; i < out.n; ++i) {
    for (int j = 0; j < in.n; ++j) MOE_TRY(apart(out.v[i], in.v[j]));
    for (int j = 0; j < i; ++j) MOE_TRY(apart(out.v[i], out.v[j]));
  }
  return MOE_OK;
}
void add_sequences(Spans& s, const moe::SeqArgs& q) {
  s.add(q.offsets, (int64_t)q.n + 1, 4, "sequence offsets");
  s.add(q.lens, q.n, 4, "sequence lens");
}

moe_status_t check_grad_plan(const moe_grad_plan_t* p, const void* image) {
  if (!p) return fail(MOE_ERR_INVALID_ARG, "plan must not be NULL");
  if (p->n_tensors < 0 || p->n_chunks < 0 || p->n_chunks > MAX_ROWS)
    return fail(MOE_ERR_INVALID_ARG, "plan was not filled by moe_grad_plan");
  return p->n_chunks ? need(image, "image") : MOE_OK;
}

}  // namespace

namespace moe {
moe_status_t check_route_apart(const moe_config_t* c, int64_t T, const void* x, const float* router_w, const float* bias,
                               const int32_t* topk_idx, const float* topk_w, const float* logits, const void* ws, size_t ws_bytes) {
  const int64_t E = c->num_experts, K = c->num_experts_per_tok, H = c->hidden_size;
  Spans in, out;
  in.add(x, T * H, 2, "x");
  in.add(router_w, E * H, 4, "router_w");
  in.add(bias, E, 4, "expert_bias");
  out.add(topk_idx, T * K, 4, "topk_idx");
  out.add(topk_w, T * K, 4, "topk_w");
  out.add(logits, T * E, 4, "logits");
  out.add(ws, (int64_t)ws_bytes, 1, "workspace");
  return all_apart(out, in);
}
}  // namespace moe

extern "C" {

moe_status_t moe_router_workspace_size(const moe_config_t* cfg, int64_t T, int32_t n_seq, size_t* bytes) {
  moe::set_last_error("");
  MOE_TRY(moe::check_config(cfg, T));
  if (!bytes) return fail(MOE_ERR_INVALID_ARG, "bytes must not be NULL");
  if (n_seq < 1) return fail(MOE_ERR_INVALID_ARG, "n_seq %d must be >= 1", n_seq);
  if (n_seq > MAX_SEQ) return fail(MOE_ERR_UNSUPPORTED, "n_seq %d is above %d", n_seq, MAX_SEQ);
  // of any call, also for fewer tokens, of which some take more parts or chunks
  const Layout L = layout(cfg, T, n_seq, moe::balance_chunks_bound(T, n_seq),
                          moe::router_grad_parts_bound(T, cfg->num_experts, cfg->hidden_size));
  *bytes = std::max(L.balance, L.backward);
  return MOE_OK;
}

moe_status_t moe_balance_loss(const moe_config_t* cfg, int64_t T, const moe_sequences_t* sequences, const float* logits,
                              const int32_t* topk_idx, float coef, int32_t* counts, float* probs, float* loss, void* ws,
                              size_t ws_bytes, void* stream) {
  moe::set_last_error("");
  MOE_TRY(moe::check_config(cfg, T));
  moe::BalanceArgs a{};
  MOE_TRY(check_sequences(T, sequences, &a.seq));
  if (!std::isfinite(coef)) return fail(MOE_ERR_INVALID_ARG, "coef is not finite");
  if (T > 0) {
    MOE_TRY(need(logits, "logits"));
    MOE_TRY(need(topk_idx, "topk_idx"));
  }
  MOE_TRY(need(counts, "counts"));
  MOE_TRY(need(probs, "probs"));
  MOE_TRY(need(loss, "loss", 4));
  const int64_t E = cfg->num_experts, K = cfg->num_experts_per_tok, B = a.seq.n;
  a.chunk = moe::balance_chunk(T, a.seq.n);
  const Layout L = layout(cfg, T, a.seq.n, std::max<int64_t>((T + a.chunk - 1) / a.chunk, 1), 1);
  MOE_TRY(check_ws(ws, ws_bytes, L.balance));
  Spans in, out;
  in.add(logits, T * E, 4, "logits");
  in.add(topk_idx, T * K, 4, "topk_idx");
  add_sequences(in, a.seq);
  out.add(counts, B * E, 4, "counts");
  out.add(probs, B * E, 4, "probs");
  out.add(loss, 1, 4, "loss");
  out.add(ws, (int64_t)L.balance, 1, "workspace");
  MOE_TRY(all_apart(out, in));
  char* w = (char*)ws;
  a.E = (int)E;
  a.K = (int)K;
  a.coef = coef;
  a.logits = logits;
  a.topk_idx = topk_idx;
  a.done = (int*)(w + L.done);
  a.part = (double*)(w + L.parts);
  a.psum = (float*)(w + L.psum);
  a.pcnt = (int32_t*)(w + L.pcnt);
  a.counts = counts;
  a.probs = probs;
  a.loss = loss;
  return done(moe::launch_balance(a, (hipStream_t)stream), "balance loss launch");
}

moe_status_t moe_router_backward(const moe_config_t* cfg, int64_t T, const moe_sequences_t* sequences,
                                 const moe_router_backward_t* g, void* ws, size_t ws_bytes, void* stream) {
  moe::set_last_error("");
  MOE_TRY(moe::check_config(cfg, T));
  if (!g) return fail(MOE_ERR_INVALID_ARG, "the gradients must not be NULL");
  moe::DlogitsArgs d{};
  MOE_TRY(check_sequences(T, sequences, &d.seq));
  // (without tokens an array may have no address)
  if (T > 0 && !g->dtopk_w && !g->counts) return fail(MOE_ERR_INVALID_ARG, "dtopk_w or counts must be given");
  if (T > 0 && !g->dlogits && !g->drouter_w && !g->dx) return fail(MOE_ERR_INVALID_ARG, "dlogits, drouter_w or dx must be given");
  if ((g->drouter_w || g->dx) && cfg->hidden_size > MAX_HIDDEN)
    return fail(MOE_ERR_UNSUPPORTED, "hidden_size %d is above %d", cfg->hidden_size, MAX_HIDDEN);
  if (!std::isfinite(g->balance_coef)) return fail(MOE_ERR_INVALID_ARG, "balance_coef is not finite");
  if (g->dx && g->dx_dtype != MOE_DTYPE_BF16 && g->dx_dtype != MOE_DTYPE_FP32)
    return fail(MOE_ERR_INVALID_ARG, "dx: dtype %d is unknown", g->dx_dtype);
  if (g->dx && g->accumulate_x && g->dx_dtype != MOE_DTYPE_FP32)
    return fail(MOE_ERR_UNSUPPORTED, "dx: accumulation needs fp32 (a bf16 sum would round at every call)");
  if (T > 0) {
    MOE_TRY(need(g->logits, "logits"));
    if (g->dtopk_w) MOE_TRY(need(g->topk_idx, "topk_idx"));
    if (g->drouter_w) MOE_TRY(need(g->x, "x"));
    if (g->dx) MOE_TRY(need(g->router_w, "router_w"));
  }
  MOE_TRY(need_opt(g->dtopk_w, "dtopk_w", 16));
  MOE_TRY(need_opt(g->counts, "counts", 16));
  MOE_TRY(need_opt(g->dloss, "dloss", 4));
  MOE_TRY(need_opt(g->dlogits, "dlogits", 16));
  MOE_TRY(need_opt(g->drouter_w, "drouter_w", 16));
  MOE_TRY(need_opt(g->dx, "dx", 16));
  const int64_t E = cfg->num_experts, K = cfg->num_experts_per_tok, H = cfg->hidden_size;
  const bool products = g->drouter_w || g->dx;
  moe::RouterGradPlan plan{};
  if (products) plan = moe::router_grad_plan(T, (int)E, (int)H, g->drouter_w, g->dx);
  const Layout L = layout(cfg, T, d.seq.n, 0, plan.nsplit);
  if (products) MOE_TRY(check_ws(ws, ws_bytes, L.backward));
  Spans in, out;
  in.add(g->logits, T * E, 4, "logits");
  if (g->dtopk_w) in.add(g->topk_idx, T * K, 4, "topk_idx");
  in.add(g->dtopk_w, T * K, 4, "dtopk_w");
  in.add(g->counts, d.seq.n * E, 4, "counts");
  in.add(g->dloss, 1, 4, "dloss");
  if (g->drouter_w) in.add(g->x, T * H, 2, "x");
  if (g->dx) in.add(g->router_w, E * H, 4, "router_w");
  if (g->counts) add_sequences(in, d.seq);
  out.add(g->dlogits, T * E, 4, "dlogits");
  out.add(g->drouter_w, E * H, 4, "drouter_w");
  out.add(g->dx, T * H, dsize(g->dx_dtype), "dx");
  if (products) out.add(ws, (int64_t)L.backward, 1, "workspace");
  MOE_TRY(all_apart(out, in));
  char* w = (char*)ws;
  d.E = (int)E;
  d.K = (int)K;
  d.norm = cfg->norm_topk_prob != 0;
  d.scale = cfg->routed_scaling_factor;
  d.logits = g->logits;
  d.topk_idx = g->topk_idx;
  d.dtopk_w = g->dtopk_w;
  d.counts = g->counts;
  d.coef = g->balance_coef;
  d.dloss = g->dloss;
  d.dlogits = g->dlogits;
  if (g->drouter_w) {
    d.bf = (uint16_t*)(w + L.bf);
    d.live = (uint8_t*)(w + L.live);
  }
  if (g->dx) {
    d.hf = (uint16_t*)(w + L.hf);
    d.hexp = (int32_t*)(w + L.hexp);
    d.w = g->router_w;
    d.H = (int)H;
    d.wt = (uint16_t*)(w + L.wt);
    d.wexp = (int32_t*)(w + L.wexp);
  }
  MOE_TRY(done(moe::launch_dlogits(d, (hipStream_t)stream), "router backward launch"));
  if (!products) return MOE_OK;
  moe::RouterGradArgs a{};
  a.plan = plan;
  a.T = (int)T;
  a.E = (int)E;
  a.H = (int)H;
  a.dl = d.bf;
  a.live = d.live;
  a.x = (const uint16_t*)g->x;
  a.part = (float*)(w + L.part);
  a.dh = d.hf;
  a.dexp = d.hexp;
  a.wt = d.wt;
  a.wexp = d.wexp;
  a.dw = g->drouter_w;
  a.acc_w = g->accumulate_w != 0;
  a.dx = g->dx;
  a.dx_f32 = g->dx_dtype == MOE_DTYPE_FP32;
  a.acc_x = g->accumulate_x != 0;
  return done(moe::launch_router_grad(a, (hipStream_t)stream), "router gradient launch");
}

moe_status_t moe_grad_plan(int64_t n_tensors, const moe_grad_tensor_t* tensors, moe_grad_plan_t* plan, void* image,
                           size_t image_bytes) {
  moe::set_last_error("");
  if (!plan) return fail(MOE_ERR_INVALID_ARG, "plan must not be NULL");
  if (n_tensors < 0) return fail(MOE_ERR_INVALID_ARG, "n_tensors = %lld must be >= 0", (long long)n_tensors);
  if (n_tensors > MAX_ROWS) return fail(MOE_ERR_UNSUPPORTED, "n_tensors = %lld is too large", (long long)n_tensors);
  if (n_tensors && !tensors) return fail(MOE_ERR_INVALID_ARG, "tensors must not be NULL");
  int64_t chunks = 0;
  for (int64_t i = 0; i < n_tensors; ++i) {
    const moe_grad_tensor_t& t = tensors[i];
    for (int32_t d : {t.grad_dtype, t.out_dtype})
      if (d != MOE_DTYPE_BF16 && d != MOE_DTYPE_FP32) return fail(MOE_ERR_INVALID_ARG, "tensor %lld: dtype %d is unknown", (long long)i, d);
    if (t.numel < 0) return fail(MOE_ERR_INVALID_ARG, "tensor %lld: numel = %lld must be >= 0", (long long)i, (long long)t.numel);
    if (t.numel > ((int64_t)1 << 40)) return fail(MOE_ERR_UNSUPPORTED, "tensor %lld: numel = %lld is too large", (long long)i, (long long)t.numel);
    if (t.numel == 0) continue;
    char name[64];
    snprintf(name, sizeof(name), "tensor %lld: grad", (long long)i);
    MOE_TRY(need(t.grad, name));
    snprintf(name, sizeof(name), "tensor %lld: out", (long long)i);
    MOE_TRY(need_opt(t.out, name, 16));
    if ((!t.out || t.out == t.grad) && t.out_dtype != t.grad_dtype)
      return fail(MOE_ERR_INVALID_ARG, "tensor %lld: a gradient clipped in place keeps its type", (long long)i);
    chunks += (t.numel + moe::GRAD_CHUNK - 1) / moe::GRAD_CHUNK;
  }
  if (chunks > MAX_ROWS) return fail(MOE_ERR_UNSUPPORTED, "%lld values are too many for one plan", (long long)(chunks * moe::GRAD_CHUNK));
  plan->n_tensors = n_tensors;
  plan->n_chunks = chunks;
  plan->workspace_bytes = moe::GRAD_MAX_PARTIALS * sizeof(double);
  plan->image_bytes = sizeof(moe::GradHeader) + (size_t)chunks * sizeof(moe::GradChunk);
  if (!image) return MOE_OK;
  if (image_bytes < plan->image_bytes)
    return fail(MOE_ERR_WORKSPACE, "plan image has %zu bytes, %zu needed", image_bytes, plan->image_bytes);

  // what the clipping writes must be apart from everything else (in place: one array)
  try {
    struct Range { uintptr_t lo, hi; int64_t tensor; bool written; };
    std::vector<Range> all;
    for (int64_t i = 0; i < n_tensors; ++i) {
      const moe_grad_tensor_t& t = tensors[i];
      if (!t.numel) continue;
      const bool in_place = !t.out || t.out == t.grad;
      all.push_back({(uintptr_t)t.grad, (uintptr_t)t.grad + (uintptr_t)(t.numel * dsize(t.grad_dtype)), i, in_place});
      if (!in_place) all.push_back({(uintptr_t)t.out, (uintptr_t)t.out + (uintptr_t)(t.numel * dsize(t.out_dtype)), i, true});
    }
    std::sort(all.begin(), all.end(), [](const Range& a, const Range& b) { return a.lo < b.lo; });
    uintptr_t end_any = 0, end_written = 0;
    for (const Range& r : all) {
      if (r.lo < end_written || (r.written && r.lo < end_any))
        return fail(MOE_ERR_INVALID_ARG, "tensor %lld: an array that the clipping writes overlaps another", (long long)r.tensor);
      end_any = std::max(end_any, r.hi);
      if (r.written) end_written = std::max(end_written, r.hi);
    }
  } catch (const std::bad_alloc&) {
    return fail(MOE_ERR_INVALID_ARG, "no host memory for %lld tensors", (long long)n_tensors);
  }

  uint8_t* at = (uint8_t*)image;
  const moe::GradHeader hd{moe::GRAD_MAGIC, n_tensors, chunks, 0};
  memcpy(at, &hd, sizeof(hd));
  at += sizeof(hd);
  for (int64_t i = 0; i < n_tensors; ++i) {
    const moe_grad_tensor_t& t = tensors[i];
    const int32_t flags = (t.grad_dtype == MOE_DTYPE_FP32 ? moe::GRAD_IN_F32 : 0) | (t.out_dtype == MOE_DTYPE_FP32 ? moe::GRAD_OUT_F32 : 0);
    for (int64_t c = 0; c < t.numel; c += moe::GRAD_CHUNK) {
      const moe::GradChunk k{(const char*)t.grad + c * dsize(t.grad_dtype), (char*)(t.out ? t.out : t.grad) + c * dsize(t.out_dtype),
                             (int32_t)std::min<int64_t>(t.numel - c, moe::GRAD_CHUNK), flags};
      memcpy(at, &k, sizeof(k));
      at += sizeof(k);
    }
  }
  return MOE_OK;
}

moe_status_t moe_grad_norm(const moe_grad_plan_t* plan, const void* image, double max_norm, double scale, float* norm, float* coef,
                           void* ws, size_t ws_bytes, void* stream) {
  moe::set_last_error("");
  MOE_TRY(check_grad_plan(plan, image));
  if (!(max_norm >= 0)) return fail(MOE_ERR_INVALID_ARG, "max_norm %g must be >= 0", max_norm);
  if (!std::isfinite(scale)) return fail(MOE_ERR_INVALID_ARG, "scale is not finite");
  MOE_TRY(need(norm, "norm", 4));
  MOE_TRY(need_opt(coef, "coef", 4));
  const size_t want = moe::GRAD_MAX_PARTIALS * sizeof(double);
  MOE_TRY(check_ws(ws, ws_bytes, want));
  Spans in, out;
  in.add(image, (int64_t)plan->image_bytes, 1, "image");
  out.add(norm, 1, 4, "norm");
  out.add(coef, 1, 4, "coef");
  out.add(ws, (int64_t)want, 1, "workspace");
  MOE_TRY(all_apart(out, in));
  moe::GradArgs a{};
  a.image = (const uint8_t*)image;
  a.n_tensors = plan->n_tensors;
  a.n_chunks = plan->n_chunks;
  a.scale = scale;
  a.max_norm = max_norm;
  a.partial = (double*)ws;
  a.norm = norm;
  a.coef_out = coef;
  return done(moe::launch_grad_norm(a, (hipStream_t)stream), "gradient norm launch");
}

moe_status_t moe_grad_clip(const moe_grad_plan_t* plan, const void* image, const float* coef, void* stream) {
  moe::set_last_error("");
  MOE_TRY(check_grad_plan(plan, image));
  MOE_TRY(need(coef, "coef", 4));
  moe::GradArgs a{};
  a.image = (const uint8_t*)image;
  a.n_tensors = plan->n_tensors;
  a.n_chunks = plan->n_chunks;
  a.coef = coef;
  return done(moe::launch_grad_clip(a, (hipStream_t)stream), "gradient clipping launch");
}

}  // extern "C"
