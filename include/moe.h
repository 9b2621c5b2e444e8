/*
 * moe.h -- C ABI of libmoe: the forward pass of one BailingMoeV3 sparse MoE layer
 * (Ling-3.0-flash / Ling-3.0-flash-VL) on one AMD Instinct MI355X (gfx950).
 *
 * What the layer computes (Ling-3.0-flash-VL routing walk-through page, lqnn.cn,
 * "MoE 稀疏路由机制"):
 *   section 三.1  router: one raw score per routed expert from the hidden state, then
 *                 an element-wise sigmoid (score_function "sigmoid");
 *   section 三.3  a per-expert bias is added to the score used for selection
 *                 (moe_router_enable_expert_bias);
 *   section 三.2  the experts form n_group equal groups; keep the topk_group groups
 *                 with the largest in-group maximum, then the num_experts_per_tok best
 *                 experts inside the kept groups;
 *   section 四    router in fp32 (router_dtype), weights renormalised to sum to 1
 *                 (norm_topk_prob) and multiplied by routed_scaling_factor; SwiGLU
 *                 activations optionally clamped (expert_swiglu_limit_list);
 *   section 二    each expert is a SwiGLU FFN (gate, up: hidden -> intermediate;
 *                 down: intermediate -> hidden) and one shared expert sees every token.
 * Routed-expert weights may be MXFP4 (hybrid-attention page, lpnh.cn, table 模型一览).
 * The block is BailingMoeV3SparseMoeBlock (Ling-3.0-flash page, wmrh.cn, section
 * 稀疏MoE设计).
 *
 * Conventions for every entry point
 *   - Pointers marked "device" are HIP device pointers the caller owns; the library
 *     keeps no pointer and no state after a call returns and allocates no device memory
 *     (moe_forward's second stream, below, is the one object it keeps).
 *     Every device pointer must be 16-byte aligned.  Outputs must not alias inputs.
 *   - `stream` is a hipStream_t passed as void* (NULL = the default stream).  Calls
 *     only enqueue work: they return before the GPU finishes, and a fault inside a
 *     kernel surfaces at the caller's next synchronisation as a HIP error.
 *   - Argument errors are found on the host before anything is enqueued and return a
 *     negative status; moe_last_error() then describes the failure (thread-local).
 *   - T (tokens) may be 0: the call returns MOE_OK and enqueues nothing.
 *   - Matrices are row-major.  bf16 tensors are passed as raw 16-bit patterns.
 *   - Results are bitwise reproducible run to run: no reduction uses atomics.
 *
 * Shapes (T tokens; symbols used below)
 *   H = hidden_size, E = num_experts, K = num_experts_per_tok, I = moe_intermediate_size,
 *   S = num_shared_experts (0 or 1), P = T*K + T*S sorted positions.
 */
#ifndef MOE_H_
#define MOE_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  MOE_OK = 0,
  MOE_ERR_INVALID_ARG = -1, /* a size, flag or pointer is out of range or NULL */
  MOE_ERR_UNSUPPORTED = -2, /* a valid configuration these kernels do not implement */
  MOE_ERR_ALIGNMENT = -3,   /* a device pointer is not 16-byte aligned */
  MOE_ERR_WORKSPACE = -4,   /* workspace NULL or smaller than moe_workspace_size() */
  MOE_ERR_HIP = -5          /* a HIP launch failed; moe_last_error() has the HIP text */
} moe_status_t;

typedef enum {
  MOE_WEIGHTS_BF16 = 0,
  MOE_WEIGHTS_MXFP4 = 1,
  MOE_WEIGHTS_MXFP8 = 2,
  MOE_WEIGHTS_MXFP4_TILED = 3, /* MXFP4 in the kernels' tiled order (moe_pack_mxfp4) */
  MOE_WEIGHTS_MXFP8_TILED = 4  /* MXFP8 in the kernels' tiled order (moe_pack_mxfp8) */
} moe_weight_format_t;

/* Activations of the routed experts' two matrix products.  MOE_ACT_BF16: x as given (bf16)
 * and h kept as one fp16 plane (11 significant bits; one bf16 plane for MXFP4 weights).  MOE_ACT_MXFP8 (MXFP4 or MXFP8
 * weights only): x and h rounded to MXFP8 -- E4M3 values with one e8m0 scale per 32
 * consecutive values along the reduction (OCP MX v1.0: scale = 2^(floor(log2 amax) - 8),
 * round to nearest even, saturate at 448) -- and multiplied by gfx950's scaled MFMA; the
 * shared expert keeps bf16 activations.  The hybrid-attention page (table 模型一览) lists the
 * quantised model as "FP8 + MXFP4". */
typedef enum { MOE_ACT_BF16 = 0, MOE_ACT_MXFP8 = 1 } moe_act_format_t;

/* Layer configuration.  Field names follow the model's config.json text_config as the
 * routing walk-through page quotes them (sections 二, 三.2 and 四). */
typedef struct {
  int32_t hidden_size;              /* H; multiple of 128 */
  int32_t num_experts;              /* E routed experts; multiple of 64, at most 1024 */
  int32_t num_experts_per_tok;      /* K, 1..16 and at most topk_group*E/n_group */
  int32_t n_group;                  /* groups; divides 64 and E */
  int32_t topk_group;               /* kept groups, 1..n_group */
  int32_t moe_intermediate_size;    /* I; multiple of 128 */
  int32_t num_shared_experts;       /* S: 0 or 1 */
  int32_t shared_intermediate_size; /* must equal I when S == 1 */
  int32_t norm_topk_prob;           /* nonzero: renormalise the K weights to sum to 1 */
  float routed_scaling_factor;      /* multiplies the routed weights (2.5) */
  float swiglu_limit;               /* > 0: clamp routed activations to [-limit, limit] */
  float shared_swiglu_limit;        /* > 0: clamp shared-expert activations */
  int32_t expert_weight_format;     /* moe_weight_format_t of the routed experts */
  int32_t expert_act_format;        /* moe_act_format_t of the routed experts (0: bf16) */
} moe_config_t;

/* Expert weights, all device pointers, PyTorch [out_features, in_features] layout.
 *   MOE_WEIGHTS_BF16:  gate [E,I,H], up [E,I,H], down [E,H,I] bf16; *_scale NULL.
 *   MOE_WEIGHTS_MXFP4: gate [E,I,H/2], up [E,I,H/2], down [E,H,I/2] uint8, two e2m1
 *                      codes per byte (low nibble = even k, nibble = sign<<3 | code),
 *                      gate_scale/up_scale [E,I,H/32], down_scale [E,H,I/32] e8m0
 *                      bytes (value = e2m1 * 2^(scale-127), one scale per 32 k).
 *   MOE_WEIGHTS_MXFP8: gate [E,I,H], up [E,I,H], down [E,H,I] uint8 E4M3 codes (OCP FP8:
 *                      sign<<7 | exponent (bias 7)<<3 | mantissa; 0x7f/0xff NaN, never
 *                      given), scales as for MXFP4 (value = e4m3 * 2^(scale-127)).
 *   MOE_WEIGHTS_MXFP4_TILED: the MXFP4 arrays (same values, same sizes) in the order the
 *                      expert kernels read them, written by moe_pack_mxfp4; needs H and I
 *                      multiples of 256.  Each matrix [N, Kd] (gate, up: N = I, Kd = H;
 *                      down: N = H, Kd = I) is stored in blocks of 16 rows:
 *                      codes: 1 KB per 16 rows x 128 values, block (b, s) at byte
 *                        (b*(Kd/128) + s)*1024; in it, the 16 bytes at 16*(16*q + r) hold
 *                        row 16b + r's values k = 128s + 32q .. +31 (two per byte, low
 *                        nibble first), q = 0..3, r = 0..15;
 *                      scales: 128 bytes per 16 rows x 256 values, block (b, t) at byte
 *                        (b*(Kd/256) + t)*128; in it, byte 8*r + i is the scale of row
 *                        16b + r's 32-value block 8t + i.
 *                      A 16-lane x 4 load then reads 1 KB of contiguous codes per step (the
 *                      row-major layout spreads it over 16 rows' half cache lines).
 *   MOE_WEIGHTS_MXFP8_TILED: the MXFP8 arrays in the same manner (moe_pack_mxfp8; H and I
 *                      multiples of 256): codes 2 KB per 16 rows x 128 values, block (b, s) at
 *                      byte (b*(Kd/128) + s)*2048; in it, the 16 bytes at 1024*p + 16*(16*q + r)
 *                      hold row 16b + r's values k = 128s + 64p + 16q .. +15 (p = 0, 1: the
 *                      scaled MFMA's E4M3 operand halves); scales as for MOE_WEIGHTS_MXFP4_TILED.
 *   Shared expert (bf16, required when S == 1, else ignored):
 *                      shared_gate [I,H], shared_up [I,H], shared_down [H,I]. */
typedef struct {
  const void* gate;
  const void* up;
  const void* down;
  const uint8_t* gate_scale;
  const uint8_t* up_scale;
  const uint8_t* down_scale;
  const void* shared_gate;
  const void* shared_up;
  const void* shared_down;
} moe_expert_weights_t;

/* Bytes of device workspace that any entry point needs for T tokens (host call). */
moe_status_t moe_workspace_size(const moe_config_t* cfg, int64_t T, size_t* bytes);

/* Router (sections 三.1-三.3 and 四 of the routing walk-through page).
 *   x           device bf16 [T,H]   hidden states
 *   router_w    device fp32 [E,H]   router weight
 *   expert_bias device fp32 [E]     selection bias; NULL means no bias
 *   topk_idx    device int32 [T,K]  chosen experts of each token, ascending id
 *   topk_w      device fp32 [T,K]   their mixing weights, same order
 *   ws          device workspace of at least moe_workspace_size() bytes
 * Logits are computed in fp32 (bf16 x times fp32 W_r, fp32 accumulation); sigmoid,
 * bias, group scores and the selection are fp32.  Exact ties go to the lower group or
 * expert index.  The weight of a chosen expert is its unbiased sigmoid score. */
moe_status_t moe_route(const moe_config_t* cfg, int64_t T, const void* x, const float* router_w,
                       const float* expert_bias, int32_t* topk_idx, float* topk_w, void* ws,
                       size_t ws_bytes, void* stream);

/* Dispatch: group the T*K (token, slot) pairs by expert.
 *   topk_idx       device int32 [T,K] (each token's K ids distinct and in [0,E);
 *                  out-of-range ids are ignored: their slot gets inv_perm = -1 and they
 *                  are in no count)
 *   expert_counts  device int32 [E+1] tokens per expert; entry E = shared expert (T*S)
 *   expert_offsets device int32 [E+2] offsets[e] = sum of counts[0..e-1] for e < E;
 *                  offsets[E] = T*K and offsets[E+1] = T*K + T*S always
 *   sorted_token   device int32 [P]   positions offsets[e]..offsets[e]+counts[e]-1 hold the
 *                  tokens of expert e in ascending order; the shared expert's block
 *                  (from T*K) holds 0..T-1; positions no token fills (those of ignored
 *                  pairs, at the end of the last routed expert's range) hold -1
 *   inv_perm       device int32 [T,K] sorted position of each (token, slot) */
moe_status_t moe_dispatch(const moe_config_t* cfg, int64_t T, const int32_t* topk_idx,
                          int32_t* expert_counts, int32_t* expert_offsets, int32_t* sorted_token,
                          int32_t* inv_perm, void* ws, size_t ws_bytes, void* stream);

/* Expert FFNs (section 二 and 四): for every sorted position p of expert e and token
 * t = sorted_token[p],  y_sorted[p] = down_e( clamp( silu(gate_e x_t) * up_e x_t ) ).
 *   x              device bf16 [T,H]
 *   expert_offsets device int32 [E+2], sorted_token device int32 [P] (from moe_dispatch)
 *   weights        host pointer to the device weight table above
 *   y_sorted       device fp32 [P,H]  (rows of the shared expert at T*K + t)
 * gate/up runs on bf16 MFMA with fp32 accumulation.  The activation between the two
 * products is kept as one fp16 plane (11 significant bits) for bf16 and MXFP8 expert
 * weights, whose down product then runs on fp16 MFMA with the weights converted (bf16) or
 * decoded (MXFP8) exactly to fp16; as one bf16 plane for MXFP4 weights with bf16
 * activations; as MXFP8 with MXFP8 activations.  Block-format gate/up weights are decoded
 * exactly to bf16 in registers. */
moe_status_t moe_expert_ffn(const moe_config_t* cfg, int64_t T, const void* x,
                            const int32_t* expert_offsets, const int32_t* sorted_token,
                            const moe_expert_weights_t* weights, void* y_sorted, void* ws,
                            size_t ws_bytes, void* stream);

/* Combine: out[t] = sum_k topk_w[t,k] * y_sorted[inv_perm[t,k]]  (k ascending, fp32)
 *                   + y_sorted[T*K + t] when S == 1,   rounded once to bf16.
 *   y_sorted device fp32 [P,H], inv_perm device int32 [T,K], topk_w device fp32 [T,K],
 *   out device bf16 [T,H].  Slots with inv_perm < 0 contribute nothing. */
moe_status_t moe_combine(const moe_config_t* cfg, int64_t T, const void* y_sorted,
                         const int32_t* inv_perm, const float* topk_w, void* out, void* stream);

/* The whole layer: route, dispatch, expert FFNs, combine.
 *   out                device bf16 [T,H]
 *   topk_idx_out, topk_w_out, expert_counts_out: optional device copies of the
 *   routing ([T,K] int32, [T,K] fp32, [E+1] int32); NULL to skip.
 * Equivalent to the four calls above in order, with the same results bit for bit.
 * With block-format experts and a shared expert, the shared expert's kernels (which read x
 * only) run on a second stream of the library's, created once per device on its first such
 * call (default priority), forked from `stream` before the router and joined back into
 * `stream` before the combine: everything the call enqueues is still ordered after the
 * work already on `stream` and before the work enqueued on it afterwards. */
moe_status_t moe_forward(const moe_config_t* cfg, int64_t T, const void* x, const float* router_w,
                         const float* expert_bias, const moe_expert_weights_t* weights, void* out,
                         int32_t* topk_idx_out, float* topk_w_out, int32_t* expert_counts_out,
                         void* ws, size_t ws_bytes, void* stream);

/* Dense SwiGLU FFN, the layers before the MoE stack (routing walk-through page, section 二:
 * first_k_dense_replace = 2, the first two of the 42 layers use an ordinary dense FFN; the
 * page gives no intermediate size, so it is a parameter, and the FFN is read as the experts'
 * own SwiGLU form):  out[t] = ( silu(x[t] gate^T) * (x[t] up^T) ) down^T, the activation
 * clamped to +-swiglu_limit when it is > 0, fp32 accumulation, one rounding to bf16.
 * Up to 10 tokens it runs on two kernels of its own (gate/up, then down writing out); up to
 * 4096, on the kernels of moe_expert_ffn with tiles computed from T and the output written by
 * the down GEMM (or, up to 512 tokens, by a last kernel adding the down GEMM's split
 * reduction in order); above, as a layer with a single routed expert that every token takes with
 * weight 1, on the kernels of moe_expert_ffn and moe_combine.  Up to 10 tokens h is kept as
 * two bf16 planes (about 16 significand bits), above as one fp16 plane (11); every path sums
 * in a fixed order.
 *   x device bf16 [T,H]; gate, up device bf16 [I,H]; down device bf16 [H,I]; out device
 *   bf16 [T,H]; ws device, 256-byte aligned, moe_dense_ffn_workspace_size bytes.
 *   H and I multiples of 128 (MOE_ERR_UNSUPPORTED otherwise); T = 0 is a no-op.
 * Results are deterministic. */
moe_status_t moe_dense_ffn_workspace_size(int32_t hidden_size, int32_t intermediate_size, int64_t T,
                                          size_t* bytes);
moe_status_t moe_dense_ffn(int32_t hidden_size, int32_t intermediate_size, float swiglu_limit, int64_t T,
                           const void* x, const void* gate, const void* up, const void* down, void* out,
                           void* ws, size_t ws_bytes, void* stream);

/* MXFP8 rounding of bf16 activations, the step the MOE_ACT_MXFP8 path applies to x before
 * the routed experts' gate/up products (the same device code rounds h in the gate/up
 * epilogue): for each block of 32 consecutive values of a row, scale = 2^X with
 * X = floor(log2 max|v|) - 8 clamped to [-127, 127] (-127 for an all-zero block), and each
 * v / 2^X rounded to the nearest E4M3 value, ties to even, saturated at 448 (OCP MX v1.0).
 *   x       device bf16 [rows, cols]; cols a positive multiple of 32
 *   codes   device uint8 [rows, cols]     E4M3 codes (16-byte aligned)
 *   scales  device uint8 [rows, cols/32]  e8m0 bytes X + 127
 * Enqueued on `stream`; rows = 0 is a no-op. */
moe_status_t moe_quantise_mxfp8(const void* x, int64_t rows, int32_t cols, uint8_t* codes, uint8_t* scales,
                                void* stream);

/* MXFP4 weights from the row-major MOE_WEIGHTS_MXFP4 arrays into MOE_WEIGHTS_MXFP4_TILED
 * order (the layout above), for `mats` consecutive matrices of N x Kd values each; weights
 * are static, so this runs once when they are loaded (the hybrid-attention page, table
 * 模型一览, gives the routed experts in MXFP4; their memory order is not fixed there).
 *   codes      device uint8 [mats, N, Kd/2]   row-major E2M1 codes (16-byte aligned)
 *   scales     device uint8 [mats, N, Kd/32]  row-major e8m0 scales (8-byte aligned)
 *   codes_out  device uint8, mats * N * Kd/2 bytes (16-byte aligned; must not overlap codes)
 *   scales_out device uint8, mats * N * Kd/32 bytes (8-byte aligned; must not overlap scales)
 *   N          multiple of 16; Kd multiple of 256
 * MOE_ERR_INVALID_ARG for a NULL pointer, bad sizes or overlapping buffers, MOE_ERR_ALIGNMENT
 * for a misaligned pointer; mats = 0 is a no-op.  Enqueued on `stream`. */
moe_status_t moe_pack_mxfp4(const uint8_t* codes, const uint8_t* scales, int64_t mats, int32_t N, int32_t Kd,
                            uint8_t* codes_out, uint8_t* scales_out, void* stream);

/* The same for MXFP8 weights (MOE_WEIGHTS_MXFP8 -> MOE_WEIGHTS_MXFP8_TILED): codes [mats, N, Kd]
 * (one E4M3 code per byte) and scales [mats, N, Kd/32], outputs of the same sizes; the same
 * requirements and errors as moe_pack_mxfp4. */
moe_status_t moe_pack_mxfp8(const uint8_t* codes, const uint8_t* scales, int64_t mats, int32_t N, int32_t Kd,
                            uint8_t* codes_out, uint8_t* scales_out, void* stream);

/* Expert-bias update, the step after the layer in training (routing walk-through page,
 * section 三.3: every routed expert's selection bias is lowered when it is busy and raised
 * when it is idle, balancing the load without an auxiliary loss).  The page gives neither the
 * rule nor the rate; this library takes the sign rule with a caller-chosen step gamma:
 *   bias[e] += gamma   if counts[e] * E < sum(counts)   (below the mean count)
 *   bias[e] -= gamma   if counts[e] * E > sum(counts)   (above it; unchanged at the mean)
 * computed as bias[e] + gamma * (+1 | -1 | 0) in fp32, the decision taken in integers.
 *   expert_counts  device int32 [E]: the routed counts of a step (the first E entries of the
 *                  expert_counts of moe_dispatch or moe_forward; the shared expert's is not read)
 *   expert_bias    device fp32 [E], updated in place (the array moe_route/moe_forward read)
 *   gamma          the step; any finite value (MOE_ERR_INVALID_ARG otherwise)
 * Enqueued on `stream`; it reads the counts when it runs, so it may follow the forward that
 * writes them on the same stream without a host synchronisation. */
moe_status_t moe_update_expert_bias(const moe_config_t* cfg, const int32_t* expert_counts,
                                    float* expert_bias, float gamma, void* stream);

/* moe_forward with a timing trace, for profiling (same results).  events[0] is recorded on
 * `stream` before the first kernel and events[i+1] right after the i-th kernel launch; the
 * caller creates the events (hipEvent_t, passed as void*) and later reads the elapsed times;
 * a NULL entry records nothing (each recorded event costs a few microseconds of queue time,
 * so a caller timing one kernel passes only the two events around it).
 * kernel_names (host array of max_events - 1 pointers) receives static kernel names and
 * *n_kernels the number of kernels launched.  Returns MOE_ERR_INVALID_ARG (after running
 * the layer) if max_events is smaller than n_kernels + 1. */
moe_status_t moe_forward_traced(const moe_config_t* cfg, int64_t T, const void* x, const float* router_w,
                                const float* expert_bias, const moe_expert_weights_t* weights, void* out,
                                void* ws, size_t ws_bytes, void* stream, void* const* events,
                                int32_t max_events, const char** kernel_names, int32_t* n_kernels);

/* moe_forward with one kernel timed by events bound to its own dispatch (the AMD launch
 * extension hipExtLaunchKernel): start_event and stop_event (hipEvent_t created by the caller,
 * passed as void*) take that kernel's start and end times, and no other queue packets are
 * added, so the step runs as fast as moe_forward (same results).  kernel_index counts the
 * kernels in the order moe_forward_traced names them (0 = the first); a step that launches
 * several kernels under one name is timed by its first.  Returns MOE_ERR_INVALID_ARG (after
 * running the layer) if the forward launched no kernel with that index. */
moe_status_t moe_forward_timed(const moe_config_t* cfg, int64_t T, const void* x, const float* router_w,
                               const float* expert_bias, const moe_expert_weights_t* weights, void* out,
                               void* ws, size_t ws_bytes, void* stream, int32_t kernel_index,
                               void* start_event, void* stop_event);

/* moe_forward without a caller workspace, for callers that cannot allocate device memory
 * (code under HIP graph capture, tight serving loops, harnesses that forbid allocation).
 * Same arguments and results as moe_forward (bit for bit), minus ws/ws_bytes: the workspace
 * is a static device array inside the library, 64 MiB on each GPU the library runs on, held
 * until the process ends (its device address is looked up on the first call on a device,
 * which must be current).  The call allocates nothing.  T whose workspace
 * (moe_workspace_size) exceeds 64 MiB is rejected with MOE_ERR_WORKSPACE before anything is
 * enqueued: for the full-size layer (hidden 2560, 512 experts, intermediate 768) that is T
 * above about 970 tokens.  Every call on one GPU uses the same array and leaves its contents
 * behind (each call rewrites what it reads), so calls that overlap on one GPU -- on
 * different streams, or from different threads without ordering -- race. */
moe_status_t moe_forward_noalloc(const moe_config_t* cfg, int64_t T, const void* x, const float* router_w,
                                 const float* expert_bias, const moe_expert_weights_t* weights, void* out,
                                 int32_t* topk_idx_out, float* topk_w_out, int32_t* expert_counts_out,
                                 void* stream);

/* ---- Training the experts -----------------------------------------------------------------
 * The operators of a training step beside the forward: products grouped by expert whose
 * operands and results stay with the caller (forward, input gradient, weight gradient), the
 * SwiGLU activation with its gradient, and the AdamW step.  One layer, positions p in
 * moe_dispatch's order, topk_w [T,K] and inv_perm [T,K] flattened:
 *   g = moe_grouped_gemm(x by sorted_token, gate)     u = the same with up          (bf16)
 *   h = moe_swiglu(g, u; row_w = topk_w, pos = inv_perm)                            (bf16)
 *   y_sorted = moe_grouped_gemm(h, down) (fp32);  out = moe_combine(y_sorted, ones): the
 *     routing weights are in h already
 *   dh = moe_grouped_gemm_dgrad(dout by sorted_token, down)                         (bf16)
 *   d_down = moe_grouped_gemm_wgrad(dout by sorted_token, h)
 *   dg, du, d_topk_w = moe_swiglu_backward(g, u, dh; topk_w, inv_perm)
 *   dx_sorted = moe_grouped_gemm_dgrad(dg, gate, du, up) (fp32); dx = moe_combine(dx_sorted, ones)
 *   d_gate = moe_grouped_gemm_wgrad(dg, x by sorted_token); d_up likewise
 *   moe_adamw_step on the expert weights; moe_update_expert_bias on the selection bias
 * The shared expert's T rows are one group at position T*K of every buffer, whatever the routing: its
 * calls take the matrices from that row on, x and dout by token without a map, groups = 1, rows = T
 * and offsets {0, T}.  (groups = 1 with offsets = expert_offsets + E on the whole buffers computes the
 * same, but tiles are chosen for groups of rows / groups positions, here all P: 44 us instead of 18
 * for the gate product of 1024 tokens at 2560 x 768.)
 * Outputs must not overlap inputs (offsets, maps, positions and weights among them) or each other:
 * MOE_ERR_INVALID_ARG.  Matrices of one row stride may lie side by side in the rows of one buffer,
 * and a vector between two rows of a matrix. */
typedef enum { MOE_DTYPE_BF16 = 0, MOE_DTYPE_FP32 = 1 } moe_dtype_t;

/* Groups of positions: group g holds positions offsets[g] <= p < offsets[g+1] (the first
 * groups + 1 entries of moe_dispatch's expert_offsets, or that many from expert e on), each
 * group with its own [out_features, in_features] weight.  Offsets are read on the device and
 * taken as clamped to [0, rows]; a group may be empty. */
typedef struct {
  int32_t groups;         /* 1..1025 */
  int32_t out_features;   /* N: multiple of 8, at most 65536 */
  int32_t in_features;    /* K: multiple of 8, at most 65536; N * K below 2^31 - 128 */
  int64_t rows;           /* positions; below 2^31 - 4096 */
  const int32_t* offsets; /* device [groups + 1], 4-byte aligned, not decreasing */
} moe_groups_t;

/* A bf16 operand by position: position p is row row_map[p] of the matrix (device int32 [rows],
 * 4-byte aligned; moe_dispatch's sorted_token), or row p with row_map NULL.  A position whose
 * row lies outside [0, rows) counts as a row of zeros and is never read. */
typedef struct {
  const void* data;       /* device bf16, row stride ld; NULL only with rows 0 */
  int64_t rows;           /* rows of the matrix; with row_map NULL at least the positions */
  int64_t ld;             /* values between rows: at least the columns, multiple of 8, at most 2^22 */
  const int32_t* row_map;
} moe_rows_t;

/* y[p] = w_g x[p] (fp32 accumulation) for every position p of every group g.
 *   x  [.., in_features]; w device bf16 [groups, out_features, in_features]
 *   y  device bf16 or fp32 (y_dtype) [rows, out_features], row stride ldy (multiple of 8).  Rows
 *      of no group are left as they are.  accumulate != 0 adds to y (fp32 only).
 * No workspace; results do not depend on the launch (no atomics).  `rows` and `groups` choose the
 * tiles, so rows should be about what the groups hold.  An infinity or NaN of one row
 * or group reaches that row's or group's results only. */
moe_status_t moe_grouped_gemm(const moe_groups_t* groups, const moe_rows_t* x, const void* w, void* y, int64_t ldy,
                              int32_t y_dtype, int32_t accumulate, void* stream);

/* Input gradient: dx[p] = dy[p] w_g (+ dy2[p] w2_g, both or neither), summed in fp32 and rounded
 * once.  dy, dy2 [.., out_features], with the same rows, row stride and row map; w, w2 as above; dx bf16 or fp32 [rows, in_features]. */
moe_status_t moe_grouped_gemm_dgrad(const moe_groups_t* groups, const moe_rows_t* dy, const void* w,
                                    const moe_rows_t* dy2, const void* w2, void* dx, int64_t lddx, int32_t dx_dtype,
                                    int32_t accumulate, void* stream);

/* Weight gradient: dw_g = sum over the group's positions of dy[p]^T x[p]; an empty group's is
 * zero (or unchanged with accumulate != 0, which adds to dw; fp32 only).  A position counts only
 * if its rows exist in both operands.
 *   dw device bf16 or fp32 [groups, out_features, in_features] */
moe_status_t moe_grouped_gemm_wgrad(const moe_groups_t* groups, const moe_rows_t* dy, const moe_rows_t* x, void* dw,
                                    int32_t dw_dtype, int32_t accumulate, void* stream);

/* SwiGLU with clamp and routing weight over stored products: for i < n and row r = pos[i] (i
 * with pos NULL),  h[r] = row_w[i] * clamp(silu(gate[r]) * up[r], -limit, limit), rounded once.
 *   gate, up  device bf16 [mat_rows, cols], row stride ld; h likewise with ldh; cols a multiple
 *             of 8, strides multiples of 8.  (bf16 only: the products are kept for the backward
 *             pass, and in fp32 they would double what both directions read and what is kept.)
 *   limit     > 0: clamp; 0, negative or infinite: none
 *   row_w     device fp32 [n] or NULL (1);  pos device int32 [n] or NULL, entries distinct; an
 *             entry outside [0, mat_rows) is skipped (moe_dispatch's -1)
 * Rows that no entry names are left as they are. */
moe_status_t moe_swiglu(int64_t n, int64_t mat_rows, int32_t cols, float limit, const void* gate, const void* up,
                        int64_t ld, const float* row_w, const int32_t* pos, void* h, int64_t ldh, void* stream);

/* Its gradient from dh: dgate, dup device bf16 [mat_rows, cols] (row stride ldd) and, unless NULL,
 * drow_w device fp32 [n] (0 for a skipped entry).  A value that the clamp cuts, |silu(g) u| >
 * limit, passes no gradient to gate and up. */
moe_status_t moe_swiglu_backward(int64_t n, int64_t mat_rows, int32_t cols, float limit, const void* gate,
                                 const void* up, int64_t ld, const void* dh, int64_t lddh, const float* row_w,
                                 const int32_t* pos, void* dgate, void* dup, int64_t ldd, float* drow_w, void* stream);

/* AdamW over many tensors in one launch:
 *   m' = beta1 m + (1 - beta1) g;  v' = beta2 v + (1 - beta2) g^2      (each operation rounded
 *        to fp32; g = grad, times *grad_scale if that is given)
 *   p' = p (1 - lr weight_decay) - lr m' / (1 - beta1^step) / (sqrt(v' / (1 - beta2^step)) + eps)
 * (with eps 0, a value that never had a gradient becomes NaN: 0 / 0).
 * Parameters and gradients are bf16 or fp32; with bf16 parameters an fp32 master copy may hold
 * the exact values (then the parameters are its rounding).  States are fp32, or 8 bits:
 * MOE_STATE_8BIT keeps blocks of 128 consecutive values of a tensor as one code byte each and an
 * fp32 scale, the block's largest magnitude / 1.875:
 *   exp_avg     code = sign << 7 | e << 3 | f: (1 + f/8) 2^(e-15) scale, zero for e = f = 0
 *   exp_avg_sq  code = e << 3 | f:             (1 + f/8) 2^(e-31) scale
 * rounded stochastically by a hash of (seed, step, tensor's index in the plan, value's index):
 * the same call gives the same codes.  Rounding is unbiased from 1.125 2^-15 (exp_avg) and 2^-31
 * (exp_avg_sq) of the scale on.  Smaller second moments are raised to 2^-31; first moments up to 2^-15 of
 * the scale become zero, so an element whose gradients stay below 1.6e-5 of its block's largest is not
 * moved: tensors that mix such sizes within 128 values keep MOE_STATE_FP32.  Both moments start as
 * zero codes with zero scales.  A block with an infinite or NaN value, which has no code, reads back
 * as not finite. */
typedef enum { MOE_STATE_FP32 = 0, MOE_STATE_8BIT = 1 } moe_state_format_t;

typedef struct {           /* device arrays of one tensor, 16-byte aligned (scales 4-byte) */
  void* param;             /* [numel] param_dtype, updated */
  float* master;           /* [numel] fp32, updated; NULL for all tensors or for none */
  const void* grad;        /* [numel] grad_dtype */
  void* exp_avg;           /* [numel] fp32 or codes, updated */
  void* exp_avg_sq;
  float* exp_avg_scale;    /* [ceil(numel / 128)] fp32, MOE_STATE_8BIT only */
  float* exp_avg_sq_scale;
  int64_t numel;           /* may be 0 */
  float weight_decay;
  int32_t reserved;
} moe_adamw_tensor_t;

typedef struct {
  int64_t n_tensors, n_chunks;
  uint64_t flags;
  size_t image_bytes;      /* size of the plan's image */
} moe_adamw_plan_t;

typedef struct {
  double lr, beta1, beta2, eps;
  int64_t step;            /* 1 for the first step */
  uint32_t seed;           /* of the stochastic rounding */
  /* device scalars outside the arrays that the step writes (which is not checked) */
  const float* lr_ptr;     /* device; if given, read when the step runs instead of lr */
  const int64_t* step_ptr; /* device; likewise for step (a captured step can then be replayed); below 1
                              the step writes nothing */
  const float* grad_scale; /* device; if given, multiplies every gradient */
} moe_adamw_config_t;

/* Host call: fills *plan and, with image (host memory, plan->image_bytes), the table that the
 * step reads.  The caller copies the image to device memory once (16-byte aligned) and keeps it as
 * long as the arrays stay where they are.  Arrays that the step writes must overlap no other. */
moe_status_t moe_adamw_plan(int64_t n_tensors, const moe_adamw_tensor_t* tensors, int32_t param_dtype,
                            int32_t grad_dtype, int32_t state_format, moe_adamw_plan_t* plan, void* image,
                            size_t image_bytes);

/* One step.  image: the device copy of the plan's image.  Memory that does not hold an image, or one
 * of other numbers of tensors and chunks or other types, is recognised by the kernel, which then
 * writes nothing (an image of the same numbers and types is taken for this plan's). */
moe_status_t moe_adamw_step(const moe_adamw_config_t* cfg, const moe_adamw_plan_t* plan, const void* image,
                            void* stream);

/* Values of an 8-bit state array: out[i] (device fp32) = the value that codes[i] stands for.
 * is_signed != 0: exp_avg's codes, 0: exp_avg_sq's. */
moe_status_t moe_adamw_dequantise(const uint8_t* codes, const float* scales, int64_t numel, int32_t is_signed,
                                  float* out, void* stream);

/* Static text for a status code. */
const char* moe_status_string(moe_status_t status);

/* Description of the last failed call on this thread ("" if none). */
const char* moe_last_error(void);

#ifdef __cplusplus
}
#endif
#endif /* MOE_H_ */
