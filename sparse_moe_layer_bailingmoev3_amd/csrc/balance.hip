// Balance loss of a router: how evenly the tokens of each sequence load the experts.
//
//   p_te = s_te / sum_j s_tj,  s = sigmoid(logits)      P_be = mean of p_te over the tokens of sequence b
//   c_be = (token, slot) pairs of sequence b at e       f_be = E c_be / (K n_b)
//   loss = coef sum_b (n_b / N) sum_e f_be P_be  =  coef E / (K N) sum_be c_be P_be
//
// Two launches.  The first cuts the tokens into chunks; a workgroup walks the sequences that its
// chunk touches, its waves taking four tokens at a time (a lane EPL experts of each), and leaves one
// row of sums and counts per (chunk c, sequence b) in slot c + b of the workspace.  (Both grow along the
// walk and one of them at every step, so no two pairs share a slot.)  The second adds a sequence's
// slots, 64 experts a workgroup or wave, and its last workgroup to finish adds the parts of the loss.  A small
// batch is done by one workgroup in one launch.  Every sum has a fixed order.
//
// Counts are integers: LDS atomics, whose order does not matter.
//
// What bounds it, on one MI355X: 8192 tokens of 512 experts 13.8 us, of which the logits' 17 MB are 3.  The
// first launch takes 6.2 (about 2.8 of vector work, 80 cycles a score, behind the first loads), the second 6.0,
// a chain of latencies: the sequence's ends, its slots, the parts of the loss, the counter (2.5 with what
// follows it), the parts again.
#include "router_scores.h"

namespace moe {

namespace {

// sums over the tokens [lo, hi) of one sequence and their counts, left in sums[0] and hist
template <int EPL, int WAVES>
__device__ __forceinline__ void balance_run(const BalanceArgs& a, int lo, int hi, float (*sums)[EPL * 64], int* hist) {
  constexpr int E = EPL * 64, AHEAD = EPL > 8 ? 2 : 4;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  float acc[EPL] = {};
  const int64_t p0 = (int64_t)lo * a.K + threadIdx.x, p1 = (int64_t)hi * a.K;
  const int e0 = p0 < p1 ? a.topk_idx[p0] : -1;  // (asked for before the scores, which take longer)
  for (int t = lo + wave * AHEAD; t < hi; t += WAVES * AHEAD) {
    float l[AHEAD][EPL];
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) Row<EPL>::load(a.logits + (int64_t)min(t + k, hi - 1) * E, lane, l[k]);
    float total[AHEAD], least = 1.f;
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      total[k] = 0.f;
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        l[k][i] = score_of(l[k][i]).s;
        total[k] += l[k][i];
      }
      total[k] = wave_sum(total[k]);
      least = fminf(least, total[k]);
    }
    if (least < SCORES_TINY) {
#pragma unroll
      for (int k = 0; k < AHEAD; ++k) {
        if (!(total[k] < SCORES_TINY)) continue;
        Row<EPL>::load(a.logits + (int64_t)min(t + k, hi - 1) * E, lane, l[k]);
        total[k] = 0.f;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
          l[k][i] = tiny_score(l[k][i]);
          total[k] += l[k][i];
        }
        total[k] = wave_sum(total[k]);
      }
    }
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      const float inv = total[k] == 0.f || t + k >= hi ? 0.f : 1.0f / total[k];
#pragma unroll
      for (int i = 0; i < EPL; ++i) acc[i] = t + k < hi ? __builtin_fmaf(l[k][i], inv, acc[i]) : acc[i];
    }
  }
  if ((unsigned)e0 < (unsigned)E) atomicAdd(&hist[e0], 1);
  for (int64_t p = p0 + WAVES * 64; p < p1; p += WAVES * 64) {
    const int e = a.topk_idx[p];
    if ((unsigned)e < (unsigned)E) atomicAdd(&hist[e], 1);
  }
  Row<EPL>::store(sums[wave], lane, acc);
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += WAVES * 64) {
    float v = sums[0][e];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) v += sums[w][e];
    sums[0][e] = v;
  }
}

constexpr int BAL_WAVES = 8;

template <int EPL>
__global__ __launch_bounds__(BAL_WAVES * 64) void balance_partial_kernel(BalanceArgs a) {
  constexpr int E = EPL * 64;
  __shared__ __align__(16) float sums[BAL_WAVES][E];
  __shared__ int hist[E];
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.done = 0;
  const int t0 = blockIdx.x * a.chunk, t1 = (int)min((int64_t)t0 + a.chunk, (int64_t)a.seq.T);
  for (int i = threadIdx.x; i < E; i += BAL_WAVES * 64) hist[i] = 0;
  const Seqs seqs(a.seq);
  int b = seqs.first(t0);
  __syncthreads();
  for (; b < a.seq.n; ++b) {
    const Seq q = seqs.at(b);
    if (q.begin >= t1) break;
    const int lo = max(q.begin, t0), hi = min(q.end, t1);
    if (lo < hi) {
      balance_run<EPL, BAL_WAVES>(a, lo, hi, sums, hist);
      const int64_t slot = (int64_t)blockIdx.x + b;
      for (int e = threadIdx.x; e < E; e += BAL_WAVES * 64) {
        a.psum[slot * E + e] = sums[0][e];
        a.pcnt[slot * E + e] = hist[e];
        hist[e] = 0;
      }
      __syncthreads();
    }
    if (q.next >= t1) break;
  }
}

// one chunk of tokens: all of it
template <int EPL>
__global__ __launch_bounds__(1024) void balance_small_kernel(BalanceArgs a) {
  constexpr int E = EPL * 64, WAVES = 16;
  __shared__ __align__(16) float sums[WAVES][E];
  __shared__ int hist[E];
  __shared__ double parts[WAVES];
  __shared__ int tokens;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int i = threadIdx.x; i < E; i += 1024) hist[i] = 0;
  const Seqs seqs(a.seq);
  const int N = seqs.tokens(&tokens);
  __syncthreads();
  double part = 0;
  for (int b = 0; b < a.seq.n; ++b) {
    const Seq q = seqs.at(b);
    const int n = q.end - q.begin;
    if (n > 0) balance_run<EPL, WAVES>(a, q.begin, q.end, sums, hist);
    for (int e = threadIdx.x; e < E; e += 1024) {
      const double mean = n > 0 ? (double)sums[0][e] / n : 0.0;
      a.probs[(int64_t)b * E + e] = (float)mean;
      a.counts[(int64_t)b * E + e] = hist[e];
      part += hist[e] * mean;
      hist[e] = 0;
    }
    __syncthreads();
  }
  part = wave_sum_f64(part);
  if (lane == 0) parts[wave] = part;
  __syncthreads();
  if (threadIdx.x == 0) {
    part = 0;
    for (int w = 0; w < WAVES; ++w) part += parts[w];
    *a.loss = N > 0 ? (float)((double)a.coef * E * part / ((double)a.K * N)) : 0.f;
  }
}

// A pair is a sequence and 64 experts.  Few pairs: a workgroup each, whose waves take turns at the slots.
// MANY: a wave each, 16 a workgroup, as launching and meeting at the counter cost each workgroup its turn.
template <bool MANY>
__global__ __launch_bounds__(1024) void balance_finish_kernel(BalanceArgs a) {
  constexpr int WAVES = MANY ? 1 : 16;  // of a pair
  __shared__ double sums[16][64];
  __shared__ int cnts[16][64];
  __shared__ int tokens, last;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, turn = MANY ? 0 : wave;
  const int blocks = a.E / 64, pairs = a.seq.n * blocks;
  const int pair = __builtin_amdgcn_readfirstlane(MANY ? blockIdx.x * 16 + wave : blockIdx.x);
  const int b = pair / blocks, e = (pair - b * blocks) * 64 + lane;
  const Seqs seqs(a.seq);
  const bool late = a.seq.lens && !seqs.few;  // lens that the last workgroup adds
  int N = late ? 0 : seqs.tokens(&tokens);
  const Seq q = pair < pairs ? seqs.at(b) : Seq{0, 0, 0};
  double sum = 0;
  int cnt = 0;
  if (q.begin < q.end) {
    const int c1 = __builtin_amdgcn_readfirstlane((q.end - 1) / a.chunk);
    for (int c = __builtin_amdgcn_readfirstlane(q.begin / a.chunk + turn); c <= c1; c += 16 * WAVES) {
      float v[16];  // sixteen slots' loads at once
      int n[16];
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        if (c + WAVES * k > c1) break;
        const int64_t at = ((int64_t)(c + WAVES * k) + b) * a.E + e;
        v[k] = a.psum[at];
        n[k] = a.pcnt[at];
      }
#pragma unroll
      for (int k = 0; k < 16; ++k)
        if (c + WAVES * k <= c1) {
          sum += v[k];
          cnt += n[k];
        }
    }
  }
  if constexpr (!MANY) {
    sums[wave][lane] = sum;
    cnts[wave][lane] = cnt;
    __syncthreads();
    if (wave > 0) return;
    for (int w = 1; w < WAVES; ++w) {
      sum += sums[w][lane];
      cnt += cnts[w][lane];
    }
  }
  if (pair < pairs) {
    const int len = q.end - q.begin;
    const double mean = len > 0 ? sum / len : 0.0;
    const int64_t at = (int64_t)b * a.E + e;
    a.counts[at] = cnt;
    a.probs[at] = (float)mean;
    const double part = wave_sum_f64(cnt * mean);
    if (lane == 0) {
      // An exchange has taken place where all dies see it once its old value is here: no cache need be written
      // back, as a fence would do for every pair (8192 pairs: 30 us a call, 172 with fences).
      const unsigned long long old = __hip_atomic_exchange((unsigned long long*)(a.part + pair), __double_as_longlong(part),
                                                           __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      asm volatile("" ::"v"(old) : "memory");
    }
  }
  int is_last = 0;
  if constexpr (MANY) __syncthreads();
  if (threadIdx.x == 0) is_last = atomicAdd(a.done, 1) == (int)gridDim.x - 1;
  if constexpr (MANY) {
    if (threadIdx.x == 0) last = is_last;
    __syncthreads();
    is_last = last;
  }
  if (!__builtin_amdgcn_readfirstlane(is_last)) return;
  // the last workgroup: all parts in order, read past the caches that do not see other dies' stores
  __threadfence();
  constexpr int STEP = MANY ? 1024 : 64;
  double total = 0;
  for (int i = threadIdx.x; i < pairs; i += STEP) total += __hip_atomic_load(a.part + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  total = wave_sum_f64(total);
  if (late) {
    for (int i = threadIdx.x; i < a.seq.n; i += STEP) {
      const Seq s = seq_at(a.seq, i);
      N += s.end - s.begin;
    }
    N = wave_sum_i32(N);
  }
  if constexpr (MANY) {
    if (lane == 0) {
      sums[0][wave] = total;
      cnts[0][wave] = N;
    }
    __syncthreads();
    total = 0;
    if (late) N = 0;
    for (int w = 0; w < 16; ++w) {
      total += sums[0][w];
      if (late) N += cnts[0][w];
    }
  }
  if (threadIdx.x == 0) *a.loss = N > 0 ? (float)((double)a.coef * a.E * total / ((double)a.K * N)) : 0.f;
}

// ---- fp32 values in 16-bit pieces -------------------------------------------------------------

// the exponent that brings values of magnitude up to `top` (as bits) below 2^15, the largest to 2^14 or
// more (subnormal ones too, whose largest is below 2^-126)
__device__ __forceinline__ int half_exponent(uint32_t top) { return 14 + 127 - (int)(top >> 23); }
// two values times 2^ex -> two fp16 pieces each; infinities and NaN end as NaN
__device__ __forceinline__ void half_pieces(float v0, float v1, int ex, uint32_t& hi, uint32_t& lo) {
  typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
  v0 = __builtin_amdgcn_ldexpf(v0, ex);
  v1 = __builtin_amdgcn_ldexpf(v1, ex);
  const f16x2 h = {(_Float16)v0, (_Float16)v1};
  const f16x2 l = {(_Float16)(v0 - (float)h[0]), (_Float16)(v1 - (float)h[1])};
  hi = __builtin_bit_cast(uint32_t, h);
  lo = __builtin_bit_cast(uint32_t, l);
}
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, true));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, true));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xF, 0xF, true));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x140, 0xF, 0xF, true));
  auto at = [&](int l) { return (uint32_t)__builtin_amdgcn_readlane((int)v, l); };
  return max(max(at(0), at(16)), max(at(32), at(48)));
}

// three bf16 (upper halves of words) that add up to v exactly; infinities and NaN end as NaN
__device__ __forceinline__ void bf16_pieces(float v, uint32_t (&p)[3]) {
  p[0] = __float_as_uint(v) & 0xFFFF0000u;
  v -= __uint_as_float(p[0]);
  p[1] = __float_as_uint(v) & 0xFFFF0000u;
  p[2] = __float_as_uint(v - __uint_as_float(p[1])) & 0xFFFF0000u;
}

// a lane's share of a row in P planes of 16-bit pieces
template <int EPL, int P>
struct Pieces {
  uint32_t w[P][(EPL + 1) / 2];
  // where(e): where expert e's value lies in the first plane
  template <typename At>
  __device__ __forceinline__ void store(uint16_t* base, int64_t plane, int lane, At where) const {
#pragma unroll
    for (int p = 0; p < P; ++p) {
#pragma unroll
      for (int j = 0; j < Row<EPL>::NJ; ++j) {
        uint16_t* const at = base + p * plane + where(Row<EPL>::at(lane, j));
        if constexpr (EPL == 1) *at = (uint16_t)w[p][0];
        else if constexpr (EPL == 2) *(uint32_t*)at = w[p][0];
        else *(u32x2*)at = u32x2{w[p][2 * j], w[p][2 * j + 1]};
      }
    }
  }
};

// 16 columns of router_w, transposed, in scaled fp16 pieces: a thread takes N = 4 EPL consecutive experts of
// a column, which lie side by side in the planes, 16 of them beside those of the next column.
template <int EPL>
__device__ __forceinline__ void split_weight(const DlogitsArgs& a, int block, uint32_t* lds) {
  constexpr int E = EPL * 64, N = 4 * EPL, V = N < 8 ? N / 2 : 4;  // words of a store
  typedef uint32_t vec __attribute__((ext_vector_type(V)));
  const int col = threadIdx.x & 15, grp = threadIdx.x >> 4, h0 = block * 16;
  float v[N];
  uint32_t top = 0;
  const float* src = a.w + (int64_t)grp * N * a.H + h0 + col;
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = src[(int64_t)i * a.H];
#pragma unroll
  for (int i = 0; i < N; ++i) top = max(top, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  lds[threadIdx.x] = top;
  __syncthreads();
#pragma unroll
  for (int g = 0; g < 16; ++g) top = max(top, lds[g * 16 + col]);
  const int ex = half_exponent(top);
  if (grp == 0) a.wexp[h0 + col] = ex;
#pragma unroll
  for (int i = 0; i < N; i += 2 * V) {
    vec w[2];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      uint32_t hi, lo;
      half_pieces(v[i + 2 * j], v[i + 2 * j + 1], ex, hi, lo);
      w[0][j] = hi;
      w[1][j] = lo;
    }
#pragma unroll
    for (int p = 0; p < 2; ++p) *(vec*)(a.wt + p * plane_size(a.H, E) + plane_at(h0 + col, grp * N + i, E)) = w[p];
  }
}

// ---- the gradient of the logits ------------------------------------------------------------------
//   through the mixing weights, w_k = c s_k / sum_j s_j (or c s_k):
//     dl_k = (g_k - sum_j g_j q_j) q_k (1 - s_k),  g = c dw, q = s / sum s      (or g_k s_k (1 - s_k))
//   through the balance loss (the counts are constants to it):
//     dl_e += dloss coef / N (f_e - sum_j f_j p_j) p_e (1 - s_e)
// A wave takes `run` consecutive tokens, a lane EPL experts of each; the K chosen experts' part is
// computed by K lanes and handed to the experts' lanes through LDS.  The gradient leaves in fp32 if it is
// asked for, and in the 16-bit pieces that the products take; other workgroups take router_w apart meanwhile.
//
// What bounds it, on one MI355X: 8192 tokens of 512 experts with both products' pieces 15.5-18 us, 28 MB read
// and 50 written at the copy's rate; 16,384 tokens of 256 experts, fp32 alone, 12.0 us against 5 of traffic: latency
// and vector work of four tokens a wave.  router_w's part (512 x 2560) takes 8 alone, so it goes first.
template <int EPL>
__global__ __launch_bounds__(256) void dlogits_kernel(DlogitsArgs a) {
  constexpr int E = EPL * 64;
  __shared__ __align__(16) uint32_t lds[4 * E];  // a row of every wave, or a maximum of every thread
  __shared__ int tokens;
  if ((int)blockIdx.x < a.weight_blocks) {  // (first: they take longest)
    split_weight<EPL>(a, blockIdx.x, lds);
    return;
  }
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  float(*const rows)[E] = (float(*)[E])lds;
  const int64_t base = (int64_t)((int)blockIdx.x - a.weight_blocks) * 4 * a.run;
  Seq q{0, 0, 0};
  float f[EPL] = {};
  bool have = false;
  const int64_t t0 = base + (int64_t)wave * a.run, t1 = min(t0 + a.run, (int64_t)a.seq.T);
  // the next token's loads are under way while one is computed
  float ahead[EPL] = {};
  int e_ahead = -1;
  float g_ahead = 0.f;
  auto fetch = [&](int64_t t) {
    if (t >= t1) return;
    Row<EPL>::load(a.logits + t * E, lane, ahead);
    if (a.dtopk_w && lane < a.K) {
      e_ahead = a.topk_idx[t * a.K + lane];
      g_ahead = a.dtopk_w[t * a.K + lane];
    }
  };
  fetch(t0);
  const Seqs seqs(a.seq, a.counts != nullptr);
  int b = 0;
  float g0 = 0.f;
  if (a.counts) {
    b = seqs.first((int)base);
    const int N = seqs.tokens(&tokens);
    g0 = N > 0 ? a.coef / (float)N : 0.f;
    if (a.dloss) g0 *= *a.dloss;
  }
  for (int64_t t = t0; t < t1; ++t) {
    float l[EPL], d[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) l[i] = ahead[i];
    const int e = (unsigned)e_ahead < (unsigned)E ? e_ahead : -1;
    const float dw = g_ahead;
    fetch(t + 1);
    Score s[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      s[i] = score_of(l[i]);
      d[i] = 0.f;
    }
    if (a.counts) {
      while (b < a.seq.n && (!have || q.next <= t)) {  // on to the token's sequence
        if (have) ++b;
        if (b >= a.seq.n) break;
        q = seqs.at(b);
        have = true;
        if (q.next <= t) continue;
        int32_t c[EPL];
        Row<EPL>::load(a.counts + (int64_t)b * E, lane, c);
        const float per = q.end > q.begin ? (float)E / ((float)a.K * (float)(q.end - q.begin)) : 0.f;
#pragma unroll
        for (int i = 0; i < EPL; ++i) f[i] = (float)c[i] * per;
      }
      if (b < a.seq.n && t >= q.begin && t < q.end) {
        float total = 0.f, load = 0.f;
        auto add = [&]() {
          total = load = 0.f;
#pragma unroll
          for (int i = 0; i < EPL; ++i) {
            total += s[i].s;
            load += f[i] * s[i].s;
          }
          total = wave_sum(total);
          load = wave_sum(load);
        };
        add();
        if (total < SCORES_TINY) {
#pragma unroll
          for (int i = 0; i < EPL; ++i) s[i].s = tiny_score(l[i]);
          add();
          // shares in place of scores: a large gradient times this sum's reciprocal may leave fp32's range
          const float part = total == 0.f ? 0.f : 1.0f / total;
#pragma unroll
          for (int i = 0; i < EPL; ++i) s[i].s *= part;
          load *= part;
          total = 1.f;
        }
        const float inv = 1.0f / total, mean = load * inv, g = g0 * inv;
#pragma unroll
        for (int i = 0; i < EPL; ++i) d[i] = g * (f[i] - mean) * s[i].s * s[i].r;
      }
    }
    if (a.dtopk_w) {
      // the chosen experts' logits to their lanes, their gradients back, through the wave's row in LDS (a wave's
      // LDS accesses run in order; the compiler, which sees one lane, must keep them so)
      Row<EPL>::store(rows[wave], lane, l);
      asm volatile("" ::: "memory");
      Score k{0.f, 0.f};
      float g = 0.f, v = 0.f, chosen = 0.f;
      if (e >= 0) {
        chosen = rows[wave][e];
        k = score_of(chosen);
        g = dw * a.scale;
      }
      const float zero[EPL] = {};
      asm volatile("" ::: "memory");
      Row<EPL>::store(rows[wave], lane, zero);
      if (a.norm) {
        float total = lane_of(row_sum(k.s), 0);  // (K <= 16: one row of lanes)
        if (total < SCORES_TINY) {
          k.s = e >= 0 ? tiny_score(chosen) : 0.f;
          total = lane_of(row_sum(k.s), 0);
        }
        const float share = total == 0.f ? 0.f : k.s / total;
        const float mean = lane_of(row_sum(g * share), 0);
        v = (g - mean) * share * k.r;
      } else {
        v = g * k.s * k.r;
      }
      asm volatile("" ::: "memory");
      if (e >= 0) atomicAdd(&rows[wave][e], v);
      asm volatile("" ::: "memory");
      float add[EPL];
      Row<EPL>::load(rows[wave], lane, add);
#pragma unroll
      for (int i = 0; i < EPL; ++i) d[i] += add[i];
    }
    if (a.dlogits) Row<EPL>::store(a.dlogits + t * E, lane, d);
    uint32_t top = 0;
    if (a.bf || a.hf) {
#pragma unroll
      for (int i = 0; i < EPL; ++i) top = max(top, __float_as_uint(d[i]) & 0x7FFFFFFFu);
      top = wave_max_u32(top);
    }
    if (a.bf) {
      if (lane == 0) a.live[t] = top != 0;
      Pieces<EPL, 3> p;
#pragma unroll
      for (int i = 0; i < EPL; i += 2) {
        uint32_t x[3], y[3];
        bf16_pieces(d[i], x);
        bf16_pieces(i + 1 < EPL ? d[i + 1] : 0.f, y);
#pragma unroll
        for (int k = 0; k < 3; ++k) p.w[k][i / 2] = x[k] >> 16 | y[k];
      }
      p.store(a.bf, (int64_t)a.seq.T * E, lane, [&](int e) { return t * E + e; });
    }
    if (a.hf) {
      const int ex = half_exponent(top);
      Pieces<EPL, 2> p;
#pragma unroll
      for (int i = 0; i < EPL; i += 2) half_pieces(d[i], i + 1 < EPL ? d[i + 1] : 0.f, ex, p.w[0][i / 2], p.w[1][i / 2]);
      p.store(a.hf, plane_size(a.seq.T, E), lane, [&](int e) { return plane_at(t, e, E); });
      if (lane == 0) a.hexp[t] = ex;
    }
  }
}

}  // namespace

// Up to so many tokens and logits one workgroup does it all, one sequence after another.  Sides measured (us a
// call, one launch / two): 64 tokens of 512 experts 7.8 / 9.7, in 2 sequences 8.8 / 10.5, in 3 11.7 / 10.8; 128 tokens
// 11.9 / 10.9; 256 tokens of 64 experts 8.7 / 9.9, in 4 sequences 9.7 / 10.1, in 6 11.7 / 9.8; 512 tokens 14.2 / 10.8.
constexpr int BALANCE_SMALL_T = 256, BALANCE_SMALL_SEQ = 4;
constexpr int64_t BALANCE_SMALL = 32768, BALANCE_SMALL_RUNS = 65536;

// Tokens of a chunk: about one workgroup for each of the MI355X's 256 compute units, from 32 (four a wave, whose
// loads are under way at once) to 256.  Sides measured (us a call, 512 experts): 8192 tokens 16 14.2, 32 12.8, 64 15.1; 16,384 32
// 17.7, 64 15.2, 128 20.4; 32,768 64 23.8, 128 22.5, 256 32.3; 200,000 128 107, 256 105.  But no longer than a
// sequence on average, down to 4, as a workgroup takes its sequences one after another: 65 tokens in 16
// sequences 10.8, in chunks of 32 25.3; 257 tokens of 64 experts in 64 sequences 10.0, 14.6.
int balance_chunk(int64_t T, int n_seq) {
  int c = 32;
  while (c < 256 && T > (int64_t)c * 256) c *= 2;
  while (c > 4 && (int64_t)c * n_seq > T) c /= 2;
  return c;
}

// The number of chunks falls where their size steps up: the most lie at the last T of each size.
int64_t balance_chunks_bound(int64_t T, int n_seq) {
  auto chunks = [&](int64_t t) {
    const int c = balance_chunk(t, n_seq);
    return (t + c - 1) / c;
  };
  int64_t most = std::max<int64_t>(chunks(T), 1);
  for (int64_t c = 8; c <= 256; c *= 2) {  // the first T of chunks of c tokens
    const int64_t from = std::max<int64_t>(c * n_seq, c > 32 ? c / 2 * 256 + 1 : 0);
    if (from <= T) most = std::max(most, chunks(from - 1));
  }
  return most;
}

#define MOE_EPL(E, F)          \
  switch ((E) / WAVE) {        \
    case 1: F(1); break;       \
    case 2: F(2); break;       \
    case 4: F(4); break;       \
    case 8: F(8); break;       \
    case 16: F(16); break;     \
    default: return hipErrorInvalidValue; \
  }

hipError_t launch_balance(const BalanceArgs& a, hipStream_t s) {
  if (a.seq.T <= BALANCE_SMALL_T && a.seq.T * a.E <= BALANCE_SMALL && a.seq.n <= BALANCE_SMALL_SEQ &&
      a.seq.T * a.E * a.seq.n <= BALANCE_SMALL_RUNS) {
#define MOE_BAL(N) hipLaunchKernelGGL(balance_small_kernel<N>, dim3(1), dim3(1024), 0, s, a)
    MOE_EPL(a.E, MOE_BAL)
#undef MOE_BAL
    return hipGetLastError();
  }
  const unsigned chunks = (unsigned)(((int64_t)a.seq.T + a.chunk - 1) / a.chunk);
#define MOE_BAL(N) hipLaunchKernelGGL(balance_partial_kernel<N>, dim3(std::max(chunks, 1u)), dim3(BAL_WAVES * 64), 0, s, a)
  MOE_EPL(a.E, MOE_BAL)
#undef MOE_BAL
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  // Sides measured (us a call, a workgroup each / a wave each): 128 pairs 13.1 / 15.5, 256 14.7 / 15.3, 512 18.3 /
  // 15.2, 2048 47 / 21, 8192 145 / 30.
  const int pairs = a.seq.n * (a.E / 64);
  if (pairs <= 256)
    hipLaunchKernelGGL(balance_finish_kernel<false>, dim3((unsigned)pairs), dim3(1024), 0, s, a);
  else
    hipLaunchKernelGGL(balance_finish_kernel<true>, dim3((unsigned)((pairs + 15) / 16)), dim3(1024), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_dlogits(DlogitsArgs a, hipStream_t s) {
  if (a.seq.T == 0) return hipSuccess;
  // 4096 waves, four on each SIMD, until a wave has eight tokens.  Measured (us, 16,384 tokens of 256 experts):
  // 2048 waves 14.0, 4096 12.3, 8192 13.2, 16,384 15.6 (each finds its sequence and loads its counts)
  a.run = (int)std::min<int64_t>(std::max<int64_t>(a.seq.T / 4096, 1), 8);
  a.weight_blocks = a.hf ? a.H / 16 : 0;
  const unsigned grid = (unsigned)(a.weight_blocks + ((int64_t)a.seq.T + 4 * a.run - 1) / (4 * a.run));
#define MOE_DL(N) hipLaunchKernelGGL(dlogits_kernel<N>, dim3(grid), dim3(256), 0, s, a)
  MOE_EPL(a.E, MOE_DL)
#undef MOE_DL
  return hipGetLastError();
}

}  // namespace moe
