// Device code shared by the kernels that read the router's logits: sigmoid scores, sums over a
// wave, the sequences of a batch.
#pragma once
#include "moe_common.h"
#include "moe_internal.h"

namespace moe {

// exp(a) 2^up for a <= 0, through the hardware's power of two, which gives zero below fp32's normal range.  The
// product a log2(e) is carried with its rounding (else its 2^-24 would be multiplied by a).
__device__ __forceinline__ float exp_scaled(float a, float up) {
  a = a < -200.f ? -200.f : a;  // (far below what any use can tell from zero; NaN stays)
  const float t = a * 1.44269504f;
  const float lo = __builtin_fmaf(a, 1.44269504f, -t) + a * 1.92596299e-8f;
  float at;
  {
#pragma clang fp contract(off)
    at = t + up;  // (exact; as one operation with the product it would leave nothing for `lo` to correct)
  }
  const float e = __builtin_amdgcn_exp2f(at);
  return __builtin_fmaf(e, lo * 0.693147181f, e);
}

// sigmoid of a logit and its complement, both to a few ulp of themselves in fp32's normal range, zero below it
// (from |l| = 87.3 on): from e = exp(-|l|) <= 1 the larger is 1 / (1 + e), the smaller e times that.
struct Score {
  float s, r;  // sigmoid(l), 1 - sigmoid(l)
};
__device__ __forceinline__ Score score_of(float l) {
  const float e = exp_scaled(-fabsf(l), 0.f);
  const float big = __builtin_amdgcn_rcpf(1.0f + e), small = e * big;
  return l < 0.f ? Score{small, big} : Score{big, small};
}

// Quotients of scores whose sum is below SCORES_TINY are taken from 2^64 times the scores, or fp32 would hold
// the scores in few bits or none while their quotients are ordinary numbers.  Every logit is below -44 then: the
// sigmoid is exp(l), in full precision down to l = -131 and zero below that.
constexpr float SCORES_TINY = 0x1p-64f;
__device__ __forceinline__ float tiny_score(float l) { return exp_scaled(l, 64.f); }

// sum over the wave, in every lane: rows of 16 lanes by lane permutations (xor 1, xor 2, mirrors of 8
// and 16), the four rows by lane reads
template <int CTRL>
__device__ __forceinline__ float dpp_add(float v) {
  return v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, true));
}
__device__ __forceinline__ float row_sum(float v) {  // over 16 lanes
  v = dpp_add<0xB1>(v);
  v = dpp_add<0x4E>(v);
  v = dpp_add<0x141>(v);
  return dpp_add<0x140>(v);
}
__device__ __forceinline__ float lane_of(float v, int l) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), l));
}
__device__ __forceinline__ float wave_sum(float v) {
  v = row_sum(v);
  return (lane_of(v, 0) + lane_of(v, 16)) + (lane_of(v, 32) + lane_of(v, 48));
}

// A lane's experts of a row of E = 64 EPL values: pieces j of V consecutive ones, j * 64 V + lane * V,
// so that a piece of the wave is contiguous.
template <int EPL>
struct Row {
  static constexpr int V = EPL < 4 ? EPL : 4, NJ = EPL / V;
  typedef float vec __attribute__((ext_vector_type(V)));
  typedef int32_t ivec __attribute__((ext_vector_type(V)));
  static __device__ __forceinline__ int at(int lane, int j) { return j * 64 * V + lane * V; }
  static __device__ __forceinline__ void load(const float* p, int lane, float (&v)[EPL]) {
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const vec x = *(const vec*)(p + at(lane, j));
#pragma unroll
      for (int i = 0; i < V; ++i) v[j * V + i] = x[i];
    }
  }
  static __device__ __forceinline__ void load(const int32_t* p, int lane, int32_t (&v)[EPL]) {
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const ivec x = *(const ivec*)(p + at(lane, j));
#pragma unroll
      for (int i = 0; i < V; ++i) v[j * V + i] = x[i];
    }
  }
  static __device__ __forceinline__ void store(float* p, int lane, const float (&v)[EPL]) {
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      vec x;
#pragma unroll
      for (int i = 0; i < V; ++i) x[i] = v[j * V + i];
      *(vec*)(p + at(lane, j)) = x;
    }
  }
};

// The tokens of sequence b (begin <= t < end) and where the next sequence's run begins; all within
// [0, T] whatever the arrays hold.
struct Seq {
  int begin, end, next;
};
__device__ __forceinline__ Seq seq_at(const SeqArgs& q, int b) {
  Seq r{0, q.T, q.T};
  if (q.offsets) {
    r.begin = min(max(q.offsets[b], 0), q.T);
    r.next = r.end = min(max(q.offsets[b + 1], r.begin), q.T);
  }
  if (q.lens) r.end = r.begin + min(max(q.lens[b], 0), r.end - r.begin);
  return r;
}

__device__ __forceinline__ int wave_sum_i32(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0xB1, 0xF, 0xF, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x4E, 0xF, 0xF, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x141, 0xF, 0xF, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x140, 0xF, 0xF, true);
  auto at = [&](int l) { return __builtin_amdgcn_readlane(v, l); };
  return (at(0) + at(16)) + (at(32) + at(48));
}

// The sequences as a wave sees them.  Up to 64: one a lane, read at once, all questions answered without
// memory or other waves (balance loss of 16,384 tokens in 16 sequences 18.0 us a call, 20.6 the other way).
// More, or a single run: read as they are asked for, counted by the whole workgroup.
struct Seqs {
  const SeqArgs& q;
  bool few;
  Seq mine;
  // read: whether any question will be asked
  __device__ __forceinline__ explicit Seqs(const SeqArgs& args, bool read = true)
      : q(args), few(read && args.offsets && args.n <= 64), mine{0, 0, 0} {
    const int lane = threadIdx.x & 63;
    if (few && lane < q.n) mine = seq_at(q, lane);
  }
  // sequence b, the same in all lanes
  __device__ __forceinline__ Seq at(int b) const {
    if (!few) return seq_at(q, b);
    const int l = __builtin_amdgcn_readfirstlane(b);
    return {__builtin_amdgcn_readlane(mine.begin, l), __builtin_amdgcn_readlane(mine.end, l), __builtin_amdgcn_readlane(mine.next, l)};
  }
  // The first sequence whose run ends behind token t (n if none; 0 where there is but one): up to 64, counted;
  // more, sought in steps of 64 parts.
  __device__ __forceinline__ int first(int t) const {
    if (!q.offsets || q.n == 1) return 0;
    const int lane = threadIdx.x & 63;
    if (few) return __builtin_popcountll(__ballot(lane < q.n && mine.next <= t));
    int lo = 0;
    for (int n = q.n; n > 0;) {  // lo .. lo + n holds the answer
      const int part = (n + 63) / 64, at = (lane + 1) * part;  // each lane asks for the last of its part
      const int k = __builtin_popcountll(__ballot(at <= n && q.offsets[lo + min(at, n)] <= t));
      lo += k * part;
      n = min(part - 1, n - k * part);
    }
    return lo;
  }
  // Tokens of all sequences.  `count`: one int in LDS.
  __device__ __forceinline__ int tokens(int* count) const {
    if (few) return wave_sum_i32(mine.end - mine.begin);
    if (!q.lens) return q.offsets ? max(min(q.offsets[q.n], q.T) - max(q.offsets[0], 0), 0) : q.T;
    if (threadIdx.x == 0) *count = 0;
    __syncthreads();
    int c = 0;
    for (int b = threadIdx.x; b < q.n; b += blockDim.x) {
      const Seq s = seq_at(q, b);
      c += s.end - s.begin;
    }
    if (c) atomicAdd(count, c);
    __syncthreads();
    return *count;
  }
};

}  // namespace moe
