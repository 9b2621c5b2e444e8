// AdamW over many tensors in one launch, with optimiser states in 32 or 8 bits.
//
//   m' = b1 m + (1-b1) g;   v' = b2 v + (1-b2) g^2
//   p' = p (1 - lr wd) - lr / (1-b1^t) * m' / (sqrt(v' / (1-b2^t)) + eps)
//
// Every product and sum of m' and v' is rounded to fp32 by itself (no fused multiply-add), so the
// 8-bit codes below follow bit for bit from the same operations in any fp32 arithmetic.
//
// 8-bit states: 128 consecutive values of a tensor share an fp32 scale, their largest magnitude /
// 1.875, so the largest is always a code of its own and the whole block can shrink by its scale.
//   first moment   sign, 4 exponent and 3 mantissa bits: (1 + f/8) 2^(e-15), code 0 is zero
//   second moment  5 exponent and 3 mantissa bits:       (1 + f/8) 2^(e-31) (never zero unless
//                  the block is, so the quotient m / sqrt(v) cannot run away)
// A moment moves by 0.1 % a step where its code's step is 6-12 %, so rounding to the nearest
// would hold it in place; the codes are rounded stochastically instead, by 16 bits of a hash of
// (seed, step, tensor, element) added below the kept bits: the same on every run, and unbiased within
// the codes' range.  Below it the rounding is not: a first moment of at most 2^-15 of its block's scale
// (1.6e-5 of the largest magnitude) becomes zero, and between that and the smallest code, 1.125 2^-15,
// the mean read back rises from zero to the value; a second moment below 2^-31 of its scale is raised
// to it.  So an element whose gradients stay 60,000 times below its block's largest is not moved.
// The two moments of an element are rounded by the same bits: each alone is unbiased, their errors are
// not independent.
//
// One workgroup takes a chunk of 8192 values found by one load from the plan; a lane takes 8
// consecutive values at a time, so 16 lanes (one DPP row) hold a block and its maximum takes four
// lane permutations, no LDS.  Streaming: 10 + 16/128 bytes per value with bf16 parameters and
// 8-bit states, 22 with 32-bit states, 28 with master weights besides.  755 M values of 384 tensors
// in 8 bits on one MI355X: 1.42-1.48 ms, 5.2-5.4 TB/s (eps 1e-15: 1.55 ms); both moments read out as
// fp32: 1.27 ms, 6.0 TB/s (a copy moves 4.9, a fill 6.9).  The vector units are near their limit there
// (about 60 operations a value), which is why the codes are packed by byte permutes.
#include "moe_common.h"
#include "moe_internal.h"

namespace moe {

namespace {

constexpr float STATE_TOP = 1.875f;  // the largest code
constexpr int M_BIAS = (127 - 15) << 3, V_BIAS = (127 - 31) << 3;

__device__ __forceinline__ uint32_t dpp_max16(uint32_t v) {
  // xor 1, xor 2 (quad permutations), then the mirrors of 8 and of 16 lanes
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, true));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, true));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xF, 0xF, true));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x140, 0xF, 0xF, true));
  return v;
}

// 32 random bits of a pair of values: an index hash of multiplications by odd constants and shifts
// (`x`: pair * HASH_STEP + key, which the pairs of a lane reach by additions).  The three multipliers are
// those of the grid-cell hash in Ericson, Real-Time Collision Detection (2005), chapter 7; the key's
// (0x9E3779B9, 0x7F4A7C15) are the halves of 2^64 divided by the golden ratio.
constexpr uint32_t HASH_STEP = 0x8DA6B343u;
__device__ __forceinline__ uint32_t pair_bits(uint32_t x) {
  x ^= x >> 15;
  x *= 0xD8163841u;
  x ^= x >> 13;
  x *= 0xCB1AB31Fu;
  x ^= x >> 16;
  return x;
}

template <bool SIGNED>
__device__ __forceinline__ float decode(uint32_t c, float scale) {
  if constexpr (SIGNED) {
    const uint32_t mag = c & 127u;
    const uint32_t bits = ((mag << 20) + ((uint32_t)M_BIAS << 20)) | ((c & 128u) << 24);
    return (mag ? __uint_as_float(bits) : 0.f) * scale;
  } else {
    return __uint_as_float((c << 20) + ((uint32_t)V_BIAS << 20)) * scale;
  }
}

// A code still among the bits above it (bits 8 and up are not cleared): |x| / scale with 16 random
// bits added below the kept ones.  The bias of the exponent field is no more than set bits above
// the code (and its bit 7, which the sign replaces), so nothing is subtracted.
template <bool SIGNED>
__device__ __forceinline__ uint32_t encode(float x, float inv, uint32_t r16) {
  static_assert(V_BIAS == 0x300 && M_BIAS == 0x380, "the biases lie above the codes");
  constexpr int LO = SIGNED ? M_BIAS : V_BIAS, HI = LO + (SIGNED ? 127 : 255);
  const int bits = (__float_as_int(fabsf(x) * inv) + (int)(r16 << 4)) >> 20;
  const uint32_t c = (uint32_t)min(max(bits, LO), HI);
  return SIGNED ? (c & 0x7Fu) | (__float_as_uint(x) >> 24 & ~0x7Fu) : c;
}

// eight values -> their block's scale, the codes in two words
template <bool SIGNED>
__device__ __forceinline__ float encode8(const float (&x)[8], const uint32_t (&rnd)[4], u32x2& codes) {
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(x[j]) & 0x7FFFFFFFu);
  float scale = __uint_as_float(dpp_max16(top)) * (1.0f / STATE_TOP);
  if (scale < 0x1p-126f) scale = 0.f;  // below the normal range: the block is stored as zeros
  const float inv = scale > 0.f ? 1.0f / scale : 0.f;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t c[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t r = rnd[h * 2 + j / 2];
      c[j] = encode<SIGNED>(x[h * 4 + j], inv, j & 1 ? r >> 16 : r & 0xFFFFu);
    }
    // the low bytes of four words
    const uint32_t lo = __builtin_amdgcn_perm(c[1], c[0], 0x0C0C0400u), hi = __builtin_amdgcn_perm(c[3], c[2], 0x0C0C0400u);
    codes[h] = lo | hi << 16;
  }
  return scale;
}

// eight consecutive values from i on, zeros past n
template <bool F32>
__device__ __forceinline__ void load8(const void* p, int64_t i, int64_t n, float (&v)[8]) {
  if (i + 8 <= n) {
    if constexpr (F32) {
      const floatx4 a = *(const floatx4*)((const float*)p + i), b = *(const floatx4*)((const float*)p + i + 4);
#pragma unroll
      for (int j = 0; j < 4; ++j) { v[j] = a[j]; v[4 + j] = b[j]; }
    } else {
      const u32x4 a = *(const u32x4*)((const uint16_t*)p + i);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[2 * j] = __uint_as_float(a[j] << 16);
        v[2 * j + 1] = __uint_as_float(a[j] & 0xFFFF0000u);
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      v[j] = i + j >= n ? 0.f : F32 ? ((const float*)p)[i + j] : bf16_bits_to_f32(((const uint16_t*)p)[i + j]);
  }
}

template <bool F32>
__device__ __forceinline__ void store8(void* p, int64_t i, int64_t n, const float (&v)[8]) {
  if (i + 8 <= n) {
    if constexpr (F32) {
      *(floatx4*)((float*)p + i) = floatx4{v[0], v[1], v[2], v[3]};
      *(floatx4*)((float*)p + i + 4) = floatx4{v[4], v[5], v[6], v[7]};
    } else {
      *(u32x4*)((uint16_t*)p + i) = u32x4{f32x2_to_bf16x2(v[0], v[1]), f32x2_to_bf16x2(v[2], v[3]),
                                          f32x2_to_bf16x2(v[4], v[5]), f32x2_to_bf16x2(v[6], v[7])};
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (i + j < n) {
        if constexpr (F32) ((float*)p)[i + j] = v[j];
        else ((uint16_t*)p)[i + j] = (uint16_t)f32x2_to_bf16x2(v[j], 0.f);
      }
  }
}

__device__ __forceinline__ u32x2 load_codes(const uint8_t* p, int64_t i, int64_t n) {
  if (i + 8 <= n) return *(const u32x2*)(p + i);
  u32x2 r{0, 0};
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (i + j < n) r[j / 4] |= (uint32_t)p[i + j] << (8 * (j & 3));
  return r;
}

__device__ __forceinline__ void store_codes(uint8_t* p, int64_t i, int64_t n, const u32x2& c) {
  if (i + 8 <= n) {
    *(u32x2*)(p + i) = c;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (i + j < n) p[i + j] = (uint8_t)(c[j / 4] >> (8 * (j & 3)));
  }
}

// m / (sqrt(v inv_c2) + eps).  The hardware's square root and reciprocal take values below 2^-126 as
// zero.  With eps of 2^-39 or more that is at most 2^-63 / 2^-39 of the quotient, a rounding; with less
// (EXACT), v is scaled up under its root and the quotient is divided out.  A branch of the whole launch:
// the division alone is ten operations a value.
template <bool EXACT>
__device__ __forceinline__ float quotient(float m, float v, float inv_c2, float eps) {
#pragma clang fp contract(off)
  if constexpr (!EXACT) return m * __builtin_amdgcn_rcpf(__builtin_amdgcn_sqrtf(v * inv_c2) + eps);
  const bool small = v < 0x1p-96f;
  const float root = __builtin_amdgcn_sqrtf((small ? v * 0x1p32f : v) * inv_c2);
  return m / ((small ? root * 0x1p-16f : root) + eps);
}
constexpr float EPS_EXACT = 0x1p-39f;

template <bool PF32, bool GF32, bool EIGHT, bool MASTER>
__global__ __launch_bounds__(256) void adamw_kernel(AdamWArgs a) {
#pragma clang fp contract(off)
  const AdamWHeader* hd = (const AdamWHeader*)a.image;
  // what is no image, or one of other sizes or types, is not followed
  if (hd->magic != ADAMW_MAGIC || hd->n_tensors != a.n_tensors || hd->n_chunks != a.n_chunks || hd->flags != a.flags)
    return;
  const AdamWTensor* ts = (const AdamWTensor*)(hd + 1);
  const AdamWChunk ck = ((const AdamWChunk*)(ts + a.n_tensors))[blockIdx.x];
  const AdamWTensor t = ts[ck.tensor];

  float lr = a.lr, inv_c1 = a.inv_c1, inv_c2 = a.inv_c2;
  uint32_t step = a.step;
  if (a.lr_ptr) lr = *a.lr_ptr;
  if (a.step_ptr) {
    __shared__ float corr[2];
    const int64_t st = *a.step_ptr;
    if (st < 1) return;  // no step: its bias corrections would make every parameter infinite or NaN
    if (threadIdx.x == 0) {
      corr[0] = (float)(1.0 / (1.0 - pow(a.beta1, (double)st)));
      corr[1] = (float)(1.0 / (1.0 - pow(a.beta2, (double)st)));
    }
    __syncthreads();
    inv_c1 = corr[0];
    inv_c2 = corr[1];
    step = (uint32_t)st;
  }
  const float gscale = a.grad_scale ? *a.grad_scale : 1.f;
  const float decay = 1.f - lr * t.weight_decay, rate = lr * inv_c1;
  const uint32_t key = (uint32_t)ck.tensor * 0x9E3779B9u + a.seed + step * 0x7F4A7C15u;
  const int64_t n = t.numel;

#pragma unroll 1
  for (int it = 0; it < ADAMW_CHUNK / 2048; ++it) {
    const int64_t i = (int64_t)ck.chunk * ADAMW_CHUNK + it * 2048 + threadIdx.x * 8;
    // whole blocks of 128 leave together: their 16 lanes share a maximum
    if (i / ADAMW_BLOCK * ADAMW_BLOCK >= n) break;
    float g[8], m[8], v[8], p[8];
    load8<GF32>(t.grad, i, n, g);
    if (a.grad_scale) {
#pragma unroll
      for (int j = 0; j < 8; ++j) g[j] = g[j] * gscale;
    }
    if constexpr (MASTER) load8<true>(t.master, i, n, p);
    else load8<PF32>(t.param, i, n, p);
    if constexpr (EIGHT) {
      const u32x2 mc = load_codes((const uint8_t*)t.m, i, n), vc = load_codes((const uint8_t*)t.v, i, n);
      const float ms = t.ms[i / ADAMW_BLOCK], vs = t.vs[i / ADAMW_BLOCK];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        m[j] = decode<true>((mc[j / 4] >> (8 * (j & 3))) & 255u, ms);
        v[j] = decode<false>((vc[j / 4] >> (8 * (j & 3))) & 255u, vs);
      }
    } else {
      load8<true>(t.m, i, n, m);
      load8<true>(t.v, i, n, v);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      m[j] = m[j] * a.b1 + g[j] * a.omb1;
      v[j] = v[j] * a.b2 + g[j] * g[j] * a.omb2;
    }
    if (a.eps >= EPS_EXACT) {
#pragma unroll
      for (int j = 0; j < 8; ++j) p[j] = __builtin_fmaf(quotient<false>(m[j], v[j], inv_c2, a.eps), -rate, p[j] * decay);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) p[j] = __builtin_fmaf(quotient<true>(m[j], v[j], inv_c2, a.eps), -rate, p[j] * decay);
    }
    if (EIGHT && i + 8 > n) {  // past the end: no part of the block's maximum
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (i + j >= n) m[j] = v[j] = 0.f;
    }
    if constexpr (MASTER) store8<true>(t.master, i, n, p);
    store8<PF32>(t.param, i, n, p);
    if constexpr (EIGHT) {
      uint32_t rnd[4];
      const uint32_t hash0 = (uint32_t)(i >> 1) * HASH_STEP + key;
#pragma unroll
      for (int j = 0; j < 4; ++j) rnd[j] = pair_bits(hash0 + j * HASH_STEP);
      u32x2 mc, vc;
      const float ms = encode8<true>(m, rnd, mc), vs = encode8<false>(v, rnd, vc);
      store_codes((uint8_t*)t.m, i, n, mc);
      store_codes((uint8_t*)t.v, i, n, vc);
      if ((threadIdx.x & 15) == 0) {
        t.ms[i / ADAMW_BLOCK] = ms;
        t.vs[i / ADAMW_BLOCK] = vs;
      }
    } else {
      store8<true>(t.m, i, n, m);
      store8<true>(t.v, i, n, v);
    }
  }
}

template <bool SIGNED>
__global__ __launch_bounds__(256) void dequantise_kernel(const uint8_t* codes, const float* scales, int64_t n, float* out) {
  for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8; i < n; i += (int64_t)gridDim.x * 2048) {
    const u32x2 c = load_codes(codes, i, n);
    const float s = scales[i / ADAMW_BLOCK];
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = decode<SIGNED>((c[j / 4] >> (8 * (j & 3))) & 255u, s);
    store8<true>(out, i, n, v);
  }
}

}  // namespace

hipError_t launch_adamw(const AdamWArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)a.n_chunks), block(256);
  const bool pf = a.flags & ADAMW_PARAM_F32, gf = a.flags & ADAMW_GRAD_F32, e = a.flags & ADAMW_EIGHT, m = a.flags & ADAMW_MASTER;
#define MOE_ADAMW(PF, GF, E, M) \
  if (pf == PF && gf == GF && e == E && m == M) hipLaunchKernelGGL((adamw_kernel<PF, GF, E, M>), grid, block, 0, s, a)
  MOE_ADAMW(false, false, false, false);
  MOE_ADAMW(false, false, false, true);
  MOE_ADAMW(false, false, true, false);
  MOE_ADAMW(false, false, true, true);
  MOE_ADAMW(false, true, false, false);
  MOE_ADAMW(false, true, false, true);
  MOE_ADAMW(false, true, true, false);
  MOE_ADAMW(false, true, true, true);
  MOE_ADAMW(true, false, false, false);
  MOE_ADAMW(true, false, true, false);
  MOE_ADAMW(true, true, false, false);
  MOE_ADAMW(true, true, true, false);
#undef MOE_ADAMW
  return hipGetLastError();
}

hipError_t launch_adamw_dequantise(const uint8_t* codes, const float* scales, int64_t n, bool is_signed, float* out,
                                   hipStream_t s) {
  const int64_t grid = std::min<int64_t>((n + 2047) / 2048, (int64_t)1 << 20);
  if (is_signed) hipLaunchKernelGGL(dequantise_kernel<true>, dim3((unsigned)grid), dim3(256), 0, s, codes, scales, n, out);
  else hipLaunchKernelGGL(dequantise_kernel<false>, dim3((unsigned)grid), dim3(256), 0, s, codes, scales, n, out);
  return hipGetLastError();
}

}  // namespace moe
