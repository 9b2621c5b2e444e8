// Norm over many gradients, and clipping.
//
//   norm = |scale| sqrt(sum over all tensors of g^2);   coef = scale (1 if norm <= max_norm, else max_norm / norm)
//   out = coef g
//
// The gradients are read once, in chunks of GRAD_CHUNK values that a table lists; the workgroups are
// as many as fit the card and take every grid-th chunk, each leaving one sum in 64 bits; a second
// launch of one workgroup adds them in order.  Squares are summed in fp32 within a lane's share of a
// chunk (32 values), in 64 bits from there on.  A share whose sum leaves 2^-60 .. 2^120 (all zeros
// apart) is read again with squares in 64 bits: gradients whose squares overflow or vanish in fp32 have
// a norm too.
//
// What bounds it, on one MI355X: HBM.  755 M bf16 values in 388 tensors 250 us a call, 6.05 TB/s (the reading
// kernel 239-247, the adding one 4-5); 94.5 M fp32 values with clipping into bf16 175, of which the norm 70-74
// and the clipping 87-90: 945 MB in all at 5.4 TB/s.  1.3 M values: three launches of 2.9, 2.0 and 3.4 us, and
// as long on the host.  Chunks of 16,384 values were as fast (249 and 181 us); loads one after another instead of a
// chunk's at once, and a table of tensors behind the chunks', took 286 and 6.6 us (small) for the norm.
#include <type_traits>

#include "moe_common.h"
#include "moe_internal.h"

namespace moe {

namespace {

// eight values from i on, zeros past n
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

// A lane's share of a chunk of n values, squared in fp32, or (WIDE) in 64 bits.  `any`: the bits of its
// values, or-ed, signs apart.
template <bool F32, bool WIDE>
__device__ __forceinline__ double chunk_sum(const void* p, int n, uint32_t& any) {
  typedef std::conditional_t<WIDE, double, float> sum_t;
  sum_t s[2] = {0, 0};
  any = 0;
  auto add = [&](float v, int j) {
    if constexpr (WIDE) s[j] += (double)v * (double)v;
    else s[j] = __builtin_fmaf(v, v, s[j]);
  };
  if (n == GRAD_CHUNK) {
    constexpr int W = GRAD_CHUNK / 2048 * (F32 ? 2 : 1);
    u32x4 w[W];  // all loads at once
#pragma unroll
    for (int i = 0; i < W; ++i) w[i] = ((const u32x4*)p)[i * 256 + threadIdx.x];
#pragma unroll
    for (int i = 0; i < W; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        any |= w[i][j] & (F32 ? 0x7FFFFFFFu : 0x7FFF7FFFu);
        if constexpr (F32) {
          add(__uint_as_float(w[i][j]), j & 1);
        } else {
          add(__uint_as_float(w[i][j] << 16), 0);
          add(__uint_as_float(w[i][j] & 0xFFFF0000u), 1);
        }
      }
  } else {
    for (int i = threadIdx.x * 8; i < n; i += 2048) {
      float v[8];
      load8<F32>(p, i, n, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        any |= __float_as_uint(v[j]) & 0x7FFFFFFFu;
        add(v[j], j & 1);
      }
    }
  }
  return (double)s[0] + (double)s[1];
}
template <bool F32>
__device__ __forceinline__ double chunk_sum(const void* p, int n) {
  uint32_t any;
  const double s = chunk_sum<F32, false>(p, n, any);
  if (s < 0x1p120 && (s > 0x1p-60 || any == 0)) return s;
  return chunk_sum<F32, true>(p, n, any);
}

// what is no image, or one of other sizes, is not followed
__device__ __forceinline__ bool is_image(const GradArgs& a) {
  const GradHeader* hd = (const GradHeader*)a.image;
  return hd->magic == GRAD_MAGIC && hd->n_tensors == a.n_tensors && hd->n_chunks == a.n_chunks;
}
__device__ __forceinline__ const GradChunk* chunks_of(const GradArgs& a) { return (const GradChunk*)(a.image + sizeof(GradHeader)); }

__global__ __launch_bounds__(256) void grad_norm_kernel(GradArgs a) {
  __shared__ double sums[4];
  double total = 0;
  if (is_image(a)) {
    GradChunk next = chunks_of(a)[blockIdx.x];
    for (int64_t c = blockIdx.x; c < a.n_chunks;) {
      const GradChunk ck = next;
      c += gridDim.x;
      if (c < a.n_chunks) next = chunks_of(a)[c];
      total += ck.flags & GRAD_IN_F32 ? chunk_sum<true>(ck.in, ck.n) : chunk_sum<false>(ck.in, ck.n);
    }
  }
  total = wave_sum_f64(total);
  if ((threadIdx.x & 63) == 0) sums[threadIdx.x >> 6] = total;
  __syncthreads();
  if (threadIdx.x == 0) a.partial[blockIdx.x] = (sums[0] + sums[1]) + (sums[2] + sums[3]);
}

__global__ __launch_bounds__(1024) void grad_norm_finish_kernel(GradArgs a, int n) {
  __shared__ double sums[16];
  double v[GRAD_MAX_PARTIALS / 1024], s = 0;
  if (n > 0) {
#pragma unroll
    for (int i = 0; i < GRAD_MAX_PARTIALS / 1024; ++i) v[i] = a.partial[min(i * 1024 + (int)threadIdx.x, n - 1)];
    if (!is_image(a)) return;
#pragma unroll
    for (int i = 0; i < GRAD_MAX_PARTIALS / 1024; ++i) s += i * 1024 + (int)threadIdx.x < n ? v[i] : 0.0;
  }
  s = wave_sum_f64(s);
  if ((threadIdx.x & 63) == 0) sums[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    s = 0;
    for (int w = 0; w < 16; ++w) s += sums[w];
    const double norm = fabs(a.scale) * sqrt(s);
    *a.norm = (float)norm;
    // (a NaN norm gives a NaN coefficient, an infinite one zero, also where max_norm is infinite)
    if (a.coef_out) *a.coef_out = (float)(a.scale * (isinf(norm) ? 0.0 : norm <= a.max_norm ? 1.0 : a.max_norm / norm));
  }
}

template <bool IF32, bool OF32>
__device__ __forceinline__ void clip_chunk(const GradChunk& ck, float c) {
  if (ck.n == GRAD_CHUNK) {  // the loads of half a chunk at once
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      constexpr int N = GRAD_CHUNK / 4096;
      u32x4 w[N][IF32 ? 2 : 1];
#pragma unroll
      for (int i = 0; i < N; ++i)
#pragma unroll
        for (int k = 0; k < (IF32 ? 2 : 1); ++k)
          w[i][k] = ((const u32x4*)ck.in)[((h * N + i) * 256 + threadIdx.x) * (IF32 ? 2 : 1) + k];
#pragma unroll
      for (int i = 0; i < N; ++i) {
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if constexpr (IF32) v[j] = __uint_as_float(w[i][j / 4][j & 3]) * c;
          else v[j] = __uint_as_float(j & 1 ? w[i][0][j / 2] & 0xFFFF0000u : w[i][0][j / 2] << 16) * c;
        }
        store8<OF32>(ck.out, ((int64_t)(h * N + i) * 256 + threadIdx.x) * 8, GRAD_CHUNK, v);
      }
    }
  } else {
    for (int i = threadIdx.x * 8; i < ck.n; i += 2048) {
      float v[8];
      load8<IF32>(ck.in, i, ck.n, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] *= c;
      store8<OF32>(ck.out, i, ck.n, v);
    }
  }
}

__global__ __launch_bounds__(256) void grad_clip_kernel(GradArgs a) {
  const float c = *a.coef;
  if (!is_image(a)) return;
  // from the last chunk to the first: what the norm read last is still in the Infinity Cache
  const GradChunk ck = chunks_of(a)[a.n_chunks - 1 - blockIdx.x];
  if (ck.in == ck.out && c == 1.f) return;  // in place: nothing changes
  switch (ck.flags & (GRAD_IN_F32 | GRAD_OUT_F32)) {
    case 0: clip_chunk<false, false>(ck, c); break;
    case GRAD_IN_F32: clip_chunk<true, false>(ck, c); break;
    case GRAD_OUT_F32: clip_chunk<false, true>(ck, c); break;
    default: clip_chunk<true, true>(ck, c);
  }
}

}  // namespace

hipError_t launch_grad_norm(const GradArgs& a, hipStream_t s) {
  const int cus = device_cu_count();
  if (cus <= 0) return hipErrorInvalidDevice;
  // as many workgroups as the card holds: few sums to add, no second round
  const int grid = (int)std::min<int64_t>(std::min<int64_t>(a.n_chunks, (int64_t)cus * 8), GRAD_MAX_PARTIALS);
  if (grid > 0) hipLaunchKernelGGL(grad_norm_kernel, dim3((unsigned)grid), dim3(256), 0, s, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(grad_norm_finish_kernel, dim3(1), dim3(1024), 0, s, a, grid);
  return hipGetLastError();
}

hipError_t launch_grad_clip(const GradArgs& a, hipStream_t s) {
  if (a.n_chunks == 0) return hipSuccess;
  hipLaunchKernelGGL(grad_clip_kernel, dim3((unsigned)a.n_chunks), dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace moe
