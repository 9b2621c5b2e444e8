// Norm over many gradients, and clipping.
//
//   norm = |scale| sqrt(sum over all tensors of g^2);   coef = scale (1 if norm <= max_norm, else max_norm / norm)
//   out = coef g
//
// The gradients are read once, in chunks of GRAD_CHUNK values that a table lists; the workgroups are
// as many as fit the card and take every grid-th chunk, each leaving one sum in 64 bits; a second
// launch of one workgroup adds them in order.  Squares are summed in fp32 within a lane's share of a
// chunk (at most 64 values), in 64 bits from there on.  A chunk whose sum leaves 2^-60 .. 2^120 is
// read again with squares in 64 bits: gradients whose squares overflow or vanish in fp32 have a
// norm too.
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

struct Table {
  const GradTensor* tensors;
  const GradChunk* chunks;
};
__device__ __forceinline__ bool open_table(const uint8_t* image, int64_t n_tensors, int64_t n_chunks, Table& t) {
  const GradHeader* hd = (const GradHeader*)image;
  // what is no image, or one of other sizes, is not followed
  if (hd->magic != GRAD_MAGIC || hd->n_tensors != n_tensors || hd->n_chunks != n_chunks) return false;
  t.tensors = (const GradTensor*)(hd + 1);
  t.chunks = (const GradChunk*)(t.tensors + n_tensors);
  return true;
}

// a lane's share of the chunk from value `base` on
template <bool F32>
__device__ __forceinline__ double chunk_sum(const void* p, int64_t base, int64_t n) {
  float s[2] = {0.f, 0.f};
#pragma unroll
  for (int it = 0; it < GRAD_CHUNK / 2048; ++it) {
    float v[8];
    load8<F32>(p, base + it * 2048 + threadIdx.x * 8, n, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) s[j & 1] = __builtin_fmaf(v[j], v[j], s[j & 1]);
  }
  return (double)s[0] + (double)s[1];
}
template <bool F32>
__device__ double chunk_sum_wide(const void* p, int64_t base, int64_t n) {
  double s = 0;
  for (int it = 0; it < GRAD_CHUNK / 2048; ++it) {
    float v[8];
    load8<F32>(p, base + it * 2048 + threadIdx.x * 8, n, v);
    for (int j = 0; j < 8; ++j) s += (double)v[j] * (double)v[j];
  }
  return s;
}

__device__ __forceinline__ double wave_sum_f64(double v) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) v += __shfl_xor(v, m, WAVE);
  return v;
}

__global__ __launch_bounds__(256) void grad_norm_kernel(GradArgs a) {
  __shared__ double sums[4];
  Table tb;
  double total = 0;
  if (open_table(a.image, a.n_tensors, a.n_chunks, tb)) {
    for (int64_t c = blockIdx.x; c < a.n_chunks; c += gridDim.x) {
      const GradChunk ck = tb.chunks[c];
      const GradTensor t = tb.tensors[ck.tensor];
      const int64_t base = (int64_t)ck.chunk * GRAD_CHUNK;
      double s = t.flags & GRAD_IN_F32 ? chunk_sum<true>(t.in, base, t.numel) : chunk_sum<false>(t.in, base, t.numel);
      // (a lane alone decides for its share; zeros need no second look, but come cheap)
      if (!(s > 0x1p-60 && s < 0x1p120)) s = t.flags & GRAD_IN_F32 ? chunk_sum_wide<true>(t.in, base, t.numel) : chunk_sum_wide<false>(t.in, base, t.numel);
      total += s;
    }
  }
  total = wave_sum_f64(total);
  if ((threadIdx.x & 63) == 0) sums[threadIdx.x >> 6] = total;
  __syncthreads();
  if (threadIdx.x == 0) a.partial[blockIdx.x] = (sums[0] + sums[1]) + (sums[2] + sums[3]);
}

__global__ __launch_bounds__(1024) void grad_norm_finish_kernel(GradArgs a, int n) {
  __shared__ double sums[16];
  const GradHeader* hd = (const GradHeader*)a.image;
  if (a.n_chunks && (hd->magic != GRAD_MAGIC || hd->n_tensors != a.n_tensors || hd->n_chunks != a.n_chunks)) return;
  double s = 0;
  for (int i = threadIdx.x; i < n; i += 1024) s += a.partial[i];
  s = wave_sum_f64(s);
  if ((threadIdx.x & 63) == 0) sums[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    s = 0;
    for (int w = 0; w < 16; ++w) s += sums[w];
    const double norm = fabs(a.scale) * sqrt(s);
    *a.norm = (float)norm;
    // (a NaN norm gives a NaN coefficient, an infinite one zero)
    if (a.coef_out) *a.coef_out = (float)(a.scale * (norm <= a.max_norm ? 1.0 : a.max_norm / norm));
  }
}

template <bool IF32, bool OF32>
__device__ __forceinline__ void clip_chunk(const GradTensor& t, int64_t base, float c) {
#pragma unroll
  for (int it = 0; it < GRAD_CHUNK / 2048; ++it) {
    const int64_t i = base + it * 2048 + threadIdx.x * 8;
    if (i >= t.numel) break;
    float v[8];
    load8<IF32>(t.in, i, t.numel, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] *= c;
    store8<OF32>(t.out, i, t.numel, v);
  }
}

__global__ __launch_bounds__(256) void grad_clip_kernel(GradArgs a) {
  Table tb;
  if (!open_table(a.image, a.n_tensors, a.n_chunks, tb)) return;
  const float c = *a.coef;
  const GradChunk ck = tb.chunks[blockIdx.x];
  const GradTensor t = tb.tensors[ck.tensor];
  if (t.in == t.out && c == 1.f) return;  // in place: nothing changes
  const int64_t base = (int64_t)ck.chunk * GRAD_CHUNK;
  switch (t.flags & (GRAD_IN_F32 | GRAD_OUT_F32)) {
    case 0: clip_chunk<false, false>(t, base, c); break;
    case GRAD_IN_F32: clip_chunk<true, false>(t, base, c); break;
    case GRAD_OUT_F32: clip_chunk<false, true>(t, base, c); break;
    default: clip_chunk<true, true>(t, base, c);
  }
}

}  // namespace

hipError_t launch_grad_norm(const GradArgs& a, hipStream_t s) {
  const int cus = device_cu_count();
  if (cus <= 0) return hipErrorInvalidDevice;
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
