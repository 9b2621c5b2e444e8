// The two products of the router's backward pass, from the gradient dl [T,E] of the logits:
//
//   d router_w[e,h] = sum_t dl[t,e] x[t,h]        dx[t,h] = sum_e dl[t,e] router_w[e,h]
//
// A 64 x 64 tile a workgroup, 4 x 4 values a thread, fp32.
#include "moe_common.h"
#include "moe_internal.h"

namespace moe {

namespace {

template <bool DW, bool F32>
__global__ __launch_bounds__(256) void router_product_kernel(RouterGradArgs a) {
  constexpr int KS = 16;
  __shared__ float A[KS][68], B[KS][68];
  const int tr = threadIdx.x / 16, tc = threadIdx.x % 16;
  const int64_t r0 = (int64_t)blockIdx.y * 64;
  const int c0 = blockIdx.x * 64;
  const int64_t rows = DW ? a.E : a.T, red = DW ? a.T : a.E;
  float acc[4][4] = {};
  for (int64_t k0 = 0; k0 < red; k0 += KS) {
    for (int i = threadIdx.x; i < KS * 64; i += 256) {
      if constexpr (DW) {
        const int k = i / 64, c = i % 64;
        const int64_t t = k0 + k;
        A[k][c] = t < red && r0 + c < rows ? a.dl[t * a.E + r0 + c] : 0.f;
        B[k][c] = t < red ? bf16_bits_to_f32(a.x[t * a.H + c0 + c]) : 0.f;
      } else {
        const int64_t t = r0 + i / KS;
        A[i % KS][i / KS] = t < rows ? a.dl[t * a.E + k0 + i % KS] : 0.f;
        B[i / 64][i % 64] = a.w[(k0 + i / 64) * a.H + c0 + i % 64];
      }
    }
    __syncthreads();
    for (int k = 0; k < KS; ++k)
      for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) acc[i][j] = __builtin_fmaf(A[k][tr * 4 + i], B[k][tc * 4 + j], acc[i][j]);
    __syncthreads();
  }
  for (int i = 0; i < 4; ++i) {
    const int64_t r = r0 + tr * 4 + i;
    if (r >= rows) continue;
    for (int j = 0; j < 4; ++j) {
      const int64_t at = r * a.H + c0 + tc * 4 + j;
      if constexpr (DW) a.dw[at] = a.acc_w ? a.dw[at] + acc[i][j] : acc[i][j];
      else if constexpr (F32) ((float*)a.dx)[at] = a.acc_x ? ((float*)a.dx)[at] + acc[i][j] : acc[i][j];
      else ((uint16_t*)a.dx)[at] = (uint16_t)f32x2_to_bf16x2(acc[i][j], 0.f);
    }
  }
}

}  // namespace

hipError_t launch_router_grad(const RouterGradArgs& a, hipStream_t s) {
  if (a.dw) hipLaunchKernelGGL((router_product_kernel<true, true>), dim3(a.H / 64, a.E / 64), dim3(256), 0, s, a);
  if (a.dx && a.T > 0) {
    const dim3 grid(a.H / 64, (unsigned)((a.T + 63) / 64));
    if (a.dx_f32) hipLaunchKernelGGL((router_product_kernel<false, true>), grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((router_product_kernel<false, false>), grid, dim3(256), 0, s, a);
  }
  return hipGetLastError();
}

}  // namespace moe
