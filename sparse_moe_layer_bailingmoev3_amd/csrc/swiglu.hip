// SwiGLU with an optional clamp and routing weight, forward and backward, over stored gate and up
// products (the activation between the grouped products when a layer is trained).
//
//   s = clamp(silu(g) u, +-L);   h = w s
//   ds = w dh;  dg = 1[|silu(g) u| <= L] ds u silu'(g);  du = 1[..] ds silu(g);  dw = sum dh s
//
// The routing weight scales h, so the down product already carries it: the combine then only
// sums, and dw is a sum over the intermediate size instead of the hidden size.  Row i of the
// weights is matrix row pos[i] (the dispatch's inv_perm, flattened), so w and dw stay in [T,K]
// order and no permuted copy of them is made.
//
// Pure streaming: 6 (forward) or 10 (backward) bytes per value.  LPR lanes share a row, each
// taking 8 consecutive values (16 bytes) at a time, so a row's reads are contiguous.  65,536 rows
// of 768 on one MI355X: 63 us forward, 105 us backward, both 4.8 TB/s, the rate of a copy; 776
// rows of 136: 7.8-8.5 us a call, the host's cost of a call (the kernel takes 3.6).
#include "moe_common.h"
#include "moe_internal.h"

namespace moe {

namespace {

__device__ __forceinline__ float lo_f32(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float hi_f32(uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); }

// Whether |a| <= L for a = silu(g) u computed in fp32.  Next to the border the fp32 product does
// not decide it: there it is computed again in 64 bits (g and u are exact).
__device__ __forceinline__ bool inside(float a, float g, float u, float L) {
  const float m = fabsf(a);
  if (fabsf(m - L) <= 1e-5f * L) {
    const double gd = g;
    return fabs(gd / (1.0 + exp(-gd)) * (double)u) <= (double)L;
  }
  return !(m > L);  // NaN passes
}

template <int LPR, bool BWD>
__global__ __launch_bounds__(256) void swiglu_kernel(SwigluArgs a) {
  const int sub = threadIdx.x % LPR;
  const int chunks = a.cols / 8;
  constexpr int ROWS = 256 / LPR;
  for (int64_t i = (int64_t)blockIdx.x * ROWS + threadIdx.x / LPR; i < a.n; i += (int64_t)gridDim.x * ROWS) {
    const int64_t row = a.pos ? a.pos[i] : i;
    if ((uint64_t)row >= (uint64_t)a.mat_rows) {  // a slot that was dispatched nowhere
      if (BWD && a.drow_w && sub == 0) a.drow_w[i] = 0.f;
      continue;
    }
    const float w = a.row_w ? a.row_w[i] : 1.f;
    const float L = a.limit;
    float dw = 0.f;
    for (int c = sub; c < chunks; c += LPR) {
      const u32x4 gv = *(const u32x4*)(a.gate + row * a.ld + c * 8);
      const u32x4 uv = *(const u32x4*)(a.up + row * a.ld + c * 8);
      u32x4 dv{};
      if (BWD) dv = *(const u32x4*)(a.dh + row * a.ldh + c * 8);
      u32x4 o0, o1;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float r0[2], r1[2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const float g = t ? hi_f32(gv[j]) : lo_f32(gv[j]), u = t ? hi_f32(uv[j]) : lo_f32(uv[j]);
          // sigmoid of g and of -g from e = exp(-|g|), squared up from its root so that it reaches
          // down through fp32's subnormal range and never overflows
          const float root = __expf(-0.5f * fabsf(g)), e = root * root, top = __builtin_amdgcn_rcpf(1.f + e);
          const float sig = g >= 0.f ? top : e * top, rest = g >= 0.f ? e * top : top;
          const float silu = g * sig;
          float s = silu * u;
          bool free = true;
          if (L > 0.f) {
            free = inside(s, g, u, L);
            if (!free) s = s > 0.f ? L : -L;
          }
          if (!BWD) {
            r0[t] = w * s;
          } else {
            const float dh = t ? hi_f32(dv[j]) : lo_f32(dv[j]);
            dw += dh * s;
            const float da = free ? w * dh : 0.f;
            r0[t] = da * u * (sig * (1.f + g * rest));
            r1[t] = da * silu;
          }
        }
        o0[j] = f32x2_to_bf16x2(r0[0], r0[1]);
        if (BWD) o1[j] = f32x2_to_bf16x2(r1[0], r1[1]);
      }
      if (!BWD) {
        *(u32x4*)(a.h + row * a.ldh + c * 8) = o0;
      } else {
        *(u32x4*)(a.dgate + row * a.ldd + c * 8) = o0;
        *(u32x4*)(a.dup + row * a.ldd + c * 8) = o1;
      }
    }
    if (BWD && a.drow_w) {  // fixed order: the lanes' partial sums in a tree
#pragma unroll
      for (int d = LPR / 2; d; d >>= 1) dw += __shfl_xor(dw, d, 64);
      if (sub == 0) a.drow_w[i] = dw;
    }
  }
}

template <int LPR, bool BWD>
hipError_t run(const SwigluArgs& a, hipStream_t s) {
  constexpr int ROWS = 256 / LPR;
  const int64_t grid = std::min<int64_t>((a.n + ROWS - 1) / ROWS, (int64_t)1 << 20);
  hipLaunchKernelGGL((swiglu_kernel<LPR, BWD>), dim3((unsigned)grid), dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace

// Lanes per row: the width of 64, 32 or 16 that leaves the fewest idle (768 columns are 96 chunks:
// three rounds of 32 lanes, where 64 would idle a quarter of the time).
hipError_t launch_swiglu(const SwigluArgs& a, bool backward, hipStream_t s) {
  const int chunks = a.cols / 8;
  auto lanes = [&](int l) { return (chunks + l - 1) / l * l; };
  if (lanes(64) <= lanes(32) && lanes(64) <= lanes(16)) return backward ? run<64, true>(a, s) : run<64, false>(a, s);
  if (lanes(32) <= lanes(16)) return backward ? run<32, true>(a, s) : run<32, false>(a, s);
  return backward ? run<16, true>(a, s) : run<16, false>(a, s);
}

}  // namespace moe
