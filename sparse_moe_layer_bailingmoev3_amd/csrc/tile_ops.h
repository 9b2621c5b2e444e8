// Device code shared by the tile kernels that stage operands through LDS by direct loads: the loads,
// gfx950's transposing LDS read, counted waits, swizzles, the transposition of result fragments.
#pragma once
#include <utility>

#include "moe_common.h"

namespace moe {

// 16 bytes per lane, global -> LDS: lane l writes lds_off + 16*l (an LDS byte offset, wave-uniform).
// Written as an instruction because the compiler, which cannot tell the stages of the ring apart,
// waits for every outstanding direct load before the next LDS read; the kernel's own counted
// waits are what keeps the loads of later stages in flight.  It has no register result; m0, which
// the compiler reserves, is used by nothing else in the files that include this.
__device__ __forceinline__ void dma16(const void* g, uint32_t lds_off) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(lds_off), "v"(g) : "memory");
}
__device__ __forceinline__ uint32_t lds_offset(const void* p) {
  return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void*)p;
}

// The same through a buffer descriptor of BUF_MAX bytes: an offset past its end gives zeros.
constexpr uint32_t BUF_OUT = 0xFFFFFFF0u;
constexpr int64_t BUF_MAX = 0xFFFFFF00ll;
__device__ __forceinline__ u32x4 buffer_at(uint64_t base) {
  return u32x4{(uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)base),
               (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(base >> 32)), (uint32_t)BUF_MAX, 0x00020000u};
}
__device__ __forceinline__ void dma16(uint32_t off, const u32x4& rsrc, uint32_t lds_off) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(lds_off), "v"(off), "s"(rsrc)
               : "memory");
}

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4* lds_s16x4;

// Transposing LDS read.  The 16 lanes of a group address 4 rows of 16 values (lane i: row i/4,
// values 4*(i%4)..+3); lane i receives column i of that block, rows 0..3.
__device__ __forceinline__ u32x2 lds_read_tr(const uint8_t* p) {
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)p));
}

// (the empty asm keeps the compiler from moving memory accesses across)
__device__ __forceinline__ void lds_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0); vmcnt and expcnt left alone
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

template <int N>
__device__ __forceinline__ void wait_vmcnt() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 0xF) | ((N >> 4) << 14) | (0x7 << 4) | (0xF << 8));
}

// 16-byte chunk swizzle of an LDS row of W values whose 32-byte blocks are read by the transposing
// load: one read touches rows 8q..8q+3 (or 8q+4..8q+7) of lane groups q, told apart by bits 0, 1 and
// 3 of the row.
template <int W>
__device__ __forceinline__ int swz_tr(int row) {
  static_assert(W >= 64, "rows of at least 128 bytes");
  if constexpr (W >= 128) return ((row & 3) | ((row >> 1) & 4)) << 1;
  return (((row >> 1) & 1) | ((row >> 2) & 2)) << 1;  // 128-byte rows: bit 0 is the half
}

// v[j] of lane b of every quad <-> v[b] of lane j
__device__ __forceinline__ void quad_transpose(floatx4 (&v)[4]) {
  const bool b0 = threadIdx.x & 1, b1 = threadIdx.x & 2;
  auto swap = [](float& x, float& y, bool up, auto ctrl) {  // lower lane keeps x, upper keeps y
    const float t = __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(up ? x : y), decltype(ctrl)::value, 0xF, 0xF, true));
    x = up ? t : x;
    y = up ? y : t;
  };
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float w[4] = {v[0][i], v[1][i], v[2][i], v[3][i]};
    swap(w[0], w[1], b0, std::integral_constant<int, 0xB1>{});  // quad_perm 1 0 3 2
    swap(w[2], w[3], b0, std::integral_constant<int, 0xB1>{});
    swap(w[0], w[2], b1, std::integral_constant<int, 0x4E>{});  // quad_perm 2 3 0 1
    swap(w[1], w[3], b1, std::integral_constant<int, 0x4E>{});
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j][i] = w[j];
  }
}

// f(0) .. f(N-1), written out by the front end (a loop over registers that the optimiser unrolls
// too late leaves them in memory)
template <typename F, int... I>
__device__ __forceinline__ void each_impl(F& f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>{}), ...);
}
template <int N, typename F>
__device__ __forceinline__ void each(F f) {
  each_impl(f, std::make_integer_sequence<int, N>{});
}

}  // namespace moe
