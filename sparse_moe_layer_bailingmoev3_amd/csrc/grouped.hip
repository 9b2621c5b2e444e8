// Matrix products grouped by expert with ragged sizes: forward, input gradient, weight gradient.
//
//   forward   y[p,n]    = sum_k x[m(p),k] W_g[n,k]
//   dgrad     dx[p,k]   = sum_n dy[m(p),n] W_g[n,k]  (+ sum_n dy2[m(p),n] W2_g[n,k])
//   wgrad     dW_g[n,k] = sum_{p in g} dy[md(p),n] x[mx(p),k]
//
// for the positions offsets[g] <= p < offsets[g+1] of group g (bf16 operands, fp32 accumulation).
// One engine: an output tile of BR rows by BC contiguous columns is the sum over reduction steps
// of 64, each step one X tile (feeding the rows) and one Y tile (feeding the columns) that direct
// global->LDS loads bring into a ring of NST stages.  The operands differ in which way their
// reduction index runs in memory:
//   * along a row (forward's x and W, dgrad's dy): LDS rows of 64 values, 16-byte fragments read
//     as they lie;
//   * across rows (dgrad's W, both operands of wgrad): LDS keeps the rows as they come and the
//     fragments are read through gfx950's transposing LDS load (each 16 lanes turn a 4 x 16 block
//     of 16-bit values), so no operand is ever transposed in memory.
// Every stage slot is XOR-swizzled by the row (on the global side: the direct load writes LDS in
// lane order, so each lane picks the 16 bytes that belong in its slot), which spreads the rows of
// one fragment read over all LDS banks.
//
// Masking is done by address: a lane whose row or column does not exist (ragged ends, rows outside
// the matrix, sizes that fill no tile) loads 16 zero bytes from a constant, so no masked value is
// ever read and an infinity or NaN outside the group cannot reach a sum.
//
// The workgroups are persistent and need no list from another kernel: each builds the prefix of
// row tiles over the groups in LDS from `offsets`, and XCD x's workgroups walk the contiguous x-th
// eighth of the tiles together, so tiles that share operand rows or weights run side by side in
// one L2.
#include <atomic>

#include "moe_common.h"
#include "moe_internal.h"

namespace moe {

namespace {

constexpr int OP_FWD = 0, OP_DGRAD = 1, OP_WGRAD = 2;
constexpr int G_KS = 64;                 // reduction values per step
constexpr int G_MAX_GROUPS = 1025;       // 1024 routed experts and a shared one

__device__ __align__(16) const uint32_t grouped_zeros[4] = {0, 0, 0, 0};

// 16 bytes per lane, global -> LDS: lane l writes lds_off + 16*l (an LDS byte offset, wave-uniform).
// Written as an instruction because the compiler, which cannot tell the stages of the ring apart,
// waits for every outstanding direct load before the next LDS read; the kernel's own counted
// waits are what keeps the loads of later stages in flight.  It has no register result; m0, which
// the compiler reserves, is used by nothing else in this file.
__device__ __forceinline__ void dma16(const void* g, uint32_t lds_off) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(lds_off), "v"(g) : "memory");
}
__device__ __forceinline__ uint32_t lds_offset(const void* p) {
  return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void*)p;
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

// 16-byte chunk swizzles of an LDS row: rows of 64 reduction values (8 chunks), and rows of W
// output values whose 32-byte blocks are read by the transposing load: one read touches rows
// 8q..8q+3 (or 8q+4..8q+7) of lane groups q, told apart by bits 0, 1 and 3 of the row.
__device__ __forceinline__ int swz_k(int row) { return (row >> 1) & 7; }
template <int W>
__device__ __forceinline__ int swz_tr(int row) {
  if constexpr (W >= 128) return ((row & 3) | ((row >> 1) & 4)) << 1;
  if constexpr (W == 64) return (((row >> 1) & 1) | ((row >> 2) & 2)) << 1;  // 128-byte rows: bit 0 is the half
  return (((row >> 3) & 1)) << 1;                                            // 64-byte rows
}

template <int OP, int BR, int BC, int WR, int WC, int NST, bool F32>
__global__ __launch_bounds__(WR* WC * 64, 2) void grouped_kernel(GroupedArgs a) {
  constexpr bool XT = OP == OP_WGRAD, YT = OP != OP_FWD;  // operands read through the transposing load
  constexpr int NW = WR * WC;
  constexpr int X_BYTES = BR * G_KS * 2, Y_BYTES = BC * G_KS * 2, ST_BYTES = X_BYTES + Y_BYTES;
  constexpr int XN = X_BYTES / (NW * 1024), YN = Y_BYTES / (NW * 1024);  // loads per wave and step
  static_assert(XN * NW * 1024 == X_BYTES && YN * NW * 1024 == Y_BYTES, "a stage must split evenly over the waves");
  static_assert(OP != OP_WGRAD || BR == BC, "both operands of wgrad share their row indices");
  constexpr int NLOAD = XN + YN;  // (wgrad's row index loads, in between, only make the waits stricter)
  constexpr int D = NST - 1;  // steps in flight
  constexpr int RJ = BR / WR / 16, CJ = BC / WC / 16;
  static_assert(RJ * WR * 16 == BR && CJ * WC * 16 == BC, "wave tiles of 16");
  // lanes per LDS row and rows per load of a transposed operand
  constexpr int XL = BR / 8, YL = BC / 8, XR = 64 / XL, YR = 64 / YL;

  __shared__ __align__(16) uint8_t lds[NST * ST_BYTES];
  __shared__ int32_t prefix[OP == OP_WGRAD ? 1 : G_MAX_GROUPS + 1];

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, q = lane >> 4;
  const int wr = wave / WC, wc = wave % WC;
  const int G = a.groups;
  const int Rdim = OP == OP_WGRAD ? a.N : 0;               // wgrad's row extent
  const int Cdim = OP == OP_FWD ? a.N : a.K;               // contiguous output extent
  const int Red = OP == OP_FWD ? a.K : a.N;                // reduction extent (forward, dgrad)
  const int nct = (Cdim + BC - 1) / BC;
  const int nrt = OP == OP_WGRAD ? (Rdim + BR - 1) / BR : 0;

  // positions of group g, clamped so that no offset leads outside the caller's rows
  auto begin_of = [&](int g) { return min(max(a.offsets[g], 0), a.rows); };
  auto count_of = [&](int g) { const int b = begin_of(g); return max(min(a.offsets[g + 1], a.rows) - b, 0); };

  // ---- the prefix of row tiles (forward, dgrad): wave 0 scans 64 groups at a time
  if constexpr (OP != OP_WGRAD) {
    if (wave == 0) {
      int run = 0;
      for (int g0 = 0; g0 < G; g0 += 64) {
        const int g = g0 + lane;
        int v = g < G ? (count_of(g) + BR - 1) / BR : 0;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
          const int t = __shfl_up(v, d, 64);
          if (lane >= d) v += t;
        }
        if (g < G) prefix[g + 1] = run + v;
        run += __shfl(v, 63, 64);
      }
      if (lane == 0) prefix[0] = 0;
    }
    __syncthreads();
  }
  const int ntile = OP == OP_WGRAD ? G * nrt : prefix[G];

  // ---- LDS read addresses, constant per lane
  // row-major operand: row j*16 + r16, chunk (4u + q); transposed: block cb of 16 columns
  int xa[XT ? RJ : 2], ya[YT ? CJ : 2];
  if constexpr (XT) {
    const int row = 8 * q + (r16 >> 2);
#pragma unroll
    for (int j = 0; j < RJ; ++j)
      xa[j] = row * BR * 2 + ((((wr * RJ + j) * 2) ^ swz_tr<BR>(row)) << 4) + (r16 & 3) * 8;
  } else {
#pragma unroll
    for (int u = 0; u < 2; ++u) xa[u] = (wr * RJ * 16 + r16) * 128 + (((4 * u + q) ^ swz_k(r16)) << 4);
  }
  if constexpr (YT) {
    const int row = 8 * q + (r16 >> 2);
#pragma unroll
    for (int j = 0; j < CJ; ++j)
      ya[j] = X_BYTES + row * BC * 2 + ((((wc * CJ + j) * 2) ^ swz_tr<BC>(row)) << 4) + (r16 & 3) * 8;
  } else {
#pragma unroll
    for (int u = 0; u < 2; ++u) ya[u] = X_BYTES + (wc * CJ * 16 + r16) * 128 + (((4 * u + q) ^ swz_k(r16)) << 4);
  }

  const int64_t total = (int64_t)ntile * nct;
  const int64_t per = (total + 7) >> 3;
  const int64_t first = (int64_t)(blockIdx.x & 7) * per;
  const int64_t last = min(first + per, total);
  const int slots = gridDim.x >> 3;
  int e = 0;  // group of the current tile (tiles of a workgroup only grow)

  for (int64_t item = first + (blockIdx.x >> 3); item < last; item += slots) {
    const int tile = (int)(item / nct), ct = (int)(item - (int64_t)tile * nct);
    int r0;  // first row of the tile: position (forward, dgrad) or weight row (wgrad)
    if constexpr (OP == OP_WGRAD) {
      e = tile / nrt;
      r0 = (tile - e * nrt) * BR;
    } else {
      while (prefix[e + 1] <= tile) ++e;
      r0 = (tile - prefix[e]) * BR;
    }
    const int p0 = begin_of(e), cnt = count_of(e);
    const int c0 = ct * BC;
    const int nred = OP == OP_WGRAD ? cnt : Red;
    const int steps1 = (nred + G_KS - 1) / G_KS;
    const int nsteps = (OP == OP_DGRAD && a.w1) ? 2 * steps1 : steps1;

    // ---- load sources
    const char* xs[XN];
    const char* ys[YN];
    int xinc[XN];
    int64_t yinc[YN];
    const char* const zero = (const char*)grouped_zeros;
    auto set_x = [&](const RowsArg& m) {  // row-major operand of the rows
      if constexpr (!XT) {
#pragma unroll
        for (int i = 0; i < XN; ++i) {
          const int row = (wave * XN + i) * 8 + (lane >> 3);
          int src = -1;
          if (r0 + row < cnt) src = m.map ? m.map[p0 + r0 + row] : p0 + r0 + row;
          const bool ok = (unsigned)src < (unsigned)m.rows;
          const int ch = (lane & 7) ^ swz_k(row);
          xs[i] = ok ? (const char*)m.data + ((int64_t)src * m.ld + ch * 8) * 2 : zero;
          xinc[i] = ok ? G_KS * 2 : 0;
        }
      }
    };
    auto set_y = [&](const uint16_t* w) {  // the group's weights
      const char* wb = (const char*)(w + (int64_t)e * a.N * a.K);
      if constexpr (OP == OP_FWD) {
#pragma unroll
        for (int i = 0; i < YN; ++i) {
          const int row = (wave * YN + i) * 8 + (lane >> 3);
          const bool ok = c0 + row < a.N;
          ys[i] = ok ? wb + ((int64_t)(c0 + row) * a.K + ((lane & 7) ^ swz_k(row)) * 8) * 2 : zero;
          yinc[i] = ok ? G_KS * 2 : 0;
        }
      } else if constexpr (OP == OP_DGRAD) {
#pragma unroll
        for (int i = 0; i < YN; ++i) {
          const int row = (wave * YN + i) * YR + lane / YL;
          const int col = c0 + ((lane % YL) ^ swz_tr<BC>(row)) * 8;
          const bool ok = col < a.K;
          ys[i] = ok ? wb + ((int64_t)row * a.K + col) * 2 : zero;
          yinc[i] = ok ? (int64_t)G_KS * a.K * 2 : 0;
        }
      }
    };
    // wgrad: the step's row indices, one per lane (lane l: row wave*XN*XR + l mod (XN*XR)), loaded
    // one step ahead; a row counts only if it exists in both matrices
    int idx_d = -1, idx_x = -1, cur_d = -1, cur_x = -1;
    auto load_idx = [&](int s) {
      if constexpr (OP == OP_WGRAD) {
        const int row = s * G_KS + wave * (XN * XR) + (lane & (XN * XR - 1));
        const int p = p0 + min(row, cnt - 1);
        const int md = (a.x0.map ? a.x0.map : a.offsets)[a.x0.map ? p : 0];
        const int mx = (a.x1.map ? a.x1.map : a.offsets)[a.x1.map ? p : 0];
        idx_d = a.x0.map ? md : p;
        idx_x = a.x1.map ? mx : p;
        if (row >= cnt) idx_d = -1;
      }
    };
    auto take_idx = [&]() {
      const bool ok = (unsigned)idx_d < (unsigned)a.x0.rows && (unsigned)idx_x < (unsigned)a.x1.rows;
      cur_d = ok ? idx_d : -1;
      cur_x = ok ? idx_x : -1;
    };

    // loads of step s into its stage (s counts through the item; a second operand pair follows the first)
    auto issue = [&](int s) {
      const uint32_t st = __builtin_amdgcn_readfirstlane(lds_offset(lds) + (s % NST) * ST_BYTES);
      if constexpr (OP == OP_WGRAD) {
#pragma unroll
        for (int i = 0; i < XN; ++i) {
          const int row = (wave * XN + i) * XR + lane / XL;
          const int ch = (lane % XL) ^ swz_tr<BR>(row);
          const int d = __shfl(cur_d, i * XR + lane / XL, 64), x = __shfl(cur_x, i * XR + lane / XL, 64);
          const int cn = r0 + ch * 8, ck = c0 + ch * 8;
          const char* pd = d >= 0 && cn < a.N ? (const char*)a.x0.data + ((int64_t)d * a.x0.ld + cn) * 2 : zero;
          const char* px = x >= 0 && ck < a.K ? (const char*)a.x1.data + ((int64_t)x * a.x1.ld + ck) * 2 : zero;
          dma16(pd, st + (wave * XN + i) * 1024);
          dma16(px, st + X_BYTES + (wave * XN + i) * 1024);
        }
      } else {
        if (OP == OP_DGRAD && s == steps1) {
          set_x(a.x1);
          set_y(a.w1);
        }
        const int k0 = (s >= steps1 ? s - steps1 : s) * G_KS;
        const bool tail = k0 + G_KS > nred;
#pragma unroll
        for (int i = 0; i < XN; ++i) {
          const char* p = xs[i];
          if (tail) {
            const int row = (wave * XN + i) * 8 + (lane >> 3);
            if (k0 + ((lane & 7) ^ swz_k(row)) * 8 >= nred) p = zero;
          }
          dma16(p, st + (wave * XN + i) * 1024);
          xs[i] += xinc[i];
        }
#pragma unroll
        for (int i = 0; i < YN; ++i) {
          const char* p = ys[i];
          if (tail) {
            if constexpr (OP == OP_FWD) {
              const int row = (wave * YN + i) * 8 + (lane >> 3);
              if (k0 + ((lane & 7) ^ swz_k(row)) * 8 >= nred) p = zero;
            } else {
              const int row = (wave * YN + i) * YR + lane / YL;
              if (k0 + row >= nred) p = zero;
            }
          }
          dma16(p, st + X_BYTES + (wave * YN + i) * 1024);
          ys[i] += yinc[i];
        }
      }
    };

    floatx4 acc[CJ][RJ];
#pragma unroll
    for (int c = 0; c < CJ; ++c)
#pragma unroll
      for (int r = 0; r < RJ; ++r) acc[c][r] = floatx4{0.f, 0.f, 0.f, 0.f};

    auto compute = [&](int s) {
      const uint8_t* st = lds + (s % NST) * ST_BYTES;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        u32x4 xf[RJ], yf[CJ];
#pragma unroll
        for (int j = 0; j < RJ; ++j) {
          if constexpr (XT) {
            const u32x2 lo = lds_read_tr(st + xa[j] + u * 32 * BR * 2), hi = lds_read_tr(st + xa[j] + (u * 32 + 4) * BR * 2);
            xf[j] = u32x4{lo[0], lo[1], hi[0], hi[1]};
          } else {
            xf[j] = *(const u32x4*)(st + xa[u] + j * 16 * 128);
          }
        }
#pragma unroll
        for (int j = 0; j < CJ; ++j) {
          if constexpr (YT) {
            const u32x2 lo = lds_read_tr(st + ya[j] + u * 32 * BC * 2), hi = lds_read_tr(st + ya[j] + (u * 32 + 4) * BC * 2);
            yf[j] = u32x4{lo[0], lo[1], hi[0], hi[1]};
          } else {
            yf[j] = *(const u32x4*)(st + ya[u] + j * 16 * 128);
          }
        }
#pragma unroll
        for (int c = 0; c < CJ; ++c)
#pragma unroll
          for (int r = 0; r < RJ; ++r) acc[c][r] = mfma16(yf[c], xf[r], acc[c][r]);
      }
    };

    // ---- prologue: every wave has left the previous item's stages
    lds_barrier();
    if constexpr (OP != OP_WGRAD) {
      set_x(a.x0);
      set_y(a.w0);
    }
    if (nsteps > 0) {
      load_idx(0);
#pragma unroll
      for (int s = 0; s < D; ++s) {
        if (s < nsteps) {
          take_idx();
          load_idx(s + 1);
          issue(s);
        }
      }
    }
    // ---- steps: wait until only the loads of the later steps are outstanding, meet the other
    // waves (their loads of this stage are in, their reads of the stage to be refilled are done),
    // refill, multiply
    const bool live = OP == OP_WGRAD ? r0 + wr * RJ * 16 < a.N : r0 + wr * RJ * 16 < cnt;
    for (int s = 0; s < nsteps; ++s) {
      const int ahead = min(nsteps - 1 - s, D - 1);
      if (ahead >= 2) wait_vmcnt<2 * NLOAD>();
      else if (ahead == 1) wait_vmcnt<NLOAD>();
      else wait_vmcnt<0>();
      lds_barrier();
      if (s + D < nsteps) {
        take_idx();
        load_idx(s + D + 1);
        issue(s + D);
      }
      if (live) compute(s);
    }

    // ---- epilogue: lane holds columns c..c+3 of one output row
#pragma unroll
    for (int r = 0; r < RJ; ++r) {
      const int row = r0 + (wr * RJ + r) * 16 + r16;
      const bool rok = OP == OP_WGRAD ? row < a.N : row < cnt;
      if (!rok) continue;
      const int64_t ob = OP == OP_WGRAD ? ((int64_t)e * a.N + row) * a.K : (int64_t)(p0 + row) * a.ldo;
#pragma unroll
      for (int c = 0; c < CJ; ++c) {
        const int col = c0 + (wc * CJ + c) * 16 + 4 * q;
        if (col >= Cdim) continue;
        if constexpr (F32) {
          floatx4* o = (floatx4*)((float*)a.out + ob + col);
          *o = a.accumulate ? *o + acc[c][r] : acc[c][r];
        } else {
          *(u32x2*)((uint16_t*)a.out + ob + col) =
              u32x2{f32x2_to_bf16x2(acc[c][r][0], acc[c][r][1]), f32x2_to_bf16x2(acc[c][r][2], acc[c][r][3])};
        }
      }
    }
  }
  wait_vmcnt<0>();  // no direct-to-LDS load may outlive the workgroup
}

template <int OP, int BR, int BC, int WR, int WC, int NST>
hipError_t run_grouped(const GroupedArgs& a, int64_t max_items, int wg_per_cu, hipStream_t s) {
  const int cus = device_cu_count();
  if (cus <= 0) return hipErrorInvalidDevice;
  const int64_t grid = std::min<int64_t>((int64_t)(cus / 8 * 8) * wg_per_cu, (max_items + 7) / 8 * 8);
  if (grid <= 0) return hipSuccess;
  if (a.out_f32)
    hipLaunchKernelGGL((grouped_kernel<OP, BR, BC, WR, WC, NST, true>), dim3((unsigned)grid), dim3(WR * WC * 64), 0, s, a);
  else
    hipLaunchKernelGGL((grouped_kernel<OP, BR, BC, WR, WC, NST, false>), dim3((unsigned)grid), dim3(WR * WC * 64), 0, s, a);
  return hipGetLastError();
}

}  // namespace

int device_cu_count() {
  static std::atomic<int> cache[64];
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0) return 0;
  if (dev < 64 && cache[dev].load() > 0) return cache[dev].load();
  int n = 0;
  if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess) return 0;
  if (dev < 64) cache[dev].store(n);
  return n;
}

// Tiles: no group count is known on the host, only the number of positions and groups.
hipError_t launch_grouped_rows(const GroupedArgs& a, bool dgrad, hipStream_t s) {
  const int64_t nct = ((dgrad ? a.K : a.N) + 127) / 128;
  // at most one partial tile per group that holds a position
  auto items = [&](int br) { return (a.rows / br + std::min<int64_t>(a.groups, a.rows)) * nct; };
  if (a.rows <= (int64_t)24 * a.groups)
    return dgrad ? run_grouped<OP_DGRAD, 32, 128, 1, 4, 3>(a, items(32), 2, s)
                 : run_grouped<OP_FWD, 32, 128, 1, 4, 3>(a, items(32), 2, s);
  return dgrad ? run_grouped<OP_DGRAD, 128, 128, 2, 2, 2>(a, items(128), 2, s)
               : run_grouped<OP_FWD, 128, 128, 2, 2, 2>(a, items(128), 2, s);
}

hipError_t launch_grouped_wgrad(const GroupedArgs& a, hipStream_t s) {
  const int64_t items = (int64_t)a.groups * ((a.N + 127) / 128) * ((a.K + 127) / 128);
  return run_grouped<OP_WGRAD, 128, 128, 2, 2, 2>(a, items, 2, s);
}

}  // namespace moe
