// Matrix products grouped by expert with ragged sizes: forward, input gradient, weight gradient.
//
//   forward   y[p,n]    = sum_k x[m(p),k] W_g[n,k]
//   dgrad     dx[p,k]   = sum_n dy[m(p),n] W_g[n,k]  (+ sum_n dy2[m(p),n] W2_g[n,k])
//   wgrad     dW_g[n,k] = sum_{p in g} dy[md(p),n] x[mx(p),k]
//
// for the positions offsets[g] <= p < offsets[g+1] of group g (bf16 operands, fp32 accumulation).
// One engine: an output tile of BR rows by BC contiguous columns is the sum over reduction steps
// of KS values (64; 128 in the 16 x 64 form for few rows), each step one X tile (feeding the rows)
// and one Y tile (feeding the columns) that direct global->LDS loads bring into a ring of NST
// stages.  The operands differ in which way their reduction index runs in memory:
//   * along a row (forward's x and W, dgrad's dy): LDS rows of KS values, 16-byte fragments read
//     as they lie;
//   * across rows (dgrad's W, both operands of wgrad): LDS keeps the rows as they come and the
//     fragments are read through gfx950's transposing LDS load (each 16 lanes turn a 4 x 16 block
//     of 16-bit values), so no operand is ever transposed in memory.
// Every stage slot is XOR-swizzled by the row (on the global side: the direct load writes LDS in
// lane order, so each lane picks the 16 bytes that belong in its slot), which spreads the rows of
// one fragment read over all LDS banks.
//
// Masking is done by address: the direct loads go through buffer descriptors, and a lane whose row
// or column does not exist (ragged ends, rows outside the matrix, sizes that fill no tile) takes
// an offset past the descriptor's end, for which the load writes zeros to LDS.  No masked value is
// ever read, and an infinity or NaN outside the group cannot reach a sum.  Descriptors also keep
// the address arithmetic off the vector units: a lane's offset in the tile stays, and the
// descriptor's base moves from step to step.
//
// The workgroups are persistent and need no list from another kernel: each builds the prefix of
// row tiles over the groups in LDS from `offsets`, and XCD x's workgroups walk the contiguous x-th
// eighth of the tiles together, so tiles that share operand rows or weights run side by side in
// one L2.  The loads run NST-1 steps ahead of the products and on into the next tile, so a tile's
// end does not empty the pipeline.
//
// What bounds it, on one MI355X (a copy moves 4.9 TB/s here, reads alone 6.3, fills 6.9; the bf16
// library product reaches 1.23 PFLOP/s), 512 groups of 768 x 2560 weights, 8 a token:
//   few rows (forward, 64 tokens)          204-212 us, 6.0-6.3 TB/s of weights: the read rate
//   forward down, 8192 tokens, fp32 out    554 us, 5.0 TB/s: the copy rate
//   dgrad down, 8192 tokens                463-470 us, 4.6 TB/s (5.2 as fetched: a token's row comes
//                                          in once for each of its eight positions)
//   wgrad added to fp32, 8192 tokens       1660 us, 4.9 TB/s: the copy rate
//   the same, 64 tokens (324 groups)       1060 us, 4.9 TB/s; 1 token (8 groups): 162 us, in which
//                                          every workgroup steps through 60 tiles, most of them of
//                                          empty groups (read and written: nothing)
// With 1024 rows a group (64 groups) the products bound it: forward 1.02, dgrad 0.87 (0.73 with fp32
// results), wgrad 0.80 PFLOP/s; LDS reads and matrix instructions of a step do not overlap fully (one
// barrier a step), and the 256 x 256 dgrad form with fp32 results spills 6 vector registers (28 bytes
// a lane; it and wgrad's also keep 60-75 scalar values in lanes).  LDS bank conflicts are zero in every
// form.  Measured and not kept: steps of 32 values (dgrad +40 %: the barriers), nontemporal results
// (wgrad +22 %), fragments read a sub-step ahead (no change, or slower by the registers they hold),
// 128 x 128 tiles per wave (78-540 vector registers spilled), a group's row tiles before its column
// tiles (skewed dgrad +6 %), raised wave priority around the products (no change).
#include <atomic>
#include <cmath>

#include "moe_common.h"
#include "moe_internal.h"
#include "tile_ops.h"

namespace moe {

namespace {

constexpr int OP_FWD = 0, OP_DGRAD = 1, OP_WGRAD = 2;
constexpr int G_MAX_GROUPS = 1025;       // 1024 routed experts and a shared one

__device__ __align__(16) const uint32_t grouped_zeros[4] = {0, 0, 0, 0};

// 16-byte chunk swizzle of an LDS row of KS reduction values (of the others: swz_tr)
template <int KS>
__device__ __forceinline__ int swz_k(int row) { return KS == 64 ? (row >> 1) & 7 : row & 15; }

// Loads through the scalar data cache (uniform addresses of data the kernel never writes): they are
// counted by lgkmcnt, so finding the next tile's rows never waits on the loads of the tiles' data.
typedef const __attribute__((address_space(4))) int32_t* sptr;

template <int OP, int KS, int BR, int BC, int WR, int WC, int NST, bool F32>
__global__ __launch_bounds__(WR* WC * 64, (WR * WC == 4 && NST * (BR + BC) * KS * 2 > 72 * 1024) ? 1 : 2) void grouped_kernel(GroupedArgs a) {
  constexpr bool XT = OP == OP_WGRAD, YT = OP != OP_FWD;  // operands read through the transposing load
  constexpr int NW = WR * WC;
  constexpr int X_BYTES = BR * KS * 2, Y_BYTES = BC * KS * 2, ST_BYTES = X_BYTES + Y_BYTES;
  constexpr int XN = X_BYTES / (NW * 1024), YN = Y_BYTES / (NW * 1024);  // loads per wave and step
  static_assert(XN * NW * 1024 == X_BYTES && YN * NW * 1024 == Y_BYTES, "a stage must split evenly over the waves");
  static_assert(OP != OP_WGRAD || BR == BC, "both operands of wgrad share their row indices");
  constexpr int D = NST - 1;  // steps in flight
  constexpr int KB = KS * 2, KC = KS / 8;  // bytes and 16-byte chunks of a row of reduction values
  constexpr int KR = 64 / KC;              // such rows per load
  constexpr int RJ = BR / WR / 16, CJ = BC / WC / 16;
  static_assert(RJ * WR * 16 == BR && CJ * WC * 16 == BC, "wave tiles of 16");
  // lanes per LDS row and rows per load of a transposed operand
  constexpr int XL = BR / 8, YL = BC / 8, XR = 64 / XL, YR = 64 / YL;

  __shared__ __align__(16) uint8_t lds[NST * ST_BYTES];
  __shared__ int32_t prefix[OP == OP_WGRAD ? 1 : G_MAX_GROUPS + 65];  // row tiles before each group
  __shared__ int32_t wave_total[NW];

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, q = lane >> 4;
  const int wr = wave / WC, wc = wave % WC;
  const int G = a.groups;
  const int Cdim = OP == OP_FWD ? a.N : a.K;  // contiguous output extent
  const int Red = OP == OP_FWD ? a.K : a.N;   // reduction extent (forward, dgrad)
  const int nct = (Cdim + BC - 1) / BC;
  const int nrt = OP == OP_WGRAD ? (a.N + BR - 1) / BR : 0;

  // ---- the prefix of row tiles over the groups (forward, dgrad), a group per thread and round
  if constexpr (OP != OP_WGRAD) {
    int run = 0;
    for (int g0 = 0; g0 < G; g0 += NW * 64) {
      const int g = g0 + threadIdx.x;
      int v = 0;
      if (g < G) {
        const int b = min(max(a.offsets[g], 0), a.rows);
        v = (max(min(a.offsets[g + 1], a.rows) - b, 0) + BR - 1) / BR;
      }
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const int t = __shfl_up(v, d, 64);
        if (lane >= d) v += t;
      }
      if (lane == 63) wave_total[wave] = v;
      __syncthreads();
      int before = run;
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        if (w < wave) before += wave_total[w];
        run += wave_total[w];
      }
      if (g < G) prefix[g + 1] = before + v;
      __syncthreads();
    }
    // 64 entries past the last group end the lanes' search
    if (threadIdx.x < 64) prefix[G + 1 + threadIdx.x] = 0x7FFFFFFF;
    if (threadIdx.x == 0) prefix[0] = 0;
    __syncthreads();
  }
  const int ntile = OP == OP_WGRAD ? G * nrt : __builtin_amdgcn_readfirstlane(prefix[G]);

  // ---- LDS read addresses, constant per lane
  // row-major operand: row j*16 + r16, chunk (4u + q); transposed: block cb of 16 columns
  int xa[XT ? RJ : KS / 32], ya[YT ? CJ : KS / 32];
  if constexpr (XT) {
    const int row = 8 * q + (r16 >> 2);
#pragma unroll
    for (int j = 0; j < RJ; ++j)
      xa[j] = row * BR * 2 + ((((wr * RJ + j) * 2) ^ swz_tr<BR>(row)) << 4) + (r16 & 3) * 8;
  } else {
#pragma unroll
    for (int u = 0; u < KS / 32; ++u) xa[u] = (wr * RJ * 16 + r16) * KB + (((4 * u + q) ^ swz_k<KS>(r16)) << 4);
  }
  if constexpr (YT) {
    const int row = 8 * q + (r16 >> 2);
#pragma unroll
    for (int j = 0; j < CJ; ++j)
      ya[j] = X_BYTES + row * BC * 2 + ((((wc * CJ + j) * 2) ^ swz_tr<BC>(row)) << 4) + (r16 & 3) * 8;
  } else {
#pragma unroll
    for (int u = 0; u < KS / 32; ++u) ya[u] = X_BYTES + (wc * CJ * 16 + r16) * KB + (((4 * u + q) ^ swz_k<KS>(r16)) << 4);
  }

  // ---- this workgroup's tiles.  The loads run D steps ahead of the products, across tiles, so
  // the two sides walk the tiles separately.
  const int slots = gridDim.x >> 3;
  const int dtile = slots / nct, dct = slots - dtile * nct;
  struct Walk {
    int64_t left;  // tiles after this one's position in the XCD's range
    int tile, ct;
    int e, p0, cnt, r0, c0, nsteps, steps1;
  };
  const sptr offsets = (sptr)a.offsets;
  auto locate = [&](Walk& w) {
    if constexpr (OP == OP_WGRAD) {
      w.e = w.tile / nrt;
      w.r0 = (w.tile - w.e * nrt) * BR;
    } else {
      // the lanes look at 64 groups at a time
      for (;;) {
        const int n = __popcll(__ballot(prefix[w.e + 1 + lane] <= w.tile));
        w.e += n;
        if (n < 64) break;
      }
      w.e = min(__builtin_amdgcn_readfirstlane(w.e), G - 1);
      w.r0 = (w.tile - __builtin_amdgcn_readfirstlane(prefix[w.e])) * BR;
    }
    w.p0 = min(max(offsets[w.e], 0), a.rows);
    w.cnt = max(min(offsets[w.e + 1], a.rows) - w.p0, 0);
    w.c0 = w.ct * BC;
    // an empty group's gradient is one step of zeros
    w.steps1 = OP == OP_WGRAD ? max((w.cnt + KS - 1) / KS, 1) : (Red + KS - 1) / KS;
    w.nsteps = (OP == OP_DGRAD && a.w1) ? 2 * w.steps1 : w.steps1;
  };
  auto advance = [&](Walk& w) -> bool {
    w.left -= slots;
    if (w.left <= 0) return false;
    w.tile += dtile;
    w.ct += dct;
    if (w.ct >= nct) {
      w.ct -= nct;
      ++w.tile;
    }
    locate(w);
    return true;
  };
  Walk ld;
  {
    const int64_t total = (int64_t)ntile * nct, per = (total + 7) >> 3;
    const int64_t first = (int64_t)(blockIdx.x & 7) * per + (blockIdx.x >> 3);
    ld.left = min((int64_t)(blockIdx.x & 7) * per + per, total) - first;
    if (ld.left <= 0) return;
    ld.tile = (int)(first / nct);
    ld.ct = (int)(first - (int64_t)ld.tile * nct);
    ld.e = 0;
    locate(ld);
  }
  Walk cw = ld;  // the products' side
  int ls = 0;    // next step to load of tile `ld`
  bool more = true;

  // ---- load sources: descriptor bases that move with the steps, offsets that stay for the tile
  uint64_t xb = 0, yb = 0;
  int64_t xstep = 0, ystep = 0;
  uint32_t xo[XN], yo[YN];  // (the rows of a mapped matrix of more than BUF_MAX bytes: row numbers)
  int xn = XN;         // row loads that hold a row of the tile
  int left = 0;        // reduction values from step `ls` on
  const char* const zero = (const char*)grouped_zeros;
  auto wide = [&](const RowsArg& m) { return m.map && (int64_t)m.rows * m.ld * 2 > BUF_MAX; };
  const bool wide0 = wide(a.x0), wide1 = OP == OP_WGRAD && wide(a.x1);
  // the n consecutive rows of a load: row `sub` of positions p.., through the map
  auto mapped = [&](const RowsArg& m, int p, int last, int sub, auto n) {
    int src = 0;
    const sptr map = (sptr)m.map;
    each<decltype(n)::value>([&](auto k) {
      const int t = map[min(p + k, last)];
      src = sub == k ? t : src;
    });
    return src;
  };
  auto set_x = [&](const RowsArg& m) {  // row-major operand of the rows; load i holds rows (i*NW + wave)*KR ..
    if constexpr (!XT) {
      const int n = ld.cnt - ld.r0;
      xn = min((n + NW * KR - 1) / (NW * KR), XN);
      xb = (uint64_t)m.data + (m.map ? 0 : (int64_t)(ld.p0 + ld.r0) * m.ld * 2);
      xstep = KB;
      each<XN>([&](auto i) {
        const int row0 = (i * NW + wave) * KR, row = row0 + lane / KC;
        const int ch = (lane % KC) ^ swz_k<KS>(row);
        uint32_t o = (uint32_t)row * (uint32_t)(m.ld * 2) + ch * 16;
        bool ok = row < n;
        if (m.map) {
          int src = -1;
          if (row0 < n) src = mapped(m, ld.p0 + ld.r0 + row0, ld.p0 + ld.cnt - 1, lane / KC, std::integral_constant<int, KR>{});
          ok = ok && (unsigned)src < (unsigned)m.rows;
          o = wide0 ? (uint32_t)src : (uint32_t)src * (uint32_t)(m.ld * 2) + ch * 16;
        }
        xo[i] = ok ? o : BUF_OUT;
      });
    }
  };
  auto set_y = [&](const uint16_t* w) {  // the group's weights
    yb = (uint64_t)(w + (int64_t)ld.e * a.N * a.K);
    if constexpr (OP == OP_FWD) {
      yb += (int64_t)ld.c0 * a.K * 2;
      ystep = KB;
      each<YN>([&](auto i) {
        const int row = (wave * YN + i) * KR + lane / KC;
        yo[i] = ld.c0 + row < a.N ? (uint32_t)row * (uint32_t)(a.K * 2) + ((lane % KC) ^ swz_k<KS>(row)) * 16 : BUF_OUT;
      });
    } else if constexpr (OP == OP_DGRAD) {
      yb += (int64_t)ld.c0 * 2;
      ystep = (int64_t)KS * a.K * 2;
      each<YN>([&](auto i) {
        const int row = (wave * YN + i) * YR + lane / YL;
        const int col = ((lane % YL) ^ swz_tr<BC>(row)) * 8;
        yo[i] = ld.c0 + col < a.K ? (uint32_t)row * (uint32_t)(a.K * 2) + col * 2 : BUF_OUT;
      });
    }
  };
  auto set_sources = [&]() {
    if constexpr (OP == OP_WGRAD) {
      left = ld.cnt;
      xb = (uint64_t)a.x0.data + ld.r0 * 2 + (a.x0.map ? 0 : (int64_t)ld.p0 * a.x0.ld * 2);
      xstep = a.x0.map ? 0 : KS * a.x0.ld * 2;
      yb = (uint64_t)a.x1.data + ld.c0 * 2 + (a.x1.map ? 0 : (int64_t)ld.p0 * a.x1.ld * 2);
      ystep = a.x1.map ? 0 : KS * a.x1.ld * 2;
      each<XN>([&](auto i) {
        const int row = (wave * XN + i) * XR + lane / XL, ch = (lane % XL) ^ swz_tr<BR>(row);
        xo[i] = ld.r0 + ch * 8 < a.N ? (uint32_t)row * (uint32_t)(a.x0.ld * 2) + ch * 16 : BUF_OUT;
        yo[i] = ld.c0 + ch * 8 < a.K ? (uint32_t)row * (uint32_t)(a.x1.ld * 2) + ch * 16 : BUF_OUT;
      });
    } else {
      left = Red;
      set_x(a.x0);
      set_y(a.w0);
    }
  };

  // wgrad through maps: the rows of the next step's loads, read one step ahead (a step waits for
  // all loads of the one before, these among them)
  int di[XT ? XN : 1], xi[XT ? XN : 1];
  auto load_rows = [&]() {
    if constexpr (OP == OP_WGRAD) {
      static_assert(D == 1, "row indices are one step ahead");
      if (a.x0.map || a.x1.map) {
        each<XN>([&](auto i) {
          const int p = ld.p0 + max(min(ls * KS + (wave * XN + i) * XR + lane / XL, ld.cnt - 1), 0);
          int d = 0, x = 0;
          if (ld.cnt > 0) {
            if (a.x0.map) d = a.x0.map[p];
            if (a.x1.map) x = a.x1.map[p];
          }
          di[i] = d;
          xi[i] = x;
        });
      }
    }
  };

  // loads of step `ls` of tile `ld` into the stage at LDS offset st
  auto issue = [&](uint32_t st) {
    if constexpr (OP == OP_WGRAD) {
      const u32x4 xr = buffer_at(xb), yr = buffer_at(yb);
      const uint32_t xt = st + wave * XN * 1024;
      if (!a.x0.map && !a.x1.map) {
        if (left >= KS) {
          each<XN>([&](auto i) {
            dma16(xo[i], xr, xt + i * 1024);
            dma16(yo[i], yr, xt + X_BYTES + i * 1024);
          });
        } else {
          each<XN>([&](auto i) {
            const bool ok = (wave * XN + i) * XR + lane / XL < left;
            dma16(ok ? xo[i] : BUF_OUT, xr, xt + i * 1024);
            dma16(ok ? yo[i] : BUF_OUT, yr, xt + X_BYTES + i * 1024);
          });
        }
      } else {
        // a row counts only if it exists in both matrices
        each<XN>([&](auto i) {
          const int row = (wave * XN + i) * XR + lane / XL, ch = (lane % XL) ^ swz_tr<BR>(row);
          const int d = di[i], x = xi[i];
          const bool ok = row < left && (unsigned)d < (unsigned)a.x0.rows && (unsigned)x < (unsigned)a.x1.rows;
          const bool okd = ok && xo[i] != BUF_OUT, okx = ok && yo[i] != BUF_OUT;
          const uint32_t od = a.x0.map ? (uint32_t)d * (uint32_t)(a.x0.ld * 2) + ch * 16 : xo[i];
          const uint32_t ox = a.x1.map ? (uint32_t)x * (uint32_t)(a.x1.ld * 2) + ch * 16 : yo[i];
          if (wide0) dma16(okd ? (const char*)a.x0.data + ((int64_t)d * a.x0.ld + ld.r0 + ch * 8) * 2 : zero, xt + i * 1024);
          else dma16(okd ? od : BUF_OUT, xr, xt + i * 1024);
          if (wide1) dma16(okx ? (const char*)a.x1.data + ((int64_t)x * a.x1.ld + ld.c0 + ch * 8) * 2 : zero, xt + X_BYTES + i * 1024);
          else dma16(okx ? ox : BUF_OUT, yr, xt + X_BYTES + i * 1024);
        });
      }
    } else {
      if (OP == OP_DGRAD && ls == ld.steps1) {  // the second operand pair
        left = Red;
        set_x(a.x1);
        set_y(a.w1);
      }
      const u32x4 xr = buffer_at(xb), yr = buffer_at(yb);
      const uint32_t xt = st + wave * 1024, yt = st + X_BYTES + wave * YN * 1024;
      if (!wide0 && left >= KS) {
        each<XN>([&](auto i) {
          if (XN == 1 || i < xn) dma16(xo[i], xr, xt + i * NW * 1024);
        });
        each<YN>([&](auto i) { dma16(yo[i], yr, yt + i * 1024); });
      } else {
        // the last step of a reduction that is no multiple of KS: what follows in memory is the next
        // row, or the next group
        each<XN>([&](auto i) {
          if (XN == 1 || i < xn) {
            const int row = (i * NW + wave) * KR + lane / KC;
            const int k = ((lane % KC) ^ swz_k<KS>(row)) * 8;
            const bool past = k >= left;
            if (wide0) {  // a mapped matrix: row number to 64-bit address
              const RowsArg& m = OP == OP_DGRAD && ls >= ld.steps1 ? a.x1 : a.x0;
              const char* p = (const char*)m.data + ((int64_t)xo[i] * m.ld + (Red - left) + k) * 2;
              dma16(past || xo[i] == BUF_OUT ? zero : p, xt + i * NW * 1024);
            } else dma16(past ? BUF_OUT : xo[i], xr, xt + i * NW * 1024);
          }
        });
        each<YN>([&](auto i) {
          const int row = OP == OP_FWD ? (wave * YN + i) * KR + lane / KC : (wave * YN + i) * YR + lane / YL;
          const bool past = (OP == OP_FWD ? ((lane % KC) ^ swz_k<KS>(row)) * 8 : row) >= left;
          dma16(past ? BUF_OUT : yo[i], yr, yt + i * 1024);
        });
      }
    }
    left -= KS;
    xb += xstep;
    yb += ystep;
  };
  const uint32_t lds0 = lds_offset(lds);
  uint32_t lst = lds0;  // stage of the next step to load
  int flying = 0;       // steps loaded or in flight and not yet computed
  int n_last = 0;       // loads of the last of them
  auto issue_next = [&]() {  // `ld`, `ls` and the sources stand at the step to load
    if (!more) return;
    issue(__builtin_amdgcn_readfirstlane(lst));
    lst = lst == lds0 + (NST - 1) * ST_BYTES ? lds0 : lst + ST_BYTES;
    n_last = xn;
    ++flying;
    if (++ls == ld.nsteps) {
      more = advance(ld);
      ls = 0;
      if (more) set_sources();
    }
    if (more) load_rows();
  };

  floatx4 acc[CJ][RJ];
  auto clear = [&]() {
#pragma unroll
    for (int c = 0; c < CJ; ++c)
#pragma unroll
      for (int r = 0; r < RJ; ++r) acc[c][r] = floatx4{0.f, 0.f, 0.f, 0.f};
  };
  clear();

  auto compute = [&](const uint8_t* st) {
#pragma unroll
    for (int u = 0; u < KS / 32; ++u) {
      u32x4 xf[RJ], yf[CJ];
#pragma unroll
      for (int j = 0; j < RJ; ++j) {
        if constexpr (XT) {
          const u32x2 lo = lds_read_tr(st + xa[j] + u * 32 * BR * 2), hi = lds_read_tr(st + xa[j] + (u * 32 + 4) * BR * 2);
          xf[j] = u32x4{lo[0], lo[1], hi[0], hi[1]};
        } else {
          xf[j] = *(const u32x4*)(st + xa[u] + j * 16 * KB);
        }
      }
#pragma unroll
      for (int j = 0; j < CJ; ++j) {
        if constexpr (YT) {
          const u32x2 lo = lds_read_tr(st + ya[j] + u * 32 * BC * 2), hi = lds_read_tr(st + ya[j] + (u * 32 + 4) * BC * 2);
          yf[j] = u32x4{lo[0], lo[1], hi[0], hi[1]};
        } else {
          yf[j] = *(const u32x4*)(st + ya[u] + j * 16 * KB);
        }
      }
#pragma unroll
      for (int c = 0; c < CJ; ++c)
#pragma unroll
        for (int r = 0; r < RJ; ++r) acc[c][r] = mfma16(yf[c], xf[r], acc[c][r]);
    }
  };

  // Lane (r16, q) holds columns 16c + 4q .. +3 of output row r16 for the fragments c.  Four
  // fragments are first turned within each quad of lanes, after which lane (4a + b, q) holds
  // columns 16b + 4q .. of rows 4a .. 4a+3: 16 lanes then write (and, adding, read) one row's 64
  // columns side by side, whole cache lines instead of 64-byte pieces of them.
  auto epilogue = [&]() {
    const int rows = OP == OP_WGRAD ? a.N : cw.cnt;
    const int64_t ob = OP == OP_WGRAD ? (int64_t)cw.e * a.N * a.K : (int64_t)cw.p0 * a.ldo;
    const int64_t ldo = OP == OP_WGRAD ? a.K : a.ldo;
    // row and first column of piece j of fragment row r
    constexpr bool TURN = CJ == 4;
    const int row0 = cw.r0 + wr * RJ * 16 + (TURN ? r16 & 12 : r16);
    const int col0 = cw.c0 + wc * CJ * 16 + 4 * q + (TURN ? (r16 & 3) * 16 : 0);
    auto at = [&](int r, int j, bool& ok) -> int64_t {
      const int row = row0 + r * 16 + (TURN ? j : 0), col = col0 + (TURN ? 0 : j * 16);
      ok = row < rows && col < Cdim;
      return ob + (int64_t)row * ldo + col;
    };
    if constexpr (TURN) {
#pragma unroll
      for (int r = 0; r < RJ; ++r) {
        floatx4 v[4] = {acc[0][r], acc[1][r], acc[2][r], acc[3][r]};
        quad_transpose(v);
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[j][r] = v[j];
      }
    }
    if constexpr (F32) {
      if (a.accumulate) {
        // the old values of many pieces at once: added one by one, each would wait for its own load
        constexpr int RP = RJ > 4 ? 1 : RJ;
#pragma unroll
        for (int r0 = 0; r0 < RJ; r0 += RP) {
          floatx4 old[CJ][RP];
#pragma unroll
          for (int r = 0; r < RP; ++r)
#pragma unroll
            for (int j = 0; j < CJ; ++j) {
              bool ok;
              const int64_t i = at(r0 + r, j, ok);
              old[j][r] = *(const floatx4*)((const float*)a.out + (ok ? i : ob));
            }
#pragma unroll
          for (int r = 0; r < RP; ++r)
#pragma unroll
            for (int j = 0; j < CJ; ++j) acc[j][r0 + r] += old[j][r];
        }
      }
    }
#pragma unroll
    for (int r = 0; r < RJ; ++r)
#pragma unroll
      for (int j = 0; j < CJ; ++j) {
        bool ok;
        const int64_t i = at(r, j, ok);
        if (!ok) continue;
        if constexpr (F32) *(floatx4*)((float*)a.out + i) = acc[j][r];
        else *(u32x2*)((uint16_t*)a.out + i) = u32x2{f32x2_to_bf16x2(acc[j][r][0], acc[j][r][1]), f32x2_to_bf16x2(acc[j][r][2], acc[j][r][3])};
      }
  };

  set_sources();
  load_rows();
#pragma unroll
  for (int j = 0; j < D; ++j) issue_next();

  // ---- steps: wait until only the loads of the later steps are outstanding (stores of an earlier
  // tile, which may end out of order, only make the wait stricter), meet the other waves (their
  // loads of this stage are in, their reads of the stage to be refilled are done), refill, multiply
  int cs = 0, stage = 0;
  for (;;) {
    --flying;
    if (flying < D - 1) {  // the end: at most D - 1 of these waits in a launch
      wait_vmcnt<0>();
    } else if constexpr (OP == OP_WGRAD || XN == 1) {
      wait_vmcnt<(D - 1) * (XN + YN)>();
    } else {
      static_assert(D == 1 || (D == 2 && XN == 2), "counts of one later step");
      if (D == 1) wait_vmcnt<0>();
      else if (n_last == 2) wait_vmcnt<2 + YN>();
      else wait_vmcnt<1 + YN>();
    }
    lds_barrier();
    issue_next();
    const bool live = OP == OP_WGRAD ? cw.r0 + wr * RJ * 16 < a.N : cw.r0 + wr * RJ * 16 < cw.cnt;
    if (live) compute(lds + stage);
    stage = stage == (NST - 1) * ST_BYTES ? 0 : stage + ST_BYTES;
    if (++cs == cw.nsteps) {
      // (adding, an empty group's gradient stays as it is: not even read)
      if (live && !(OP == OP_WGRAD && F32 && a.accumulate && cw.cnt == 0)) epilogue();
      clear();
      cs = 0;
      if (!advance(cw)) break;
    }
  }
  wait_vmcnt<0>();  // no direct-to-LDS load may outlive the workgroup
}

template <int OP, int KS, int BR, int BC, int WR, int WC, int NST>
hipError_t run_grouped(const GroupedArgs& a, int64_t max_items, int wg_per_cu, hipStream_t s) {
  const int cus = device_cu_count();
  if (cus <= 0) return hipErrorInvalidDevice;
  const int64_t grid = std::min<int64_t>((int64_t)(cus / 8 * 8) * wg_per_cu, (max_items + 7) / 8 * 8);
  if (grid <= 0) return hipSuccess;
  if (a.out_f32)
    hipLaunchKernelGGL((grouped_kernel<OP, KS, BR, BC, WR, WC, NST, true>), dim3((unsigned)grid), dim3(WR * WC * 64), 0, s, a);
  else
    hipLaunchKernelGGL((grouped_kernel<OP, KS, BR, BC, WR, WC, NST, false>), dim3((unsigned)grid), dim3(WR * WC * 64), 0, s, a);
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

// ---- which tile --------------------------------------------------------------------------------
// The group sizes are on the device; the host knows the positions and groups.  Each tile shape is
// priced for groups of equal size and the cheapest is taken:
//   rounds of the tiles over the workgroups that fit the card x (steps x step + tile), or what the
//   weights and results take at the memory's rate if that is more (then the first shape in order).
// `step` and `tile` (us, the end of a tile included) were fitted to sweeps over 1 to 8192 tokens,
// 1 to 512 groups and weights of 136 x 520 to 2560 x 768; `alone` is a step with one workgroup on
// its compute unit.  Sides measured (us, forward, 768 x 2560 weights, 8 of 512 groups a token):
//   1 token: 16x64 12, 32x128 19, 64x256 23, 128x256 31, 256x256 38
//   2048:    16x64 556, 32x128 422, 64x256 351, 128x256 351, 256x256 395
//   8192:    16x64 1740, 32x128 918, 64x256 579, 128x256 532, 256x256 489
struct Shape {
  int br, bc, ks, wgs;  // tile, reduction values per step, workgroups per compute unit
  float alone, step, tile;
};
constexpr double MEMORY_BYTES_PER_US = 5.8e6;

static double price(const Shape& v, double items, double steps64, int cus) {
  const double n = std::min<double>(v.wgs, std::max(1.0, items / cus));
  const double step = std::max<double>(v.alone, v.step * n / v.wgs);
  return std::ceil(items / ((double)cus * v.wgs)) * (std::ceil(steps64 * 64 / v.ks) * step + v.tile);
}

hipError_t launch_grouped_rows(const GroupedArgs& a, bool dgrad, hipStream_t s) {
  const int cols = dgrad ? a.K : a.N, red = dgrad ? a.N : a.K, cus = device_cu_count();
  if (cus <= 0) return hipErrorInvalidDevice;
  const int pair = a.w1 ? 2 : 1;
  static const Shape shapes[2][6] = {
      // the reduction along the weights' rows (forward): order of preference where memory bounds all
      {{16, 64, 128, 1, .30f, .48f, 1.f}, {128, 256, 64, 1, .6f, 1.13f, 3.f}, {64, 256, 64, 1, .42f, .86f, 2.5f},
       {32, 128, 64, 2, .32f, .55f, 1.5f}, {64, 64, 64, 3, .33f, .77f, .7f}, {256, 256, 64, 1, .8f, 1.5f, 7.f}},
      // across them (dgrad)
      {{128, 256, 64, 1, .6f, 1.25f, 3.f}, {64, 256, 64, 1, .42f, .82f, 2.5f}, {32, 128, 64, 2, .32f, .67f, 1.5f},
       {16, 64, 128, 1, .30f, .42f, 1.f}, {64, 64, 64, 3, .33f, 1.1f, .7f}, {256, 256, 64, 1, .8f, 1.6f, 7.5f}}};
  const double avg = (double)a.rows / a.groups, filled = a.groups * -std::expm1(-avg);
  const double floor = (filled * a.N * (double)a.K * 2 * pair + (double)a.rows * cols * (a.out_f32 ? 4 : 2)) / MEMORY_BYTES_PER_US;
  const Shape* best = nullptr;
  double cost = 0;
  for (const Shape& v : shapes[dgrad]) {
    const double in_group = std::max(avg, a.rows / std::max(filled, 1e-9));
    const double tiles = filled * std::max(1.0, in_group / v.br + (a.groups > 1 ? 0.5 : 0.0));
    const double c = std::max(floor, price(v, tiles * ((cols + v.bc - 1) / v.bc), pair * ((red + 63) / 64), cus));
    if (!best || c < cost) best = &v, cost = c;
  }
  // at most one partial tile per group that holds a position
  auto items = [&](int br, int bc) { return (a.rows / br + std::min<int64_t>(a.groups, a.rows)) * ((cols + bc - 1) / bc); };
#define MOE_GROUPED(KS, BR, BC, WR, WC, NST, WGS)                                                   \
  if (best->br == BR && best->bc == BC)                                                             \
    return dgrad ? run_grouped<OP_DGRAD, KS, BR, BC, WR, WC, NST>(a, items(BR, BC), WGS, s)         \
                 : run_grouped<OP_FWD, KS, BR, BC, WR, WC, NST>(a, items(BR, BC), WGS, s)
  MOE_GROUPED(128, 16, 64, 1, 4, 7, 1);
  MOE_GROUPED(64, 32, 128, 1, 4, 3, 2);
  MOE_GROUPED(64, 64, 64, 2, 2, 3, 3);
  MOE_GROUPED(64, 64, 256, 2, 4, 3, 1);
  MOE_GROUPED(64, 128, 256, 2, 4, 3, 1);
  MOE_GROUPED(64, 256, 256, 2, 4, 2, 1);
#undef MOE_GROUPED
  return hipErrorInvalidValue;
}

// Weight gradient: square tiles (both operands share their rows), the same pricing.  Sides measured
// (us, fp32 results): 512 groups of 768 x 2560, 8192 tokens: 64 2004, 128 1164, 256 871; one group,
// 8192 rows: 64 74, 128 97, 256 192; 64 groups of 136 x 520, 1024 tokens: 64 9.5, 128 12, 256 14.
hipError_t launch_grouped_wgrad(const GroupedArgs& a, hipStream_t s) {
  const int cus = device_cu_count();
  if (cus <= 0) return hipErrorInvalidDevice;
  static const Shape shapes[3] = {{256, 256, 64, 1, 1.5f, 2.3f, 9.4f}, {128, 128, 64, 2, .75f, 1.4f, 4.9f}, {64, 64, 64, 4, .55f, 1.4f, 2.f}};
  auto items = [&](int64_t b) { return a.groups * ((a.N + b - 1) / b) * ((a.K + b - 1) / b); };
  const double steps = std::max(1.0, (double)a.rows / a.groups / 64 + 0.5);
  const Shape* best = nullptr;
  double cost = 0;
  for (const Shape& v : shapes) {
    const double c = price(v, (double)items(v.br), steps, cus);
    if (!best || c < cost) best = &v, cost = c;
  }
  if (best->br == 256) return run_grouped<OP_WGRAD, 64, 256, 256, 2, 4, 2>(a, items(256), 1, s);
  if (best->br == 128) return run_grouped<OP_WGRAD, 64, 128, 128, 2, 2, 2>(a, items(128), 2, s);
  return run_grouped<OP_WGRAD, 64, 64, 64, 2, 2, 2>(a, items(64), 4, s);
}

}  // namespace moe
