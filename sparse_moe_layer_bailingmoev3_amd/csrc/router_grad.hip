// The two products of the router's backward pass, from the gradient dl [T,E] of the logits:
//
//   d router_w[e,h] = sum_t dl[t,e] x[t,h]        dx[t,h] = sum_e dl[t,e] router_w[e,h]
//
// dl and router_w are fp32, the matrix units take 16 bits.  Each fp32 value is taken apart into 16-bit
// pieces, and products are formed piece by piece with fp32 accumulation:
//   * d router_w: dl in three bf16 pieces (exactly: 8 bits each), x is bf16 itself.  Three products.
//     (Two rounded pieces lose 2.4e-6 in the norm, twice what a product in fp32 throughout loses.)
//   * dx: both operands in fp16, each row of dl and each column of router_w scaled by a power of two
//     that brings its largest value to 2^14..2^15, so that fp16's range covers 2^-38 of the largest; the
//     result is scaled back.  Two pieces each (22 bits), hi hi + hi lo + lo hi; what is left out is 2^-22 of
//     the magnitudes.  Three products, against six with three bf16 pieces each.  A result in bf16 is the same
//     sum rounded once.  (The first pieces alone, one product: 8192 tokens 115 instead of 144 us, 3e-4 in the norm,
//     but a sum that cancels was off by any number of steps of bf16.)
// The pieces are written by the kernel that computes dl (balance.hip), router_w's transposed.
//
// Both products are tiles of one launch, the weight gradient's (longer ones) first: the tokens' tiles,
// which end in reading and writing dx, then run beside them on the same compute units.
//
// One tile engine: BR rows by BC columns of the result, reduction steps of KS values, both operands'
// planes brought into a ring of NST LDS stages by direct loads, products on the 32 x 32 x 16 matrix
// instruction.  dx's planes run along the reduction and are read as they lie; d router_w's run across it
// and are read through the transposing LDS load.  Rows past the end are offsets past a buffer
// descriptor's end: zeros.
//
// What bounds it, on one MI355X: 8192 tokens of 512 x 2560, dx added to in fp32, 122 us at first and up to 167
// back to back (the card's power then holds its clock down): 129 GFLOP of products, 1.06 to 0.77 PFLOP/s (the
// library's bf16 product reaches 1.31 in short runs), matrix units busy 48 % of the cycles; LDS reads of a
// step (16 KB a wave for 24 products of 32 x 32 x 16) and what the loads write there take about as long as the
// products, no bank conflicts.  Calls for one product, 6400 tokens: d router_w 70 us, dx 59 in fp32, 54 in bf16.
// Measured and not kept: 256 x 256 tiles, as 16 waves of 64 x 64 or 4 waves of 128 x 128 that read the next
// fragments between the products (1.5 PFLOP/s within a tile, but 480 long items on 256 places end unevenly:
// 157 against 158 us a call), 256 x 128, steps of 16; dx's planes in rows of E values instead of blocks
// (dx alone 90 against 54 us: a load of 16 or 32 rows touched as many cache lines by halves or quarters);
// the tiles of both products mixed, or dx's first (+15 to +40 %); two rounded bf16 pieces of dl (-20 us, see
// above); the parts of d router_w added by the workgroup that finishes a tile last instead of a second launch
// (its fences write back a whole L2: +50 us at 8192 tokens, +20 at 1333; a join without fences, as the balance loss
// has it, is not tried); five stages for the 64 x 64 tiles (the same times).
#include <type_traits>

#include "moe_common.h"
#include "moe_internal.h"
#include "tile_ops.h"

namespace moe {

namespace {

constexpr int OP_DW = 0, OP_DX = 1;

typedef float floatx16 __attribute__((ext_vector_type(16)));

// 32 x 32 x 16 products.  Operands: lane l holds row l % 32, reduction values 8 (l / 32) .. +7.  Result:
// lane l holds column l % 32 (of b), rows 8g + 4 (l / 32) .. +3 (of a) in elements 4g .. 4g+3.
template <int OP>
__device__ __forceinline__ floatx16 mfma32(const u32x4& a, const u32x4& b, floatx16 c) {
  if constexpr (OP == OP_DW)
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// what a tile of BR x BC takes from LDS
template <int OP, int BR, int BC, int KS_>
struct Stage {
  static constexpr int KS = KS_, PX = OP == OP_DW ? 3 : 2, PY = OP == OP_DW ? 1 : 2;  // planes
  static constexpr int X_BYTES = BR * KS * 2, Y_BYTES = BC * KS * 2, BYTES = PX * X_BYTES + PY * Y_BYTES;
};

// 16-byte chunk swizzles.  Rows of 16 reduction values (2 chunks): the 16-byte LDS read serves lanes 0-3,
// 12-15, 20-23, 24-27 of each half wave together, then the others.
__device__ __forceinline__ int swz_row(int row) { return (row >> 4) & 1; }
// Rows of W output values under the transposing read, which touches rows r..r+3 and two blocks of 32 bytes
// in each half wave.
template <int W>
__device__ __forceinline__ int swz_cols(int row) { return W >= 128 ? (row & 3) << 2 : (row & 2) << 1; }

template <int OP, int BR, int BC, int WR, int WC, int KS, int NST, bool F32>
__device__ __forceinline__ void router_tile(const RouterGradArgs& a, int block, int blocks, uint8_t* lds) {
  typedef Stage<OP, BR, BC, KS> St;
  constexpr int NW = WR * WC, PX = St::PX, PY = St::PY;
  constexpr int X_BYTES = St::X_BYTES, Y_BYTES = St::Y_BYTES, ST_BYTES = St::BYTES;
  constexpr int XN = X_BYTES / (NW * 1024), YN = Y_BYTES / (NW * 1024), LN = PX * XN + PY * YN;  // loads per wave
  static_assert(XN * NW * 1024 == X_BYTES && YN * NW * 1024 == Y_BYTES, "a plane must split evenly over the waves");
  constexpr int RJ = BR / WR / 32, CJ = BC / WC / 32;
  constexpr int NA = RJ * CJ == 1 ? 2 : 1;   // sums that take turns (one alone would wait for itself)

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r32 = lane & 31, half = lane >> 5;
  const int wr = wave / WC, wc = wave % WC;

  // ---- which tile: consecutive ones (the column tiles of a row tile, the tiles of a split) on one XCD
  const int nct = (a.H + BC - 1) / BC;
  const int nrt = ((OP == OP_DW ? a.E : a.T) + BR - 1) / BR;
  const int tiles = nct * nrt, total = OP == OP_DW ? tiles * a.plan.nsplit : tiles;
  const int item = (block & 7) * (blocks >> 3) + (block >> 3);  // (blocks: total, rounded up to a multiple of 8)
  if (item >= total) return;
  const int split = item / tiles, tile = item - split * tiles;
  const int rt = tile / nct, r0 = rt * BR, c0 = (tile - rt * nct) * BC;
  const int red0 = OP == OP_DW ? split * a.plan.split_steps * 32 : 0;
  const int red = OP == OP_DW ? max(min(a.T - red0, a.plan.split_steps * 32), 0) : a.E;
  const int nsteps = (red + KS - 1) / KS;

  // ---- loads
  uint64_t xb[PX], yb[PY];
  uint32_t xo[XN], yo[YN], xstep, ystep;
  int xrow[XN], yrow[YN];  // reduction row of the loads (d router_w: masked in the last step)
  if constexpr (OP == OP_DX) {
    // planes in blocks of 32 rows by 16 values (plane_at): a load is one block
    each<PX>([&](auto p) { xb[p] = (uint64_t)(a.dh + p * plane_size(a.T, a.E) + (int64_t)r0 * a.E); });
    each<PY>([&](auto p) { yb[p] = (uint64_t)(a.wt + p * plane_size(a.H, a.E) + (int64_t)c0 * a.E); });
    xstep = ystep = KS * 64;
    auto offset = [&](int load, int blocks, int rows) {
      const int u = load / blocks, r = load % blocks * 32, row = lane / 2;
      return r + row < rows ? (uint32_t)(r * a.E * 2 + u * 1024 + row * 32 + (((lane & 1) ^ swz_row(row)) << 4)) : BUF_OUT;
    };
    each<XN>([&](auto i) { xo[i] = offset(wave * XN + i, BR / 32, a.T - r0); });
    each<YN>([&](auto i) { yo[i] = offset(wave * YN + i, BC / 32, a.H - c0); });
  } else {
    constexpr int XL = BR / 8, YL = BC / 8;
    each<PX>([&](auto p) { xb[p] = (uint64_t)(a.dl + ((int64_t)p * a.T + red0) * a.E + r0); });
    yb[0] = (uint64_t)(a.x + (int64_t)red0 * a.H + c0);
    xstep = KS * a.E * 2;
    ystep = KS * a.H * 2;
    each<XN>([&](auto i) {
      const int row = xrow[i] = (wave * XN + i) * (64 / XL) + lane / XL, ch = (lane % XL) ^ swz_cols<BR>(row);
      xo[i] = r0 + ch * 8 < a.E ? (uint32_t)(row * a.E * 2 + ch * 16) : BUF_OUT;
    });
    each<YN>([&](auto i) {
      const int row = yrow[i] = (wave * YN + i) * (64 / YL) + lane / YL, ch = (lane % YL) ^ swz_cols<BC>(row);
      yo[i] = c0 + ch * 8 < a.H ? (uint32_t)(row * a.H * 2 + ch * 16) : BUF_OUT;
    });
  }
  const uint32_t lds0 = lds_offset(lds);
  int left = red;  // reduction values from the next step to load on
  uint32_t lst = lds0;
  // Rows of x whose tokens have no gradient are not read (zeros instead): x may hold anything there, and 0
  // times an infinity is no part of the sum.  One byte a token, read through the scalar cache a step ahead;
  // a load's rows are 4 or 8 consecutive ones.
  constexpr int YROWS = 64 * 8 / BC;  // rows of a load of x
  typedef std::conditional_t<YROWS == 8, uint64_t, uint32_t> live_t;
  static_assert(YROWS == 8 || YROWS == 4, "a load's bytes in one word");
  typedef const __attribute__((address_space(4))) live_t* live_ptr;
  const uint8_t* live_at = a.live + red0;
  live_t live[YN] = {};
  auto load_live = [&]() {
    if constexpr (OP == OP_DW) {
      if (left <= 0) return;
      each<YN>([&](auto i) { live[i] = *(live_ptr)(uint64_t)(live_at + (wave * YN + i) * YROWS); });
      live_at += KS;
    }
  };
  load_live();
  auto issue = [&]() {
    const uint32_t st = __builtin_amdgcn_readfirstlane(lst);
    const bool whole = OP == OP_DX || left >= KS;
    each<PX>([&](auto p) {
      const u32x4 rs = buffer_at(xb[p]);
      each<XN>([&](auto i) {
        dma16(whole || xrow[i] < left ? xo[i] : BUF_OUT, rs, st + p * X_BYTES + (wave * XN + i) * 1024);
      });
      xb[p] += xstep;
    });
    each<PY>([&](auto p) {
      const u32x4 rs = buffer_at(yb[p]);
      each<YN>([&](auto i) {
        bool ok = whole || yrow[i] < left;
        if constexpr (OP == OP_DW) ok = ok && (live[i] >> (lane / (BC / 8) * 8) & 1);
        dma16(ok ? yo[i] : BUF_OUT, rs, st + PX * X_BYTES + p * Y_BYTES + (wave * YN + i) * 1024);
      });
      yb[p] += ystep;
    });
    left -= KS;
    load_live();
    lst = lst == lds0 + (NST - 1) * ST_BYTES ? lds0 : lst + ST_BYTES;
  };

  // ---- LDS read addresses.  Transposed: lanes 16g .. 16g+15 read rows 8 (g/2) .. of column block g%2.
  int xa[OP == OP_DW ? RJ : 1], ya[OP == OP_DW ? CJ : 1];
  if constexpr (OP == OP_DW) {
    const int row = 8 * half + ((lane & 15) >> 2), block16 = (lane >> 4) & 1, in = (lane & 3) * 8;
#pragma unroll
    for (int j = 0; j < RJ; ++j)
      xa[j] = row * BR * 2 + ((((wr * RJ + j) * 4 + block16 * 2) ^ swz_cols<BR>(row)) << 4) + in;
#pragma unroll
    for (int j = 0; j < CJ; ++j)
      ya[j] = PX * X_BYTES + row * BC * 2 + ((((wc * CJ + j) * 4 + block16 * 2) ^ swz_cols<BC>(row)) << 4) + in;
  } else {
    const int in = r32 * 32 + ((half ^ swz_row(r32)) << 4);
    xa[0] = wr * RJ * 1024 + in;
    ya[0] = PX * X_BYTES + wc * CJ * 1024 + in;
  }
  auto frag = [&](const uint8_t* st, const int* at, int j, int u, int row_bytes) {
    if constexpr (OP == OP_DW) {
      const uint8_t* const p = st + at[j] + u * 16 * row_bytes;
      const u32x2 lo = lds_read_tr(p), hi = lds_read_tr(p + 4 * row_bytes);
      return u32x4{lo[0], lo[1], hi[0], hi[1]};
    } else {
      return *(const u32x4*)(st + at[0] + u * 16 * row_bytes + j * 1024);
    }
  };

  floatx16 acc[NA][CJ][RJ];
#pragma unroll
  for (int n = 0; n < NA; ++n)
#pragma unroll
    for (int c = 0; c < CJ; ++c)
#pragma unroll
      for (int r = 0; r < RJ; ++r)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[n][c][r][i] = 0.f;

  auto compute = [&](const uint8_t* st) {
#pragma unroll
    for (int u = 0; u < KS / 16; ++u) {
      u32x4 yf[PY][CJ];
#pragma unroll
      for (int p = 0; p < PY; ++p)
#pragma unroll
        for (int c = 0; c < CJ; ++c) yf[p][c] = frag(st + p * Y_BYTES, ya, c, u, BC * 2);
#pragma unroll
      for (int r = 0; r < RJ; ++r) {
        u32x4 xf[PX];
#pragma unroll
        for (int p = 0; p < PX; ++p) xf[p] = frag(st + p * X_BYTES, xa, r, u, BR * 2);
        // small terms first
#pragma unroll
        for (int p = PX + PY - 2; p >= 0; --p)
#pragma unroll
          for (int c = 0; c < CJ; ++c) {
            floatx16& s = acc[(u * (PX + PY - 1) + p) % NA][c][r];
            if constexpr (OP == OP_DW) s = mfma32<OP>(yf[0][c], xf[p], s);
            else s = mfma32<OP>(yf[p == 2][c], xf[p == 1], s);
          }
      }
    }
  };

  // ---- steps: wait for this stage's loads (those of later stages stay in flight), meet the other
  // waves, refill the stage that all have left, multiply
#pragma unroll
  for (int j = 0; j < NST - 1; ++j)
    if (j < nsteps) issue();
  int stage = 0;
  for (int s = 0; s < nsteps; ++s) {
    if (nsteps - 1 - s >= NST - 2) wait_vmcnt<(NST - 2) * LN>();
    else wait_vmcnt<0>();
    lds_barrier();
    if (s + NST - 1 < nsteps) issue();
    compute(lds + stage);
    stage = stage == (NST - 1) * ST_BYTES ? 0 : stage + ST_BYTES;
  }

  // ---- result: four pieces of four columns a lane, turned within quads of lanes: 4 lanes of both half
  // waves then hold 32 columns of one row side by side (whole cache lines)
  const int rows = OP == OP_DW ? a.E : a.T;
  float* const o32 = OP == OP_DX ? (float*)a.dx : a.plan.nsplit > 1 ? a.part + (int64_t)split * a.E * a.H : a.dw;
  const bool add = OP == OP_DX ? a.acc_x : a.acc_w && a.plan.nsplit == 1;
  const int row0 = r0 + wr * RJ * 32 + (r32 & 28), col0 = c0 + wc * CJ * 32 + 8 * (r32 & 3) + 4 * half;
  // everything that the tile's end reads is asked for at once, or, the old values, a column of fragments
  // ahead of their use: one after another, each would wait for itself
  int er[RJ][4] = {}, ec[CJ][4] = {};
  if constexpr (OP == OP_DX) {  // (the exponents' arrays reach to the end of the last tile)
#pragma unroll
    for (int r = 0; r < RJ; ++r) {
      const int4 e = *(const int4*)(a.dexp + row0 + r * 32);
      er[r][0] = e.x, er[r][1] = e.y, er[r][2] = e.z, er[r][3] = e.w;
    }
#pragma unroll
    for (int c = 0; c < CJ; ++c) {
      const int4 e = *(const int4*)(a.wexp + col0 + c * 32);
      ec[c][0] = e.x, ec[c][1] = e.y, ec[c][2] = e.z, ec[c][3] = e.w;
    }
  }
  auto load_old = [&](auto c, floatx4 (&old)[RJ][4]) {
    if (!(F32 && add)) return;
    const int col = col0 + c * 32;
#pragma unroll
    for (int r = 0; r < RJ; ++r)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int row = row0 + r * 32 + j;
        old[r][j] = *(const floatx4*)(o32 + (row < rows && col < a.H ? (int64_t)row * a.H + col : 0));
      }
  };
  auto finish = [&](auto c, const floatx4 (&old)[RJ][4]) {
    const int col = col0 + c * 32;
#pragma unroll
    for (int r = 0; r < RJ; ++r) {
      floatx4 v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[j][i] = acc[0][c][r][4 * j + i];
          if constexpr (NA == 2) v[j][i] += acc[NA - 1][c][r][4 * j + i];
        }
      quad_transpose(v);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int row = row0 + r * 32 + j;
        if (row >= rows || col >= a.H) continue;
        const int64_t at = (int64_t)row * a.H + col;
        if constexpr (OP == OP_DX) {
#pragma unroll
          for (int i = 0; i < 4; ++i) v[j][i] = __builtin_amdgcn_ldexpf(v[j][i], -(er[r][j] + ec[c][i]));
        }
        if (F32 && add) v[j] += old[r][j];
        if constexpr (F32) *(floatx4*)(o32 + at) = v[j];
        else *(u32x2*)((uint16_t*)a.dx + at) = u32x2{f32x2_to_bf16x2(v[j][0], v[j][1]), f32x2_to_bf16x2(v[j][2], v[j][3])};
      }
    }
  };
  floatx4 old0[RJ][4], old1[RJ][4];
  load_old(std::integral_constant<int, 0>{}, old0);
  each<CJ>([&](auto c) {
    constexpr int C = decltype(c)::value;
    auto& now = C % 2 ? old1 : old0;
    if constexpr (C + 1 < CJ) load_old(std::integral_constant<int, C + 1>{}, C % 2 ? old0 : old1);
    finish(c, now);
  });
}

// d router_w = (d router_w +) the splits' parts in order
__global__ __launch_bounds__(256) void router_join_kernel(RouterGradArgs a) {
  const int64_t n = (int64_t)a.E * a.H, i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (i >= n) return;
  floatx4 v{0.f, 0.f, 0.f, 0.f};
  if (a.acc_w) v = *(const floatx4*)(a.dw + i);
  floatx4 s{0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
  for (int p = 0; p < a.plan.nsplit; ++p) s += *(const floatx4*)(a.part + p * n + i);
  *(floatx4*)(a.dw + i) = v + s;
}

template <int BR, int BC, int WR, int WC, int KS, int NW, int NX, bool F32>
__global__ __launch_bounds__(WR* WC * 64, 2) void router_products_kernel(RouterGradArgs a, int dw_blocks) {
  constexpr int DW = NW * Stage<OP_DW, BR, BC, KS>::BYTES, DX = NX * Stage<OP_DX, BR, BC, KS>::BYTES;
  __shared__ __align__(16) uint8_t lds[DW > DX ? DW : DX];
  const int block = blockIdx.x;
  if (block < dw_blocks) router_tile<OP_DW, BR, BC, WR, WC, KS, NW, true>(a, block, dw_blocks, lds);
  else router_tile<OP_DX, BR, BC, WR, WC, KS, NX, F32>(a, block - dw_blocks, (int)gridDim.x - dw_blocks, lds);
}

template <int BR, int BC, int WR, int WC, int KS, int NW, int NX>
void run_products(const RouterGradArgs& a, hipStream_t s) {
  auto blocks = [&](int64_t rows, int n) { return (int)(((rows + BR - 1) / BR * ((a.H + BC - 1) / BC) * n + 7) / 8 * 8); };
  // (no tokens: zeros, or what lay there to the bit)
  const int dw = a.dw && (a.T > 0 || !a.acc_w) ? blocks(a.E, a.plan.nsplit) : 0, dx = a.dx && a.T > 0 ? blocks(a.T, 1) : 0;
  if (dw + dx == 0) return;
  if (a.dx_f32)
    hipLaunchKernelGGL((router_products_kernel<BR, BC, WR, WC, KS, NW, NX, true>), dim3((unsigned)(dw + dx)), dim3(WR * WC * 64), 0, s, a, dw);
  else
    hipLaunchKernelGGL((router_products_kernel<BR, BC, WR, WC, KS, NW, NX, false>), dim3((unsigned)(dw + dx)), dim3(WR * WC * 64), 0, s, a, dw);
}

}  // namespace

// Parts of d router_w's reduction over tokens that a plan takes at most: so many that its tiles are all under way
// at once (two workgroups a compute unit), up to 32.  More would wait for places, and cost their bytes besides: no
// plan of 64 x 128 to 1024 x 7168 and 1 to 300,000 tokens priced more as best.
constexpr int PRODUCT_PLACES = 512, MAX_PARTS = 32;
static int64_t most_parts(int64_t steps, int64_t tiles) {
  return std::min<int64_t>(std::min<int64_t>(steps, MAX_PARTS), std::max<int64_t>(PRODUCT_PLACES / std::max<int64_t>(tiles, 1), 1));
}
static int64_t token_steps(int64_t T) { return std::max<int64_t>((T + 31) / 32, 1); }
int router_grad_parts_bound(int64_t T, int E, int H) {
  return (int)most_parts(token_steps(T), (int64_t)((E + 127) / 128) * ((H + 127) / 128));
}

// Tile size and the parts of the weight gradient's reduction, by price: a step of one product of a tile
// takes `full` us on a place with all `wgs` places of its compute unit taken, `alone` at least; `end` is a tile's
// beginning and end, 5 us what a third launch costs, besides the parts' bytes.  The weight gradient's items
// are started first, the others fill the places that they leave.  For the MI355X's 256 compute units; fitted to
// sweeps over 16 to 8192 tokens at 64 x 512 to 1024 x 2560.  Sides measured (us a call, 512 x 2560, fp32 dx):
//   512 tokens:  128 26.4, 64 28.6     2048: 128 in 2 parts 50.5, 4 56.7; 64 62.4     8192: 128 148, 64 206
//   512 tokens of 128 x 640: 64 in one part 14.5, 2 17.4; 4096: 64 in 8 parts 22.0, 128 24.6
RouterGradPlan router_grad_plan(int64_t T, int E, int H, bool dw, bool dx) {
  struct Shape {
    int tile, wgs;
    float alone, full, end;
  };
  static const Shape shapes[2] = {{128, 2, .25f, .45f, 4.f}, {64, 2, .05f, .17f, 2.5f}};
  const int64_t steps = token_steps(T);
  RouterGradPlan best{};
  double cost = -1;
  for (const Shape& v : shapes) {
    const double places = PRODUCT_PLACES;
    const int64_t ct = (H + v.tile - 1) / v.tile, dwt = dw ? (E + v.tile - 1) / v.tile * ct : 0, dxt = dx ? (T + v.tile - 1) / v.tile * ct : 0;
    for (int64_t n = 1; n <= (dw ? most_parts(steps, dwt) : 1); ++n) {
      const int64_t per = (steps + n - 1) / n;
      if ((steps + per - 1) / per != n) continue;
      const double items = (double)dwt * n, load = std::min<double>(v.wgs, std::max(1.0, (items + dxt) / 256));
      const double step = std::max<double>(v.alone, v.full * load / v.wgs);
      const double len = per * 3 * step + v.end, dx_len = dxt ? (E / 32) * 3 * step + v.end : 0;
      const double c = std::max(std::ceil(items / places) * len, (items * len + dxt * dx_len) / places + .5 * dx_len) +
                       (n > 1 ? 5 + n * (double)E * H * 8 / 5e6 : 0);
      if (cost < 0 || c < cost) {
        cost = c;
        best = {v.tile, (int)n, (int)per};
      }
    }
  }
  return best;
}

hipError_t launch_router_grad(const RouterGradArgs& a, hipStream_t s) {
  if (a.plan.tile == 128) run_products<128, 128, 2, 2, 32, 2, 2>(a, s);
  else run_products<64, 64, 2, 2, 32, 4, 4>(a, s);
  if (a.dw && a.plan.nsplit > 1)
    hipLaunchKernelGGL(router_join_kernel, dim3((unsigned)(((int64_t)a.E * a.H + 1023) / 1024)), dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace moe
