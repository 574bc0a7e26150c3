// 4-bit weights: their quantisation (E2M1 codes, one power-of-two scale per 32 elements along
// K) and products of few rows with them, dense or over expert segments, plain or gated:
//     y = x W^T,   or  h = g * sigmoid(g) * u  with g, u the two halves of x W^T.
// Bound by the stream of the weights from HBM (4.25 bits each) for up to 16 rows: 36864 x 7168 with one row 31 us, at
// 4.5 TB/s; 29 experts of 4096 x 7168 with 128 rows 96 us, at 4.7.  With more rows of X by what a tile costs a
// wavefront: its instructions that widen W, and X's way through L2 and LDS (48 rows, 7168 x 18432: 34-36 us, 2.0 TB/s).
//
// The products run on the bf16 matrix cores: every E2M1 value times its power of two, and
// every E4M3 value, is a bf16 value, so each product is exact and the sums are fp32.
#include <type_traits>

#include "activation.h"
#include "fp4_shape.h"
#include "gemm_fp8_tile.h"
#include "launch.h"
#include "lanes.h"

namespace fp8fg {
namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// ---------------------------------------------------------------- quantisation
// Four lanes per group of 32, eight elements each.
template <bool BF16>
__global__ void __launch_bounds__(256) fp4_quant_kernel(const void* __restrict__ w, int64_t octets, int64_t per_row,
                                                        int64_t ld, uint8_t* __restrict__ q,
                                                        uint8_t* __restrict__ scales) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= octets) return;  // (whole groups: K is a multiple of 128)
  const int64_t row = i / per_row, at = row * ld + (i - row * per_row) * 8;
  float f[8];
  if constexpr (BF16) {
    const u32x4 u = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(w) + at));
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      f[2 * k] = __uint_as_float(u[k] << 16);
      f[2 * k + 1] = __uint_as_float(u[k] & 0xFFFF0000u);
    }
  } else {
    const f32x4* p = reinterpret_cast<const f32x4*>(static_cast<const float*>(w) + at);
    const f32x4 lo = __builtin_nontemporal_load(p), hi = __builtin_nontemporal_load(p + 1);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      f[k] = lo[k];
      f[4 + k] = hi[k];
    }
  }
  float top = 0.0f;
#pragma unroll
  for (int k = 0; k < 8; ++k) top = fmaxf(top, fabsf(f[k]));
  top = fmaxf(top, dpp<0xB1>(top));
  top = fmaxf(top, dpp<0x4E>(top));
  // 6 = 1.5 * 2^2: the exponent two below that of the largest, one more above 1.5
  const uint32_t b = __float_as_uint(top);
  int e = static_cast<int>(b >> 23) - 2 + ((b & 0x7FFFFFu) > 0x400000u ? 1 : 0);
  e = e < 1 ? 1 : e;
  const float inv = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
  uint32_t code = 0;
  code = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(code, f[0] * inv, f[1] * inv, 1.0f, 0);
  code = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(code, f[2] * inv, f[3] * inv, 1.0f, 1);
  code = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(code, f[4] * inv, f[5] * inv, 1.0f, 2);
  code = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(code, f[6] * inv, f[7] * inv, 1.0f, 3);
  reinterpret_cast<uint32_t*>(q)[i] = code;
  if ((threadIdx.x & 3) == 0) scales[i >> 2] = static_cast<uint8_t>(e);
}

// ---------------------------------------------------------------- products
// Eight E2M1 codes times 2^(e - 127) as bf16, exact.
__device__ __forceinline__ bf16x8 widen_fp4(uint32_t c, float scale) {
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 0);
  const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 1);
  const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 2);
  const bf16x2 e = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 3);
  return bf16x8{a[0], a[1], b[0], b[1], d[0], d[1], e[0], e[1]};
}
// Eight E4M3 codes as bf16, exact.
__device__ __forceinline__ bf16x8 widen_e4m3(uint32_t lo, uint32_t hi) {
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false);
  const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
  const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false);
  const bf16x2 e = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
  return bf16x8{a[0], a[1], b[0], b[1], d[0], d[1], e[0], e[1]};
}

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// Tiles of the output are numbered by segment, then column, then row, so that the row tiles of one
// column tile, which read the same weights, come next to each other.
struct Segment {
  int e, lo, hi;      // expert, its rows
  int first, end;     // its tiles
};

// The segments of 256 experts, four to a lane: their bounds, held to [0, M], and the row tiles of ROWS rows before the
// lane's.  rising: no offset is below the one before it; only then are the tiles no more than the host counted.
template <int ROWS>
struct SegmentTable {
  int lo[4], hi[4], before, total;
  bool rising;

  __device__ __forceinline__ int tiles(int i) const { return fp4_row_tiles(lo[i], hi[i], ROWS); }
  __device__ __forceinline__ void load(const Fp4Args& a, int64_t base) {
    const int lane = threadIdx.x & 63, M = static_cast<int>(a.M);
    int v[5];
#pragma unroll
    for (int i = 0; i < 5; ++i) {
      const int64_t g = base + 4 * lane + i;
      v[i] = a.offsets[g < a.G ? g : a.G];
    }
    int sum = 0;
    bool falls = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      falls |= v[i + 1] < v[i];
      lo[i] = v[i] < 0 ? 0 : (v[i] > M ? M : v[i]);
      hi[i] = v[i + 1] < lo[i] ? lo[i] : (v[i + 1] > M ? M : v[i + 1]);
      if (base + 4 * lane + i >= a.G) hi[i] = lo[i];
      sum += tiles(i);
    }
    int incl = sum;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_up(incl, d);
      if (lane >= d) incl += o;
    }
    before = incl - sum;
    rising = __ballot(falls) == 0;
    total = __builtin_amdgcn_readlane(incl, 63);
  }
  // The segment of tile t, numbered from the table's first; false: it lies behind the table.
  __device__ __forceinline__ bool find(int t, int col_tiles, int64_t base, int number, Segment& s) const {
    int first = before * col_tiles, at = -1, f = 0, n = 0, l = 0, h = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int cnt = tiles(i) * col_tiles;
      if (t >= first && t < first + cnt) {
        at = i;
        f = first;
        n = cnt;
        l = lo[i];
        h = hi[i];
      }
      first += cnt;
    }
    const uint64_t who = __ballot(at >= 0);
    if (!who) return false;
    const int src = __ffsll(static_cast<unsigned long long>(who)) - 1;
    s.e = static_cast<int>(base) + 4 * src + __builtin_amdgcn_readlane(at, src);
    s.lo = __builtin_amdgcn_readlane(l, src);
    s.hi = __builtin_amdgcn_readlane(h, src);
    s.first = number + __builtin_amdgcn_readlane(f, src);
    s.end = s.first + __builtin_amdgcn_readlane(n, src);
    return true;
  }
};

// A tile of LDS rows of C chunks of 16 bytes, filled by whole-wavefront DMAs of 64 chunks: where
// row r's chunk c lies.  The permutation keeps the 16 rows of a fragment read on different banks.
template <int C>
__device__ __forceinline__ int place(int r, int c) {
  return r * C + (c ^ (C >= 8 ? r & 7 : (r >> 1) & 3));
}

// The rings' loads are issued as x(t + SX - 1), w(t + SW - 1) in stage t, and return in that order.
// Loads issued after all of stage t's own when it is waited for, `left` more stages following it
// (those of the scales come on top).
constexpr int later_loads(int LX, int LW, int SX, int SW, int left) {
  const int x = left < SX - 1 ? left : SX - 1;
  const int w = (left < SW - 1 ? left : SW - 1) - (SX == SW ? 0 : SW - SX - 1);
  return LX * x + LW * (w > 0 ? w : 0);
}
// The wait of the last stages, behind which no load of W has been issued.
template <int LX, int LW, int SX, int SW, int L = 0>
__device__ __forceinline__ void wait_last(int left) {
  if constexpr (L < SW - 1) {
    if (left == L)
      asm volatile("s_waitcnt vmcnt(%0)" ::"i"(later_loads(LX, LW, SX, SW, L)) : "memory");
    else
      wait_last<LX, LW, SX, SW, L + 1>(left);
  }
}

// Sub-tiles whose partial sums a wavefront puts into `room` KB at a time: a divisor of all of them.
constexpr int sums_at_once(int all, int room) {
  int n = all;
  while (n > room || all % n != 0) --n;
  return n;
}

// A workgroup walks over tiles of XR rows of X by NF sub-tiles of 16 rows of W (gated: 8 gate
// rows and the 8 up rows of the same columns).  Its KW wavefronts take a part of K each; every
// wavefront moves its own operands, KU values of K at a time, into rings of its own in LDS (SW
// stages of W, SX of X) and waits for its own loads only: the stream of weights goes on from
// tile to tile.  A tile's partial sums meet in LDS and are added in the order of K.
// (One tile per workgroup, without the walk, left every tile its own start: 128 rows over 32 experts of 4096 x
// 7168 took 135 us instead of 97.  Loading straight into the MFMA layout, 64 bytes of 16 rows at a time, reached
// 2.4 TB/s where the rings reach 4.4.)
// Of an MFMA's operands a lane holds row lane % 16 and the 32 values 32 (lane / 16) .. + 31 of
// each 128 along K, eight to an instruction.
template <bool CODES, bool GATED, bool GROUPED, int XR, int NF, int KW, int SW, int SX, int KU>
__global__ void __launch_bounds__(KW * 64) fp4_gemm_kernel(Fp4Args a) {
  constexpr int MF = (XR + 15) / 16;
  constexpr int COLS = (GATED ? 8 : 16) * NF;
  constexpr int ES = CODES ? 1 : 2;
  constexpr int XC = KU * ES / 16, WC = KU / 32;                   // chunks of 16 bytes per row
  constexpr int XD = (XR * XC + 63) / 64, WD = NF * 16 * WC / 64;  // DMAs per stage
  constexpr int SR = KU / 128;                                     // dwords of scales per row
  constexpr int SD = NF * 16 * SR * 4 / 64, SXD = CODES ? (XR * SR + 63) / 64 : 0;  // (W's: of four stages)
  constexpr int LX = XD + SXD, LW = WD;
  constexpr int WAIT = later_loads(LX, LW, SX, SW, SW - 1);
  constexpr int W_STAGE = WD * 1024, X_STAGE = XD * 1024 + SXD * 256, S_STAGE = SD * 256, SS = SW;
  constexpr int S_AT = SW * W_STAGE, X_AT = S_AT + SS * S_STAGE;
  constexpr int RING = X_AT + SX * X_STAGE;
  constexpr int SUMS = sums_at_once(MF * NF, WD + XD);
  static_assert(SW >= SX && WAIT < 64, "the wait counter");
  static_assert(KW * RING <= 163840, "LDS");
  __shared__ __attribute__((aligned(1024))) uint8_t lds[KW * RING];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int row = lane & 15, j = lane >> 4;
  const int KB = static_cast<int>(a.K / 128);
  const int col_tiles = static_cast<int>((a.N + COLS - 1) / COLS);
  const bool indexed = GROUPED && a.row_index;

  // tiles [t0, t1) of this workgroup
  SegmentTable<XR> table{};  // of the first 256 experts; those behind are loaded again where they are needed
  int row_tiles = static_cast<int>((a.M + XR - 1) / XR);
  if constexpr (GROUPED) {
    table.load(a, 0);
    row_tiles = table.total;
    bool rising = table.rising;
    for (int64_t base = 256; base < a.G; base += 256) {
      SegmentTable<XR> more;
      more.load(a, base);
      row_tiles += more.total;
      rising &= more.rising;
    }
    if (!rising) return;
  }
  const int all = row_tiles * col_tiles;
  const int each = uniform(all / static_cast<int>(gridDim.x)), rest = all - each * static_cast<int>(gridDim.x);
  // workgroups of one XCD (every eighth) take neighbouring tiles: those of the same columns of W share its L2
  // (512 rows over 32 experts of 4096 x 7168: 151 -> 140 us; 48 rows, 7168 x 18432: 38 -> 34)
  const int xcd = static_cast<int>(blockIdx.x) & 7, grid = static_cast<int>(gridDim.x);
  const int block =
      xcd * (grid >> 3) + (xcd < (grid & 7) ? xcd : grid & 7) + (static_cast<int>(blockIdx.x) >> 3);
  const int t0 = block * each + (block < rest ? block : rest), t1 = t0 + each + (block < rest ? 1 : 0);
  if (t0 >= t1) return;
  auto locate = [&](int t, Segment& s, int& lo, int& hi, int& n0) {
    if constexpr (GROUPED) {
      if (t < s.first || t >= s.end) {
        int number = table.total * col_tiles;
        if (t < number) {
          table.find(t, col_tiles, 0, 0, s);
        } else {
          for (int64_t base = 256; base < a.G; base += 256) {
            SegmentTable<XR> more;
            more.load(a, base);
            if (more.find(t - number, col_tiles, base, number, s)) break;
            number += more.total * col_tiles;
          }
        }
      }
    }
    const int rt = fp4_row_tiles(s.lo, s.hi, XR), r = t - s.first, c = rt == 1 ? r : uniform(r / rt);
    lo = s.lo + (r - c * rt) * XR;
    hi = s.hi - lo > XR ? lo + XR : s.hi;
    n0 = c * COLS;
  };

  const int NU = (KB + SR - 1) / SR;  // stages of the whole K
  const int begin = wave * NU / KW, n = (wave + 1) * NU / KW - begin;
  const int64_t stages = static_cast<int64_t>(t1 - t0) * n;
  uint8_t* ring = lds + wave * RING;
  const uint32_t ring_at = __builtin_amdgcn_readfirstlane(lds_addr(ring));
  // In the last, half stage of an odd number of blocks the chunks of the second half are those
  // of the first again: this much further back.
  const uint32_t w_back = SR == 2 && (place<WC>(lane / WC, lane % WC) % WC) >= WC / 2 ? WC * 8 : 0;
  const uint32_t x_back = SR == 2 && (place<XC>(lane / XC, lane % XC) % XC) >= XC / 2 ? XC * 8 : 0;

  struct Cursor {
    Segment s;
    int64_t stage;
    int tile, u, slot;
  };
  // W's cursor: where the next stage of weights and scales comes from
  Cursor cw{Segment{0, 0, GROUPED ? 0 : static_cast<int>(a.M), 0, GROUPED ? 0 : all}, 0, t0, 0, 0}, cx = cw;
  Segment sc = cw.s;
  const uint8_t* w_base = nullptr;
  uint32_t w_off[WD];
  const uint8_t* s_ptr[SD];
  int s_slot = 0;
  auto aim_w = [&]() {
    int lo, hi, n0;
    locate(cw.tile, cw.s, lo, hi, n0);
    const int64_t wrows = GATED ? 2 * a.N : a.N;
    w_base = a.w + (cw.s.e * wrows + n0) * (a.K / 2);
    const uint8_t* sw = a.sw + cw.s.e * wrows * (a.K / 32);
    auto w_row = [&](int f, int r) -> int64_t {  // columns past the end: the last one again
      int64_t c = static_cast<int64_t>(n0) + (GATED ? f * 8 + (r & 7) : f * 16 + r);
      c = c < a.N ? c : a.N - 1;
      return c + (GATED && r >= 8 ? a.N : 0);
    };
#pragma unroll
    for (int i = 0; i < WD; ++i) {
      const int p = 64 * i + lane, r = p / WC;
      w_off[i] =
          static_cast<uint32_t>((w_row(r / 16, r % 16) - n0) * (a.K / 2)) + (place<WC>(r, p % WC) - r * WC) * 16;
    }
#pragma unroll
    for (int i = 0; i < SD; ++i) {
      const int r = (64 * i + lane) / (4 * SR);
      s_ptr[i] = sw + w_row(r / 16, r % 16) * (a.K / 32);
    }
  };
  auto issue_w = [&]() {
    if (cw.u == 0) aim_w();
    const int64_t u = begin + cw.u;
    const bool half = SR == 2 && 2 * u + 1 >= KB;
    const uint32_t at = uniform(ring_at + static_cast<uint32_t>(cw.slot) * W_STAGE);
    if (half) {
#pragma unroll
      for (int d = 0; d < WD; ++d) dma16(w_base + u * (KU / 2), w_off[d] - w_back, at + d * 1024);
    } else {
#pragma unroll
      for (int d = 0; d < WD; ++d) dma16(w_base + u * (KU / 2), w_off[d], at + d * 1024);
    }
    if (cw.u % 4 == 0) {
      // the scales of four stages at a time, 32 bytes of a row instead of 8 (one token, 7168 x 18432: 15.8 ->
      // 15.1 us); blocks past the row's end: its last
      const int64_t k = u * SR + lane % (4 * SR), kb = k < KB ? k : KB - 1;
      const uint32_t to = uniform(ring_at + S_AT + static_cast<uint32_t>(s_slot) * S_STAGE);
#pragma unroll
      for (int d = 0; d < SD; ++d) dma4(s_ptr[d] + kb * 4, to + d * 256);
      s_slot = s_slot == SS - 1 ? 0 : s_slot + 1;
    }
    ++cw.stage;
    cw.slot = cw.slot == SW - 1 ? 0 : cw.slot + 1;
    if (++cw.u == n) {
      cw.u = 0;
      ++cw.tile;
    }
  };
  // X's cursor
  const uint8_t* x_base = nullptr;
  uint32_t x_off[XD];
  const float* sx_ptr[CODES ? SXD : 1];
  int x_lo = -1;
  auto aim_x = [&]() {
    int lo, hi, n0;
    locate(cx.tile, cx.s, lo, hi, n0);
    if (lo == x_lo) return;
    x_lo = lo;
    auto x_row = [&](int r) -> int64_t {  // rows past the end: the last one again, not stored
      const int m = r < hi - lo ? lo + r : hi - 1;
      if (!indexed) return m;
      const int64_t v = a.row_index[m];
      return v < 0 ? 0 : (v >= a.T ? a.T - 1 : v);
    };
    const int64_t first = indexed ? 0 : lo;
    x_base = static_cast<const uint8_t*>(a.x) + first * a.K * ES;
#pragma unroll
    for (int i = 0; i < XD; ++i) {
      const int p = 64 * i + lane, r = p / XC;
      x_off[i] = static_cast<uint32_t>((x_row(r) - first) * a.K * ES) + (place<XC>(r, p % XC) - r * XC) * 16;
    }
    if constexpr (CODES) {
#pragma unroll
      for (int i = 0; i < SXD; ++i) sx_ptr[i] = a.sx + x_row((64 * i + lane) / SR) * KB + lane % SR;
    }
  };
  auto issue_x = [&]() {
    if (cx.u == 0) aim_x();
    const int64_t u = begin + cx.u;
    const bool half = SR == 2 && 2 * u + 1 >= KB;
    const uint32_t at = uniform(ring_at + X_AT + static_cast<uint32_t>(cx.slot) * X_STAGE);
    if (half) {
#pragma unroll
      for (int d = 0; d < XD; ++d) dma16(x_base + u * (KU * ES), x_off[d] - x_back, at + d * 1024);
    } else {
#pragma unroll
      for (int d = 0; d < XD; ++d) dma16(x_base + u * (KU * ES), x_off[d], at + d * 1024);
    }
    if constexpr (CODES) {
#pragma unroll
      for (int d = 0; d < SXD; ++d) dma4(sx_ptr[d] + u * SR - (half ? lane % SR : 0), at + XD * 1024 + d * 256);
    }
    ++cx.stage;
    cx.slot = cx.slot == SX - 1 ? 0 : cx.slot + 1;
    if (++cx.u == n) {
      cx.u = 0;
      ++cx.tile;
    }
  };

  f32x4 acc[MF][NF];
  auto multiply = [&](int u, const uint8_t* wst, const uint8_t* sst, const uint8_t* xst) {
    const u32x4* ws = reinterpret_cast<const u32x4*>(wst);
    const u32x4* xs = reinterpret_cast<const u32x4*>(xst);
#pragma unroll
    for (int b = 0; b < SR; ++b) {
      if (b == 1 && 2 * (begin + u) + 1 >= KB) continue;
      u32x4 wv[NF], xv[MF][2 * ES];
      float sc[NF];
#pragma unroll
      for (int f = 0; f < NF; ++f) {
        wv[f] = ws[place<WC>(f * 16 + row, 4 * b + j)];
        sc[f] = __uint_as_float(static_cast<uint32_t>(sst[(f * 16 + row) * (KU / 8) + 4 * b + j]) << 23);
      }
#pragma unroll
      for (int m = 0; m < MF; ++m)
#pragma unroll
        for (int c = 0; c < 2 * ES; ++c)
          xv[m][c] = xs[place<XC>(m * 16 + (XR < 16 ? row & (XR - 1) : row), (8 * b + 2 * j) * ES + c)];
      f32x4 p[MF][NF];
#pragma unroll
      for (int m = 0; m < MF; ++m)
#pragma unroll
        for (int f = 0; f < NF; ++f) p[m][f] = CODES ? f32x4{0.0f, 0.0f, 0.0f, 0.0f} : acc[m][f];
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        bf16x8 wf[NF];
#pragma unroll
        for (int f = 0; f < NF; ++f) wf[f] = widen_fp4(wv[f][s], sc[f]);
#pragma unroll
        for (int m = 0; m < MF; ++m) {
          bf16x8 xf;
          if constexpr (CODES)
            xf = widen_e4m3(xv[m][s >> 1][2 * (s & 1)], xv[m][s >> 1][2 * (s & 1) + 1]);
          else
            xf = __builtin_bit_cast(bf16x8, xv[m][s]);
#pragma unroll
          for (int f = 0; f < NF; ++f) p[m][f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xf, wf[f], p[m][f], 0, 0, 0);
        }
      }
#pragma unroll
      for (int m = 0; m < MF; ++m) {
        if constexpr (CODES) {
          const float* sx = reinterpret_cast<const float*>(xst + XD * 1024);
          float k[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int r = 16 * m + 4 * j + q;
            k[q] = sx[(XR < 16 ? r & (XR - 1) : r) * SR + b];
          }
#pragma unroll
          for (int f = 0; f < NF; ++f)
#pragma unroll
            for (int q = 0; q < 4; ++q) acc[m][f][q] = fmaf(p[m][f][q], k[q], acc[m][f][q]);
        } else {
#pragma unroll
          for (int f = 0; f < NF; ++f) acc[m][f] = p[m][f];
        }
      }
    }
  };
  // The order of the loads is that of the loop below from the start: x's first stage is followed
  // by one of w and SX - 1 of both when the loop waits for it.
  if (n > 0) {
#pragma unroll
    for (int i = 0; i < SW - 1; ++i) {
      if (i >= SW - SX && cx.stage < stages) issue_x();
      if (cw.stage < stages) issue_w();
    }
  }
  // Where a wavefront v's partial sums of sub-tile q lie: in the slots that it has read last, which are not loaded into
  // before its next stage.  (Room of their own, and with it one barrier's wait less, is no faster, and the room is
  // better spent on longer stages: 16 rows of 7168 x 18432 24.3 -> 21.5 us.)
  auto sums_of = [&](int v, int q, int tiles) -> f32x4* {
    const uint32_t nv = (v + 1) * NU / KW - v * NU / KW, n = tiles;  // (a wavefront without stages: any slot)
    uint8_t* own = lds + v * RING;
    return reinterpret_cast<f32x4*>(q < WD ? own + (n % SW * nv + SW - 1) % SW * W_STAGE + q * 1024
                                           : own + X_AT + (n % SX * nv + SX - 1) % SX * X_STAGE + (q - WD) * 1024);
  };
  int w_slot = 0, x_slot = 0, r_slot = 0;
  int64_t stage = 0;
  for (int t = t0; t < t1; ++t) {
#pragma unroll
    for (int m = 0; m < MF; ++m)
#pragma unroll
      for (int f = 0; f < NF; ++f) acc[m][f] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    for (int u = 0; u < n; ++u) {
      // the slots read in the previous stage: their reads have returned
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      if (cx.stage < stages) issue_x();
      if (cw.stage < stages) {
        issue_w();
        asm volatile("s_waitcnt vmcnt(%0)" ::"i"(WAIT) : "memory");
      } else {
        wait_last<LX, LW, SX, SW>(static_cast<int>(stages - 1 - stage));
      }
      if (u % 4 == 0 && stage > 0) r_slot = r_slot == SS - 1 ? 0 : r_slot + 1;
      ++stage;
      multiply(u, ring + w_slot * W_STAGE, ring + S_AT + r_slot * S_STAGE + (u % 4) * (KU / 32),
               ring + X_AT + x_slot * X_STAGE);
      w_slot = w_slot == SW - 1 ? 0 : w_slot + 1;
      x_slot = x_slot == SX - 1 ? 0 : x_slot + 1;
    }
    int lo, hi, n0;
    locate(t, sc, lo, hi, n0);
    const int tiles = t - t0 + 1;
#pragma unroll
    for (int r0 = 0; r0 < MF * NF; r0 += SUMS) {
#pragma unroll
      for (int q = 0; q < SUMS; ++q) sums_of(wave, q, tiles)[lane] = acc[(r0 + q) / NF][(r0 + q) % NF];
      asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
      constexpr int MINE = (SUMS + KW - 1) / KW;
      f32x4 total[MINE];
#pragma unroll
      for (int i = 0; i < MINE; ++i) {
        const int q = i * KW + wave;
        total[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        if (q >= SUMS) continue;
#pragma unroll
        for (int v = 0; v < KW; ++v) total[i] += sums_of(v, q, tiles)[lane];
      }
      // (the sums have been read: the slots may be written again)
      asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
#pragma unroll
      for (int i = 0; i < MINE; ++i) {
        const int r = r0 + i * KW + wave;
        if (r >= r0 + SUMS) continue;
        // lane: row `row` of W's sub-tile, rows 4j .. 4j + 3 of X's
        const int64_t m0 = static_cast<int64_t>(lo) + 16 * (r / NF) + 4 * j;
        const int64_t c = static_cast<int64_t>(n0) + (GATED ? (r % NF) * 8 + (row & 7) : (r % NF) * 16 + row);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float v = total[i][k];
          if constexpr (GATED) {
            const float up = __shfl_xor(v, 8);
            v = v * sigmoid(v) * up;
          }
          if (m0 + k >= hi || c >= a.N || (GATED && row >= 8)) continue;
          const int64_t at = (m0 + k) * a.N + c;
          if (a.y_bf16)
            static_cast<uint16_t*>(a.y)[at] = static_cast<uint16_t>(pack_bf16(v, 0.0f));
          else
            static_cast<float*>(a.y)[at] = v;
        }
      }
    }
  }
}

template <bool CODES, bool GATED, bool GROUPED, int I>
hipError_t launch_shape(const Fp4Args& a, int shape, hipStream_t s) {
  constexpr Fp4Shape t = kFp4Shapes[CODES][I];
  if (shape == I) {
    const int64_t tiles = fp4_tiles(a.M, a.N, a.G, a.offsets != nullptr, a.gated, t);
    const int cus = device_cus();
    const int64_t most = cus > 0 ? cus : 256;
    hipLaunchKernelGGL((fp4_gemm_kernel<CODES, GATED, GROUPED, t.xr, t.nf, t.kw, t.sw, t.sx, t.ku>),
                       dim3(static_cast<unsigned>(tiles < most ? tiles : most)), dim3(t.kw * 64), 0, s, a);
    return hipGetLastError();
  }
  if constexpr (I + 1 < kFp4ShapeCount) return launch_shape<CODES, GATED, GROUPED, I + 1>(a, shape, s);
  return hipErrorInvalidValue;
}

int shape_of(const Fp4Args& a) {
  const int cus = device_cus();
  return choose_fp4_shape(a.M, a.N, a.G, a.offsets != nullptr, a.gated, a.sx != nullptr, cus > 0 ? cus : 256);
}

}  // namespace

hipError_t launch_fp4_quant(const void* w, bool bf16, int64_t N, int64_t K, int64_t ld, uint8_t* q, uint8_t* scales,
                            hipStream_t s) {
  const int64_t octets = N * (K / 8);
  const dim3 grid(static_cast<unsigned>((octets + 255) / 256));
  if (bf16)
    hipLaunchKernelGGL(fp4_quant_kernel<true>, grid, dim3(256), 0, s, w, octets, K / 8, ld, q, scales);
  else
    hipLaunchKernelGGL(fp4_quant_kernel<false>, grid, dim3(256), 0, s, w, octets, K / 8, ld, q, scales);
  return hipGetLastError();
}

hipError_t launch_fp4_gemm(const Fp4Args& a, hipStream_t s) {
  const int shape = shape_of(a);
  auto form = [&](auto codes, auto gated) {
    constexpr bool CODES = decltype(codes)::value, GATED = decltype(gated)::value;
    return a.offsets ? launch_shape<CODES, GATED, true, 0>(a, shape, s)
                     : launch_shape<CODES, GATED, false, 0>(a, shape, s);
  };
  if (a.sx) return a.gated ? form(std::true_type{}, std::true_type{}) : form(std::true_type{}, std::false_type{});
  return a.gated ? form(std::false_type{}, std::true_type{}) : form(std::false_type{}, std::false_type{});
}

}  // namespace fp8fg
