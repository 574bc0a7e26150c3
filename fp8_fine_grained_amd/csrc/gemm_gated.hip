// The gated pair of block-scaled FP8 products of a feed-forward block,
//     g = deq(A) deq(Wg)^T,  u = deq(A) deq(Wu)^T,  h = g * sigmoid(g) * u,
// in one kernel: the gate and up values stay in the accumulators, and only h
// (bf16, fp32 or already 1x128-quantised) and, for training, the values its
// gradient reads leave the chip.
#include "gated_shape.h"
#include "gemm_fp8_tile.h"
#include "lanes.h"

namespace fp8fg {
namespace {

FParams gated_params(const GemmArgs& g) {
  FParams p{};
  p.a = g.a; p.sa = g.sa; p.b = g.b; p.sb = g.sb; p.y = g.y; p.offsets = g.offsets; p.rows = g.row_index;
  p.M = g.M; p.N = g.N; p.K = g.K; p.G = g.G; p.T = g.T;
  p.KB = static_cast<int>(g.K / 128);
  p.ys = g.y_scales;
  p.gu = g.gu;
  p.gu_bf16 = g.gu_bf16;
  p.pow2 = g.pow2;
  return p;
}

int64_t row_tiles(const GemmArgs& g, int BM) { return gated_row_tiles(g.M, g.G, g.offsets != nullptr, BM); }

template <int CFG, bool EXACT, bool SCALED, bool GROUPED>
hipError_t launch_tiles(const GemmArgs& g, hipStream_t s) {
  using C = Cfg<CFG>;
  const int64_t MT = row_tiles(g, C::BM);
  FParams p = gated_params(g);
  p.MT = static_cast<int>(MT);
  p.NT = static_cast<int>(g.N / C::BN);
  p.T_full = static_cast<int>(MT * p.NT);
  p.split = 1;
  const dim3 grid(static_cast<unsigned>(p.T_full)), block(C::WM * C::WN * 64);
  auto go = [&](auto bf16, auto quantised) {
    hipLaunchKernelGGL((gemm_fp8_block_kernel<C::BM, C::BN, C::WM, C::WN, C::ST, EXACT, false, decltype(bf16)::value,
                                              GROUPED, GROUPED, SCALED, decltype(quantised)::value ? 3 : 0, true>),
                       grid, block, 0, s, p);
  };
  if (g.y_scales)
    go(std::false_type{}, std::true_type{});
  else if (g.y_bf16)
    go(std::true_type{}, std::false_type{});
  else
    go(std::false_type{}, std::false_type{});
  return hipGetLastError();
}

// ---------------------------------------------------------------- few tiles
// When the 256-wide tiles would leave most compute units idle (one token, small
// batches, narrow pairs), a workgroup takes a small output tile and splits K
// over its wavefronts, so that many more units stream the weights:
//  * KW wavefronts take a part of K each, and all the tile's MF x NF sub-tiles of
//    16 tokens by 8 output columns.  One MFMA operand carries the 8
//    gate rows and the 8 up rows of those columns, so g and u of an output end
//    up 32 lanes apart in one wavefront.
//  * Every wavefront moves its own operands, a K block at a time, into its own
//    ring of S stages in LDS, and waits for its own loads only: there is no
//    barrier in the K loop, and KW x S blocks are in flight per workgroup.
//    (Loading straight into the MFMA layout needs no LDS, but there 16
//    consecutive lanes read 16 bytes each of 16 rows; the vector cache serves
//    one line at a time and such loads reached 11 bytes a clock and compute
//    unit: 30 us for 128 tokens, 2048 x 7168, where the ring takes 17.)
//  * The KW partial sums meet in LDS and are added in the order of K: the result
//    does not depend on timing.
enum { kFp8 = 0, kExact = 1, kScaled = 2 };

// Expert and rows [lo, hi) of row tile t (BM rows each) of the grouped problem,
// found by the wavefront together; e < 0: no such tile.
__device__ __forceinline__ void segment_tile(const FParams& p, int t, int BM, int& e, int64_t& lo, int64_t& hi) {
  const int lane = threadIdx.x & 63;
  int before = 0;
  e = -1;
  for (int64_t base = 0; base < p.G; base += 64) {
    const int64_t g = base + lane;
    int64_t l = 0, h = 0;
    if (g < p.G) {
      l = p.offsets[g];
      h = p.offsets[g + 1];
      l = l < 0 ? 0 : (l > p.M ? p.M : l);
      h = h < l ? l : (h > p.M ? p.M : h);
    }
    const int cnt = static_cast<int>((h - l + BM - 1) / BM);
    int incl = cnt;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_up(incl, d);
      if (lane >= d) incl += o;
    }
    const int excl = before + incl - cnt;
    const unsigned long long who = __ballot(cnt > 0 && t >= excl && t < excl + cnt);
    if (who) {
      const int src = __ffsll(who) - 1;
      auto of = [&](int v) { return __builtin_amdgcn_readfirstlane(__shfl(v, src)); };
      e = static_cast<int>(base) + src;
      const int64_t last = of(static_cast<int>(h));
      lo = of(static_cast<int>(l)) + static_cast<int64_t>(t - of(excl)) * BM;
      hi = lo + BM < last ? lo + BM : last;
      return;
    }
    before += __shfl(incl, 63);
  }
}

// A8: 8-row loads of tokens (MF = A8 / 2 sub-tiles, rounded up).
template <int MODE, bool BF16OUT, int A8, int NF, int KW, int S, bool GROUPED>
__global__ void __launch_bounds__(KW * 64) gated_split_kernel(FParams p) {
  constexpr int MF = (A8 + 1) / 2;
  constexpr int FR = MF * NF;               // sub-tiles of a wavefront
  constexpr int R = FR < 8 ? FR : 8;        // sub-tiles per reduction round
  constexpr int COLS = 8 * NF;              // output columns of the workgroup
  constexpr int BM = 8 * A8;
  constexpr int SCALES = 16 * MF + 2 <= 64 ? 1 : 2;          // scale loads per stage
  constexpr int STAGE = (NF + MF) * 2048 + SCALES * 256;     // weights, tokens, scales
  constexpr int LOADS = 2 * NF + A8 + SCALES;                // loads per stage
  constexpr int RED = KW * R * 1024;
  constexpr int RING = KW * S * STAGE;
  static_assert(FR % R == 0 && 128 % COLS == 0, "whole rounds; columns inside one weight block");
  static_assert((S - 1) * LOADS < 64, "the wait counter");
  __shared__ __attribute__((aligned(1024))) uint8_t lds[RING > RED ? RING : RED];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int row = lane & 15, j = lane >> 4;
  const int64_t I = p.N / 2;

  int64_t lo = static_cast<int64_t>(blockIdx.y) * BM, hi = lo + BM < p.M ? lo + BM : p.M;
  const uint8_t* w = p.b;
  const float* sw = p.sb;
  if constexpr (GROUPED) {
    int e;
    segment_tile(p, blockIdx.y, BM, e, lo, hi);  // every wavefront finds the same
    if (e < 0) return;
    w += static_cast<int64_t>(e) * p.N * p.K;
    sw += static_cast<int64_t>(e) * (p.N / 128) * p.KB;
  }
  const int64_t c0 = static_cast<int64_t>(blockIdx.x) * COLS;  // the workgroup's first output column
  // Row of A of tile row r: rows past the end repeat the last one and are not stored.
  auto a_row = [&](int r) -> int64_t {
    int64_t m = lo + r;
    m = m < hi ? m : hi - 1;
    if (GROUPED && p.rows) {
      m = p.rows[m];
      m = m < 0 ? 0 : (m >= p.T ? p.T - 1 : m);
    }
    return m;
  };
  // An 8-row load: lane L fills the 16 bytes at L of 1 KB, physical chunk L % 8 of
  // row L / 8, with logical chunk (L % 8) ^ (L / 8) (the layout frag() reads).
  const int lrow = lane >> 3, lchunk = ((lane & 7) ^ lrow) * 16;
  const uint32_t w_off = static_cast<uint32_t>(lrow * static_cast<int>(p.K) + lchunk);
  const uint8_t* w_base = uniform_ptr(w + c0 * p.K);
  // token rows: offsets from the tile's first row (below BM * K < 2^32), or from A
  // when the rows are indexed (below T * K < 2^32)
  const int64_t a0 = GROUPED && p.rows ? 0 : lo;
  const uint8_t* a_base = uniform_ptr(p.a + a0 * p.K);
  uint32_t a_off[A8];
#pragma unroll
  for (int i = 0; i < A8; ++i) a_off[i] = static_cast<uint32_t>((a_row(8 * i + lrow) - a0) * p.K + lchunk);
  // Scale loads: one value per token row, then the gate and the up block's.
  const float* s_ptr[SCALES];
#pragma unroll
  for (int i = 0; i < SCALES; ++i) {
    const int r = 64 * i + lane;
    s_ptr[i] = r < 16 * MF ? p.sa + a_row(r) * p.KB : sw + (c0 / 128 + (r == 16 * MF ? 0 : I / 128)) * p.KB;
  }
  uint8_t* ring = lds + wave * (S * STAGE);
  const uint32_t ring_at = __builtin_amdgcn_readfirstlane(lds_addr(ring));

  const int begin = static_cast<int>(static_cast<int64_t>(wave) * p.KB / KW);
  const int n = static_cast<int>(static_cast<int64_t>(wave + 1) * p.KB / KW) - begin;  // K blocks of this wavefront
  auto issue = [&](int i, int slot) {
    const int64_t kof = static_cast<int64_t>(begin + i) * 128;
    const uint32_t at = ring_at + static_cast<uint32_t>(slot) * STAGE;
#pragma unroll
    for (int f = 0; f < NF; ++f) {
      dma16(w_base + static_cast<int64_t>(f) * 8 * p.K + kof, w_off, at + f * 2048);
      dma16(w_base + (I + f * 8) * p.K + kof, w_off, at + f * 2048 + 1024);
    }
#pragma unroll
    for (int f = 0; f < A8; ++f) dma16(a_base + kof, a_off[f], at + NF * 2048 + f * 1024);
#pragma unroll
    for (int f = 0; f < SCALES; ++f) dma4(s_ptr[f] + begin + i, at + (NF + MF) * 2048 + f * 256);
  };

  v4f acc[NF][MF];
#pragma unroll
  for (int f = 0; f < NF; ++f)
#pragma unroll
    for (int m = 0; m < MF; ++m) acc[f][m] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  auto multiply = [&](int slot) {
    const uint8_t* st = ring + slot * STAGE;
    const float* sc = reinterpret_cast<const float*>(st + (NF + MF) * 2048);
    v8i wf[NF], af[MF];
    float sa[MF];
#pragma unroll
    for (int f = 0; f < NF; ++f) wf[f] = frag(st + f * 2048, 0, lane);
#pragma unroll
    for (int m = 0; m < MF; ++m) {
      af[m] = frag(st + (NF + m) * 2048, 0, lane);
      sa[m] = sc[m * 16 + row];
    }
    // Weight scale: by the half the lane's result rows lie in (lanes 0-31 hold gate
    // rows), or, as an operand of the scaled MFMA, by the half its weight row lies in.
    const float swv = sc[16 * MF + ((MODE == kScaled ? row >= 8 : lane >= 32) ? 1 : 0)];
    WideFrag wide[MODE == kExact ? MF : 1];
    if constexpr (MODE == kExact) {
#pragma unroll
      for (int m = 0; m < MF; ++m) wide[m] = widen(af[m]);
    }
#pragma unroll
    for (int f = 0; f < NF; ++f) {
      WideFrag ww;
      if constexpr (MODE == kExact) ww = widen(wf[f]);
#pragma unroll
      for (int m = 0; m < MF; ++m) {
        if constexpr (MODE == kScaled) {
          const int ew = static_cast<int>((__float_as_uint(swv) >> 23) & 0xFFu);
          const int ea = static_cast<int>((__float_as_uint(sa[m]) >> 23) & 0xFFu);
          acc[f][m] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wf[f], af[m], acc[f][m], 0, 0, 0, ew, 0, ea);
        } else {
          v4f P = {0.0f, 0.0f, 0.0f, 0.0f};
          if constexpr (MODE == kExact) {
#pragma unroll
            for (int q = 0; q < 4; ++q) P = __builtin_amdgcn_mfma_f32_16x16x32_f16(ww.q[q], wide[m].q[q], P, 0, 0, 0);
          } else {
            P = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wf[f], af[m], P, 0, 0, 0, 0, 0, 0);
          }
          const float k = sa[m] * swv;
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[f][m][r] = fmaf(P[r], k, acc[f][m][r]);
        }
      }
    }
  };

#pragma unroll
  for (int i = 0; i < S - 1; ++i)
    if (i < n) issue(i, i);
  int slot = 0;
  for (int i = 0; i < n; ++i) {
    if (i + S - 1 < n) {
      // the slot read in the previous iteration: its reads have returned
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      issue(i + S - 1, slot == 0 ? S - 1 : slot - 1);
      asm volatile("s_waitcnt vmcnt(%0)" ::"i"((S - 1) * LOADS) : "memory");
    } else {
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    }
    multiply(slot);
    slot = slot == S - 1 ? 0 : slot + 1;
  }
  __syncthreads();  // every wavefront is done with its ring (and has no load in flight)

  // ---- join the KW partial sums, R sub-tiles at a time
  v4f(*red)[R][64] = reinterpret_cast<v4f(*)[R][64]>(lds);
  auto store = [](void* to, bool bf16, int64_t at, const v4f& v) {
    if (bf16)
      *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(to) + at) =
          u32x2{bf16x2_rne(v[0], v[1]), bf16x2_rne(v[2], v[3])};
    else
      *reinterpret_cast<v4f*>(static_cast<float*>(to) + at) = v;
  };
#pragma unroll
  for (int r0 = 0; r0 < FR; r0 += R) {
    if (r0 > 0) __syncthreads();
#pragma unroll
    for (int r = 0; r < R; ++r) red[wave][r][lane] = acc[(r0 + r) / MF][(r0 + r) % MF];
    __syncthreads();
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (r % KW != wave) continue;
      const int f = (r0 + r) / MF, mi = (r0 + r) % MF;
      v4f v = red[0][r][lane];
#pragma unroll
      for (int k = 1; k < KW; ++k) v += red[k][r][lane];
      // lanes 0-31: g of token `row`, columns 4j .. 4j+3; lanes 32-63: u of columns 4(j-2) ..
      const int64_t m = lo + mi * 16 + row;
      const int64_t c = c0 + f * 8 + (j & 1) * 4;
      if (p.gu && m < hi) {
        const int64_t at = m * p.N + (j >> 1) * I + c;
        store(p.gu, BF16OUT || p.gu_bf16, at, v);
      }
      v4f h;
#pragma unroll
      for (int i = 0; i < 4; ++i) h[i] = gate_product<MODE == kExact>(v[i], __shfl_xor(v[i], 32));
      if (lane < 32 && m < hi) {
        store(p.y, BF16OUT, m * I + c, h);
      }
    }
  }
}

template <int MODE, int A8, int NF, int KW, int S>
hipError_t launch_split(const GemmArgs& g, hipStream_t s) {
  const FParams p = gated_params(g);
  const dim3 grid(static_cast<unsigned>(g.N / 2 / (8 * NF)), static_cast<unsigned>(row_tiles(g, 8 * A8)));
  auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, dim3(KW * 64), 0, s, p); };
  if (g.offsets)
    g.y_bf16 ? go(gated_split_kernel<MODE, true, A8, NF, KW, S, true>)
             : go(gated_split_kernel<MODE, false, A8, NF, KW, S, true>);
  else
    g.y_bf16 ? go(gated_split_kernel<MODE, true, A8, NF, KW, S, false>)
             : go(gated_split_kernel<MODE, false, A8, NF, KW, S, false>);
  return hipGetLastError();
}

// The 1x128 quantisation of h [M, I] (fp32) that the small tiles left in the
// workspace: 16 lanes per group, by the rule that the tiles' own epilogue follows.
__global__ void __launch_bounds__(256) gated_quant_kernel(const float* __restrict__ h, int64_t groups, bool pow2,
                                                          uint8_t* __restrict__ q, float* __restrict__ scales) {
  using O = Octet<false>;
  const int part = threadIdx.x & 15;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * 16 + (threadIdx.x >> 4);
  if (t >= groups) return;  // 16 whole lanes; only those exchange below
  float v[8], s, inv;
  O::widen(O::load(reinterpret_cast<const char*>(h + t * 128), part), v);
  group_scale(pow2, group_amax(v), s, inv);
  O::store_codes(q + t * 128, part, v, inv);
  if (part == 0) scales[t] = s;
}

template <int MODE>
hipError_t launch_mode(const GemmArgs& g, int shape, hipStream_t s) {
  switch (shape) {
    case 0: return launch_split<MODE, 2, 1, 8, 4>(g, s);
    case 1: return launch_split<MODE, 2, 2, 8, 3>(g, s);
    case 2: return launch_split<MODE, 2, 4, 4, 3>(g, s);
    case 3: return launch_split<MODE, 4, 2, 8, 2>(g, s);
    case 4: return launch_split<MODE, 4, 4, 4, 3>(g, s);
    case 5: return launch_split<MODE, 8, 4, 4, 2>(g, s);
    case kTile128:
      return g.offsets ? launch_tiles<1, MODE == kExact, MODE == kScaled, true>(g, s)
                       : launch_tiles<1, MODE == kExact, MODE == kScaled, false>(g, s);
    default:
      if constexpr (MODE == kExact)
        return hipErrorInvalidValue;  // not chosen: its fp16 fragments need the registers
      else
        // (scaled: four wavefronts of 128 x 128, 888 -> 838 us at 4096 x 18432 x 7168)
        return launch_tiles<MODE == kScaled ? 3 : 0, false, MODE == kScaled, false>(g, s);
  }
}

int choose_shape(const GemmArgs& g, bool quantised, bool tiles_only) {
  GatedProblem p{};
  p.M = g.M; p.I = g.N / 2; p.K = g.K; p.G = g.G;
  p.grouped = g.offsets != nullptr; p.exact = g.exact; p.quantised = quantised; p.tiles_only = tiles_only;
  const int found = device_cus();
  return choose_gated_shape(p, found > 0 ? found : 256);
}

hipError_t launch_shape(const GemmArgs& g, int shape, hipStream_t s) {
  if (g.exact) return launch_mode<kExact>(g, shape, s);
  return g.scaled ? launch_mode<kScaled>(g, shape, s) : launch_mode<kFp8>(g, shape, s);
}

}  // namespace

bool gated_quant_takes_workspace(const GemmArgs& g) { return choose_shape(g, true, false) < kTile128; }

hipError_t launch_gated_gemm(const GemmArgs& g, float* workspace, hipStream_t s) {
  if (!g.y_scales) return launch_shape(g, choose_shape(g, false, false), s);
  const int shape = choose_shape(g, true, workspace == nullptr);
  if (shape >= kTile128) return launch_shape(g, shape, s);
  // Small tiles do not hold whole 1x128 groups: h goes through the workspace in
  // fp32 and is quantised by a second launch.
  GemmArgs f = g;
  f.y = workspace;
  f.y_scales = nullptr;
  f.y_bf16 = false;
  f.gu_bf16 = true;
  const hipError_t e = launch_shape(f, shape, s);
  if (e != hipSuccess) return e;
  const int64_t groups = g.M * (g.N / 256);
  hipLaunchKernelGGL(gated_quant_kernel, dim3(static_cast<unsigned>((groups + 15) / 16)), dim3(256), 0, s, workspace,
                     groups, g.pow2, static_cast<uint8_t*>(g.y), g.y_scales);
  return hipGetLastError();
}

}  // namespace fp8fg
