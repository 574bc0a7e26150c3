// The gated pair of block-scaled FP8 products of a feed-forward block,
//     g = deq(A) deq(Wg)^T,  u = deq(A) deq(Wu)^T,  h = g * sigmoid(g) * u,
// in one kernel: the gate and up values stay in the accumulators, and only h
// (bf16, fp32 or already 1x128-quantised) and, for training, the values its
// gradient reads leave the chip.
#include "gemm_fp8_tile.h"

namespace fp8fg {
namespace {

template <int CFG, bool EXACT, bool SCALED, bool GROUPED>
hipError_t launch_tiles(const GemmArgs& g, hipStream_t s) {
  using C = Cfg<CFG>;
  const int64_t MT = GROUPED ? g.M / C::BM + g.G : (g.M + C::BM - 1) / C::BM;
  FParams p{};
  p.a = g.a; p.sa = g.sa; p.b = g.b; p.sb = g.sb; p.y = g.y; p.offsets = g.offsets; p.rows = g.row_index;
  p.M = g.M; p.N = g.N; p.K = g.K; p.G = g.G; p.T = g.T;
  p.KB = static_cast<int>(g.K / 128);
  p.MT = static_cast<int>(MT);
  p.NT = static_cast<int>(g.N / C::BN);
  p.ys = g.y_scales;
  p.T_full = static_cast<int>(MT * p.NT);
  p.split = 1;
  p.gu = g.gu;
  p.pow2 = g.pow2;
  const dim3 grid(static_cast<unsigned>(p.T_full)), block(C::WM * C::WN * 64);
  auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, block, 0, s, p); };
  if (g.y_scales)
    go(gemm_fp8_block_kernel<C::BM, C::BN, C::WM, C::WN, C::ST, EXACT, false, false, GROUPED, GROUPED, SCALED, 3, true>);
  else if (g.y_bf16)
    go(gemm_fp8_block_kernel<C::BM, C::BN, C::WM, C::WN, C::ST, EXACT, false, true, GROUPED, GROUPED, SCALED, 0, true>);
  else
    go(gemm_fp8_block_kernel<C::BM, C::BN, C::WM, C::WN, C::ST, EXACT, false, false, GROUPED, GROUPED, SCALED, 0, true>);
  return hipGetLastError();
}

}  // namespace

// Tiles as the plain GEMM takes them: 256 x 256 (128 output columns) for dense FP8
// sums, 128 x 256 for the exact sums and for expert segments.
hipError_t launch_gated_gemm(const GemmArgs& g, hipStream_t s) {
  if (g.offsets) {
    if (g.exact) return launch_tiles<1, true, false, true>(g, s);
    return g.scaled ? launch_tiles<1, false, true, true>(g, s) : launch_tiles<1, false, false, true>(g, s);
  }
  if (g.exact) return launch_tiles<1, true, false, false>(g, s);
  return g.scaled ? launch_tiles<0, false, true, false>(g, s) : launch_tiles<0, false, false, false>(g, s);
}

}  // namespace fp8fg
