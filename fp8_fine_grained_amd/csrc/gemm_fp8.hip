// Launches of the throughput kernel (gemm_fp8_tile.h) for the dense projection
// and the MoE grouped GEMM: tile choice, K split of fp32 outputs.
#include <atomic>

#include "gemm_fp8_tile.h"

namespace fp8fg {
namespace {

// Zeroes the fp32 output of the K-split tiles (tiles T_full .. T_full +
// gridDim.x - 1 of the dense order) before their parts add into it.  A kernel,
// not a memset, so the sequence can be captured in a graph.
template <int BM, int BN>
__global__ void __launch_bounds__(256) zero_split_tiles_kernel(float* __restrict__ y, int64_t M, int64_t N, int MT,
                                                               int NT, int T_full) {
  int mt, nt;
  dense_tile_coords(T_full + static_cast<int>(blockIdx.x), MT, NT, mt, nt);
  const int64_t r0 = static_cast<int64_t>(mt) * BM, c0 = static_cast<int64_t>(nt) * BN;
  for (int idx = threadIdx.x; idx < BM * (BN / 4); idx += 256) {
    const int r = idx / (BN / 4), c = idx % (BN / 4);
    if (r0 + r < M) *reinterpret_cast<v4f*>(y + (r0 + r) * N + c0 + 4 * c) = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  }
}

}  // namespace

// Compute units of the current device, queried once per device.
int device_cus() {
  static std::atomic<int> cache[64];
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return 0;
  int v = cache[dev].load(std::memory_order_relaxed);
  if (v == 0) {
    if (hipDeviceGetAttribute(&v, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess) return 0;
    cache[dev].store(v, std::memory_order_relaxed);
  }
  return v;
}

namespace {

template <int CFG, bool EXACT, bool ROWS, bool BF16OUT, bool GROUPED, bool GATHER, bool SCALED, int QOUT = 0>
hipError_t launch_cfg(const GemmArgs& g, hipStream_t s) {
  using C = Cfg<CFG>;
  const int64_t MT = GROUPED ? g.M / C::BM + g.G : (g.M + C::BM - 1) / C::BM;
  FParams p{g.a, g.sa, g.b, g.sb, g.y, g.offsets, g.row_index, g.M, g.N, g.K, g.G, g.T,
            static_cast<int>(g.K / 128), static_cast<int>(MT), static_cast<int>(g.N / C::BN), g.y_scales};
  const int64_t T = MT * p.NT;
  p.T_full = static_cast<int>(T);
  p.split = 1;
  if constexpr (!GROUPED && !BF16OUT && QOUT == 0) {
    // fp32 output filling at least one round of the CUs: the tiles of the
    // partial last round are split along K over the CUs that round would leave
    // idle (the weight-gradient shape 7168 x 7168 has 1568 tiles of 128 x 256,
    // 6.125 rounds of 256 CUs; its last 32 tiles run as 8 parts each).  The
    // parts add in whatever order they finish, so those tiles' last bits can
    // differ between runs.  Smaller problems are not split, which keeps their
    // results equal bit for bit to the same sums computed by other tile shapes
    // (the grouped and the output-quantising kernels).
    const int ncu = device_cus();
    if (ncu > 0 && T >= ncu) {
      const int64_t full = (T / ncu) * ncu, rest = T - full;
      int64_t parts = rest > 0 ? ncu / rest : 1;
      parts = parts < p.KB ? parts : p.KB;
      if (parts >= 2) {
        p.T_full = static_cast<int>(full);
        p.split = static_cast<int>(parts);
        hipLaunchKernelGGL((zero_split_tiles_kernel<C::BM, C::BN>), dim3(static_cast<unsigned>(rest)), dim3(256), 0,
                           s, static_cast<float*>(g.y), g.M, g.N, p.MT, p.NT, p.T_full);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
      }
    }
  }
  const unsigned blocks = static_cast<unsigned>(p.T_full + (T - p.T_full) * p.split);
  hipLaunchKernelGGL(
      (gemm_fp8_block_kernel<C::BM, C::BN, C::WM, C::WN, C::ST, EXACT, ROWS, BF16OUT, GROUPED, GATHER, SCALED,
                             QOUT>),
      dim3(blocks), dim3(C::WM * C::WN * 64), 0, s, p);
  return hipGetLastError();
}

template <int CFG, bool EXACT, bool ROWS, bool GROUPED, bool GATHER = false, bool SCALED = false>
hipError_t launch_out(const GemmArgs& g, hipStream_t s) {
  return g.y_bf16 ? launch_cfg<CFG, EXACT, ROWS, true, GROUPED, GATHER, SCALED>(g, s)
                  : launch_cfg<CFG, EXACT, ROWS, false, GROUPED, GATHER, SCALED>(g, s);
}

}  // namespace

bool fp8_block_kernel_applies(const GemmArgs& g) {
  // (the DMA lane offsets are 32-bit: 256 rows x K bytes must stay below 4 GiB)
  if (g.K >= (int64_t(1) << 24)) return false;
  if (g.N % 256 == 0) return true;
  // 224-wide tiles: dense, 128x128 weight scales, FP8 or scaled accumulation
  return g.N % 224 == 0 && g.offsets == nullptr && !g.exact && !g.row_scales;
}

namespace {

// Width of the 256-row dense tiles: 256 whenever N allows it, else 224.
// Measured on 4096 x 7168 x 7168, 224-wide tiles (512 tiles, exactly two
// rounds of the 256 CUs) run 5-8% slower than 256-wide ones (448 tiles, 1.75
// rounds): the per-block costs (barrier, A fragments, scales) are spread over
// 7/8 of the MFMAs, and the last round of 256-wide tiles runs on a partly idle
// chip at a higher clock.  So 224 serves only N that 256 does not divide.
int dense_tile_width(const GemmArgs& g) { return g.N % 256 == 0 ? 256 : 224; }

}  // namespace

// Block-scaled FP8 accumulation: dense GEMMs use the 256 x 256 tile (least L2
// and LDS traffic per flop), grouped GEMMs the 128-row tile (expert segments of
// ~256 rows then waste less of their last m-tile).  The exact mode (fp16
// operands, twice the fragment registers) uses the 64 x 64 wavefront tile; the
// row-scaled FP8 mode (one more multiply and four row scales per sub-tile) the
// dense 256 x 256 tile.
// The scaled mode (power-of-two scales applied by the matrix cores) takes the
// same tiles as the FP8 mode.
hipError_t launch_grouped_gemm_gather(const GemmArgs& g, hipStream_t s) {
  if (g.scaled) return launch_out<1, false, false, true, true, true>(g, s);
  return g.exact ? launch_out<1, true, false, true, true>(g, s) : launch_out<1, false, false, true, true>(g, s);
}

hipError_t launch_fp8_block_gemm(const GemmArgs& g, bool grouped, hipStream_t s) {
  if (grouped) {
    if (g.scaled) return launch_out<1, false, false, true, false, true>(g, s);
    return g.exact ? launch_out<1, true, false, true>(g, s) : launch_out<1, false, false, true>(g, s);
  }
  if (g.exact)
    return g.row_scales ? launch_out<1, true, true, false>(g, s) : launch_out<1, true, false, false>(g, s);
  // Row-scaled B with FP8 accumulation fits the 256 x 256 tile (244 VGPRs with
  // the four row scales per sub-tile): 10% faster than 128 x 256 on the weight
  // gradient 7168 x 7168 x 16384.  Exact mode keeps 128 x 256 (its fp16
  // fragments need the registers).
  if (g.row_scales) return launch_out<0, false, true, false>(g, s);
  const bool narrow = dense_tile_width(g) == 224;
  // (scaled mode: four wavefronts of 128 x 128 on 256 x 256 tiles, 2.5% faster
  // than eight of 64 x 128 on 4096 x 7168 x 7168: half the fragment reads and
  // half the wavefronts at each barrier)
  if (g.scaled)
    return narrow ? launch_out<2, false, false, false, false, true>(g, s)
                  : launch_out<3, false, false, false, false, true>(g, s);
  return narrow ? launch_out<2, false, false, false>(g, s) : launch_out<0, false, false, false>(g, s);
}

// GEMM whose output leaves 1x128-quantised (256 x 256 dense tiles: a
// wavefront's 128 columns are one group).  FP8 or scaled accumulation.
hipError_t launch_fp8_block_gemm_quant(const GemmArgs& g, bool pow2, hipStream_t s) {
  // (the scaled mode keeps eight wavefronts here: with four, the quantising
  // epilogue needs more than the 512 registers of a wavefront and spills)
  if (g.scaled)
    return pow2 ? launch_cfg<0, false, false, false, false, false, true, 2>(g, s)
                : launch_cfg<0, false, false, false, false, false, true, 1>(g, s);
  return pow2 ? launch_cfg<0, false, false, false, false, false, false, 2>(g, s)
              : launch_cfg<0, false, false, false, false, false, false, 1>(g, s);
}

}  // namespace fp8fg
