// The workgroup shapes of the gated products (gemm_gated.hip) and the choice among
// them.  Plain host C++, so that the choice can be looked at without a GPU.
#pragma once
#include <cmath>
#include <cstdint>

namespace fp8fg {

// Output columns and rows of a workgroup, and the time of one round of the compute
// units, start + per_block * K/128 (us).  The last two are the tile kernel's
// 128 x 256 and 256 x 256 tiles, the others the kernel of few tiles.
struct GatedShape {
  int cols, rows;
  float start, per_block;
};
constexpr GatedShape kGatedShapes[] = {{8, 16, 0.8f, 0.073f},  {16, 16, 0.5f, 0.14f}, {32, 16, 0.7f, 0.19f},
                                       {16, 32, 0.9f, 0.155f}, {32, 32, 1.8f, 0.22f}, {32, 64, 2.9f, 0.32f},
                                       {128, 128, 2.1f, 1.0f}, {128, 256, 1.9f, 1.6f}};
constexpr int kTile128 = 6, kTile256 = 7;

struct GatedProblem {
  int64_t M, I, K, G;  // G: experts, when grouped
  bool grouped;
  bool exact;       // fp16 matrix cores
  bool quantised;   // h leaves 1x128-quantised
  bool tiles_only;  // no workspace for the small shapes' h
};

// Row tiles of `rows` rows: exact when dense, an upper bound over segments.
inline int64_t gated_row_tiles(int64_t M, int64_t G, bool grouped, int rows) {
  if (!grouped) return (M + rows - 1) / rows;
  return M / rows + (G < M ? G : M);
}

// The shape of the least estimated time: rounds of the compute units times the
// time of a round.  The times are fitted to every shape's measured times on 256 units
// (FP8 and exact sums; 1 to 8192 rows, up to 256 experts).  On 143 problems the choice
// costs 0.1% over the best shape with dense operands on average (4% at worst), with
// experts 0.1% for FP8 sums and 6% for exact ones (27% at worst: 64 experts of 4 rows).
// Against the tile kernel alone: one token of 2048 x 7168 7.6 instead of 83 us, 64 rows 13 instead of 90;
// against 256-row tiles alone: 777 rows 50 instead of 88.
// Quantised outputs of the small tiles take a second launch, 3 us.
inline int choose_gated_shape(const GatedProblem& p, double cus) {
  const int64_t KB = p.K / 128;
  // Segments that may hold rows, and the rows of one: a quarter more than the mean,
  // since the fuller half of the experts decides.
  const int64_t groups = p.grouped ? (p.G < p.M ? p.G : p.M) : 1;
  const int64_t mean = (p.M + groups - 1) / groups;
  const int64_t rows = p.grouped ? (5 * mean + 3) / 4 : mean;
  int best = kTile128;
  double least = 0;
  for (int i = p.tiles_only ? kTile128 : 0; i <= (p.exact || p.grouped ? kTile128 : kTile256); ++i) {
    const GatedShape& t = kGatedShapes[i];
    // (more rows than the problem has: the time per round would go into repeated rows)
    if (i < kTile128 &&
        ((t.rows > 16 && t.rows >= 2 * mean) || gated_row_tiles(p.M, p.G, p.grouped, t.rows) > 65535))
      continue;
    double per_block = t.per_block;
    if (i == kTile128) per_block *= (p.exact ? 1.55 : 1.0) * (rows <= 64 ? 0.7 : 1.0);
    const double wgs = static_cast<double>(groups * ((rows + t.rows - 1) / t.rows)) * ((p.I + t.cols - 1) / t.cols);
    double time = std::ceil(wgs / cus) * (t.start + KB * per_block);
    if (p.quantised && i < kTile128) time += 3.0;
    if (least == 0 || time < least) {
      least = time;
      best = i;
    }
  }
  return best;
}

}  // namespace fp8fg
