// The workgroup shapes of the products with 4-bit weights (fp4.hip) and the choice among
// them.  Plain host C++, so that the choice can be looked at without a GPU.
#pragma once
#include <cstdint>

namespace fp8fg {

// Rows of X and sub-tiles of 16 rows of W in a tile, wavefronts that share K, stages of the rings of W and of
// X, values of K in a stage, and the time of a tile per 128 values of K (us; with the compute units busy).
struct Fp4Shape {
  int xr, nf, kw, sw, sx, ku;
  float per_block;
};
// Of X in bf16, and in E4M3 codes, whose smaller stages leave 32 rows of X twice as long ones or twice the
// wavefronts (7168 x 18432, 32 rows: 30.6 -> 27.8 us; 48 rows: 39 -> 34).  Up to 16 rows both types
// take the same times.
constexpr int kFp4ShapeCount = 12;
constexpr Fp4Shape kFp4Shapes[2][kFp4ShapeCount] = {
    {{2, 1, 8, 4, 4, 256, 0.054f},
     {2, 2, 8, 3, 2, 256, 0.085f},
     {2, 3, 4, 4, 4, 256, 0.112f},
     {8, 1, 8, 4, 2, 256, 0.055f},
     {8, 2, 8, 2, 2, 256, 0.102f},
     {8, 3, 4, 3, 3, 256, 0.120f},
     {16, 1, 8, 4, 3, 128, 0.100f},
     {16, 2, 4, 3, 3, 256, 0.130f},
     {16, 3, 4, 3, 2, 256, 0.175f},
     {16, 4, 4, 2, 2, 256, 0.210f},
     {32, 2, 4, 4, 2, 128, 0.175f},
     {32, 4, 4, 3, 2, 128, 0.270f}},
    {{2, 1, 8, 4, 4, 256, 0.054f},
     {2, 2, 8, 3, 2, 256, 0.085f},
     {2, 3, 4, 4, 4, 256, 0.112f},
     {8, 1, 8, 4, 2, 256, 0.055f},
     {8, 2, 8, 2, 2, 256, 0.102f},
     {8, 3, 4, 3, 3, 256, 0.120f},
     {16, 1, 8, 4, 3, 128, 0.100f},
     {16, 2, 4, 3, 3, 256, 0.130f},
     {16, 3, 4, 3, 2, 256, 0.175f},
     {16, 4, 4, 2, 2, 256, 0.210f},
     {32, 2, 4, 4, 2, 256, 0.158f},
     {32, 4, 8, 2, 2, 128, 0.245f}}};

// Tiles of `rows` rows that cover rows lo .. hi - 1, lo <= hi.  (Unsigned: hi - lo may be up to 2^31 - 1.)
constexpr int fp4_row_tiles(int lo, int hi, int rows) {
  return static_cast<int>((static_cast<uint32_t>(hi) - static_cast<uint32_t>(lo) + static_cast<uint32_t>(rows - 1)) /
                          static_cast<uint32_t>(rows));
}

// Tiles of a launch; over segments an upper bound.
inline int64_t fp4_tiles(int64_t M, int64_t N, int64_t G, bool grouped, bool gated, const Fp4Shape& s) {
  const int64_t cols = (gated ? 8 : 16) * s.nf;
  const int64_t rows = grouped ? M / s.xr + (G < M ? G : M) : (M + s.xr - 1) / s.xr;
  return rows * ((N + cols - 1) / cols);
}

// The shape of the least estimated time: rounds of the compute units times the time of a tile (which has
// the same number of blocks in every shape).  Over segments the fuller half decides: a quarter more rows than
// the mean and one, but two rows where most tokens' experts differ.
// Measured at 1 to 64 rows, 1024 to 36864 columns and 2048 to 18432 of K.
inline int choose_fp4_shape(int64_t M, int64_t N, int64_t G, bool grouped, bool gated, bool codes, int64_t cus) {
  const int64_t groups = grouped ? (G < M ? G : M) : 1;
  const int64_t mean = (M + groups - 1) / groups;
  const int64_t rows = !grouped ? M : 2 * M <= G ? 2 : (5 * mean + 3) / 4 + 1;
  int best = 0;
  double least = 0;
  for (int i = 0; i < kFp4ShapeCount; ++i) {
    const Fp4Shape& s = kFp4Shapes[codes][i];
    const int64_t cols = (gated ? 8 : 16) * s.nf;
    const int64_t tiles = groups * ((rows + s.xr - 1) / s.xr) * ((N + cols - 1) / cols);
    const double time = static_cast<double>((tiles + cus - 1) / cus) * s.per_block;
    if (i == 0 || time < least) {
      least = time;
      best = i;
    }
  }
  return best;
}

}  // namespace fp8fg
