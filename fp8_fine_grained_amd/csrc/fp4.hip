// 4-bit weights: their quantisation (E2M1 codes, one power-of-two scale per 32 elements along
// K) and products of few rows with them, dense or over expert segments, plain or gated:
//     y = x W^T,   or  h = g * sigmoid(g) * u  with g, u the two halves of x W^T.
// Bound by the stream of the weights from HBM (4.25 bits each).
//
// The products run on the bf16 matrix cores: every E2M1 value times its power of two, and
// every E4M3 value, is a bf16 value, so each product is exact and the sums are fp32.
#include "activation.h"
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
constexpr int kRows = 16;  // of X in a workgroup's tile, and of W in a sub-tile
constexpr int kWaves = kFp4Threads / 64;

// Eight E2M1 codes times 2^(e - 127) as bf16, exact.
__device__ __forceinline__ bf16x8 widen_fp4(uint32_t c, float scale) {
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 0);
  const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 1);
  const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 2);
  const bf16x2 e = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 3);
  return bf16x8{a[0], a[1], b[0], b[1], d[0], d[1], e[0], e[1]};
}
// Eight E4M3 codes as bf16, exact.
__device__ __forceinline__ bf16x8 widen_e4m3(u32x2 c) {
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[0], 1.0f, false);
  const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[0], 1.0f, true);
  const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[1], 1.0f, false);
  const bf16x2 e = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[1], 1.0f, true);
  return bf16x8{a[0], a[1], b[0], b[1], d[0], d[1], e[0], e[1]};
}

// Expert and rows [lo, hi) of row tile t of the grouped problem, found by every wavefront
// for itself; false: no such tile.
__device__ __forceinline__ bool segment_of_tile(const Fp4Args& a, int64_t t, int64_t& e, int64_t& lo, int64_t& hi) {
  const int lane = threadIdx.x & 63;
  int64_t before = 0;
  for (int64_t base = 0; base < a.G; base += 64) {
    const int64_t g = base + lane;
    int64_t l = 0, h = 0;
    if (g < a.G) {
      l = a.offsets[g];
      h = a.offsets[g + 1];
      l = l < 0 ? 0 : (l > a.M ? a.M : l);
      h = h < l ? l : (h > a.M ? a.M : h);
    }
    const int64_t cnt = (h - l + kRows - 1) / kRows;
    int64_t incl = cnt;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int64_t o = __shfl_up(incl, d);
      if (lane >= d) incl += o;
    }
    const int64_t excl = before + incl - cnt;
    const uint64_t who = __ballot(cnt > 0 && t >= excl && t < excl + cnt);
    if (who) {
      const int src = __ffsll(static_cast<unsigned long long>(who)) - 1;
      e = base + src;
      const int64_t last = __shfl(h, src);
      lo = __shfl(l, src) + (t - __shfl(excl, src)) * kRows;
      hi = lo + kRows < last ? lo + kRows : last;
      return true;
    }
    before += __shfl(incl, 63);
  }
  return false;
}

// A workgroup takes 16 rows of X by 16 columns of Y; its wavefronts take a part of K each and
// their sums meet in LDS, in the order of K.  A lane holds row lane % 16 of both operands and
// the 32 values 32 (lane / 16) .. + 31 of each 128 along K, eight to an instruction.
template <bool CODES, bool GATED, bool GROUPED>
__global__ void __launch_bounds__(kFp4Threads) fp4_gemm_kernel(Fp4Args a) {
  constexpr int NF = GATED ? 2 : 1;
  __shared__ __attribute__((aligned(16))) f32x4 sums[kWaves][NF][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int row = lane & 15, j = lane >> 4;
  const int64_t tiles = (a.N + 15) / 16;
  const int64_t n0 = (blockIdx.x % tiles) * 16, mt = blockIdx.x / tiles;
  int64_t lo = mt * kRows, hi = lo + kRows < a.M ? lo + kRows : a.M;
  const uint8_t* w = a.w;
  const uint8_t* sw = a.sw;
  const int64_t KB = a.K / 128, wrows = GATED ? 2 * a.N : a.N;
  if constexpr (GROUPED) {
    int64_t e;
    if (!segment_of_tile(a, mt, e, lo, hi)) return;
    w += e * wrows * (a.K / 2);
    sw += e * wrows * (a.K / 32);
  }
  // rows past an edge repeat the last one and are not stored
  int64_t m = lo + row < hi ? lo + row : hi - 1;
  auto x_row = [&](int64_t r) -> int64_t {
    if (!GROUPED || !a.row_index) return r;
    const int64_t v = a.row_index[r];
    return v < 0 ? 0 : (v >= a.T ? a.T - 1 : v);
  };
  m = x_row(m);
  const int64_t n = n0 + row < a.N ? n0 + row : a.N - 1;
  const uint8_t* wp[NF];
  const uint8_t* sp[NF];
#pragma unroll
  for (int f = 0; f < NF; ++f) {
    wp[f] = w + (f * a.N + n) * (a.K / 2) + 16 * j;
    sp[f] = sw + (f * a.N + n) * (a.K / 32) + j;
  }
  const uint8_t* xp = static_cast<const uint8_t*>(a.x) + (m * a.K + 32 * j) * (CODES ? 1 : 2);
  const float* sx[4];
  if constexpr (CODES) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t r = lo + 4 * j + i < hi ? lo + 4 * j + i : hi - 1;
      sx[i] = a.sx + x_row(r) * KB;
    }
  }
  f32x4 acc[NF] = {};
  const int64_t begin = wave * KB / kWaves, end = (wave + 1) * KB / kWaves;
  for (int64_t kb = begin; kb < end; ++kb) {
    bf16x8 xf[4];
    if constexpr (CODES) {
      const u32x4 c0 = *reinterpret_cast<const u32x4*>(xp + kb * 128);
      const u32x4 c1 = *reinterpret_cast<const u32x4*>(xp + kb * 128 + 16);
      xf[0] = widen_e4m3(u32x2{c0[0], c0[1]});
      xf[1] = widen_e4m3(u32x2{c0[2], c0[3]});
      xf[2] = widen_e4m3(u32x2{c1[0], c1[1]});
      xf[3] = widen_e4m3(u32x2{c1[2], c1[3]});
    } else {
#pragma unroll
      for (int s = 0; s < 4; ++s) xf[s] = *reinterpret_cast<const bf16x8*>(xp + kb * 256 + 16 * s);
    }
#pragma unroll
    for (int f = 0; f < NF; ++f) {
      const u32x4 c = *reinterpret_cast<const u32x4*>(wp[f] + kb * 64);
      const float scale = __uint_as_float(static_cast<uint32_t>(sp[f][kb * 4]) << 23);
      f32x4 p = {0.0f, 0.0f, 0.0f, 0.0f};
      if constexpr (!CODES) p = acc[f];
#pragma unroll
      for (int s = 0; s < 4; ++s)
        p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xf[s], widen_fp4(c[s], scale), p, 0, 0, 0);
      if constexpr (CODES) {
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[f][i] = fmaf(p[i], sx[i][kb], acc[f][i]);
      } else {
        acc[f] = p;
      }
    }
  }
#pragma unroll
  for (int f = 0; f < NF; ++f) sums[wave][f][lane] = acc[f];
  __syncthreads();
  if (wave != 0) return;
  f32x4 y[NF];
#pragma unroll
  for (int f = 0; f < NF; ++f) {
    y[f] = sums[0][f][lane];
#pragma unroll
    for (int v = 1; v < kWaves; ++v) y[f] += sums[v][f][lane];
  }
  // lane: column row, rows 4j .. 4j + 3
  if (n0 + row >= a.N) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t r = lo + 4 * j + i;
    if (r >= hi) continue;
    float v = y[0][i];
    if constexpr (GATED) v = v * sigmoid(v) * y[NF - 1][i];
    const int64_t at = r * a.N + n0 + row;
    if (a.y_bf16)
      static_cast<uint16_t*>(a.y)[at] = static_cast<uint16_t>(pack_bf16(v, 0.0f));
    else
      static_cast<float*>(a.y)[at] = v;
  }
}

int64_t row_tiles(const Fp4Args& a) {
  if (!a.offsets) return (a.M + kRows - 1) / kRows;
  return a.M / kRows + (a.G < a.M ? a.G : a.M);
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

int64_t fp4_workgroups(const Fp4Args& a) { return row_tiles(a) * ((a.N + 15) / 16); }

hipError_t launch_fp4_gemm(const Fp4Args& a, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>(fp4_workgroups(a)));
  auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, dim3(kFp4Threads), 0, s, a); };
  auto form = [&](auto codes, auto gated) {
    a.offsets ? go(fp4_gemm_kernel<decltype(codes)::value, decltype(gated)::value, true>)
              : go(fp4_gemm_kernel<decltype(codes)::value, decltype(gated)::value, false>);
  };
  if (a.sx)
    a.gated ? form(std::true_type{}, std::true_type{}) : form(std::true_type{}, std::false_type{});
  else
    a.gated ? form(std::false_type{}, std::true_type{}) : form(std::false_type{}, std::false_type{});
  return hipGetLastError();
}

}  // namespace fp8fg
