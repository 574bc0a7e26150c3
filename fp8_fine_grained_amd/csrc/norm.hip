// Residual addition, root-mean-square norm and 1x128 quantisation in one pass,
// and the norm's gradient.
//
// Forward, per row of H elements (all in fp32 until the stores):
//     z = x + r,  rstd = 1 / sqrt(mean(z^2) + eps),  y = (z * rstd) * w,
//     codes and scales of y per 128 elements by the quantisers' rule;
//     h = z rounded to the input type (the residual stream passed on).
// y is taken from the unrounded z: rounding the residual stream is a property
// of its storage, and the norm need not inherit it.
// Backward, with n = h * rstd and d = dy * w:
//     dx = rstd * (d - n * mean(d * n)) + dh,    dw = sum over rows of dy * n.
//
// Both are bound by HBM: a row is read once and kept in registers between the
// row statistic and the outputs.
#include <type_traits>

#include "launch.h"
#include "lanes.h"

namespace fp8fg {
namespace {

// Four consecutive elements of the norm weight, of its own type, as fp32.
__device__ __forceinline__ f32x4 weight4(const void* w, bool bf16, int64_t i) {
  if (!bf16) return *reinterpret_cast<const f32x4*>(static_cast<const float*>(w) + i);
  const u32x2 u = *reinterpret_cast<const u32x2*>(static_cast<const uint16_t*>(w) + i);
  return f32x4{__uint_as_float(u[0] << 16), __uint_as_float(u[0] & 0xFFFF0000u), __uint_as_float(u[1] << 16),
               __uint_as_float(u[1] & 0xFFFF0000u)};
}
// The weights of a lane's octet of group g.
template <bool BF16>
__device__ __forceinline__ void weight_octet(const void* w, bool w_bf16, int g, int part, float (&f)[8]) {
  const f32x4 lo = weight4(w, w_bf16, g * 128 + Octet<BF16>::col(part, 0));
  const f32x4 hi = weight4(w, w_bf16, g * 128 + Octet<BF16>::col(part, 4));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[i] = lo[i];
    f[4 + i] = hi[i];
  }
}

// ---------------------------------------------------------------- forward
// WPR wavefronts own a row; 16 consecutive lanes own one 128-element group, so
// a step of the WPR wavefronts covers 512 * WPR elements and CH steps the row.
template <bool BF16, int WPR, int CH>
__global__ void __launch_bounds__(WPR > 4 ? WPR * 64 : 256) rmsnorm_quant_kernel(NormArgs a) {
  using O = Octet<BF16>;
  constexpr int ROWS = WPR >= 4 ? 1 : 4 / WPR;  // rows per workgroup
  __shared__ float partial[WPR > 1 ? WPR : 1];
  const int wave = threadIdx.x >> 6;
  const int64_t m = static_cast<int64_t>(blockIdx.x) * ROWS + (ROWS > 1 ? wave / WPR : 0);
  if (ROWS > 1 && m >= a.M) return;  // whole wavefronts, and no barrier below when ROWS > 1
  const int t = threadIdx.x % (WPR * 64);
  const int part = t & 15;
  const int G = static_cast<int>(a.H >> 7);
  const char* x = static_cast<const char*>(a.x) + m * a.ld_x * O::ES;
  const char* r = static_cast<const char*>(a.r) + m * a.ld_r * O::ES;
  float z[CH][8];
  typename O::Raw xr[CH], rr[CH];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int g = c * (WPR * 4) + (t >> 4);
    if (g < G) {
      xr[c] = O::load(x + static_cast<int64_t>(g) * 128 * O::ES, part);
      if (a.r) rr[c] = O::load(r + static_cast<int64_t>(g) * 128 * O::ES, part);
    }
  }
  float ss = 0.0f;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int g = c * (WPR * 4) + (t >> 4);
    if (g < G) {
      O::widen(xr[c], z[c]);
      if (a.r) {
        float v[8];
        O::widen(rr[c], v);
#pragma unroll
        for (int i = 0; i < 8; ++i) z[c][i] += v[i];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(z[c][i], z[c][i], ss);
      if (a.h) O::store(static_cast<char*>(a.h) + (m * a.H + g * 128) * O::ES, part, z[c]);
    }
  }
  ss = sum64(ss);
  if constexpr (WPR > 1) {
    if ((t & 63) == 0) partial[wave] = ss;
    __syncthreads();
    ss = 0.0f;
#pragma unroll
    for (int w = 0; w < WPR; ++w) ss += partial[w];
  }
  const float rstd = 1.0f / sqrtf(ss / static_cast<float>(a.H) + a.eps);
  if (t == 0 && a.rstd) a.rstd[m] = rstd;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int g = c * (WPR * 4) + (t >> 4);
    if (g < G) {
      float w[8];
      weight_octet<BF16>(a.w, a.w_bf16, g, part, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) z[c][i] = z[c][i] * rstd * w[i];
      float s, inv;
      group_scale(a.pow2, group_amax(z[c]), s, inv);
      O::store_codes(a.q + m * a.H + g * 128, part, z[c], inv);
      if (part == 0) a.scales[m * G + g] = s;
      if (a.y) O::store(static_cast<char*>(a.y) + (m * a.H + g * 128) * O::ES, part, z[c]);
    }
  }
}

// ---------------------------------------------------------------- backward
// A workgroup of NW wavefronts holds NW / WPR rows at a time and walks the rows
// with a stride of the grid, adding dy * n into registers; at its end its row
// slots are summed through LDS, in order, into one partial of dw per workgroup,
// and a second kernel sums the partials, in order: dw is the same on every run.
template <bool BF16, int WPR, int CH, int NW>
__global__ void __launch_bounds__(NW * 64) rmsnorm_backward_kernel(NormGradArgs a) {
  using O = Octet<BF16>;
  constexpr int SLOTS = NW / WPR;
  __shared__ float part_sum[2][NW];
  extern __shared__ __attribute__((aligned(16))) float dw_sum[];  // [H], when SLOTS > 1 and dw is asked for
  const int wave = threadIdx.x >> 6;
  const int slot = wave / WPR;
  const int t = threadIdx.x % (WPR * 64);
  const int part = t & 15;
  const int G = static_cast<int>(a.H >> 7);
  float acc[CH][8];
#pragma unroll
  for (int c = 0; c < CH; ++c)
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[c][i] = 0.0f;

  const int64_t stride = static_cast<int64_t>(gridDim.x) * SLOTS;
  int flip = 0;
  // every slot makes the same number of steps, so that the workgroup's barriers agree
  for (int64_t m0 = static_cast<int64_t>(blockIdx.x) * SLOTS; m0 < a.M; m0 += stride) {
    const int64_t m = m0 + slot;
    const bool live = m < a.M;
    float d[CH][8], n[CH][8];
    float dot = 0.0f, rstd = 0.0f;
    typename O::Raw gr[CH];
    if (live) {
      typename O::Raw yr[CH], hr[CH];
      rstd = a.rstd[m];
      const char* dy = static_cast<const char*>(a.dy) + m * a.ld_dy * O::ES;
      const char* h = static_cast<const char*>(a.h) + m * a.ld_h * O::ES;
      const char* dh = static_cast<const char*>(a.dh) + m * a.ld_dh * O::ES;
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int g = c * (WPR * 4) + (t >> 4);
        if (g < G) {
          yr[c] = O::load(dy + static_cast<int64_t>(g) * 128 * O::ES, part);
          hr[c] = O::load(h + static_cast<int64_t>(g) * 128 * O::ES, part);
          if (a.dh) gr[c] = O::load(dh + static_cast<int64_t>(g) * 128 * O::ES, part);
        }
      }
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int g = c * (WPR * 4) + (t >> 4);
        if (g < G) {
          float w[8];
          weight_octet<BF16>(a.w, a.w_bf16, g, part, w);
          O::widen(yr[c], d[c]);
          O::widen(hr[c], n[c]);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            n[c][i] *= rstd;
            acc[c][i] = fmaf(d[c][i], n[c][i], acc[c][i]);
            d[c][i] *= w[i];
            dot = fmaf(d[c][i], n[c][i], dot);
          }
        }
      }
    }
    dot = sum64(dot);
    if constexpr (WPR > 1) {
      // two buffers: a slow wavefront's reads of one row never meet the next row's writes
      if ((t & 63) == 0) part_sum[flip][wave] = dot;
      __syncthreads();
      dot = 0.0f;
#pragma unroll
      for (int w = 0; w < WPR; ++w) dot += part_sum[flip][slot * WPR + w];
      flip ^= 1;
    }
    if (live) {
      const float c0 = dot / static_cast<float>(a.H);
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int g = c * (WPR * 4) + (t >> 4);
        if (g < G) {
          float o[8];
          if (a.dh) O::widen(gr[c], o);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float v = rstd * fmaf(-n[c][i], c0, d[c][i]);
            o[i] = a.dh ? v + o[i] : v;
          }
          O::store(static_cast<char*>(a.dx) + (m * a.H + g * 128) * O::ES, part, o);
        }
      }
    }
  }
  if (!a.partial) return;
  float* out = a.partial + blockIdx.x * a.H;
#pragma unroll 1
  for (int s = 0; s < SLOTS; ++s) {
    if (slot == s) {
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int g = c * (WPR * 4) + (t >> 4);
        if (g < G) {
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const int j = g * 128 + O::col(part, 4 * half);
            f32x4 v = {acc[c][4 * half], acc[c][4 * half + 1], acc[c][4 * half + 2], acc[c][4 * half + 3]};
            if (s > 0) v += *reinterpret_cast<const f32x4*>(dw_sum + j);
            if (s == SLOTS - 1)
              *reinterpret_cast<f32x4*>(out + j) = v;
            else
              *reinterpret_cast<f32x4*>(dw_sum + j) = v;
          }
        }
      }
    }
    if constexpr (SLOTS > 1) __syncthreads();
  }
}

// dw[j] = sum of the P partials of column j.  A workgroup takes 32 columns: 8
// lanes of four columns by 32 strided row sums, added pairwise through LDS.
__global__ void __launch_bounds__(256) rmsnorm_dw_kernel(const float* __restrict__ partial, int P, int64_t H,
                                                         float* __restrict__ dw) {
  __shared__ __attribute__((aligned(16))) f32x4 sums[32][8];
  const int c = threadIdx.x & 7, r = threadIdx.x >> 3;
  const int64_t j = static_cast<int64_t>(blockIdx.x) * 32 + c * 4;
  f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int p = r; p < P; p += 32) v += *reinterpret_cast<const f32x4*>(partial + p * H + j);
  sums[r][c] = v;
#pragma unroll
  for (int n = 16; n >= 1; n >>= 1) {
    __syncthreads();
    if (r < n) sums[r][c] += sums[r + n][c];
  }
  if (r == 0) *reinterpret_cast<f32x4*>(dw + j) = sums[0][c];
}

// Wavefronts per row and steps per row for H: the fewest registers per lane that
// still hold a row (CH octets of 8 elements).
template <typename F>
hipError_t with_shape(int64_t H, F&& f) {
  using std::integral_constant;
#define FP8FG_SHAPE(WPR, CH) f(integral_constant<int, WPR>{}, integral_constant<int, CH>{})
  if (H <= 512) return FP8FG_SHAPE(1, 1);
  if (H <= 1024) return FP8FG_SHAPE(1, 2);
  if (H <= 2048) return FP8FG_SHAPE(4, 1);
  if (H <= 4096) return FP8FG_SHAPE(4, 2);
  if (H <= 8192) return FP8FG_SHAPE(4, 4);
  if (H <= 16384) return FP8FG_SHAPE(16, 2);
  return FP8FG_SHAPE(16, 4);  // H <= 32768
#undef FP8FG_SHAPE
}

// Wavefronts of a backward workgroup, and the most workgroups of one pass.
constexpr int grad_waves(int wpr) { return wpr > 8 ? wpr : 8; }
constexpr int kGradBlocks = 512;

}  // namespace

hipError_t launch_rmsnorm_quant(const NormArgs& a, hipStream_t s) {
  return with_shape(a.H, [&](auto wpr, auto ch) {
    constexpr int WPR = decltype(wpr)::value, CH = decltype(ch)::value;
    constexpr int ROWS = WPR >= 4 ? 1 : 4 / WPR;
    const dim3 grid(static_cast<unsigned>((a.M + ROWS - 1) / ROWS)), block(WPR > 4 ? WPR * 64 : 256);
    if (a.bf16)
      hipLaunchKernelGGL((rmsnorm_quant_kernel<true, WPR, CH>), grid, block, 0, s, a);
    else
      hipLaunchKernelGGL((rmsnorm_quant_kernel<false, WPR, CH>), grid, block, 0, s, a);
    return hipGetLastError();
  });
}

int64_t rmsnorm_backward_partials(int64_t M, int64_t H) {
  int64_t p = 0;
  (void)with_shape(H, [&](auto wpr, auto) {
    constexpr int WPR = decltype(wpr)::value, SLOTS = grad_waves(WPR) / WPR;
    p = (M + SLOTS - 1) / SLOTS;
    return hipSuccess;
  });
  return p < kGradBlocks ? p : kGradBlocks;
}

hipError_t launch_rmsnorm_backward(const NormGradArgs& a, float* dw, hipStream_t s) {
  const int64_t P = rmsnorm_backward_partials(a.M, a.H);
  hipError_t e = hipSuccess;
  if (P > 0) {
    e = with_shape(a.H, [&](auto wpr, auto ch) {
      constexpr int WPR = decltype(wpr)::value, CH = decltype(ch)::value;
      constexpr int NW = grad_waves(WPR);
      const size_t lds = NW > WPR && a.partial ? a.H * sizeof(float) : 0;
      const dim3 grid(static_cast<unsigned>(P)), block(NW * 64);
      if (a.bf16)
        hipLaunchKernelGGL((rmsnorm_backward_kernel<true, WPR, CH, NW>), grid, block, lds, s, a);
      else
        hipLaunchKernelGGL((rmsnorm_backward_kernel<false, WPR, CH, NW>), grid, block, lds, s, a);
      return hipGetLastError();
    });
    if (e != hipSuccess) return e;
  }
  if (dw) {
    hipLaunchKernelGGL(rmsnorm_dw_kernel, dim3(static_cast<unsigned>(a.H / 32)), dim3(256), 0, s, a.partial,
                       static_cast<int>(P), a.H, dw);
    e = hipGetLastError();
  }
  return e;
}

}  // namespace fp8fg
