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
// Rows of a workgroup whose rows take WPR wavefronts each: four wavefronts at least.
constexpr int norm_rows(int wpr) { return wpr >= 4 ? 1 : 4 / wpr; }

// WPR wavefronts own a row; 16 consecutive lanes own one 128-element group, so
// a step of the WPR wavefronts covers 512 * WPR elements and CH steps the row.
// (Fewer workgroups, each walking over rows with the next row's loads ahead, as the
// backward pass does, were slower: 44 us and more against 37.5 at 4096 x 7168.)
template <bool BF16, int WPR, int CH, bool RES>
__global__ void __launch_bounds__(norm_rows(WPR) * WPR * 64) rmsnorm_quant_kernel(NormArgs a) {
  using O = Octet<BF16>;
  constexpr int ROWS = norm_rows(WPR);
  __shared__ float partial[ROWS * WPR];
  const int slot = ROWS == 1 ? 0 : (threadIdx.x >> 6) / WPR;
  int64_t m = static_cast<int64_t>(blockIdx.x) * ROWS + slot;
  const bool live = m < a.M;
  m = live ? m : a.M - 1;  // past the end: the last row again, not stored
  const int t = threadIdx.x % (WPR * 64);
  const int part = t & 15;
  const int G = static_cast<int>(a.H >> 7);
  typename O::Raw xr[CH], rr[CH];
  const char* x = static_cast<const char*>(a.x) + m * a.ld_x * O::ES;
  const char* r = static_cast<const char*>(a.r) + m * a.ld_r * O::ES;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int g = c * (WPR * 4) + (t >> 4);
    if (g >= G) continue;
    xr[c] = O::load(x + static_cast<int64_t>(g) * 128 * O::ES, part);
    if constexpr (RES) rr[c] = O::load(r + static_cast<int64_t>(g) * 128 * O::ES, part);
  }
  float z[CH][8];
  float ss = 0.0f;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int g = c * (WPR * 4) + (t >> 4);
    if (g >= G) continue;
    O::widen(xr[c], z[c]);
    if constexpr (RES) {
      float v[8];
      O::widen(rr[c], v);
#pragma unroll
      for (int i = 0; i < 8; ++i) z[c][i] += v[i];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(z[c][i], z[c][i], ss);
    // (the next reader of h comes after the GEMMs: it need not stay in the caches;
    // 41.1 -> 39.5 us at 4096 x 7168)
    if (a.h && live) O::template store<true>(static_cast<char*>(a.h) + (m * a.H + g * 128) * O::ES, part, z[c]);
  }
  ss = sum64(ss);
  if constexpr (WPR > 1) {
    if ((t & 63) == 0) partial[threadIdx.x >> 6] = ss;
    __syncthreads();
    ss = 0.0f;
#pragma unroll
    for (int w = 0; w < WPR; ++w) ss += partial[slot * WPR + w];
  }
  if (!live) return;
  // A row of zeros without eps (or one whose squares vanish in fp32) has no direction:
  // zero, not 0 * infinity, here and, through rstd, in the gradient.
  const float mean = ss / static_cast<float>(a.H) + a.eps;
  const float rstd = mean == 0.0f ? 0.0f : 1.0f / sqrtf(mean);
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
// Wavefronts of a workgroup, and the most workgroups of a pass: one per compute
// unit (twice as many write twice the partials: 46.4 -> 54.5 us at 4096 x 7168).
constexpr int kGradWaves = 8;
constexpr int kGradBlocks = 256;

// A workgroup of eight wavefronts holds 8 / WPR rows at a time and walks the rows
// with a stride of the grid, adding dy * n into registers; at its end its row
// slots are summed through LDS, in order, into one partial of dw per workgroup,
// and a second kernel sums the partials, in order: dw is the same on every run.
template <bool BF16, int WPR, int CH, bool DH>
__global__ void __launch_bounds__(kGradWaves * 64) rmsnorm_backward_kernel(NormGradArgs a) {
  using O = Octet<BF16>;
  constexpr int SLOTS = kGradWaves / WPR;
  // Long rows leave no registers for a second row and the weights.
  constexpr bool AHEAD = CH <= (BF16 ? 3 : 2);
  __shared__ float part_sum[2][kGradWaves];
  extern __shared__ __attribute__((aligned(16))) float dw_sum[];  // [H], when SLOTS > 1 and dw is asked for
  const int wave = threadIdx.x >> 6;
  const int slot = wave / WPR;
  const int t = threadIdx.x % (WPR * 64);
  const int part = t & 15;
  const int G = static_cast<int>(a.H >> 7);
  // Octets past the row's end read its last group again and count as zero.
  int col[CH];
  bool in_row[CH];
  float acc[CH][8], w[AHEAD ? CH : 1][8];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int g = c * (WPR * 4) + (t >> 4);
    in_row[c] = g < G;
    col[c] = (g < G ? g : G - 1) * 128;
    if constexpr (AHEAD) weight_octet<BF16>(a.w, a.w_bf16, col[c] >> 7, part, w[c]);
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[c][i] = 0.0f;
  }
  struct Row {
    typename O::Raw y[CH], h[CH], dh[CH];
    float rstd;
  };
  // The row's loads, in a straight line (behind a branch the compiler could not
  // count them and would wait for the next row's before using this one's); rows
  // past the end read the last one.
  auto load = [&](Row& r, int64_t m) {
    m = m < a.M ? m : a.M - 1;
    const char* dy = static_cast<const char*>(a.dy) + m * a.ld_dy * O::ES;
    const char* h = static_cast<const char*>(a.h) + m * a.ld_h * O::ES;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      r.y[c] = O::load(dy + static_cast<int64_t>(col[c]) * O::ES, part);
      r.h[c] = O::load(h + static_cast<int64_t>(col[c]) * O::ES, part);
    }
    if constexpr (DH) {
      const char* dh = static_cast<const char*>(a.dh) + m * a.ld_dh * O::ES;
#pragma unroll
      for (int c = 0; c < CH; ++c) r.dh[c] = O::load(dh + static_cast<int64_t>(col[c]) * O::ES, part);
    }
    r.rstd = a.rstd[m];
  };
  int flip = 0;
  auto process = [&](Row& r, int64_t m) __attribute__((always_inline)) {
    const bool live = m < a.M;
    // dy and n of octet c, and its weights
    auto form = [&](int c, float (&y)[8], float (&n)[8], float (&wc)[8]) __attribute__((always_inline)) {
      O::widen(r.y[c], y);
      O::widen(r.h[c], n);
      if constexpr (!AHEAD) {
        int g = col[c] >> 7;
        asm volatile("" : "+v"(g));  // else the compiler keeps every weight in registers over the rows
        weight_octet<BF16>(a.w, a.w_bf16, g, part, wc);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        n[i] *= r.rstd;
        if constexpr (AHEAD) wc[i] = w[c][i];
      }
    };
    float dot = 0.0f;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      float y[8], n[8], wc[8];
      form(c, y, n, wc);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (live && in_row[c]) acc[c][i] = fmaf(y[i], n[i], acc[c][i]);
        if (in_row[c]) dot = fmaf(y[i] * wc[i], n[i], dot);
      }
      if constexpr (!AHEAD) __builtin_amdgcn_sched_barrier(0);  // octet by octet: fewer live registers
    }
    dot = sum64(dot);
    if constexpr (WPR > 1) {
      // two buffers: a slow wavefront's reads of one row never meet the next row's writes
      if ((t & 63) == 0) part_sum[flip][wave] = dot;
      __syncthreads();
      dot = 0.0f;
#pragma unroll
      for (int v = 0; v < WPR; ++v) dot += part_sum[flip][slot * WPR + v];
      flip ^= 1;
    }
    const float c0 = dot / static_cast<float>(a.H);
    if (live) {
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        if (in_row[c]) {
          float y[8], n[8], wc[8], o[8];
          if constexpr (!AHEAD) {
            // formed again from the loaded values, which this hides from the
            // compiler: kept in fp32 they would spill
#pragma unroll
            for (int k = 0; k < (BF16 ? 1 : 2); ++k) asm volatile("" : "+v"(r.y[c].v[k]), "+v"(r.h[c].v[k]));
          }
          form(c, y, n, wc);
          if constexpr (DH) O::widen(r.dh[c], o);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float v = r.rstd * fmaf(-n[i], c0, y[i] * wc[i]);
            o[i] = DH ? v + o[i] : v;
          }
          O::store(static_cast<char*>(a.dx) + (m * a.H + col[c]) * O::ES, part, o);
        }
        if constexpr (!AHEAD) __builtin_amdgcn_sched_barrier(0);
      }
    }
  };
  // Every slot makes the same number of steps, so that the workgroup's barriers
  // agree.  The next row loads while this one is reduced and written (54.6 -> 46.4
  // us at 4096 x 7168).
  const int64_t stride = static_cast<int64_t>(gridDim.x) * SLOTS;
  int64_t m0 = static_cast<int64_t>(blockIdx.x) * SLOTS;
  if constexpr (AHEAD) {
    Row r0, r1;
    load(r0, m0 + slot);
    for (; m0 < a.M; m0 += 2 * stride) {
      load(r1, m0 + stride + slot);
      process(r0, m0 + slot);
      if (m0 + stride >= a.M) break;
      load(r0, m0 + 2 * stride + slot);
      process(r1, m0 + stride + slot);
    }
  } else {
    for (; m0 < a.M; m0 += stride) {
      Row r;
      load(r, m0 + slot);
      process(r, m0 + slot);
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

// dw[j] = sum of the P <= kGradBlocks partials of column j.  A workgroup takes 32 columns: 8
// lanes of four columns by 32 strided row sums, added pairwise through LDS.
__global__ void __launch_bounds__(256) rmsnorm_dw_kernel(const float* __restrict__ partial, int P, int64_t H,
                                                         float* __restrict__ dw) {
  __shared__ __attribute__((aligned(16))) f32x4 sums[32][8];
  const int c = threadIdx.x & 7, r = threadIdx.x >> 3;
  const int64_t j = static_cast<int64_t>(blockIdx.x) * 32 + c * 4;
  f32x4 part[kGradBlocks / 32];  // loaded together: one latency instead of eight
#pragma unroll
  for (int i = 0; i < kGradBlocks / 32; ++i) {
    const int p = r + 32 * i;
    part[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    if (p < P) part[i] = *reinterpret_cast<const f32x4*>(partial + p * H + j);
  }
  f32x4 v = part[0];
#pragma unroll
  for (int i = 1; i < kGradBlocks / 32; ++i) v += part[i];
  sums[r][c] = v;
#pragma unroll
  for (int n = 16; n >= 1; n >>= 1) {
    __syncthreads();
    if (r < n) sums[r][c] += sums[r + n][c];
  }
  if (r == 0) *reinterpret_cast<f32x4*>(dw + j) = sums[0][c];
}

// Wavefronts per row and octets per lane for rows of H elements.  More wavefronts
// shorten a row's latency, fewer leave less of them idle; at 7168 (4096 rows, bf16)
// 8 x 2 octets take 38.8 us forward and 46.4 backward, 4 x 4 39.9 and 57.3, 16 x 1
// 43.7 and 46.7, and one row alone takes 3.5, 4.7 and 3.1 us forward.  The backward
// pass, which keeps dw in registers as well, stays at eight wavefronts, with 256
// registers a lane (18432, 4096 rows: 16 x 3 spilled, 363 us; 8 x 5 takes 144 bf16 and
// 251 fp32).  Six and eight octets a lane spill (4 to 163 registers): 24576 and 32768
// take 211 and 529 us in bf16, 426 and 809 in fp32, against 164, 218, 327 and 437 at
// the copy rate.
#define FP8FG_SHAPE(WPR, CH) f(std::integral_constant<int, WPR>{}, std::integral_constant<int, CH>{})
template <typename F>
hipError_t with_short_shape(int64_t H, F&& f) {
  if (H <= 512) return FP8FG_SHAPE(1, 1);
  if (H <= 1024) return FP8FG_SHAPE(2, 1);
  if (H <= 2048) return FP8FG_SHAPE(4, 1);
  if (H <= 4096) return FP8FG_SHAPE(8, 1);
  return FP8FG_SHAPE(8, 2);  // H <= 8192
}
template <typename F>
hipError_t with_forward_shape(int64_t H, F&& f) {
  if (H <= 8192) return with_short_shape(H, f);
  if (H <= 16384) return FP8FG_SHAPE(16, 2);
  if (H <= 24576) return FP8FG_SHAPE(16, 3);
  return FP8FG_SHAPE(16, 4);  // kNormMaxH
}
template <typename F>
hipError_t with_backward_shape(int64_t H, F&& f) {
  if (H <= 8192) return with_short_shape(H, f);
  if (H <= 12288) return FP8FG_SHAPE(8, 3);
  if (H <= 16384) return FP8FG_SHAPE(8, 4);
  if (H <= 20480) return FP8FG_SHAPE(8, 5);
  if (H <= 24576) return FP8FG_SHAPE(8, 6);
  return FP8FG_SHAPE(8, 8);  // kNormMaxH
}
#undef FP8FG_SHAPE

}  // namespace

hipError_t launch_rmsnorm_quant(const NormArgs& a, hipStream_t s) {
  return with_forward_shape(a.H, [&](auto wpr, auto ch) {
    constexpr int WPR = decltype(wpr)::value, CH = decltype(ch)::value;
    constexpr int ROWS = norm_rows(WPR);
    constexpr int64_t kMost = kMaxWorkItems / (ROWS * WPR * 64) * ROWS;  // rows of a launch: 2^26 or 2^23, nearly
    const int64_t es = a.bf16 ? 2 : 4;
    auto rows = [](auto* p, int64_t bytes) {
      return p ? reinterpret_cast<decltype(p)>(reinterpret_cast<uintptr_t>(p) + bytes) : p;
    };
    for (int64_t m0 = 0; m0 < a.M; m0 += kMost) {
      NormArgs b = a;
      b.M = a.M - m0 < kMost ? a.M - m0 : kMost;
      b.x = rows(a.x, m0 * a.ld_x * es);
      b.r = rows(a.r, m0 * a.ld_r * es);
      b.h = rows(a.h, m0 * a.H * es);
      b.y = rows(a.y, m0 * a.H * es);
      b.q = rows(a.q, m0 * a.H);
      b.scales = rows(a.scales, m0 * (a.H / 128) * 4);
      b.rstd = rows(a.rstd, m0 * 4);
      const dim3 grid(static_cast<unsigned>((b.M + ROWS - 1) / ROWS)), block(ROWS * WPR * 64);
      auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, block, 0, s, b); };
      if (a.bf16)
        a.r ? go(rmsnorm_quant_kernel<true, WPR, CH, true>) : go(rmsnorm_quant_kernel<true, WPR, CH, false>);
      else
        a.r ? go(rmsnorm_quant_kernel<false, WPR, CH, true>) : go(rmsnorm_quant_kernel<false, WPR, CH, false>);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
    return hipSuccess;
  });
}

int64_t rmsnorm_backward_partials(int64_t M, int64_t H) {
  int64_t p = 0;
  (void)with_backward_shape(H, [&](auto wpr, auto) {
    constexpr int WPR = decltype(wpr)::value, SLOTS = kGradWaves / WPR;
    p = (M + SLOTS - 1) / SLOTS;
    return hipSuccess;
  });
  return p < kGradBlocks ? p : kGradBlocks;
}

hipError_t launch_rmsnorm_backward(const NormGradArgs& a, float* dw, hipStream_t s) {
  const int64_t P = rmsnorm_backward_partials(a.M, a.H);
  hipError_t e = hipSuccess;
  if (P > 0) {
    e = with_backward_shape(a.H, [&](auto wpr, auto ch) {
      constexpr int WPR = decltype(wpr)::value, CH = decltype(ch)::value;
      const size_t lds = WPR < kGradWaves && a.partial ? a.H * sizeof(float) : 0;
      const dim3 grid(static_cast<unsigned>(P)), block(kGradWaves * 64);
      auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, block, lds, s, a); };
      if (a.bf16)
        a.dh ? go(rmsnorm_backward_kernel<true, WPR, CH, true>) : go(rmsnorm_backward_kernel<true, WPR, CH, false>);
      else
        a.dh ? go(rmsnorm_backward_kernel<false, WPR, CH, true>)
             : go(rmsnorm_backward_kernel<false, WPR, CH, false>);
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
