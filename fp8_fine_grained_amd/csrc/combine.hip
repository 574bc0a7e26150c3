// Combination of the experts' rows and its gradient.
//     y[t] = base[t] + sum_j w[t, j] * rows[p[t, j]]             (fp32, in the order of j)
//     drows[p[t, j]] = w[t, j] * dy[t],  dw[t, j] = <dy[t], rows[p[t, j]]>
// Bound by HBM: every row is read (and written) once.
#include <type_traits>

#include "launch.h"
#include "lanes.h"

namespace fp8fg {
namespace {

constexpr int kThreads = 256;
constexpr int64_t kMostBlocks = int64_t(1) << 23;  // of kThreads work-items

// Eight consecutive elements as fp32.
template <bool BF16>
__device__ __forceinline__ void load8(const void* p, int64_t i, float (&f)[8]) {
  if constexpr (BF16) {
    const u32x4 u = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(p) + i);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      f[2 * k] = __uint_as_float(u[k] << 16);
      f[2 * k + 1] = __uint_as_float(u[k] & 0xFFFF0000u);
    }
  } else {
    const f32x4* v = reinterpret_cast<const f32x4*>(static_cast<const float*>(p) + i);
    const f32x4 lo = v[0], hi = v[1];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      f[k] = lo[k];
      f[4 + k] = hi[k];
    }
  }
}
template <bool BF16>
__device__ __forceinline__ void store8(void* p, int64_t i, const float (&f)[8]) {
  if constexpr (BF16) {
    *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(p) + i) =
        u32x4{pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7])};
  } else {
    f32x4* v = reinterpret_cast<f32x4*>(static_cast<float*>(p) + i);
    v[0] = f32x4{f[0], f[1], f[2], f[3]};
    v[1] = f32x4{f[4], f[5], f[6], f[7]};
  }
}

// A workgroup per token.
template <bool BF16>
__global__ void __launch_bounds__(kThreads) combine_kernel(CombineArgs a) {
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    for (int64_t c = threadIdx.x * 8; c < a.H; c += kThreads * 8) {
      float y[8] = {};
      if (a.base) load8<BF16>(a.base, t * a.ld_base + c, y);
      for (int j = 0; j < a.k; ++j) {
        const int32_t p = a.positions[t * a.k + j];
        if (p < 0 || p >= a.R) continue;
        const float w = a.weights ? a.weights[t * a.k + j] : 1.0f;
        float r[8];
        load8<BF16>(a.rows, p * a.ld_rows + c, r);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = fmaf(w, r[i], y[i]);
      }
      store8<BF16>(a.y, t * a.H + c, y);
    }
  }
}

// A wavefront per entry (token, place).
template <bool BF16, bool QUANT>
__global__ void __launch_bounds__(kThreads) combine_backward_kernel(CombineGradArgs a) {
  using O = Octet<BF16>;
  const int lane = threadIdx.x & 63;
  const int64_t n = a.T * a.k, waves = static_cast<int64_t>(gridDim.x) * (kThreads / 64);
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * (kThreads / 64) + (threadIdx.x >> 6); i < n; i += waves) {
    const int64_t t = i / a.k;
    const int64_t p = a.positions[i];
    if (p < 0 || p >= a.R) {
      if (a.dw && lane == 0) a.dw[i] = 0.0f;
      continue;
    }
    const float w = a.weights ? a.weights[i] : 1.0f;
    float dot = 0.0f;
    if constexpr (QUANT) {
      const int part = lane & 15;
      for (int64_t g = lane >> 4; g < a.H / 128; g += 4) {
        float d[8], v[8];
        O::widen(O::template load<false>(static_cast<const char*>(a.dy) + (t * a.ld_dy + g * 128) * O::ES, part), d);
        if (a.dw) {
          O::widen(O::load(static_cast<const char*>(a.rows) + (p * a.ld_rows + g * 128) * O::ES, part), v);
#pragma unroll
          for (int k = 0; k < 8; ++k) dot = fmaf(d[k], v[k], dot);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) d[k] *= w;
        float s, inv;
        group_scale(a.pow2, group_amax(d), s, inv);
        O::store_codes(static_cast<uint8_t*>(a.drows) + p * a.H + g * 128, part, d, inv);
        if (part == 0) a.scales[p * (a.H / 128) + g] = s;
      }
    } else {
      for (int64_t c = lane * 8; c < a.H; c += 512) {
        float d[8], v[8];
        load8<BF16>(a.dy, t * a.ld_dy + c, d);
        if (a.dw) {
          load8<BF16>(a.rows, p * a.ld_rows + c, v);
#pragma unroll
          for (int k = 0; k < 8; ++k) dot = fmaf(d[k], v[k], dot);
        }
        if (a.drows) {
#pragma unroll
          for (int k = 0; k < 8; ++k) d[k] *= w;
          store8<BF16>(a.drows, p * a.H + c, d);
        }
      }
    }
    if (a.dw) {
      dot = sum64(dot);
      if (lane == 0) a.dw[i] = dot;
    }
  }
}

unsigned blocks(int64_t n) { return static_cast<unsigned>(n < kMostBlocks ? n : kMostBlocks); }

}  // namespace

hipError_t launch_combine(const CombineArgs& a, hipStream_t s) {
  if (a.bf16)
    hipLaunchKernelGGL(combine_kernel<true>, dim3(blocks(a.T)), dim3(kThreads), 0, s, a);
  else
    hipLaunchKernelGGL(combine_kernel<false>, dim3(blocks(a.T)), dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_combine_backward(const CombineGradArgs& a, hipStream_t s) {
  const dim3 grid(blocks((a.T * a.k + kThreads / 64 - 1) / (kThreads / 64)));
  auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, dim3(kThreads), 0, s, a); };
  if (a.scales)
    a.bf16 ? go(combine_backward_kernel<true, true>) : go(combine_backward_kernel<false, true>);
  else
    a.bf16 ? go(combine_backward_kernel<true, false>) : go(combine_backward_kernel<false, false>);
  return hipGetLastError();
}

}  // namespace fp8fg
