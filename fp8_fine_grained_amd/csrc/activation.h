// The sigmoid of the gated activation, shared by its forward (the epilogues of
// gemm_fp8_tile.h and gemm_gated.hip) and its gradient (gated_backward.hip).
#pragma once
#include <hip/hip_runtime.h>

namespace fp8fg {

// 1 / (1 + exp(-g)) to about an ulp.  exp(-g) = 2^t with t = -g log2(e) taken in two
// parts, hi + lo: the hardware exponential of hi alone would carry hi's rounding,
// |t| / 2 ulp.  The reciprocal takes one Newton step.  Nine instructions, where the
// library's exponential and an exact division take 22 (rows of the 8192 x 2048 gradient:
// 31.9 -> 27.8 us).  g is held to where the result changes: at -88.7 the exponential is
// just finite and its reciprocal, below the normal range, is zero.
__device__ __forceinline__ float sigmoid(float g) {
  constexpr float kLog2e = 1.44269504f, kLog2eRest = 1.92596303e-8f, kLn2 = 0.693147181f;
  g = __builtin_amdgcn_fmed3f(g, -88.7f, 100.0f);
  const float hi = -g * kLog2e;
  const float lo = fmaf(-g, kLog2e, -hi) - g * kLog2eRest;
  float e = __builtin_amdgcn_exp2f(hi);
  e = fmaf(e, lo * kLn2, e);
  const float x = 1.0f + e;
  const float r = __builtin_amdgcn_rcpf(x);
  return fmaf(fmaf(-x, r, 1.0f), r, r);
}

}  // namespace fp8fg
