// Routing of tokens to experts and its gradient.
//
// Forward, per token: s = softmax(z) or sigmoid(z), c = s + bias; the best groups by the sum
// of their one or two largest c, the k largest c in them, and the weights
// scale * s_j (/ the sum of the chosen s).
// Backward, with t_j = s_j dL/ds_j through the weights and u = dscores * s:
//     sigmoid: dz = (t + u)(1 - s),   softmax: dz = t + u - s * sum(t + u).
#include "activation.h"
#include "launch.h"
#include "lanes.h"

namespace fp8fg {
namespace {

constexpr int kWaves = 4;                       // tokens of a workgroup
constexpr int64_t kMostBlocks = int64_t(1) << 20;
constexpr int kSteps = kRouteMaxE / 64;         // experts of a lane: lane, lane + 64, ...
constexpr double kNotANumber = -1e300;          // ranks below every fp32 number, above what is out

template <bool BF16>
__device__ __forceinline__ float element(const void* p, int64_t i) {
  if constexpr (BF16) return __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(p)[i]) << 16);
  return static_cast<const float*>(p)[i];
}

template <typename T>
__device__ __forceinline__ T wave_max(T v) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) {
    const T o = __shfl_xor(v, d);
    v = o > v ? o : v;
  }
  return v;
}
template <typename T>
__device__ __forceinline__ T wave_sum(T v) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d);
  return v;
}

// Scores of a token's logits; lanes without an expert hold -infinity.  A logit of -infinity
// has score 0, whatever the others are.
template <typename F>
__device__ __forceinline__ void scores(bool sigmoidal, const float (&z)[kSteps], F (&s)[kSteps]) {
  if (sigmoidal) {
#pragma unroll
    for (int i = 0; i < kSteps; ++i) s[i] = F(1) / (F(1) + exp(-static_cast<F>(z[i])));
  } else {
    float m = -__builtin_inff();
#pragma unroll
    for (int i = 0; i < kSteps; ++i) m = fmaxf(m, z[i]);
    m = wave_max(m);
    F sum = 0;
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      s[i] = z[i] == -__builtin_inff() ? F(0) : exp(static_cast<F>(z[i]) - static_cast<F>(m));
      sum += s[i];
    }
    sum = wave_sum(sum);
#pragma unroll
    for (int i = 0; i < kSteps; ++i) s[i] = s[i] == F(0) ? F(0) : s[i] / sum;
  }
}

// A chosen expert's score times a factor that is the same for all of its token's (m: the
// largest chosen logit), for their shares: fp32 holds it however small the scores are.
__device__ __forceinline__ float share(bool sigmoidal, float z, float m) {
  if (z == -__builtin_inff()) return 0.0f;
  if (!sigmoidal) return expf(z - m);
  return z >= 0.0f ? 1.0f / (1.0f + expf(-z)) : expf(z - fminf(m, 0.0f)) / (1.0f + expf(z));
}
// Lane j < k: the share of the j-th chosen expert's logit among them; the other lanes (and
// places without an expert) hold -infinity.
__device__ __forceinline__ float shares(bool sigmoidal, float z) {
  const float f = share(sigmoidal, z, wave_max(z));
  const float sum = wave_sum(f);
  return f == 0.0f ? 0.0f : f / sum;
}

// One wavefront per token; every choice in 64 bits.
template <bool BF16>
__global__ void __launch_bounds__(kWaves * 64) route_kernel(RouteArgs a) {
  __shared__ double value[kWaves][kRouteMaxE];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const float out = -__builtin_inff();
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * kWaves + wave; t < a.T;
       t += static_cast<int64_t>(gridDim.x) * kWaves) {
    float z[kSteps], s[kSteps];
    double key[kSteps], wide[kSteps];
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const int e = lane + 64 * i;
      z[i] = e < a.E ? element<BF16>(a.z, t * a.ld + e) : out;
    }
    scores(a.sigmoid, z, s);
    scores(a.sigmoid, z, wide);
    if (a.scores) {
#pragma unroll
      for (int i = 0; i < kSteps; ++i)
        if (lane + 64 * i < a.E) a.scores[t * a.E + lane + 64 * i] = s[i];
    }
    if (a.mask && a.mask[t] == 0) {
      if (lane < a.k) {
        a.experts[t * a.k + lane] = -1;
        a.weights[t * a.k + lane] = 0.0f;
      }
      continue;
    }
    // what experts are ranked by, and what group scores are made of
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const int e = lane + 64 * i;
      const float b = a.bias && e < a.E ? a.bias[e] : 0.0f;
      const bool gone = z[i] == out || b == out;
      const double c = wide[i] + static_cast<double>(b);
      auto rank = [&](double v) { return gone ? static_cast<double>(out) : v == v ? v : kNotANumber; };
      key[i] = rank(a.bias ? c : static_cast<double>(z[i]));
      wide[i] = a.bias || a.terms == 2 ? rank(c) : key[i];
    }
    if (a.kept < a.groups) {
#pragma unroll
      for (int i = 0; i < kSteps; ++i)
        if (lane + 64 * i < a.E) value[wave][lane + 64 * i] = wide[i];
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      const int size = a.E / a.groups;
      double first = out, second = out;
      if (lane < a.groups) {
        for (int i = 0; i < size; ++i) {
          const double v = value[wave][lane * size + i];
          if (v > first) {
            second = first;
            first = v;
          } else if (v > second) {
            second = v;
          }
        }
      }
      const double score = a.terms == 1 ? first : second == out ? static_cast<double>(out) : first + second;
      int before = 0;  // groups that come before this lane's
      for (int g = 0; g < a.groups; ++g) {
        const double o = __shfl(score, g);
        if (o > score || (o == score && g < lane)) ++before;
      }
      const uint64_t stay = __ballot(lane < a.groups && before < a.kept && score != out);
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        const int e = lane + 64 * i;
        if (e < a.E && !((stay >> (e / size)) & 1)) key[i] = out;
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
    int mine = -1;  // lane j: the j-th expert, its score (or its logit, for the shares)
    float chosen = a.renormalise ? out : 0.0f;
    for (int j = 0; j < a.k; ++j) {
      double best = out;
      int at = kRouteMaxE;
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        if (key[i] > best) {
          best = key[i];
          at = lane + 64 * i;
        }
      }
#pragma unroll
      for (int d = 32; d >= 1; d >>= 1) {
        const double o = __shfl_xor(best, d);
        const int oa = __shfl_xor(at, d);
        if (o > best || (o == best && oa < at)) {
          best = o;
          at = oa;
        }
      }
      if (at == kRouteMaxE) break;  // none left
      float v = 0.0f;
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        if (at == lane + 64 * i) {
          v = a.renormalise ? z[i] : s[i];
          key[i] = out;
        }
      }
      v = __shfl(v, at & 63);
      if (lane == j) {
        mine = at;
        chosen = v;
      }
    }
    const float w = a.renormalise ? shares(a.sigmoid, chosen) : chosen;
    if (lane < a.k) {
      a.experts[t * a.k + lane] = mine;
      a.weights[t * a.k + lane] = mine < 0 ? 0.0f : a.scale * w;
    }
  }
}

// One wavefront per token; lane j holds the j-th chosen expert's t.
template <bool BF16>
__global__ void __launch_bounds__(kWaves * 64) route_backward_kernel(RouteGradArgs a) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const float out = -__builtin_inff();
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * kWaves + wave; t < a.T;
       t += static_cast<int64_t>(gridDim.x) * kWaves) {
    float z[kSteps], s[kSteps], d[kSteps];
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const int e = lane + 64 * i;
      z[i] = e < a.E ? element<BF16>(a.z, t * a.ld + e) : out;
    }
    scores(a.sigmoid, z, s);
    int mine = lane < a.k ? a.experts[t * a.k + lane] : -1;
    if (mine >= a.E) mine = -1;
    const float dw = mine >= 0 ? a.scale * a.dw[t * a.k + lane] : 0.0f;
    float tj;
    if (a.renormalise) {
      const float p = shares(a.sigmoid, mine >= 0 ? element<BF16>(a.z, t * a.ld + mine) : out);
      tj = p * (dw - wave_sum(dw * p));
    } else {
      float chosen = 0.0f;
      for (int j = 0; j < a.k; ++j) {
        const int e = __builtin_amdgcn_readfirstlane(__shfl(mine, j));
        if (e < 0) continue;
        float v = 0.0f;
#pragma unroll
        for (int i = 0; i < kSteps; ++i)
          if (i == (e >> 6)) v = s[i];
        v = __shfl(v, e & 63);
        if (lane == j) chosen = v;
      }
      tj = chosen * dw;
    }
    float total = 0.0f;
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const int e = lane + 64 * i;
      d[i] = a.ds && e < a.E ? a.ds[t * a.E + e] * s[i] : 0.0f;
      total += d[i];
    }
    for (int j = 0; j < a.k; ++j) {
      const int e = __builtin_amdgcn_readfirstlane(__shfl(mine, j));
      const float v = __shfl(tj, j);
      if (e < 0) continue;
#pragma unroll
      for (int i = 0; i < kSteps; ++i)
        if (i == (e >> 6) && lane == (e & 63)) d[i] += v;
    }
    if (!a.sigmoid) {
      // (renormalised weights do not change with a common factor: their t sum to zero)
      total = wave_sum(a.renormalise ? total : total + tj);
    }
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const int e = lane + 64 * i;
      if (e >= a.E) continue;
      float v = a.sigmoid ? d[i] * (1.0f - s[i]) : d[i] - s[i] * total;
      if (z[i] == out) v = 0.0f;
      if constexpr (BF16)
        static_cast<uint16_t*>(a.dz)[t * a.E + e] = static_cast<uint16_t>(pack_bf16(v, 0.0f));
      else
        static_cast<float*>(a.dz)[t * a.E + e] = v;
    }
  }
}

dim3 token_blocks(int64_t T) {
  const int64_t n = (T + kWaves - 1) / kWaves;
  return dim3(static_cast<unsigned>(n < kMostBlocks ? n : kMostBlocks));
}

}  // namespace

hipError_t launch_route(const RouteArgs& a, hipStream_t s) {
  if (a.bf16)
    hipLaunchKernelGGL(route_kernel<true>, token_blocks(a.T), dim3(kWaves * 64), 0, s, a);
  else
    hipLaunchKernelGGL(route_kernel<false>, token_blocks(a.T), dim3(kWaves * 64), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_route_backward(const RouteGradArgs& a, hipStream_t s) {
  if (a.bf16)
    hipLaunchKernelGGL(route_backward_kernel<true>, token_blocks(a.T), dim3(kWaves * 64), 0, s, a);
  else
    hipLaunchKernelGGL(route_backward_kernel<false>, token_blocks(a.T), dim3(kWaves * 64), 0, s, a);
  return hipGetLastError();
}

}  // namespace fp8fg
