// Routing of tokens to experts and its gradient.
//
// Forward, per token: s = softmax(z) or sigmoid(z), c = s + bias; the best groups by the sum
// of their one or two largest c, the k largest c in them, and the weights
// scale * s_j (/ the sum of the chosen s).
// Backward, with t_j = s_j dL/ds_j through the weights and u = dscores * s:
//     sigmoid: dz = (t + u)(1 - s),   softmax: dz = t + u - s * sum(t + u).
#include <type_traits>

#include "activation.h"
#include "launch.h"
#include "lanes.h"

namespace fp8fg {
namespace {

constexpr int kWaves = 4;                       // wavefronts of a workgroup
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
template <typename F, int STEPS>
__device__ __forceinline__ void scores(bool sigmoidal, const float (&z)[STEPS], F (&s)[STEPS]) {
  if (sigmoidal) {
#pragma unroll
    for (int i = 0; i < STEPS; ++i) s[i] = F(1) / (F(1) + exp(-static_cast<F>(z[i])));
  } else {
    float m = -__builtin_inff();
#pragma unroll
    for (int i = 0; i < STEPS; ++i) m = fmaxf(m, z[i]);
    m = wave_max(m);
    F sum = 0;
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
      s[i] = z[i] == -__builtin_inff() ? F(0) : exp(static_cast<F>(z[i]) - static_cast<F>(m));
      sum += s[i];
    }
    sum = wave_sum(sum);
#pragma unroll
    for (int i = 0; i < STEPS; ++i) s[i] = s[i] == F(0) ? F(0) : s[i] / sum;
  }
}

// The sigmoid of a logit: 0 for -infinity, and what is not a number stays so.
__device__ __forceinline__ float score(float z) {
  const float v = z == z ? sigmoid(z) : z;
  return z == -__builtin_inff() ? 0.0f : v;
}

// Reductions over aligned groups of L = 16, 32 or 64 lanes.
template <int L>
__device__ __forceinline__ float max_of(float v) {
  v = max16(v);
  if constexpr (L >= 32) v = fmaxf(v, __shfl_xor(v, 16));
  if constexpr (L == 64) v = fmaxf(v, __shfl_xor(v, 32));
  return v;
}
template <int L>
__device__ __forceinline__ float sum_of(float v) {
  v += dpp<0xB1>(v);
  v += dpp<0x4E>(v);
  v += dpp<0x141>(v);
  v += dpp<0x140>(v);
  if constexpr (L >= 32) v += __shfl_xor(v, 16);
  if constexpr (L == 64) v += __shfl_xor(v, 32);
  return v;
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
  const float f = share(sigmoidal, z, max_of<64>(z));
  const float sum = sum64(f);
  return f == 0.0f ? 0.0f : f / sum;
}

// ---------------------------------------------------------------- choices in 64 bits
// A token by a whole wavefront, every choice in 64 bits: what the fast kernel below leaves over, and more than 15
// experts per token.  Rare, so its values lie in LDS (value [E]) and not in the fast kernel's registers.
template <bool BF16>
__device__ __forceinline__ void route_token(const RouteArgs& a, int64_t t, double* value) {
  const int lane = threadIdx.x & 63;
  const double out = -__builtin_inf();
  const float outf = -__builtin_inff();
  auto logit = [&](int e) { return element<BF16>(a.z, t * a.ld + e); };
  double top = out, total = 0.0;
  if (!a.sigmoid) {
    float m = outf;
    for (int e = lane; e < a.E; e += 64) m = fmaxf(m, logit(e));
    top = wave_max(m);
    for (int e = lane; e < a.E; e += 64) total += logit(e) == outf ? 0.0 : exp(static_cast<double>(logit(e)) - top);
    total = wave_sum(total);
  }
  // what experts are ranked by (score: also without a bias)
  auto bias = [&](int e) { return a.bias ? static_cast<double>(a.bias[e]) : 0.0; };
  auto score_of = [&](int e) {
    const double z = logit(e), f = a.sigmoid ? 1.0 / (1.0 + exp(-z)) : exp(z - top);
    return a.sigmoid || f == 0.0 ? f : f / total;
  };
  auto rank = [&](int e, bool score) -> double {
    const double z = logit(e), b = bias(e);
    if (z == out || b == out) return out;
    const double c = score || a.bias ? score_of(e) + b : z;
    return c == c ? c : kNotANumber;
  };
  uint64_t stay = ~uint64_t(0);
  const int size = a.E / a.groups;
  if (a.kept < a.groups) {
    for (int e = lane; e < a.E; e += 64) value[e] = rank(e, a.terms == 2);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    double first = out, second = out;
    if (lane < a.groups) {
      for (int i = 0; i < size; ++i) {
        const double v = value[lane * size + i];
        second = fmax(second, fmin(first, v));
        first = fmax(first, v);
      }
    }
    double score = a.terms == 1 ? first : second == out ? out : first + second;
    const bool sum = a.terms == 2 && a.bias && second > kNotANumber && score < -out;
    // how far the sums' roundings may bring two of them
    const double apart = 0x1p-49 * max_of<64>(sum ? static_cast<float>(fabs(first) + fabs(second)) : 0.0f);
    int before;  // groups that come before this lane's
    bool close;
    auto compare = [&]() {
      before = 0;
      close = false;
      for (int g = 0; g < a.groups; ++g) {
        const double o = __shfl(score, g);
        if (o > score || (o == score && g < lane)) ++before;
        close |= g != lane && fabs(o - score) <= apart;
      }
      close &= sum;
    };
    compare();
    if (__ballot(close)) {
      // Scores and biases for themselves: sums that tie as real numbers are equal whichever bias goes with which score.
      if (sum) {
        int at = -1, next = -1;
        for (int e = lane * size; e < (lane + 1) * size; ++e) {
          if (at < 0 && value[e] == first)
            at = e;
          else if (value[e] == second)
            next = e;
        }
        score = (score_of(at) + score_of(next)) + (bias(at) + bias(next));
      }
      compare();
    }
    stay = __ballot(lane < a.groups && before < a.kept && score != out);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  }
  for (int e = lane; e < a.E; e += 64) value[e] = (stay >> (e / size & 63)) & 1 ? rank(e, false) : out;
  int mine = -1;  // lane j: the j-th expert
  for (int j = 0; j < a.k; ++j) {
    double best = out;
    int at = kRouteMaxE;
    for (int e = lane; e < a.E; e += 64) {
      if (value[e] > best) {
        best = value[e];
        at = e;
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
    if ((at & 63) == lane) value[at] = out;
    if (lane == j) mine = at;
  }
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  const float z = mine >= 0 ? logit(mine) : outf;
  float w;
  if (a.renormalise)
    w = shares(a.sigmoid, z);
  else
    w = z == outf ? 0.0f : a.sigmoid ? 1.0f / (1.0f + expf(-z)) : expf(z - static_cast<float>(top)) /
                                                                      static_cast<float>(total);
  if (lane < a.k) {
    a.experts[t * a.k + lane] = mine;
    a.weights[t * a.k + lane] = mine < 0 ? 0.0f : a.scale * w;
  }
}

template <bool BF16>
__global__ void __launch_bounds__(kWaves * 64) route_wide_kernel(RouteArgs a) {
  __shared__ double value[kWaves][kRouteMaxE];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * kWaves + wave; t < a.T;
       t += static_cast<int64_t>(gridDim.x) * kWaves) {
    if (a.scores) {
      float z[kSteps], s[kSteps];
#pragma unroll
      for (int i = 0; i < kSteps; ++i)
        z[i] = lane + 64 * i < a.E ? element<BF16>(a.z, t * a.ld + lane + 64 * i) : -__builtin_inff();
      scores<float, kSteps>(a.sigmoid, z, s);
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
    route_token<BF16>(a, t, value[wave]);
  }
}

// ---------------------------------------------------------------- the fast kernel
// Signed integers in the order of finite floats (without -0), and back: the same exchange.
__device__ __forceinline__ int ordered(int b) { return b ^ ((b >> 31) & 0x7FFFFFFF); }
__device__ __forceinline__ int dpp_max(int v, int o) { return o > v ? o : v; }
template <int L>
__device__ __forceinline__ int max_of(int v) {
  v = dpp_max(v, __builtin_amdgcn_update_dpp(v, v, 0xB1, 0xF, 0xF, false));
  v = dpp_max(v, __builtin_amdgcn_update_dpp(v, v, 0x4E, 0xF, 0xF, false));
  v = dpp_max(v, __builtin_amdgcn_update_dpp(v, v, 0x141, 0xF, 0xF, false));
  v = dpp_max(v, __builtin_amdgcn_update_dpp(v, v, 0x140, 0xF, 0xF, false));
  if constexpr (L >= 32) v = dpp_max(v, __shfl_xor(v, 16));
  if constexpr (L == 64) v = dpp_max(v, __shfl_xor(v, 32));
  return v;
}
// Descending order of a lane's keys: odd-even merging (63 exchanges of a maximum and a minimum for 16 keys).
template <int V>
__device__ __forceinline__ void sort_keys(int (&k)[V]) {
#pragma unroll
  for (int p = 1; p < V; p *= 2) {
#pragma unroll
    for (int q = p; q >= 1; q /= 2) {
#pragma unroll
      for (int j = q % p; j + q < V; j += 2 * q) {
#pragma unroll
        for (int i = 0; i < q; ++i) {
          if (i + j + q < V && (i + j) / (2 * p) == (i + j + q) / (2 * p)) {
            const int x = k[i + j], y = k[i + j + q];
            k[i + j] = x > y ? x : y;
            k[i + j + q] = x > y ? y : x;
          }
        }
      }
    }
  }
}

template <int CTRL>
__device__ __forceinline__ int dpp_int(int v) {
  return __builtin_amdgcn_update_dpp(v, v, CTRL, 0xF, 0xF, false);
}
// The two largest of a set, of which v, or another part's two largest f and s, are met.
__device__ __forceinline__ int larger(int a, int b) { return a > b ? a : b; }
__device__ __forceinline__ void merge_one(int& first, int& second, int v) {
  second = larger(second, first < v ? first : v);
  first = larger(first, v);
}
__device__ __forceinline__ void merge_two(int& first, int& second, int f, int s) {
  second = larger(first < f ? first : f, larger(second, s));
  first = larger(first, f);
}

// L lanes per token, V consecutive experts per lane (so that the lowest index is the first lane's first).  Choices go
// through 32-bit keys, in the order of the fp32 values, whose low bits say where they come from.  A lane sorts its keys
// once; then each round takes the largest of the lanes' first keys, and the lane it came from moves up by one.
// (Unsorted keys, searched and struck out in every round: 15.1 us instead of 12.2 at 8192 x 256.)
//  * bf16 logits without a bias leave room for the whole index: the keys are exact, ties and all;
//  * other keys give up four bits for the place in the lane.  Neighbours that lie closer than those bits and the
//    rounding of a score are put in order by their 64-bit values.  Where that does not do (three in one place at the
//    border, sums of groups that lie close) the token is done again in 64 bits, and so is one with a value that is not
//    a number or +infinity.
// Bound by the instructions of its rounds and their fetch, not by the logits' bytes (8192 x 256 fp32 in 8 groups: 12.2
// us, 1.7 for the bytes), so four tokens of up to 256 experts share a wavefront: a round costs the same for one.  (A
// wavefront per token, all in 64 bits: 83 us.)
template <bool BF16, bool BIAS, int L, int V>
__global__ void __launch_bounds__(kWaves * 64) route_kernel(RouteArgs a) {
  constexpr bool EXACT = BF16 && !BIAS;
  constexpr int TOKENS = 64 / L;
  constexpr float kInf = __builtin_inff();
  constexpr int kOut = static_cast<int>(0x80000000), kLowest = static_cast<int>(0x80800000);  // (the largest negative)
  __shared__ double wide[kWaves][L * V];             // of tokens that are done again
  __shared__ int narrow[kWaves][TOKENS][L * V];    // choices, where groups lie across lanes
  __shared__ __attribute__((aligned(16))) float group_score[kWaves][TOKENS][kRouteMaxGroups + 4];
  __shared__ float group_off[kWaves][TOKENS][kRouteMaxGroups];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int l = lane & (L - 1), slot = lane / L;
  const int e0 = l * V;
  constexpr uint64_t kToken = L == 64 ? ~uint64_t(0) : (uint64_t(1) << (L & 63)) - 1;  // lanes of the first token
  auto of_token = [&](uint64_t ballot) -> uint64_t { return L == 64 ? ballot : (ballot >> (slot * L)) & kToken; };
  float bias[BIAS ? V : 1];
  if constexpr (BIAS) {
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      if (e0 + i + 4 <= a.E && (reinterpret_cast<uintptr_t>(a.bias) & 15) == 0) {
        const f32x4 b = *reinterpret_cast<const f32x4*>(a.bias + e0 + i);
        bias[i] = b[0]; bias[i + 1] = b[1]; bias[i + 2] = b[2]; bias[i + 3] = b[3];
      } else {
#pragma unroll
        for (int q = i; q < i + 4; ++q) bias[q] = e0 + q < a.E ? a.bias[e0 + q] : 0.0f;
      }
    }
  }
  const int size = a.E / a.groups, lanes = size / V, shift = lanes > 0 ? __builtin_ctz(lanes) : 0;
  const bool grouped = a.kept < a.groups;
  const bool sums = grouped && a.terms == 2;  // sums of two scores are compared
  const bool whole = size % V == 0 && (lanes & (lanes - 1)) == 0 && lanes <= 16;  // a group is 1, 2, 4, .. lanes
  const bool scored = BIAS || sums || a.scores || (!a.sigmoid && !a.renormalise);
  constexpr int VEC = BF16 ? 8 : 4;  // elements of a 16-byte load
  const bool vector = V % VEC == 0 && a.E % VEC == 0 && (a.ld * (BF16 ? 2 : 4)) % 16 == 0 &&
                      reinterpret_cast<uintptr_t>(a.z) % 16 == 0;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kWaves * TOKENS;
  for (int64_t t0 = (static_cast<int64_t>(blockIdx.x) * kWaves + wave) * TOKENS; t0 < a.T; t0 += stride) {
    const bool live = t0 + slot < a.T;
    const int64_t t = live ? t0 + slot : a.T - 1;  // past the end: the last token again, not stored
    int E = a.E;
    asm volatile("" : "+s"(E));  // (else its comparisons leave the loop, and fill and spill scalar registers)
    float z[V];
    if (vector) {
      if constexpr (V % VEC == 0) {
#pragma unroll
        for (int q = 0; q < V / VEC; ++q) {
          const int e = e0 + q * VEC < E ? e0 + q * VEC : 0;
          const u32x4 u =
              *reinterpret_cast<const u32x4*>(static_cast<const char*>(a.z) + (t * a.ld + e) * (BF16 ? 2 : 4));
#pragma unroll
          for (int i = 0; i < VEC; ++i) {
            uint32_t v = BF16 ? (i % 2 ? u[i / 2] & 0xFFFF0000u : u[i / 2] << 16) : u[i % 4];
            z[q * VEC + i] = e0 + q * VEC < E ? __uint_as_float(v) : -kInf;
          }
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) z[i] = e0 + i < E ? element<BF16>(a.z, t * a.ld + e0 + i) : -kInf;
    }
    float s[V], top = 0.0f, total = 1.0f, largest = 1.0f;
    if (scored) {
      if (a.sigmoid) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          s[i] = score(z[i]);
        }
      } else {
        top = -kInf;
#pragma unroll
        for (int i = 0; i < V; ++i) top = fmaxf(top, z[i]);
        top = max_of<L>(top);
        total = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          s[i] = z[i] == -kInf ? 0.0f : expf(z[i] - top);
          total += s[i];
        }
        total = sum_of<L>(total);
        largest = 1.0f / total;
#pragma unroll
        for (int i = 0; i < V; ++i) s[i] = s[i] == 0.0f ? 0.0f : s[i] * largest;
      }
      if (a.scores && live) {
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (e0 + i < E) a.scores[t * E + e0 + i] = s[i];
      }
    }
    // how far an fp32 score may be off: the sigmoid's roundings; or exponential, argument, sum and quotient
    const float off = a.sigmoid ? 0x1p-23f : 0x1p-18f * largest;
    // Choices as ordered integers; the tests of all of them at once: what is not a number lies beyond an infinity.
    int ord[V], most = kLowest, least = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float c = BIAS ? s[i] + bias[i] : z[i] + 0.0f;  // (no -0: it equals 0)
      if (BIAS && z[i] == -kInf) c = -kInf;
      ord[i] = ordered(__float_as_int(c));
      most = ord[i] > most ? ord[i] : most;
      least = ord[i] < least ? ord[i] : least;
    }
    bool again = most >= ordered(0x7F800000) || least < ordered(static_cast<int>(0xFF800000));
    uint64_t stay = ~uint64_t(0);  // groups
    if (grouped) {
      // the two largest choices of every group
      auto choice = [&](int i) { return BIAS || !sums || ord[i] < kLowest ? ord[i] : __float_as_int(s[i]); };
      auto value = [&](int first, int second) {
        float v = __int_as_float(ordered(first));
        if (first < kLowest || (sums && second < kLowest)) return -kInf;
        if (sums) v += __int_as_float(ordered(second));
        again |= fabsf(v) == kInf;  // (a sum past fp32's range is no reason to leave a group out)
        return v;
      };
      // How far it may be off: its terms' scores, their roundings (a term may be far above the sum), the sum's.
      auto error = [&](int first, int second) {
        const float f = 0x1p-23f * fabsf(__int_as_float(ordered(first)));
        return 2.0f * off + (sums ? fmaf(0x1p-23f, fabsf(__int_as_float(ordered(second))), f) : f);
      };
      float* of_group = group_score[wave][slot];
      float* off_group = group_off[wave][slot];
      if (whole) {
        int first = kOut, second = kOut;
#pragma unroll
        for (int i = 0; i < V; ++i) merge_one(first, second, choice(i));
        if (lanes >= 2) merge_two(first, second, dpp_int<0xB1>(first), dpp_int<0xB1>(second));
        if (lanes >= 4) merge_two(first, second, dpp_int<0x4E>(first), dpp_int<0x4E>(second));
        if (lanes >= 8) merge_two(first, second, dpp_int<0x141>(first), dpp_int<0x141>(second));
        if (lanes >= 16) merge_two(first, second, dpp_int<0x140>(first), dpp_int<0x140>(second));
        if ((l & (lanes - 1)) == 0 && (l >> shift) < a.groups) {
          of_group[l >> shift] = value(first, second);
          off_group[l >> shift] = error(first, second);
        }
      } else {
        int* c = narrow[wave][slot];
#pragma unroll
        for (int i = 0; i < V; ++i) c[e0 + i] = choice(i);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        for (int g = l; g < a.groups; g += L) {
          int first = kOut, second = kOut;
          int at = g % size;  // (groups start at different banks)
          for (int i = 0; i < size; ++i) {
            merge_one(first, second, c[g * size + at]);
            at = at + 1 == size ? 0 : at + 1;
          }
          of_group[g] = value(first, second);
          off_group[g] = error(first, second);
        }
      }
      if (l < 3) of_group[a.groups + l] = -kInf;  // (read below, four at a time)
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      // Groups with fewer than `kept` before them stay.  Maxima of logits compare exactly; of scores and sums the
      // least that one that stays may be has to lie above the most that one that does not may be (equal ones are left
      // to the 64-bit form).
      const bool exact = !BIAS && !sums;
      stay = 0;
      float low = kInf;
      for (int g0 = 0; g0 < a.groups; g0 += L) {
        const int g = g0 + l;
        const float mine = g < a.groups ? of_group[g] : -kInf;
        int before = 0;
        for (int o = 0; o < a.groups; o += 4) {
          const f32x4 other = *reinterpret_cast<const f32x4*>(of_group + o);
#pragma unroll
          for (int q = 0; q < 4; ++q) before += other[q] > mine || (exact && other[q] == mine && o + q < g) ? 1 : 0;
        }
        const bool keep = mine > -kInf && before < a.kept;
        stay |= of_token(__ballot(keep)) << g0;
        if (keep) low = fminf(low, mine);
      }
      if (!exact) {
        low = -max_of<L>(-low);
        float staying = kInf, leaving = -kInf;  // (above `low`: differences at the border are exact)
        for (int g = l; g < a.groups; g += L) {
          const float d = of_group[g] - low;
          if ((stay >> g) & 1)
            staying = fminf(staying, d - off_group[g]);
          else
            leaving = fmaxf(leaving, d + off_group[g]);
        }
        staying = -max_of<L>(-staying);
        leaving = max_of<L>(leaving);
        again |= (leaving > -kInf && !(staying > leaving)) || __popcll(stay) > a.kept;
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
    int code[V];
#pragma unroll
    for (int i = 0; i < V; ++i) code[i] = EXACT ? (ord[i] & ~0xFFFF) | (1023 - (e0 + i)) : (ord[i] & ~15) | (15 - i);
    if (grouped && whole) {
      const bool keep = (stay >> (l >> shift & 63)) & 1;
#pragma unroll
      for (int i = 0; i < V; ++i) code[i] = keep ? code[i] : kOut;
    } else if (grouped) {
      int g = e0 / size, next = (g + 1) * size;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if (e0 + i == next) {
          ++g;
          next += size;
        }
        if (!((stay >> (g & 63)) & 1)) code[i] = kOut;
      }
    }
    sort_keys(code);
    // Lane j: the j-th expert; of inexact keys one more than asked for, which may yet change places with the last.
    const int found = EXACT ? a.k : a.k + 1;
    int mine = -1;
    float before = kInf, last = kInf;  // the choice before, the last that is asked for
    bool close = false;
    for (int j = 0;; ++j) {
      const int m = max_of<L>(code[0]);
      if constexpr (!EXACT) {
        const float c = __int_as_float(ordered(m & ~15));
        const float apart = (BIAS ? 2.0f * off : 0.0f) + 0x1p-17f * fmaxf(fabsf(before), fabsf(c));
        if (j < found) close |= j > 0 && m >= kLowest && !(before - c > apart);
        if (j == a.k - 1) last = c;
        if (j == found) again |= m >= kLowest && !(last - c > apart);  // three of a kind at the border
        before = c;
      }
      if (j == found) break;
      const int from = __ffsll(static_cast<unsigned long long>(of_token(__ballot(code[0] == m)))) - 1;
      const int e = EXACT ? 1023 - (m & 1023) : from * V + 15 - (m & 15);
      if (l == j) mine = m >= kLowest ? e : -1;
      const bool moves = l == from;
#pragma unroll
      for (int i = 0; i < V - 1; ++i) code[i] = moves ? code[i + 1] : code[i];
      code[V - 1] = moves ? kOut : code[V - 1];
    }
    if constexpr (!EXACT) {
      // Neighbours that the keys cannot tell apart, found in any order: in the order of the logits themselves, or of
      // 64-bit sums.
      if (__ballot(close)) {
        double all = 1.0;
        if (BIAS && !a.sigmoid) {
          all = 0.0;
#pragma unroll 1
          for (int e = e0; e < e0 + V && e < a.E; ++e)
            all += exp(static_cast<double>(element<BF16>(a.z, t * a.ld + e)) - static_cast<double>(top));
#pragma unroll
          for (int d = 1; d < L; d <<= 1) all += __shfl_xor(all, d);
        }
        double c = -__builtin_inf();
        if (mine >= 0) {
          c = static_cast<double>(element<BF16>(a.z, t * a.ld + mine));
          if constexpr (BIAS)
            c = (a.sigmoid ? 1.0 / (1.0 + exp(-c)) : exp(c - static_cast<double>(top)) / all) +
                static_cast<double>(a.bias[mine]);
        }
        int place = 0;
        for (int o = 0; o < found; ++o) {
          const int from = slot * L + o, eo = __shfl(mine, from);
          const double co = __shfl(c, from);
          if (co > c || (co == c && eo >= 0 && eo < mine)) ++place;
        }
        int sorted = -1;
        for (int o = 0; o < found; ++o) {
          const int from = slot * L + o, eo = __shfl(mine, from), po = __shfl(place, from);
          if (po == l && eo >= 0) sorted = eo;
        }
        if (close) mine = sorted;
      }
      if (l >= a.k) mine = -1;
    }
    const bool masked = a.mask && a.mask[t] == 0;
    if (masked) mine = -1;
    const uint64_t redo = __ballot(again && live && !masked);
    // the chosen logits again (from the caches), and their weights
    const float zc = mine >= 0 ? element<BF16>(a.z, t * a.ld + mine) : -kInf;
    float w;
    if (a.renormalise) {
      w = share(a.sigmoid, zc, max_of<L>(zc));
      const float sum = sum_of<L>(w);
      w = w == 0.0f ? 0.0f : w / sum;
    } else {
      w = mine < 0 ? 0.0f : a.sigmoid ? sigmoid(zc) : expf(zc - top) / total;
    }
    if (live && l < a.k && of_token(redo) == 0) {
      a.experts[t * a.k + l] = mine;
      a.weights[t * a.k + l] = mine < 0 ? 0.0f : a.scale * w;
    }
    if (redo) {
#pragma unroll 1
      for (int q = 0; q < TOKENS; ++q)
        if ((redo >> (q * L)) & kToken) route_token<BF16>(a, t0 + q, wide[wave]);
    }
  }
}

// ---------------------------------------------------------------- gradient
// One wavefront per token, STEPS experts per lane; lane j holds the j-th chosen expert's t, and hands it to the lane of
// the expert (one scalar comparison per step, no search).  Bound by HBM at large T: the logits in, their gradient out.
template <bool BF16, int STEPS>
__global__ void __launch_bounds__(kWaves * 64) route_backward_kernel(RouteGradArgs a) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const float out = -__builtin_inff();
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * kWaves + wave; t < a.T;
       t += static_cast<int64_t>(gridDim.x) * kWaves) {
    int mine = lane < a.k ? a.experts[t * a.k + lane] : -1;
    float dw = lane < a.k ? a.dw[t * a.k + lane] : 0.0f;
    float z[STEPS], s[STEPS], d[STEPS];
    float rest[STEPS];  // 1 - s of the sigmoid: a confident expert's is far below the rounding of s
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
      const int e = lane + 64 * i;
      z[i] = e < a.E ? element<BF16>(a.z, t * a.ld + e) : out;
      d[i] = a.ds && e < a.E ? a.ds[t * a.E + e] : 0.0f;
    }
    if (mine >= a.E) mine = -1;
    dw = mine >= 0 ? a.scale * dw : 0.0f;
    const float zc = mine >= 0 ? element<BF16>(a.z, t * a.ld + mine) : out;  // (on its way before the scores)
    float top = out, total = 1.0f;
    if (a.sigmoid) {
#pragma unroll
      for (int i = 0; i < STEPS; ++i) {
        sigmoid_and_rest(z[i], s[i], rest[i]);
        if (z[i] == out) s[i] = 0.0f;
        if (z[i] != z[i]) s[i] = rest[i] = z[i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < STEPS; ++i) top = fmaxf(top, z[i]);
      top = max_of<64>(top);
      total = 0.0f;
#pragma unroll
      for (int i = 0; i < STEPS; ++i) {
        s[i] = z[i] == out ? 0.0f : expf(z[i] - top);
        total += s[i];
      }
      total = sum64(total);
#pragma unroll
      for (int i = 0; i < STEPS; ++i) s[i] = s[i] == 0.0f ? 0.0f : s[i] / total;
    }
    float tj;
    if (a.renormalise) {
      const float p = shares(a.sigmoid, zc);
      tj = p * (dw - sum64(dw * p));
    } else {
      const float f = a.sigmoid ? score(zc) : zc == out ? 0.0f : expf(zc - top) / total;
      tj = f * dw;
    }
    float u = 0.0f;
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
      d[i] = a.ds ? d[i] * s[i] : 0.0f;
      u += d[i];
    }
    for (int j = 0; j < a.k; ++j) {
      const int e = __builtin_amdgcn_readlane(mine, j);
      const float v = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(tj), j));
      if (e < 0) continue;
#pragma unroll
      for (int i = 0; i < STEPS; ++i)
        if (i == (e >> 6)) d[i] += lane == (e & 63) ? v : 0.0f;
    }
    // (renormalised weights do not change with a common factor: their t sum to zero)
    if (!a.sigmoid) u = sum64(a.renormalise ? u : u + tj);
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
      const int e = lane + 64 * i;
      if (e >= a.E) continue;
      float v = a.sigmoid ? d[i] * rest[i] : d[i] - s[i] * u;
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
  if (a.k > 15) {
    if (a.bf16)
      hipLaunchKernelGGL(route_wide_kernel<true>, token_blocks(a.T), dim3(kWaves * 64), 0, s, a);
    else
      hipLaunchKernelGGL(route_wide_kernel<false>, token_blocks(a.T), dim3(kWaves * 64), 0, s, a);
    return hipGetLastError();
  }
  auto shape = [&](auto bf16, auto bias) {
    constexpr bool BF16 = decltype(bf16)::value, BIAS = decltype(bias)::value;
    const dim3 narrow = token_blocks((a.T + 3) / 4), half = token_blocks((a.T + 1) / 2), full = token_blocks(a.T),
               block(kWaves * 64);
    if (a.E > 64 && a.E <= 256 && a.T <= 512)  // (less code to fetch: one token 6.7 -> 5.1 us)
      hipLaunchKernelGGL((route_kernel<BF16, BIAS, 64, 4>), full, block, 0, s, a);
    else if (a.E <= 64)
      hipLaunchKernelGGL((route_kernel<BF16, BIAS, 16, 4>), narrow, block, 0, s, a);
    else if (a.E <= 128)
      hipLaunchKernelGGL((route_kernel<BF16, BIAS, 16, 8>), narrow, block, 0, s, a);
    else if (a.E <= 256)
      hipLaunchKernelGGL((route_kernel<BF16, BIAS, 16, 16>), narrow, block, 0, s, a);
    else if (a.E <= 512)
      hipLaunchKernelGGL((route_kernel<BF16, BIAS, 32, 16>), half, block, 0, s, a);
    else
      hipLaunchKernelGGL((route_kernel<BF16, BIAS, 64, 16>), full, block, 0, s, a);
    return hipGetLastError();
  };
  if (a.bf16) return a.bias ? shape(std::true_type{}, std::true_type{}) : shape(std::true_type{}, std::false_type{});
  return a.bias ? shape(std::false_type{}, std::true_type{}) : shape(std::false_type{}, std::false_type{});
}

hipError_t launch_route_backward(const RouteGradArgs& a, hipStream_t s) {
  auto form = [&](auto bf16) {
    constexpr bool BF16 = decltype(bf16)::value;
    auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, token_blocks(a.T), dim3(kWaves * 64), 0, s, a); };
    if (a.E <= 64)
      go(route_backward_kernel<BF16, 1>);
    else if (a.E <= 128)
      go(route_backward_kernel<BF16, 2>);
    else if (a.E <= 256)
      go(route_backward_kernel<BF16, 4>);
    else if (a.E <= 512)
      go(route_backward_kernel<BF16, 8>);
    else
      go(route_backward_kernel<BF16, 16>);
    return hipGetLastError();
  };
  return a.bf16 ? form(std::true_type{}) : form(std::false_type{});
}

}  // namespace fp8fg
