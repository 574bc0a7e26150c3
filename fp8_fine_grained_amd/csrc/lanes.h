// Device helpers of the element-wise kernels around the GEMM (norm.hip,
// gated_backward.hip, clip.hip): eight consecutive-lane elements as fp32,
// reductions over a row's 16 lanes and over a wavefront, bf16 rounding.
#pragma once
#include <hip/hip_runtime.h>
#include <cstdint>

#include "quant_rule.h"

namespace fp8fg {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, false));
}
// Max over each aligned group of 16 lanes (quad xor 1 and 2, half-row mirror, row mirror).
__device__ __forceinline__ float max16(float v) {
  v = fmaxf(v, dpp<0xB1>(v));
  v = fmaxf(v, dpp<0x4E>(v));
  v = fmaxf(v, dpp<0x141>(v));
  return fmaxf(v, dpp<0x140>(v));
}
// Sum over the 64-lane wavefront, the same value in every lane.
__device__ __forceinline__ float sum64(float v) {
  v += dpp<0xB1>(v);
  v += dpp<0x4E>(v);
  v += dpp<0x141>(v);
  v += dpp<0x140>(v);
  v += __shfl_xor(v, 16);
  return v + __shfl_xor(v, 32);
}

// Two fp32 values as packed bf16, round to nearest even (low half a).
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  const bf16x2 v = {static_cast<__bf16>(a), static_cast<__bf16>(b)};
  return __builtin_bit_cast(uint32_t, v);
}

// A 128-element group read by 16 lanes, 8 elements each, so that every load
// instruction of the 16 lanes reads whole contiguous runs: a bf16 lane holds
// elements 8*part .. +7 (one 16-byte load), an fp32 lane 4*part .. +3 and
// 64 + 4*part .. +3 (two 16-byte loads, each covering 256 contiguous bytes).
template <bool BF16>
struct Octet {
  static constexpr int ES = BF16 ? 2 : 4;
  // column within the group of the lane's element i
  static __device__ __forceinline__ int col(int part, int i) {
    return BF16 ? 8 * part + i : (i < 4 ? 4 * part + i : 60 + 4 * part + i);
  }
  struct Raw {
    u32x4 v[BF16 ? 1 : 2];
  };
  // The lane's octet of the group starting at `g` (16-byte aligned).
  template <bool NT = true>
  static __device__ __forceinline__ Raw load(const void* g, int part) {
    const u32x4* p = static_cast<const u32x4*>(g) + part;
    Raw r;
    r.v[0] = NT ? __builtin_nontemporal_load(p) : *p;
    if constexpr (!BF16) r.v[1] = NT ? __builtin_nontemporal_load(p + 16) : p[16];
    return r;
  }
  static __device__ __forceinline__ void widen(const Raw& r, float (&f)[8]) {
    if constexpr (BF16) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(r.v[0][i] << 16);
        f[2 * i + 1] = __uint_as_float(r.v[0][i] & 0xFFFF0000u);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f[i] = __uint_as_float(r.v[0][i]);
        f[4 + i] = __uint_as_float(r.v[1][i]);
      }
    }
  }
  template <bool NT = false>
  static __device__ __forceinline__ void store(void* g, int part, const float (&f)[8]) {
    u32x4* p = static_cast<u32x4*>(g) + part;
    auto put = [](const u32x4& v, u32x4* to) {
      if constexpr (NT)
        __builtin_nontemporal_store(v, to);
      else
        *to = v;
    };
    if constexpr (BF16) {
      put(u32x4{pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7])}, p);
    } else {
      put(u32x4{__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3])}, p);
      put(u32x4{__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]), __float_as_uint(f[7])}, p + 16);
    }
  }
  // The lane's 8 codes into the group's 128-byte code row.
  static __device__ __forceinline__ void store_codes(uint8_t* g, int part, const float (&f)[8], float inv) {
    const uint32_t lo = cvt4(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv);
    const uint32_t hi = cvt4(f[4] * inv, f[5] * inv, f[6] * inv, f[7] * inv);
    if constexpr (BF16) {
      *reinterpret_cast<u32x2*>(g + 8 * part) = u32x2{lo, hi};
    } else {
      *reinterpret_cast<uint32_t*>(g + 4 * part) = lo;
      *reinterpret_cast<uint32_t*>(g + 64 + 4 * part) = hi;
    }
  }
};

// max|f| over a lane's octet and the 16 lanes of its group
__device__ __forceinline__ float group_amax(const float (&f)[8]) {
  float a = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) a = fmaxf(a, fabsf(f[i]));
  return max16(a);
}

// The group rule with the scale form chosen at run time, and with the same bits as
// group_scale<>() from quant_rule.h in fewer instructions: a quotient by a constant
// is its product with the rounded reciprocal plus one correction, and 1/s one
// Newton step on the hardware reciprocal.  (Both are then the correctly rounded
// divisions; the tests compare them with the quantisers over every mantissa.)  An
// infinite amax has an infinite scale and 1/s = 0, as the rule has it.  Below the
// rule's range (s under the smallest normal, where 1/s may be infinite) the codes are
// zero: the caller of a fused operator does not see the values that are quantised,
// and cannot keep them out of it.
__device__ __forceinline__ void group_scale(bool pow2, float amax, float& s, float& inv) {
  if (pow2) {
    group_scale<true>(amax, s, inv);
    return;
  }
  constexpr float kInv448 = 1.0f / kE4M3Max;
  constexpr int kPositiveNormal = 0x100;
  const float q = amax * kInv448;
  s = amax < __builtin_inff() ? fmaf(fmaf(-kE4M3Max, q, amax), kInv448, q) : amax;
  const float r = __builtin_amdgcn_rcpf(s);
  inv = __builtin_amdgcn_classf(s, kPositiveNormal) ? fmaf(fmaf(-s, r, 1.0f), r, r) : 0.0f;
}

}  // namespace fp8fg
