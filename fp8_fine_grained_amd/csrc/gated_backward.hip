// Gradient of the gated activation h = g sigmoid(g) u, quantised for the two
// products of the backward pass as it is formed.  With p = sigmoid(g):
//     dg = dh u p (1 + g (1 - p)),   du = dh g p,   h = g p u  (formed again)
// (dg, du) [M, 2I] leaves 1x128-quantised along its columns (operand of the data
// gradient dX = dGU W) and, transposed, along the tokens (operand of the weight
// gradient dW = dGU^T X); h leaves transposed for the down projection's weight
// gradient dW2 = dY^T h.  One pass: dh, g and u are read once, 11 bytes move per
// (token, column) in bf16, and HBM is the bound.
#include "activation.h"
#include "launch.h"
#include "lanes.h"

namespace fp8fg {
namespace {

// The lane's octets of dg, du and h of one row's 128 columns.
template <bool BF16>
struct Grads {
  float g[8], u[8], h[8];
  // dh, gate and up octets as loaded
  using O = Octet<BF16>;
  __device__ __forceinline__ void form(const typename O::Raw& rd, const typename O::Raw& rg,
                                       const typename O::Raw& ru) {
    float d[8];
    O::widen(rd, d);
    O::widen(rg, g);
    O::widen(ru, u);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float p = sigmoid(g[i]);
      const float gp = g[i] * p;
      h[i] = gp * u[i];
      const float dg = d[i] * u[i] * p * fmaf(g[i], 1.0f - p, 1.0f);
      u[i] = d[i] * gp;
      g[i] = dg;
    }
  }
};

// ---------------------------------------------------------------- rows only
// 16 lanes own one (token, 128 columns) pair and write its two groups of codes.
template <bool BF16>
__global__ void __launch_bounds__(256) gated_backward_rows_kernel(GatedGradArgs a) {
  using O = Octet<BF16>;
  const int part = threadIdx.x & 15;
  const int64_t G = a.I >> 7;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * 16 + (threadIdx.x >> 4);
  if (t >= a.M * G) return;  // 16 whole lanes; only those exchange below
  const int64_t m = t / G, c = (t - m * G) * 128;
  const char* gu = static_cast<const char*>(a.gu) + (m * 2 * a.I + c) * O::ES;
  Grads<BF16> v;
  v.form(O::load(static_cast<const char*>(a.dh) + (m * a.ld_dh + c) * O::ES, part), O::load(gu, part),
         O::load(gu + a.I * O::ES, part));
  float s, inv;
  group_scale(a.pow2, group_amax(v.g), s, inv);
  O::store_codes(a.q + m * 2 * a.I + c, part, v.g, inv);
  if (part == 0) a.s[m * 2 * G + (c >> 7)] = s;
  group_scale(a.pow2, group_amax(v.u), s, inv);
  O::store_codes(a.q + m * 2 * a.I + a.I + c, part, v.u, inv);
  if (part == 0) a.s[m * 2 * G + G + (c >> 7)] = s;
}

// ------------------------------------------------------- rows and columns
// A 512-thread workgroup takes tiles of 128 tokens x 128 columns of dh, g and u.
// ALL: every output is asked for, which leaves the loads and stores without branches.  Thread
// (rg, part) holds rows 4 rg .. 4 rg + 3 and the 8 columns of lane `part`, so its
// four tokens of a column are one dword of the transposed codes.  Column maxima
// meet in LDS; the transposed codes are staged there as well and leave as whole
// 128-byte runs.  LDS rows are 36 dwords apart and their 16-byte
// pieces permuted by the column, so the 64 lanes of a store hit 64 banks.
constexpr int kPitch = 36;

template <bool BF16>
__device__ __forceinline__ int piece_key(int c) {
  return BF16 ? (c >> 4) & 7 : (c >> 4) & 3;
}

template <bool BF16, bool ALL>
__global__ void __launch_bounds__(512) gated_backward_tile_kernel(GatedGradArgs a) {
  using O = Octet<BF16>;
  __shared__ __attribute__((aligned(16))) union {
    uint32_t tile[3][128 * kPitch];
    float max[3][32][128];  // before the codes
  } lds;
  __shared__ float inverse[3][128];
  const int tid = threadIdx.x;
  const int part = tid & 15, rg = tid >> 4;
  const int TG = static_cast<int>(a.M >> 7), G = static_cast<int>(a.I >> 7);
  // Tiles are numbered token group fastest; each XCD (workgroup id mod 8) takes one
  // contiguous range and its workgroups stride through it, so the 128-byte runs and
  // the scales of an output column come through one L2.
  const int tiles = TG * G, per_xcd = (tiles + 7) / 8;
  const int first = (blockIdx.x % 8) * per_xcd;
  const int end = first + per_xcd < tiles ? first + per_xcd : tiles;
  const int stride = gridDim.x / 8;
  // bf16 inputs leave registers to load the next tile ahead (8192 x 2048: 54 -> 47.7
  // us); fp32 ones take a tile per workgroup (4096 x 2048: 41 with, 35 us without).
  constexpr bool AHEAD = BF16;
  struct Raw {
    typename O::Raw d[4], g[4], u[4];
  };
  auto load = [&](Raw& r, int t) {
    const int64_t tg = t % TG, c0 = static_cast<int64_t>(t / TG) * 128;
    const char* dh = static_cast<const char*>(a.dh) + ((tg * 128 + 4 * rg) * a.ld_dh + c0) * O::ES;
    const char* gu = static_cast<const char*>(a.gu) + ((tg * 128 + 4 * rg) * 2 * a.I + c0) * O::ES;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      r.d[i] = O::load(dh + i * a.ld_dh * O::ES, part);
      r.g[i] = O::load(gu + i * 2 * a.I * O::ES, part);
      r.u[i] = O::load(gu + (2 * i + 1) * a.I * O::ES, part);
    }
  };
  int t = first + blockIdx.x / 8;
  if (t >= end) return;
  Raw raw;
  if constexpr (AHEAD) load(raw, t);
  for (; t < end; t += stride) {
    if constexpr (!AHEAD) load(raw, t);
    const int64_t tg = t % TG, c0 = static_cast<int64_t>(t / TG) * 128;
    Grads<BF16> v[4];
    {
      uint8_t* q = a.q + (tg * 128 + 4 * rg) * 2 * a.I + c0;
      float* s_out = a.s + (tg * 128 + 4 * rg) * 2 * G + (c0 >> 7);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[i].form(raw.d[i], raw.g[i], raw.u[i]);
        if (ALL || a.q) {
          float s, inv;
          group_scale(a.pow2, group_amax(v[i].g), s, inv);
          O::store_codes(q + 2 * i * a.I, part, v[i].g, inv);
          if (part == 0) s_out[2 * i * G] = s;
          group_scale(a.pow2, group_amax(v[i].u), s, inv);
          O::store_codes(q + (2 * i + 1) * a.I, part, v[i].u, inv);
          if (part == 0) s_out[(2 * i + 1) * G] = s;
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    if constexpr (AHEAD) {
      load(raw, t + stride < end ? t + stride : t);  // the next tile, while this one's columns are formed
      __builtin_amdgcn_sched_barrier(0);
    }
    // column maxima: the thread's four rows, then the workgroup's 32 row groups
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      float mx[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        mx[e] = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          mx[e] = fmaxf(mx[e], fabsf(k == 0 ? v[i].g[e] : k == 1 ? v[i].u[e] : v[i].h[e]));
      }
#pragma unroll
      for (int h = 0; h < 2; ++h)
        *reinterpret_cast<f32x4*>(&lds.max[k][rg][O::col(part, 4 * h)]) =
            f32x4{mx[4 * h], mx[4 * h + 1], mx[4 * h + 2], mx[4 * h + 3]};
    }
    __syncthreads();
    if (tid < 384) {
      const int k = tid >> 7, c = tid & 127;
      float mx = 0.0f;
#pragma unroll
      for (int r = 0; r < 32; ++r) mx = fmaxf(mx, lds.max[k][r][c]);
      float s, inv;
      group_scale(a.pow2, mx, s, inv);
      inverse[k][c] = inv;
      float* out = k < 2 ? a.s_t : a.s_ht;
      if (ALL || out) out[((k == 1 ? a.I : 0) + c0 + c) * TG + tg] = s;
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int c = O::col(part, e);
      const int at = c * kPitch + (rg ^ (piece_key<BF16>(c) << 2));
      const float ig = inverse[0][c], iu = inverse[1][c], ih = inverse[2][c];
      lds.tile[0][at] = cvt4(v[0].g[e] * ig, v[1].g[e] * ig, v[2].g[e] * ig, v[3].g[e] * ig);
      lds.tile[1][at] = cvt4(v[0].u[e] * iu, v[1].u[e] * iu, v[2].u[e] * iu, v[3].u[e] * iu);
      lds.tile[2][at] = cvt4(v[0].h[e] * ih, v[1].h[e] * ih, v[2].h[e] * ih, v[3].h[e] * ih);
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      uint8_t* out = k < 2 ? a.q_t : a.q_ht;
      if (!ALL && !out) continue;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int c = (tid + 512 * j) >> 3, ch = tid & 7;
        *reinterpret_cast<u32x4*>(out + ((k == 1 ? a.I : 0) + c0 + c) * a.M + tg * 128 + ch * 16) =
            *reinterpret_cast<const u32x4*>(&lds.tile[k][c * kPitch + 4 * (ch ^ piece_key<BF16>(c))]);
      }
    }
    __syncthreads();  // the staged codes have been read
  }
}

}  // namespace

hipError_t launch_gated_backward(const GatedGradArgs& a, hipStream_t s) {
  const int64_t G = a.I >> 7;
  if (a.q_t || a.q_ht) {
    // a multiple of the 8 XCDs; bf16: one workgroup per compute unit (its registers
    // hold one), walking over the tiles
    const int cus = device_cus();
    const int64_t tiles = (a.M >> 7) * G, most = cus >= 8 ? cus / 8 * 8 : 256;
    const dim3 grid(static_cast<unsigned>(a.bf16 && tiles > most ? most : (tiles + 7) / 8 * 8));
    auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, dim3(512), 0, s, a); };
    const bool all = a.q && a.q_t && a.q_ht;
    if (a.bf16)
      all ? go(gated_backward_tile_kernel<true, true>) : go(gated_backward_tile_kernel<true, false>);
    else
      all ? go(gated_backward_tile_kernel<false, true>) : go(gated_backward_tile_kernel<false, false>);
  } else {
    const dim3 grid(static_cast<unsigned>((a.M * G + 15) / 16));
    if (a.bf16)
      hipLaunchKernelGGL(gated_backward_rows_kernel<true>, grid, dim3(256), 0, s, a);
    else
      hipLaunchKernelGGL(gated_backward_rows_kernel<false>, grid, dim3(256), 0, s, a);
  }
  return hipGetLastError();
}

}  // namespace fp8fg
