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
  __device__ __forceinline__ void form(const typename O::Raw& rd, const typename O::Raw& rg, const typename O::Raw& ru) {
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
// A 512-thread workgroup owns 128 tokens x 128 columns of dh, g and u.  Thread
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

template <bool BF16>
__global__ void __launch_bounds__(512) gated_backward_tile_kernel(GatedGradArgs a) {
  using O = Octet<BF16>;
  __shared__ __attribute__((aligned(16))) union {
    uint32_t tile[3][128 * kPitch];
    float max[3][32][128];  // before the codes
  } lds;
  __shared__ float inverse[3][128];
  const int tid = threadIdx.x;
  const int part = tid & 15, rg = tid >> 4;
  const int64_t TG = a.M >> 7, G = a.I >> 7;
  // Token group fastest, each XCD (workgroup id mod 8) one contiguous range: the
  // 128-byte runs and the scales of an output column come through one L2.
  const int n = static_cast<int>(gridDim.x);
  const int b = n % 8 == 0 ? (blockIdx.x % 8) * (n / 8) + blockIdx.x / 8 : blockIdx.x;
  const int64_t tg = b % TG, c0 = b / TG * 128;
  Grads<BF16> v[4];
  {
    // Every load goes out first; then row by row, so that a row's loaded registers
    // are free before the next row's results need theirs.
    typename O::Raw rd[4], rgt[4], ru[4];
    const char* dh = static_cast<const char*>(a.dh) + ((tg * 128 + 4 * rg) * a.ld_dh + c0) * O::ES;
    const char* gu = static_cast<const char*>(a.gu) + ((tg * 128 + 4 * rg) * 2 * a.I + c0) * O::ES;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      rd[i] = O::load(dh + i * a.ld_dh * O::ES, part);
      rgt[i] = O::load(gu + i * 2 * a.I * O::ES, part);
      ru[i] = O::load(gu + (2 * i + 1) * a.I * O::ES, part);
    }
    uint8_t* q = a.q + (tg * 128 + 4 * rg) * 2 * a.I + c0;
    float* s_out = a.s + (tg * 128 + 4 * rg) * 2 * G + (c0 >> 7);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i].form(rd[i], rgt[i], ru[i]);
      if (a.q) {
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
    if (out) out[((k == 1 ? a.I : 0) + c0 + c) * TG + tg] = s;
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
    if (!out) continue;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int c = (tid + 512 * j) >> 3, ch = tid & 7;
      *reinterpret_cast<u32x4*>(out + ((k == 1 ? a.I : 0) + c0 + c) * a.M + tg * 128 + ch * 16) =
          *reinterpret_cast<const u32x4*>(&lds.tile[k][c * kPitch + 4 * (ch ^ piece_key<BF16>(c))]);
    }
  }
}

}  // namespace

hipError_t launch_gated_backward(const GatedGradArgs& a, hipStream_t s) {
  const int64_t G = a.I >> 7;
  if (a.q_t || a.q_ht) {
    const dim3 grid(static_cast<unsigned>((a.M >> 7) * G));
    if (a.bf16)
      hipLaunchKernelGGL(gated_backward_tile_kernel<true>, grid, dim3(512), 0, s, a);
    else
      hipLaunchKernelGGL(gated_backward_tile_kernel<false>, grid, dim3(512), 0, s, a);
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
