// Combination of the experts' rows and its gradient.
//     y[t] = base[t] + sum_j w[t, j] * rows[p[t, j]]             (fp32, in the order of j)
//     drows[p[t, j]] = w[t, j] * dy[t],  dw[t, j] = <dy[t], rows[p[t, j]]>
// Bound by HBM: every row is read (and written) once.  8192 tokens of 8 x 7168 bf16: 211 us (5.6 TB/s, most of it
// read), the gradient with quantised rows 317 us (4.9 TB/s, read and written).
#include <type_traits>

#include "launch.h"
#include "lanes.h"

namespace fp8fg {
namespace {

constexpr int kThreads = 256;
constexpr int kPerGroup = kThreads / 64;           // wavefronts of a workgroup
constexpr int64_t kMostBlocks = int64_t(1) << 23;  // of kThreads work-items

// A wavefront's piece of a row: 512 columns from `base`, eight to a lane, in whole contiguous runs per load (bf16:
// 8 lane .. + 7; fp32: 4 lane .. + 3 of either half).  Columns past the row's end read its first ones.
template <bool BF16>
struct Piece {
  static constexpr int ES = BF16 ? 2 : 4, LOADS = BF16 ? 1 : 2;
  struct Raw {
    u32x4 v[LOADS];
  };
  static __device__ __forceinline__ int64_t column(int64_t base, int lane, int half) {
    return base + (BF16 ? 8 * lane : 256 * half + 4 * lane);
  }
  template <bool NT = false>
  static __device__ __forceinline__ Raw load(const void* row, int64_t base, int lane, int64_t H) {
    Raw r;
#pragma unroll
    for (int h = 0; h < LOADS; ++h) {
      const int64_t c = column(base, lane, h);
      const u32x4* p = reinterpret_cast<const u32x4*>(static_cast<const char*>(row) + (c < H ? c : 0) * ES);
      r.v[h] = NT ? __builtin_nontemporal_load(p) : *p;
    }
    return r;
  }
  static __device__ __forceinline__ void widen(const Raw& r, float (&f)[8]) {
    if constexpr (BF16) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        f[2 * k] = __uint_as_float(r.v[0][k] << 16);
        f[2 * k + 1] = __uint_as_float(r.v[0][k] & 0xFFFF0000u);
      }
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) f[k] = __uint_as_float(r.v[k / 4][k % 4]);
    }
  }
  // Zeros for the columns past the row's end.
  static __device__ __forceinline__ void cut(float (&f)[8], int64_t base, int lane, int64_t H) {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (column(base, lane, BF16 ? 0 : k / 4) >= H) f[k] = 0.0f;
  }
  template <bool NT = false>
  static __device__ __forceinline__ void store(void* row, int64_t base, int lane, int64_t H, const float (&f)[8]) {
#pragma unroll
    for (int h = 0; h < LOADS; ++h) {
      const int64_t c = column(base, lane, h);
      u32x4 v;
      if constexpr (BF16)
        v = u32x4{pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7])};
      else
        v = u32x4{__float_as_uint(f[4 * h]), __float_as_uint(f[4 * h + 1]), __float_as_uint(f[4 * h + 2]),
                  __float_as_uint(f[4 * h + 3])};
      u32x4* p = reinterpret_cast<u32x4*>(static_cast<char*>(row) + c * ES);
      if (c < H) {
        if constexpr (NT)
          __builtin_nontemporal_store(v, p);
        else
          *p = v;
      }
    }
  }
};

__device__ __forceinline__ float lane_of(float v, int lane) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), lane));
}

// A wavefront per piece of a token.  One lane each reads a place's row number and weight; the loads of J rows go out
// together, in a straight line: places without a row read row 0 and are not counted.  (Place after place, each
// waiting for its row: 247 us instead of 226 at 8192 tokens of 8 x 7168 bf16, and 10.1 instead of 2.8 for 4 tokens.)
template <bool BF16, int J>
__global__ void __launch_bounds__(kThreads) combine_kernel(CombineArgs a, int64_t pieces) {
  using P = Piece<BF16>;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t n = a.T * pieces, waves = static_cast<int64_t>(gridDim.x) * kPerGroup;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kPerGroup + wave; i < n; i += waves) {
    const int64_t t = i / pieces, base = (i - t * pieces) * 512;
    int p = lane < a.k ? a.positions[t * a.k + lane] : -1;
    const float w = lane < a.k ? (a.weights ? a.weights[t * a.k + lane] : 1.0f) : 0.0f;
    if (p >= a.R) p = -1;
    float y[8] = {};
    if (a.base)
      P::widen(P::load(static_cast<const char*>(a.base) + t * a.ld_base * P::ES, base, lane, a.H), y);
    for (int j0 = 0; j0 < a.k; j0 += J) {
      typename P::Raw r[J];
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const int at = __builtin_amdgcn_readlane(p, j0 + j);
        r[j] = P::template load<true>(static_cast<const char*>(a.rows) + (at < 0 ? 0 : at) * a.ld_rows * P::ES, base,
                                      lane, a.H);
      }
#pragma unroll
      for (int j = 0; j < J; ++j) {
        if (__builtin_amdgcn_readlane(p, j0 + j) < 0) continue;
        const float wj = lane_of(w, j0 + j);
        float f[8];
        P::widen(r[j], f);
#pragma unroll
        for (int q = 0; q < 8; ++q) y[q] = fmaf(wj, f[q], y[q]);
      }
    }
    P::store(static_cast<char*>(a.y) + t * a.H * P::ES, base, lane, a.H, y);
  }
}

// W wavefronts per token take the pieces in turn, J places at a time, so that dy is read once for all of them and J
// rows' loads are in flight; the dot products' parts meet in LDS, in the order of the wavefronts.  One wavefront does
// for short rows (100000 tokens of 2 x 256, quantised: 311 -> 68 us), sixteen share few tokens (one of 8 x 7168: 8.5
// -> 5.5 us).
// DW: dweights are asked for (the rows are read).
template <bool BF16, bool QUANT, bool DW, int J, int W>
__global__ void __launch_bounds__(W == 1 ? kThreads : W * 64) combine_backward_kernel(CombineGradArgs a) {
  constexpr int TOKENS = W == 1 ? kPerGroup : 1;  // of a workgroup
  using P = Piece<BF16>;
  using O = Octet<BF16>;
  __shared__ float part[W][J];
  const int lane = threadIdx.x & 63, id = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wave = W == 1 ? 0 : id;
  const int64_t pieces = (a.H + 511) / 512, G = a.H / 128;
  // QUANT: a lane's octet of the group g = base / 128 + lane / 16; groups past the row's end read the first
  auto load = [&](auto nt, const void* row, int64_t base) {
    if constexpr (QUANT) {
      const int64_t g = base / 128 + (lane >> 4);
      return O::template load<decltype(nt)::value>(static_cast<const char*>(row) + (g < G ? g : 0) * 128 * O::ES,
                                                   lane & 15);
    } else {
      return P::template load<decltype(nt)::value>(row, base, lane, a.H);
    }
  };
  auto widen = [&](const auto& raw, float (&f)[8], int64_t base) {
    if constexpr (QUANT) {
      O::widen(raw, f);
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (base / 128 + (lane >> 4) >= G) f[q] = 0.0f;
    } else {
      P::widen(raw, f);
      P::cut(f, base, lane, a.H);
    }
  };
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * TOKENS + (W == 1 ? id : 0); t < a.T;
       t += static_cast<int64_t>(gridDim.x) * TOKENS) {
    const char* dy = static_cast<const char*>(a.dy) + t * a.ld_dy * P::ES;
    int p = lane < a.k ? a.positions[t * a.k + lane] : -1;
    const float w = lane < a.k ? (a.weights ? a.weights[t * a.k + lane] : 1.0f) : 0.0f;
    if (p >= a.R) p = -1;
    for (int j0 = 0; j0 < a.k; j0 += J) {
      float dot[J];
#pragma unroll
      for (int j = 0; j < J; ++j) dot[j] = 0.0f;
      for (int64_t piece = wave; piece < pieces; piece += W) {
        const int64_t base = piece * 512;
        decltype(load(std::true_type{}, dy, base)) r[DW ? J : 1];
        const auto rd = load(std::false_type{}, dy, base);
        if constexpr (DW) {
#pragma unroll
          for (int j = 0; j < J; ++j) {
            const int at = __builtin_amdgcn_readlane(p, j0 + j);
            r[j] = load(std::true_type{},
                        static_cast<const char*>(a.rows) + (at < 0 ? 0 : at) * a.ld_rows * P::ES, base);
          }
        }
        float d[8];
        widen(rd, d, base);
#pragma unroll
        for (int j = 0; j < J; ++j) {
          const int64_t at = __builtin_amdgcn_readlane(p, j0 + j);
          if (at < 0) continue;
          if constexpr (DW) {
            float f[8];
            widen(r[j], f, base);
#pragma unroll
            for (int q = 0; q < 8; ++q) dot[j] = fmaf(d[q], f[q], dot[j]);
          }
          if (!a.drows) continue;
          const float wj = lane_of(w, j0 + j);
          float o[8];
#pragma unroll
          for (int q = 0; q < 8; ++q) o[q] = d[q] * wj;
          if constexpr (QUANT) {
            const int64_t g = base / 128 + (lane >> 4);
            float s, inv;
            group_scale(a.pow2, group_amax(o), s, inv);
            if (g < G) {
              O::store_codes(static_cast<uint8_t*>(a.drows) + at * a.H + g * 128, lane & 15, o, inv);
              if ((lane & 15) == 0) a.scales[at * G + g] = s;
            }
          } else {
            P::template store<true>(static_cast<char*>(a.drows) + at * a.H * P::ES, base, lane, a.H, o);
          }
        }
      }
      if constexpr (DW) {
        float mine = 0.0f;  // lane j: the wavefront's part of dot j
#pragma unroll
        for (int j = 0; j < J; ++j) {
          const float v = sum64(dot[j]);
          if (lane == j) mine = v;
        }
        if constexpr (W > 1) {
          if (lane < J) part[wave][lane] = mine;
          __syncthreads();
          if (wave == 0 && lane < J) {
            mine = part[0][lane];
#pragma unroll
            for (int q = 1; q < W; ++q) mine += part[q][lane];
          }
          __syncthreads();
        }
        if (wave == 0 && lane < J && j0 + lane < a.k) a.dw[t * a.k + j0 + lane] = mine;
      }
    }
  }
}

unsigned blocks(int64_t n) { return static_cast<unsigned>(n < kMostBlocks ? n : kMostBlocks); }

}  // namespace

hipError_t launch_combine(const CombineArgs& args, hipStream_t s) {
  CombineArgs a = args;
  if (a.R == 0) a.k = 0;  // (no row to read in a place's stead)
  const int64_t pieces = (a.H + 511) / 512;
  const dim3 grid(blocks((a.T * pieces + kPerGroup - 1) / kPerGroup));
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, dim3(kThreads), 0, s, a, pieces);
    return hipGetLastError();
  };
  if (a.bf16)
    return a.k <= 2   ? go(combine_kernel<true, 2>)
           : a.k <= 4 ? go(combine_kernel<true, 4>)
                      : go(combine_kernel<true, 8>);
  return a.k <= 2 ? go(combine_kernel<false, 2>) : go(combine_kernel<false, 4>);
}

hipError_t launch_combine_backward(const CombineGradArgs& args, hipStream_t s) {
  CombineGradArgs a = args;
  if (a.H == 0) a.drows = nullptr;
  if (a.R == 0) {  // no row to read in a place's stead, and none to write: dweights are zero
    a.rows = a.dy;
    a.ld_rows = 0;
    a.drows = nullptr;
  }
  const int64_t pieces = (a.H + 511) / 512;
  // Wavefronts per token: one for rows of one piece, sixteen where the tokens are fewer than the compute units.
  const int w = pieces <= 1 ? 1 : a.T <= 128 ? 16 : 4;
  auto form = [&](auto bf16, auto quant, auto dw) {
    constexpr bool BF16 = decltype(bf16)::value, QUANT = decltype(quant)::value, DW = decltype(dw)::value;
    auto go = [&](auto j) {
      constexpr int J = decltype(j)::value;
      const dim3 grid(blocks(w == 1 ? (a.T + kPerGroup - 1) / kPerGroup : a.T));
      if (w == 1)
        hipLaunchKernelGGL((combine_backward_kernel<BF16, QUANT, DW, J, 1>), grid, dim3(kThreads), 0, s, a);
      else if (w == 4)
        hipLaunchKernelGGL((combine_backward_kernel<BF16, QUANT, DW, J, 4>), grid, dim3(256), 0, s, a);
      else
        hipLaunchKernelGGL((combine_backward_kernel<BF16, QUANT, DW, J, 16>), grid, dim3(1024), 0, s, a);
    };
    if (a.k <= 2)
      go(std::integral_constant<int, 2>{});
    else if (a.k <= 4 || !BF16)  // (an fp32 piece takes twice the registers)
      go(std::integral_constant<int, 4>{});
    else
      go(std::integral_constant<int, 8>{});
    return hipGetLastError();
  };
  auto outputs = [&](auto bf16, auto quant) {
    return a.dw ? form(bf16, quant, std::true_type{}) : form(bf16, quant, std::false_type{});
  };
  if (a.scales)
    return a.bf16 ? outputs(std::true_type{}, std::true_type{}) : outputs(std::false_type{}, std::true_type{});
  return a.bf16 ? outputs(std::true_type{}, std::false_type{}) : outputs(std::false_type{}, std::false_type{});
}

}  // namespace fp8fg
