// Global norm over many gradients, and clipping by it.
//
//     norm = sqrt(sum over all tensors of g^2),
//     c = norm <= max_norm ? 1 : max_norm / norm,   out = c * g.
//
// Squares are summed in 64 bits: 1e8 values lose nothing to rounding, and no
// finite fp32 gradient overflows or vanishes when squared.  Sums are taken in a
// fixed order (per thread, per workgroup, over the workgroups), so the norm is
// the same on every run.  HBM is the bound: every gradient is read twice, since
// no output can be written before the whole norm is known.
//
// Tensors come as kernel arguments, kGradBatch per launch, so nothing has to be
// copied to the device first.  A tensor is cut into chunks of kChunk elements;
// workgroups walk the chunks of all tensors of their launch.
#include "launch.h"
#include "lanes.h"

namespace fp8fg {
namespace {

constexpr int kChunk = 8192;  // elements, 32 per thread

struct Batch {
  const void* in[kGradBatch];
  int64_t count[kGradBatch];
  int first[kGradBatch + 1];  // first chunk of each tensor; [n] is the number of chunks
  bool bf16[kGradBatch];
  int n;
};
struct Outs {
  void* out[kGradBatch];
};

// The tensor that chunk c belongs to (first[] is non-decreasing, first[0] == 0).
__device__ __forceinline__ int tensor_of(const Batch& b, int c) {
  int lo = 0, hi = b.n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (b.first[mid] <= c)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// Sixteen bytes at any element address: global memory takes them unaligned, so
// a view into a flat gradient buffer costs no scalar path.
typedef u32x4 u32x4_any __attribute__((aligned(2)));

// The 16-byte pieces of a chunk that lie whole inside it, PIECES per thread, as
// raw registers; the rest of the chunk is left to the element loop.
template <int PIECES>
__device__ __forceinline__ void load_pieces(const char* p, int whole, u32x4 (&u)[PIECES]) {
#pragma unroll
  for (int i = 0; i < PIECES; ++i) {
    const int j = threadIdx.x + 256 * i;
    u[i] = u32x4{0u, 0u, 0u, 0u};
    if (j < whole) u[i] = *reinterpret_cast<const u32x4_any*>(p + 16 * j);
  }
}

__device__ __forceinline__ float element(const void* p, bool bf16, int64_t i) {
  return bf16 ? __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(p)[i]) << 16)
              : static_cast<const float*>(p)[i];
}

// Sum over the workgroup's 256 threads, the same value in every thread.
__device__ __forceinline__ double block_sum(double v, double* lds) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d);
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  return (lds[0] + lds[1]) + (lds[2] + lds[3]);
}

__global__ void __launch_bounds__(256) grad_square_kernel(Batch b, double* __restrict__ partial) {
  __shared__ double lds[4];
  const int chunks = b.first[b.n];
  double sum = 0.0;
  for (int c = blockIdx.x; c < chunks; c += gridDim.x) {
    const int k = tensor_of(b, c);
    const int64_t i0 = static_cast<int64_t>(c - b.first[k]) * kChunk;
    const int64_t left = b.count[k] - i0;
    const bool bf16 = b.bf16[k];
    const int n = static_cast<int>(left < kChunk ? left : kChunk);
    const char* p = static_cast<const char*>(b.in[k]) + i0 * (bf16 ? 2 : 4);
    if (bf16) {
      u32x4 u[4];
      load_pieces(p, n / 8, u);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const double lo = __uint_as_float(u[i][e] << 16), hi = __uint_as_float(u[i][e] & 0xFFFF0000u);
          sum = fma(lo, lo, sum);
          sum = fma(hi, hi, sum);
        }
    } else {
      u32x4 u[8];
      load_pieces(p, n / 4, u);
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const double d = __uint_as_float(u[i][e]);
          sum = fma(d, d, sum);
        }
    }
    // the elements past the last whole piece: fewer than 8
    const int i = (bf16 ? n & ~7 : n & ~3) + threadIdx.x;
    if (i < n) {
      const double d = element(p, bf16, i);
      sum = fma(d, d, sum);
    }
  }
  sum = block_sum(sum, lds);
  if (threadIdx.x == 0) partial[blockIdx.x] = sum;
}

// The norm from all partial sums, in the same order in every workgroup.
__device__ __forceinline__ float norm_of(const double* __restrict__ partial, int parts, double* lds) {
  double sum = 0.0;
  for (int i = threadIdx.x; i < parts; i += 256) sum += partial[i];
  return static_cast<float>(sqrt(block_sum(sum, lds)));
}

__global__ void __launch_bounds__(256) grad_norm_kernel(const double* __restrict__ partial, int parts,
                                                        float* __restrict__ norm) {
  __shared__ double lds[4];
  const float v = norm_of(partial, parts, lds);
  if (threadIdx.x == 0) *norm = v;
}

// Every workgroup forms the norm from the partial sums itself (a few KB from
// L2), which saves a launch between the two passes.
__global__ void __launch_bounds__(256) grad_clip_kernel(Batch b, Outs o, const double* __restrict__ partial, int parts,
                                                        float max_norm, float* __restrict__ norm) {
  __shared__ double lds[4];
  const float total = norm_of(partial, parts, lds);
  if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = total;
  // a norm that is not a number scales everything to NaN: it must not pass unseen
  const float c = total <= max_norm ? 1.0f : max_norm / total;
  const int chunks = b.first[b.n];
  for (int j = blockIdx.x; j < chunks; j += gridDim.x) {
    const int chunk = chunks - 1 - j;
    const int k = tensor_of(b, chunk);
    const int64_t i0 = static_cast<int64_t>(chunk - b.first[k]) * kChunk;
    const int64_t left = b.count[k] - i0;
    const bool bf16 = b.bf16[k];
    const int n = static_cast<int>(left < kChunk ? left : kChunk);
    const char* p = static_cast<const char*>(b.in[k]) + i0 * (bf16 ? 2 : 4);
    char* q = static_cast<char*>(o.out[k]) + i0 * (bf16 ? 2 : 4);
    if (c == 1.0f && p == q) continue;  // nothing to change
    if (bf16) {
      u32x4 u[4];
      load_pieces(p, n / 8, u);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          u[i][e] = pack_bf16(__uint_as_float(u[i][e] << 16) * c, __uint_as_float(u[i][e] & 0xFFFF0000u) * c);
        const int j = threadIdx.x + 256 * i;
        if (j < n / 8) *reinterpret_cast<u32x4_any*>(q + 16 * j) = u[i];
      }
    } else {
      u32x4 u[8];
      load_pieces(p, n / 4, u);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
#pragma unroll
        for (int e = 0; e < 4; ++e) u[i][e] = __float_as_uint(__uint_as_float(u[i][e]) * c);
        const int j = threadIdx.x + 256 * i;
        if (j < n / 4) *reinterpret_cast<u32x4_any*>(q + 16 * j) = u[i];
      }
    }
    const int i = (bf16 ? n & ~7 : n & ~3) + threadIdx.x;
    if (i < n) {
      const float d = element(p, bf16, i) * c;
      if (bf16)
        reinterpret_cast<uint16_t*>(q)[i] = static_cast<uint16_t>(pack_bf16(d, 0.0f) & 0xFFFFu);
      else
        reinterpret_cast<float*>(q)[i] = d;
    }
  }
}

// The tensors [t0, t0 + kGradBatch) of the list as kernel arguments.
void fill(const GradList& g, int64_t t0, Batch& b, Outs& o) {
  b.n = static_cast<int>(g.n - t0 < kGradBatch ? g.n - t0 : kGradBatch);
  b.first[0] = 0;
  for (int i = 0; i < b.n; ++i) {
    const int64_t k = t0 + i;
    b.in[i] = g.grads[k];
    b.count[i] = g.counts[k];
    o.out[i] = g.outs ? g.outs[k] : nullptr;
    b.bf16[i] = g.dtypes[k] == 1;  // FP8FG_BF16
    b.first[i + 1] = b.first[i] + static_cast<int>((g.counts[k] + kChunk - 1) / kChunk);
  }
}

}  // namespace

hipError_t launch_grad_norm(const GradList& g, float max_norm, float* norm, double* partial, hipStream_t s) {
  int parts = 0;
  Batch b{};
  Outs o{};
  for (int64_t t0 = 0; t0 < g.n; t0 += kGradBatch) {
    fill(g, t0, b, o);
    const int blocks = b.first[b.n] < kGradPartials ? b.first[b.n] : kGradPartials;
    if (blocks == 0) continue;  // empty tensors only
    hipLaunchKernelGGL(grad_square_kernel, dim3(blocks), dim3(256), 0, s, b, partial + parts);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    parts += blocks;
  }
  if (!g.outs || parts == 0) {
    hipLaunchKernelGGL(grad_norm_kernel, dim3(1), dim3(256), 0, s, partial, parts, norm);
    return hipGetLastError();
  }
  for (int64_t t0 = 0; t0 < g.n; t0 += kGradBatch) {
    fill(g, t0, b, o);
    const int blocks = b.first[b.n] < 2 * kGradPartials ? b.first[b.n] : 2 * kGradPartials;
    if (blocks == 0) continue;
    hipLaunchKernelGGL(grad_clip_kernel, dim3(blocks), dim3(256), 0, s, b, o, partial, parts, max_norm, norm);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    norm = nullptr;  // written once
  }
  return hipSuccess;
}

}  // namespace fp8fg
