// Row segments of chosen experts: a stable counting sort of n entries by expert.
//
// A unit of the sort is one wavefront's run of consecutive entries.  The first pass counts
// every unit's entries per expert; the second sums those counts over the units (all of them
// for the segments' starts, the earlier ones for the unit's own), and each unit then places
// its entries in order, 64 at a time: an entry's place among the 64 is the number of earlier
// lanes with the same expert, found by ballots over the bits of the expert's number.  No
// atomics between wavefronts, so the order is the entries' own.
// Entries of no local expert form a last bin of their own behind the segments.
#include "launch.h"

namespace fp8fg {
namespace {

constexpr int kUnitWaves = 4;                        // units of a workgroup
constexpr int64_t kUnit = 512;                       // entries of a unit
constexpr int64_t kMostUnits = 1024;                 // (longer inputs take longer units)

int64_t unit_length(int64_t n) {
  const int64_t u = (n + kMostUnits - 1) / kMostUnits;
  return u <= kUnit ? kUnit : (u + 63) / 64 * 64;
}

__device__ __forceinline__ int bin_of(const SegmentArgs& a, int64_t i) {
  const int64_t e = static_cast<int64_t>(a.experts[i]) - a.first;
  return e >= 0 && e < a.G ? static_cast<int>(e) : a.G;
}
// Lanes of the wavefront with the same bin (0 for a lane that takes no part).
__device__ __forceinline__ uint64_t same_bin(int bin, bool live, int bits) {
  uint64_t m = __ballot(live);
  for (int b = 0; b < bits; ++b) {
    const uint64_t v = __ballot((bin >> b) & 1);
    m &= (bin >> b) & 1 ? v : ~v;
  }
  return live ? m : 0;
}

// counts[unit][bin]
__global__ void __launch_bounds__(kUnitWaves * 64) count_kernel(SegmentArgs a, int64_t unit, int bits) {
  __shared__ int32_t c[kUnitWaves][kSegmentMaxG + 1];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t u = static_cast<int64_t>(blockIdx.x) * kUnitWaves + wave;
  for (int g = lane; g <= a.G; g += 64) c[wave][g] = 0;
  __syncthreads();
  const int64_t begin = u * unit, end = begin + unit < a.n ? begin + unit : a.n;
  for (int64_t i = begin + lane; i - lane < end; i += 64) {
    const bool live = i < end;
    const int bin = live ? bin_of(a, i) : 0;
    const uint64_t m = same_bin(bin, live, bits);
    if (live && __ffsll(static_cast<unsigned long long>(m)) - 1 == lane) c[wave][bin] += __popcll(m);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  }
  if (begin < a.n)
    for (int g = lane; g <= a.G; g += 64) a.counts[u * (a.G + 1) + g] = c[wave][g];
}

__global__ void __launch_bounds__(kUnitWaves * 64) place_kernel(SegmentArgs a, int64_t unit, int bits) {
  __shared__ int32_t at[kUnitWaves][kSegmentMaxG + 1];  // where the unit's next entry of a bin goes
  __shared__ int32_t start[kSegmentMaxG + 1];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int bins = a.G + 1;
  const int64_t units = (a.n + unit - 1) / unit;
  const int64_t u0 = static_cast<int64_t>(blockIdx.x) * kUnitWaves;
  for (int g = threadIdx.x; g < bins; g += kUnitWaves * 64) {
    int32_t total = 0;
    for (int64_t u = 0; u < units; ++u) {
      if (u >= u0 && u < u0 + kUnitWaves) at[u - u0][g] = total;
      total += a.counts[u * bins + g];
    }
    start[g] = total;
  }
  __syncthreads();
  if (wave == 0) {  // exclusive sums of the bins' totals
    int32_t before = 0;
    for (int g0 = 0; g0 < bins; g0 += 64) {
      const int g = g0 + lane;
      const int32_t v = g < bins ? start[g] : 0;
      int32_t incl = v;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const int32_t o = __shfl_up(incl, d);
        if (lane >= d) incl += o;
      }
      if (g < bins) {
        start[g] = before + incl - v;
        if (blockIdx.x == 0) a.offsets[g] = before + incl - v;
      }
      before += __shfl(incl, 63);
    }
  }
  __syncthreads();
  const int64_t begin = (u0 + wave) * unit, end = begin + unit < a.n ? begin + unit : a.n;
  for (int64_t i = begin + lane; i - lane < end; i += 64) {
    const bool live = i < end;
    const int bin = live ? bin_of(a, i) : 0;
    const uint64_t m = same_bin(bin, live, bits);
    const int rank = __popcll(m & ((uint64_t(1) << lane) - 1));
    if (live) {
      const int32_t p = start[bin] + at[wave][bin] + rank;
      a.positions[i] = bin < a.G ? p : -1;
      a.row_index[p] = bin < a.G ? static_cast<int32_t>(static_cast<uint32_t>(i) / static_cast<uint32_t>(a.k)) : 0;
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    if (live && rank == 0) at[wave][bin] += __popcll(m);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  }
}

__global__ void zero_offsets_kernel(int32_t* offsets, int n) {
  for (int i = threadIdx.x; i < n; i += 64) offsets[i] = 0;
}

}  // namespace

int64_t segments_workspace(int64_t n, int64_t G) {
  const int64_t unit = unit_length(n);
  return (n + unit - 1) / unit * (G + 1);
}

hipError_t launch_segments(const SegmentArgs& a, hipStream_t s) {
  if (a.n == 0) {
    hipLaunchKernelGGL(zero_offsets_kernel, dim3(1), dim3(64), 0, s, a.offsets, a.G + 1);
    return hipGetLastError();
  }
  const int64_t unit = unit_length(a.n), units = (a.n + unit - 1) / unit;
  int bits = 0;
  while (a.G >> bits) ++bits;
  const dim3 grid(static_cast<unsigned>((units + kUnitWaves - 1) / kUnitWaves)), block(kUnitWaves * 64);
  hipLaunchKernelGGL(count_kernel, grid, block, 0, s, a, unit, bits);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(place_kernel, grid, block, 0, s, a, unit, bits);
  return hipGetLastError();
}

}  // namespace fp8fg
