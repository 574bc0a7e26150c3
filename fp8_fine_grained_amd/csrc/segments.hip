// Row segments of chosen experts: a stable counting sort of n entries by expert.
//
// A workgroup takes a run of consecutive entries, each of its wavefronts a part of it, 64
// entries at a time.  An entry's place among the 64 is the number of earlier lanes with the
// same expert, found by ballots over the bits of the expert's number; counts per wavefront
// and expert are kept in LDS, and each wavefront's start in a segment is the sum of the
// counts before it.  No atomics between wavefronts, so the order is the entries' own.
// With more entries than one workgroup takes, a first launch counts every workgroup's
// entries per expert, and each workgroup of the second sums the table (all of it for the
// segments' starts, the rows before its own for its own).
// Entries of no local expert form a last bin of their own behind the segments.
// Bound by its dependent steps, not by its few bytes: 8 entries take 3.7 us, 65536 over 256 experts 4 us to count
// and 8 us to place.
#include <type_traits>

#include "launch.h"

namespace fp8fg {
namespace {

constexpr int kFewWaves = 8, kFewRounds = 2;      // 1024 entries: the workgroups of many, or a single small one
constexpr int kManyWaves = 16, kManyRounds = 5;   // 5120 entries: the most of a single workgroup (8192: 16 us, not 12)
constexpr int64_t kFewRun = kFewWaves * kFewRounds * 64, kManyRun = kManyWaves * kManyRounds * 64;
constexpr int64_t kMostGroups = 1024;             // (longer inputs: longer runs)

// Entries of a workgroup when there are several.
int64_t run_length(int64_t n) { return ((n + kMostGroups - 1) / kMostGroups + kFewRun - 1) / kFewRun * kFewRun; }

// A wavefront's entries begin + 64 r + lane of r = 0 .. R - 1: their bins (-1 past `end`), all loaded together.
template <int R>
__device__ __forceinline__ void load_bins(const SegmentArgs& a, int64_t begin, int64_t end, int (&bin)[R]) {
  const int lane = threadIdx.x & 63;
  int32_t e[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int64_t i = begin + 64 * r + lane;
    e[r] = a.experts[i < end ? i : end - 1];
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int64_t g = static_cast<int64_t>(e[r]) - a.first;
    bin[r] = g >= 0 && g < a.G ? static_cast<int>(g) : a.G;
    if (begin + 64 * r + lane >= end) bin[r] = -1;
  }
}
// Lanes of the wavefront with the same bin (0 for a lane without an entry).
__device__ __forceinline__ uint64_t same_bin(int bin, int bits) {
  uint64_t m = __ballot(bin >= 0);
  for (int b = 0; b < bits; ++b) {
    const uint64_t v = __ballot((bin >> b) & 1);
    m &= (bin >> b) & 1 ? v : ~v;
  }
  return bin >= 0 ? m : 0;
}
// Lanes before this one in m.
__device__ __forceinline__ int rank_in(uint64_t m) {
  return __builtin_amdgcn_mbcnt_hi(static_cast<uint32_t>(m >> 32),
                                   __builtin_amdgcn_mbcnt_lo(static_cast<uint32_t>(m), 0));
}
__device__ __forceinline__ void wave_fence() { __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront"); }

// The lanes with the same bin, for every round that holds entries.
template <int R>
__device__ __forceinline__ void match(const int (&bin)[R], int64_t begin, int64_t end, int bits, uint64_t (&m)[R]) {
#pragma unroll
  for (int r = 0; r < R; ++r) m[r] = begin + 64 * r < end ? same_bin(bin[r], bits) : 0;
}
// Adds a wavefront's entries to its counts.
template <int R>
__device__ __forceinline__ void count(const int (&bin)[R], const uint64_t (&m)[R], int32_t* c) {
#pragma unroll
  for (int r = 0; r < R; ++r) {
    if (m[r] != 0 && rank_in(m[r]) == 0) c[bin[r]] += __popcll(m[r]);
    wave_fence();
  }
}

// counts[workgroup][bin]
__global__ void __launch_bounds__(kFewWaves * 64) count_kernel(SegmentArgs a, int64_t run, int bits) {
  __shared__ int32_t c[kFewWaves][kSegmentMaxG + 1];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t part = run / kFewWaves;
  const int64_t begin = blockIdx.x * run + wave * part, end = begin + part < a.n ? begin + part : a.n;
  for (int g = lane; g <= a.G; g += 64) c[wave][g] = 0;
  wave_fence();
  for (int64_t i = begin; i < end; i += kFewRounds * 64) {
    int bin[kFewRounds];
    uint64_t m[kFewRounds];
    load_bins(a, i, end, bin);
    match(bin, i, end, bits, m);
    count(bin, m, c[wave]);
  }
  __syncthreads();
  for (int g = threadIdx.x; g <= a.G; g += kFewWaves * 64) {
    int32_t v = 0;
#pragma unroll
    for (int w = 0; w < kFewWaves; ++w) v += c[w][g];
    a.counts[blockIdx.x * (a.G + 1) + g] = v;
  }
}

// WAVES wavefronts with R rounds at a time; ONE: a single workgroup, without the table.
template <int WAVES, int R, bool ONE>
__global__ void __launch_bounds__(WAVES * 64) place_kernel(SegmentArgs a, int64_t run, int bits) {
  __shared__ int32_t at[WAVES][kSegmentMaxG + 1];  // counts, then where the wavefront's next entry of a bin goes
  __shared__ int32_t start[kSegmentMaxG + 1];
  __shared__ int32_t base[ONE ? 1 : kSegmentMaxG + 1];
  __shared__ int32_t chunk[(kSegmentMaxG + 64) / 64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int bins = a.G + 1;
  const int64_t part = run / WAVES;
  const int64_t begin = blockIdx.x * run + wave * part, end = begin + part < a.n ? begin + part : a.n;
  for (int g = lane; g < bins; g += 64) at[wave][g] = 0;
  int bin[R];           // of the first R * 64 entries, all of them but for very long inputs
  uint64_t same[R];
  if (begin < end) load_bins(a, begin, end, bin);
  // The table's sums: entries of all workgroups, and of those before this one.  (Their loads go out with the entries'
  // own: one latency instead of two.)
  if constexpr (!ONE) {
    const int groups = gridDim.x, mine = blockIdx.x;
    for (int g = threadIdx.x; g < bins; g += WAVES * 64) {
      int32_t before = 0, total = 0;
      for (int b0 = 0; b0 < groups; b0 += 16) {
        int32_t v[16];
#pragma unroll
        for (int q = 0; q < 16; ++q) v[q] = a.counts[static_cast<int64_t>(b0 + q < groups ? b0 + q : 0) * bins + g];
#pragma unroll
        for (int q = 0; q < 16; ++q) {
          const int32_t c = b0 + q < groups ? v[q] : 0;
          total += c;
          before += b0 + q < mine ? c : 0;
        }
      }
      start[g] = total;
      base[g] = before;
    }
  }
  wave_fence();
  match(bin, begin, end, bits, same);
  count(bin, same, at[wave]);
  for (int64_t i = begin + R * 64; i < end; i += R * 64) {
    int more[R];
    uint64_t m[R];
    load_bins(a, i, end, more);
    match(more, i, end, bits, m);
    count(more, m, at[wave]);
  }
  __syncthreads();
  for (int g = threadIdx.x; g < bins; g += WAVES * 64) {
    // the wavefronts' counts become the counts before them
    int32_t before = ONE ? 0 : base[g];
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
      const int32_t c = at[w][g];
      at[w][g] = before;
      before += c;
    }
    if constexpr (ONE) start[g] = before;
  }
  __syncthreads();
  // exclusive sums of the bins' totals, a chunk of 64 per wavefront, then over the chunks
  for (int g0 = wave * 64; g0 < bins; g0 += WAVES * 64) {
    const int g = g0 + lane;
    const int32_t v = g < bins ? start[g] : 0;
    int32_t incl = v;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int32_t o = __shfl_up(incl, d);
      if (lane >= d) incl += o;
    }
    if (g < bins) start[g] = incl - v;
    if (lane == 63) chunk[g0 / 64] = incl;
  }
  __syncthreads();
  for (int g = threadIdx.x; g < bins; g += WAVES * 64) {
    int32_t v = start[g];
    for (int c = 0; c < g / 64; ++c) v += chunk[c];
    if (blockIdx.x == 0) a.offsets[g] = v;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) at[w][g] += v;
  }
  __syncthreads();
  for (int64_t i = begin; i < end; i += R * 64) {
    if (i > begin) {
      load_bins(a, i, end, bin);
      match(bin, i, end, bits, same);
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (i + 64 * r >= end) break;
      const uint64_t m = same[r];
      const int rank = rank_in(m);
      const int64_t k = i + 64 * r + lane;
      if (m != 0) {
        const int32_t p = at[wave][bin[r]] + rank;
        a.positions[k] = bin[r] < a.G ? p : -1;
        a.row_index[p] = bin[r] < a.G ? static_cast<int32_t>(static_cast<uint32_t>(k) / static_cast<uint32_t>(a.k)) : 0;
      }
      wave_fence();
      if (m != 0 && rank == 0) at[wave][bin[r]] += __popcll(m);
      wave_fence();
    }
  }
}

__global__ void zero_offsets_kernel(int32_t* offsets, int n) {
  for (int i = threadIdx.x; i < n; i += 64) offsets[i] = 0;
}

}  // namespace

int64_t segments_workspace(int64_t n, int64_t G) {
  if (n <= kManyRun) return 0;
  const int64_t run = run_length(n);
  return (n + run - 1) / run * (G + 1);
}

hipError_t launch_segments(const SegmentArgs& a, hipStream_t s) {
  if (a.n == 0) {
    hipLaunchKernelGGL(zero_offsets_kernel, dim3(1), dim3(64), 0, s, a.offsets, a.G + 1);
    return hipGetLastError();
  }
  int bits = 0;
  while (a.G >> bits) ++bits;
  // (a single workgroup's wavefronts share the entries evenly)
  auto shared = [&](int64_t waves) { return (a.n + waves * 64 - 1) / (waves * 64) * waves * 64; };
  if (a.n <= kFewRun) {
    hipLaunchKernelGGL((place_kernel<kFewWaves, kFewRounds, true>), dim3(1), dim3(kFewWaves * 64), 0, s, a,
                       shared(kFewWaves), bits);
    return hipGetLastError();
  }
  if (a.n <= kManyRun) {
    hipLaunchKernelGGL((place_kernel<kManyWaves, kManyRounds, true>), dim3(1), dim3(kManyWaves * 64), 0, s, a,
                       shared(kManyWaves), bits);
    return hipGetLastError();
  }
  const int64_t run = run_length(a.n);
  const dim3 grid(static_cast<unsigned>((a.n + run - 1) / run)), block(kFewWaves * 64);
  hipLaunchKernelGGL(count_kernel, grid, block, 0, s, a, run, bits);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((place_kernel<kFewWaves, kFewRounds, false>), grid, block, 0, s, a, run, bits);
  return hipGetLastError();
}

}  // namespace fp8fg
