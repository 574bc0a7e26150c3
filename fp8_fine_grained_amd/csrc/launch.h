// Internal launcher interface between the C-ABI layer (capi.cpp) and the
// HIP kernels.  Arguments reaching these functions have been validated.
#pragma once
#include <hip/hip_runtime.h>
#include <cstdint>

namespace fp8fg {

// pow2: power-of-two (E8M0) group scales instead of amax/448.
// 1x128 quantisation, row-contiguous input (stride_k == 1).
hipError_t launch_quant_act_rows(const void* x, bool bf16, bool pow2, int64_t M, int64_t K, int64_t ld,
                                 uint8_t* q, float* scales, hipStream_t s);
// 1x128 quantisation along K of a column-contiguous input (stride_m == 1):
// x is physically [K, ld] row-major, element (m, k) at k*ld + m.
hipError_t launch_quant_act_cols(const void* x, bool bf16, bool pow2, int64_t M, int64_t K, int64_t ld,
                                 uint8_t* q, float* scales, hipStream_t s);
// One scale for the whole row-contiguous [M, K] tensor, written into all
// n_scales entries of `scales` (M * K/128 or (M/128) * (K/128) of them).
hipError_t launch_quant_per_tensor(const void* x, bool bf16, int64_t M, int64_t K, int64_t ld, uint8_t* q,
                                   float* scales, int64_t n_scales, hipStream_t s);
// 128x128 quantisation.
hipError_t launch_quant_weight(const void* w, bool bf16, bool pow2, int64_t N, int64_t K, int64_t ld,
                               uint8_t* q, float* scales, hipStream_t s);
// 128x128 quantisation of w and 1x128 quantisation of the row-contiguous x in one
// launch (either part may be empty: M == 0 or N == 0).
hipError_t launch_quant_act_weight(const void* x, bool x_bf16, int64_t M, int64_t K_x, int64_t ld_x, uint8_t* q_x,
                                   float* s_x, const void* w, bool w_bf16, int64_t N, int64_t K_w, int64_t ld_w,
                                   uint8_t* q_w, float* s_w, bool pow2, hipStream_t s);
// 128x128 quantisation writing q [N,K] and the transposed q_t [K,N] (+ scales, scales_t).
hipError_t launch_quant_weight_dual(const void* w, bool bf16, bool pow2, int64_t N, int64_t K, int64_t ld,
                                    uint8_t* q, float* scales, uint8_t* qt, float* scales_t, hipStream_t s);

struct GemmArgs {
  const uint8_t* a;
  const float* sa;
  const uint8_t* b;
  const float* sb;
  void* y;
  const int32_t* offsets;  // grouped only
  int64_t M, N, K, G;
  bool row_scales;  // B scales per row (1x128) instead of per 128x128 block
  bool exact;       // exact products (fp16 matrix cores) instead of FP8 MFMA
  bool scaled;      // power-of-two scales applied by the matrix cores (E8M0), FP32 accumulation in the MFMA
  bool y_bf16;
  const int32_t* row_index = nullptr;  // grouped with gather: row r of A is a[row_index[r]]
  int64_t T = 0;                       // rows of a (and sa) when gathering
  float* y_scales = nullptr;           // quantised output: scales [M, N/128] (y = codes [M, N])
  void* gu = nullptr;                  // gated: gate and up values [M, N] (of y's type; bf16 when quantised), or null
  bool gu_bf16 = false;                // gated: gu in bf16 although y is fp32
  bool pow2 = false;                   // gated, quantised: power-of-two scales
};
hipError_t launch_block_gemm(const GemmArgs& g, hipStream_t s);
hipError_t launch_grouped_gemm(const GemmArgs& g, hipStream_t s);
// Grouped GEMM gathering A rows by index (requires fp8_block_kernel_applies).
hipError_t launch_grouped_gemm_gather(const GemmArgs& g, hipStream_t s);

// 256x256-tile FP8-accumulation kernel for 128x128 weight scales (gemm_fp8.hip).
bool fp8_block_kernel_applies(const GemmArgs& g);
hipError_t launch_fp8_block_gemm(const GemmArgs& g, bool grouped, hipStream_t s);
// Dense GEMM writing its output as 1x128-quantised E4M3 codes (g.y) and scales
// (g.y_scales); requires N % 256 == 0, block-scaled B, FP8 or scaled accumulation.
hipError_t launch_fp8_block_gemm_quant(const GemmArgs& g, bool pow2, hipStream_t s);

// Gated pair of products h = g * sigmoid(g) * u (gemm_gated.hip): b holds the N/2
// gate rows and then the N/2 up rows, y is [M, N/2].  Grouped when g.offsets is
// set (rows read through g.row_index, or in order when it is null).  workspace:
// M * N/2 floats for a quantised output of few rows, or null (one kernel, slower
// for few rows); gated_quant_takes_workspace: whether it would be used.
hipError_t launch_gated_gemm(const GemmArgs& g, float* workspace, hipStream_t s);
bool gated_quant_takes_workspace(const GemmArgs& g);

// Work-items that one launch may have along x: HIP counts them in 32 bits.
constexpr int64_t kMaxWorkItems = 0xFFFFFFFF;

// Compute units of the current device (0 if it cannot be asked).
int device_cus();

// Gradient of the gated activation, quantised along its columns (q, s), along
// the tokens (q_t, s_t), and h along the tokens (q_ht, s_ht); each pair may be
// null, the transposed ones need M % 128 == 0 (gated_backward.hip).
struct GatedGradArgs {
  const void* dh;
  const void* gu;
  uint8_t* q;
  float* s;
  uint8_t* q_t;
  float* s_t;
  uint8_t* q_ht;
  float* s_ht;
  int64_t M, I, ld_dh;
  bool bf16, pow2;
};
hipError_t launch_gated_backward(const GatedGradArgs& a, hipStream_t s);

// Residual addition, RMS norm and 1x128 quantisation (norm.hip).
struct NormArgs {
  const void* x;
  const void* r;  // residual, or null
  const void* w;
  void* h;        // x + r in the input type, or null
  void* y;        // the normed rows in the input type, or null
  uint8_t* q;
  float* scales;
  float* rstd;    // or null
  int64_t M, H, ld_x, ld_r;
  float eps;
  bool bf16, w_bf16, pow2;
};
hipError_t launch_rmsnorm_quant(const NormArgs& a, hipStream_t s);

// Its gradient: dx, and the weight's gradient through per-workgroup partials
// [rmsnorm_backward_partials(M, H), H].
struct NormGradArgs {
  const void* dy;
  const void* h;
  const void* dh;  // gradient arriving along the residual stream, or null
  const float* rstd;
  const void* w;
  void* dx;
  float* partial;  // null: no weight gradient
  int64_t M, H, ld_dy, ld_h, ld_dh;
  bool bf16, w_bf16;
};
constexpr int64_t kNormMaxH = 32768;  // a row stays in a workgroup's registers
int64_t rmsnorm_backward_partials(int64_t M, int64_t H);
hipError_t launch_rmsnorm_backward(const NormGradArgs& a, float* dw, hipStream_t s);

// Global gradient norm and clipping (clip.hip).
struct GradList {
  const void* const* grads;
  void* const* outs;  // null: norm only
  const int64_t* counts;
  const int* dtypes;
  int64_t n;
};
constexpr int kGradBatch = 120;        // tensors per launch (kernel arguments)
constexpr int kGradPartials = 1024;    // workgroups, hence partial sums, per launch
hipError_t launch_grad_norm(const GradList& g, float max_norm, float* norm, double* partial, hipStream_t s);

// Routing (route.hip): scores, the k chosen experts of every token and their weights.
struct RouteArgs {
  const void* z;        // logits [T, E], row pitch ld
  const float* bias;    // or null
  const uint8_t* mask;  // or null
  int32_t* experts;
  float* weights;
  float* scores;  // or null
  int64_t T, ld;
  int E, groups, kept, terms, k;
  float scale;
  bool bf16, sigmoid, renormalise;
};
constexpr int kRouteMaxE = 1024, kRouteMaxK = 32, kRouteMaxGroups = 64;
hipError_t launch_route(const RouteArgs& a, hipStream_t s);

struct RouteGradArgs {
  const float* dw;
  const int32_t* experts;
  const void* z;
  const float* ds;  // or null
  void* dz;
  int64_t T, ld;
  int E, k;
  float scale;
  bool bf16, sigmoid, renormalise;
};
hipError_t launch_route_backward(const RouteGradArgs& a, hipStream_t s);

// Row segments of the n = T * k chosen experts (segments.hip): a stable counting sort.
// workspace: segments_workspace(n, G) ints.
struct SegmentArgs {
  const int32_t* experts;
  int32_t* offsets;
  int32_t* row_index;
  int32_t* positions;
  int32_t* counts;  // the workspace
  int64_t n, first;
  int k, G;
};
constexpr int kSegmentMaxG = 1024;
int64_t segments_workspace(int64_t n, int64_t G);
hipError_t launch_segments(const SegmentArgs& a, hipStream_t s);

// Combination of the experts' rows and its gradient (combine.hip).
struct CombineArgs {
  const void* rows;
  const int32_t* positions;
  const float* weights;  // or null: ones
  const void* base;      // or null
  void* y;
  int64_t R, H, ld_rows, ld_base, T;
  int k;
  bool bf16;
};
constexpr int kCombineMaxK = 32;
hipError_t launch_combine(const CombineArgs& a, hipStream_t s);

struct CombineGradArgs {
  const void* dy;
  const void* rows;  // null: no dw
  const int32_t* positions;
  const float* weights;  // or null: ones
  void* drows;           // of dy's type, or codes when scales is set; or null
  float* scales;
  float* dw;  // or null
  int64_t R, H, ld_dy, ld_rows, T;
  int k;
  bool bf16, pow2;
};
hipError_t launch_combine_backward(const CombineGradArgs& a, hipStream_t s);

// 4-bit weights (fp4.hip): their quantisation, and products of few rows with them.
hipError_t launch_fp4_quant(const void* w, bool bf16, int64_t N, int64_t K, int64_t ld, uint8_t* q, uint8_t* scales,
                            hipStream_t s);
struct Fp4Args {
  const void* x;
  const float* sx;  // null: x is bf16
  const uint8_t* w;
  const uint8_t* sw;
  void* y;
  const int32_t* offsets;  // grouped only
  const int32_t* row_index;
  int64_t M, N, K, G, T;  // N: output columns (w has 2N rows when gated)
  bool gated, y_bf16;
};
hipError_t launch_fp4_gemm(const Fp4Args& a, hipStream_t s);

}  // namespace fp8fg
