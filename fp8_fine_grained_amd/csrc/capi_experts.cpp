// C-ABI entry points declared in include/fp8fg_experts.h: argument validation on the
// host, then the launches.  Validation runs before any HIP call.
#include "fp8fg_experts.h"

#include <cmath>
#include <cstdint>
#include <limits>

#include "fp4_shape.h"
#include "launch.h"

namespace {

constexpr int64_t kInt32Max = std::numeric_limits<int32_t>::max();
constexpr int64_t kUint32Max = std::numeric_limits<uint32_t>::max();
constexpr int64_t kInt64Max = std::numeric_limits<int64_t>::max();

bool aligned(const void* p, unsigned a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
int64_t elem_size(int dtype) { return dtype == FP8FG_BF16 ? 2 : 4; }
bool valid_dtype(int d) { return d == FP8FG_F32 || d == FP8FG_BF16; }
bool flag(int v) { return v == 0 || v == 1; }
int hip_status(hipError_t e) { return e == hipSuccess ? FP8FG_OK : FP8FG_ERR_HIP; }

// A row-major operand, `ld` elements between rows, of which `rows` are addressed.
int check_rows(const void* p, int dtype, int64_t rows, int64_t H, int64_t ld) {
  if (!p || ld < H) return FP8FG_ERR_INVALID_ARG;
  if (ld > kInt64Max / 16 / (rows + 1)) return FP8FG_ERR_UNSUPPORTED;
  if (!aligned(p, 16) || (ld * elem_size(dtype)) % 16 != 0) return FP8FG_ERR_MISALIGNED;
  return FP8FG_OK;
}

// What both routing calls take.
int check_route(const void* logits, int dtype, int64_t T, int64_t E, int64_t ld, int score, int64_t k,
                int renormalise, float scale) {
  if (!valid_dtype(dtype) || T < 0 || E < 0 || k < 0 || !flag(renormalise)) return FP8FG_ERR_INVALID_ARG;
  if (score != FP8FG_SCORE_SOFTMAX && score != FP8FG_SCORE_SIGMOID) return FP8FG_ERR_INVALID_ARG;
  if (!std::isfinite(scale)) return FP8FG_ERR_INVALID_ARG;
  if (E < 1 || E > fp8fg::kRouteMaxE || k < 1 || k > fp8fg::kRouteMaxK || k > E || T > kInt32Max)
    return FP8FG_ERR_UNSUPPORTED;
  if (T == 0) return FP8FG_OK;
  if (!logits || ld < E) return FP8FG_ERR_INVALID_ARG;
  if (ld > kInt64Max / 16 / (T + 1)) return FP8FG_ERR_UNSUPPORTED;
  if (!aligned(logits, static_cast<unsigned>(elem_size(dtype)))) return FP8FG_ERR_MISALIGNED;
  return FP8FG_OK;
}

}  // namespace

extern "C" {

int fp8fg_route_experts(const void* logits, int dtype, int64_t T, int64_t E, int64_t ld, const float* bias,
                        const uint8_t* mask, int score, int64_t groups, int64_t groups_kept, int group_terms,
                        int64_t k, int renormalise, float scale, int32_t* experts, float* weights, float* scores,
                        fp8fg_stream_t stream) {
  const int c = check_route(logits, dtype, T, E, ld, score, k, renormalise, scale);
  if (c != FP8FG_OK) return c;
  if (groups < 1 || groups_kept < 1 || groups_kept > groups || (group_terms != 1 && group_terms != 2))
    return FP8FG_ERR_INVALID_ARG;
  if (groups > fp8fg::kRouteMaxGroups || E % groups != 0 || k > groups_kept * (E / groups))
    return FP8FG_ERR_UNSUPPORTED;
  if (groups_kept < groups && group_terms > E / groups) return FP8FG_ERR_UNSUPPORTED;
  if (T == 0) return FP8FG_OK;
  if (!experts || !weights) return FP8FG_ERR_INVALID_ARG;
  if (!aligned(bias, 4) || !aligned(experts, 4) || !aligned(weights, 4) || !aligned(scores, 4))
    return FP8FG_ERR_MISALIGNED;
  fp8fg::RouteArgs a{};
  a.z = logits; a.bias = bias; a.mask = mask; a.experts = experts; a.weights = weights; a.scores = scores;
  a.T = T; a.ld = ld; a.E = static_cast<int>(E); a.groups = static_cast<int>(groups);
  a.kept = static_cast<int>(groups_kept); a.terms = group_terms; a.k = static_cast<int>(k); a.scale = scale;
  a.bf16 = dtype == FP8FG_BF16; a.sigmoid = score == FP8FG_SCORE_SIGMOID; a.renormalise = renormalise == 1;
  return hip_status(fp8fg::launch_route(a, static_cast<hipStream_t>(stream)));
}

int fp8fg_route_experts_backward(const float* dweights, const int32_t* experts, const void* logits, int dtype,
                                 int64_t T, int64_t E, int64_t ld, int score, int64_t k, int renormalise, float scale,
                                 const float* dscores, void* dlogits, fp8fg_stream_t stream) {
  const int c = check_route(logits, dtype, T, E, ld, score, k, renormalise, scale);
  if (c != FP8FG_OK) return c;
  if (T == 0) return FP8FG_OK;
  if (!dweights || !experts || !dlogits) return FP8FG_ERR_INVALID_ARG;
  if (!aligned(dweights, 4) || !aligned(experts, 4) || !aligned(dscores, 4) ||
      !aligned(dlogits, static_cast<unsigned>(elem_size(dtype))))
    return FP8FG_ERR_MISALIGNED;
  fp8fg::RouteGradArgs a{};
  a.dw = dweights; a.experts = experts; a.z = logits; a.ds = dscores; a.dz = dlogits;
  a.T = T; a.ld = ld; a.E = static_cast<int>(E); a.k = static_cast<int>(k); a.scale = scale;
  a.bf16 = dtype == FP8FG_BF16; a.sigmoid = score == FP8FG_SCORE_SIGMOID; a.renormalise = renormalise == 1;
  return hip_status(fp8fg::launch_route_backward(a, static_cast<hipStream_t>(stream)));
}

int64_t fp8fg_expert_segments_workspace(int64_t T, int64_t k, int64_t G) {
  if (T <= 0 || k <= 0 || G <= 0 || G > fp8fg::kSegmentMaxG || T > kInt32Max / k) return 0;
  return fp8fg::segments_workspace(T * k, G) * static_cast<int64_t>(sizeof(int32_t));
}

int fp8fg_expert_segments(const int32_t* experts, int64_t T, int64_t k, int64_t first, int64_t G, int32_t* offsets,
                          int32_t* row_index, int32_t* positions, void* workspace, int64_t workspace_bytes,
                          fp8fg_stream_t stream) {
  if (T < 0 || k < 0 || first < 0 || G < 0) return FP8FG_ERR_INVALID_ARG;
  if (G < 1 || G > fp8fg::kSegmentMaxG || first > kInt32Max - G) return FP8FG_ERR_UNSUPPORTED;
  if (k > 0 && T > (kInt32Max - (int64_t(1) << 20)) / k) return FP8FG_ERR_UNSUPPORTED;
  if (!offsets) return FP8FG_ERR_INVALID_ARG;
  if (T > 0 && k > 0) {
    if (!experts || !row_index || !positions) return FP8FG_ERR_INVALID_ARG;
    const int64_t need = fp8fg_expert_segments_workspace(T, k, G);
    if (need > 0 && (!workspace || workspace_bytes < need)) return FP8FG_ERR_INVALID_ARG;
  }
  if (!aligned(experts, 4) || !aligned(offsets, 4) || !aligned(row_index, 4) || !aligned(positions, 4) ||
      !aligned(workspace, 4))
    return FP8FG_ERR_MISALIGNED;
  fp8fg::SegmentArgs a{};
  a.experts = experts; a.offsets = offsets; a.row_index = row_index; a.positions = positions;
  a.counts = static_cast<int32_t*>(workspace);
  a.n = T * k; a.first = first; a.k = static_cast<int>(k); a.G = static_cast<int>(G);
  return hip_status(fp8fg::launch_segments(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"

namespace {

int check_combine(int dtype, int64_t R, int64_t H, int64_t T, int64_t k) {
  if (!valid_dtype(dtype) || R < 0 || H < 0 || T < 0 || k < 0) return FP8FG_ERR_INVALID_ARG;
  if (H % 8 != 0 || H > kInt32Max || R > kInt32Max || T > kInt32Max || k > fp8fg::kCombineMaxK)
    return FP8FG_ERR_UNSUPPORTED;
  return FP8FG_OK;
}

int combine_backward(const void* dy, const void* rows, int dtype, int64_t R, int64_t H, int64_t ld_dy, int64_t ld_rows,
                     const int32_t* positions, const float* weights, int64_t T, int64_t k, void* drows, float* scales,
                     int pow2, float* dweights, fp8fg_stream_t stream) {
  int c = check_combine(dtype, R, H, T, k);
  if (c != FP8FG_OK) return c;
  if (T == 0 || k == 0) return FP8FG_OK;
  const bool any = R > 0 && H > 0;  // (rows and their gradient without elements may have no address)
  if (!positions || (any && ((!drows && !dweights) || (dweights && !rows)))) return FP8FG_ERR_INVALID_ARG;
  if (!aligned(positions, 4) || !aligned(weights, 4) || !aligned(dweights, 4) ||
      (any && (!aligned(scales, 4) || !aligned(drows, 16))))
    return FP8FG_ERR_MISALIGNED;
  if (H > 0 && (c = check_rows(dy, dtype, T, H, ld_dy)) != FP8FG_OK) return c;
  if (any && dweights && (c = check_rows(rows, dtype, R, H, ld_rows)) != FP8FG_OK) return c;
  if (!any && !dweights) return FP8FG_OK;
  fp8fg::CombineGradArgs a{};
  a.dy = dy; a.rows = rows; a.positions = positions; a.weights = weights; a.drows = drows; a.scales = scales;
  a.dw = dweights; a.R = R; a.H = H; a.ld_dy = ld_dy; a.ld_rows = ld_rows; a.T = T; a.k = static_cast<int>(k);
  a.bf16 = dtype == FP8FG_BF16; a.pow2 = pow2 == 1;
  return hip_status(fp8fg::launch_combine_backward(a, static_cast<hipStream_t>(stream)));
}

}  // namespace

extern "C" {

int fp8fg_combine_experts(const void* rows, int dtype, int64_t R, int64_t H, int64_t ld_rows,
                          const int32_t* positions, const float* weights, int64_t T, int64_t k, const void* base,
                          int64_t ld_base, void* y, fp8fg_stream_t stream) {
  int c = check_combine(dtype, R, H, T, k);
  if (c != FP8FG_OK) return c;
  if (T == 0 || H == 0) return FP8FG_OK;
  if (!y || (k > 0 && !positions)) return FP8FG_ERR_INVALID_ARG;
  if (!aligned(y, 16) || !aligned(positions, 4) || !aligned(weights, 4)) return FP8FG_ERR_MISALIGNED;
  if (R > 0 && k > 0 && (c = check_rows(rows, dtype, R, H, ld_rows)) != FP8FG_OK) return c;
  if (base && (c = check_rows(base, dtype, T, H, ld_base)) != FP8FG_OK) return c;
  fp8fg::CombineArgs a{};
  a.rows = rows; a.positions = positions; a.weights = weights; a.base = base; a.y = y;
  a.R = R; a.H = H; a.ld_rows = ld_rows; a.ld_base = ld_base; a.T = T; a.k = static_cast<int>(k);
  a.bf16 = dtype == FP8FG_BF16;
  return hip_status(fp8fg::launch_combine(a, static_cast<hipStream_t>(stream)));
}

int fp8fg_combine_experts_backward(const void* dy, const void* rows, int dtype, int64_t R, int64_t H, int64_t ld_dy,
                                   int64_t ld_rows, const int32_t* positions, const float* weights, int64_t T,
                                   int64_t k, void* drows, float* dweights, fp8fg_stream_t stream) {
  return combine_backward(dy, rows, dtype, R, H, ld_dy, ld_rows, positions, weights, T, k, drows, nullptr, 0, dweights,
                          stream);
}

int fp8fg_combine_experts_backward_quant(const void* dy, const void* rows, int dtype, int64_t R, int64_t H,
                                         int64_t ld_dy, int64_t ld_rows, const int32_t* positions,
                                         const float* weights, int64_t T, int64_t k, int pow2, uint8_t* q,
                                         float* scales, float* dweights, fp8fg_stream_t stream) {
  if (!flag(pow2)) return FP8FG_ERR_INVALID_ARG;
  if (H >= 0 && H % 128 != 0) return FP8FG_ERR_UNSUPPORTED;
  if (T > 0 && k > 0 && R > 0 && H > 0 && (!q || !scales)) return FP8FG_ERR_INVALID_ARG;
  return combine_backward(dy, rows, dtype, R, H, ld_dy, ld_rows, positions, weights, T, k, q, scales, pow2, dweights,
                          stream);
}

int fp4_quant_weight_1x32(const void* w, int w_dtype, int64_t N, int64_t K, int64_t ld_w, uint8_t* q, uint8_t* scales,
                          fp8fg_stream_t stream) {
  if (!valid_dtype(w_dtype) || N < 0 || K < 0) return FP8FG_ERR_INVALID_ARG;
  if (N == 0 || K == 0) return FP8FG_OK;
  if (K % 128 != 0 || N > kInt64Max / 16 / K || N * (K / 8) > fp8fg::kMaxWorkItems - 256) return FP8FG_ERR_UNSUPPORTED;
  if (!q || !scales) return FP8FG_ERR_INVALID_ARG;
  const int c = check_rows(w, w_dtype, N, K, ld_w);
  if (c != FP8FG_OK) return c;
  if (!aligned(q, 16) || !aligned(scales, 4)) return FP8FG_ERR_MISALIGNED;
  return hip_status(fp8fg::launch_fp4_quant(w, w_dtype == FP8FG_BF16, N, K, ld_w, q, scales,
                                            static_cast<hipStream_t>(stream)));
}

}  // extern "C"

namespace {

// N: columns of y; a gated w has 2N rows.
int fp4_product(const void* x, const float* sx, int64_t T, const int32_t* row_index, const int32_t* offsets,
                bool grouped, int64_t G, const uint8_t* w, const uint8_t* sw, void* y, int y_dtype, bool gated,
                int64_t M, int64_t N, int64_t K, fp8fg_stream_t stream) {
  if (!valid_dtype(y_dtype) || M < 0 || N < 0 || K < 0 || G < 0 || T < 0) return FP8FG_ERR_INVALID_ARG;
  if (M == 0 || N == 0 || G == 0) return FP8FG_OK;
  if (K == 0 || K % 128 != 0 || K >= (int64_t(1) << 24) || M > kInt32Max || N > kInt32Max || G > kInt32Max ||
      T > kInt32Max)
    return FP8FG_ERR_UNSUPPORTED;
  if (!x || !w || !sw || !y) return FP8FG_ERR_INVALID_ARG;
  if (grouped && (T == 0 || !offsets || (!row_index && T != M))) return FP8FG_ERR_INVALID_ARG;
  // The weights' bytes are counted in 64 bits, tiles in 31, lanes' offsets (from a tile's gate rows to its up
  // rows, from the first token to the last) in 32.
  if (G > kInt64Max / 2 / (gated ? 2 : 1) / N / K) return FP8FG_ERR_UNSUPPORTED;
  for (const fp8fg::Fp4Shape& s : fp8fg::kFp4Shapes[sx != nullptr])
    if (fp8fg::fp4_tiles(M, N, G, grouped, gated, s) > kInt32Max) return FP8FG_ERR_UNSUPPORTED;
  if (gated && (N + 128) * (K / 2) > kUint32Max) return FP8FG_ERR_UNSUPPORTED;
  if (grouped && row_index && T * K * (sx ? 1 : 2) > kUint32Max) return FP8FG_ERR_UNSUPPORTED;
  if (!aligned(x, 16) || !aligned(w, 16) || !aligned(sx, 4) || !aligned(sw, 4) ||
      !aligned(y, static_cast<unsigned>(elem_size(y_dtype))) || !aligned(offsets, 4) || !aligned(row_index, 4))
    return FP8FG_ERR_MISALIGNED;
  fp8fg::Fp4Args a{};
  a.x = x; a.sx = sx; a.w = w; a.sw = sw; a.y = y;
  a.offsets = offsets; a.row_index = row_index;
  a.M = M; a.N = N; a.K = K; a.G = G; a.T = T;
  a.gated = gated;
  a.y_bf16 = y_dtype == FP8FG_BF16;
  return hip_status(fp8fg::launch_fp4_gemm(a, static_cast<hipStream_t>(stream)));
}

}  // namespace

extern "C" {

int fp4_gemm(const void* x, const float* sx, const uint8_t* w, const uint8_t* sw, void* y, int y_dtype, int64_t M,
             int64_t N, int64_t K, fp8fg_stream_t stream) {
  return fp4_product(x, sx, M, nullptr, nullptr, false, 1, w, sw, y, y_dtype, false, M, N, K, stream);
}

int fp4_gated_gemm(const void* x, const float* sx, const uint8_t* w, const uint8_t* sw, void* h, int h_dtype,
                   int64_t M, int64_t I, int64_t K, fp8fg_stream_t stream) {
  return fp4_product(x, sx, M, nullptr, nullptr, false, 1, w, sw, h, h_dtype, true, M, I, K, stream);
}

int fp4_grouped_gemm(const void* x, const float* sx, int64_t T, const int32_t* row_index,
                     const int32_t* group_offsets, int64_t G, const uint8_t* w, const uint8_t* sw, void* y,
                     int y_dtype, int64_t M_total, int64_t N, int64_t K, fp8fg_stream_t stream) {
  return fp4_product(x, sx, T, row_index, group_offsets, true, G, w, sw, y, y_dtype, false, M_total, N, K, stream);
}

int fp4_grouped_gated_gemm(const void* x, const float* sx, int64_t T, const int32_t* row_index,
                           const int32_t* group_offsets, int64_t G, const uint8_t* w, const uint8_t* sw, void* h,
                           int h_dtype, int64_t M_total, int64_t I, int64_t K, fp8fg_stream_t stream) {
  return fp4_product(x, sx, T, row_index, group_offsets, true, G, w, sw, h, h_dtype, true, M_total, I, K, stream);
}

}  // extern "C"
