// C-ABI entry points declared in include/fp8fg_layer.h: argument validation on
// the host, then the launches.  Validation runs before any HIP call.
#include "fp8fg_layer.h"

#include <algorithm>
#include <cstdint>
#include <limits>
#include <memory>
#include <new>

#include "launch.h"

namespace {

constexpr int64_t kInt32Max = std::numeric_limits<int32_t>::max();

// Launches of workgroups of 512 work-items (their number rounded up to a multiple of
// 8), and of 16 work-items per group.
constexpr int64_t kMostTiles = fp8fg::kMaxWorkItems / 512 / 8 * 8;
constexpr int64_t kMostRowGroups = fp8fg::kMaxWorkItems / 256 * 16;

bool aligned(const void* p, unsigned a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
int64_t elem_size(int dtype) { return dtype == FP8FG_BF16 ? 2 : 4; }
bool valid_dtype(int d) { return d == FP8FG_F32 || d == FP8FG_BF16; }
int hip_status(hipError_t e) { return e == hipSuccess ? FP8FG_OK : FP8FG_ERR_HIP; }

// A row-major operand of a norm call, `ld` elements between rows.
int check_rows(const void* p, int dtype, int64_t H, int64_t ld) {
  if (!p || ld < H) return FP8FG_ERR_INVALID_ARG;
  if (ld > std::numeric_limits<int64_t>::max() / 16) return FP8FG_ERR_UNSUPPORTED;
  if (!aligned(p, 16) || (ld * elem_size(dtype)) % 16 != 0) return FP8FG_ERR_MISALIGNED;
  return FP8FG_OK;
}

int check_norm_sizes(int dtype, int w_dtype, int64_t M, int64_t H) {
  if (!valid_dtype(dtype) || !valid_dtype(w_dtype) || M < 0 || H < 0) return FP8FG_ERR_INVALID_ARG;
  if (H % 128 != 0 || H > fp8fg::kNormMaxH || M > kInt32Max) return FP8FG_ERR_UNSUPPORTED;
  return FP8FG_OK;
}

}  // namespace

extern "C" {

int fp8_add_rmsnorm_quant_1x128(const void* x, const void* residual, int dtype, int64_t M, int64_t H, int64_t ld_x,
                                int64_t ld_r, const void* weight, int w_dtype, float eps, int pow2, void* h, void* y,
                                uint8_t* q, float* scales, float* rstd, fp8fg_stream_t stream) {
  int c = check_norm_sizes(dtype, w_dtype, M, H);
  if (c != FP8FG_OK) return c;
  if (!(eps >= 0.0f) || (pow2 != 0 && pow2 != 1)) return FP8FG_ERR_INVALID_ARG;
  if (M == 0 || H == 0) return FP8FG_OK;
  if ((c = check_rows(x, dtype, H, ld_x)) != FP8FG_OK) return c;
  if (residual && (c = check_rows(residual, dtype, H, ld_r)) != FP8FG_OK) return c;
  if (!weight || !q || !scales) return FP8FG_ERR_INVALID_ARG;
  if (!aligned(weight, 16) || !aligned(h, 16) || !aligned(y, 16) || !aligned(q, 16) || !aligned(scales, 4) ||
      !aligned(rstd, 4))
    return FP8FG_ERR_MISALIGNED;
  fp8fg::NormArgs a{};
  a.x = x; a.r = residual; a.w = weight; a.h = h; a.y = y; a.q = q; a.scales = scales; a.rstd = rstd;
  a.M = M; a.H = H; a.ld_x = ld_x; a.ld_r = ld_r; a.eps = eps;
  a.bf16 = dtype == FP8FG_BF16; a.w_bf16 = w_dtype == FP8FG_BF16; a.pow2 = pow2 == 1;
  return hip_status(fp8fg::launch_rmsnorm_quant(a, static_cast<hipStream_t>(stream)));
}

int64_t fp8_rmsnorm_backward_workspace(int64_t M, int64_t H) {
  if (M < 0 || H < 0 || H > fp8fg::kNormMaxH) return 0;
  return fp8fg::rmsnorm_backward_partials(M, H) * H * static_cast<int64_t>(sizeof(float));
}

int fp8_rmsnorm_backward(const void* dy, const void* h, const void* dh, int dtype, int64_t M, int64_t H, int64_t ld_dy,
                         int64_t ld_h, int64_t ld_dh, const float* rstd, const void* weight, int w_dtype, void* dx,
                         float* dw, void* workspace, int64_t workspace_bytes, fp8fg_stream_t stream) {
  int c = check_norm_sizes(dtype, w_dtype, M, H);
  if (c != FP8FG_OK) return c;
  if (H == 0 || (M == 0 && !dw)) return FP8FG_OK;
  if (dw) {
    if (!aligned(dw, 16)) return FP8FG_ERR_MISALIGNED;
    const int64_t need = fp8_rmsnorm_backward_workspace(M, H);
    if (need > 0 && (!workspace || workspace_bytes < need)) return FP8FG_ERR_INVALID_ARG;
    if (!aligned(workspace, 16)) return FP8FG_ERR_MISALIGNED;
  }
  if (M > 0) {
    if ((c = check_rows(dy, dtype, H, ld_dy)) != FP8FG_OK || (c = check_rows(h, dtype, H, ld_h)) != FP8FG_OK) return c;
    if (dh && (c = check_rows(dh, dtype, H, ld_dh)) != FP8FG_OK) return c;
    if (!rstd || !weight || !dx) return FP8FG_ERR_INVALID_ARG;
    if (!aligned(rstd, 4) || !aligned(weight, 16) || !aligned(dx, 16)) return FP8FG_ERR_MISALIGNED;
  }
  fp8fg::NormGradArgs a{};
  a.dy = dy; a.h = h; a.dh = dh; a.rstd = rstd; a.w = weight; a.dx = dx;
  a.partial = dw ? static_cast<float*>(workspace) : nullptr;
  a.M = M; a.H = H; a.ld_dy = ld_dy; a.ld_h = ld_h; a.ld_dh = ld_dh;
  a.bf16 = dtype == FP8FG_BF16; a.w_bf16 = w_dtype == FP8FG_BF16;
  return hip_status(fp8fg::launch_rmsnorm_backward(a, dw, static_cast<hipStream_t>(stream)));
}

}  // extern "C"

namespace {

// Checks of a gated product and its launch arguments: FP8FG_OK, an error status,
// or -1 when there is nothing to do.
int check_gated(const uint8_t* a, const float* sa, const uint8_t* w, const float* sw, int accum, const void* h,
                int h_dtype, const void* gu, int64_t M, int64_t I, int64_t K) {
  if (!valid_dtype(h_dtype) || M < 0 || I < 0 || K < 0) return FP8FG_ERR_INVALID_ARG;
  if (accum != FP8FG_ACCUM_FP8_MFMA && accum != FP8FG_ACCUM_EXACT && accum != FP8FG_ACCUM_SCALED_MFMA)
    return FP8FG_ERR_INVALID_ARG;
  if (M == 0 || I == 0) return -1;
  if (K == 0 || K % 128 != 0 || I % 128 != 0) return FP8FG_ERR_UNSUPPORTED;
  if (!a || !sa || !w || !sw || !h) return FP8FG_ERR_INVALID_ARG;
  // (the tile loads' lane offsets are 32-bit: 256 rows of K bytes)
  if (M > kInt32Max || I > kInt32Max / 2 || K >= (int64_t(1) << 24)) return FP8FG_ERR_UNSUPPORTED;
  if (!aligned(a, 16) || !aligned(w, 16) || !aligned(h, 16) || !aligned(gu, 16) || !aligned(sa, 4) || !aligned(sw, 4))
    return FP8FG_ERR_MISALIGNED;
  return FP8FG_OK;
}

fp8fg::GemmArgs gated_args(const uint8_t* a, const float* sa, const uint8_t* w, const float* sw, int accum, void* h,
                           int h_dtype, void* gu, int64_t M, int64_t I, int64_t K) {
  fp8fg::GemmArgs g{};
  g.a = a; g.sa = sa; g.b = w; g.sb = sw; g.y = h;
  g.M = M; g.N = 2 * I; g.K = K; g.G = 1; g.T = M;
  g.exact = accum == FP8FG_ACCUM_EXACT;
  g.scaled = accum == FP8FG_ACCUM_SCALED_MFMA;
  g.y_bf16 = h_dtype == FP8FG_BF16;
  g.gu = gu;
  return g;
}

int gated(const uint8_t* a, const float* sa, const uint8_t* w, const float* sw, int accum, void* h, int h_dtype,
          float* s_h, int pow2, void* gu, void* workspace, int64_t M, int64_t I, int64_t K, fp8fg_stream_t stream) {
  const int c = check_gated(a, sa, w, sw, accum, h, h_dtype, gu, M, I, K);
  if (c != FP8FG_OK) return c < 0 ? FP8FG_OK : c;
  if (((M + 127) / 128) * (I / 128) > kMostTiles) return FP8FG_ERR_UNSUPPORTED;
  fp8fg::GemmArgs g = gated_args(a, sa, w, sw, accum, h, h_dtype, gu, M, I, K);
  g.y_scales = s_h;
  g.pow2 = pow2 == 1;
  return hip_status(fp8fg::launch_gated_gemm(g, static_cast<float*>(workspace), static_cast<hipStream_t>(stream)));
}

int grouped_gated(const uint8_t* a, const float* sa, int64_t T, const int32_t* row_index,
                  const int32_t* group_offsets, int64_t G, const uint8_t* w, const float* sw, int accum, void* h,
                  int h_dtype, float* s_h, int pow2, void* gu, void* workspace, int64_t M_total, int64_t I, int64_t K,
                  fp8fg_stream_t stream) {
  if (G < 0 || T < 0) return FP8FG_ERR_INVALID_ARG;
  const int c = check_gated(a, sa, w, sw, accum, h, h_dtype, gu, M_total, I, K);
  if (c > 0) return c;
  if (c < 0 || G == 0) return FP8FG_OK;
  if (T == 0 || !group_offsets || (!row_index && T != M_total)) return FP8FG_ERR_INVALID_ARG;
  if (!aligned(group_offsets, 4) || !aligned(row_index, 4)) return FP8FG_ERR_MISALIGNED;
  if (G > kInt32Max || (M_total / 128 + G) * (I / 128) > kMostTiles) return FP8FG_ERR_UNSUPPORTED;
  if (T > kInt32Max || T * K >= (int64_t(1) << 32)) return FP8FG_ERR_UNSUPPORTED;  // 32-bit row offsets
  fp8fg::GemmArgs g = gated_args(a, sa, w, sw, accum, h, h_dtype, gu, M_total, I, K);
  g.offsets = group_offsets;
  g.row_index = row_index;
  g.G = G;
  g.T = T;
  g.y_scales = s_h;
  g.pow2 = pow2 == 1;
  return hip_status(fp8fg::launch_gated_gemm(g, static_cast<float*>(workspace), static_cast<hipStream_t>(stream)));
}

// Checks of a quantised output; a workspace too small to be used becomes null.
int check_quant_out(const float* s_h, int pow2, void*& workspace, int64_t bytes, int64_t M, int64_t I) {
  if ((pow2 != 0 && pow2 != 1) || bytes < 0) return FP8FG_ERR_INVALID_ARG;
  if (M > 0 && I > 0 && !s_h) return FP8FG_ERR_INVALID_ARG;
  if (!aligned(s_h, 4) || !aligned(workspace, 16)) return FP8FG_ERR_MISALIGNED;
  if (M > 0 && I > 0 && bytes / 4 / I < M) workspace = nullptr;
  return FP8FG_OK;
}

}  // namespace

extern "C" {

int fp8_block_gated_gemm(const uint8_t* a, const float* sa, const uint8_t* w, const float* sw, int accum, void* h,
                         int h_dtype, void* gu, int64_t M, int64_t I, int64_t K, fp8fg_stream_t stream) {
  return gated(a, sa, w, sw, accum, h, h_dtype, nullptr, 0, gu, nullptr, M, I, K, stream);
}

int fp8_block_gated_gemm_quant(const uint8_t* a, const float* sa, const uint8_t* w, const float* sw, int accum,
                               int pow2, uint8_t* q_h, float* s_h, void* gu, void* workspace, int64_t workspace_bytes,
                               int64_t M, int64_t I, int64_t K, fp8fg_stream_t stream) {
  const int c = check_quant_out(s_h, pow2, workspace, workspace_bytes, M, I);
  return c != FP8FG_OK ? c : gated(a, sa, w, sw, accum, q_h, FP8FG_BF16, s_h, pow2, gu, workspace, M, I, K, stream);
}

int64_t fp8_block_gated_gemm_quant_workspace(int accum, int64_t M, int64_t I, int64_t K, int64_t G) {
  if (M <= 0 || I <= 0 || K <= 0 || G < 0 || M > kInt32Max || I > kInt32Max / 2) return 0;
  fp8fg::GemmArgs g = gated_args(nullptr, nullptr, nullptr, nullptr, accum, nullptr, FP8FG_BF16, nullptr, M, I, K);
  const int32_t grouped = 0;
  if (G > 0) {
    g.G = G;
    g.offsets = &grouped;  // (only whether it is set is looked at)
  }
  return fp8fg::gated_quant_takes_workspace(g) ? M * I * 4 : 0;
}

int fp8_block_grouped_gated_gemm(const uint8_t* a, const float* sa, int64_t T, const int32_t* row_index,
                                 const int32_t* group_offsets, int64_t G, const uint8_t* w, const float* sw,
                                 int accum, void* h, int h_dtype, void* gu, int64_t M_total, int64_t I, int64_t K,
                                 fp8fg_stream_t stream) {
  return grouped_gated(a, sa, T, row_index, group_offsets, G, w, sw, accum, h, h_dtype, nullptr, 0, gu, nullptr,
                       M_total, I, K, stream);
}

int fp8_block_grouped_gated_gemm_quant(const uint8_t* a, const float* sa, int64_t T, const int32_t* row_index,
                                       const int32_t* group_offsets, int64_t G, const uint8_t* w, const float* sw,
                                       int accum, int pow2, uint8_t* q_h, float* s_h, void* gu, void* workspace,
                                       int64_t workspace_bytes, int64_t M_total, int64_t I, int64_t K,
                                       fp8fg_stream_t stream) {
  const int c = check_quant_out(s_h, pow2, workspace, workspace_bytes, M_total, I);
  return c != FP8FG_OK ? c : grouped_gated(a, sa, T, row_index, group_offsets, G, w, sw, accum, q_h, FP8FG_BF16, s_h,
                                           pow2, gu, workspace, M_total, I, K, stream);
}

int fp8_gated_backward_quant(const void* dh, const void* gu, int dtype, int64_t M, int64_t I, int64_t ld_dh, int pow2,
                             uint8_t* q, float* s, uint8_t* q_t, float* s_t, uint8_t* q_ht, float* s_ht,
                             fp8fg_stream_t stream) {
  if (!valid_dtype(dtype) || M < 0 || I < 0 || (pow2 != 0 && pow2 != 1)) return FP8FG_ERR_INVALID_ARG;
  if (!q != !s || !q_t != !s_t || !q_ht != !s_ht) return FP8FG_ERR_INVALID_ARG;  // half a pair
  if (M == 0 || I == 0) return FP8FG_OK;
  if (!q && !q_t && !q_ht) return FP8FG_ERR_INVALID_ARG;
  if (I % 128 != 0 || ((q_t || q_ht) && M % 128 != 0)) return FP8FG_ERR_UNSUPPORTED;
  // launch grids: one workgroup of 512 work-items per 128 x 128 tile (bf16 walks over
  // the tiles), or 16 work-items per group of a row
  if (M > kInt32Max || I > kInt32Max || M * (I / 128) > kInt32Max - 8) return FP8FG_ERR_UNSUPPORTED;
  if (q_t || q_ht ? dtype == FP8FG_F32 && (M / 128) * (I / 128) > kMostTiles : M * (I / 128) > kMostRowGroups)
    return FP8FG_ERR_UNSUPPORTED;
  const int c = check_rows(dh, dtype, I, ld_dh);
  if (c != FP8FG_OK) return c;
  if (!gu) return FP8FG_ERR_INVALID_ARG;
  if (!aligned(gu, 16) || !aligned(q, 16) || !aligned(q_t, 16) || !aligned(q_ht, 16) || !aligned(s, 4) ||
      !aligned(s_t, 4) || !aligned(s_ht, 4))
    return FP8FG_ERR_MISALIGNED;
  fp8fg::GatedGradArgs a{};
  a.dh = dh; a.gu = gu; a.q = q; a.s = s; a.q_t = q_t; a.s_t = s_t; a.q_ht = q_ht; a.s_ht = s_ht;
  a.M = M; a.I = I; a.ld_dh = ld_dh;
  a.bf16 = dtype == FP8FG_BF16; a.pow2 = pow2 == 1;
  return hip_status(fp8fg::launch_gated_backward(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"

namespace {

// Whether an output of a clip overlaps another output, another tensor's gradient, or
// part of its own: workgroups would then read what others have already scaled.
int check_disjoint(const void* const* grads, void* const* outs, const int64_t* counts, const int* dtypes, int64_t n) {
  struct Range {
    uintptr_t begin, end;
    bool written;
  };
  constexpr int64_t kFew = 128;  // kept on the stack
  Range few[kFew];
  std::unique_ptr<Range[]> many;
  Range* r = few;
  if (2 * n > kFew) {
    many.reset(new (std::nothrow) Range[2 * n]);
    if (!many) return FP8FG_ERR_UNSUPPORTED;
    r = many.get();
  }
  int64_t k = 0;
  for (int64_t i = 0; i < n; ++i) {
    if (counts[i] == 0) continue;
    const uintptr_t bytes = static_cast<uintptr_t>(counts[i] * elem_size(dtypes[i]));
    const uintptr_t in = reinterpret_cast<uintptr_t>(grads[i]), out = reinterpret_cast<uintptr_t>(outs[i]);
    r[k++] = Range{out, out + bytes, true};
    if (in != out) r[k++] = Range{in, in + bytes, false};
  }
  std::sort(r, r + k, [](const Range& a, const Range& b) { return a.begin < b.begin; });
  uintptr_t read_end = 0, written_end = 0;
  for (int64_t i = 0; i < k; ++i) {
    if (r[i].begin < written_end || (r[i].written && r[i].begin < read_end)) return FP8FG_ERR_INVALID_ARG;
    uintptr_t& end = r[i].written ? written_end : read_end;
    end = std::max(end, r[i].end);
  }
  return FP8FG_OK;
}

int grad_norm(const void* const* grads, void* const* outs, bool clip, const int64_t* counts, const int* dtypes,
              int64_t n, float max_norm, float* norm, void* workspace, int64_t workspace_bytes,
              fp8fg_stream_t stream) {
  if (n < 0 || !norm || (n > 0 && (!grads || !counts || !dtypes || (clip && !outs)))) return FP8FG_ERR_INVALID_ARG;
  if (clip && !(max_norm > 0.0f)) return FP8FG_ERR_INVALID_ARG;
  if (n > 0 && (!workspace || workspace_bytes < fp8fg_grad_norm_workspace(n))) return FP8FG_ERR_INVALID_ARG;
  if (!aligned(norm, 4) || !aligned(workspace, 8)) return FP8FG_ERR_MISALIGNED;
  // (120 tensors of 2^36 elements are 2^30 chunks of 8192: a launch numbers them with 32 bits)
  constexpr int64_t kMostElements = int64_t(1) << 36;
  for (int64_t i = 0; i < n; ++i) {
    if (!valid_dtype(dtypes[i]) || counts[i] < 0) return FP8FG_ERR_INVALID_ARG;
    if (counts[i] == 0) continue;
    if (!grads[i] || (clip && !outs[i])) return FP8FG_ERR_INVALID_ARG;
    if (counts[i] > kMostElements) return FP8FG_ERR_UNSUPPORTED;
    const unsigned es = static_cast<unsigned>(elem_size(dtypes[i]));
    if (!aligned(grads[i], es) || (clip && !aligned(outs[i], es))) return FP8FG_ERR_MISALIGNED;
  }
  if (clip) {
    const int c = check_disjoint(grads, outs, counts, dtypes, n);
    if (c != FP8FG_OK) return c;
  }
  fp8fg::GradList g{};
  g.grads = grads; g.outs = clip ? outs : nullptr; g.counts = counts; g.dtypes = dtypes; g.n = n;
  return hip_status(fp8fg::launch_grad_norm(g, max_norm, norm, static_cast<double*>(workspace),
                                            static_cast<hipStream_t>(stream)));
}

}  // namespace

extern "C" {

int64_t fp8fg_grad_norm_workspace(int64_t n) {
  if (n <= 0) return 0;
  return (n + fp8fg::kGradBatch - 1) / fp8fg::kGradBatch * fp8fg::kGradPartials * static_cast<int64_t>(sizeof(double));
}

int fp8fg_grad_norm(const void* const* grads, const int64_t* counts, const int* dtypes, int64_t n, float* norm,
                    void* workspace, int64_t workspace_bytes, fp8fg_stream_t stream) {
  return grad_norm(grads, nullptr, false, counts, dtypes, n, 0.0f, norm, workspace, workspace_bytes, stream);
}

int fp8fg_clip_grad_norm(const void* const* grads, void* const* outs, const int64_t* counts, const int* dtypes,
                         int64_t n, float max_norm, float* norm, void* workspace, int64_t workspace_bytes,
                         fp8fg_stream_t stream) {
  return grad_norm(grads, outs, true, counts, dtypes, n, max_norm, norm, workspace, workspace_bytes, stream);
}

}  // extern "C"
