// C ABI of the quantised linear layer's operators (pipe_linear.h): argument
// checks, before any HIP call, then the launches.
#include <hip/hip_runtime.h>

#include "pipe_kernels.hpp"
#include "pipe_linear.h"
#include "pipe_linear.hpp"

namespace {

using namespace pipe;

bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

// Device code forms byte offsets in int64: a matrix must span fewer than 2^62
// bytes (row counts are at most 2^31 - 1).
bool pitch_fits(int64_t ld) { return ld <= int64_t(1) << 28; }

// The e4m3 product's kernels reach the 256 rows of a tile by 32-bit offsets.
constexpr int64_t kFp8PitchEnd = int64_t(1) << 24;

pipe_status_t hip_status(hipError_t e) { return e == hipSuccess ? PIPE_OK : PIPE_ERR_HIP; }

bool is16(pipe_dtype_t t) { return t == PIPE_BF16 || t == PIPE_FP16; }

pipe_status_t fill_zero(void* C, int64_t M, int64_t N, int64_t ldc, pipe_dtype_t type,
                        hipStream_t st) {
  return hip_status(type == PIPE_FP32
                        ? launch_fill_f32(static_cast<float*>(C), M, N, ldc, 0.f, st)
                        : launch_fill_u16(static_cast<uint16_t*>(C), M, N, ldc, 0, st));
}

pipe_status_t norm_shape(int64_t M, int64_t N) {
  if (M < 0 || N < 0 || M > INT32_MAX || N % 8 != 0 || N > PIPE_RMSNORM_MAX_N)
    return PIPE_ERR_SHAPE;
  return PIPE_OK;
}

// A matrix of the norm: pitch and alignment of `elem`-byte elements.
pipe_status_t norm_operand(const void* base, int64_t ld, int64_t N, int elem) {
  if (base == nullptr) return PIPE_ERR_NULL;
  if (ld < N || !pitch_fits(ld)) return PIPE_ERR_SHAPE;
  if (!aligned(base, 8 * elem) || ld % 8 != 0) return PIPE_ERR_ALIGN;
  return PIPE_OK;
}

}  // namespace

extern "C" {

pipe_status_t pipe_rmsnorm(const void* x, const void* residual, const void* weight, void* y,
                           float* y_scales, void* h, int64_t M, int64_t N, int64_t ld_x,
                           int64_t ld_residual, int64_t ld_y, int64_t ld_h, float eps,
                           pipe_dtype_t type, pipe_dtype_t out_type, void* stream) {
  if (!is16(type) || (out_type != type && out_type != PIPE_E4M3)) return PIPE_ERR_CONFIG;
  if (!(eps >= 0.f)) return PIPE_ERR_CONFIG;
  pipe_status_t s = norm_shape(M, N);
  if (s != PIPE_OK) return s;
  if (M == 0 || N == 0) return PIPE_OK;
  const bool q8 = out_type == PIPE_E4M3;
  s = norm_operand(x, ld_x, N, 2);
  if (s != PIPE_OK) return s;
  s = norm_operand(y, ld_y, N, q8 ? 1 : 2);
  if (s != PIPE_OK) return s;
  if ((residual == nullptr) != (h == nullptr) || weight == nullptr) return PIPE_ERR_NULL;
  if (residual != nullptr) {
    s = norm_operand(residual, ld_residual, N, 2);
    if (s != PIPE_OK) return s;
    s = norm_operand(h, ld_h, N, 2);
    if (s != PIPE_OK) return s;
  }
  if (!aligned(weight, 16)) return PIPE_ERR_ALIGN;
  if (q8) {
    if (y_scales == nullptr) return PIPE_ERR_NULL;
    if (!aligned(y_scales, 4)) return PIPE_ERR_ALIGN;
  }
  NormParams p{};
  p.x = static_cast<const uint8_t*>(x);
  p.residual = static_cast<const uint8_t*>(residual);
  p.weight = static_cast<const uint8_t*>(weight);
  p.y = static_cast<uint8_t*>(y);
  p.h = static_cast<uint8_t*>(h);
  p.scales = y_scales;
  p.ld_x = ld_x * 2;
  p.ld_residual = residual != nullptr ? ld_residual * 2 : 0;
  p.ld_y = q8 ? ld_y : ld_y * 2;
  p.ld_h = h != nullptr ? ld_h * 2 : 0;
  p.M = M;
  p.chunks = (int32_t)(N / 8);
  p.inv_n = 1.0f / (float)N;
  p.eps = eps;
  return hip_status(launch_rmsnorm(p, type, q8, static_cast<hipStream_t>(stream)));
}

pipe_status_t pipe_rmsnorm_backward_workspace_bytes(int64_t M, int64_t N, size_t* bytes) {
  if (bytes == nullptr) return PIPE_ERR_NULL;
  *bytes = 0;
  const pipe_status_t s = norm_shape(M, N);
  if (s != PIPE_OK) return s;
  *bytes = (size_t)rmsnorm_grad_partials(M, N) * (size_t)N * sizeof(float);
  return PIPE_OK;
}

pipe_status_t pipe_rmsnorm_backward(const void* dy, const void* x, const void* weight,
                                    const void* dh, void* dx, float* dweight, int64_t M,
                                    int64_t N, int64_t ld_dy, int64_t ld_x, int64_t ld_dh,
                                    int64_t ld_dx, float eps, pipe_dtype_t type,
                                    void* workspace, size_t workspace_bytes, void* stream) {
  if (!is16(type) || !(eps >= 0.f)) return PIPE_ERR_CONFIG;
  size_t need = 0;
  pipe_status_t s = pipe_rmsnorm_backward_workspace_bytes(M, N, &need);
  if (s != PIPE_OK) return s;
  if (N == 0) return PIPE_OK;
  if (dweight == nullptr) return PIPE_ERR_NULL;
  if (!aligned(dweight, 16)) return PIPE_ERR_ALIGN;
  if (M > 0) {
    s = norm_operand(dy, ld_dy, N, 2);
    if (s == PIPE_OK) s = norm_operand(x, ld_x, N, 2);
    if (s == PIPE_OK) s = norm_operand(dx, ld_dx, N, 2);
    if (s == PIPE_OK && dh != nullptr) s = norm_operand(dh, ld_dh, N, 2);
    if (s != PIPE_OK) return s;
    if (weight == nullptr) return PIPE_ERR_NULL;
    if (!aligned(weight, 16)) return PIPE_ERR_ALIGN;
    if (need > 0) {
      if (workspace == nullptr || workspace_bytes < need) return PIPE_ERR_WORKSPACE;
      if (!aligned(workspace, 16)) return PIPE_ERR_ALIGN;
    }
  }
  NormGradParams p{};
  p.dy = static_cast<const uint8_t*>(dy);
  p.x = static_cast<const uint8_t*>(x);
  p.weight = static_cast<const uint8_t*>(weight);
  p.dh = static_cast<const uint8_t*>(dh);
  p.dx = static_cast<uint8_t*>(dx);
  p.partials = static_cast<float*>(workspace);
  p.ld_dy = ld_dy * 2;
  p.ld_x = ld_x * 2;
  p.ld_dh = dh != nullptr ? ld_dh * 2 : 0;
  p.ld_dx = ld_dx * 2;
  p.M = M;
  p.chunks = (int32_t)(N / 8);
  p.inv_n = 1.0f / (float)N;
  p.eps = eps;
  return hip_status(launch_rmsnorm_grad(p, dweight, type, static_cast<hipStream_t>(stream)));
}

pipe_status_t pipe_gemm_fp8_workspace_bytes(int64_t M, int64_t N, int64_t K, size_t* bytes) {
  if (bytes == nullptr) return PIPE_ERR_NULL;
  *bytes = 0;
  if (M < 0 || N < 0 || K < 0 || M > INT32_MAX || N > INT32_MAX || K > INT32_MAX || N % 8 != 0 ||
      K % 16 != 0)
    return PIPE_ERR_SHAPE;
  if (M == 0 || N == 0 || K == 0) return PIPE_OK;
  if ((M + 127) / 128 * ((N + 127) / 128) > INT32_MAX) return PIPE_ERR_SHAPE;  // output tiles
  *bytes = (size_t)gemm_fp8_partials(M, N, K) * sizeof(float);
  return PIPE_OK;
}

pipe_status_t pipe_gemm_fp8(const void* A, const float* a_scales, const void* B,
                            const float* b_scales, void* C, int64_t M, int64_t N, int64_t K,
                            int64_t lda, int64_t ldb, int64_t ldc, pipe_dtype_t out_type,
                            void* workspace, size_t workspace_bytes, void* stream) {
  if (!is16(out_type) && out_type != PIPE_FP32) return PIPE_ERR_CONFIG;
  size_t need = 0;
  const pipe_status_t s = pipe_gemm_fp8_workspace_bytes(M, N, K, &need);
  if (s != PIPE_OK) return s;
  if (lda < K || ldb < K || ldc < N || lda >= kFp8PitchEnd || ldb >= kFp8PitchEnd || !pitch_fits(ldc))
    return PIPE_ERR_SHAPE;
  if (M == 0 || N == 0) return PIPE_OK;
  if (C == nullptr) return PIPE_ERR_NULL;
  if (!aligned(C, 16) || ldc % 8 != 0) return PIPE_ERR_ALIGN;
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (K == 0) return fill_zero(C, M, N, ldc, out_type, st);
  if (A == nullptr || B == nullptr || a_scales == nullptr || b_scales == nullptr)
    return PIPE_ERR_NULL;
  if (!aligned(A, 16) || !aligned(B, 16) || lda % 16 != 0 || ldb % 16 != 0 ||
      !aligned(a_scales, 4) || !aligned(b_scales, 4))
    return PIPE_ERR_ALIGN;
  if (need > 0) {
    if (workspace == nullptr || workspace_bytes < need) return PIPE_ERR_WORKSPACE;
    if (!aligned(workspace, 16)) return PIPE_ERR_ALIGN;
  }
  Fp8Params p{};
  p.A = static_cast<const uint8_t*>(A);
  p.B = static_cast<const uint8_t*>(B);
  p.a_scales = a_scales;
  p.b_scales = b_scales;
  p.C = C;
  p.partials = static_cast<float*>(workspace);
  p.lda = lda;
  p.ldb = ldb;
  p.ldc = ldc;
  p.M = (int32_t)M;
  p.N = (int32_t)N;
  p.K = (int32_t)K;
  return hip_status(launch_gemm_fp8(p, out_type, st));
}

pipe_status_t pipe_gemm_w4_workspace_bytes(int64_t M, int64_t N, int64_t K, size_t* bytes) {
  if (bytes == nullptr) return PIPE_ERR_NULL;
  *bytes = 0;
  if (M < 0 || N < 0 || K < 0 || M > INT32_MAX || N > INT32_MAX || K > INT32_MAX - 1024 ||
      N % 8 != 0 || K % 32 != 0)
    return PIPE_ERR_SHAPE;
  if (M == 0 || N == 0 || K == 0) return PIPE_OK;
  if ((M + 15) / 16 * ((N + 127) / 128) > INT32_MAX) return PIPE_ERR_SHAPE;  // output tiles
  *bytes = (size_t)gemm_w4_partials(M, N, K) * sizeof(float);
  return PIPE_OK;
}

pipe_status_t pipe_gemm_w4(const void* A, const void* codes, const void* scales,
                           const void* zeros, void* C, int64_t M, int64_t N, int64_t K,
                           int64_t group, int64_t lda, int64_t ld_codes, int64_t ld_scales,
                           int64_t ld_zeros, int64_t ldc, pipe_dtype_t type, void* workspace,
                           size_t workspace_bytes, void* stream) {
  if (!is16(type)) return PIPE_ERR_CONFIG;
  size_t need = 0;
  const pipe_status_t shape = pipe_gemm_w4_workspace_bytes(M, N, K, &need);
  if (shape != PIPE_OK) return shape;
  const bool pow2 = group >= 32 && (group & (group - 1)) == 0;
  if (K > 0 && !(group == K || (pow2 && K % group == 0))) return PIPE_ERR_SHAPE;
  const int64_t groups = K > 0 ? K / group : 0;
  if (lda < K || ld_codes < K / 2 || ld_scales < groups || ldc < N ||
      (zeros != nullptr && ld_zeros < groups))
    return PIPE_ERR_SHAPE;
  if (!pitch_fits(lda) || !pitch_fits(ld_codes) || !pitch_fits(ld_scales) || !pitch_fits(ldc) ||
      (zeros != nullptr && !pitch_fits(ld_zeros)))
    return PIPE_ERR_SHAPE;
  if (M == 0 || N == 0) return PIPE_OK;
  if (C == nullptr) return PIPE_ERR_NULL;
  if (!aligned(C, 16) || ldc % 8 != 0) return PIPE_ERR_ALIGN;
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (K == 0) return fill_zero(C, M, N, ldc, type, st);
  if (A == nullptr || codes == nullptr || scales == nullptr) return PIPE_ERR_NULL;
  if (!aligned(A, 16) || lda % 8 != 0 || !aligned(codes, 16) || ld_codes % 16 != 0 ||
      !aligned(scales, 2))
    return PIPE_ERR_ALIGN;
  if (need > 0) {
    if (workspace == nullptr || workspace_bytes < need) return PIPE_ERR_WORKSPACE;
    if (!aligned(workspace, 16)) return PIPE_ERR_ALIGN;
  }
  W4Params p{};
  p.partials = static_cast<float*>(workspace);
  p.A = static_cast<const uint8_t*>(A);
  p.codes = static_cast<const uint8_t*>(codes);
  p.scales = static_cast<const uint16_t*>(scales);
  p.zeros = static_cast<const uint8_t*>(zeros);
  p.C = static_cast<uint8_t*>(C);
  p.lda = lda * 2;
  p.ld_codes = ld_codes;
  p.ld_scales = ld_scales;
  p.ld_zeros = zeros != nullptr ? ld_zeros : 0;
  p.ldc = ldc;
  p.M = (int32_t)M;
  p.N = (int32_t)N;
  p.K = (int32_t)K;
  p.group_shift = 31;
  if (group != K)
    for (p.group_shift = 5; (int64_t(1) << p.group_shift) < group;) ++p.group_shift;
  return hip_status(launch_gemm_w4(p, type, st));
}

}  // extern "C"
