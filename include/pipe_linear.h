/*
 * pipe_linear -- the operators of a quantised linear layer, exported by the
 * same library as pipe_tile.h: RMS norm with the residual's addition and a
 * 16-bit or e4m3 output, its gradient, products of e4m3 rows with e4m3
 * weights, and products of 16-bit rows with 4-bit weights; layer norm with the
 * residual's addition and a 16-bit, e4m3 or microscaled 4-bit output, its
 * gradient, the microscaled 4-bit form of 16- and 32-bit rows and back, and
 * products of rows and weights in it.
 *
 * The conventions of pipe_tile.h hold: device pointers owned by the caller,
 * row-major matrices with a leading dimension in elements, asynchronous calls
 * on `stream`, every argument checked before anything is enqueued, no
 * allocation and no host state. Status codes and their names are
 * pipe_status_t's. None of these calls uses the library's status word: their
 * kernels have no bounded waits.
 *
 * Results are deterministic: no atomics, every sum in an order that depends
 * on the shapes alone.
 */
#ifndef PIPE_LINEAR_H
#define PIPE_LINEAR_H

#include "pipe_tile.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  PIPE_BF16 = 0,
  PIPE_FP16 = 1,
  PIPE_FP32 = 2,
  PIPE_E4M3 = 3,          /* OCP 8-bit float, 448 the largest */
  PIPE_MXFP4 = 4,         /* OCP microscaled 4-bit float, below */
  PIPE_DTYPE_RANGE_MIN_ = -0x7fffffff - 1,
  PIPE_DTYPE_RANGE_MAX_ = 0x7fffffff
} pipe_dtype_t;

/* The widest row of the norm and its gradient, in elements. */
#define PIPE_RMSNORM_MAX_N 32768

/* RMS norm of each row, after an optional addition:
 *   h = x + residual, rounded to `type` (h = x without a residual)
 *   y = h * rsqrt(mean(h^2) + eps) * weight
 * with the sums in fp32. out_type == type: y rounded to it (y_scales is not
 * used). out_type == PIPE_E4M3: with s = max(max|y| of the row, 2^-100) / 448,
 * y_scales[row] = s and y = y / s in e4m3; a row with a NaN, or with an
 * infinity, has a NaN scale and NaN values.
 *   type: PIPE_BF16 or PIPE_FP16, of x, residual, weight and h.
 *   N % 8 == 0 and N <= PIPE_RMSNORM_MAX_N (else PIPE_ERR_SHAPE); M arbitrary;
 *   M == 0 or N == 0 is a no-op. Bases 16-byte aligned (y 8-byte aligned where
 *   it is e4m3, y_scales 4-byte aligned), pitches >= N and multiples of 8
 *   (else PIPE_ERR_SHAPE / PIPE_ERR_ALIGN).
 *   residual and h: both NULL, or both given (else PIPE_ERR_NULL). h may be x
 *   or residual itself, y (16 bits) may be x itself, each with the same pitch;
 *   other overlaps are the caller's error. */
pipe_status_t pipe_rmsnorm(const void* x, const void* residual, const void* weight, void* y,
                           float* y_scales, void* h, int64_t M, int64_t N, int64_t ld_x,
                           int64_t ld_residual, int64_t ld_y, int64_t ld_h, float eps,
                           pipe_dtype_t type, pipe_dtype_t out_type, void* stream);

/* Bytes of workspace pipe_rmsnorm_backward needs: fp32 partials of dweight,
 * none for a few rows. */
pipe_status_t pipe_rmsnorm_backward_workspace_bytes(int64_t M, int64_t N, size_t* bytes);

/* Gradient of y = x * r * weight, r = rsqrt(mean(x^2) + eps), for the input x
 * that was normalised (pipe_rmsnorm's h):
 *   g  = dy * weight
 *   dx = r * g - x * r^3 * mean(g * x)  (+ dh), rounded once to `type`
 *   dweight = sum over the rows of dy * x * r, fp32
 * dh (nullable) is the gradient that reaches h by the residual stream; dx is
 * then the gradient of both x and residual of the forward call. dx may be dy
 * or dh itself with the same pitch. M == 0 gives dweight = 0; N == 0 is a
 * no-op. Shapes, pitches and alignment as above; dweight and workspace
 * 16-byte aligned. One or two kernels are enqueued. */
pipe_status_t pipe_rmsnorm_backward(const void* dy, const void* x, const void* weight,
                                    const void* dh, void* dx, float* dweight, int64_t M,
                                    int64_t N, int64_t ld_dy, int64_t ld_x, int64_t ld_dh,
                                    int64_t ld_dx, float eps, pipe_dtype_t type,
                                    void* workspace, size_t workspace_bytes, void* stream);

/* Bytes of workspace pipe_gemm_fp8 needs for a shape: fp32 partial products
 * where the K axis is split over workgroups, else 0. */
pipe_status_t pipe_gemm_fp8_workspace_bytes(int64_t M, int64_t N, int64_t K, size_t* bytes);

/* C[m][n] = (sum_k A[m][k] * B[n][k]) * a_scales[m] * b_scales[n], A (M x K)
 * and B (N x K, the transpose of the K x N right operand: lda, ldb >= K) in
 * e4m3, C in PIPE_BF16, PIPE_FP16 or PIPE_FP32. For fp16 and fp32 C the sum is
 * an fp32 sum. For bf16 C and five rows of A or more it is that of the 8-bit
 * matrix instructions, at twice the rate: of each eight neighbouring k's
 * products are cut off 13 bits below the largest one's leading bit, and added
 * up in fp32 from there on (1.5e-5 to 2e-4 of the result's norm, measured on
 * normal inputs and on sums that cancel; bf16's own rounding is 1.6e-3).
 *   N % 8 == 0, K % 16 == 0, M arbitrary (else PIPE_ERR_SHAPE); M == 0 or
 *   N == 0 is a no-op, K == 0 gives C = 0 (scales unread). A, B, C bases
 *   16-byte aligned, lda and ldb multiples of 16 and below 2^24 (else
 *   PIPE_ERR_SHAPE), ldc a multiple of 8, scales 4-byte and the workspace
 *   16-byte aligned (else PIPE_ERR_ALIGN). */
pipe_status_t pipe_gemm_fp8(const void* A, const float* a_scales, const void* B,
                            const float* b_scales, void* C, int64_t M, int64_t N, int64_t K,
                            int64_t lda, int64_t ldb, int64_t ldc, pipe_dtype_t out_type,
                            void* workspace, size_t workspace_bytes, void* stream);

/* Bytes of workspace pipe_gemm_w4 needs for a shape, as above. */
pipe_status_t pipe_gemm_w4_workspace_bytes(int64_t M, int64_t N, int64_t K, size_t* bytes);

/* C[m][n] = sum_k A[m][k] * (q[n][k] - z[n][k / group]) * scales[n][k / group]
 * with A (M x K), scales (N x K / group) and C in `type` (PIPE_BF16 or
 * PIPE_FP16), 4-bit codes q (two a byte, the even k's in the low half; rows of
 * ld_codes bytes) and zero points z (one uint8 of 0..15 each; NULL: 8
 * everywhere). Codes and zero points enter the products as the integers they
 * are, the scale is applied to the fp32 sum of each group, and C is rounded
 * once. A group's product is s (sum a q - z sum a): the fp32 errors are those
 * of these two sums, which may be larger than their difference. Where one of
 * them passes fp32's range (an infinite A, or bf16 values near the end of the
 * range) C is NaN, though the single weights' products may add up to a number
 * or an infinity.
 *   group: a power of two >= 32 that divides K, or K itself if K % 32 == 0
 *   (else PIPE_ERR_SHAPE). N % 8 == 0, M arbitrary (the kernels are laid out
 *   for up to 64 rows; more run in passes of 64). M == 0 or N == 0 is a no-op,
 *   K == 0 gives C = 0. A, codes and C bases 16-byte aligned, lda and ldc
 *   multiples of 8, ld_codes a multiple of 16 and >= K / 2; ld_scales and
 *   ld_zeros >= K / group, scales 2-byte, the workspace 16-byte aligned. */
pipe_status_t pipe_gemm_w4(const void* A, const void* codes, const void* scales,
                           const void* zeros, void* C, int64_t M, int64_t N, int64_t K,
                           int64_t group, int64_t lda, int64_t ld_codes, int64_t ld_scales,
                           int64_t ld_zeros, int64_t ldc, pipe_dtype_t type, void* workspace,
                           size_t workspace_bytes, void* stream);

/* The microscaled 4-bit form of a matrix of M rows and K columns, K % 32 == 0:
 *   codes: e2m1 values, two a byte, the even column's in the low half: rows of
 *   ld_codes bytes. The eight codes from 0 are 0, 0.5, 1, 1.5, 2, 3, 4, 6, the
 *   next eight their negatives.
 *   scales: a byte for 32 neighbours of a row, the exponent plus 127 of the
 *   power of two that they are multiplied by (e8m0; 255: all 32 are NaN): rows
 *   of ld_scales bytes.
 * Bases are 16-byte aligned and pitches multiples of 16 (else PIPE_ERR_ALIGN),
 * ld_scales below 2^24 (else PIPE_ERR_SHAPE).
 * Rows of scales are read in whole groups of 16 bytes: the memory up to the next
 * multiple of 16 behind a row's K / 32 bytes must exist; what it holds is not
 * used. Only the K / 32 bytes are written. */

/* Brings x (PIPE_BF16, PIPE_FP16 or PIPE_FP32) into that form. A block's power
 * of two is the largest one not above its largest magnitude, divided by 4, and
 * 2^-127 at least; the values divided by it are rounded to codes, to nearest,
 * ties to the even code; what passes 6 becomes 6 (a largest magnitude of 7
 * scales becomes 6). A block with a NaN or an infinity is NaN.
 *   K % 32 == 0, M * K at most 2^40 (else PIPE_ERR_SHAPE); M == 0 or K == 0 is
 *   a no-op. x: base 16-byte aligned, ld_x >= K and a multiple of 8. */
pipe_status_t pipe_quantize_mxfp4(const void* x, void* codes, void* scales, int64_t M, int64_t K,
                                  int64_t ld_x, int64_t ld_codes, int64_t ld_scales,
                                  pipe_dtype_t type, void* stream);

/* The values that the form stands for, rounded once to out_type (PIPE_BF16,
 * PIPE_FP16 or PIPE_FP32; only fp16 rounds, and what passes a type's range is an
 * infinity: values of 2^128 and more, which pipe_quantize_mxfp4 never makes).
 * Conditions as above, out for x. */
pipe_status_t pipe_dequantize_mxfp4(const void* codes, const void* scales, void* out, int64_t M,
                                    int64_t K, int64_t ld_codes, int64_t ld_scales, int64_t ld_out,
                                    pipe_dtype_t out_type, void* stream);

/* The widest row of the layer norm and its gradient, in elements. */
#define PIPE_LAYERNORM_MAX_N 32768

/* Layer norm of each row, after an optional addition:
 *   h = x + residual, rounded to `type` (h = x without a residual)
 *   m = mean(h), y = (h - m) * rsqrt(mean((h - m)^2) + eps) * weight + bias
 * with the sums in fp32 and the deviations from the mean itself; bias may be
 * NULL. A row with a NaN or an infinity is NaN; one of finite values whose squared
 * deviations add up past fp32's range (bf16's largest values) gives y = bias; with
 * eps == 0 one whose squared deviations are all zero in fp32 is not finite.
 * out_type == type: y rounded to it. PIPE_E4M3: y_scales are fp32, one a
 * row, as pipe_rmsnorm's. PIPE_MXFP4: y in the form above (N for K, y and ld_y
 * for codes and ld_codes, y_scales for scales), N % 32 == 0; y is rounded once,
 * to its code. ld_scales is not used but there.
 *   type: PIPE_BF16 or PIPE_FP16, of x, residual, weight, bias and h.
 *   N % 8 == 0 and N <= PIPE_LAYERNORM_MAX_N (else PIPE_ERR_SHAPE); M arbitrary;
 *   M == 0 or N == 0 is a no-op. Alignment and pitches as pipe_rmsnorm's, and
 *   so are residual and h, and what may overlap. */
pipe_status_t pipe_layernorm(const void* x, const void* residual, const void* weight,
                             const void* bias, void* y, void* y_scales, void* h, int64_t M,
                             int64_t N, int64_t ld_x, int64_t ld_residual, int64_t ld_y,
                             int64_t ld_scales, int64_t ld_h, float eps, pipe_dtype_t type,
                             pipe_dtype_t out_type, void* stream);

/* Bytes of workspace pipe_layernorm_backward needs: fp32 partials of dweight and
 * dbias, none where one workgroup takes all rows. */
pipe_status_t pipe_layernorm_backward_workspace_bytes(int64_t M, int64_t N, size_t* bytes);

/* Gradient of y = u * weight + bias, u = (x - m) * r, r = rsqrt(mean((x - m)^2) +
 * eps), for the input x that was normalised (pipe_layernorm's h):
 *   g  = dy * weight
 *   dx = r * (g - mean(g) - u * mean(g * u))  (+ dh), rounded once to `type`
 *   dweight = sum over the rows of dy * u, dbias = sum over the rows of dy, fp32
 * dh (nullable) and overlaps as pipe_rmsnorm_backward's. M == 0 gives dweight =
 * dbias = 0; N == 0 is a no-op. Shapes, pitches and alignment as above; dweight,
 * dbias and workspace 16-byte aligned. One or two kernels are enqueued. A row's dx
 * does not depend on how many rows there are, nor do pipe_layernorm's y and h. A row
 * of finite values whose squared deviations add up past fp32's range has u = 0 and
 * dx = 0 (+ dh). dy * weight * (x - m) and its sum over a row are fp32 values: where
 * one passes that range, the row's dx is not finite. */
pipe_status_t pipe_layernorm_backward(const void* dy, const void* x, const void* weight,
                                      const void* dh, void* dx, float* dweight, float* dbias,
                                      int64_t M, int64_t N, int64_t ld_dy, int64_t ld_x,
                                      int64_t ld_dh, int64_t ld_dx, float eps, pipe_dtype_t type,
                                      void* workspace, size_t workspace_bytes, void* stream);

/* Bytes of workspace pipe_gemm_mxfp4 needs for a shape: fp32 partial products
 * where the K axis is split over workgroups, both operands' scales laid out anew
 * for the largest products, else 0. */
pipe_status_t pipe_gemm_mxfp4_workspace_bytes(int64_t M, int64_t N, int64_t K, size_t* bytes);

/* C[m][n] = sum_k A[m][k] * W[n][k], A (M x K) and W (N x K) in the form above
 * (lda and ldw in bytes, >= K / 2), C in PIPE_BF16, PIPE_FP16 or PIPE_FP32. A
 * block's 32 products add up exactly, the blocks in fp32; what is below fp32's
 * normal range may count as zero.
 *   N % 8 == 0, K % 32 == 0, M arbitrary (else PIPE_ERR_SHAPE); M == 0 or N == 0
 *   is a no-op, K == 0 gives C = 0. lda and ldw below 2^24 (else
 *   PIPE_ERR_SHAPE), C's base and the workspace 16-byte aligned, ldc a multiple
 *   of 8 (else PIPE_ERR_ALIGN). */
pipe_status_t pipe_gemm_mxfp4(const void* A, const void* a_scales, const void* W,
                              const void* w_scales, void* C, int64_t M, int64_t N, int64_t K,
                              int64_t lda, int64_t ld_a_scales, int64_t ldw, int64_t ld_w_scales,
                              int64_t ldc, pipe_dtype_t out_type, void* workspace,
                              size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* PIPE_LINEAR_H */
