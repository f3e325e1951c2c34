// The microscaled 4-bit form: 32 neighbours of a row share one power of two, held
// as its exponent plus 127 (e8m0; 255 is a NaN), and each is an e2m1 value, 0, 0.5,
// 1, 1.5, 2, 3, 4, 6 or a negative of these, two a byte.
#pragma once

#include "pipe_norm.hpp"

namespace pipe {

constexpr int kMxBlock = 32;   // neighbours that share a scale

struct MxQuantParams {
  const uint8_t *x, *codes_in, *scales_in;
  uint8_t *codes, *scales, *out;
  int64_t ld_x, ld_codes, ld_scales, ld_out;  // bytes
  int64_t chunks;       // chunks of 16 bytes of the 16- or 32-bit side in all
  uint32_t row_chunks;  // in a row
  uint32_t reciprocal;  // floor(2^32 / row_chunks)
};

struct MxGemmParams {
  const uint8_t *A, *W, *a_scales, *w_scales;
  void* C;
  float* partials;  // the workspace: scales laid out anew, if any, then [splits][M][N] where splits > 1
  int64_t lda, ldw, ld_as, ld_ws, ldc;  // bytes, but ldc: elements
  int64_t step_as, step_ws;             // bytes between the scales of two pairs of stages
  int32_t M, N, bytes;                  // bytes of a row: K / 2
  int32_t tiles_m, tiles_n, splits, steps;  // K steps of a whole row
};

hipError_t launch_mx_quantize(const MxQuantParams& p, int type, hipStream_t stream);
hipError_t launch_mx_dequantize(const MxQuantParams& p, int type, hipStream_t stream);
int64_t gemm_mx_partials(int64_t M, int64_t N, int64_t K);  // floats of workspace
hipError_t launch_gemm_mx(MxGemmParams p, int out_type, hipStream_t stream);

// A block's e8m0 byte from the bits of its largest magnitude: the largest power of
// two not above it, divided by 4 (e2m1's largest power of two), 2^-127 at least.
// A NaN or an infinity makes the block NaN.
__device__ __forceinline__ uint32_t mx_exponent(uint32_t top) {
  const uint32_t e = top >> 23;
  return e == 255 ? 255 : e < 2 ? 0 : e - 2;
}
// The power of two that an e8m0 byte stands for.
__device__ __forceinline__ float mx_scale(uint32_t e) {
  return __uint_as_float(e == 0 ? 0x00400000u : e == 255 ? 0x7FC00000u : e << 23);
}
// Largest of the magnitudes' bits over a block: 8 elements each of four lanes, or 4
// of eight.
template <int COUNT>
__device__ __forceinline__ uint32_t mx_top(const float (&f)[COUNT]) {
  uint32_t top = 0;
#pragma unroll
  for (int e = 0; e < COUNT; ++e) top = max(top, abs_bits(f[e]));
  top = dpp_max<0xB1, 0xF>(top);   // quad permutations [1,0,3,2] and [2,3,0,1]
  top = dpp_max<0x4E, 0xF>(top);
  if constexpr (COUNT == 4) top = dpp_max<0x141, 0xF>(top);   // lane 7 - i of each eight
  return top;
}
// Values divided by the scale and rounded to codes, to nearest, ties to the even
// code; what passes 6 becomes 6.
template <int COUNT>
__device__ __forceinline__ uint32_t mx_codes(const float (&f)[COUNT], float scale) {
  uint32_t w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, f[0], f[1], scale, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f[2], f[3], scale, 1);
  if constexpr (COUNT == 8) {
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f[4], f[5], scale, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f[6], f[7], scale, 3);
  }
  return w;
}

}  // namespace pipe
