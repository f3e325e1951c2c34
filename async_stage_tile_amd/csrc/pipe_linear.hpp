// Shared pieces of the quantised linear layer's kernels: launch parameters,
// 16-bit types, wave reductions.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace pipe {

struct NormParams {
  const uint8_t *x, *residual, *weight;
  uint8_t *y, *h;
  float* scales;
  int64_t ld_x, ld_residual, ld_y, ld_h;  // bytes
  int64_t M;
  int32_t chunks;  // 8-element chunks in a row
  float inv_n, eps;
};

struct NormGradParams {
  const uint8_t *dy, *x, *weight, *dh;
  uint8_t* dx;
  float* partials;  // [workgroups][N]
  int64_t ld_dy, ld_x, ld_dh, ld_dx;  // bytes
  int64_t M;
  int32_t chunks;
  float inv_n, eps;
};

struct LayerNormParams {
  const uint8_t *x, *residual, *weight, *bias;
  uint8_t *y, *h, *scales;  // scales: fp32, one a row, or e8m0
  int64_t ld_x, ld_residual, ld_y, ld_h, ld_scales;  // bytes
  int64_t M;
  int32_t chunks;  // 8-element chunks in a row
  float inv_n, eps;
};

struct LayerNormGradParams {
  const uint8_t *dy, *x, *weight, *dh;
  uint8_t* dx;
  float *sum_weight, *sum_bias;  // a workgroup's are sum_stride floats further each
  int64_t sum_stride;
  int64_t ld_dy, ld_x, ld_dh, ld_dx;  // bytes
  int64_t M;
  int32_t chunks;
  float inv_n, eps;
};

struct Fp8Params {
  const uint8_t *A, *B;
  const float *a_scales, *b_scales;
  void* C;
  float* partials;                    // [splits][M][N] where splits > 1
  int64_t lda, ldb, ldc;              // bytes, bytes, elements
  int32_t M, N, K;
  int32_t tiles_m, tiles_n, splits, steps;  // K steps of a whole row
};

struct W4Params {
  const uint8_t *A, *codes, *zeros;
  const uint16_t* scales;
  uint8_t* C;
  float* partials;                    // [splits][M][N] where splits > 1
  int64_t lda, ld_codes, ld_scales, ld_zeros, ldc;  // bytes, bytes, elements, bytes, elements
  int32_t M, N, K;
  int32_t group_shift;  // log2 of the group size; 31 for one group a row
  int32_t splits;
};

// Each launcher takes what its entry point has checked. Types: 0 bf16, 1 fp16,
// 2 fp32, 3 e4m3 (pipe_dtype_t).
hipError_t launch_rmsnorm(const NormParams& p, int type, bool q8, hipStream_t stream);
int64_t rmsnorm_grad_partials(int64_t M, int64_t N);  // rows of N floats
hipError_t launch_rmsnorm_grad(NormGradParams p, float* dweight, int type, hipStream_t stream);
hipError_t launch_layernorm(const LayerNormParams& p, int type, int out, hipStream_t stream);  // out: 0 type, 1 e4m3, 2 4-bit
int64_t layernorm_grad_partials(int64_t M, int64_t N);  // rows of N floats
hipError_t launch_layernorm_grad(LayerNormGradParams p, float* partials, float* dweight, float* dbias,
                                 int type, hipStream_t stream);
int64_t gemm_fp8_partials(int64_t M, int64_t N, int64_t K);  // floats of workspace
hipError_t launch_gemm_fp8(Fp8Params p, int out_type, hipStream_t stream);
int64_t gemm_w4_partials(int64_t M, int64_t N, int64_t K);  // floats of workspace
hipError_t launch_gemm_w4(W4Params p, int type, hipStream_t stream);

// A one-dimensional grid of any length in two dimensions (a launch takes fewer
// than 2^32 threads along x). Workgroups past the end leave at once or compute
// what is dropped.
inline dim3 long_grid(int64_t workgroups) {
  constexpr int64_t kWide = 1 << 20;
  if (workgroups <= kWide) return dim3((unsigned)workgroups);
  return dim3((unsigned)kWide, (unsigned)((workgroups + kWide - 1) / kWide));
}
__device__ __forceinline__ int64_t long_block() {
  return (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
}

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

// A 16-bit type T as pairs in 32-bit words. Rounding is to nearest even.
template <class T>
struct Pair;
template <>
struct Pair<__bf16> {
  static __device__ __forceinline__ float lo(uint32_t w) { return __uint_as_float(w << 16); }
  static __device__ __forceinline__ float hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    const f32x2 v = {a, b};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
  }
};
template <>
struct Pair<_Float16> {
  static __device__ __forceinline__ float lo(uint32_t w) {
    return (float)__builtin_bit_cast(f16x2, w)[0];
  }
  static __device__ __forceinline__ float hi(uint32_t w) {
    return (float)__builtin_bit_cast(f16x2, w)[1];
  }
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    const f32x2 v = {a, b};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, f16x2));
  }
};

// One step of a reduction to lane 63: v combined with v of the lanes that the
// DPP control names; lanes without a source combine with 0.
template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp_add(float v) {
  return v + __uint_as_float(__builtin_amdgcn_update_dpp(0u, __float_as_uint(v), CTRL, ROWS, 0xF, false));
}
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp_max(uint32_t v) {
  const uint32_t o = __builtin_amdgcn_update_dpp(0u, v, CTRL, ROWS, 0xF, false);
  return v > o ? v : o;
}

// Sum and unsigned maximum over the 64 lanes, wave-uniform results: shifts by
// 1, 2, 4, 8 within rows of 16, then broadcasts of lane 15 and lane 31.
__device__ __forceinline__ float wave_sum(float v) {
  v = dpp_add<0x111, 0xF>(v);
  v = dpp_add<0x112, 0xF>(v);
  v = dpp_add<0x114, 0xF>(v);
  v = dpp_add<0x118, 0xF>(v);
  v = dpp_add<0x142, 0xA>(v);
  v = dpp_add<0x143, 0xC>(v);
  return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), 63));
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  v = dpp_max<0x111, 0xF>(v);
  v = dpp_max<0x112, 0xF>(v);
  v = dpp_max<0x114, 0xF>(v);
  v = dpp_max<0x118, 0xF>(v);
  v = dpp_max<0x142, 0xA>(v);
  v = dpp_max<0x143, 0xC>(v);
  return __builtin_amdgcn_readlane(v, 63);
}

// Sum over each aligned group of N lanes (8, 16 or 32), in every lane of it.
template <int N>
__device__ __forceinline__ float group_sum(float s) {
  s = dpp_add<0xB1, 0xF>(s);    // quad permutations [1,0,3,2] and [2,3,0,1]
  s = dpp_add<0x4E, 0xF>(s);
  s = dpp_add<0x141, 0xF>(s);   // mirror of 8 lanes
  if constexpr (N >= 16) s = dpp_add<0x140, 0xF>(s);   // mirror of 16
  if constexpr (N >= 32) {
    const u32x2 x = __builtin_amdgcn_permlane16_swap(__float_as_uint(s), __float_as_uint(s), false,
                                                     false);
    s = __uint_as_float(x[0]) + __uint_as_float(x[1]);
  }
  return s;
}

// Sums over the 64 lanes of eight registers: each swap and addition halves the
// registers and keeps, in each part of the lanes, another one's sums. Row
// 4 q + {0, 2, 1, 3}[lane / 16] of the eight ends up in out[q].
__device__ __forceinline__ void sum_rows(const float (&v)[8], float (&out)[2]) {
  float h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const u32x2 x = __builtin_amdgcn_permlane32_swap(__float_as_uint(v[2 * i]),
                                                     __float_as_uint(v[2 * i + 1]), false, false);
    h[i] = __uint_as_float(x[0]) + __uint_as_float(x[1]);
  }
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const u32x2 x = __builtin_amdgcn_permlane16_swap(__float_as_uint(h[2 * q]),
                                                     __float_as_uint(h[2 * q + 1]), false, false);
    float s = __uint_as_float(x[0]) + __uint_as_float(x[1]);
    s = dpp_add<0x121, 0xF>(s);   // rotations within rows of 16 lanes
    s = dpp_add<0x122, 0xF>(s);
    s = dpp_add<0x124, 0xF>(s);
    out[q] = dpp_add<0x128, 0xF>(s);
  }
}

// Store four consecutive outputs of type OUT (0 bf16, 1 fp16, 2 fp32).
template <int OUT>
__device__ __forceinline__ void store4(void* c, int64_t at, f32x4 v) {
  if constexpr (OUT == 2) {
    *reinterpret_cast<f32x4*>(static_cast<float*>(c) + at) = v;
  } else {
    u32x2 w;
    if constexpr (OUT == 0) {
      w = u32x2{Pair<__bf16>::pack(v[0], v[1]), Pair<__bf16>::pack(v[2], v[3])};
    } else {
      w = u32x2{Pair<_Float16>::pack(v[0], v[1]), Pair<_Float16>::pack(v[2], v[3])};
    }
    *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(c) + at) = w;
  }
}

}  // namespace pipe
