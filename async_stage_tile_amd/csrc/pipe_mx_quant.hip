// 16-bit and 32-bit rows into the microscaled 4-bit form, and back.
//
// A thread takes chunks of 8 elements; the four lanes of a block of 32 find its
// largest magnitude by two exchanges. Dividing by the block's power of two is
// exact, so each value is rounded once, to its code; on the way back the product
// of code and power of two is exact in fp32 and rounded once, to the output's
// type. Both are bound by memory: a few operations for every byte moved.
#include "pipe_mx.hpp"

namespace pipe {

namespace {

constexpr int kThreads = 256, kChunks = 4;   // chunks a thread, all loads ahead of the first use

template <int TYPE>
struct Elem;   // 0 bf16, 1 fp16, 2 fp32: a chunk of 8 in words, and its values
template <>
struct Elem<2> {
  static constexpr int kWords = 8;
  static __device__ __forceinline__ void get(const uint32_t (&w)[8], float (&f)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = __uint_as_float(w[e]);
  }
  static __device__ __forceinline__ void put(const float (&f)[8], uint32_t (&w)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = __float_as_uint(f[e]);
  }
};
template <class T>
struct Elem16 {
  static constexpr int kWords = 4;
  static __device__ __forceinline__ void get(const uint32_t (&w)[4], float (&f)[8]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      f[2 * e] = Pair<T>::lo(w[e]);
      f[2 * e + 1] = Pair<T>::hi(w[e]);
    }
  }
  static __device__ __forceinline__ void put(const float (&f)[8], uint32_t (&w)[4]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = Pair<T>::pack(f[2 * e], f[2 * e + 1]);
  }
};
template <>
struct Elem<0> : Elem16<__bf16> {};
template <>
struct Elem<1> : Elem16<_Float16> {};

// Row and place in it of a workgroup's chunks. One division of 64 bits a
// workgroup; a chunk's by the reciprocal, whose quotient is the true one or one
// less for every 32-bit number.
struct Place {
  int64_t row;
  uint32_t col;
};
struct Walk {
  int64_t first_row;
  uint32_t rest;
  __device__ __forceinline__ Walk(const MxQuantParams& p, int64_t first) {
    first_row = first / p.row_chunks;
    rest = (uint32_t)(first - first_row * p.row_chunks);
  }
  __device__ __forceinline__ Place at(const MxQuantParams& p, uint32_t i) const {
    const uint32_t n = rest + i;
    uint32_t q = __umulhi(n, p.reciprocal);
    uint32_t r = n - q * p.row_chunks;
    if (r >= p.row_chunks) {
      ++q;
      r -= p.row_chunks;
    }
    return Place{first_row + q, r};
  }
};

template <int TYPE>
__global__ void __launch_bounds__(kThreads) mx_quantize_kernel(MxQuantParams p) {
  using E = Elem<TYPE>;
  const int64_t first = long_block() * (kThreads * kChunks);
  if (first >= p.chunks) return;
  const Walk walk(p, first);
  Place at[kChunks];
  uint32_t w[kChunks][E::kWords];
#pragma unroll
  for (int i = 0; i < kChunks; ++i) {
    const uint32_t u = threadIdx.x + kThreads * i;
    at[i] = walk.at(p, u);
    if (first + u < p.chunks) {
      const u32x4* src = reinterpret_cast<const u32x4*>(p.x + at[i].row * p.ld_x) + (int64_t)at[i].col * (E::kWords / 4);
#pragma unroll
      for (int q = 0; q < E::kWords / 4; ++q) {
        const u32x4 v = __builtin_nontemporal_load(src + q);
#pragma unroll
        for (int e = 0; e < 4; ++e) w[i][4 * q + e] = v[e];
      }
    } else {
#pragma unroll
      for (int e = 0; e < E::kWords; ++e) w[i][e] = 0;
    }
  }
#pragma unroll
  for (int i = 0; i < kChunks; ++i) {
    float f[8];
    E::get(w[i], f);
    const uint32_t exponent = mx_exponent(mx_top(f));
    const uint32_t codes = mx_codes(f, mx_scale(exponent));
    if (first + threadIdx.x + kThreads * i < p.chunks) {
      *reinterpret_cast<uint32_t*>(p.codes + at[i].row * p.ld_codes + (int64_t)at[i].col * 4) = codes;
      if ((threadIdx.x & 3) == 0) p.scales[at[i].row * p.ld_scales + (at[i].col >> 2)] = (uint8_t)exponent;
    }
  }
}

template <int TYPE>
__global__ void __launch_bounds__(kThreads) mx_dequantize_kernel(MxQuantParams p) {
  using E = Elem<TYPE>;
  const int64_t first = long_block() * (kThreads * kChunks);
  if (first >= p.chunks) return;
  const Walk walk(p, first);
  Place at[kChunks];
  uint32_t codes[kChunks], exponent[kChunks];
#pragma unroll
  for (int i = 0; i < kChunks; ++i) {
    const uint32_t u = threadIdx.x + kThreads * i;
    at[i] = walk.at(p, u);
    codes[i] = exponent[i] = 0;
    if (first + u < p.chunks) {
      codes[i] = __builtin_nontemporal_load(
          reinterpret_cast<const uint32_t*>(p.codes_in + at[i].row * p.ld_codes + (int64_t)at[i].col * 4));
      exponent[i] = p.scales_in[at[i].row * p.ld_scales + (at[i].col >> 2)];
    }
  }
#pragma unroll
  for (int i = 0; i < kChunks; ++i) {
    const float scale = mx_scale(exponent[i]);
    const f32x2 v[4] = {__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes[i], 1.f, 0),
                        __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes[i], 1.f, 1),
                        __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes[i], 1.f, 2),
                        __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes[i], 1.f, 3)};
    float f[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = v[e >> 1][e & 1] * scale;
    uint32_t w[E::kWords];
    E::put(f, w);
    if (first + threadIdx.x + kThreads * i < p.chunks) {
      u32x4* out = reinterpret_cast<u32x4*>(p.out + at[i].row * p.ld_out) + (int64_t)at[i].col * (E::kWords / 4);
#pragma unroll
      for (int q = 0; q < E::kWords / 4; ++q)
        out[q] = u32x4{w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]};
    }
  }
}

hipError_t launch(void (*kernel)(MxQuantParams), const MxQuantParams& p, hipStream_t stream) {
  constexpr int kEach = kThreads * kChunks;
  hipLaunchKernelGGL(kernel, long_grid((p.chunks + kEach - 1) / kEach), dim3(kThreads), 0, stream, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_mx_quantize(const MxQuantParams& p, int type, hipStream_t stream) {
  return launch(type == 0   ? mx_quantize_kernel<0>
                : type == 1 ? mx_quantize_kernel<1>
                            : mx_quantize_kernel<2>,
                p, stream);
}

hipError_t launch_mx_dequantize(const MxQuantParams& p, int type, hipStream_t stream) {
  return launch(type == 0   ? mx_dequantize_kernel<0>
                : type == 1 ? mx_dequantize_kernel<1>
                            : mx_dequantize_kernel<2>,
                p, stream);
}

}  // namespace pipe
