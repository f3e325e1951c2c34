// 16-bit and 32-bit rows into the microscaled 4-bit form, and back.
//
// A thread takes chunks of 16 bytes of the wide side; the four or eight lanes of a
// block of 32 find its largest magnitude by two or three exchanges. Dividing by the block's power of two is
// exact, so each value is rounded once, to its code; on the way back the product
// of code and power of two is exact in fp32 and rounded once, to the output's
// type. Both are bound by memory: a few operations for every byte moved.
//
// 28672 x 8192 bf16 there and back takes 173 to 185 us (6.4 TB/s or more): codes are
// written and read through the caches, since what reads them comes next (212 with
// non-temporal stores of them), wide rows past them (209 with cached stores on the way
// back); 28672 x 4096 fp32 168 us (197 and 194). Into the form with four chunks a thread,
// 99 us (100 with two, 104 with eight); back with one, 82 us over the same output again
// (84 with two, 85 with four) and 114 over others.
#include "pipe_mx.hpp"

namespace pipe {

namespace {

constexpr int kThreads = 256;
constexpr int kChunks = 4;   // a thread, into the form; all loads ahead of the first use

// A chunk's 16 bytes and its values, in bf16, fp16 or fp32; the unsigned type of its codes.
template <int TYPE>
struct Elem;
template <>
struct Elem<2> {
  static constexpr int kCount = 4;
  using Codes = uint16_t;
  static __device__ __forceinline__ void get(u32x4 w, float (&f)[4]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) f[e] = __uint_as_float(w[e]);
  }
  static __device__ __forceinline__ u32x4 put(const float (&f)[4]) {
    u32x4 w;
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = __float_as_uint(f[e]);
    return w;
  }
};
template <class T>
struct Elem16 {
  static constexpr int kCount = 8;
  using Codes = uint32_t;
  static __device__ __forceinline__ void get(u32x4 w, float (&f)[8]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      f[2 * e] = Pair<T>::lo(w[e]);
      f[2 * e + 1] = Pair<T>::hi(w[e]);
    }
  }
  static __device__ __forceinline__ u32x4 put(const float (&f)[8]) {
    u32x4 w;
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = Pair<T>::pack(f[2 * e], f[2 * e + 1]);
    return w;
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
  using Codes = typename E::Codes;
  constexpr int kLanes = kMxBlock / E::kCount;   // of a block
  const int64_t first = long_block() * (kThreads * kChunks);
  if (first >= p.chunks) return;
  const Walk walk(p, first);
  Place at[kChunks];
  u32x4 w[kChunks];
#pragma unroll
  for (int i = 0; i < kChunks; ++i) {
    const uint32_t u = threadIdx.x + kThreads * i;
    at[i] = walk.at(p, u);
    if (first + u < p.chunks)
      w[i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p.x + at[i].row * p.ld_x) + at[i].col);
    else
      w[i] = u32x4{0, 0, 0, 0};
  }
#pragma unroll
  for (int i = 0; i < kChunks; ++i) {
    float f[E::kCount];
    E::get(w[i], f);
    const uint32_t exponent = mx_exponent(mx_top(f));
    const Codes codes = (Codes)mx_codes(f, mx_scale(exponent));
    if (first + threadIdx.x + kThreads * i < p.chunks) {
      reinterpret_cast<Codes*>(p.codes + at[i].row * p.ld_codes)[at[i].col] = codes;
      if (threadIdx.x % kLanes == 0)
        p.scales[at[i].row * p.ld_scales + at[i].col / kLanes] = (uint8_t)exponent;
    }
  }
}

template <int TYPE>
__global__ void __launch_bounds__(kThreads) mx_dequantize_kernel(MxQuantParams p) {
  using E = Elem<TYPE>;
  using Codes = typename E::Codes;
  constexpr int kLanes = kMxBlock / E::kCount;   // of a block
  const int64_t first = long_block() * kThreads;
  if (first + threadIdx.x >= p.chunks) return;
  const Place at = Walk(p, first).at(p, threadIdx.x);
  const uint32_t codes = reinterpret_cast<const Codes*>(p.codes_in + at.row * p.ld_codes)[at.col];
  const float scale = mx_scale(p.scales_in[at.row * p.ld_scales + at.col / kLanes]);
  const f32x2 v[4] = {__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.f, 0),
                      __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.f, 1),
                      __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.f, 2),
                      __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.f, 3)};
  float f[E::kCount];
#pragma unroll
  for (int e = 0; e < E::kCount; ++e) f[e] = v[e >> 1][e & 1] * scale;
  __builtin_nontemporal_store(E::put(f), reinterpret_cast<u32x4*>(p.out + at.row * p.ld_out) + at.col);
}

hipError_t launch(void (*kernel)(MxQuantParams), const MxQuantParams& p, int chunks, hipStream_t stream) {
  const int each = kThreads * chunks;
  hipLaunchKernelGGL(kernel, long_grid((p.chunks + each - 1) / each), dim3(kThreads), 0, stream, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_mx_quantize(const MxQuantParams& p, int type, hipStream_t stream) {
  return launch(type == 0   ? mx_quantize_kernel<0>
                : type == 1 ? mx_quantize_kernel<1>
                            : mx_quantize_kernel<2>,
                p, kChunks, stream);
}

hipError_t launch_mx_dequantize(const MxQuantParams& p, int type, hipStream_t stream) {
  return launch(type == 0   ? mx_dequantize_kernel<0>
                : type == 1 ? mx_dequantize_kernel<1>
                            : mx_dequantize_kernel<2>,
                p, 1, stream);
}

}  // namespace pipe
