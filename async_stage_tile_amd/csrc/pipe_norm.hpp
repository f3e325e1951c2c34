// Shared pieces of the norms' kernels: the e4m3 output's constants, packed
// rows in registers.
#pragma once

#include "pipe_linear.hpp"

namespace pipe {

constexpr float kE4m3Max = 448.f;
constexpr float kAmaxMin = 0x1p-100f;  // keeps the scale and its reciprocal normal numbers

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// Keeps the 16-bit pairs as what stays in registers across a reduction: without
// it the compiler keeps their fp32 values, twice the registers.
template <int CH>
__device__ __forceinline__ void keep_packed(u32x4 (&v)[CH]) {
#pragma unroll
  for (int i = 0; i < CH; ++i) asm("" : "+v"(v[i]));
}

}  // namespace pipe
