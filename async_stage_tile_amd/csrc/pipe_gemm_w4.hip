// Products of 16-bit rows with 4-bit weights: C = A ((q - z) s)^T, a scale and
// a zero point for each group of K.
//
// For up to 64 rows the call is bound by reading the weights once: N K / 2
// bytes of codes, for a few operations each. So the codes go from memory
// straight into registers, 16 bytes (32 codes) a lane, become 16-bit integers
// there, and enter v_mfma_f32_16x16x32 with the rows of A as the other
// operand. The waves of a workgroup share 16 NT weight rows and split K
// between them in blocks of 128, each next block going to the next wave, so
// that the workgroup as a whole reads long runs of each row; their sums meet
// in LDS at the end, in wave order.
//
// Integers: a byte 0..15 is, read as e4m3, q * 2^-9 (the subnormals and the
// first binade are evenly spaced), so one v_cvt_scalef32_pk with scale 2^9
// turns two of them into 16-bit floats exactly: 7 operations for 8 codes,
// shift and masks included.
//
// Scales and zero points: over one group (q - z) s = s q - s z, so with
// P = sum_k a q and S = sum_k a of the group, acc += s P - (s z) S. P is the
// MFMA's sum over the group and S that of one more MFMA, against ones, that
// the wave's NT column tiles share. Everything is exact or fp32; no weight is
// rounded to 16 bits.
//
// K order: within a lane's 8 codes of an MFMA the order is even k's, then odd
// (as the masks leave them), and A's pairs are permuted alike. Over the lanes,
// groups of 128 and more take a lane's four words as they come: word t of
// quarter q (16 lanes) holds k = 32 q + 8 t .. + 7, and A's lanes load that.
// Smaller groups need every MFMA inside 32 consecutive k's: the words of the
// four quarters are transposed first (two 16-lane and two 32-lane swaps), after
// which word t of quarter q holds k = 32 t + 8 q .. + 7.
#include "pipe_linear.hpp"

namespace pipe {

namespace {

template <class T>
struct Mma;
template <>
struct Mma<__bf16> {
  static constexpr uint32_t kOnes = 0x3F803F80u;
  static __device__ __forceinline__ uint32_t codes_lo(uint32_t b) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 512.f, false));
  }
  static __device__ __forceinline__ uint32_t codes_hi(uint32_t b) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 512.f, true));
  }
  static __device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  }
  static __device__ __forceinline__ float to_float(uint16_t v) { return Pair<__bf16>::lo(v); }
  static __device__ __forceinline__ uint32_t pack(float a, float b) { return Pair<__bf16>::pack(a, b); }
};
template <>
struct Mma<_Float16> {
  static constexpr uint32_t kOnes = 0x3C003C00u;
  static __device__ __forceinline__ uint32_t codes_lo(uint32_t b) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, 512.f, false));
  }
  static __device__ __forceinline__ uint32_t codes_hi(uint32_t b) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, 512.f, true));
  }
  static __device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                  __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  }
  static __device__ __forceinline__ float to_float(uint16_t v) { return Pair<_Float16>::lo(v); }
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    return Pair<_Float16>::pack(a, b);
  }
};

// 8 codes as 16-bit floats: k0 k2 | k4 k6 | k1 k3 | k5 k7.
template <class T>
__device__ __forceinline__ u32x4 expand(uint32_t codes) {
  const uint32_t even = codes & 0x0F0F0F0Fu, odd = (codes >> 4) & 0x0F0F0F0Fu;
  return u32x4{Mma<T>::codes_lo(even), Mma<T>::codes_hi(even), Mma<T>::codes_lo(odd),
               Mma<T>::codes_hi(odd)};
}

// A's 8 values in the order of expand().
__device__ __forceinline__ u32x4 even_odd(u32x4 a) {
  return u32x4{__builtin_amdgcn_perm(a[1], a[0], 0x05040100u),
               __builtin_amdgcn_perm(a[3], a[2], 0x05040100u),
               __builtin_amdgcn_perm(a[1], a[0], 0x07060302u),
               __builtin_amdgcn_perm(a[3], a[2], 0x07060302u)};
}

// Word t of quarter q <- word q of quarter t.
__device__ __forceinline__ u32x4 transpose_quarters(u32x4 w) {
  const u32x2 a = __builtin_amdgcn_permlane16_swap(w[0], w[1], false, false);
  const u32x2 b = __builtin_amdgcn_permlane16_swap(w[2], w[3], false, false);
  const u32x2 c = __builtin_amdgcn_permlane32_swap(a[0], b[0], false, false);
  const u32x2 d = __builtin_amdgcn_permlane32_swap(a[1], b[1], false, false);
  return u32x4{c[0], d[0], c[1], d[1]};
}

// Scales and zero points of the groups of one block, at any alignment.
template <int N>
struct Packed;
template <>
struct Packed<1> {
  typedef uint16_t scales;
  typedef uint8_t zeros;
};
template <>
struct Packed<2> {
  typedef uint16_t scales __attribute__((ext_vector_type(2), aligned(2)));
  typedef uint8_t zeros __attribute__((ext_vector_type(2), aligned(1)));
};
template <>
struct Packed<4> {
  typedef uint16_t scales __attribute__((ext_vector_type(4), aligned(2)));
  typedef uint8_t zeros __attribute__((ext_vector_type(4), aligned(1)));
};

// What a wave holds of one block of 128 k's.
template <int MT, int NT, int FLUSHES>
struct Block {
  u32x4 w[NT];
  u32x4 a[MT][4];
  uint16_t s[NT][FLUSHES];
  uint8_t z[NT][FLUSHES];
};

// MT, NT: 16-row tiles of A and of the weights that a wave holds. WAVES split
// K. F: k's between two scalings, the group size or 128 if that is larger.
// Rows past M and N are read from the last row and dropped.
template <class T, int MT, int NT, int WAVES, int F, bool ZEROS>
__global__ void __launch_bounds__(64 * WAVES) gemm_w4_kernel(W4Params p) {
  constexpr int kFlushes = 128 / F;   // scalings in a block
  constexpr int kTiles = MT * NT;
  using Blk = Block<MT, NT, kFlushes>;
  __shared__ f32x4 red[WAVES][kTiles][64];
  const int lane = (int)(threadIdx.x & 63);
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int li = lane & 15, lq = lane >> 4;
  // Workgroups that share weight rows are neighbours.
  const int m_tiles = (p.M + 16 * MT - 1) / (16 * MT);
  const int64_t wg = long_block();
  if (wg >= (int64_t)m_tiles * ((p.N + 16 * NT - 1) / (16 * NT))) return;
  const int n0 = (int)(wg / m_tiles) * (16 * NT), m0 = (int)(wg % m_tiles) * (16 * MT);

  const uint8_t* code_row[NT];
  const uint16_t* scale_row[NT];
  const uint8_t* zero_row[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int n = min(n0 + 16 * j + li, p.N - 1);
    code_row[j] = p.codes + (int64_t)n * p.ld_codes + 16 * lq;
    scale_row[j] = p.scales + (int64_t)n * p.ld_scales;
    zero_row[j] = ZEROS ? p.zeros + (int64_t)n * p.ld_zeros : nullptr;
  }
  const uint8_t* a_row[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) a_row[i] = p.A + (int64_t)min(m0 + 16 * i + li, p.M - 1) * p.lda;
  f32x4 acc[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  const u32x4 ones = {Mma<T>::kOnes, Mma<T>::kOnes, Mma<T>::kOnes, Mma<T>::kOnes};

  // A's k's of MFMA step t in this lane.
  const auto a_k = [&](int t) { return F < 128 ? 32 * t + 8 * lq : 32 * lq + 8 * t; };
  const auto load = [&](Blk& blk, int k0) {
#pragma unroll
    for (int j = 0; j < NT; ++j)
      blk.w[j] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(code_row[j] + (k0 >> 1)));
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int g = k0 >> p.group_shift;
      using P = Packed<kFlushes>;
      *reinterpret_cast<typename P::scales*>(&blk.s[j]) =
          *reinterpret_cast<const typename P::scales*>(scale_row[j] + g);
      if constexpr (ZEROS)
        *reinterpret_cast<typename P::zeros*>(&blk.z[j]) =
            *reinterpret_cast<const typename P::zeros*>(zero_row[j] + g);
    }
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int t = 0; t < 4; ++t)
        blk.a[i][t] = *reinterpret_cast<const u32x4*>(a_row[i] + 2 * (int64_t)(k0 + a_k(t)));
  };
  // The last block of a K that is no multiple of 128: addresses stay in the
  // row, and A and the scales are zeros past K.
  const auto load_tail = [&](Blk& blk, int k0) {
    const u32x4 zero4 = {0, 0, 0, 0};
    const int back = k0 + 32 * lq < p.K ? 0 : 16 * lq;
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      blk.w[j] = *reinterpret_cast<const u32x4*>(code_row[j] + (k0 >> 1) - back);
#pragma unroll
      for (int f = 0; f < kFlushes; ++f) {
        const int k = k0 + f * F, g = min(k, p.K - 1) >> p.group_shift;
        blk.s[j][f] = k < p.K ? scale_row[j][g] : 0;
        if constexpr (ZEROS) blk.z[j][f] = zero_row[j][g];
      }
    }
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const int k = k0 + a_k(t);
        const u32x4 v = *reinterpret_cast<const u32x4*>(a_row[i] + 2 * (int64_t)min(k, p.K - 8));
        blk.a[i][t] = k < p.K ? v : zero4;
      }
  };
  const auto compute = [&](Blk& blk) {
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int t = 0; t < 4; ++t) blk.a[i][t] = even_odd(blk.a[i][t]);
    if constexpr (F < 128) {
#pragma unroll
      for (int j = 0; j < NT; ++j) blk.w[j] = transpose_quarters(blk.w[j]);
    }
#pragma unroll
    for (int f = 0; f < kFlushes; ++f) {
      f32x4 sum[MT], part[MT][NT];
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        sum[i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < NT; ++j) part[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
      }
#pragma unroll
      for (int t = f * (F / 32); t < (f + 1) * (F / 32); ++t) {
#pragma unroll
        for (int i = 0; i < MT; ++i) sum[i] = Mma<T>::mfma(blk.a[i][t], ones, sum[i]);
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const u32x4 q = expand<T>(blk.w[j][t]);
#pragma unroll
          for (int i = 0; i < MT; ++i) part[i][j] = Mma<T>::mfma(blk.a[i][t], q, part[i][j]);
        }
      }
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const float s = Mma<T>::to_float(blk.s[j][f]);
        const float z = ZEROS ? (float)blk.z[j][f] : 8.f;
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][j][e] += s * (part[i][j][e] - z * sum[i][e]);
      }
    }
  };
  // A block's loads go out before the block ahead of it is used.
  const int full = p.K >> 7;
  int b = wave;
  if (b < full) {
    Blk x, y;
    load(x, b << 7);
    for (;;) {
      b += WAVES;
      if (b < full) load(y, b << 7);
      compute(x);
      if (b >= full) break;
      b += WAVES;
      if (b < full) load(x, b << 7);
      compute(y);
      if (b >= full) break;
    }
  }
  if ((p.K & 127) != 0 && wave == full % WAVES) {
    Blk x;
    load_tail(x, full << 7);
    compute(x);
  }
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) red[wave][i * NT + j][lane] = acc[i][j];
  __syncthreads();
  // An output value is element e of lane (16 (m / 4 % 4) + n % 16) of its tile,
  // e = m % 4. A thread adds up one pair of neighbouring columns of one row.
  constexpr int kPairs = kTiles * 128;
  uint32_t* C = reinterpret_cast<uint32_t*>(p.C);
  for (int u = (int)threadIdx.x; u < kPairs; u += 64 * WAVES) {
    const int pair = u & 7, tile = (u >> 3) % NT, r = (u >> 3) / NT;   // row of the workgroup's rows
    const int m = m0 + r, n = n0 + 16 * tile + 2 * pair;
    if (m >= p.M || n >= p.N) continue;
    const int src = ((r >> 2) & 3) * 16 + 2 * pair, e = r & 3, at = (r >> 4) * NT + tile;
    float lo = 0.f, hi = 0.f;
#pragma unroll
    for (int v = 0; v < WAVES; ++v) {
      lo += reinterpret_cast<const float*>(&red[v][at][src])[e];
      hi += reinterpret_cast<const float*>(&red[v][at][src + 1])[e];
    }
    C[((int64_t)m * p.ldc + n) >> 1] = Mma<T>::pack(lo, hi);
  }
}

template <class T, int MT, int NT, int WAVES, int F>
hipError_t launch_w4_shape(const W4Params& p, hipStream_t stream) {
  const dim3 grid = long_grid(((int64_t)p.N + 16 * NT - 1) / (16 * NT) *
                              (((int64_t)p.M + 16 * MT - 1) / (16 * MT)));
  void (*k)(W4Params) = p.zeros != nullptr ? gemm_w4_kernel<T, MT, NT, WAVES, F, true>
                                           : gemm_w4_kernel<T, MT, NT, WAVES, F, false>;
  hipLaunchKernelGGL(k, grid, dim3(64 * WAVES), 0, stream, p);
  return hipGetLastError();
}

template <class T, int MT, int NT, int WAVES>
hipError_t launch_w4_group(const W4Params& p, hipStream_t stream) {
  if (p.group_shift == 5) return launch_w4_shape<T, MT, NT, WAVES, 32>(p, stream);
  if (p.group_shift == 6) return launch_w4_shape<T, MT, NT, WAVES, 64>(p, stream);
  return launch_w4_shape<T, MT, NT, WAVES, 128>(p, stream);
}

template <class T>
hipError_t launch_w4_type(const W4Params& p, hipStream_t stream) {
  if (p.M <= 16) return launch_w4_group<T, 1, 1, 8>(p, stream);
  if (p.M <= 32) return launch_w4_group<T, 2, 2, 8>(p, stream);
  return launch_w4_group<T, 4, 2, 8>(p, stream);
}

}  // namespace

hipError_t launch_gemm_w4(const W4Params& p, int type, hipStream_t stream) {
  return type == 0 ? launch_w4_type<__bf16>(p, stream) : launch_w4_type<_Float16>(p, stream);
}

}  // namespace pipe
