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
  static __device__ __forceinline__ float dot2(uint32_t a, uint32_t b, float c) {
    return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, a),
                                           __builtin_bit_cast(bf16x2, b), c, false);
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
  static __device__ __forceinline__ float dot2(uint32_t a, uint32_t b, float c) {
    return __builtin_amdgcn_fdot2(__builtin_bit_cast(f16x2, a), __builtin_bit_cast(f16x2, b), c,
                                  false);
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

// MT, NT: 16-row tiles of A and of the weights that a wave holds. WAVES split
// K into runs of blocks of 128. F: k's between two scalings, the group size or
// 128 if that is larger. Rows of A and of the weights past the end are read
// from the last row and dropped.
//
// K is taken in chunks of at most kChunkGroups groups, whose scales and zero
// points the workgroup first turns into pairs of floats in LDS: a 2-byte and a
// 1-byte load in every block cost more than the block's codes.
//
// Loads run ahead of their use without a second set of registers: the codes of
// a block are followed at once by those of the block four further on. Loads
// return in order, so a fragment of A has to be asked for as far ahead or it
// would wait for younger codes: also four blocks with one row tile, where
// registers allow it; with more tiles A's loads are the longer part, and each
// fragment is followed by the next block's.
constexpr int kChunkGroups = 128;

template <class T, int MT, int NT, int WAVES, int F, bool ZEROS>
__global__ void __launch_bounds__(64 * WAVES) gemm_w4_kernel(W4Params p) {
  constexpr int kFlushes = 128 / F;   // scalings in a block
  constexpr int kTiles = MT * NT, kRows = 16 * NT;
  constexpr int kAhead = MT == 1 ? 4 : 1;
  constexpr int kPitch = kChunkGroups + 1;
  __shared__ union {
    f32x4 red[WAVES][kTiles][64];
    f32x2 groups[kRows][kPitch];      // scale, zero point
  } lds;
  const int lane = (int)(threadIdx.x & 63);
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int li = lane & 15, lq = lane >> 4;
  // Workgroups that share weight rows are neighbours.
  const int m_tiles = (p.M + 16 * MT - 1) / (16 * MT);
  const int64_t wg = long_block();
  if (wg >= (int64_t)m_tiles * ((p.N + kRows - 1) / kRows)) return;
  const int n0 = (int)(wg / m_tiles) * kRows, m0 = (int)(wg % m_tiles) * (16 * MT);

  const uint8_t* code_row[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j)
    code_row[j] = p.codes + (int64_t)min(n0 + 16 * j + li, p.N - 1) * p.ld_codes + 16 * lq;
  const uint8_t* a_row[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) a_row[i] = p.A + (int64_t)min(m0 + 16 * i + li, p.M - 1) * p.lda;
  f32x4 acc[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  const u32x4 ones = {Mma<T>::kOnes, Mma<T>::kOnes, Mma<T>::kOnes, Mma<T>::kOnes};

  u32x4 w[4][NT], a[kAhead][4][MT];
  const auto load_codes = [&](int i, int b) {
#pragma unroll
    for (int j = 0; j < NT; ++j)
      w[i][j] = __builtin_nontemporal_load(
          reinterpret_cast<const u32x4*>(code_row[j] + ((int64_t)b << 6)));
  };
  // A's k's of MFMA step t in this lane.
  const auto a_k = [&](int t) { return F < 128 ? 32 * t + 8 * lq : 32 * lq + 8 * t; };
  const auto load_a = [&](int i, int t, int b) {
#pragma unroll
    for (int m = 0; m < MT; ++m)
      a[i][t][m] = *reinterpret_cast<const u32x4*>(a_row[m] + 2 * (((int64_t)b << 7) + a_k(t)));
  };
  // One block: its codes, its A fragments (`next` follows the use of step t),
  // its groups from `at` on in the chunk.
  const auto compute = [&](u32x4(&wb)[NT], u32x4(&ab)[4][MT], int at, auto next) {
    if constexpr (F < 128) {
#pragma unroll
      for (int j = 0; j < NT; ++j) wb[j] = transpose_quarters(wb[j]);
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
        u32x4 av[MT];
#pragma unroll
        for (int i = 0; i < MT; ++i) av[i] = even_odd(ab[t][i]);
        next(t);
#pragma unroll
        for (int i = 0; i < MT; ++i) sum[i] = Mma<T>::mfma(av[i], ones, sum[i]);
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const u32x4 q = expand<T>(wb[j][t]);
#pragma unroll
          for (int i = 0; i < MT; ++i) part[i][j] = Mma<T>::mfma(av[i], q, part[i][j]);
        }
      }
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const f32x2 g = lds.groups[16 * j + li][at + f];
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][j][e] += g[0] * (part[i][j][e] - g[1] * sum[i][e]);
      }
    }
  };

  // Chunks: equal numbers of blocks (groups of more than 128 are counted as
  // blocks here: each block finds its own copy of the group's pair).
  const int full = p.K >> 7, blocks = (p.K + 127) >> 7;   // whole blocks; all
  constexpr int kMost = kChunkGroups / kFlushes;
  const int chunks = (blocks + kMost - 1) / kMost, chunk = (blocks + chunks - 1) / chunks;
  for (int c0 = 0; c0 < blocks; c0 += chunk) {
    const int c1 = min(c0 + chunk, blocks);
    const int each = (min(c1, full) - c0 + WAVES - 1) / WAVES;
    int b = c0 + wave * each;
    const int end = min(b + each, min(c1, full));
    const bool work = b < end;

    // This thread's part of the scales: wave r takes rows r, r + WAVES, ...,
    // its lanes the pairs of a row.
    const int pairs = (c1 - c0) * kFlushes;
    uint16_t sv[2][kRows / WAVES];
    uint8_t zv[2][kRows / WAVES];
    static_assert(kRows % WAVES == 0 && kChunkGroups == 128, "two pairs a lane and row");
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int g = min(((c0 << 7) + (lane + 64 * h) * F), p.K - 1) >> p.group_shift;
#pragma unroll
      for (int r = 0; r < kRows / WAVES; ++r) {
        const int64_t n = min(n0 + wave + r * WAVES, p.N - 1);
        sv[h][r] = p.scales[n * p.ld_scales + g];
        if constexpr (ZEROS) zv[h][r] = p.zeros[n * p.ld_zeros + g];
      }
    }
    if (work) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        load_codes(i, min(b + i, end - 1));
        if (i < kAhead)
#pragma unroll
          for (int t = 0; t < 4; ++t) load_a(i, t, min(b + i, end - 1));
      }
    }
    if (c0 > 0) __syncthreads();   // the last chunk's pairs are no longer read
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int r = 0; r < kRows / WAVES; ++r)
        if (lane + 64 * h < pairs) {
          // Past K: zeros, which the tail's products are multiplied by.
          const bool in = (c0 << 7) + (lane + 64 * h) * F < p.K;
          const float s = in ? Mma<T>::to_float(sv[h][r]) : 0.f;
          lds.groups[wave + r * WAVES][lane + 64 * h] = f32x2{s, ZEROS ? (float)zv[h][r] : 8.f};
        }
    __syncthreads();

    if (work) {
      for (; b + 4 < end; b += 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int far = min(b + i + 4, end - 1);
          if constexpr (kAhead == 4)
            compute(w[i], a[i], (b + i - c0) * kFlushes, [&](int t) { load_a(i, t, far); });
          else
            compute(w[i], a[0], (b + i - c0) * kFlushes, [&](int t) { load_a(0, t, b + i + 1); });
          load_codes(i, far);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (b + i < end) {
          if constexpr (kAhead == 4)
            compute(w[i], a[i], (b + i - c0) * kFlushes, [](int) {});
          else
            compute(w[i], a[0], (b + i - c0) * kFlushes,
                    [&](int t) { load_a(0, t, min(b + i + 1, end - 1)); });
        }
      }
    }
    if (c1 > full && wave == WAVES - 1) {
      // The last block of a K that is no multiple of 128: addresses stay in the
      // row, and A and the scales are zeros past K.
      const int k0 = full << 7;
      const u32x4 zero4 = {0, 0, 0, 0};
      const int back = k0 + 32 * lq < p.K ? 0 : 16 * lq;
#pragma unroll
      for (int j = 0; j < NT; ++j)
        w[0][j] = *reinterpret_cast<const u32x4*>(code_row[j] + (k0 >> 1) - back);
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          const int k = k0 + a_k(t);
          const u32x4 v = *reinterpret_cast<const u32x4*>(a_row[i] + 2 * (int64_t)min(k, p.K - 8));
          a[0][t][i] = k < p.K ? v : zero4;
        }
      compute(w[0], a[0], (full - c0) * kFlushes, [](int) {});
    }
  }
  __syncthreads();   // the pairs' place is the sums' now
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) lds.red[wave][i * NT + j][lane] = acc[i][j];
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
      lo += reinterpret_cast<const float*>(&lds.red[v][at][src])[e];
      hi += reinterpret_cast<const float*>(&lds.red[v][at][src + 1])[e];
    }
    C[((int64_t)m * p.ldc + n) >> 1] = Mma<T>::pack(lo, hi);
  }
}

// ---------------------------------------------------------------------------
// One to four rows of A. A lane keeps the values of 32 k's of every row in
// registers (LPR lanes make up a row of weights, a wave's slice of K) and meets
// them with the codes of kVecRows weight rows, one 16-byte load each: a wave
// reads 1 KiB of a row at a time, and all loads of its rows are in flight
// together. A lane's 32 k's lie in one group, whatever its size, so the scale
// and the zero point are applied to the lane's own sum. v_dot2 adds up two
// products at a time in fp32.
// ---------------------------------------------------------------------------
constexpr int kVecRows = 8;
constexpr int kVecWaves = 8;    // at most, each with slices of K of its own
constexpr int kVecSlice = 2048;

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

template <class T, int MM, int LPR, bool ZEROS>
__global__ void __launch_bounds__(64 * kVecWaves) gemv_w4_kernel(W4Params p) {
  constexpr int kRowsPer = 64 / LPR;   // weight rows a load
  __shared__ float red[kVecWaves][MM][kVecRows * kRowsPer];
  const int lane = (int)(threadIdx.x & 63);
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int waves = (int)(blockDim.x >> 6);
  const int64_t wg = long_block();
  const int64_t row0 = wg * (kVecRows * kRowsPer);
  if (row0 >= p.N) return;
  float acc[MM][kVecRows];
#pragma unroll
  for (int m = 0; m < MM; ++m)
#pragma unroll
    for (int r = 0; r < kVecRows; ++r) acc[m][r] = 0.f;
  const int slices = LPR < 64 ? 1 : (p.K + kVecSlice - 1) / kVecSlice;
  for (int slice = wave; slice < slices; slice += waves) {
    const int k = slice * kVecSlice + (lane % LPR) * 32;
    const bool in = k < p.K;
    const int kk = in ? k : 0;      // lanes past K: values of the row's start times zeros
    u32x4 a[MM][4];
#pragma unroll
    for (int m = 0; m < MM; ++m)
#pragma unroll
      for (int t = 0; t < 4; ++t)
        a[m][t] = *reinterpret_cast<const u32x4*>(p.A + min(m, p.M - 1) * p.lda +
                                                  2 * (int64_t)kk + 16 * t);
    u32x4 w[kVecRows];
    uint16_t s[kVecRows];
    uint8_t z[kVecRows];
    const int g = kk >> p.group_shift;
#pragma unroll
    for (int r = 0; r < kVecRows; ++r) {
      int64_t n = row0 + r * kRowsPer;
      if constexpr (LPR < 64) n += lane / LPR;
      if (n > p.N - 1) n = p.N - 1;
      w[r] = __builtin_nontemporal_load(
          reinterpret_cast<const u32x4*>(p.codes + n * p.ld_codes + (kk >> 1)));
      s[r] = p.scales[n * p.ld_scales + g];
      if constexpr (ZEROS) z[r] = p.zeros[n * p.ld_zeros + g];
    }
    const u32x4 zero4 = {0, 0, 0, 0};
    float total[MM];                 // of the lane's A values
#pragma unroll
    for (int m = 0; m < MM; ++m) {
      total[m] = 0.f;
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        a[m][t] = in ? even_odd(a[m][t]) : zero4;
#pragma unroll
        for (int e = 0; e < 4; ++e) total[m] = Mma<T>::dot2(a[m][t][e], Mma<T>::kOnes, total[m]);
      }
    }
#pragma unroll
    for (int r = 0; r < kVecRows; ++r) {
      float part[MM];
#pragma unroll
      for (int m = 0; m < MM; ++m) part[m] = 0.f;
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const u32x4 q = expand<T>(w[r][t]);
#pragma unroll
        for (int m = 0; m < MM; ++m)
#pragma unroll
          for (int e = 0; e < 4; ++e) part[m] = Mma<T>::dot2(a[m][t][e], q[e], part[m]);
      }
      const float sc = in ? Mma<T>::to_float(s[r]) : 0.f;
      const float zp = ZEROS ? (float)z[r] : 8.f;
#pragma unroll
      for (int m = 0; m < MM; ++m) acc[m][r] += sc * (part[m] - zp * total[m]);
    }
  }
#pragma unroll
  for (int m = 0; m < MM; ++m) {
    if constexpr (LPR == 64) {
      float out[2];
      sum_rows(acc[m], out);
      if ((lane & 15) == 0) {
        const int part = (lane >> 4), at = ((part & 1) << 1) | (part >> 1);
        red[wave][m][at] = out[0];
        red[wave][m][4 + at] = out[1];
      }
    } else {
#pragma unroll
      for (int r = 0; r < kVecRows; ++r) {
        float v = acc[m][r];
#pragma unroll
        for (int off = LPR / 2; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
        if (lane % LPR == 0) red[wave][m][r * kRowsPer + lane / LPR] = v;
      }
    }
  }
  __syncthreads();
  constexpr int kPairs = MM * kVecRows * kRowsPer / 2;
  uint32_t* C = reinterpret_cast<uint32_t*>(p.C);
  for (int u = (int)threadIdx.x; u < kPairs; u += (int)blockDim.x) {
    const int m = u / (kPairs / MM), r = u % (kPairs / MM) * 2;
    const int64_t n = row0 + r;
    if (m >= p.M || n >= p.N) continue;
    float lo = 0.f, hi = 0.f;
    for (int v = 0; v < waves; ++v) {
      lo += red[v][m][r];
      hi += red[v][m][r + 1];
    }
    C[(m * p.ldc + n) >> 1] = Mma<T>::pack(lo, hi);
  }
}

template <class T, int MM, int LPR>
hipError_t launch_w4_vec(const W4Params& p, hipStream_t stream) {
  constexpr int kRows = kVecRows * (64 / LPR);
  const int slices = LPR < 64 ? 1 : (p.K + kVecSlice - 1) / kVecSlice;
  const int turns = (slices + kVecWaves - 1) / kVecWaves;
  const int waves = (slices + turns - 1) / turns;
  void (*k)(W4Params) = p.zeros != nullptr ? gemv_w4_kernel<T, MM, LPR, true>
                                           : gemv_w4_kernel<T, MM, LPR, false>;
  hipLaunchKernelGGL(k, long_grid(((int64_t)p.N + kRows - 1) / kRows), dim3(64 * waves), 0, stream, p);
  return hipGetLastError();
}

// A row of weights takes 32 k's a lane: as many lanes as K has, up to a wave.
template <class T, int MM>
hipError_t launch_w4_vec_k(const W4Params& p, hipStream_t stream) {
  if (p.K <= 8 * 32) return launch_w4_vec<T, MM, 8>(p, stream);
  if (p.K <= 16 * 32) return launch_w4_vec<T, MM, 16>(p, stream);
  if (p.K <= 32 * 32) return launch_w4_vec<T, MM, 32>(p, stream);
  return launch_w4_vec<T, MM, 64>(p, stream);
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
  if (p.M == 1) return launch_w4_vec_k<T, 1>(p, stream);
  if (p.M == 2) return launch_w4_vec_k<T, 2>(p, stream);
  if (p.M <= 4) return launch_w4_vec_k<T, 4>(p, stream);
  if (p.M <= 16) return launch_w4_group<T, 1, 2, 8>(p, stream);
  if (p.M <= 32) return launch_w4_group<T, 2, 2, 8>(p, stream);
  if (p.M <= 48) return launch_w4_group<T, 3, 2, 8>(p, stream);
  return launch_w4_group<T, 4, 2, 8>(p, stream);
}

}  // namespace

hipError_t launch_gemm_w4(const W4Params& p, int type, hipStream_t stream) {
  return type == 0 ? launch_w4_type<__bf16>(p, stream) : launch_w4_type<_Float16>(p, stream);
}

}  // namespace pipe
