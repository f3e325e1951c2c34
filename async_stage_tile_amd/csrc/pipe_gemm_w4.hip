// Products of 16-bit rows with 4-bit weights: C = A ((q - z) s)^T, a scale and
// a zero point for each group of K.
//
// For a few rows the call is bound by reading the weights once: N K / 2 bytes
// of codes, for a few operations each. One row of A, or two, meets them on the
// vector units (gemv_w4_kernel), up to eight on the small MFMAs
// (gemm_w4_quad_kernel), more rows or weights on the large ones
// (gemm_w4_tile_kernel).
//
// Integers: a byte 0..15 is, read as e4m3, q * 2^-9 (the subnormals and the
// first binade are evenly spaced), so one v_cvt_scalef32_pk with scale 2^9
// turns two of them into 16-bit floats exactly: 7 operations for 8 codes,
// shift and masks included.
//
// Scales and zero points: over one group (q - z) s = s q - s z, so with
// P = sum_k a q and S = sum_k a of the group, acc += s (P - z S). On the MFMAs S
// is one more product, against ones. Everything is exact or fp32; no weight is
// rounded to 16 bits. P and z S may be larger than their difference, and their
// fp32 errors with them: on loud channels, activations of one sign and sums that
// cancel they stay within sqrt(K) 2^-24 of the two sums.
#include "pipe_device.hpp"
#include "pipe_linear.hpp"

namespace pipe {

namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));

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
  static __device__ __forceinline__ f32x4 mfma4(uint32_t a0, uint32_t a1, uint32_t b0, uint32_t b1,
                                                f32x4 c) {
    return __builtin_amdgcn_mfma_f32_4x4x4bf16_1k(__builtin_bit_cast(s16x4, u32x2{a0, a1}),
                                                  __builtin_bit_cast(s16x4, u32x2{b0, b1}), c, 0, 0, 0);
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
  static __device__ __forceinline__ f32x4 mfma4(uint32_t a0, uint32_t a1, uint32_t b0, uint32_t b1,
                                                f32x4 c) {
    return __builtin_amdgcn_mfma_f32_4x4x4f16(__builtin_bit_cast(f16x4, u32x2{a0, a1}),
                                              __builtin_bit_cast(f16x4, u32x2{b0, b1}), c, 0, 0, 0);
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

// The value of the lane N places on among its 16, around.
template <int N>
__device__ __forceinline__ float rotate16(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v),
                                                               0x120 + N, 0xf, 0xf, false));
}

// A's 8 values in the order of expand().
__device__ __forceinline__ u32x4 even_odd(u32x4 a) {
  return u32x4{__builtin_amdgcn_perm(a[1], a[0], 0x05040100u),
               __builtin_amdgcn_perm(a[3], a[2], 0x05040100u),
               __builtin_amdgcn_perm(a[1], a[0], 0x07060302u),
               __builtin_amdgcn_perm(a[3], a[2], 0x07060302u)};
}

// 8 codes as 16-bit floats in their own order.
template <class T>
__device__ __forceinline__ u32x4 expand_in_order(uint32_t codes) {
  const uint32_t even = codes & 0x0F0F0F0Fu, odd = (codes >> 4) & 0x0F0F0F0Fu;
  const uint32_t lo = __builtin_amdgcn_perm(odd, even, 0x05010400u);   // k0 k1 k2 k3
  const uint32_t hi = __builtin_amdgcn_perm(odd, even, 0x07030602u);   // k4 k5 k6 k7
  return u32x4{Mma<T>::codes_lo(lo), Mma<T>::codes_hi(lo), Mma<T>::codes_lo(hi),
               Mma<T>::codes_hi(hi)};
}

// ---------------------------------------------------------------------------
// More rows of A. A workgroup computes 16 MT rows of A times TN weight
// rows; stages of 256 k pass through an LDS ring, filled by direct-to-LDS loads
// alone, so that one wait count covers a stage: codes (TN rows of 128 bytes,
// 16-byte chunk c of row r at place c ^ ((r >> 1) & 7)) and A (rows of 512
// bytes, chunk c of row r at c ^ (r & 15)). The scales and zero points of as
// many stages as there is room for are copied to a table in LDS between stages,
// a row's groups at a time: fetched stage by stage, they cost a cache line a row
// for each few bytes, more requests than the codes themselves. Wave (wn, kh)
// takes weight rows 32 wn .. + 31 and part kh of the stage's k's; with the codes
// of 8 k's in one LDS word, an MFMA step of 32 k's reads its operand as it lies:
// quarter q of the lanes holds k = 8 q .. 8 q + 7. The parts' sums meet in LDS at
// the end.
//
// One barrier a stage: at its top a wave's own loads of the stage have landed
// and its reads of the stage before have returned. After the barrier that
// holds for every wave, and the slot of the stage before takes the next one
// that is not under way.
//
// Where the tiles leave compute units idle K is split over workgroups, which
// then write fp32 partial products for gemm_w4_join_kernel to add up in order.
// Rows past M and N are read from the last row and dropped; of the last stage
// only the MFMA steps and groups inside K are used, and loads past K take the
// stage's first chunk or the last group instead.
//
// Bound by turning codes into MFMA operands and by the MFMAs, S's among them,
// on the way through each stage: 16 rows against 28672 x 8192 take 36 us (the
// codes alone would take 19). 47 against 6000 x 4096 take 15.6, of which 12 are
// left without any of that: two launches, the ring's start, the join.
// ---------------------------------------------------------------------------
template <bool B>
struct W4Flag {
  static constexpr bool value = B;
};

constexpr int kW4StageK = 256, kW4Waves = 8;

template <int MT, int F, int TN>
struct W4Tile {
  static constexpr int kAcross = TN / 32;                  // waves along N, and along K:
  static constexpr int kParts = kW4Waves / kAcross;
  static constexpr int kSpan = kW4StageK / kParts;         // k's of a part
  static constexpr int kSum = F < kSpan ? F : kSpan;       // k's between two scalings
  static constexpr int kGroups = kW4StageK / F;            // groups of a stage
  static constexpr int kCodes = TN * kW4StageK / 2;  // bytes of a slot's parts
  static constexpr int kA = 16 * MT * kW4StageK * 2;
  static constexpr int kSlot = kCodes + kA;
  static constexpr int kPitch = TN + 4;              // floats of a row of sums
  static constexpr int kLds = 163840;
  static constexpr int kFit = (kLds - 8192) / kSlot;
  static constexpr int kSlots = kFit > 5 ? 5 : kFit;
  static constexpr int kTable = kLds - kSlots * kSlot;     // scales (2 bytes), zero points (1)
  static constexpr int kRoom = kTable / (3 * TN * kGroups);
  static constexpr int kChunk = kRoom < 32 ? kRoom : 32;   // stages of a table
  static constexpr int kChunkGroups = kChunk * kGroups;
  static constexpr int kCodeLoads = TN / 8 / kW4Waves, kALoads = MT;
  static constexpr int kLoads = kCodeLoads + kALoads;      // a wave and stage
  static_assert(kSlots >= 3 && kChunk >= 1 && 16 * MT * kPitch * 4 <= kSlots * kSlot, "LDS");
};

template <class T, int MT, int F, int TN, bool ZEROS>
__global__ void __launch_bounds__(64 * kW4Waves) gemm_w4_tile_kernel(W4Params p) {
  using Tile = W4Tile<MT, F, TN>;
  constexpr int kSteps = Tile::kSpan / 32, kSums = Tile::kSpan / Tile::kSum;
  __shared__ __align__(1024) uint8_t lds[Tile::kLds];
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int lane = lane_id();
  const int li = lane & 15, lq = lane >> 4;
  const int wn = wave % Tile::kAcross, kh = wave / Tile::kAcross;
  const uint32_t base = uniform(lds_addr(&lds[0]));
  const int64_t wg = long_block();
  // Neighbours share weight rows, then lie along N. Their number is below 2^31:
  // the host checks the tiles', and K is split for fewer than 256 tiles only.
  const int m_tiles = (p.M - 1) / (16 * MT) + 1, n_tiles = (p.N + TN - 1) / TN;
  if (wg >= (int64_t)m_tiles * n_tiles * p.splits) return;
  const int split = p.splits == 1 ? 0 : (int)wg / (m_tiles * n_tiles);
  const int tile = (int)wg - split * (m_tiles * n_tiles);
  const int along = m_tiles == 1 ? tile : tile / m_tiles;
  const int m0 = (tile - along * m_tiles) * (16 * MT), n0 = along * TN;
  const int stages = (p.K + kW4StageK - 1) / kW4StageK;
  const int per = (stages + p.splits - 1) / p.splits;
  const int first = split * per, count = min(per, stages - first);   // >= 1

  // This wave's loads of a stage.
  const uint8_t* code_src[Tile::kCodeLoads];
  int code_k[Tile::kCodeLoads];
#pragma unroll
  for (int j = 0; j < Tile::kCodeLoads; ++j) {
    const int r = (wave * Tile::kCodeLoads + j) * 8 + (lane >> 3);
    const int c = (lane & 7) ^ ((r >> 1) & 7);
    code_src[j] = p.codes + (int64_t)min(n0 + r, p.N - 1) * p.ld_codes;
    code_k[j] = 32 * c;
  }
  const uint8_t* a_src[Tile::kALoads];
  int a_k[Tile::kALoads];
#pragma unroll
  for (int j = 0; j < Tile::kALoads; ++j) {
    const int r = (wave * Tile::kALoads + j) * 2 + (lane >> 5);
    a_src[j] = p.A + (int64_t)min(m0 + r, p.M - 1) * p.lda;
    a_k[j] = 8 * ((lane & 31) ^ (r & 15));
  }
  auto load = [&](int ks, int slot) {
    const int k0 = (first + min(ks, count - 1)) * kW4StageK;
    const uint32_t to = base + slot * Tile::kSlot;
#pragma unroll
    for (int j = 0; j < Tile::kCodeLoads; ++j) {
      const int k = k0 + (k0 + code_k[j] < p.K ? code_k[j] : 0);
      dma_block_nt(code_src[j] + (k >> 1), to + (wave * Tile::kCodeLoads + j) * kBlockBytes);
    }
#pragma unroll
    for (int j = 0; j < Tile::kALoads; ++j) {
      const int k = k0 + (k0 + a_k[j] < p.K ? a_k[j] : 0);
      dma_block(a_src[j] + 2 * (int64_t)k, to + Tile::kCodes + (wave * Tile::kALoads + j) * kBlockBytes);
    }
  };
  // The table of the stages from ks on: this wave takes an eighth of the rows,
  // 4 at a time, 16 groups of each. Group g of the table's n-th row lies at [g][n].
  uint16_t* table_s = reinterpret_cast<uint16_t*>(&lds[Tile::kSlots * Tile::kSlot]);
  uint8_t* table_z = reinterpret_cast<uint8_t*>(table_s + Tile::kChunkGroups * TN);
  constexpr int kRounds = (Tile::kChunkGroups + 15) / 16;
  auto fill_table = [&](int ks) {
    const int g_end = min(Tile::kChunk, count - ks) * Tile::kGroups;
    for (int h = 0; h < kRounds && 16 * h < g_end; ++h) {
      const int g = 16 * h + li;
      const int at = min((first + ks) * kW4StageK + g * F, p.K - 1) >> p.group_shift;
      constexpr int kQuads = TN / 4 / kW4Waves;
      uint16_t sv[kQuads];
      uint8_t zv[kQuads];
#pragma unroll
      for (int r = 0; r < kQuads; ++r) {
        const int64_t n = min(n0 + 4 * (kQuads * wave + r) + lq, p.N - 1);
        sv[r] = p.scales[n * p.ld_scales + at];
        if constexpr (ZEROS) zv[r] = p.zeros[n * p.ld_zeros + at];
      }
#pragma unroll
      for (int r = 0; r < kQuads; ++r)
        if (g < g_end) {
          const int to = g * TN + 4 * (kQuads * wave + r) + lq;
          table_s[to] = sv[r];
          if constexpr (ZEROS) table_z[to] = zv[r];
        }
    }
  };

  f32x4 acc[MT][2];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  const u32x4 ones = {Mma<T>::kOnes, Mma<T>::kOnes, Mma<T>::kOnes, Mma<T>::kOnes};

  // This wave's part of a slot, of which `left` k's are inside K.
  auto compute = [&](int slot, int table, auto CUT, int left) {   // table: the stage's first group there
    constexpr bool cut = decltype(CUT)::value;
    const uint8_t* codes = &lds[slot * Tile::kSlot] + (32 * wn + li) * 128 + 4 * lq;
    const uint8_t* rows = &lds[slot * Tile::kSlot + Tile::kCodes] + li * 512;
    // All LDS reads of the part go out first: left to the compiler they
    // come one MFMA step at a time, each with its own wait.
    u32x4 a[kSteps][MT];
    uint32_t word[kSteps][2];
    float scale[kSums][2], zero[kSums][2];
#pragma unroll
    for (int t = 0; t < kSteps; ++t) {
#pragma unroll
      for (int j = 0; j < 2; ++j)   // row 16 j + li of the wave's: (r >> 1) & 7 is (li >> 1) & 7
        word[t][j] = *reinterpret_cast<const uint32_t*>(
            codes + j * 16 * 128 + ((kSteps * kh + t) ^ ((li >> 1) & 7)) * 16);
#pragma unroll
      for (int i = 0; i < MT; ++i)
        a[t][i] = *reinterpret_cast<const u32x4*>(rows + i * 16 * 512 +
                                                  ((4 * (kSteps * kh + t) + lq) ^ li) * 16);
    }
#pragma unroll
    for (int f = 0; f < kSums; ++f)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int at = (table + (kh * Tile::kSpan + f * Tile::kSum) / F) * TN + 32 * wn + 16 * j + li;
        scale[f][j] = Mma<T>::to_float(table_s[at]);
        zero[f][j] = ZEROS ? (float)table_z[at] : 8.f;
      }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int f = 0; f < kSums; ++f) {
      if (cut && f * Tile::kSum >= left) break;
      f32x4 sum[MT], part[MT][2];
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        sum[i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < 2; ++j) part[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
      }
#pragma unroll
      for (int t = f * (Tile::kSum / 32); t < (f + 1) * (Tile::kSum / 32); ++t) {
        if (cut && 32 * t >= left) break;
#pragma unroll
        for (int i = 0; i < MT; ++i) sum[i] = Mma<T>::mfma(a[t][i], ones, sum[i]);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const u32x4 q = expand_in_order<T>(word[t][j]);
#pragma unroll
          for (int i = 0; i < MT; ++i) part[i][j] = Mma<T>::mfma(a[t][i], q, part[i][j]);
        }
      }
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            acc[i][j][e] += scale[f][j] * (part[i][j][e] - zero[f][j] * sum[i][e]);
    }
  };

  for (int i = 0; i < Tile::kSlots - 1; ++i) load(i, i);
  fill_table(0);   // seen by the other waves after the first stage's barrier
  int slot = 0, turn = 0;   // the stage's slot, and its place in the table
  auto begin = [&](int ks) {
    wait_vmcnt<(Tile::kSlots - 2) * Tile::kLoads>();   // those of younger stages
    wait_lgkmcnt0();
    __syncthreads();
    if (turn == Tile::kChunk) {
      turn = 0;
      fill_table(ks);
      __syncthreads();
    }
    load(ks + Tile::kSlots - 1, slot == 0 ? Tile::kSlots - 1 : slot - 1);
  };
  auto end = [&]() {
    slot = slot + 1 == Tile::kSlots ? 0 : slot + 1;
    ++turn;
  };
  // Whole stages, then what K leaves of the last one (apart: with both in one
  // loop the accumulators are copied to and fro between the two).
  const int whole = (first + count) * kW4StageK <= p.K ? count : count - 1;
  for (int ks = 0; ks < whole; ++ks) {
    begin(ks);
    compute(slot, turn * Tile::kGroups, W4Flag<false>{}, Tile::kSpan);
    end();
  }
  if (whole < count) {
    begin(whole);
    const int left = p.K - (first + whole) * kW4StageK - Tile::kSpan * kh;
    if (left > 0) compute(slot, turn * Tile::kGroups, W4Flag<true>{}, left);
  }
  // The ring's last loads have landed and its last reads returned: its place
  // holds the sums now, a row of A each.
  wait_vmcnt<0>();
  wait_lgkmcnt0();
  __syncthreads();
  float* sums = reinterpret_cast<float*>(&lds[0]);
  auto at = [&](int i, int j, int e) {
    return (16 * i + 4 * lq + e) * Tile::kPitch + 32 * wn + 16 * j + li;
  };
#pragma unroll
  for (int part = Tile::kParts - 1; part >= 0; --part) {
    if (kh == part) {
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            sums[at(i, j, e)] =
                part == Tile::kParts - 1 ? acc[i][j][e] : acc[i][j][e] + sums[at(i, j, e)];
    }
    __syncthreads();
  }
  for (int u = (int)threadIdx.x; u < 16 * MT * (TN / 8); u += 64 * kW4Waves) {
    const int r = u / (TN / 8), c = u % (TN / 8) * 8;
    const int m = m0 + r, n = n0 + c;
    if (m >= p.M || n >= p.N) continue;
    const f32x4 lo = *reinterpret_cast<const f32x4*>(&sums[r * Tile::kPitch + c]);
    const f32x4 hi = *reinterpret_cast<const f32x4*>(&sums[r * Tile::kPitch + c + 4]);
    if (p.splits > 1) {
      f32x4* to = reinterpret_cast<f32x4*>(p.partials + ((int64_t)split * p.M + m) * p.N + n);
      to[0] = lo;
      to[1] = hi;
    } else {
      *reinterpret_cast<u32x4*>(p.C + ((int64_t)m * p.ldc + n) * 2) =
          u32x4{Mma<T>::pack(lo[0], lo[1]), Mma<T>::pack(lo[2], lo[3]),
                Mma<T>::pack(hi[0], hi[1]), Mma<T>::pack(hi[2], hi[3])};
    }
  }
}

// The splits' partial products added up in order: eight columns a thread.
// Bound by a launch and trips to memory, 2 to 4 us, so four splits' loads go out
// together (40 x 512 x 28672, 28 splits, 15.4 us in all; one at a time 21.2).
template <class T>
__global__ void __launch_bounds__(256) gemm_w4_join_kernel(W4Params p) {
  const int octets = p.N >> 3;
  const int64_t i = long_block() * 256 + threadIdx.x;
  if (i >= (int64_t)p.M * octets) return;
  const int64_t m = i / octets, n = i % octets * 8;
  const float* src = p.partials + m * p.N + n;
  f32x4 lo = {0.f, 0.f, 0.f, 0.f}, hi = lo;
#pragma unroll 4
  for (int s = 0; s < p.splits; ++s, src += (int64_t)p.M * p.N) {
    lo += *reinterpret_cast<const f32x4*>(src);
    hi += *reinterpret_cast<const f32x4*>(src + 4);
  }
  *reinterpret_cast<u32x4*>(p.C + (m * p.ldc + n) * 2) =
      u32x4{Mma<T>::pack(lo[0], lo[1]), Mma<T>::pack(lo[2], lo[3]), Mma<T>::pack(hi[0], hi[1]),
            Mma<T>::pack(hi[2], hi[3])};
}

// ---------------------------------------------------------------------------
// One or two rows of A. A lane keeps the values of 32 k's of every row in
// registers (a wave takes a slice of 2048) and meets them with the codes of
// kVecRows weight rows, one 16-byte load each: a wave reads 1 KiB of a row at a
// time, and all loads of its rows are in flight together. 1 x 28672 x 8192 takes 23 us (5.3 TB/s), bound by reading the codes
// and then by turning them into floats (codes masked into the mantissa of a
// large float instead: 27 us). A lane's 32 k's lie in one group, whatever its size, so the scale
// and the zero point are applied to the lane's own sum. v_dot2 adds up two
// products at a time in fp32.
// ---------------------------------------------------------------------------
constexpr int kVecRows = 8;
constexpr int kVecWaves = 8;    // at most, each with slices of K of its own
constexpr int kVecSlice = 2048;

template <class T, int MM, bool ZEROS>
__global__ void __launch_bounds__(64 * kVecWaves) gemv_w4_kernel(W4Params p) {
  __shared__ float red[kVecWaves][MM][kVecRows];
  const int lane = (int)(threadIdx.x & 63);
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int waves = (int)(blockDim.x >> 6);
  const int64_t wg = long_block();
  const int64_t row0 = wg * kVecRows;
  if (row0 >= p.N) return;
  float acc[MM][kVecRows];
#pragma unroll
  for (int m = 0; m < MM; ++m)
#pragma unroll
    for (int r = 0; r < kVecRows; ++r) acc[m][r] = 0.f;
  const int slices = (p.K + kVecSlice - 1) / kVecSlice;
  for (int slice = wave; slice < slices; slice += waves) {
    const int k = slice * kVecSlice + lane * 32;
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
      int64_t n = row0 + r;
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
      const float zp = ZEROS ? (float)z[r] : 8.f;
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
#pragma unroll
      for (int m = 0; m < MM; ++m)
        acc[m][r] += sc * (part[m] - zp * total[m]);
    }
  }
#pragma unroll
  for (int m = 0; m < MM; ++m) {
    float out[2];
    sum_rows(acc[m], out);
    if ((lane & 15) == 0) {
      const int part = (lane >> 4), at = ((part & 1) << 1) | (part >> 1);
      red[wave][m][at] = out[0];
      red[wave][m][4 + at] = out[1];
    }
  }
  __syncthreads();
  constexpr int kPairs = MM * kVecRows / 2;
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

template <class T, int MM>
hipError_t launch_w4_vec(const W4Params& p, hipStream_t stream) {
  const int slices = (p.K + kVecSlice - 1) / kVecSlice;
  const int turns = (slices + kVecWaves - 1) / kVecWaves;
  const int waves = (slices + turns - 1) / turns;
  void (*k)(W4Params) = p.zeros != nullptr ? gemv_w4_kernel<T, MM, true>
                                           : gemv_w4_kernel<T, MM, false>;
  hipLaunchKernelGGL(k, long_grid(((int64_t)p.N + kVecRows - 1) / kVecRows), dim3(64 * waves), 0,
                     stream, p);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// One to eight rows of A against smaller layers. v_mfma_f32_4x4x4 multiplies 16
// blocks apart, four rows by four columns by four k's each: lane 4 b + j holds
// values of A's row j and of weight row j, at the 32 k's of block b, that one
// 16-byte load of codes brings. KB blocks lie along K, 64 / KB weight rows make
// up a load, and a lane's 32 k's lie in one group, so scale and zero point are
// applied to the block's product in the lane, sum_k a times the zero point by one
// more product, against ones. No LDS on the way in, and the vector units only
// expand the codes, where v_dot2 would take 8 cycles for every 128 products too:
// 4 x 4096 x 4096 5.8 us (on v_dot2 7.7), 4 x 3544 x 22464 16.6 (25.2), 1 x 4096
// x 4096 4.7 (4.8).
// Bound by a launch and a trip to memory there, and by the reads, in pieces of
// 256 bytes a row, on larger layers.
// ---------------------------------------------------------------------------
template <class T, int MM, int KB, int LOADS, bool ZEROS>
__global__ void __launch_bounds__(64 * kVecWaves) gemm_w4_quad_kernel(W4Params p) {
  constexpr int kRowsPer = 64 / KB;                  // weight rows a load
  constexpr int kRows = LOADS * kRowsPer;       // of a workgroup
  constexpr int kSlice = 32 * KB;                    // k's of a wave and turn
  constexpr int kFours = (MM + 3) / 4;
  __shared__ float red[kVecWaves][MM][LOADS][16];
  const int lane = (int)(threadIdx.x & 63);
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int waves = (int)(blockDim.x >> 6);
  const int j = lane & 3, block = lane >> 2;
  const int64_t row0 = long_block() * kRows;
  if (row0 >= p.N) return;
  const int row = block / KB * 4 + j;                // of a load's rows
  float acc[LOADS][MM];
#pragma unroll
  for (int r = 0; r < LOADS; ++r)
#pragma unroll
    for (int m = 0; m < MM; ++m) acc[r][m] = 0.f;
  const uint8_t* a_row[kFours];
#pragma unroll
  for (int f = 0; f < kFours; ++f) a_row[f] = p.A + min(4 * f + j, p.M - 1) * p.lda;
  const int slices = (p.K + kSlice - 1) / kSlice;
  for (int slice = wave; slice < slices; slice += waves) {
    const int k = slice * kSlice + block % KB * 32;
    const bool in = k < p.K;
    const int kk = in ? k : 0;        // past K: values of the row's start times zeros
    const int g = kk >> p.group_shift;
    u32x4 a[kFours][4], w[LOADS];
    uint16_t s[LOADS];
    uint8_t z[LOADS];
#pragma unroll
    for (int r = 0; r < LOADS; ++r) {
      int64_t n = row0 + r * kRowsPer + row;
      if (n > p.N - 1) n = p.N - 1;
      w[r] = __builtin_nontemporal_load(
          reinterpret_cast<const u32x4*>(p.codes + n * p.ld_codes + (kk >> 1)));
      s[r] = p.scales[n * p.ld_scales + g];
      if constexpr (ZEROS) z[r] = p.zeros[n * p.ld_zeros + g];
    }
#pragma unroll
    for (int f = 0; f < kFours; ++f)
#pragma unroll
      for (int t = 0; t < 4; ++t)
        a[f][t] = *reinterpret_cast<const u32x4*>(a_row[f] + 2 * (int64_t)kk + 16 * t);
    const f32x4 none = {0.f, 0.f, 0.f, 0.f};
    f32x4 total[kFours];              // sums of the A values
#pragma unroll
    for (int f = 0; f < kFours; ++f) {
      total[f] = none;
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        a[f][t] = in ? even_odd(a[f][t]) : u32x4{0, 0, 0, 0};
        total[f] = Mma<T>::mfma4(a[f][t][0], a[f][t][1], Mma<T>::kOnes, Mma<T>::kOnes, total[f]);
        total[f] = Mma<T>::mfma4(a[f][t][2], a[f][t][3], Mma<T>::kOnes, Mma<T>::kOnes, total[f]);
      }
    }
#pragma unroll
    for (int r = 0; r < LOADS; ++r) {
      f32x4 part[kFours];
#pragma unroll
      for (int f = 0; f < kFours; ++f) part[f] = none;
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const u32x4 q = expand<T>(w[r][t]);
#pragma unroll
        for (int f = 0; f < kFours; ++f) {
          part[f] = Mma<T>::mfma4(a[f][t][0], a[f][t][1], q[0], q[1], part[f]);
          part[f] = Mma<T>::mfma4(a[f][t][2], a[f][t][3], q[2], q[3], part[f]);
        }
      }
      const float zp = ZEROS ? (float)z[r] : 8.f;
      const float sc = in ? Mma<T>::to_float(s[r]) : 0.f;
#pragma unroll
      for (int m = 0; m < MM; ++m) acc[r][m] += sc * (part[m / 4][m % 4] - zp * total[m / 4][m % 4]);
    }
  }
  // The sums of four blocks' lanes are added up here, those of 16-lane rows and
  // waves below.
#pragma unroll
  for (int r = 0; r < LOADS; ++r)
#pragma unroll
    for (int m = 0; m < MM; ++m) {
      float v = acc[r][m];
      v += rotate16<4>(v);
      v += rotate16<8>(v);
      if ((block & 3) == 0) red[wave][m][r][(lane >> 4) * 4 + j] = v;
    }
  __syncthreads();
  constexpr int kPairs = MM * kRows / 2;
  uint32_t* C = reinterpret_cast<uint32_t*>(p.C);
  for (int u = (int)threadIdx.x; u < kPairs; u += (int)blockDim.x) {
    const int m = u / (kPairs / MM), at = u % (kPairs / MM) * 2;
    const int64_t n = row0 + at;
    if (m >= p.M || n >= p.N) continue;
    const int r = at / kRowsPer, i = at % kRowsPer;
    float lo = 0.f, hi = 0.f;
    for (int v = 0; v < waves; ++v)
#pragma unroll
      for (int b = 0; b < KB / 4; ++b) {
        const float* sum = &red[v][m][r][(i / 4 * (KB / 4) + b) * 4 + i % 4];
        lo += sum[0];
        hi += sum[1];
      }
    C[(m * p.ldc + n) >> 1] = Mma<T>::pack(lo, hi);
  }
}

template <class T, int MM, int KB, int LOADS>
hipError_t launch_w4_quad(const W4Params& p, hipStream_t stream) {
  constexpr int kRows = LOADS * (64 / KB);
  const int slices = (p.K + 32 * KB - 1) / (32 * KB);
  const int turns = (slices + kVecWaves - 1) / kVecWaves;
  const int waves = (slices + turns - 1) / turns;
  void (*k)(W4Params) = p.zeros != nullptr ? gemm_w4_quad_kernel<T, MM, KB, LOADS, true>
                                           : gemm_w4_quad_kernel<T, MM, KB, LOADS, false>;
  hipLaunchKernelGGL(k, long_grid(((int64_t)p.N + kRows - 1) / kRows), dim3(64 * waves), 0, stream, p);
  return hipGetLastError();
}

// Blocks along K: up to all 16. Four loads of codes for each of A's where that
// leaves more than 128 workgroups, else two (8 x 1024 x 8192 10.5 us with four,
// 8.5 with two; 8 x 4096 x 4096 7.1 and 8.2).
template <class T, int MM>
hipError_t launch_w4_quad_k(const W4Params& p, hipStream_t stream) {
  if (p.K <= 8 * 32)
    return p.N > 4096 ? launch_w4_quad<T, MM, 8, 4>(p, stream) : launch_w4_quad<T, MM, 8, 2>(p, stream);
  return p.N > 2048 ? launch_w4_quad<T, MM, 16, 4>(p, stream) : launch_w4_quad<T, MM, 16, 2>(p, stream);
}

template <class T, int MT, int F, int TN>
hipError_t launch_w4_tile(const W4Params& p, hipStream_t stream) {
  const int64_t tiles =
      (((int64_t)p.N + TN - 1) / TN) * (((int64_t)p.M + 16 * MT - 1) / (16 * MT));
  void (*k)(W4Params) = p.zeros != nullptr ? gemm_w4_tile_kernel<T, MT, F, TN, true>
                                           : gemm_w4_tile_kernel<T, MT, F, TN, false>;
  hipLaunchKernelGGL(k, long_grid(tiles * p.splits), dim3(64 * kW4Waves), 0, stream, p);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.splits == 1) return e;
  hipLaunchKernelGGL(gemm_w4_join_kernel<T>, long_grid(((int64_t)p.M * (p.N / 8) + 255) / 256),
                     dim3(256), 0, stream, p);
  return hipGetLastError();
}

template <class T, int MT, int TN>
hipError_t launch_w4_group(const W4Params& p, hipStream_t stream) {
  if (p.group_shift == 5) return launch_w4_tile<T, MT, 32, TN>(p, stream);
  if (p.group_shift == 6) return launch_w4_tile<T, MT, 64, TN>(p, stream);
  return launch_w4_tile<T, MT, 128, TN>(p, stream);
}

// 16-row tiles of A that a workgroup of the tile kernel takes.
int w4_m_tiles(int64_t M) { return M <= 16 ? 1 : M <= 32 ? 2 : M <= 48 ? 3 : 4; }

int64_t w4_tiles(int64_t M, int64_t N, int64_t cols) {
  const int64_t rows = 16 * w4_m_tiles(M);
  return (N + cols - 1) / cols * ((M + rows - 1) / rows);
}

// 64 weight rows a tile while the CUs take all tiles at once: fewer splits of K
// (47 x 6000 x 4096 15.6 us, 128 rows 16.9; 8 x 2048 x 11008 11.5 and 14.1). Else
// 128, which read A half as often (64 x 28672 x 8192 60 us, 64 rows 72).
int w4_cols(int64_t M, int64_t N) { return w4_tiles(M, N, 64) <= 256 ? 64 : 128; }

enum W4Kind { kW4Vec, kW4Quad, kW4Tile };

// The vector units take one row of more than 2^24 weights (1 x 28672 x 8192 23 us,
// the small MFMAs 32; 1 x 2048 x 1024 3.9 and 3.3) or of a long K (1 x 1024 x 8192
// 4.1 and 4.9), and two of more than 2^25 (2 x 28672 x 8192 30 and 34; 2 x 4096 x
// 4096 5.7 and 4.9). The small MFMAs take the rest, up to four rows of up to
// 3 * 2^25 weights (4 x 8192 x 8192 13.0 us, the tiles 16.1; 4 x 28672 x 8192 38
// and 35) and up to eight of 3 * 2^23 (8 x 4096 x 4096 7.1 and 9.3; 8 x 8192 x
// 8192 21 and 17).
W4Kind w4_kind(int64_t M, int64_t N, int64_t K) {
  const int64_t weights = N * K;
  if (M <= 2) {
    const bool vec = K > 1024 && (weights > int64_t{1} << (M == 1 ? 24 : 25) || (M == 1 && K > 4096));
    return vec ? kW4Vec : kW4Quad;
  }
  return weights <= int64_t{3} << (M <= 4 ? 25 : 23) && M <= 8 ? kW4Quad : kW4Tile;
}

// Workgroups that share a tile's K: as many as fill the CUs, two stages each at
// least (40 x 2048 x 2048 8.7 us, with four 10.0). The other kernels need none.
int w4_splits(int64_t M, int64_t N, int64_t K) {
  if (w4_kind(M, N, K) != kW4Tile) return 1;
  const int64_t tiles = w4_tiles(M, N, w4_cols(M, N));
  const int64_t stages = (K + kW4StageK - 1) / kW4StageK;
  int64_t splits = tiles < 256 ? 256 / tiles : 1;
  splits = splits < stages / 2 ? splits : stages / 2;
  if (splits <= 1) return 1;
  const int64_t per = (stages + splits - 1) / splits;
  return (int)((stages + per - 1) / per);   // no empty split
}

template <class T>
hipError_t launch_w4_type(const W4Params& p, hipStream_t stream) {
  const W4Kind kind = w4_kind(p.M, p.N, p.K);
  if (kind == kW4Vec)
    return p.M == 1 ? launch_w4_vec<T, 1>(p, stream) : launch_w4_vec<T, 2>(p, stream);
  if (kind == kW4Quad) {
    if (p.M == 1) return launch_w4_quad_k<T, 1>(p, stream);
    if (p.M == 2) return launch_w4_quad_k<T, 2>(p, stream);
    return p.M <= 4 ? launch_w4_quad_k<T, 4>(p, stream) : launch_w4_quad_k<T, 8>(p, stream);
  }
  const bool narrow = w4_cols(p.M, p.N) == 64;
  switch (w4_m_tiles(p.M)) {
    case 1: return narrow ? launch_w4_group<T, 1, 64>(p, stream) : launch_w4_group<T, 1, 128>(p, stream);
    case 2: return narrow ? launch_w4_group<T, 2, 64>(p, stream) : launch_w4_group<T, 2, 128>(p, stream);
    case 3: return narrow ? launch_w4_group<T, 3, 64>(p, stream) : launch_w4_group<T, 3, 128>(p, stream);
    default: return narrow ? launch_w4_group<T, 4, 64>(p, stream) : launch_w4_group<T, 4, 128>(p, stream);
  }
}

}  // namespace

int64_t gemm_w4_partials(int64_t M, int64_t N, int64_t K) {
  const int splits = w4_splits(M, N, K);
  return splits > 1 ? splits * M * N : 0;
}

hipError_t launch_gemm_w4(W4Params p, int type, hipStream_t stream) {
  p.splits = w4_splits(p.M, p.N, p.K);
  return type == 0 ? launch_w4_type<__bf16>(p, stream) : launch_w4_type<_Float16>(p, stream);
}

}  // namespace pipe
