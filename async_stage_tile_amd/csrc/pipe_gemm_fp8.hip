// Products of e4m3 rows with e4m3 weights: C = (A B) * a_scales * b_scales.
//
// The 8-bit MFMAs (v_mfma_f32_32x32x64_f8f6f4, twice the rate of the 16-bit and
// of the older 8-bit forms) keep fewer bits than fp32 while they add up their
// products: of each eight neighbouring k's, products are cut off 13 bits below
// the largest one's leading bit, toward zero; from there on the sums are fp32
// (measured with single products, the older forms' sums are as far off). Sums
// come out 1.5e-5 of their norm off for normal inputs, 3e-5 where one channel in
// a hundred is 11 times louder, 8e-5 where one in 500 is 300 times louder, 2e-4
// where they cancel to a fortieth, K 64 to 16384 alike. Beside bf16's rounding
// (1.6e-3 of the norm) that is nothing to see, so bf16 C takes it for five rows
// of A and more; beside fp16's (2e-4) it is. For fp16 and fp32 C the same bytes
// are turned into fp16 values, exactly, and go through the fp16 MFMAs, whose
// sums are fp32 sums (4e-8 to 9e-8 off), at half the rate: 8192^3 with
// fp16 C takes 735 us for 422, 1000 x 5000 x 4112 46 for 32, 24 x 8192 x 8192
// 16.6 for 16.1.
//
// An MFMA multiplies the bytes that the two operands hold at the same place of
// a lane, so any assignment of k's to places gives the same product as long as
// both operands use it; the loads below choose the one that reads memory or
// LDS in the best order.
//
// Few rows: the call is bound by reading B once, from memory straight into
// registers for up to four (gemv_fp8_kernel), through a deep LDS ring for up to
// 64 and for more of small layers (gemm_fp8_rows_kernel). Many rows:
// gemm_fp8_tile_kernel.
#include "pipe_gemm_tiles.hpp"

namespace pipe {

namespace {

__device__ __forceinline__ i32x8 join(u32x4 a, u32x4 b) {
  return i32x8{(int)a[0], (int)a[1], (int)a[2], (int)a[3], (int)b[0], (int)b[1], (int)b[2], (int)b[3]};
}

// Two e4m3 values as fp16: the low or the high half of a word.
__device__ __forceinline__ f16x2 e4m3_pair(uint32_t w, bool hi) {
  return hi ? __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.f, true)
            : __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.f, false);
}

// acc + x y over 64 k's, of 32 rows each; exact products and fp32 sums, but for
// bf16 C (OUT 0) those of the 8-bit MFMAs.
template <int OUT>
__device__ __forceinline__ f32x16 mma32(i32x8 x, i32x8 y, f32x16 acc) {
  if constexpr (OUT == 0) {
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(x, y, acc, 0, 0, 0, 0, 0, 0);
  } else {
#pragma unroll
    for (int t = 0; t < 8; t += 2) {
      f16x8 a, b;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const f16x2 p = e4m3_pair(x[t + (e >> 1)], e & 1), q = e4m3_pair(y[t + (e >> 1)], e & 1);
        a[2 * e] = p[0];
        a[2 * e + 1] = p[1];
        b[2 * e] = q[0];
        b[2 * e + 1] = q[1];
      }
      acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, acc, 0, 0, 0);
    }
    return acc;
  }
}

// ---------------------------------------------------------------------------
// One to four rows of A. A lane keeps 16 k's of every row in registers, as fp16
// pairs (e4m3 values are fp16 values), and meets them with the same k's of
// kVecRows rows of B, one 16-byte load each: a wave reads 1 KiB of a row at a
// time (LPR lanes make up a row where K is shorter) and all loads of its rows
// are in flight together. v_dot2 adds up two products at a time in fp32. The
// MFMAs, which want 16 rows of B side by side and so 64-byte pieces of each,
// streamed B at 3.6 TB/s where this reads 5 (8192 x 8192 in 12.7 us from HBM).
// Bound by that read; at 4096 x 4096 (4.9 us, floor 2.6) by the launch and one
// trip to memory.
// ---------------------------------------------------------------------------
constexpr int kVecRows = 8;
constexpr int kVecWaves = 8;    // at most, each with slices of K of its own
constexpr int kVecSlice = 1024;

template <int MM, int LPR, int OUT>
__global__ void __launch_bounds__(64 * kVecWaves) gemv_fp8_kernel(Fp8Params p) {
  constexpr int kRowsPer = 64 / LPR;   // rows of B a load
  __shared__ float red[kVecWaves][MM][kVecRows * kRowsPer];
  const int lane = (int)(threadIdx.x & 63);
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int waves = (int)(blockDim.x >> 6);
  const int64_t row0 = long_block() * (kVecRows * kRowsPer);
  if (row0 >= p.N) return;
  float acc[MM][kVecRows];
#pragma unroll
  for (int m = 0; m < MM; ++m)
#pragma unroll
    for (int r = 0; r < kVecRows; ++r) acc[m][r] = 0.f;
  const int slices = LPR < 64 ? 1 : (p.K + kVecSlice - 1) / kVecSlice;
  for (int slice = wave; slice < slices; slice += waves) {
    const int k = slice * kVecSlice + (lane % LPR) * 16;
    const bool in = k < p.K;
    const int kk = in ? k : 0;      // lanes past K read the row's start, and add nothing
    u32x4 a[MM], w[kVecRows];
#pragma unroll
    for (int m = 0; m < MM; ++m)
      a[m] = *reinterpret_cast<const u32x4*>(p.A + min(m, p.M - 1) * p.lda + kk);
#pragma unroll
    for (int r = 0; r < kVecRows; ++r) {
      int64_t n = row0 + r * kRowsPer;
      if constexpr (LPR < 64) n += lane / LPR;
      if (n > p.N - 1) n = p.N - 1;
      w[r] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p.B + n * p.ldb + kk));
    }
    f16x2 av[MM][8];
#pragma unroll
    for (int m = 0; m < MM; ++m)
#pragma unroll
      for (int e = 0; e < 8; ++e) av[m][e] = e4m3_pair(a[m][e >> 1], e & 1);
    if (in) {
#pragma unroll
      for (int r = 0; r < kVecRows; ++r)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const f16x2 b = e4m3_pair(w[r][e >> 1], e & 1);
#pragma unroll
          for (int m = 0; m < MM; ++m)
            acc[m][r] = __builtin_amdgcn_fdot2(av[m][e], b, acc[m][r], false);
        }
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
        const float v = group_sum<LPR>(acc[m][r]);
        if (lane % LPR == 0) red[wave][m][r * kRowsPer + lane / LPR] = v;
      }
    }
  }
  __syncthreads();
  constexpr int kQuads = MM * kVecRows * kRowsPer / 4;
  for (int u = (int)threadIdx.x; u < kQuads; u += (int)blockDim.x) {
    const int m = u / (kQuads / MM), r = u % (kQuads / MM) * 4;
    const int64_t n = row0 + r;
    if (m >= p.M || n >= p.N) continue;
    f32x4 v = {0.f, 0.f, 0.f, 0.f};
    for (int s = 0; s < waves; ++s)
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] += red[s][m][r + e];
    const float sa = p.a_scales[m];
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = v[e] * sa * p.b_scales[n + e];
    store4<OUT>(p.C, m * p.ldc + n, v);
  }
}

// ---------------------------------------------------------------------------
// Five to 64 rows, and more of small layers: bound by reading B once, through
// few CUs' worth of tiles. A workgroup of 8 waves computes 32 FM rows of A
// times 32 WN rows of B. Stages of 512 k pass through an LDS ring (rows of 512
// bytes, 16-byte chunk c of row r at place c ^ (r & 15), 2 rows a direct-to-LDS
// block); wave (wn, wk) takes 32 rows of B and part wk of the stage's k's. The
// parts' sums meet in LDS at the end. One CU's ring holds about 100 KiB of
// loads in flight, which at the memory's latency is 35 KB a us: what counts is
// that every CU has a tile, so tiles are 32 columns wide up to N = 12288, and
// with few of them a long K is split over workgroups too. 24 x 8192 x 8192
// with fp16 C takes 19.7 us from HBM (67 MB: 3.4 TB/s), 16.6 where the memory-side
// cache holds part of it, and 15.5 there without A's loads or the MFMAs: the read
// of B is all but 1 of them. B's loads are non-temporal: 53 us for 8 x 16384
// x 16384 where cached ones take 60 (they win, 14 us for 17, only for weights
// that the memory-side cache still holds from the call before).
// ---------------------------------------------------------------------------
constexpr int kRowsStageK = 512;

template <int FM, int WN>
struct Fp8Rows {
  static constexpr int kN = 32 * WN, kParts = 8 / WN;
  static constexpr int kSteps = kRowsStageK / kParts / 64;   // MFMA steps of a part
  static constexpr int kA = 32 * FM * kRowsStageK, kB = kN * kRowsStageK;
  static constexpr int kSlot = kA + kB;
  static constexpr int kSlots = 163840 / kSlot;
  static constexpr int kLoadsA = kA / kBlockBytes / 8, kLoadsB = kB / kBlockBytes / 8;
  static constexpr int kLoads = kLoadsA + kLoadsB;     // a wave and stage
  static constexpr int kPitch = kN + 4;                // floats of a row of sums
  static_assert(kSlots >= 2 && kParts * 32 * FM * kPitch * 4 <= kSlots * kSlot, "LDS");
};

template <int FM, int WN, int OUT>
__global__ void __launch_bounds__(512) gemm_fp8_rows_kernel(Fp8Params p) {
  using Tile = Fp8Rows<FM, WN>;
  constexpr int kN = Tile::kN, kSteps = Tile::kSteps;
  __shared__ __align__(1024) uint8_t lds[Tile::kSlots * Tile::kSlot];
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int lane = lane_id();
  const int li = lane & 31, lh = lane >> 5;
  const int wn = wave % WN, wk = wave / WN;
  const uint32_t base = uniform(lds_addr(&lds[0]));
  const int tiles = p.tiles_m * p.tiles_n;
  if (long_block() >= tiles * p.splits) return;   // < 2^28: splits only for few tiles
  const int wg = (int)long_block();
  const int split = p.splits == 1 ? 0 : wg / tiles, tile = wg - split * tiles;
  // The longer side's tiles go round the XCDs, so that its operand, read by all
  // workgroups along the shorter side, comes into few L2s (8192 x 64 x 8192 17.9
  // us, the other way round 29.5).
  const bool tall = p.tiles_m > p.tiles_n;
  const int shorter = p.tiles_m == 1 ? 0 : tile / (tall ? p.tiles_m : p.tiles_n);
  const int longer = tile - shorter * (tall ? p.tiles_m : p.tiles_n);
  const int m0 = (tall ? longer : shorter) * 32 * FM, n0 = (tall ? shorter : longer) * kN;
  const int per = p.splits == 1 ? p.steps : (p.steps + p.splits - 1) / p.splits;
  const int first = split * per, count = min(per, p.steps - first);   // >= 1

  const uint8_t* src[Tile::kLoads];
  int src_k[Tile::kLoads];
#pragma unroll
  for (int j = 0; j < Tile::kLoads; ++j) {
    const bool of_a = j < Tile::kLoadsA;
    const int block = of_a ? wave * Tile::kLoadsA + j : wave * Tile::kLoadsB + j - Tile::kLoadsA;
    const int r = block * 2 + (lane >> 5);
    src[j] = of_a ? p.A + (int64_t)min(m0 + r, p.M - 1) * p.lda
                  : p.B + (int64_t)min(n0 + r, p.N - 1) * p.ldb;
    src_k[j] = 16 * ((lane & 31) ^ (r & 15));
  }
  // Loads past K take the stage's first chunk.
  auto load = [&](int ks, int slot) {
    if (ks >= count) return;
    const int k0 = (first + ks) * kRowsStageK;
    const uint32_t to = base + slot * Tile::kSlot;
#pragma unroll
    for (int j = 0; j < Tile::kLoads; ++j) {
      const uint8_t* g = src[j] + k0 + (k0 + src_k[j] < p.K ? src_k[j] : 0);
      if (j < Tile::kLoadsA)
        dma_block(g, to + (wave * Tile::kLoadsA + j) * kBlockBytes);
      else
        dma_block_nt(g, to + Tile::kA + (wave * Tile::kLoadsB + j - Tile::kLoadsA) * kBlockBytes);
    }
  };
  f32x16 acc[FM];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int e = 0; e < 16; ++e) acc[i][e] = 0.f;
  // This wave's part of a slot, of which `left` k's are inside K; half h of a
  // fragment of step t takes chunks 4 t + h and 4 t + 2 + h of it.
  auto compute = [&](int slot, auto CUT, int left) {
    constexpr bool cut = decltype(CUT)::value != 0;
    const uint8_t* a_row = &lds[slot * Tile::kSlot] + li * kRowsStageK;
    const uint8_t* b_row = &lds[slot * Tile::kSlot + Tile::kA] + (32 * wn + li) * kRowsStageK;
    auto read = [&](const uint8_t* row, int t) {
      const int c = 4 * (kSteps * wk + t) + lh;
      return join(*reinterpret_cast<const u32x4*>(row + (c ^ (li & 15)) * 16),
                  *reinterpret_cast<const u32x4*>(row + ((c + 2) ^ (li & 15)) * 16));
    };
    i32x8 a[kSteps][FM], b[kSteps];
#pragma unroll
    for (int t = 0; t < kSteps; ++t) {
      b[t] = read(b_row, t);
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        a[t][i] = read(a_row + i * 32 * kRowsStageK, t);
        if constexpr (cut)
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if ((4 * t + 2 * (e >> 2) + lh) * 16 >= left) a[t][i][e] = 0;
      }
    }
#pragma unroll
    for (int t = 0; t < kSteps; ++t)
#pragma unroll
      for (int i = 0; i < FM; ++i)
        acc[i] = mma32<OUT>(b[t], a[t][i], acc[i]);
  };

  for (int i = 0; i < Tile::kSlots - 1; ++i) load(i, i);
  int slot = 0;
  auto begin = [&](int ks) {
    wait_stage<Tile::kSlots, Tile::kLoads>(ks, count);
    wait_lgkmcnt0();
    __syncthreads();
    load(ks + Tile::kSlots - 1, slot == 0 ? Tile::kSlots - 1 : slot - 1);
  };
  const int whole = (first + count) * kRowsStageK <= p.K ? count : count - 1;
  for (int ks = 0; ks < whole; ++ks) {
    begin(ks);
    compute(slot, Step<0>{}, 64 * kSteps);
    slot = slot + 1 == Tile::kSlots ? 0 : slot + 1;
  }
  if (whole < count) {
    begin(whole);
    compute(slot, Step<1>{}, p.K - (first + whole) * kRowsStageK - 64 * kSteps * wk);
  }
  // The last reads have returned (and the loads before them): the sums' place.
  wait_lgkmcnt0();
  __syncthreads();
  float* sums = reinterpret_cast<float*>(&lds[0]);
  // Lane l holds row l % 32 and columns 8 (e / 4) + 4 (l / 32) + e % 4 of a block.
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int q = 0; q < 4; ++q)
      *reinterpret_cast<f32x4*>(sums + ((wk * FM + i) * 32 + li) * Tile::kPitch + 32 * wn + 8 * q +
                                4 * lh) =
          f32x4{acc[i][4 * q], acc[i][4 * q + 1], acc[i][4 * q + 2], acc[i][4 * q + 3]};
  __syncthreads();
  for (int u = (int)threadIdx.x; u < 32 * FM * (kN / 4); u += 512) {
    const int at = u / (kN / 4), c = u % (kN / 4) * 4, m = m0 + at, n = n0 + c;
    if (m >= p.M || n >= p.N) continue;
    f32x4 v = *reinterpret_cast<const f32x4*>(sums + at * Tile::kPitch + c);
#pragma unroll
    for (int s = 1; s < Tile::kParts; ++s)
      v += *reinterpret_cast<const f32x4*>(sums + (s * 32 * FM + at) * Tile::kPitch + c);
    if (p.splits > 1) {
      *reinterpret_cast<f32x4*>(p.partials + ((int64_t)split * p.M + m) * p.N + n) = v;
    } else {
      const float sa = p.a_scales[m];
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = v[e] * sa * p.b_scales[n + e];
      store4<OUT>(p.C, (int64_t)m * p.ldc + n, v);
    }
  }
}

// ---------------------------------------------------------------------------
// Many rows. Workgroups of WM x WN waves compute tiles of 32 WM FM x 32 WN FN,
// each wave FM x FN MFMA blocks of 32 x 32. A stage of the LDS ring holds 128 k
// (128 bytes: whole cache lines) of the tile's A rows and B rows; S stages.
// 8 rows are one direct-to-LDS block; 16-byte chunk c of row r lies at place
// c ^ ((r >> 1) & 7), which spreads the reads of one chunk of 16 consecutive
// rows over all 64 banks. A stage is two MFMA steps of 64 k; half h (32 lanes)
// of a fragment of step t takes chunks 4 t + h and 4 t + 2 + h.
//
// Fragments are read one step ahead. The first step's MFMAs of a stage go with
// the reads of its second step. Then one barrier: every wave has read all of
// this stage's slot, and its own loads of the next stage have landed. The
// second step's MFMAs go with the loads of the stage S ahead, into this stage's
// slot, and the reads of the next stage's first step. The loads near the end
// fetch the last stage again, so that the loop has no branch and its wait one
// count.
//
// A load's address is a scalar base, which moves 128 bytes a stage, and a
// 32-bit offset a lane that stays: rows of up to 2^24 bytes. Rows past M and N
// are read from the last row and dropped. Lanes whose chunk lies past K (in the
// last stage) load the row's chunk 0 of that stage instead, and A's fragments
// are zeroed there, so that chunk's finite values add nothing, and a NaN in it
// is in the row's product anyway.
//
// 8192^3 with bf16 C takes 409 to 431 us (2.6 PFLOP/s): the MFMAs are at work 69 % of the
// cycles, at the 1.7 GHz that the card holds under this load; the LDS's reads and
// writes take about as many, and the two do not overlap wholly. 1000 x 5000 x
// 4112 takes 32 us in 240 tiles of 192 x 128: 33 stages of 0.72 us (0.57 where the
// pitch is a multiple of 128 bytes), about 60 KB a us and CU out of L2, and 8.7 us
// of launch, ring start and epilogue.
// ---------------------------------------------------------------------------
constexpr int kFp8StageK = 128;
constexpr int kFp8Staging = 4096;   // bytes of a wave's part of the epilogue

// Four floats at any 4-byte boundary.
typedef float f32x4_by4 __attribute__((ext_vector_type(4), aligned(4)));

template <int FM, int FN, int WM, int WN, int S>
struct Fp8Tile {
  static constexpr int kWaves = WM * WN;
  static constexpr int kRowsA = 32 * FM * WM, kRowsB = 32 * FN * WN;
  static constexpr int kLoadsA = kRowsA / 8 / kWaves, kLoadsB = kRowsB / 8 / kWaves;
  static constexpr int kLoads = kLoadsA + kLoadsB;   // blocks a wave and stage
  static constexpr int kStage = (kRowsA + kRowsB) * kFp8StageK;
  static_assert(kRowsA % (16 * kWaves) == 0 && kRowsB % (16 * kWaves) == 0,
                "a wave loads an even number of blocks of each operand");
  static_assert(S * kStage + kWaves * kFp8Staging <= 163840, "the ring and the staging fit");
};

template <int FM, int FN, int WM, int WN, int S, int PER_CU, int OUT>
__global__ void __launch_bounds__(64 * WM * WN, PER_CU) gemm_fp8_tile_kernel(Fp8Params p) {
  using Tile = Fp8Tile<FM, FN, WM, WN, S>;
  __shared__ __align__(1024) uint8_t ring[S][Tile::kStage];
  __shared__ __align__(1024) uint8_t staging[Tile::kWaves][kFp8Staging];
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int lane = lane_id();
  const int li = lane & 31, lh = lane >> 5;
  const int wm = wave / WN, wn = wave % WN;
  const uint32_t base = uniform(lds_addr(&ring[0][0]));
  const int items = p.tiles_m * p.tiles_n * p.splits;  // < 2^31, checked by the host
  const int per = (p.steps + p.splits - 1) / p.splits;

  // The stream of stages that this wave fetches, over all the workgroup's
  // items: kLoadsA blocks of A and kLoadsB of B a stage.
  const uint32_t mine_a = base + wave * Tile::kLoadsA * kBlockBytes;
  const uint32_t mine_b = base + (Tile::kRowsA / 8 + wave * Tile::kLoadsB) * kBlockBytes;
  // In a block, lane l loads the chunk that lies at place l % 8 of row l / 8;
  // this is the even blocks', odd ones' differs in one bit.
  const int chunk0 = (lane & 7) ^ (lane >> 4);
  int f_item = (int)blockIdx.x, f_stage, f_last;   // the item and stage that the next loads fetch
  const uint8_t *ga, *gb;
  uint32_t off[Tile::kLoads], shift[2];
  auto set_shift = [&](int tail) {   // tail: bytes of K in the stage
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int at = (chunk0 ^ (e << 2)) * 16;
      shift[e] = at >= tail ? at : 0;
    }
  };
  int f_k = 0;
  auto open = [&]() {
    int tm, tn, split;
    tile_item(p, f_item, items, tm, tn, split);
    const int row_a = tm * Tile::kRowsA, row_b = tn * Tile::kRowsB;
#pragma unroll
    for (int j = 0; j < Tile::kLoads; ++j) {
      const bool of_a = j < Tile::kLoadsA;
      const int q = of_a ? j : j - Tile::kLoadsA;   // block of the wave's, even with j
      const int r = (wave * (of_a ? Tile::kLoadsA : Tile::kLoadsB) + q) * 8 + (lane >> 3);
      off[j] = (uint32_t)(of_a ? min(r, p.M - row_a - 1) : min(r, p.N - row_b - 1)) *
                   (uint32_t)(of_a ? p.lda : p.ldb) +
               (uint32_t)(chunk0 ^ ((q & 1) << 2)) * 16;
    }
    f_k = split * per * kFp8StageK;
    f_stage = 0;
    f_last = min(per, p.steps - split * per) - 1;   // >= 0: the host leaves no split empty
    ga = p.A + row_a * p.lda + f_k;
    gb = p.B + row_b * p.ldb + f_k;
    set_shift(p.K - f_k);
  };
  auto advance = [&]() {
    if (f_stage < f_last) {
      ++f_stage;
      f_k += kFp8StageK;
      ga += kFp8StageK;
      gb += kFp8StageK;
      if (f_stage == f_last) set_shift(p.K - f_k);
    } else if (f_item + (int)gridDim.x < items) {
      f_item += (int)gridDim.x;
      open();
    }
  };
  auto load = [&](int slot, int j) {
    if (j < Tile::kLoadsA)
      dma_block_at(ga, off[j] - shift[j & 1], mine_a + slot * Tile::kStage + j * kBlockBytes);
    else
      dma_block_at(gb, off[j] - shift[(j - Tile::kLoadsA) & 1],
                   mine_b + slot * Tile::kStage + (j - Tile::kLoadsA) * kBlockBytes);
  };
  // Row 32 i + li of a wave's rows: (r >> 1) & 7 is (li >> 1) & 7 for every i.
  const uint8_t* frag_a = &ring[0][0] + (wm * FM * 32 + li) * kFp8StageK;
  const uint8_t* frag_b = &ring[0][0] + (Tile::kRowsA + wn * FN * 32 + li) * kFp8StageK;
  int place[2][2];
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int e = 0; e < 2; ++e) place[t][e] = ((4 * t + 2 * e + lh) ^ ((li >> 1) & 7)) * 16;
  auto read = [&](const uint8_t* row, int t) {
    return join(*reinterpret_cast<const u32x4*>(row + place[t][0]),
                *reinterpret_cast<const u32x4*>(row + place[t][1]));
  };

  open();
  for (int i = 0; i < S; ++i) {
#pragma unroll
    for (int j = 0; j < Tile::kLoads; ++j) load(i, j);
    advance();
  }
  wait_vmcnt<(S - 1) * Tile::kLoads>();
  __syncthreads();
  i32x8 fa[2][FM], fb[2][FN];

  f32x16 acc[FM][FN];
  // The MFMAs of step T on its fragments, with the reads of the next step's
  // (`ahead` is its slot) and, in the second step, the loads into `slot`. B is
  // the first operand: a lane then holds four neighbouring columns of C's row.
  auto step = [&](auto T, int slot, int ahead) {
    constexpr int t = decltype(T)::value;
    i32x8(&a)[FM] = fa[t];
    i32x8(&b)[FN] = fb[t];
    i32x8(&na)[FM] = fa[t ^ 1];
    i32x8(&nb)[FN] = fb[t ^ 1];
    const uint8_t* sa = frag_a + ahead * Tile::kStage;
    const uint8_t* sb = frag_b + ahead * Tile::kStage;
    constexpr int kBlocks = FM * FN, kReads = FM + FN;
#pragma unroll
    for (int at = 0; at < kBlocks; ++at) {
      const int i = at / FN, j = at % FN;
      acc[i][j] = mma32<OUT>(b[j], a[i], acc[i][j]);
#pragma unroll
      for (int f = at * kReads / kBlocks; f < (at + 1) * kReads / kBlocks; ++f) {
        if (f < FM) na[f] = read(sa + f * 32 * kFp8StageK, t ^ 1);
        else nb[f - FM] = read(sb + (f - FM) * 32 * kFp8StageK, t ^ 1);
      }
      if constexpr (t == 1) {
#pragma unroll
        for (int l = at * Tile::kLoads / kBlocks; l < (at + 1) * Tile::kLoads / kBlocks; ++l)
          load(slot, l);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  auto zero_past = [&](i32x8(&a)[FM], int t, int tail) {
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if ((4 * t + 2 * (e >> 2) + lh) * 16 >= tail) a[i][e] = 0;
  };

  int slot = 0;
  for (int item = (int)blockIdx.x; item < items; item += (int)gridDim.x) {
    int tm, tn, split;
    tile_item(p, item, items, tm, tn, split);
    const int first = split * per, count = min(per, p.steps - first);
    const int tail = p.K - (first + count - 1) * kFp8StageK;   // bytes of K in the last stage, and more
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.f;
    // Read here and not with the previous item's last step: the registers are
    // its epilogue's until now.
#pragma unroll
    for (int i = 0; i < FM; ++i)
      fa[0][i] = read(frag_a + slot * Tile::kStage + i * 32 * kFp8StageK, 0);
#pragma unroll
    for (int j = 0; j < FN; ++j)
      fb[0][j] = read(frag_b + slot * Tile::kStage + j * 32 * kFp8StageK, 0);
    for (int ks = 0; ks < count; ++ks) {
      const bool cut = ks == count - 1 && tail < kFp8StageK;
      const int next = slot + 1 == S ? 0 : slot + 1;
      if (cut) zero_past(fa[0], 0, tail);
      step(Step<0>{}, slot, slot);
      // At most the loads of the stages ks + 2 .. ks + S - 1 are younger than
      // those of stage ks + 1 (and the last item's stores: not counted, which
      // only makes the wait longer).
      wait_vmcnt<(S - 2) * Tile::kLoads>();
      wait_lgkmcnt0();
      __syncthreads();
      if (cut) zero_past(fa[1], 1, tail);
      step(Step<1>{}, slot, next);   // after the last stage its reads are not used
      advance();
      slot = next;
    }

    __builtin_amdgcn_sched_barrier(0);
    // Lane l holds row l % 32 and columns 8 (e / 4) + 4 (l / 32) + e % 4 of a
    // block. Rows of 128 bytes go through the wave's own staging buffer, its
    // 16-byte chunks placed as the ring's, and leave as whole cache lines,
    // while the next item's first stages arrive.
    // The lane is made anew for the compiler, which would else compute the
    // epilogue's addresses before the loop and spill them.
    int el = lane;
    asm volatile("" : "+v"(el));
    const int eli = el & 31, elh = el >> 5;
    uint8_t* mid = &staging[wave][0];
    // Unsigned: the last tile of 192 rows may end past 2^31.
    const uint32_t row0 = (uint32_t)tm * Tile::kRowsA + wm * FM * 32;
    const int col0 = tn * Tile::kRowsB + wn * FN * 32;
    const int wrow = eli * 128, wswz = (eli >> 1) & 7;
    auto flush = [&](uint8_t* out, int64_t pitch, uint32_t row, int col, int per_chunk) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int r = 8 * k + (el >> 3), c = (el & 7) ^ ((r >> 1) & 7);
        const u32x4 v = *reinterpret_cast<const u32x4*>(mid + r * 128 + (el & 7) * 16);
        if (row + r < (uint32_t)p.M && col + c * per_chunk < p.N)
          *reinterpret_cast<u32x4*>(out + (row + r) * pitch + (int64_t)col * (16 / per_chunk) + c * 16) = v;
      }
    };
    auto block32 = [&](int i, int j, float sa, const f32x4(&sb)[4], uint8_t* out, int64_t pitch) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        f32x4 v;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = acc[i][j][4 * q + e] * sa * sb[q][e];
        *reinterpret_cast<f32x4*>(mid + wrow + ((2 * q + elh) ^ wswz) * 16) = v;
      }
      flush(out, pitch, row0 + 32 * i, col0 + 32 * j, 4);
    };
    if (p.splits > 1) {
      const f32x4 one = {1.f, 1.f, 1.f, 1.f};
      const f32x4 ones[4] = {one, one, one, one};
      uint8_t* out = reinterpret_cast<uint8_t*>(p.partials + (int64_t)split * p.M * p.N);
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) block32(i, j, 1.f, ones, out, (int64_t)p.N * 4);
      continue;
    }
    f32x4 sb[FN][4];
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        sb[j][q] = *reinterpret_cast<const f32x4_by4*>(
            p.b_scales + min(col0 + 32 * j + 8 * q + 4 * elh, p.N - 4));
    uint8_t* out = static_cast<uint8_t*>(p.C);
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      const float sa = p.a_scales[min(row0 + 32 * i + eli, (uint32_t)p.M - 1)];
      if constexpr (OUT == 2) {
#pragma unroll
        for (int j = 0; j < FN; ++j) block32(i, j, sa, sb[j], out, p.ldc * 4);
      } else {
        static_assert(FN == 2, "a wave's row of 16-bit values is 128 bytes");
        using T = typename Out16<OUT>::type;
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            f32x4 v;
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = acc[i][j][4 * q + e] * sa * sb[j][q][e];
            *reinterpret_cast<u32x2*>(mid + wrow + ((4 * j + q) ^ wswz) * 16 + elh * 8) =
                u32x2{Pair<T>::pack(v[0], v[1]), Pair<T>::pack(v[2], v[3])};
          }
        flush(out, p.ldc * 2, row0 + 32 * i, col0, 8);
      }
    }
  }
  wait_vmcnt<0>();
}

// Sum of the splits' partial products in split order, scaled and rounded: four
// columns a thread. Bound by a launch and trips to memory, so four splits' loads
// go out together (30 x 512 x 16384 8.2 us in all, one at a time 9.5).
template <int OUT>
__global__ void __launch_bounds__(256) gemm_fp8_join_kernel(Fp8Params p) {
  const int quads = p.N >> 2;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= (int64_t)p.M * quads) return;
  const int m = (int)(i / quads), n = (int)(i % quads) * 4;
  const int64_t plane = (int64_t)p.M * p.N;
  const float* src = p.partials + (int64_t)m * p.N + n;
  f32x4 v = *reinterpret_cast<const f32x4*>(src);
#pragma unroll 4
  for (int s = 1; s < p.splits; ++s) v += *reinterpret_cast<const f32x4*>(src + s * plane);
  const float sa = p.a_scales[m];
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = v[e] * sa * p.b_scales[n + e];
  store4<OUT>(p.C, (int64_t)m * p.ldc + n, v);
}

// ---------------------------------------------------------------------------
// Choice of kernel.
// ---------------------------------------------------------------------------
enum Fp8Kind { kVec, kRows, kTile128, kTile128Pair, kTile192, kTile256 };

struct Fp8Plan {
  Fp8Kind kind;
  int tiles_m, tiles_n, splits, steps;
  bool wide;   // kRows: 64 columns
};

Fp8Plan fp8_plan(int64_t M, int64_t N, int64_t K) {
  Fp8Plan c{kVec, 0, 0, 1, 0, false};
  if (M <= 4) return c;
  // The few-row kernel, also for more rows while its tiles of 64 x 32 all run at
  // once and K is not long: 128 x 4096 x 4096 takes 9.7 us and in the large tiles
  // 18.7, 256 x 1024 x 4096 8.8 and 15.0; 128 x 4096 x 14336 24.8 and 22.1, and
  // with two rounds of them 128 x 8192 x 8192 35 and 23. Its tiles of 64 x 64
  // likewise up to half that K: 256 x 4096 x 4096 15.1 and 18.6, 300 x 3000 x 2000
  // 11.8 and 16.8; 1024 x 1024 x 8192 27.2 and 21.7.
  const int64_t tall = (M + 63) / 64;
  const bool few32 = tall * ((N + 31) / 32) <= 256 && K <= 8192;
  const bool few64 = tall * ((N + 63) / 64) <= 256 && K <= 4096;
  if (M <= 64 || few32 || few64) {
    c.kind = kRows;
    c.tiles_m = ceil_div(M, 64);
    c.wide = M <= 64 ? N > 192 * 64 : !few32;
    c.tiles_n = ceil_div(N, c.wide ? 64 : 32);
    c.steps = ceil_div(K, kRowsStageK);
    const int tiles = c.tiles_m * c.tiles_n;
    // K is split where that gives idle CUs enough stages to pay for the join: 16 x
    // 1024 x 3008 takes 5.0 us whole and 6.1 split, 33 x 1000 x 8192 7.9 in 6
    // parts; 24 x 4096 x 14336 14.5 in two and 18.2 whole, 8 x 4096 x 4096 7.3 and
    // 6.5.
    const int most = tiles < 96 ? 192 / tiles : tiles <= 128 && c.steps >= 16 ? 2 : 1;
    c.splits = c.steps >= 8 ? shares(c.steps, most, 2) : 1;
    return c;
  }
  // The tile kernels: of all tile shapes and splits of K, the least estimate of
  // time. A workgroup takes so many us a stage with every CU at work (8192^3 and
  // 2048 x 4096 x 4096, measured): a tile of 256 x 256 1.63, of 192 x 128 0.70,
  // of 128 x 128 alone on its CU 0.56, two of these on one CU 0.95 together.
  // Partial products cost 2 us, and 8 bytes each at 8 TB/s.
  struct Shape {
    Fp8Kind kind;
    int rows, cols, places, most;   // most: splits of K
    float us;
  };
  static constexpr Shape kShapes[] = {{kTile256, 256, 256, 256, 1, 1.63f},
                                      {kTile192, 192, 128, 256, 8, 0.70f},
                                      {kTile128, 128, 128, 256, 16, 0.56f},
                                      {kTile128Pair, 128, 128, 512, 16, 0.95f}};
  c.steps = ceil_div(K, kFp8StageK);
  float best = 0.f;
  for (const Shape& sh : kShapes) {
    const int tiles_m = ceil_div(M, sh.rows), tiles_n = ceil_div(N, sh.cols);
    const int64_t tiles = (int64_t)tiles_m * tiles_n;
    for (int want = 1; want <= sh.most; ++want) {
      const int splits = shares(c.steps, want, 4);
      if (splits != want) continue;
      const int64_t rounds = (tiles * splits + sh.places - 1) / sh.places;
      float t = (float)rounds * (float)ceil_div(c.steps, splits) * sh.us;
      if (splits > 1) t += 2.f + (float)splits * (float)M * (float)N * 1e-6f;
      if (best == 0.f || t < best) {
        best = t;
        c.kind = sh.kind;
        c.tiles_m = tiles_m;
        c.tiles_n = tiles_n;
        c.splits = splits;
      }
      if (tiles * splits >= sh.places) break;
    }
  }
  return c;
}

template <int MM, int LPR, int OUT>
hipError_t launch_fp8_vec(const Fp8Params& p, hipStream_t stream) {
  constexpr int kRows = kVecRows * (64 / LPR);
  const int slices = LPR < 64 ? 1 : ceil_div(p.K, kVecSlice);
  const int waves = ceil_div(slices, ceil_div(slices, kVecWaves));
  hipLaunchKernelGGL((gemv_fp8_kernel<MM, LPR, OUT>), long_grid(((int64_t)p.N + kRows - 1) / kRows),
                     dim3(64 * waves), 0, stream, p);
  return hipGetLastError();
}

// As many lanes a row as K has 16-byte chunks, up to a wave.
template <int MM, int OUT>
hipError_t launch_fp8_vec_k(const Fp8Params& p, hipStream_t stream) {
  if (p.K <= 16 * 16) return launch_fp8_vec<MM, 16, OUT>(p, stream);
  if (p.K <= 32 * 16) return launch_fp8_vec<MM, 32, OUT>(p, stream);
  return launch_fp8_vec<MM, 64, OUT>(p, stream);
}

template <int OUT>
hipError_t launch_fp8_out(const Fp8Params& p, Fp8Kind kind, bool wide, hipStream_t stream) {
  const int items = p.tiles_m * p.tiles_n * p.splits;
  switch (kind) {
    case kVec:
      if (p.M == 1) return launch_fp8_vec_k<1, OUT>(p, stream);
      if (p.M == 2) return launch_fp8_vec_k<2, OUT>(p, stream);
      return launch_fp8_vec_k<4, OUT>(p, stream);
    case kRows: {
      void (*k)(Fp8Params) =
          p.M <= 32 ? (wide ? gemm_fp8_rows_kernel<1, 2, OUT> : gemm_fp8_rows_kernel<1, 1, OUT>)
                    : (wide ? gemm_fp8_rows_kernel<2, 2, OUT> : gemm_fp8_rows_kernel<2, 1, OUT>);
      hipLaunchKernelGGL(k, long_grid(items), dim3(512), 0, stream, p);
      break;
    }
    case kTile128:
      hipLaunchKernelGGL((gemm_fp8_tile_kernel<2, 2, 2, 2, 4, 1, OUT>),
                         dim3(items < 256 ? items : 256), dim3(256), 0, stream, p);
      break;
    case kTile128Pair:
      hipLaunchKernelGGL((gemm_fp8_tile_kernel<2, 2, 2, 2, 2, 2, OUT>),
                         dim3(items < 512 ? items : 512), dim3(256), 0, stream, p);
      break;
    case kTile192:
      hipLaunchKernelGGL((gemm_fp8_tile_kernel<3, 2, 2, 2, 3, 1, OUT>),
                         dim3(items < 256 ? items : 256), dim3(256), 0, stream, p);
      break;
    default:
      hipLaunchKernelGGL((gemm_fp8_tile_kernel<4, 2, 2, 4, 2, 1, OUT>),
                         dim3(items < 256 ? items : 256), dim3(512), 0, stream, p);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.splits == 1) return e;
  const int64_t quads = (int64_t)p.M * (p.N / 4);
  hipLaunchKernelGGL(gemm_fp8_join_kernel<OUT>, dim3((unsigned)((quads + 255) / 256)), dim3(256), 0,
                     stream, p);
  return hipGetLastError();
}

}  // namespace

int64_t gemm_fp8_partials(int64_t M, int64_t N, int64_t K) {
  const Fp8Plan c = fp8_plan(M, N, K);
  return c.splits > 1 ? (int64_t)c.splits * M * N : 0;
}

hipError_t launch_gemm_fp8(Fp8Params p, int out_type, hipStream_t stream) {
  const Fp8Plan c = fp8_plan(p.M, p.N, p.K);
  p.tiles_m = c.tiles_m;
  p.tiles_n = c.tiles_n;
  p.splits = c.splits;
  p.steps = c.steps;
  if (out_type == 0) return launch_fp8_out<0>(p, c.kind, c.wide, stream);
  if (out_type == 1) return launch_fp8_out<1>(p, c.kind, c.wide, stream);
  return launch_fp8_out<2>(p, c.kind, c.wide, stream);
}

}  // namespace pipe
