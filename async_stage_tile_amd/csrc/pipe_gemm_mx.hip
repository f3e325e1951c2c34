// Products of rows and weights in the microscaled 4-bit form: C = A W^T.
//
// The 4-bit MFMAs (v_mfma_scale_f32_32x32x64_f8f6f4) multiply 32 k's of a lane's
// row with 32 of another's and the sum with both blocks' powers of two. A product
// of two e2m1 values is a multiple of 1/4 up to 36, so the 32 add up exactly; sums
// of blocks are fp32 sums (measured, 64 steps of random exponents: 1.05e-7 of the
// sums' norm off, as sums in fp32 one block after the other are). So every C, fp32
// among them, takes them.
//
// An MFMA multiplies what the two operands hold at the same place of a lane, so any
// assignment of blocks of k to places gives the same product as long as both
// operands and their scales use it; the loads below choose the one that reads
// memory or LDS in the best order. All offsets along K are in bytes, two k's each:
// a block of 32 is a 16-byte chunk and a byte of scale.
//
// Where a stage reaches past K, the codes there are another block's of the row and
// the scales may be anything. Both operands' scales are set to zero, 2^-127 each:
// e2m1 has no infinity and no NaN, and 2^-254 times any sum of 32 products is zero
// in fp32.
//
// Few rows: the call is bound by reading W once, from memory straight into registers
// for one and two (gemv_mx_kernel), through an LDS ring for up to 64 and for more of
// small layers (gemm_mx_rows_kernel). Many rows: gemm_mx_tile_kernel.
#include "pipe_gemm_tiles.hpp"
#include "pipe_mx.hpp"

namespace pipe {

namespace {

constexpr int kBlock = 16;   // bytes of a block of 32 k's

struct MxPackParams {
  const uint8_t *a, *w;
  uint8_t *to_a, *to_w;
  int64_t ld_a, ld_w;
  int32_t rows_a, rows_w, blocks_a, pairs;   // blocks of 64 rows
};

// acc + x y over 64 k's of 32 rows each; byte SEL of the scale words counts.
template <int SEL>
__device__ __forceinline__ f32x16 mx_mma(u32x4 x, u32x4 y, f32x16 acc, uint32_t sx, uint32_t sy) {
  const i32x8 a = {(int)x[0], (int)x[1], (int)x[2], (int)x[3], 0, 0, 0, 0};
  const i32x8 b = {(int)y[0], (int)y[1], (int)y[2], (int)y[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, acc, 4, 4, SEL, (int)sx, SEL, (int)sy);
}

// A use of a sum ahead of a branch: the compiler would else move its MFMAs behind
// it, out of the reads and loads they go with.
template <bool ACC>
__device__ __forceinline__ void keep_sum(f32x16 v) {
  if constexpr (ACC) asm volatile("" : : "a"(v));
  else asm volatile("" : : "v"(v));
}

// ---------------------------------------------------------------------------
// One or two rows of A. A lane keeps 32 k's of every row in registers, as fp16
// pairs (e2m1 values are fp16 values), and meets them with the same k's of kVecRows
// rows of W, one 16-byte load each: a wave reads 1 KiB of a row at a time (LPR lanes
// make up a row where K is shorter) and all loads of its rows are in flight
// together. v_dot2 adds up two products at a time in fp32, exactly; a block's sum is
// scaled by the sum of the two exponents. One row of 28672 x 8192 takes 21.3 us from HBM
// (5.9 TB/s), of 8192 x 8192 9.1 and of 4096 x 4096 5.3, of which a launch and one trip
// to memory are 4.
// ---------------------------------------------------------------------------
constexpr int kVecRows = 8;
constexpr int kVecWaves = 8;    // at most, each with slices of K of its own
constexpr int kVecSlice = 1024;

__device__ __forceinline__ void mx_pairs(u32x4 w, f16x2 (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[4 * i] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w[i], 1.f, 0);
    v[4 * i + 1] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w[i], 1.f, 1);
    v[4 * i + 2] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w[i], 1.f, 2);
    v[4 * i + 3] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w[i], 1.f, 3);
  }
}

template <int MM, int LPR, int OUT>
__global__ void __launch_bounds__(64 * kVecWaves) gemv_mx_kernel(MxGemmParams p) {
  constexpr int kRowsPer = 64 / LPR;   // rows of W a load
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
  const int slices = LPR < 64 ? 1 : (int)(((int64_t)p.bytes + kVecSlice - 1) / kVecSlice);
  for (int slice = wave; slice < slices; slice += waves) {
    const int k = slice * kVecSlice + (lane % LPR) * kBlock;
    const bool in = k < p.bytes;
    const int kk = in ? k : 0;      // lanes past K read the row's start, and add nothing
    u32x4 a[MM], w[kVecRows];
    int ea[MM], ew[kVecRows];
#pragma unroll
    for (int m = 0; m < MM; ++m) {
      const int row = min(m, p.M - 1);
      a[m] = *reinterpret_cast<const u32x4*>(p.A + row * p.lda + kk);
      ea[m] = p.a_scales[row * p.ld_as + kk / kBlock];
    }
#pragma unroll
    for (int r = 0; r < kVecRows; ++r) {
      int64_t n = row0 + r * kRowsPer;
      if constexpr (LPR < 64) n += lane / LPR;
      if (n > p.N - 1) n = p.N - 1;
      w[r] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p.W + n * p.ldw + kk));
      ew[r] = p.w_scales[n * p.ld_ws + kk / kBlock];
    }
    f16x2 av[MM][16];
#pragma unroll
    for (int m = 0; m < MM; ++m) mx_pairs(a[m], av[m]);
    if (in) {
#pragma unroll
      for (int r = 0; r < kVecRows; ++r) {
        f16x2 wv[16];
        mx_pairs(w[r], wv);
#pragma unroll
        for (int m = 0; m < MM; ++m) {
          float s = 0.f;
#pragma unroll
          for (int e = 0; e < 16; ++e) s = __builtin_amdgcn_fdot2(av[m][e], wv[e], s, false);
          s = ea[m] == 255 || ew[r] == 255 ? __uint_as_float(0x7FC00000u) : s;
          acc[m][r] += __builtin_amdgcn_ldexpf(s, ea[m] + ew[r] - 254);
        }
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
    store4<OUT>(p.C, m * p.ldc + n, v);
  }
}

// ---------------------------------------------------------------------------
// Two to 64 rows, and more of small layers: bound by reading W once, through few
// CUs' worth of tiles. A workgroup of 8 waves computes 32 FM rows of A times 32 WN
// rows of W. Stages of 1024 k (512 bytes of a row, and 32 of its scales) pass through
// an LDS ring: data rows of 512 bytes, 16-byte chunk c of row r at place c ^ (r & 15),
// 2 rows a direct-to-LDS block; behind them the scales, rows of 32 bytes, 32 rows a
// block, which the first waves load. Wave (wn, wk) takes 32 rows of W and part wk of
// the stage's k's. The parts' sums meet in LDS at the end. With few tiles a long K is
// split over workgroups too. 24 x 8192 x 8192 takes 10.4 us from HBM (36 MB: launch, first
// trip and tail are 5), 8 x 16384 x 16384 26 (5.5 TB/s); W's loads are non-temporal (cached
// 10.6 and 30).
// ---------------------------------------------------------------------------
constexpr int kRowsStage = 512;                            // bytes of a row
constexpr int kRowsScales = kRowsStage / kBlock;           // of its scales

template <int FM, int WN>
struct MxRows {
  static constexpr int kN = 32 * WN, kParts = 8 / WN;
  static constexpr int kSteps = kRowsStage / 32 / kParts;   // MFMA steps of a part
  static constexpr int kA = 32 * FM * kRowsStage, kB = kN * kRowsStage;
  static constexpr int kScaleBlocks = (32 * FM + kN) * kRowsScales / kBlockBytes;
  static constexpr int kSlot = kA + kB + kScaleBlocks * kBlockBytes;
  static constexpr int kSlots = 163840 / kSlot;
  static constexpr int kLoadsA = kA / kBlockBytes / 8, kLoadsB = kB / kBlockBytes / 8;
  static constexpr int kLoads = kLoadsA + kLoadsB;     // a wave and stage
  static constexpr int kPitch = kN + 4;                // floats of a row of sums
  static_assert(kSlots >= 2 && kParts * 32 * FM * kPitch * 4 <= kSlots * kSlot, "LDS");
  static_assert(kScaleBlocks <= 8 && kScaleBlocks == FM + WN, "a block of scales is one operand's");
};

template <int FM, int WN, int OUT>
__global__ void __launch_bounds__(512) gemm_mx_rows_kernel(MxGemmParams p) {
  using Tile = MxRows<FM, WN>;
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
  // workgroups along the shorter side, comes into few L2s.
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
                  : p.W + (int64_t)min(n0 + r, p.N - 1) * p.ldw;
    src_k[j] = kBlock * ((lane & 31) ^ (r & 15));
  }
  // Block `wave` of the scales: rows 32 wave + lane / 2, halves of 16 blocks.
  const bool scales = wave < Tile::kScaleBlocks;
  const int scale_half = (lane & 1) * 16;
  const uint8_t* scale_src =
      wave < FM ? p.a_scales + (int64_t)min(m0 + 32 * wave + (lane >> 1), p.M - 1) * p.ld_as
                : p.w_scales + (int64_t)min(n0 + 32 * (wave - FM) + (lane >> 1), p.N - 1) * p.ld_ws;
  const int blocks = p.bytes / kBlock;
  // Loads past K take the stage's first chunk.
  auto load = [&](int ks, int slot) {
    if (ks >= count) return;
    const int k0 = (first + ks) * kRowsStage;
    const uint32_t to = base + slot * Tile::kSlot;
#pragma unroll
    for (int j = 0; j < Tile::kLoads; ++j) {
      const uint8_t* g = src[j] + k0 + (k0 + src_k[j] < p.bytes ? src_k[j] : 0);
      if (j < Tile::kLoadsA)
        dma_block(g, to + (wave * Tile::kLoadsA + j) * kBlockBytes);
      else
        dma_block_nt(g, to + Tile::kA + (wave * Tile::kLoadsB + j - Tile::kLoadsA) * kBlockBytes);
    }
    if (scales) {
      const int b0 = k0 / kBlock;
      dma_block(scale_src + b0 + (b0 + scale_half < blocks ? scale_half : 0),
                to + Tile::kA + Tile::kB + wave * kBlockBytes);
    }
  };
  f32x16 acc[FM];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int e = 0; e < 16; ++e) acc[i][e] = 0.f;
  // This wave's part of a slot, of which `left` bytes are inside K; half h of step
  // t's fragments takes chunk 2 t + h of it.
  auto compute = [&](int slot, int left) {
    const uint8_t* at = &lds[slot * Tile::kSlot];
    const uint8_t* a_row = at + li * kRowsStage;
    const uint8_t* w_row = at + Tile::kA + (32 * wn + li) * kRowsStage;
    const uint8_t* a_scale = at + Tile::kA + Tile::kB + li * kRowsScales + wk * 2 * kSteps;
    const uint8_t* w_scale = a_scale + (32 * FM + 32 * wn) * kRowsScales;
    auto read = [&](const uint8_t* row, int t) {
      const int c = 2 * (kSteps * wk + t) + lh;
      return *reinterpret_cast<const u32x4*>(row + (c ^ (li & 15)) * kBlock);
    };
    // The scales of steps 2 q and 2 q + 1 in bytes 0 and 2.
    auto read_scales = [&](const uint8_t* row, int q) {
      return *reinterpret_cast<const uint32_t*>(row + 4 * q) >> (8 * lh);
    };
    u32x4 a[kSteps][FM], w[kSteps];
    uint32_t sa[kSteps / 2][FM], sw[kSteps / 2];
#pragma unroll
    for (int q = 0; q < kSteps / 2; ++q) {
      const int inside = (left - lh * kBlock + 31) >> 5;   // steps of this half inside K
      const uint32_t mask = inside >= 2 * q + 2 ? ~0u : inside == 2 * q + 1 ? 0xFFFFu : 0u;
      sw[q] = read_scales(w_scale, q) & mask;
#pragma unroll
      for (int i = 0; i < FM; ++i) sa[q][i] = read_scales(a_scale + 32 * i * kRowsScales, q) & mask;
    }
#pragma unroll
    for (int t = 0; t < kSteps; ++t) {
      w[t] = read(w_row, t);
#pragma unroll
      for (int i = 0; i < FM; ++i) a[t][i] = read(a_row + i * 32 * kRowsStage, t);
    }
#pragma unroll
    for (int t = 0; t < kSteps; ++t)
#pragma unroll
      for (int i = 0; i < FM; ++i)
        acc[i] = (t & 1) ? mx_mma<2>(w[t], a[t][i], acc[i], sw[t >> 1], sa[t >> 1][i])
                         : mx_mma<0>(w[t], a[t][i], acc[i], sw[t >> 1], sa[t >> 1][i]);
  };

  for (int i = 0; i < Tile::kSlots - 1; ++i) load(i, i);
  int slot = 0;
  auto begin = [&](int ks) {
    if (scales)
      wait_stage<Tile::kSlots, Tile::kLoads + 1>(ks, count);
    else
      wait_stage<Tile::kSlots, Tile::kLoads>(ks, count);
    wait_lgkmcnt0();
    __syncthreads();
    load(ks + Tile::kSlots - 1, slot == 0 ? Tile::kSlots - 1 : slot - 1);
  };
  for (int ks = 0; ks < count; ++ks) {
    begin(ks);
    compute(slot, p.bytes - (first + ks) * kRowsStage - 32 * kSteps * wk);
    slot = slot + 1 == Tile::kSlots ? 0 : slot + 1;
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
    if (p.splits > 1)
      *reinterpret_cast<f32x4*>(p.partials + ((int64_t)split * p.M + m) * p.N + n) = v;
    else
      store4<OUT>(p.C, (int64_t)m * p.ldc + n, v);
  }
}

// ---------------------------------------------------------------------------
// Many rows. Workgroups of WM x WN waves compute tiles of 32 WM FM x 32 WN FN, each
// wave FM x FN MFMA blocks of 32 x 32. A stage of the LDS ring holds 256 k (128 bytes:
// whole cache lines) of the tile's A rows and W rows; S stages. 8 rows are one
// direct-to-LDS block; 16-byte chunk c of row r lies at place c ^ ((r >> 1) & 7),
// which spreads the reads of one chunk of 16 consecutive rows over all 64 banks. A
// stage is four MFMA steps of 64 k; half h (32 lanes) of step t's fragments takes
// chunk 2 t + h.
//
// The scales of a row and two stages are 16 bytes: one direct-to-LDS block a 64 rows
// and pair of stages, into a ring of its own (S pairs: a product of K <= 256 has a
// pair for each stage).
//
// Fragments are read one step ahead, all within the first two MFMAs. Before the last
// step of a stage comes one barrier: every wave has read all of this stage's slot, and
// its own loads of the next stage have landed. The last step's MFMAs go with the loads
// of the stage S ahead, into this stage's slot, and the reads of the next stage's
// first fragments and scales; the third step's with the addresses of those loads,
// without a branch but at an item's end. The loads near the end fetch the last stage
// again, so that the wait has one count (the scales' loads come on top of it, which
// only makes the wait longer). C's stores are non-temporal, and the first wait behind
// an epilogue does not wait for them: they leave beside the next item's first stage.
//
// A load's address is a scalar base, which moves on, and a 32-bit offset a lane that
// stays: rows of up to 2^24 bytes. Rows past M and N are read from the last row and
// dropped. Lanes whose chunk lies past K (in the last stage) load the row's chunk 0 of
// that stage instead.
// ---------------------------------------------------------------------------
constexpr int kTileStage = 128;    // bytes of a row
constexpr int kStaging = 2048;     // bytes of a wave's part of the epilogue

template <int FM, int FN, int WM, int WN, int S>
struct MxTile {
  static constexpr int kWaves = WM * WN;
  static constexpr int kRowsA = 32 * FM * WM, kRowsB = 32 * FN * WN;
  static constexpr int kLoadsA = kRowsA / 8 / kWaves, kLoadsB = kRowsB / 8 / kWaves;
  static constexpr int kLoads = kLoadsA + kLoadsB;   // blocks a wave and stage
  static constexpr int kStage = (kRowsA + kRowsB) * kTileStage;
  static constexpr int kScaleBlocks = (kRowsA + kRowsB) / 64;                       // a pair
  static constexpr int kScaleLoads = (kScaleBlocks + kWaves - 1) / kWaves;           // a wave and pair, at most
  static constexpr int kScaleSlot = kScaleBlocks * kBlockBytes;
  static_assert(kRowsA % (16 * kWaves) == 0 && kRowsB % (16 * kWaves) == 0,
                "a wave loads an even number of blocks of each operand");
  static_assert(kRowsA % 64 == 0 && kRowsB % 64 == 0, "a block of scales is one operand's");
  static_assert(S * (kStage + kScaleSlot) + kWaves * kStaging <= 163840, "the rings and the staging fit");
};

template <int FM, int FN, int WM, int WN, int S, int PER_CU, int OUT>
__global__ void __launch_bounds__(64 * WM * WN, PER_CU) gemm_mx_tile_kernel(MxGemmParams p) {
  using Tile = MxTile<FM, FN, WM, WN, S>;
  __shared__ __align__(1024) uint8_t ring[S][Tile::kStage];
  __shared__ __align__(1024) uint8_t scale_ring[S][Tile::kScaleSlot];
  __shared__ __align__(1024) uint8_t staging[Tile::kWaves][kStaging];
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int lane = lane_id();
  const int li = lane & 31, lh = lane >> 5;
  const int wm = wave / WN, wn = wave % WN;
  const uint32_t base = uniform(lds_addr(&ring[0][0]));
  const uint32_t scale_base = uniform(lds_addr(&scale_ring[0][0])) + wave * kBlockBytes;
  const int items = p.tiles_m * p.tiles_n * p.splits;  // < 2^31, checked by the host
  // A split's first stage is the first of a pair.
  const int per = p.splits == 1 ? p.steps : ((p.steps + p.splits - 1) / p.splits + 1) & ~1;

  // The stream of stages that this wave fetches, over all the workgroup's
  // items: kLoadsA blocks of A and kLoadsB of W a stage.
  const uint32_t mine_a = base + wave * Tile::kLoadsA * kBlockBytes;
  const uint32_t mine_b = base + (Tile::kRowsA / 8 + wave * Tile::kLoadsB) * kBlockBytes;
  // In a block, lane l loads the chunk that lies at place l % 8 of row l / 8;
  // this is the even blocks', odd ones' differs in one bit.
  const int chunk0 = (lane & 7) ^ (lane >> 4);
  int f_item = (int)blockIdx.x, f_stage, f_last;   // the item and stage that the next loads fetch
  int f_pair = 0;                                  // the slot of its scales
  bool f_scales = true, f_more = true;             // whether they are still to be fetched
  const uint8_t *ga, *gb;
  const uint8_t* gs[Tile::kScaleLoads];
  uint32_t off[Tile::kLoads], scale_off[Tile::kScaleLoads], shift[2], last_shift[2];
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
                   (uint32_t)(of_a ? p.lda : p.ldw) +
               (uint32_t)(chunk0 ^ ((q & 1) << 2)) * kBlock;
    }
    const int f_k = split * per * kTileStage;
    f_stage = 0;
    f_last = min(per, p.steps - split * per) - 1;   // >= 0: the host leaves no split empty
    ga = p.A + row_a * p.lda + f_k;
    gb = p.W + row_b * p.ldw + f_k;
#pragma unroll
    for (int j = 0; j < Tile::kScaleLoads; ++j) {
      const int r = (j * Tile::kWaves + wave) * 64;
      const bool of_a = r < Tile::kRowsA;
      const int64_t pair = f_k / (2 * kTileStage);
      gs[j] = of_a ? p.a_scales + row_a * p.ld_as + pair * p.step_as
                   : p.w_scales + row_b * p.ld_ws + pair * p.step_ws;
      scale_off[j] = (uint32_t)(of_a ? min(r + lane, p.M - row_a - 1)
                                     : min(r - Tile::kRowsA + lane, p.N - row_b - 1)) *
                     (uint32_t)(of_a ? p.ld_as : p.ld_ws);
    }
    // Chunks past K of the last stage, as far back as its first one.
    const int tail = p.bytes - f_k - f_last * kTileStage;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int at = (chunk0 ^ (e << 2)) * kBlock;
      last_shift[e] = at >= tail ? at : 0;
    }
  };
  auto set_shift = [&]() {
#pragma unroll
    for (int e = 0; e < 2; ++e) shift[e] = f_stage == f_last ? last_shift[e] : 0u;
  };
  // On to the next stage: of this item without a branch, then of the next one.
  auto advance = [&]() {
    const bool more = f_stage < f_last;
    f_more = more;
    f_stage += more ? 1 : 0;
    ga += more ? kTileStage : 0;
    gb += more ? kTileStage : 0;
    f_scales = more && (f_stage & 1) == 0;
    f_pair = f_scales ? (f_pair + 1 == S ? 0 : f_pair + 1) : f_pair;
#pragma unroll
    for (int j = 0; j < Tile::kScaleLoads; ++j)
      gs[j] += !f_scales ? 0 : (j * Tile::kWaves + wave) * 64 < Tile::kRowsA ? p.step_as : p.step_ws;
    set_shift();
  };
  auto next_item = [&]() {
    if (f_more || f_item + (int)gridDim.x >= items) return;
    f_item += (int)gridDim.x;
    f_scales = true;
    f_pair = f_pair + 1 == S ? 0 : f_pair + 1;
    open();
    set_shift();
  };
  auto load = [&](int slot, int j) {
    if (j < Tile::kLoadsA)
      dma_block_at(ga, off[j] - shift[j & 1], mine_a + slot * Tile::kStage + j * kBlockBytes);
    else
      dma_block_at(gb, off[j] - shift[(j - Tile::kLoadsA) & 1],
                   mine_b + slot * Tile::kStage + (j - Tile::kLoadsA) * kBlockBytes);
  };
  auto load_scales = [&]() {
    if (!f_scales) return;
#pragma unroll
    for (int j = 0; j < Tile::kScaleLoads; ++j)
      if ((j + 1) * Tile::kWaves <= Tile::kScaleBlocks || j * Tile::kWaves + wave < Tile::kScaleBlocks)
        dma_block_at(gs[j], scale_off[j], scale_base + f_pair * Tile::kScaleSlot + j * Tile::kWaves * kBlockBytes);
  };
  // Row 32 i + li of a wave's rows: (r >> 1) & 7 is (li >> 1) & 7 for every i.
  const uint8_t* frag_a = &ring[0][0] + (wm * FM * 32 + li) * kTileStage;
  const uint8_t* frag_b = &ring[0][0] + (Tile::kRowsA + wn * FN * 32 + li) * kTileStage;
  const uint8_t* scale_a = &scale_ring[0][0] + (wm * FM * 32 + li) * 16;
  const uint8_t* scale_b = &scale_ring[0][0] + (Tile::kRowsA + wn * FN * 32 + li) * 16;
  auto read = [&](const uint8_t* row, int t) {
    return *reinterpret_cast<const u32x4*>(row + ((2 * t + lh) ^ ((li >> 1) & 7)) * kBlock);
  };

  open();
  set_shift();
  for (int i = 0; i < S; ++i) {
    load_scales();
#pragma unroll
    for (int j = 0; j < Tile::kLoads; ++j) load(i, j);
    if (i < S - 1) {
      advance();
      next_item();
    }
  }
  wait_vmcnt<(S - 1) * Tile::kLoads>();
  __syncthreads();
  u32x4 fa[2][FM], fb[2][FN];
  uint32_t sa[FM], sb[FN];
  u32x2 ra[FM], rb[FN];   // a stage's scales as read: eight a row, every second one this half's
  auto read_scales = [&](int f, int pair, int stage) {
    const int at = pair * Tile::kScaleSlot + (stage & 1) * 8;
    if (f < FN) rb[f] = *reinterpret_cast<const u32x2*>(scale_b + at + f * 32 * 16);
    else ra[f - FN] = *reinterpret_cast<const u32x2*>(scale_a + at + (f - FN) * 32 * 16);
  };
  auto pick_scales = [&]() {
    const uint32_t half = 0x06040200u + 0x01010101u * lh;
#pragma unroll
    for (int i = 0; i < FM; ++i) sa[i] = __builtin_amdgcn_perm(ra[i][1], ra[i][0], half);
#pragma unroll
    for (int j = 0; j < FN; ++j) sb[j] = __builtin_amdgcn_perm(rb[j][1], rb[j][0], half);
  };

  f32x16 acc[FM][FN];
  // The MFMAs of step T on its fragments, with the reads of the next step's
  // (`ahead` is its slot) and, in the last step, the loads into `slot`. W is
  // the first operand: a lane then holds four neighbouring columns of C's row.
  auto step = [&](auto T, int slot, int ahead, int pair, int stage) {
    constexpr int t = decltype(T)::value;
    u32x4(&a)[FM] = fa[t & 1];
    u32x4(&b)[FN] = fb[t & 1];
    u32x4(&na)[FM] = fa[(t & 1) ^ 1];
    u32x4(&nb)[FN] = fb[(t & 1) ^ 1];
    const uint8_t* next_a = frag_a + ahead * Tile::kStage;
    const uint8_t* next_b = frag_b + ahead * Tile::kStage;
    constexpr int kBlocks = FM * FN, kReads = FM + FN;
#pragma unroll
    for (int at = 0; at < kBlocks; ++at) {
      const int i = at / FN, j = at % FN;
      acc[i][j] = mx_mma<t>(b[j], a[i], acc[i][j], sb[j], sa[i]);
#pragma unroll
      for (int f = at * 3; f < (at + 1) * 3 && f < kReads; ++f) {
        if (f < FN) nb[f] = read(next_b + f * 32 * kTileStage, (t + 1) & 3);
        else na[f - FN] = read(next_a + (f - FN) * 32 * kTileStage, (t + 1) & 3);
      }
      if constexpr (t == 3) {
#pragma unroll
        for (int f = (at - 2) * 3; f < (at - 1) * 3; ++f)
          if (f >= 0 && f < kReads) read_scales(f, pair, stage);
#pragma unroll
        for (int l = at * Tile::kLoads / kBlocks; l < (at + 1) * Tile::kLoads / kBlocks; ++l)
          load(slot, l);
      }
      if constexpr (t == 2) {
        if (at == 3) advance();
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  auto keep_sums = [&]() {
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) keep_sum<Tile::kWaves * PER_CU == 4>(acc[i][j]);
  };

  constexpr int kStores = OUT == 2 ? 4 * FM * FN : 4 * FM;   // of a wave's whole part of C
  bool behind = false;   // the last item's stores are, all of them, under way behind this stage's loads
  int slot = 0, pair = 0;
  for (int item = (int)blockIdx.x; item < items; item += (int)gridDim.x) {
    int tm, tn, split;
    tile_item(p, item, items, tm, tn, split);
    const int first = split * per, count = min(per, p.steps - first);
    // The last stage's scales inside K, of four blocks of this half.
    const int inside = ((p.bytes - (first + count - 1) * kTileStage) / kBlock - lh + 1) >> 1;
    const uint32_t last_mask = inside >= 4 ? ~0u : (1u << (8 * inside)) - 1;
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
      fa[0][i] = read(frag_a + slot * Tile::kStage + i * 32 * kTileStage, 0);
#pragma unroll
    for (int j = 0; j < FN; ++j)
      fb[0][j] = read(frag_b + slot * Tile::kStage + j * 32 * kTileStage, 0);
#pragma unroll
    for (int f = 0; f < FM + FN; ++f) read_scales(f, pair, 0);
    for (int ks = 0; ks < count; ++ks) {
      const int next = slot + 1 == S ? 0 : slot + 1;
      pick_scales();
      if (ks == count - 1) {
#pragma unroll
        for (int i = 0; i < FM; ++i) sa[i] &= last_mask;
#pragma unroll
        for (int j = 0; j < FN; ++j) sb[j] &= last_mask;
      }
      step(Step<0>{}, slot, slot, 0, 0);
      step(Step<1>{}, slot, slot, 0, 0);
      step(Step<2>{}, slot, slot, 0, 0);
      keep_sums();
      next_item();
      if (behind)
        wait_vmcnt<(S - 2) * Tile::kLoads + kStores>();
      else
        wait_vmcnt<(S - 2) * Tile::kLoads>();
      behind = false;
      wait_lgkmcnt0();
      __syncthreads();
      // Every second stage, and an item's last, ends its pair of scales.
      if ((ks & 1) == 1 || ks == count - 1) pair = pair + 1 == S ? 0 : pair + 1;
      load_scales();
      step(Step<3>{}, slot, next, pair, ks + 1);   // after the last stage its reads are not used
      keep_sums();
      slot = next;
    }

    __builtin_amdgcn_sched_barrier(0);
    // Lane l holds row l % 32 and columns 8 (e / 4) + 4 (l / 32) + e % 4 of a
    // block. Rows of 128 bytes go, 16 at a time, through the wave's own staging
    // buffer, its 16-byte chunks placed as the ring's, and leave as whole cache
    // lines, while the next item's first stages arrive.
    // The lane is made anew for the compiler, which would else compute the
    // epilogue's addresses before the loop and spill them.
    int el = lane;
    asm volatile("" : "+v"(el));
    const int eli = el & 15, ehalf = (el >> 4) & 1, elh = el >> 5;
    uint8_t* mid = &staging[wave][0];
    // Unsigned: the last tiles may end past 2^31.
    const uint32_t row0 = (uint32_t)tm * Tile::kRowsA + wm * FM * 32;
    const uint32_t col0 = (uint32_t)tn * Tile::kRowsB + wn * FN * 32;
    const int wrow = eli * 128, wswz = (eli >> 1) & 7;
    behind = p.splits == 1 && row0 + FM * 32 <= (uint32_t)p.M && col0 + FN * 32 <= (uint32_t)p.N;
    auto flush = [&](uint8_t* out, int64_t pitch, uint32_t row, uint32_t col, int per_chunk) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int r = 8 * k + (el >> 3), c = (el & 7) ^ ((r >> 1) & 7);
        const u32x4 v = *reinterpret_cast<const u32x4*>(mid + r * 128 + (el & 7) * 16);
        if (row + r < (uint32_t)p.M && col + c * per_chunk < (uint32_t)p.N)
          __builtin_nontemporal_store(v, reinterpret_cast<u32x4*>(out + (row + r) * pitch + (int64_t)col * (16 / per_chunk) + c * 16));
      }
    };
    auto block32 = [&](int i, int j, uint8_t* out, int64_t pitch) {
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        if (ehalf == half)
#pragma unroll
          for (int q = 0; q < 4; ++q)
            *reinterpret_cast<f32x4*>(mid + wrow + ((2 * q + elh) ^ wswz) * 16) =
                f32x4{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
        flush(out, pitch, row0 + 32 * i + 16 * half, col0 + 32 * j, 4);
      }
    };
    if (p.splits > 1 || OUT == 2) {
      uint8_t* out = static_cast<uint8_t*>(p.C);
      int64_t pitch = p.ldc * 4;
      if (p.splits > 1) {
        out = reinterpret_cast<uint8_t*>(p.partials + (int64_t)split * p.M * p.N);
        pitch = (int64_t)p.N * 4;
      }
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) block32(i, j, out, pitch);
      continue;
    }
    if constexpr (OUT != 2) {
      static_assert(FN == 2, "a wave's row of 16-bit values is 128 bytes");
      using T = typename Out16<OUT>::type;
#pragma unroll
      for (int i = 0; i < FM; ++i) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          if (ehalf == half)
#pragma unroll
            for (int j = 0; j < FN; ++j)
#pragma unroll
              for (int q = 0; q < 4; ++q)
                *reinterpret_cast<u32x2*>(mid + wrow + ((4 * j + q) ^ wswz) * 16 + elh * 8) =
                    u32x2{Pair<T>::pack(acc[i][j][4 * q], acc[i][j][4 * q + 1]),
                          Pair<T>::pack(acc[i][j][4 * q + 2], acc[i][j][4 * q + 3])};
          flush(static_cast<uint8_t*>(p.C), p.ldc * 2, row0 + 32 * i + 16 * half, col0, 8);
        }
      }
    }
  }
  wait_vmcnt<0>();
}

// The scales of both operands as the tile kernel reads them fastest: the 16 bytes of
// each row and pair of stages, all rows' of one pair side by side. In rows of their
// own such 16 bytes cost the tile kernel a request for a cache line each, half as many
// again as the codes'. A workgroup turns 64 rows of 16 pairs over in LDS, so that both
// sides are whole lines.
__global__ void __launch_bounds__(256) mx_pack_scales_kernel(MxPackParams p) {
  __shared__ u32x4 part[16][64 + 1];
  const bool of_a = (int)blockIdx.x < p.blocks_a;
  const int rows = of_a ? p.rows_a : p.rows_w;
  const int row0 = (of_a ? (int)blockIdx.x : (int)blockIdx.x - p.blocks_a) * 64;
  const int pair0 = (int)blockIdx.y * 16;
  const uint8_t* src = of_a ? p.a : p.w;
  const int64_t ld = of_a ? p.ld_a : p.ld_w;
  const int pair = (int)(threadIdx.x & 15), first = (int)(threadIdx.x >> 4);
  u32x4 v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    v[i] = *reinterpret_cast<const u32x4*>(src + min(row0 + first + 16 * i, rows - 1) * ld +
                                           min(pair0 + pair, p.pairs - 1) * 16);
#pragma unroll
  for (int i = 0; i < 4; ++i) part[pair][first + 16 * i] = v[i];
  __syncthreads();
  const int lane = (int)(threadIdx.x & 63), wave = (int)(threadIdx.x >> 6);
  u32x4* dst = reinterpret_cast<u32x4*>(of_a ? p.to_a : p.to_w) + row0 + lane;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int q = wave + 4 * i;
    if (row0 + lane < rows && pair0 + q < p.pairs) dst[(int64_t)(pair0 + q) * rows] = part[q][lane];
  }
}

// Sum of the splits' partial products in split order, rounded: four columns a
// thread, four splits' loads together.
template <int OUT>
__global__ void __launch_bounds__(256) gemm_mx_join_kernel(MxGemmParams p) {
  const int quads = p.N >> 2;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= (int64_t)p.M * quads) return;
  const int m = (int)(i / quads), n = (int)(i % quads) * 4;
  const int64_t plane = (int64_t)p.M * p.N;
  const float* src = p.partials + (int64_t)m * p.N + n;
  f32x4 v = *reinterpret_cast<const f32x4*>(src);
#pragma unroll 4
  for (int s = 1; s < p.splits; ++s) v += *reinterpret_cast<const f32x4*>(src + s * plane);
  store4<OUT>(p.C, (int64_t)m * p.ldc + n, v);
}

// ---------------------------------------------------------------------------
// Choice of kernel.
// ---------------------------------------------------------------------------
enum MxKind { kVec, kRows, kTile128, kTile128Pair, kTile192, kTile256 };

struct MxPlan {
  MxKind kind;
  int tiles_m, tiles_n, splits, steps;
  bool wide;     // kRows: 64 columns
  bool packed;   // tile kernels: the scales are laid out anew
};

MxPlan mx_plan(int64_t M, int64_t N, int64_t bytes) {
  MxPlan c{kVec, 0, 0, 1, 0, false, false};
  // Turning codes into pairs makes the vector units the bound from two rows on: one row
  // of 512 x 8192 takes 3.9 us there and 6.1 in the few-row kernel, of 28672 x 8192 21.3 and
  // 24; two rows of 1024 x 16384 5.7 and 7.5, but of 4096 x 4096 5.8 and 5.2, of 14336 x 4096
  // 9.5 and 8.2.
  if (M == 1 || (M == 2 && 2 * bytes > N)) return c;
  // The few-row kernel, also for more rows, while its tiles all run at once: of 64 x
  // 32 where K is not long, and of 64 x 64. 128 x 4096 x 4096 takes 7.4 us and in the
  // large tiles 13.4, 256 x 4096 x 4096 9.4 and 13.4, 300 x 3000 x 2016 8.1 and 8.4;
  // 128 x 8192 x 14336 26.1 and 24.6, and with more tiles than CUs 64 x 28672 x 8192
  // 33.1 and 24.7, 16 x 28672 x 8192 25.0 and 23.6.
  const int64_t tall = (M + 63) / 64;
  const bool few32 = tall * ((N + 31) / 32) <= 256 && bytes <= 8192;
  const bool few64 = tall * ((N + 63) / 64) <= 256 && (M <= 64 || bytes <= 4096);
  if (few32 || few64) {
    c.kind = kRows;
    c.tiles_m = ceil_div(M, 64);
    // 64 columns for up to 64 rows too where tiles of 32 would not all run at once: 24 x
    // 8200 x 8192 takes 12.3 us so and 14.9 in 32, 48 x 11008 x 4096 9.9 and 12.5, 64 x
    // 10240 x 16384 29.5 and 38.9; 24 x 8192 x 8192 12.2 and 10.2, 64 x 8192 x 8192 16.5
    // and 12.7.
    c.wide = M <= 64 ? N > 256 * 32 : !few32;
    c.tiles_n = ceil_div(N, c.wide ? 64 : 32);
    c.steps = ceil_div(bytes, kRowsStage);
    const int tiles = c.tiles_m * c.tiles_n;
    // K is split where that gives idle CUs enough stages to pay for the join: 16 x
    // 4096 x 14336 takes 10.2 us in two parts and 11.4 whole, 40 x 2048 x 16384 10.2 in
    // four and 12.1 in two; 32 x 4096 x 8192 8.9 in two and 8.8 whole, 8 x 4096 x 4096
    // 6.5 and 5.2.
    const int most = tiles < 96 ? 256 / tiles : tiles <= 128 && c.steps >= 14 ? 2 : 1;
    c.splits = c.steps >= 8 ? shares(c.steps, most, 2) : 1;
    return c;
  }
  // The tile kernels: of all tile shapes and splits of K, the least estimate of
  // time. With every CU at work a workgroup takes so many us a stage, and so many
  // more a tile (measured from K = 1024 to 8192): the larger tiles fetch less for each
  // product, and their last round leaves more CUs idle. Two of 128 x 128 share a CU
  // where there are more than 256 of them. Partial products cost 2 us, and 8 bytes
  // each at 8 TB/s. 1500 x 8192 x 2048 takes 18.4 us in tiles of 256 x 256 (20.3 in
  // pairs of 128 x 128), 2048 x 4096 x 4096 23.8 in those pairs (25.8 in 256 x 256),
  // 1000 x 5000 x 4128 24.1 in 192 x 128 (25.4), 3000 x 1000 x 8192 23.5 in 128 x 128
  // with a CU each (25.5).
  struct Shape {
    MxKind kind;
    int rows, cols, places, most;   // most: splits of K
    float us, tile_us;
  };
  static constexpr Shape kShapes[] = {{kTile256, 256, 256, 256, 1, 1.8f, 4.5f},
                                      {kTile192, 192, 128, 256, 8, 1.0f, 2.f},
                                      {kTile128, 128, 128, 256, 16, 0.62f, 2.5f},
                                      {kTile128Pair, 128, 128, 512, 16, 1.16f, 2.f}};
  c.steps = ceil_div(bytes, kTileStage);
  float best = 0.f;
  for (const Shape& sh : kShapes) {
    const int tiles_m = ceil_div(M, sh.rows), tiles_n = ceil_div(N, sh.cols);
    const int64_t tiles = (int64_t)tiles_m * tiles_n;
    for (int want = 1; want <= sh.most; ++want) {
      // Shares of whole pairs of stages.
      const int splits = shares(ceil_div(c.steps, 2), want, 2);
      if (splits != want) continue;
      const int64_t rounds = (tiles * splits + sh.places - 1) / sh.places;
      const bool alone = sh.kind == kTile128Pair && tiles * splits <= 256;
      float t = (float)rounds * ((float)ceil_div(c.steps, splits) * (alone ? 0.72f : sh.us) +
                                 (alone ? 1.f : sh.tile_us));
      if (splits > 1) t += 2.f + (float)splits * (float)M * (float)N * 1e-6f;
      if (best == 0.f || t < best) {
        best = t;
        c.kind = sh.kind;
        c.tiles_m = tiles_m;
        c.tiles_n = tiles_n;
        c.splits = splits;
        // Laying the scales out anew pays from some 64 stages a workgroup on. Operands from
        // memory: 8192^3 (128) takes 260 us without and 248 with it, 4096 x 8192 x 8192 (64)
        // 134 and 130, 4096 x 8192 x 4096 (32) 77.0 and 75.4, 4096^3 (16) 39.8 and 40.6; from
        // the last-level cache 244 and 240, 126 and 125, 71.0 and 71.2, 40.5 and 41.1.
        c.packed = sh.kind == kTile256 && rounds * c.steps >= 64 && M + N < int64_t(1) << 29;
      }
      if (tiles * splits >= sh.places) break;
    }
  }
  return c;
}

template <int MM, int LPR, int OUT>
hipError_t launch_vec(const MxGemmParams& p, hipStream_t stream) {
  constexpr int kRows = kVecRows * (64 / LPR);
  const int slices = LPR < 64 ? 1 : ceil_div(p.bytes, kVecSlice);
  const int waves = ceil_div(slices, ceil_div(slices, kVecWaves));
  hipLaunchKernelGGL((gemv_mx_kernel<MM, LPR, OUT>), long_grid(((int64_t)p.N + kRows - 1) / kRows),
                     dim3(64 * waves), 0, stream, p);
  return hipGetLastError();
}

// As many lanes a row as K has 16-byte chunks, up to a wave.
template <int MM, int OUT>
hipError_t launch_vec_k(const MxGemmParams& p, hipStream_t stream) {
  if (p.bytes <= 16 * kBlock) return launch_vec<MM, 16, OUT>(p, stream);
  if (p.bytes <= 32 * kBlock) return launch_vec<MM, 32, OUT>(p, stream);
  return launch_vec<MM, 64, OUT>(p, stream);
}

template <int OUT>
hipError_t launch_out(const MxGemmParams& p, MxKind kind, bool wide, hipStream_t stream) {
  const int items = p.tiles_m * p.tiles_n * p.splits;
  switch (kind) {
    case kVec:
      return p.M == 1 ? launch_vec_k<1, OUT>(p, stream) : launch_vec_k<2, OUT>(p, stream);
    case kRows: {
      void (*k)(MxGemmParams) =
          p.M <= 32 ? (wide ? gemm_mx_rows_kernel<1, 2, OUT> : gemm_mx_rows_kernel<1, 1, OUT>)
                    : (wide ? gemm_mx_rows_kernel<2, 2, OUT> : gemm_mx_rows_kernel<2, 1, OUT>);
      hipLaunchKernelGGL(k, long_grid(items), dim3(512), 0, stream, p);
      break;
    }
    case kTile128:
      hipLaunchKernelGGL((gemm_mx_tile_kernel<2, 2, 2, 2, 4, 1, OUT>),
                         dim3(items < 256 ? items : 256), dim3(256), 0, stream, p);
      break;
    case kTile128Pair:
      hipLaunchKernelGGL((gemm_mx_tile_kernel<2, 2, 2, 2, 2, 2, OUT>),
                         dim3(items < 512 ? items : 512), dim3(256), 0, stream, p);
      break;
    case kTile192:
      hipLaunchKernelGGL((gemm_mx_tile_kernel<3, 2, 2, 2, 3, 1, OUT>),
                         dim3(items < 256 ? items : 256), dim3(256), 0, stream, p);
      break;
    default:
      hipLaunchKernelGGL((gemm_mx_tile_kernel<4, 2, 2, 4, 2, 1, OUT>),
                         dim3(items < 256 ? items : 256), dim3(512), 0, stream, p);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.splits == 1) return e;
  const int64_t quads = (int64_t)p.M * (p.N / 4);
  hipLaunchKernelGGL(gemm_mx_join_kernel<OUT>, dim3((unsigned)((quads + 255) / 256)), dim3(256), 0,
                     stream, p);
  return hipGetLastError();
}

}  // namespace

// Bytes of an operand's packed scales.
int64_t packed_bytes(int64_t rows, int64_t bytes) { return rows * ((bytes + 2 * kTileStage - 1) / (2 * kTileStage)) * 16; }

int64_t gemm_mx_partials(int64_t M, int64_t N, int64_t K) {
  const MxPlan c = mx_plan(M, N, K / 2);
  int64_t n = c.splits > 1 ? (int64_t)c.splits * M * N : 0;
  if (c.packed) n += (packed_bytes(M, K / 2) + packed_bytes(N, K / 2)) / 4;
  return n;
}

hipError_t launch_gemm_mx(MxGemmParams p, int out_type, hipStream_t stream) {
  const MxPlan c = mx_plan(p.M, p.N, p.bytes);
  p.tiles_m = c.tiles_m;
  p.tiles_n = c.tiles_n;
  p.splits = c.splits;
  p.steps = c.steps;
  p.step_as = p.step_ws = 16;
  if (c.packed) {
    MxPackParams q{};
    q.a = p.a_scales;
    q.w = p.w_scales;
    q.to_a = reinterpret_cast<uint8_t*>(p.partials);
    q.to_w = q.to_a + packed_bytes(p.M, p.bytes);
    q.ld_a = p.ld_as;
    q.ld_w = p.ld_ws;
    q.rows_a = p.M;
    q.rows_w = p.N;
    q.blocks_a = ceil_div(p.M, 64);
    q.pairs = ceil_div(p.bytes, 2 * kTileStage);
    hipLaunchKernelGGL(mx_pack_scales_kernel, dim3(q.blocks_a + ceil_div(p.N, 64), ceil_div(q.pairs, 16)),
                       dim3(256), 0, stream, q);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    p.a_scales = q.to_a;
    p.w_scales = q.to_w;
    p.ld_as = p.ld_ws = 16;
    p.step_as = (int64_t)p.M * 16;
    p.step_ws = (int64_t)p.N * 16;
    p.partials = reinterpret_cast<float*>(q.to_w + packed_bytes(p.N, p.bytes));
  }
  if (out_type == 0) return launch_out<0>(p, c.kind, c.wide, stream);
  if (out_type == 1) return launch_out<1>(p, c.kind, c.wide, stream);
  return launch_out<2>(p, c.kind, c.wide, stream);
}

}  // namespace pipe
