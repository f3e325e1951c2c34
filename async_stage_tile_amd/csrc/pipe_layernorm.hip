// Layer norm with the residual's addition and a 16-bit, e4m3 or microscaled 4-bit
// output, and its gradient.
//
// Forward: h = x + residual (rounded to 16 bits), m = mean(h), r = rsqrt(mean((h -
// m)^2) + eps), y = (h - m) r w + b. A row is read once and stays in registers, as
// fp32 values (the packed 16 bits, unpacked in every turn, made it bound by the
// vector units). The mean's rounding matters
// where it is much larger than the deviations, so the sums of the second turn
// correct it: with m0 the rounded mean, d = h - m0 and e = mean(d),
// mean((h - m)^2) = mean(d^2) - e^2 and y = (d - e) r w + b; d is exact or nearly
// so, and e is tiny beside the deviations.
//
// Rows of finite values whose sum of d^2 passes fp32's range (bf16 alone holds such, a
// mask's lowest value among them) have r = 0: y = b (centre, past_range).
//
// Gradient: with u = (h - m) r and g = dy w, dx = r (g - mean(g) - u mean(g u))
// (+ dh), dweight = sum_rows dy u, dbias = sum_rows dy; mean(g u) = r (mean(g d) -
// e mean(g)). A workgroup walks rows in steps of the grid and keeps its columns'
// sums in fp32; the workgroups' sums meet in a second small kernel, in a fixed
// order.
//
// Both are bound by memory: some 12 and 20 fp32 operations an element.
#include <type_traits>

#include "pipe_mx.hpp"

namespace pipe {

namespace {

// The sums over a row of N values a lane, TPR threads a row in a workgroup of WG,
// in every thread of the row. Between two uses of one buffer lies a barrier that
// every wave reaches after its reads.
template <int TPR, int WG, int N>
struct RowSums {
  float v[N][WG / 64];
};
template <int TPR, int WG, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], RowSums<TPR, WG, N>& x) {
#pragma unroll
  for (int n = 0; n < N; ++n) v[n] = wave_sum(v[n]);
  constexpr int kRowWaves = TPR / 64;
  if constexpr (kRowWaves > 1) {
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int n = 0; n < N; ++n) x.v[n][wave] = v[n];
    }
    __syncthreads();
    const int first = wave / kRowWaves * kRowWaves;
#pragma unroll
    for (int n = 0; n < N; ++n) {
      v[n] = 0.f;
#pragma unroll
      for (int i = 0; i < kRowWaves; ++i) v[n] += x.v[n][first + i];
    }
  }
}

// The rounded mean, which the row's deviations are taken from. Where it or the values'
// sum may pass fp32's range it is taken to be 0: the values are so large there that
// their squares pass it, unless they are all the same. Below 2^119 no deviation becomes
// infinite (the largest bf16 value is 2^128 - 2^120). `unit`, by which the deviations are
// multiplied in their sum, is 1, or 0 there: the sum is then zero if all values are
// finite, else NaN. (The sum and 1 / N in its place would be a register more, which
// the gradient of rows wider than 16384 does not have.)
__device__ __forceinline__ float centre(float sum, float inv_n, float& unit) {
  const float mean = sum * inv_n;
  const bool fits = fabsf(mean) < 0x1p119f;
  unit = fits ? 1.f : 0.f;
  return fits ? mean : 0.f;
}
// Whether the squares of finite values' deviations pass fp32's range. Without a branch:
// with one the gradient of 8192 x 1024 takes 20.6 us instead of 18.0.
__device__ __forceinline__ bool past_range(float unit, float sum_d, float sum_dd) {
  return (sum_dd == INFINITY) & ((unit != 0.f) | (sum_d == 0.f));
}

template <class T>
__device__ __forceinline__ void unpack(const u32x4& v, float (&f)[8]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    f[2 * e] = Pair<T>::lo(v[e]);
    f[2 * e + 1] = Pair<T>::hi(v[e]);
  }
}

// Chunk c of a row: an unsigned offset from what may be a scalar base.
__device__ __forceinline__ const u32x4* chunk(const uint8_t* row, int c) {
  return reinterpret_cast<const u32x4*>(row + (uint32_t)c * 16u);
}
__device__ __forceinline__ u32x4* chunk(uint8_t* row, int c) {
  return reinterpret_cast<u32x4*>(row + (uint32_t)c * 16u);
}

// Rows that stay in the last-level cache (KEPT) are loaded through L2, others past it.
// With a residual 1021 x 5000 takes 8.6 us so and 11.1 past it, in a chain where each
// call reads the one before's y and h 8.7 and 9.7; 4096 x 4096 (134 MB) 21.8 and 22.2
// there, 2500 x 8192 (164 MB) 31.9 and 24.9, 8192 x 8192 95 and 82. The next call reads
// y and h: written past L2 the chain of 1021 x 5000 takes 10.5 us. The gradient's dx
// meets its reader later: of rows that stay it is written past L2 (1021 x 2048 10.0 us
// and 10.4, 4096 x 1024 11.4 and 12.5), of others not (8192 x 8192 96 us and 99).
constexpr int64_t kKeptBytes = 128 << 20;
bool kept(int64_t M, int64_t chunks, int sides) { return M * chunks * 16 * sides <= kKeptBytes; }
template <bool KEPT>
__device__ __forceinline__ u32x4 load_chunk(const u32x4* from) {
  if constexpr (KEPT) return *from;
  else return __builtin_nontemporal_load(from);
}

// One row per TPR threads, WG / TPR rows a workgroup; a thread holds CH chunks of
// 8 elements, chunk index t + TPR * i. OUT: 0 the type of x, 1 e4m3, 2 4-bit. 8192 x
// 8192 with residual takes 76 us with e4m3 output (6.2 TB/s), 73 with 4-bit and 81 with
// 16-bit output (6.6 TB/s, what a copy reaches); 1021 x 5000 8.6, where a launch and one
// trip to memory are a third; one row of 4096 2.9, the two alone.
template <class T, int TPR, int WG, int CH, bool RES, bool KEPT, int OUT>
__global__ void __launch_bounds__(WG) layernorm_kernel(LayerNormParams p) {
  constexpr int kRows = WG / TPR, kRowWaves = TPR / 64;
  __shared__ RowSums<TPR, WG, 1> first_sums;
  __shared__ RowSums<TPR, WG, 2> second_sums;
  __shared__ uint32_t tops[WG / 64];
  const int t = threadIdx.x % TPR;
  const int64_t row = long_block() * kRows + threadIdx.x / TPR;
  const bool live = row < p.M;
  const int64_t at = live ? row : p.M - 1;
  const uint8_t* x = p.x + at * p.ld_x;
  const uint8_t* res = p.residual + at * p.ld_residual;
  const auto inside = [&](int i) { return min(t + TPR * i, p.chunks - 1); };
  // Threads past the row's end hold its last chunk, and leave it out of every sum.
  u32x4 v[CH], a[RES ? CH : 1], wt[CH], bs[CH];
#pragma unroll
  for (int i = 0; i < CH; ++i) v[i] = load_chunk<KEPT>(chunk(x, inside(i)));
  if constexpr (RES) {
#pragma unroll
    for (int i = 0; i < CH; ++i) a[i] = load_chunk<KEPT>(chunk(res, inside(i)));
  }
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    wt[i] = *chunk(p.weight, inside(i));
    bs[i] = u32x4{0, 0, 0, 0};
    if (p.bias != nullptr) bs[i] = *chunk(p.bias, inside(i));
  }
  float f[CH][8];   // h, then its deviations, then y
  float sum[1] = {0.f};
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    if constexpr (RES) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        v[i][e] = Pair<T>::pack(Pair<T>::lo(v[i][e]) + Pair<T>::lo(a[i][e]),
                                Pair<T>::hi(v[i][e]) + Pair<T>::hi(a[i][e]));
    }
    unpack<T>(v[i], f[i]);
    if (t + TPR * i < p.chunks) {
#pragma unroll
      for (int e = 0; e < 8; ++e) sum[0] += f[i][e];
    }
  }
  row_sums(sum, first_sums);
  // The weight and the bias are here by now: the compiler would else load them where
  // they are used, behind the stores.
  keep_packed(wt);
  keep_packed(bs);
  if constexpr (RES) {
    if (live) {
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        const int c = t + TPR * i;
        if (c < p.chunks) *chunk(p.h + row * p.ld_h, c) = v[i];
      }
    }
  }
  float unit;
  const float mean = centre(sum[0], p.inv_n, unit);
  float dev[2] = {0.f, 0.f};
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    if (t + TPR * i < p.chunks) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        f[i][e] -= mean;
        dev[0] = fmaf(f[i][e], unit, dev[0]);
        dev[1] += f[i][e] * f[i][e];
      }
    }
  }
  row_sums(dev, second_sums);
  const float off = dev[0] * p.inv_n;
  float r = 1.0f / sqrtf(fmaxf(dev[1] * p.inv_n - off * off, 0.f) + p.eps);
  float shift = -off * r;
  if (past_range(unit, dev[0], dev[1])) r = shift = 0.f;
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    float wf[8], bf[8];
    unpack<T>(wt[i], wf);
    unpack<T>(bs[i], bf);
#pragma unroll
    for (int e = 0; e < 8; ++e) f[i][e] = fmaf(fmaf(f[i][e], r, shift), wf[e], bf[e]);
    if constexpr (OUT == 1) {
      if (t + TPR * i < p.chunks) {
#pragma unroll
        for (int e = 0; e < 8; ++e) top = max(top, abs_bits(f[i][e]));
      }
    }
  }
  float scale = 0.f;
  if constexpr (OUT == 1) {
    top = wave_max(top);
    if constexpr (kRowWaves > 1) {
      const int wave = threadIdx.x >> 6;
      if ((threadIdx.x & 63) == 0) tops[wave] = top;
      __syncthreads();
      const int first = wave / kRowWaves * kRowWaves;
#pragma unroll
      for (int i = 0; i < kRowWaves; ++i) top = max(top, tops[first + i]);
    }
    // A NaN or an infinity makes the row NaN.
    float m = __uint_as_float(top >= 0x7F800000u ? 0x7FC00000u : top);
    m = m < kAmaxMin ? kAmaxMin : m;
    scale = kE4m3Max / m;
    if (live && t == 0) reinterpret_cast<float*>(p.scales)[row] = m / kE4m3Max;
  }
  if (!live) return;
  uint8_t* out = p.y + row * p.ld_y;
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = t + TPR * i;
    float(&y)[8] = f[i];
    if constexpr (OUT == 1) {
      u32x2 o;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        int q = __builtin_amdgcn_cvt_pk_fp8_f32(y[4 * e] * scale, y[4 * e + 1] * scale, 0, false);
        o[e] = __builtin_amdgcn_cvt_pk_fp8_f32(y[4 * e + 2] * scale, y[4 * e + 3] * scale, q, true);
      }
      if (c < p.chunks) reinterpret_cast<u32x2*>(out)[c] = o;
    } else if constexpr (OUT == 2) {
      // A block of 32 is that of four lanes, all inside the row or all past it.
      const uint32_t exponent = mx_exponent(mx_top(y));
      const uint32_t codes = mx_codes(y, mx_scale(exponent));
      if (c < p.chunks) {
        reinterpret_cast<uint32_t*>(out)[c] = codes;
        if ((t & 3) == 0) p.scales[row * p.ld_scales + (c >> 2)] = (uint8_t)exponent;
      }
    } else {
      u32x4 o;
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = Pair<T>::pack(y[2 * e], y[2 * e + 1]);
      if (c < p.chunks) *chunk(out, c) = o;
    }
  }
}

template <class T, int TPR, int WG, int CH, bool RES, bool KEPT>
hipError_t launch_norm_shape(const LayerNormParams& p, int out, hipStream_t stream) {
  const int64_t wgs = (p.M + WG / TPR - 1) / (WG / TPR);
  void (*k)(LayerNormParams) = out == 2   ? layernorm_kernel<T, TPR, WG, CH, RES, KEPT, 2>
                               : out == 1 ? layernorm_kernel<T, TPR, WG, CH, RES, KEPT, 1>
                                          : layernorm_kernel<T, TPR, WG, CH, RES, KEPT, 0>;
  hipLaunchKernelGGL(k, long_grid(wgs), dim3(WG), 0, stream, p);
  return hipGetLastError();
}

// One or two chunks a thread where the workgroup's 1024 threads allow it: few values
// in a thread leave many waves to a CU, and short rows to many threads. 500 x 2048 with
// 4-bit output takes 3.8 us with 256 threads a row, 4.1 with 128 and 5.0 with 64 (16384
// x 2048 43.6, 43.5, 45.3), 2000 x 16384 43.7 with 1024 and 52.2 with 512, 8192 x 8192 with
// e4m3 output 76 with 512 and 84 with 256, 1021 x 5000 9.9 with 384 and 10.3 with 512.
template <class T, bool RES, bool KEPT>
hipError_t launch_norm_type(const LayerNormParams& p, int out, hipStream_t stream) {
  if (p.chunks <= 64) return launch_norm_shape<T, 64, 256, 1, RES, KEPT>(p, out, stream);
  if (p.chunks <= 128) return launch_norm_shape<T, 128, 256, 1, RES, KEPT>(p, out, stream);
  if (p.chunks <= 256) return launch_norm_shape<T, 256, 256, 1, RES, KEPT>(p, out, stream);
  if (p.chunks <= 512) return launch_norm_shape<T, 512, 512, 1, RES, KEPT>(p, out, stream);
  if (p.chunks <= 768) return launch_norm_shape<T, 384, 384, 2, RES, KEPT>(p, out, stream);
  if (p.chunks <= 1024) return launch_norm_shape<T, 512, 512, 2, RES, KEPT>(p, out, stream);
  if (p.chunks <= 2048) return launch_norm_shape<T, 1024, 1024, 2, RES, KEPT>(p, out, stream);
  return launch_norm_shape<T, 1024, 1024, 4, RES, KEPT>(p, out, stream);
}

// ---------------------------------------------------------------------------
// Gradient. 8192 x 8192 with the residual stream's gradient takes 96 us, 4.5 of them for
// the sum of the partials (5.6 TB/s; 105 with the values unpacked in every turn and 512
// workgroups' partials); 1021 x 2048 9.8, 2.5 for the sum: launches, one trip to memory,
// two exchanges.
//
// A workgroup that fills its CU's registers (1024 threads of 128, or 512 of 256 for rows
// wider than 16384) keeps the columns' sums of dy in LDS, each
// thread its own, and reads dh where it is used; with eight chunks a thread a row's
// loads go out only when the row ahead of it is done, and the weight's with them
// and, from the caches, once more.
// ---------------------------------------------------------------------------
template <class T, int TPR, int WG, int CH, bool RES, bool KEPT>
__global__ void __launch_bounds__(WG) layernorm_grad_kernel(LayerNormGradParams p) {
  constexpr int kRows = WG / TPR;
  constexpr bool kWide = CH == 8, kFull = WG == 1024 || kWide;
  __shared__ RowSums<TPR, WG, 2> first_sums;
  __shared__ RowSums<TPR, WG, 3> second_sums;
  __shared__ f32x4 bias_lds[kFull ? 2 * CH : 1][WG];
  const int t = threadIdx.x % TPR;
  const int sub = kRows == 1 ? 0 : threadIdx.x / TPR;
  u32x4 wt[CH];
  // Threads past the row's end hold its last chunk, and leave it out of every sum.
  const auto inside = [&](int i) { return min(t + TPR * i, p.chunks - 1); };
  float dw[CH][8], db[kFull ? 1 : CH][8];
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    if constexpr (!kWide) wt[i] = *chunk(p.weight, inside(i));
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      dw[i][e] = 0.f;
      if constexpr (!kFull) db[i][e] = 0.f;
    }
    if constexpr (kFull)
      bias_lds[2 * i][threadIdx.x] = bias_lds[2 * i + 1][threadIdx.x] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  // A row's loads go out before the row ahead of it is reduced. Past the last row
  // they take the last one again: a branch around them would make the compiler
  // wait for them with the row in use.
  // dh's loads go out a row ahead too, or with four chunks for each of 512 threads, which
  // have no registers for that, ahead of the row's sums.
  constexpr bool kTop = WG == 512 && CH == 4;
  constexpr int kHeld = RES && !kFull ? CH : 1;
  u32x4 s[kHeld], nh[CH], nd[CH], ns[kTop ? 1 : kHeld];
  const auto load = [&](int64_t row) {
    const int64_t at = row < p.M ? row : p.M - 1;
    const uint8_t* dy = p.dy + at * p.ld_dy;
    const uint8_t* x = p.x + at * p.ld_x;
    const uint8_t* dh = p.dh + at * p.ld_dh;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      if constexpr (kWide) wt[i] = *chunk(p.weight, inside(i));
      nh[i] = load_chunk<KEPT>(chunk(x, inside(i)));
      nd[i] = load_chunk<KEPT>(chunk(dy, inside(i)));
    }
    if constexpr (RES && !kFull && !kTop) {
#pragma unroll
      for (int i = 0; i < CH; ++i) ns[i] = load_chunk<KEPT>(chunk(dh, inside(i)));
    }
  };
  const int64_t step = (int64_t)gridDim.x * kRows;
  if constexpr (!kWide) load((int64_t)blockIdx.x * kRows + sub);
  for (int64_t base = (int64_t)blockIdx.x * kRows; base < p.M; base += step) {
    const int64_t row = base + sub;
    if constexpr (kWide) load(row);
    // The values in fp32, once; with eight chunks a thread, unpacked in every turn.
    float fv[kWide ? 1 : CH][8], gv[kWide ? 1 : CH][8];
    const auto values = [&](int i, float(&f)[8], float(&g)[8], float(&wf)[8]) {
      if constexpr (kWide) {
        unpack<T>(nh[i], f);
        unpack<T>(nd[i], g);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          f[e] = fv[i][e];
          g[e] = gv[i][e];
        }
      }
      unpack<T>(wt[i], wf);
    };
    if constexpr (!kWide) {
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        unpack<T>(nh[i], fv[i]);
        unpack<T>(nd[i], gv[i]);
        if constexpr (RES && !kFull && !kTop) s[i] = ns[i];
      }
      if constexpr (RES && kTop) {
        const uint8_t* dh = p.dh + (row < p.M ? row : p.M - 1) * p.ld_dh;
#pragma unroll
        for (int i = 0; i < CH; ++i) s[i] = load_chunk<KEPT>(chunk(dh, inside(i)));
      }
      load(row + step);
    }
    float one[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      float f[8], g[8], wf[8];
      values(i, f, g, wf);
      if (t + TPR * i < p.chunks) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          one[0] += f[e];
          one[1] += g[e] * wf[e];
        }
      }
      if constexpr (kFull) __builtin_amdgcn_sched_barrier(0);   // one chunk's values at a time
    }
    row_sums(one, first_sums);
    if constexpr (kWide) {
      keep_packed(nh);
      keep_packed(nd);
    }
    keep_packed(wt);
    float unit;
    const float mean = centre(one[0], p.inv_n, unit);
    float two[3] = {0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      if (t + TPR * i < p.chunks) {
        float f[8], g[8], wf[8];
        values(i, f, g, wf);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float v = f[e] - mean;
          if constexpr (!kWide) fv[i][e] = v;
          two[0] = fmaf(v, unit, two[0]);
          two[1] += v * v;
          two[2] += g[e] * wf[e] * v;
        }
      }
      if constexpr (kFull) __builtin_amdgcn_sched_barrier(0);   // one chunk's values at a time
    }
    row_sums(two, second_sums);
    if constexpr (kWide) {
      keep_packed(nh);
      keep_packed(nd);
    }
    keep_packed(wt);
    if (row < p.M) {
      float off = two[0] * p.inv_n;
      float r = 1.0f / sqrtf(fmaxf(two[1] * p.inv_n - off * off, 0.f) + p.eps);
      if (past_range(unit, two[0], two[1])) off = r = two[2] = 0.f;   // no gradient through u
      const float shift = -off * r;
      const float mean_g = one[1] * p.inv_n;
      const float along = (two[2] * p.inv_n - off * mean_g) * r;
      const float less = mean_g * r, tilt = along * r;
      // The address and the place made anew for the compiler, which would else keep
      // the values.
      const uint8_t* from = p.weight;
      int place = t;
      if constexpr (kWide) {
        asm volatile("" : "+s"(from));
        asm volatile("" : "+v"(place));
      }
      uint8_t* dx = p.dx + row * p.ld_dx;
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        const int c = place + TPR * i;
        float f[8], g[8], wf[8], o[8];
        if constexpr (kWide) wt[i] = *chunk(from, min(c, p.chunks - 1));
        values(i, f, g, wf);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float u = fmaf(kWide ? f[e] - mean : f[e], r, shift);
          o[e] = fmaf(g[e] * wf[e], r, -less) - u * tilt;
          dw[i][e] += g[e] * u;
          if constexpr (!kFull) db[i][e] += g[e];
        }
        if constexpr (kFull) {
          bias_lds[2 * i][threadIdx.x] += f32x4{g[0], g[1], g[2], g[3]};
          bias_lds[2 * i + 1][threadIdx.x] += f32x4{g[4], g[5], g[6], g[7]};
        }
        if constexpr (RES) {
          float sf[8];
          u32x4 stream = {0, 0, 0, 0};
          if constexpr (!kFull) stream = s[i];
          else stream = load_chunk<KEPT>(chunk(p.dh + row * p.ld_dh, min(c, p.chunks - 1)));
          unpack<T>(stream, sf);
#pragma unroll
          for (int e = 0; e < 8; ++e) o[e] += sf[e];
        }
        u32x4 packed;
#pragma unroll
        for (int e = 0; e < 4; ++e) packed[e] = Pair<T>::pack(o[2 * e], o[2 * e + 1]);
        if (c < p.chunks) {
          if constexpr (KEPT) __builtin_nontemporal_store(packed, chunk(dx, c));
          else *chunk(dx, c) = packed;
        }
        if constexpr (kFull) __builtin_amdgcn_sched_barrier(0);
      }
    }
  }
  f32x4* out_w = reinterpret_cast<f32x4*>(p.sum_weight + (int64_t)blockIdx.x * p.sum_stride);
  f32x4* out_b = reinterpret_cast<f32x4*>(p.sum_bias + (int64_t)blockIdx.x * p.sum_stride);
  const auto bias_sum = [&](int i, int half) {
    if constexpr (kFull) return bias_lds[2 * i + half][threadIdx.x];
    else return f32x4{db[i][4 * half], db[i][4 * half + 1], db[i][4 * half + 2], db[i][4 * half + 3]};
  };
  const auto weight_sum = [&](int i, int half) {
    return f32x4{dw[i][4 * half], dw[i][4 * half + 1], dw[i][4 * half + 2], dw[i][4 * half + 3]};
  };
  if constexpr (kRows == 1) {
    // The thread's place is made anew for the compiler, which would else keep the
    // columns through the loop, in scratch memory where registers are short.
    int at = t;
    asm volatile("" : "+v"(at));
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = at + TPR * i;
      if (c < p.chunks) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          out_w[2 * c + half] = weight_sum(i, half);
          out_b[2 * c + half] = bias_sum(i, half);
        }
      }
    }
  } else {
    // The rows in flight add up in LDS first, in order.
    __shared__ f32x4 sums[kRows][2 * CH * TPR];
    const auto add_up = [&](auto sum, f32x4* out) {
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        const int c = t + TPR * i;
        sums[sub][2 * c] = sum(i, 0);
        sums[sub][2 * c + 1] = sum(i, 1);
      }
      __syncthreads();
      for (int u = (int)threadIdx.x; u < 2 * p.chunks; u += WG) {
        f32x4 a = sums[0][u];
#pragma unroll
        for (int r = 1; r < kRows; ++r) a += sums[r][u];
        out[u] = a;
      }
    };
    add_up(weight_sum, out_w);
    __syncthreads();
    add_up(bias_sum, out_b);
  }
}

// dweight and dbias: the partials' sums, rows of 2 n floats of which the first n
// are dweight's. A workgroup takes 32 columns (8 lanes of four) and 32 interleaved
// sets of partials, each summed in order; then the 8 sets of a wave, then the waves.
__global__ void __launch_bounds__(256) layernorm_columns_kernel(const float* __restrict__ partials,
                                                                float* __restrict__ dweight,
                                                                float* __restrict__ dbias, int count,
                                                                int n) {
  __shared__ f32x4 part[4][8];
  const int lane = threadIdx.x & 7, set = threadIdx.x >> 3;
  const int col = blockIdx.x * 32 + lane * 4;
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  if (col < 2 * n) {
    const float* src = partials + col;
#pragma unroll 8
    for (int i = set; i < count; i += 32)
      acc += *reinterpret_cast<const f32x4*>(src + (int64_t)i * 2 * n);
  }
#pragma unroll
  for (int step = 8; step < 64; step *= 2)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[e] += __shfl_xor(acc[e], step, 64);
  if ((set & 7) == 0) part[set >> 3][lane] = acc;
  __syncthreads();
  if (set == 0 && col < 2 * n) {
    acc = (part[0][lane] + part[1][lane]) + (part[2][lane] + part[3][lane]);
    *reinterpret_cast<f32x4*>(col < n ? dweight + col : dbias + (col - n)) = acc;
  }
}

// Each workgroup writes its partials, so there is at most one a CU, with several rows
// in flight (8192 x 8192 takes 96 us with 256 workgroups of two rows and 106 with 512 of
// one), which take equal numbers of turns, a multiple of 8 of them for the XCDs' sake.
// Few wide rows have a workgroup each: 16 x 4096 takes 6.0 us so, 6.8 in workgroups of
// two and 8.5 of four (256 x 4096 11.9 and 10.3), 16 x 8192 7.6 and 8.8. Some hundred of 4096 go four at a
// time: 1021 x 4096 14.7 us and 15.2 two at a time (256 10.4 and 10.3, 2048 20.7 and
// 19.1). Many short ones go eight at a time: 16384 x 512 16.8 us and 19.6 four at a time
// (3000 x 512 9.4 and 8.1). The threads and chunks of a row depend on its width alone, so
// that its dx does not depend on the other rows (64 threads of four chunks would take
// 48.8 us for 16384 x 2048, 256 of one take 50.4). A lone workgroup writes dweight and
// dbias itself.
struct GradShape {
  bool few, many;   // a workgroup for a row; more rows a workgroup than else
  int64_t grid;
};

GradShape grad_shape(int64_t M, int64_t chunks) {
  GradShape g{false, false, 0};
  int rows = 1;
  if (chunks <= 64) {
    g.many = M >= 4096;
    rows = g.many ? 8 : 4;
  } else if (chunks <= 128) {
    rows = 4;
  } else if (chunks <= 256) {
    rows = 2;
  } else if (chunks <= 1024) {
    g.few = M <= 64;
    g.many = chunks <= 512 && M > 256 && M < 2048;
    rows = g.few ? 1 : g.many ? 4 : 2;
  }
  const int64_t need = (M + rows - 1) / rows;
  const int64_t turns = (need + 255) / 256;
  g.grid = need <= 256 ? need : ((need + turns - 1) / turns + 7) / 8 * 8;
  return g;
}

template <class T, int TPR, int WG, int CH, bool KEPT>
hipError_t launch_grad_shape(const LayerNormGradParams& p, int64_t grid, hipStream_t stream) {
  void (*k)(LayerNormGradParams) = p.dh != nullptr ? layernorm_grad_kernel<T, TPR, WG, CH, true, KEPT>
                                                   : layernorm_grad_kernel<T, TPR, WG, CH, false, KEPT>;
  hipLaunchKernelGGL(k, dim3((unsigned)grid), dim3(WG), 0, stream, p);
  return hipGetLastError();
}

// The shapes for few rows, of up to 512 columns for fewer than 4096, and of four rows a
// workgroup have calls of 64 MiB at most: all stay in the cache.
template <class T, bool KEPT>
hipError_t launch_grad_type(const LayerNormGradParams& p, const GradShape& g, hipStream_t stream) {
  if (p.chunks <= 64)
    return g.many ? launch_grad_shape<T, 64, 512, 1, KEPT>(p, g.grid, stream)
                  : launch_grad_shape<T, 64, 256, 1, true>(p, g.grid, stream);
  if (p.chunks <= 128) return launch_grad_shape<T, 128, 512, 1, KEPT>(p, g.grid, stream);
  if (p.chunks <= 256) return launch_grad_shape<T, 256, 512, 1, KEPT>(p, g.grid, stream);
  if (p.chunks <= 512)
    return g.few    ? launch_grad_shape<T, 256, 256, 2, true>(p, g.grid, stream)
           : g.many ? launch_grad_shape<T, 256, 1024, 2, true>(p, g.grid, stream)
                    : launch_grad_shape<T, 256, 512, 2, KEPT>(p, g.grid, stream);
  if (p.chunks <= 1024)
    return g.few ? launch_grad_shape<T, 256, 256, 4, true>(p, g.grid, stream)
                 : launch_grad_shape<T, 256, 512, 4, KEPT>(p, g.grid, stream);
  if (p.chunks <= 2048) return launch_grad_shape<T, 512, 512, 4, KEPT>(p, g.grid, stream);
  return launch_grad_shape<T, 512, 512, 8, KEPT>(p, g.grid, stream);
}

}  // namespace

hipError_t launch_layernorm(const LayerNormParams& p, int type, int out, hipStream_t stream) {
  const bool res = p.residual != nullptr, keep = kept(p.M, p.chunks, res ? 4 : 2);
  const auto launch = [&](auto f16) {
    using T = std::conditional_t<decltype(f16)::value, _Float16, __bf16>;
    if (keep) return (res ? launch_norm_type<T, true, true> : launch_norm_type<T, false, true>)(p, out, stream);
    return (res ? launch_norm_type<T, true, false> : launch_norm_type<T, false, false>)(p, out, stream);
  };
  return type == 0 ? launch(std::false_type{}) : launch(std::true_type{});
}

int64_t layernorm_grad_partials(int64_t M, int64_t N) {
  const int64_t grid = grad_shape(M, N / 8).grid;
  return grid > 1 ? 2 * grid : 0;
}

hipError_t launch_layernorm_grad(LayerNormGradParams p, float* partials, float* dweight, float* dbias,
                                 int type, hipStream_t stream) {
  const GradShape g = grad_shape(p.M, p.chunks);
  const int n = p.chunks * 8;
  if (g.grid > 0) {
    p.sum_weight = g.grid == 1 ? dweight : partials;
    p.sum_bias = g.grid == 1 ? dbias : partials + n;
    p.sum_stride = 2 * (int64_t)n;
    const bool keep = kept(p.M, p.chunks, p.dh != nullptr ? 4 : 3);
    const hipError_t e =
        type == 0 ? (keep ? launch_grad_type<__bf16, true> : launch_grad_type<__bf16, false>)(p, g, stream)
                  : (keep ? launch_grad_type<_Float16, true> : launch_grad_type<_Float16, false>)(p, g, stream);
    if (e != hipSuccess || g.grid == 1) return e;
  }
  hipLaunchKernelGGL(layernorm_columns_kernel, dim3((2 * n + 31) / 32), dim3(256), 0, stream, partials,
                     dweight, dbias, (int)g.grid, n);
  return hipGetLastError();
}

}  // namespace pipe
