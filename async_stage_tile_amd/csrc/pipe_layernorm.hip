// Layer norm with the residual's addition and a 16-bit, e4m3 or microscaled 4-bit
// output, and its gradient.
//
// Forward: h = x + residual (rounded to 16 bits), m = mean(h), r = rsqrt(mean((h -
// m)^2) + eps), y = (h - m) r w + b. A row is read once and stays in registers,
// packed as the 16 bits that h is rounded to anyway. The mean's rounding matters
// where it is much larger than the deviations, so the sums of the second turn
// correct it: with m0 the rounded mean, d = h - m0 and e = mean(d),
// mean((h - m)^2) = mean(d^2) - e^2 and y = (d - e) r w + b; d is exact or nearly
// so, and e is tiny beside the deviations.
//
// Gradient: with u = (h - m) r and g = dy w, dx = r (g - mean(g) - u mean(g u))
// (+ dh), dweight = sum_rows dy u, dbias = sum_rows dy; mean(g u) = r (mean(g d) -
// e mean(g)). A workgroup walks rows in steps of the grid and keeps its columns'
// sums in fp32; the workgroups' sums meet in a second small kernel, in a fixed
// order.
//
// Both are bound by memory: some 12 and 20 fp32 operations an element.
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

// One row per TPR threads, WG / TPR rows a workgroup; a thread holds CH chunks of
// 8 elements, chunk index t + TPR * i. OUT: 0 the type of x, 1 e4m3, 2 4-bit.
template <class T, int TPR, int WG, int CH, bool RES, int OUT>
__global__ void __launch_bounds__(WG) layernorm_kernel(LayerNormParams p) {
  constexpr int kRows = WG / TPR, kRowWaves = TPR / 64;
  __shared__ RowSums<TPR, WG, 1> first_sums;
  __shared__ RowSums<TPR, WG, 2> second_sums;
  __shared__ uint32_t tops[WG / 64];
  const int t = threadIdx.x % TPR;
  const int64_t row = long_block() * kRows + threadIdx.x / TPR;
  const bool live = row < p.M;
  const int64_t at = live ? row : p.M - 1;
  const u32x4* x = reinterpret_cast<const u32x4*>(p.x + at * p.ld_x);
  const u32x4* res = reinterpret_cast<const u32x4*>(p.residual + at * p.ld_residual);
  const u32x4* w = reinterpret_cast<const u32x4*>(p.weight);
  const u32x4* b = reinterpret_cast<const u32x4*>(p.bias);
  u32x4 v[CH], a[RES ? CH : 1], wt[CH], bs[CH];
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = t + TPR * i;
    v[i] = u32x4{0, 0, 0, 0};
    if (c < p.chunks) v[i] = __builtin_nontemporal_load(x + c);
  }
  if constexpr (RES) {
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = t + TPR * i;
      a[i] = u32x4{0, 0, 0, 0};
      if (c < p.chunks) a[i] = __builtin_nontemporal_load(res + c);
    }
  }
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = t + TPR * i;
    wt[i] = bs[i] = u32x4{0, 0, 0, 0};
    if (c < p.chunks) wt[i] = w[c];
    if (b != nullptr && c < p.chunks) bs[i] = b[c];
  }
  float sum[1] = {0.f};
#pragma unroll
  for (int i = 0; i < CH; ++i) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if constexpr (RES)
        v[i][e] = Pair<T>::pack(Pair<T>::lo(v[i][e]) + Pair<T>::lo(a[i][e]),
                                Pair<T>::hi(v[i][e]) + Pair<T>::hi(a[i][e]));
      sum[0] += Pair<T>::lo(v[i][e]);
      sum[0] += Pair<T>::hi(v[i][e]);
    }
  }
  row_sums(sum, first_sums);
  keep_packed(v);
  if constexpr (RES) {
    if (live) {
      u32x4* h = reinterpret_cast<u32x4*>(p.h + row * p.ld_h);
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        const int c = t + TPR * i;
        if (c < p.chunks) h[c] = v[i];
      }
    }
  }
  const float mean = sum[0] * p.inv_n;
  float dev[2] = {0.f, 0.f};
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    if (t + TPR * i < p.chunks) {
      float f[8];
      unpack<T>(v[i], f);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float d = f[e] - mean;
        dev[0] += d;
        dev[1] += d * d;
      }
    }
  }
  row_sums(dev, second_sums);
  keep_packed(v);
  keep_packed(wt);
  keep_packed(bs);
  const float off = dev[0] * p.inv_n;
  const float r = 1.0f / sqrtf(fmaxf(dev[1] * p.inv_n - off * off, 0.f) + p.eps);
  const float shift = -off * r;
  const auto value = [&](int i, float(&y)[8]) {
    float f[8], wf[8], bf[8];
    unpack<T>(v[i], f);
    unpack<T>(wt[i], wf);
    unpack<T>(bs[i], bf);
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = fmaf(fmaf(f[e] - mean, r, shift), wf[e], bf[e]);
  };
  if constexpr (OUT == 1) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      float y[8];
      value(i, y);
      if (t + TPR * i < p.chunks)
#pragma unroll
        for (int e = 0; e < 8; ++e) top = max(top, abs_bits(y[e]));
    }
    top = wave_max(top);
    if constexpr (kRowWaves > 1) {
      const int wave = threadIdx.x >> 6;
      if ((threadIdx.x & 63) == 0) tops[wave] = top;
      __syncthreads();
      const int first = wave / kRowWaves * kRowWaves;
#pragma unroll
      for (int i = 0; i < kRowWaves; ++i) top = max(top, tops[first + i]);
    }
    if (!live) return;
    keep_packed(v);
    // A NaN or an infinity makes the row NaN.
    float m = __uint_as_float(top >= 0x7F800000u ? 0x7FC00000u : top);
    m = m < kAmaxMin ? kAmaxMin : m;
    const float inv = kE4m3Max / m;
    if (t == 0) reinterpret_cast<float*>(p.scales)[row] = m / kE4m3Max;
    u32x2* y8 = reinterpret_cast<u32x2*>(p.y + row * p.ld_y);
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = t + TPR * i;
      float y[8];
      value(i, y);
      u32x2 o;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        int q = __builtin_amdgcn_cvt_pk_fp8_f32(y[4 * e] * inv, y[4 * e + 1] * inv, 0, false);
        o[e] = __builtin_amdgcn_cvt_pk_fp8_f32(y[4 * e + 2] * inv, y[4 * e + 3] * inv, q, true);
      }
      if (c < p.chunks) y8[c] = o;
    }
  } else {
    if (!live) return;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = t + TPR * i;
      float y[8];
      value(i, y);
      if constexpr (OUT == 2) {
        // A block of 32 is that of four lanes, all inside the row or all past it.
        const uint32_t exponent = mx_exponent(mx_top(y));
        const uint32_t codes = mx_codes(y, mx_scale(exponent));
        if (c < p.chunks) {
          reinterpret_cast<uint32_t*>(p.y + row * p.ld_y)[c] = codes;
          if ((t & 3) == 0) p.scales[row * p.ld_scales + (c >> 2)] = (uint8_t)exponent;
        }
      } else {
        u32x4 o;
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = Pair<T>::pack(y[2 * e], y[2 * e + 1]);
        if (c < p.chunks) reinterpret_cast<u32x4*>(p.y + row * p.ld_y)[c] = o;
      }
    }
  }
}

template <class T, int TPR, int WG, int CH, bool RES>
hipError_t launch_norm_shape(const LayerNormParams& p, int out, hipStream_t stream) {
  const int64_t wgs = (p.M + WG / TPR - 1) / (WG / TPR);
  void (*k)(LayerNormParams) = out == 2   ? layernorm_kernel<T, TPR, WG, CH, RES, 2>
                               : out == 1 ? layernorm_kernel<T, TPR, WG, CH, RES, 1>
                                          : layernorm_kernel<T, TPR, WG, CH, RES, 0>;
  hipLaunchKernelGGL(k, long_grid(wgs), dim3(WG), 0, stream, p);
  return hipGetLastError();
}

// Rows of up to 2048 elements: one wave each, no exchange between waves. Wider
// rows: a workgroup each, of as many threads as leave each at most 4 chunks.
template <class T, bool RES>
hipError_t launch_norm_type(const LayerNormParams& p, int out, hipStream_t stream) {
  if (p.chunks <= 64) return launch_norm_shape<T, 64, 256, 1, RES>(p, out, stream);
  if (p.chunks <= 128) return launch_norm_shape<T, 64, 256, 2, RES>(p, out, stream);
  if (p.chunks <= 256) return launch_norm_shape<T, 64, 256, 4, RES>(p, out, stream);
  if (p.chunks <= 512) return launch_norm_shape<T, 256, 256, 2, RES>(p, out, stream);
  if (p.chunks <= 1024) return launch_norm_shape<T, 512, 512, 2, RES>(p, out, stream);
  if (p.chunks <= 2048) return launch_norm_shape<T, 512, 512, 4, RES>(p, out, stream);
  return launch_norm_shape<T, 1024, 1024, 4, RES>(p, out, stream);
}

// ---------------------------------------------------------------------------
// Gradient. A workgroup that fills its CU's registers (1024 threads of 128, or 512
// of 256 for rows wider than 16384) keeps the columns' sums of dy in LDS, each
// thread its own, and reads dh where it is used; with eight chunks a thread a row's
// loads go out only when the row ahead of it is done, and the weight's with them
// and, from the caches, once more.
// ---------------------------------------------------------------------------
template <class T, int TPR, int WG, int CH, bool RES>
__global__ void __launch_bounds__(WG) layernorm_grad_kernel(LayerNormGradParams p) {
  constexpr int kRows = WG / TPR;
  constexpr bool kWide = CH == 8, kFull = WG == 1024 || kWide;
  __shared__ RowSums<TPR, WG, 2> first_sums;
  __shared__ RowSums<TPR, WG, 3> second_sums;
  __shared__ f32x4 bias_lds[kFull ? 2 * CH : 1][WG];
  const int t = threadIdx.x % TPR;
  const int sub = kRows == 1 ? 0 : threadIdx.x / TPR;
  u32x4 wt[CH];
  const auto weight = [&](const uint8_t* from, int c) {
    return c < p.chunks ? *chunk(from, c) : u32x4{0, 0, 0, 0};
  };
  float dw[CH][8], db[kFull ? 1 : CH][8];
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = t + TPR * i;
    if constexpr (!kWide) wt[i] = weight(p.weight, c);
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
  constexpr int kHeld = RES && !kFull ? CH : 1;
  u32x4 h[CH], d[CH], s[kHeld], nh[CH], nd[CH], ns[kHeld];
  const auto load = [&](int64_t row) {
    const int64_t at = row < p.M ? row : p.M - 1;
    const uint8_t* dy = p.dy + at * p.ld_dy;
    const uint8_t* x = p.x + at * p.ld_x;
    const uint8_t* dh = p.dh + at * p.ld_dh;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = t + TPR * i;
      if constexpr (kWide) wt[i] = weight(p.weight, c);
      nh[i] = nd[i] = u32x4{0, 0, 0, 0};
      if (c < p.chunks) {
        nh[i] = __builtin_nontemporal_load(chunk(x, c));
        nd[i] = __builtin_nontemporal_load(chunk(dy, c));
      }
    }
    if constexpr (RES && !kFull) {
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        const int c = t + TPR * i;
        ns[i] = u32x4{0, 0, 0, 0};
        if (c < p.chunks) ns[i] = __builtin_nontemporal_load(chunk(dh, c));
      }
    }
  };
  const int64_t step = (int64_t)gridDim.x * kRows;
  if constexpr (!kWide) load((int64_t)blockIdx.x * kRows + sub);
  for (int64_t base = (int64_t)blockIdx.x * kRows; base < p.M; base += step) {
    const int64_t row = base + sub;
    if constexpr (kWide) load(row);
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      h[i] = nh[i];
      d[i] = nd[i];
      if constexpr (RES && !kFull) s[i] = ns[i];
    }
    if constexpr (!kWide) load(row + step);
    float one[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      float f[8], g[8], wf[8];
      unpack<T>(h[i], f);
      unpack<T>(d[i], g);
      unpack<T>(wt[i], wf);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        one[0] += f[e];
        one[1] += g[e] * wf[e];
      }
      if constexpr (kFull) __builtin_amdgcn_sched_barrier(0);   // one chunk's values at a time
    }
    row_sums(one, first_sums);
    keep_packed(h);
    keep_packed(d);
    keep_packed(wt);
    const float mean = one[0] * p.inv_n;
    float two[3] = {0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      if (t + TPR * i < p.chunks) {
        float f[8], g[8], wf[8];
        unpack<T>(h[i], f);
        unpack<T>(d[i], g);
        unpack<T>(wt[i], wf);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float v = f[e] - mean;
          two[0] += v;
          two[1] += v * v;
          two[2] += g[e] * wf[e] * v;
        }
      }
      if constexpr (kFull) __builtin_amdgcn_sched_barrier(0);   // one chunk's values at a time
    }
    row_sums(two, second_sums);
    keep_packed(h);
    keep_packed(d);
    keep_packed(wt);
    if (row < p.M) {
      const float off = two[0] * p.inv_n;
      const float r = 1.0f / sqrtf(fmaxf(two[1] * p.inv_n - off * off, 0.f) + p.eps);
      const float shift = -off * r;
      const float mean_g = one[1] * p.inv_n;
      const float along = (two[2] * p.inv_n - off * mean_g) * r;
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
        unpack<T>(h[i], f);
        unpack<T>(d[i], g);
        if constexpr (kWide) wt[i] = weight(from, c);
        unpack<T>(wt[i], wf);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float u = fmaf(f[e] - mean, r, shift);
          o[e] = r * (g[e] * wf[e] - mean_g - u * along);
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
          else if (c < p.chunks)
            stream = __builtin_nontemporal_load(chunk(p.dh + row * p.ld_dh, c));
          unpack<T>(stream, sf);
#pragma unroll
          for (int e = 0; e < 8; ++e) o[e] += sf[e];
        }
        u32x4 packed;
#pragma unroll
        for (int e = 0; e < 4; ++e) packed[e] = Pair<T>::pack(o[2 * e], o[2 * e + 1]);
        if (c < p.chunks) *chunk(dx, c) = packed;
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
// are dweight's. A workgroup takes 32 columns (8 threads of four) and 32
// interleaved sets of partials, each summed in order, then the 32 sums in order.
__global__ void __launch_bounds__(256) layernorm_columns_kernel(const float* __restrict__ partials,
                                                                float* __restrict__ dweight,
                                                                float* __restrict__ dbias, int count,
                                                                int n) {
  __shared__ f32x4 part[32][8];
  const int lane = threadIdx.x & 7, set = threadIdx.x >> 3;
  const int col = blockIdx.x * 32 + lane * 4;
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  if (col < 2 * n) {
    const float* src = partials + col;
#pragma unroll 4
    for (int i = set; i < count; i += 32)
      acc += *reinterpret_cast<const f32x4*>(src + (int64_t)i * 2 * n);
  }
  part[set][lane] = acc;
  __syncthreads();
  if (set == 0 && col < 2 * n) {
    acc = part[0][lane];
    for (int i = 1; i < 32; ++i) acc += part[i][lane];
    *reinterpret_cast<f32x4*>(col < n ? dweight + col : dbias + (col - n)) = acc;
  }
}

struct GradShape {
  bool tall;     // many rows: one row in flight a workgroup of 256 up to 8192 columns
  int64_t grid;
};

// Each workgroup writes a row of partials, so few rows want few workgroups with
// several rows in flight each, of 1024 threads. The few take equal numbers of
// turns, a multiple of 8 of them for the XCDs' sake. A lone workgroup writes
// dweight and dbias itself.
GradShape grad_shape(int64_t M, int64_t chunks) {
  GradShape g;
  g.tall = chunks <= 256 || M >= 4096;
  const int rows = chunks <= 256 ? 4 : g.tall ? 1 : chunks <= 512 ? 4 : chunks <= 1024 ? 2 : 1;
  const int64_t need = (M + rows - 1) / rows;
  const int64_t fill = g.tall && chunks <= 1024 ? 512 : 256;
  g.grid = need < fill ? need : fill;
  if (!g.tall && need > fill) {
    const int64_t turns = (need + fill - 1) / fill;
    g.grid = ((need + turns - 1) / turns + 7) / 8 * 8;
  }
  return g;
}

template <class T, int TPR, int WG, int CH>
hipError_t launch_grad_shape(const LayerNormGradParams& p, int64_t grid, hipStream_t stream) {
  void (*k)(LayerNormGradParams) = p.dh != nullptr ? layernorm_grad_kernel<T, TPR, WG, CH, true>
                                                   : layernorm_grad_kernel<T, TPR, WG, CH, false>;
  hipLaunchKernelGGL(k, dim3((unsigned)grid), dim3(WG), 0, stream, p);
  return hipGetLastError();
}

template <class T>
hipError_t launch_grad_type(const LayerNormGradParams& p, const GradShape& g, hipStream_t stream) {
  if (p.chunks <= 64) return launch_grad_shape<T, 64, 256, 1>(p, g.grid, stream);
  if (p.chunks <= 128) return launch_grad_shape<T, 64, 256, 2>(p, g.grid, stream);
  if (p.chunks <= 256) return launch_grad_shape<T, 64, 256, 4>(p, g.grid, stream);
  if (p.chunks <= 512)
    return g.tall ? launch_grad_shape<T, 256, 256, 2>(p, g.grid, stream)
                  : launch_grad_shape<T, 256, 1024, 2>(p, g.grid, stream);
  if (p.chunks <= 1024)
    return g.tall ? launch_grad_shape<T, 256, 256, 4>(p, g.grid, stream)
                  : launch_grad_shape<T, 512, 1024, 2>(p, g.grid, stream);
  if (p.chunks <= 2048) return launch_grad_shape<T, 1024, 1024, 2>(p, g.grid, stream);
  return launch_grad_shape<T, 512, 512, 8>(p, g.grid, stream);
}

}  // namespace

hipError_t launch_layernorm(const LayerNormParams& p, int type, int out, hipStream_t stream) {
  const bool res = p.residual != nullptr;
  if (type == 0)
    return res ? launch_norm_type<__bf16, true>(p, out, stream) : launch_norm_type<__bf16, false>(p, out, stream);
  return res ? launch_norm_type<_Float16, true>(p, out, stream)
             : launch_norm_type<_Float16, false>(p, out, stream);
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
    const hipError_t e = type == 0 ? launch_grad_type<__bf16>(p, g, stream)
                                   : launch_grad_type<_Float16>(p, g, stream);
    if (e != hipSuccess || g.grid == 1) return e;
  }
  hipLaunchKernelGGL(layernorm_columns_kernel, dim3((2 * n + 31) / 32), dim3(256), 0, stream, partials,
                     dweight, dbias, (int)g.grid, n);
  return hipGetLastError();
}

}  // namespace pipe
