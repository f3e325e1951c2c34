// RMS norm with the residual's addition and a 16-bit or e4m3 output, and its
// gradient.
//
// Forward: h = x + residual (rounded to 16 bits), r = rsqrt(mean(h^2) + eps),
// y = h r w. A row is read once: its h stays in registers, packed as the 16
// bits that it is rounded to anyway, until the row's sum of squares is known.
// The e4m3 output needs max|y| = r max|h w| before any value can be written;
// that maximum does not depend on r, so it is taken in the same pass as the sum
// and one exchange between the waves serves both. The maximum is taken over
// the bit patterns of |h w| as integers, whose order is the floats' order with
// NaN above everything: a NaN anywhere gives the row a NaN scale.
//
// Gradient: with g = dy w, dx = r g - h r^3 mean(g h) (+ dh) and
// dweight = sum_rows dy h r. A row's two sums (h^2 and g h) come from one pass
// over registers too. A workgroup walks rows in steps of the grid and keeps
// the dweight sums of its columns in fp32 registers; the sums of the
// workgroups meet in a second small kernel, in a fixed order.
//
// Both are bound by memory: a few fp32 operations for every byte moved.
#include "pipe_norm.hpp"

namespace pipe {

namespace {

// The sums of the waves of one row: TPR threads a row, in a workgroup of WG.
template <int TPR, int WG, bool MAX>
struct RowExchange {
  static constexpr int kWaves = WG / 64, kRowWaves = TPR / 64;
  float sum[2][kWaves];
  uint32_t top[MAX ? kWaves : 1];
};

// One row per TPR threads, WG / TPR rows a workgroup; a thread holds CH chunks
// of 8 elements, chunk index t + TPR * i. 8192 x 8192 with residual and e4m3
// output takes 72 us in the kernel (6.5 TB/s, what a copy reaches); 1021 x 5000
// 9 us (4.6 TB/s), where a launch and one trip to memory are half; one row of
// 4096 2.2 us, the two alone.
template <class T, int TPR, int WG, int CH, bool RES, bool Q8>
__global__ void __launch_bounds__(WG) rmsnorm_kernel(NormParams p) {
  constexpr int kRows = WG / TPR, kRowWaves = TPR / 64;
  __shared__ RowExchange<TPR, WG, Q8> ex;
  const int t = threadIdx.x % TPR;
  const int64_t row = long_block() * kRows + threadIdx.x / TPR;
  const bool live = row < p.M;
  const int64_t at = live ? row : p.M - 1;
  const u32x4* x = reinterpret_cast<const u32x4*>(p.x + at * p.ld_x);
  const u32x4* res = reinterpret_cast<const u32x4*>(p.residual + at * p.ld_residual);
  const u32x4* w = reinterpret_cast<const u32x4*>(p.weight);
  u32x4 v[CH], a[RES ? CH : 1], wt[CH];
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
    wt[i] = u32x4{0, 0, 0, 0};
    if (c < p.chunks) wt[i] = w[c];
  }
  float sum = 0.f;
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < CH; ++i) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if constexpr (RES)
        v[i][e] = Pair<T>::pack(Pair<T>::lo(v[i][e]) + Pair<T>::lo(a[i][e]),
                                Pair<T>::hi(v[i][e]) + Pair<T>::hi(a[i][e]));
      const float lo = Pair<T>::lo(v[i][e]), hi = Pair<T>::hi(v[i][e]);
      sum += lo * lo;
      sum += hi * hi;
      if constexpr (Q8) {
        const uint32_t tl = abs_bits(lo * Pair<T>::lo(wt[i][e]));
        const uint32_t th = abs_bits(hi * Pair<T>::hi(wt[i][e]));
        top = max(top, max(tl, th));
      }
    }
  }
  sum = wave_sum(sum);
  if constexpr (Q8) top = wave_max(top);
  if constexpr (kRowWaves > 1) {
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) {
      ex.sum[0][wave] = sum;
      if constexpr (Q8) ex.top[wave] = top;
    }
    __syncthreads();
    const int first = wave / kRowWaves * kRowWaves;
    sum = 0.f;
    top = 0;
#pragma unroll
    for (int i = 0; i < kRowWaves; ++i) {
      sum += ex.sum[0][first + i];
      if constexpr (Q8) top = max(top, ex.top[first + i]);
    }
  }
  if (!live) return;
  keep_packed(v);
  keep_packed(wt);
  const float r = 1.0f / sqrtf(sum * p.inv_n + p.eps);
  if constexpr (RES) {
    u32x4* h = reinterpret_cast<u32x4*>(p.h + row * p.ld_h);
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = t + TPR * i;
      if (c < p.chunks) h[c] = v[i];
    }
  }
  if constexpr (Q8) {
    float m = __uint_as_float(top) * r;
    m = m < kAmaxMin ? kAmaxMin : m;  // a NaN stays
    const float s = m / kE4m3Max;
    const float inv = kE4m3Max / m;
    if (t == 0) p.scales[row] = s;
    u32x2* y = reinterpret_cast<u32x2*>(p.y + row * p.ld_y);
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = t + TPR * i;
      float f[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        f[2 * e] = Pair<T>::lo(v[i][e]) * r * Pair<T>::lo(wt[i][e]) * inv;
        f[2 * e + 1] = Pair<T>::hi(v[i][e]) * r * Pair<T>::hi(wt[i][e]) * inv;
      }
      u32x2 o;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        int b = __builtin_amdgcn_cvt_pk_fp8_f32(f[4 * e], f[4 * e + 1], 0, false);
        o[e] = __builtin_amdgcn_cvt_pk_fp8_f32(f[4 * e + 2], f[4 * e + 3], b, true);
      }
      if (c < p.chunks) y[c] = o;
    }
  } else {
    u32x4* y = reinterpret_cast<u32x4*>(p.y + row * p.ld_y);
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = t + TPR * i;
      u32x4 o;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        o[e] = Pair<T>::pack(Pair<T>::lo(v[i][e]) * r * Pair<T>::lo(wt[i][e]),
                             Pair<T>::hi(v[i][e]) * r * Pair<T>::hi(wt[i][e]));
      if (c < p.chunks) y[c] = o;
    }
  }
}

template <class T, int TPR, int WG, int CH>
hipError_t launch_norm_shape(const NormParams& p, bool q8, hipStream_t stream) {
  const int64_t wgs = (p.M + WG / TPR - 1) / (WG / TPR);
  const bool res = p.residual != nullptr;
  void (*k)(NormParams) = res ? (q8 ? rmsnorm_kernel<T, TPR, WG, CH, true, true>
                                    : rmsnorm_kernel<T, TPR, WG, CH, true, false>)
                              : (q8 ? rmsnorm_kernel<T, TPR, WG, CH, false, true>
                                    : rmsnorm_kernel<T, TPR, WG, CH, false, false>);
  hipLaunchKernelGGL(k, long_grid(wgs), dim3(WG), 0, stream, p);
  return hipGetLastError();
}

// Rows of up to 2048 elements: one wave each, no exchange between waves. Wider
// rows: a workgroup each, of as many threads as leave each at most 4 chunks.
template <class T>
hipError_t launch_norm_type(const NormParams& p, bool q8, hipStream_t stream) {
  if (p.chunks <= 64) return launch_norm_shape<T, 64, 256, 1>(p, q8, stream);
  if (p.chunks <= 128) return launch_norm_shape<T, 64, 256, 2>(p, q8, stream);
  if (p.chunks <= 256) return launch_norm_shape<T, 64, 256, 4>(p, q8, stream);
  if (p.chunks <= 512) return launch_norm_shape<T, 256, 256, 2>(p, q8, stream);
  if (p.chunks <= 1024) return launch_norm_shape<T, 512, 512, 2>(p, q8, stream);
  if (p.chunks <= 2048) return launch_norm_shape<T, 512, 512, 4>(p, q8, stream);
  return launch_norm_shape<T, 1024, 1024, 4>(p, q8, stream);
}

// ---------------------------------------------------------------------------
// Gradient. A workgroup's rows are its grid stride's; 8192 x 8192 with the
// residual stream's gradient takes 88 us (6.1 TB/s, bound by memory: a copy
// reaches 6.5) and 4.9 for the sum of the partials, 1021 x 2048 5.8 and 3.4, of
// which bytes are 2: launches, one trip to memory and two turns of rows.
// ---------------------------------------------------------------------------
template <class T, int TPR, int WG, int CH, bool RES>
__global__ void __launch_bounds__(WG) rmsnorm_grad_kernel(NormGradParams p) {
  constexpr int kRows = WG / TPR, kRowWaves = TPR / 64;
  __shared__ RowExchange<TPR, WG, false> ex[2];
  const int t = threadIdx.x % TPR;
  const int sub = threadIdx.x / TPR;
  const int wave = threadIdx.x >> 6;
  const u32x4* w = reinterpret_cast<const u32x4*>(p.weight);
  u32x4 wt[CH];
  float dw[CH][8];
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = t + TPR * i;
    wt[i] = u32x4{0, 0, 0, 0};
    if (c < p.chunks) wt[i] = w[c];
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[i][e] = 0.f;
  }
  // A row's loads go out before the row ahead of it is reduced. Past the last
  // row they take the last one again: a branch around them would make the
  // compiler wait for them with the row in use. Not so with four chunks for each
  // of 1024 threads, rows wider than 16384: a thread has 128 registers there, and
  // two rows' worth spilled up to 115 of them (2048 x 32768 took 359 us so, and
  // takes 109; 8 x 32768 35 and 10).
  constexpr bool kAhead = WG < 1024 || CH < 4;
  u32x4 h[CH], d[CH], s[RES ? CH : 1], nh[CH], nd[CH], ns[RES ? CH : 1];
  const auto load = [&](int64_t row) {
    const int64_t at = row < p.M ? row : p.M - 1;
    const u32x4* dy = reinterpret_cast<const u32x4*>(p.dy + at * p.ld_dy);
    const u32x4* x = reinterpret_cast<const u32x4*>(p.x + at * p.ld_x);
    const u32x4* dh = reinterpret_cast<const u32x4*>(p.dh + at * p.ld_dh);
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = t + TPR * i;
      nh[i] = nd[i] = u32x4{0, 0, 0, 0};
      if (c < p.chunks) {
        nh[i] = __builtin_nontemporal_load(x + c);
        nd[i] = __builtin_nontemporal_load(dy + c);
      }
    }
    if constexpr (RES) {
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        const int c = t + TPR * i;
        ns[i] = u32x4{0, 0, 0, 0};
        if (c < p.chunks) ns[i] = __builtin_nontemporal_load(dh + c);
      }
    }
  };
  int turn = 0;
  const int64_t step = (int64_t)gridDim.x * kRows;
  if constexpr (kAhead) load((int64_t)blockIdx.x * kRows + sub);
  for (int64_t base = (int64_t)blockIdx.x * kRows; base < p.M; base += step, turn ^= 1) {
    const int64_t row = base + sub;
    const bool live = row < p.M;
    if constexpr (!kAhead) load(row);
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      h[i] = nh[i];
      d[i] = nd[i];
      if constexpr (RES) s[i] = ns[i];
    }
    if constexpr (kAhead) load(row + step);
    float hh = 0.f, gh = 0.f;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float hl = Pair<T>::lo(h[i][e]), hu = Pair<T>::hi(h[i][e]);
        hh += hl * hl;
        hh += hu * hu;
        gh += Pair<T>::lo(d[i][e]) * Pair<T>::lo(wt[i][e]) * hl;
        gh += Pair<T>::hi(d[i][e]) * Pair<T>::hi(wt[i][e]) * hu;
      }
    }
    hh = wave_sum(hh);
    gh = wave_sum(gh);
    if constexpr (kRowWaves > 1) {
      // Two exchange buffers in turn: a wave writes one again only after the
      // barrier of the other, which every wave reaches after its reads.
      if ((threadIdx.x & 63) == 0) {
        ex[turn].sum[0][wave] = hh;
        ex[turn].sum[1][wave] = gh;
      }
      __syncthreads();
      const int first = wave / kRowWaves * kRowWaves;
      hh = gh = 0.f;
#pragma unroll
      for (int i = 0; i < kRowWaves; ++i) {
        hh += ex[turn].sum[0][first + i];
        gh += ex[turn].sum[1][first + i];
      }
    }
    keep_packed(h);
    keep_packed(d);
    keep_packed(wt);
    if (live) {
      const float r = 1.0f / sqrtf(hh * p.inv_n + p.eps);
      const float k = gh * p.inv_n * r * r * r;
      u32x4* dx = reinterpret_cast<u32x4*>(p.dx + row * p.ld_dx);
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        const int c = t + TPR * i;
        u32x4 o;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float hl = Pair<T>::lo(h[i][e]), hu = Pair<T>::hi(h[i][e]);
          const float dl = Pair<T>::lo(d[i][e]), du = Pair<T>::hi(d[i][e]);
          float ol = dl * Pair<T>::lo(wt[i][e]) * r - hl * k;
          float ou = du * Pair<T>::hi(wt[i][e]) * r - hu * k;
          if constexpr (RES) {
            ol += Pair<T>::lo(s[i][e]);
            ou += Pair<T>::hi(s[i][e]);
          }
          o[e] = Pair<T>::pack(ol, ou);
          dw[i][2 * e] += dl * (hl * r);
          dw[i][2 * e + 1] += du * (hu * r);
        }
        if (c < p.chunks) dx[c] = o;
      }
    }
  }
  f32x4* out = reinterpret_cast<f32x4*>(p.partials + (int64_t)blockIdx.x * ((int64_t)p.chunks * 8));
  if constexpr (kRows == 1) {
    // The thread's place is made anew for the compiler, which would else keep
    // the columns through the loop, in scratch memory where registers are short.
    int at = t;
    asm volatile("" : "+v"(at));
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = at + TPR * i;
      if (c < p.chunks) {
        out[2 * c] = f32x4{dw[i][0], dw[i][1], dw[i][2], dw[i][3]};
        out[2 * c + 1] = f32x4{dw[i][4], dw[i][5], dw[i][6], dw[i][7]};
      }
    }
  } else {
    // The rows in flight add up in LDS first, in order.
    __shared__ f32x4 sums[kRows][2 * CH * TPR];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = t + TPR * i;
      sums[sub][2 * c] = f32x4{dw[i][0], dw[i][1], dw[i][2], dw[i][3]};
      sums[sub][2 * c + 1] = f32x4{dw[i][4], dw[i][5], dw[i][6], dw[i][7]};
    }
    __syncthreads();
    for (int u = (int)threadIdx.x; u < 2 * p.chunks; u += WG) {
      f32x4 v = sums[0][u];
#pragma unroll
      for (int r = 1; r < kRows; ++r) v += sums[r][u];
      out[u] = v;
    }
  }
}

// dweight: the partials' sum. A workgroup takes 32 columns (8 threads of four)
// and 32 interleaved sets of partials, each summed in order, then the 32 sums
// in order. 3.4 us for 256 partials of 2048 columns, 4.9 for 512 of 8192: a
// launch, and chains of loads that the caches answer.
__global__ void __launch_bounds__(256) rmsnorm_dweight_kernel(const float* __restrict__ partials,
                                                              float* __restrict__ dweight,
                                                              int count, int n) {
  __shared__ f32x4 part[32][8];
  const int lane = threadIdx.x & 7, set = threadIdx.x >> 3;
  const int col = blockIdx.x * 32 + lane * 4;
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  if (col < n) {
    const float* src = partials + col;
#pragma unroll 4
    for (int i = set; i < count; i += 32)
      acc += *reinterpret_cast<const f32x4*>(src + (int64_t)i * n);
  }
  part[set][lane] = acc;
  __syncthreads();
  if (set == 0 && col < n) {
    acc = part[0][lane];
    for (int i = 1; i < 32; ++i) acc += part[i][lane];
    *reinterpret_cast<f32x4*>(dweight + col) = acc;
  }
}

struct GradShape {
  bool tall;     // many rows: one row in flight a workgroup of 256 up to 8192 columns
  int64_t grid;
};

// Each workgroup writes a row of partials, so few rows want few workgroups with
// several rows in flight each, of 1024 threads: 1021 x 8192 takes 22.5 us with
// 256 of those and 26 with 512 of 256 threads, 8192 x 8192 100 and 95. The few
// take equal numbers of turns, a multiple of 8 of them for the XCDs' sake: 647 x
// 5520 15.3 us, in 256 workgroups of one and two turns 16.8. A lone
// workgroup writes dweight itself (a second turn of rows in it would already
// cost the second kernel's time).
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
hipError_t launch_grad_shape(const NormGradParams& p, int64_t grid, hipStream_t stream) {
  void (*k)(NormGradParams) = p.dh != nullptr ? rmsnorm_grad_kernel<T, TPR, WG, CH, true>
                                              : rmsnorm_grad_kernel<T, TPR, WG, CH, false>;
  hipLaunchKernelGGL(k, dim3((unsigned)grid), dim3(WG), 0, stream, p);
  return hipGetLastError();
}

template <class T>
hipError_t launch_grad_type(const NormGradParams& p, const GradShape& g, hipStream_t stream) {
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
  return launch_grad_shape<T, 1024, 1024, 4>(p, g.grid, stream);
}

}  // namespace

hipError_t launch_rmsnorm(const NormParams& p, int type, bool q8, hipStream_t stream) {
  return type == 0 ? launch_norm_type<__bf16>(p, q8, stream)
                   : launch_norm_type<_Float16>(p, q8, stream);
}

int64_t rmsnorm_grad_partials(int64_t M, int64_t N) {
  const int64_t grid = grad_shape(M, N / 8).grid;
  return grid > 1 ? grid : 0;
}

hipError_t launch_rmsnorm_grad(NormGradParams p, float* dweight, int type, hipStream_t stream) {
  const GradShape g = grad_shape(p.M, p.chunks);
  if (g.grid > 0) {
    if (g.grid == 1) p.partials = dweight;
    const hipError_t e = type == 0 ? launch_grad_type<__bf16>(p, g, stream)
                                   : launch_grad_type<_Float16>(p, g, stream);
    if (e != hipSuccess || g.grid == 1) return e;
  }
  const int n = p.chunks * 8;
  hipLaunchKernelGGL(rmsnorm_dweight_kernel, dim3((n + 31) / 32), dim3(256), 0, stream, p.partials,
                     dweight, (int)g.grid, n);
  return hipGetLastError();
}

}  // namespace pipe
