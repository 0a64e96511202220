// Layer norm over the rows of [M, N], forward and backward.
//
//   mean = sum x / N,  var = sum (x - mean)^2 / N,  rstd = 1 / sqrt(var + eps)
//   xh = (x - mean) rstd,  y = xh w + b
//   dx = rstd (dy w - c1 - xh c2),  c1 = sum(dy w) / N,  c2 = sum(dy w xh) / N
//   dw = sum over rows of dy xh,  db = sum over rows of dy
//
// Tensors of bf16, fp16 or fp32 (T); w and b of the same type or fp32 (W).  All arithmetic
// and all sums are fp32; each output is rounded once.
#include <type_traits>

#include "launch.hpp"
#include "rows.hpp"

namespace swg {

// ------------------------------------------------------------------ rows of any length
// Rows under 8 (a wave each) or over 16384 elements (512 threads): chunks of 8 elements and up to 7
// single ones at the end; the second and third pass over a row come from cache.  [1000, 40000]
// bf16 takes 46 us forward and 97 us backward (199 and 239 us by single elements), one row of
// 65536 14 and 19 us.

template <int n, typename W>
__device__ inline void affine_part(const W* w, int64_t c, float absent, float* f) {
  if (w) {
    load_part<n>(w + c, f);
  } else {
#pragma unroll
    for (int i = 0; i < n; ++i) f[i] = absent;
  }
}

template <typename T, typename W, int NT>
__global__ __launch_bounds__(NT) void norm_fwd_any_kernel(
    const T* x, int64_t ldx, const W* w, const W* b, T* y, int64_t ldy, float* mean, float* rstd,
    int64_t M, int64_t N, float eps) {
  __shared__ float red[NT / 64];
  for (int64_t r = blockIdx.x; r < M; r += gridDim.x) {
    const T* xr = x + r * ldx;
    T* yr = y + r * ldy;
    float s = 0.0f;
    each_part<NT>(N, [&](int64_t c, auto size) {
      constexpr int n = decltype(size)::value;
      float f[n];
      load_part<n>(xr + c, f);
#pragma unroll
      for (int i = 0; i < n; ++i) s += f[i];
    });
    const float mu = block_sum<NT>(s, red) / (float)N;
    s = 0.0f;
    each_part<NT>(N, [&](int64_t c, auto size) {
      constexpr int n = decltype(size)::value;
      float f[n];
      load_part<n>(xr + c, f);
#pragma unroll
      for (int i = 0; i < n; ++i) s = __builtin_fmaf(f[i] - mu, f[i] - mu, s);
    });
    const float rs = 1.0f / __builtin_sqrtf(block_sum<NT>(s, red) / (float)N + eps);
    each_part<NT>(N, [&](int64_t c, auto size) {
      constexpr int n = decltype(size)::value;
      float f[n], g[n], h[n];
      load_part<n>(xr + c, f);
      affine_part<n>(w, c, 1.0f, g);
      affine_part<n>(b, c, 0.0f, h);
#pragma unroll
      for (int i = 0; i < n; ++i) f[i] = __builtin_fmaf((f[i] - mu) * rs, g[i], h[i]);
      store_part<n>(yr + c, f);
    });
    if (threadIdx.x == 0) {
      if (mean) mean[r] = mu;
      if (rstd) rstd[r] = rs;
    }
  }
}

template <typename T, typename W, int NT>
__global__ __launch_bounds__(NT) void norm_dx_any_kernel(
    const T* dy, int64_t lddy, const T* x, int64_t ldx, const W* w, const float* mean,
    const float* rstd, T* dx, int64_t lddx, int64_t M, int64_t N) {
  __shared__ float red[NT / 64];
  for (int64_t r = blockIdx.x; r < M; r += gridDim.x) {
    const T* dr = dy + r * lddy;
    const T* xr = x + r * ldx;
    T* out = dx + r * lddx;
    const float mu = mean[r], rs = rstd[r];
    float s1 = 0.0f, s2 = 0.0f;
    each_part<NT>(N, [&](int64_t c, auto size) {
      constexpr int n = decltype(size)::value;
      float d[n], f[n], g[n];
      load_part<n>(dr + c, d);
      load_part<n>(xr + c, f);
      affine_part<n>(w, c, 1.0f, g);
#pragma unroll
      for (int i = 0; i < n; ++i) {
        const float h = d[i] * g[i];
        s1 += h;
        s2 = __builtin_fmaf(h, (f[i] - mu) * rs, s2);
      }
    });
    const float c1 = block_sum<NT>(s1, red) / (float)N;
    const float c2 = block_sum<NT>(s2, red) / (float)N;
    each_part<NT>(N, [&](int64_t c, auto size) {
      constexpr int n = decltype(size)::value;
      float d[n], f[n], g[n];
      load_part<n>(dr + c, d);
      load_part<n>(xr + c, f);
      affine_part<n>(w, c, 1.0f, g);
#pragma unroll
      for (int i = 0; i < n; ++i) d[i] = rs * (d[i] * g[i] - c1 - (f[i] - mu) * rs * c2);
      store_part<n>(out + c, d);
    });
  }
}

// One partial row [dw | db] of fp32 per block of rows; a thread takes 8 columns, or the up to 7
// at the end.
template <typename T>
__global__ __launch_bounds__(256) void norm_cols_any_kernel(const T* dy, int64_t lddy, const T* x,
                                                            int64_t ldx, const float* mean,
                                                            const float* rstd, float* part,
                                                            int64_t M, int64_t N, int64_t Np,
                                                            int64_t rows) {
  const int64_t c = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8;
  if (c >= N) return;
  const int n = N - c < 8 ? (int)(N - c) : 8;
  const int64_t r0 = (int64_t)blockIdx.y * rows, r1 = r0 + rows < M ? r0 + rows : M;
  float sw[8], sb[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) sw[i] = sb[i] = 0.0f;
  for (int64_t r = r0; r < r1; ++r) {
    const T* dr = dy + r * lddy + c;
    const T* xr = x + r * ldx + c;
    float d[8], f[8];
    if (n == 8) {
      load_part<8>(dr, d);
      load_part<8>(xr, f);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        d[i] = i < n ? to_f32(dr[i]) : 0.0f;
        f[i] = i < n ? to_f32(xr[i]) : 0.0f;
      }
    }
    const float mu = mean[r], rs = rstd[r];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      sw[i] = __builtin_fmaf(d[i], (f[i] - mu) * rs, sw[i]);
      sb[i] += d[i];
    }
  }
  part += (int64_t)blockIdx.y * 2 * Np;
  for (int i = 0; i < n; ++i) {
    part[c + i] = sw[i];
    part[Np + c + i] = sb[i];
  }
}

// ------------------------------------------------------------------ rows in registers
// w and b as fp32 (1 and 0 where absent)
template <typename W>
__device__ inline void load_affine(const W* w, int64_t c, float absent, float* f) {
  if (w) {
    Chunk<W> k;
    k.load(w + c);
    k.widen(f);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = absent;
  }
}

// s / n from 1 / n, with the remainder put back: the rounding of 1 / n would move the mean by up to
// its last place, and a row of equal values far from 0 would be normed by nothing but that.  An
// infinite s stays.
__device__ inline float quotient(float s, float n, float inv_n) {
  const float q = s * inv_n;
  const float r = __builtin_fmaf(__builtin_fmaf(-q, n, s), inv_n, q);
  return r == r ? r : q;
}

// Forward: the row is read once; the variance is the mean of squared differences from the mean,
// both over registers.  All workgroups are resident and walk over the rows with the next row's
// loads in flight.  Bound by memory, and closely behind by the arithmetic around the two
// reductions (a wave takes about 200 instructions a row of 512): [220000, 512] bf16, 450 MB,
// 84 us = 5.4 TB/s (469 us with one element at a time in three passes; 90 us with w and b read
// again for every row and IEEE divisions); one row of 4096 under 5 us, most of it the launch.
// Rows above 1024 columns are spread over waves (one barrier a reduction): with 4 or 8 chunks a
// thread instead of 2, one row of 14336 bf16 takes 8.0 us, not 5.5.
template <typename T, typename W, int G, int EC>
__global__ __launch_bounds__(G > 256 ? G : 256) void norm_fwd_kernel(
    const T* x, int64_t ldx, const W* w, const W* b, T* y, int64_t ldy, float* mean, float* rstd,
    int64_t M, int64_t N, float eps) {
  constexpr int ROWS = G > 256 ? 1 : 256 / G;
  __shared__ float red[2][G > 256 ? G / 64 : 4];
  const int lane = threadIdx.x % G;
  const RowMap<G, EC> map(lane, N);
  const float inv_n = 1.0f / (float)N;
  // of one chunk w and b stay in registers, of more they are read again (from cache)
  float wv[EC == 1 ? 8 : 1], bv[EC == 1 ? 8 : 1];
  if constexpr (EC == 1) {
    load_affine(w, map.col[0], 1.0f, wv);
    load_affine(b, map.col[0], 0.0f, bv);
  }
  const int64_t step = (int64_t)gridDim.x * ROWS;
  const int grp = row_group<G>();
  int64_t r = (int64_t)blockIdx.x * ROWS + grp;
  Chunk<T> cur[EC], next[EC];
#pragma unroll
  for (int j = 0; j < EC; ++j) {
    cur[j].zero();
    if (map.has(j) && r < M) cur[j].load_stream(x + r * ldx + map.col[j]);
  }
  // every thread of the workgroup makes the same number of passes (barriers)
  for (int64_t base = (int64_t)blockIdx.x * ROWS; base < M; base += step, r += step) {
#pragma unroll
    for (int j = 0; j < EC; ++j) {
      next[j].zero();
      if (map.has(j) && r + step < M) next[j].load_stream(x + (r + step) * ldx + map.col[j]);
    }
    float f[EC][8];
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < EC; ++j) {
      cur[j].widen(f[j]);
      float g[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) g[i] = f[j][i];
      drop(g, map.skip[j]);
      s += ((g[0] + g[1]) + (g[2] + g[3])) + ((g[4] + g[5]) + (g[6] + g[7]));
    }
    const float mu = quotient(row_sum<G>(s, red[0], grp * (G / 64)), (float)N, inv_n);
    s = 0.0f;
#pragma unroll
    for (int j = 0; j < EC; ++j) {
      float g[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) f[j][i] -= mu, g[i] = f[j][i];
      drop(g, map.skip[j]);
      float q = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) q = __builtin_fmaf(g[i], g[i], q);
      s += q;
    }
    const float var = row_sum<G>(s, red[1], grp * (G / 64)) * inv_n;
    const float rs = inv_root(var + eps);
    if (r < M) {
#pragma unroll
      for (int j = 0; j < EC; ++j) {
        if (!map.has(j)) continue;
        float g[8], h[8];
        if constexpr (EC == 1) {
#pragma unroll
          for (int i = 0; i < 8; ++i) g[i] = wv[i], h[i] = bv[i];
        } else {
          load_affine(w, map.col[j], 1.0f, g);
          load_affine(b, map.col[j], 0.0f, h);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) g[i] = __builtin_fmaf(f[j][i] * rs, g[i], h[i]);
        Chunk<T> o;
        o.narrow(g);
        o.store_stream(y + r * ldy + map.col[j]);
      }
      if (lane == 0) {
        if (mean) mean[r] = mu;
        if (rstd) rstd[r] = rs;
      }
    }
#pragma unroll
    for (int j = 0; j < EC; ++j) cur[j] = next[j];
  }
}

// Backward: one pass over dy and x.  A workgroup of 1024 threads walks its share of the rows,
// 1024 / G at a time; each thread keeps the sums dy xh and dy of its own columns in registers,
// and the row groups of the workgroup add theirs through LDS at the end, in a fixed order, to
// one partial row [dw | db] (dw and db themselves where there is one workgroup).  Bound by
// memory: [220000, 512] bf16, 676 MB, 117 us = 5.8 TB/s, of it 4 us for the partial rows' sums
// (963 us as two passes of single elements); [16384, 4096] fp16 with fp32 w 77 us = 5.2 TB/s;
// [8191, 1023] fp32, rows at any 4-byte boundary, 28 us.  One workgroup a CU keeps the partial
// rows few: they cost 8 N bytes a workgroup twice, which shows where rows are few and wide
// ([1000, 8192] bf16: 25 us with dw and db, 11 us without).  Above 4096 columns the 128 registers
// of 1024 threads do not hold everything: 12 to 32 bytes a lane spill.
template <typename T, typename W, int G, int EC>
__global__ __launch_bounds__(1024) void norm_bwd_kernel(NormArgs a, float* part, int64_t Np) {
  constexpr int ROWS = 1024 / G;
  __shared__ float red[2][2][16];
  __shared__ float sums[ROWS > 1 ? 1024 * EC * 8 : 1];
  const int lane = threadIdx.x % G, grp = row_group<G>(), wave0 = grp * (G / 64);
  const RowMap<G, EC> map(lane, a.N);
  const T* dy = static_cast<const T*>(a.dy);
  const T* x = static_cast<const T*>(a.x);
  T* dx = static_cast<T*>(a.dx);
  float w[EC][8], sw[EC][8], sb[EC][8];
#pragma unroll
  for (int j = 0; j < EC; ++j) {
    load_affine(static_cast<const W*>(a.w), map.col[j], 1.0f, w[j]);
    // keeps duplicates out of c1 and c2; their column sums are not written
    drop(w[j], map.skip[j]);
#pragma unroll
    for (int i = 0; i < 8; ++i) sw[j][i] = sb[j][i] = 0.0f;
  }
  const float inv_n = 1.0f / (float)a.N;
  const int64_t step = (int64_t)gridDim.x * ROWS;
  int64_t r = (int64_t)blockIdx.x * ROWS + grp;
  int half = 0;
  auto load = [&](Chunk<T>* d, Chunk<T>* f, int64_t row) {
#pragma unroll
    for (int j = 0; j < EC; ++j) {
      d[j].zero();
      f[j].zero();
      if (map.has(j) && row < a.M) {
        d[j].load_stream(dy + row * a.lddy + map.col[j]);
        f[j].load_stream(x + row * a.ldx + map.col[j]);
      }
    }
  };
  // one chunk a thread leaves registers for the next row's loads
  constexpr bool AHEAD = EC == 1;
  Chunk<T> cd[EC], cx[EC], nd[EC], nx[EC];
  if (AHEAD) load(cd, cx, r);
  for (int64_t base = (int64_t)blockIdx.x * ROWS; base < a.M; base += step, r += step) {
    const bool live = r < a.M;
    if (AHEAD) load(nd, nx, r + step);
    else load(cd, cx, r);
    const float mu = live ? a.mean[r] : 0.0f, rs = live ? a.rstd[r] : 0.0f;
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int j = 0; j < EC; ++j) {
      float d[8], f[8];
      cd[j].widen(d);
      cx[j].widen(f);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float xh = (f[i] - mu) * rs, h = d[i] * w[j][i];
        s1 += h;
        s2 = __builtin_fmaf(h, xh, s2);
        sw[j][i] = __builtin_fmaf(d[i], xh, sw[j][i]);
        sb[j][i] += d[i];
      }
    }
    if (dx) {
      s1 = lanes_sum<(G < 64 ? G : 64)>(s1);
      s2 = lanes_sum<(G < 64 ? G : 64)>(s2);
      if constexpr (G > 64) {
        if ((threadIdx.x & 63) == 0) {
          red[half][0][threadIdx.x >> 6] = s1;
          red[half][1][threadIdx.x >> 6] = s2;
        }
        __syncthreads();
        s1 = red[half][0][wave0];
        s2 = red[half][1][wave0];
#pragma unroll
        for (int i = 1; i < G / 64; ++i) {
          s1 += red[half][0][wave0 + i];
          s2 += red[half][1][wave0 + i];
        }
        half ^= 1;
      }
      const float c1 = s1 * inv_n, c2 = s2 * inv_n;
      if (live) {
#pragma unroll
        for (int j = 0; j < EC; ++j) {
          if (!map.has(j)) continue;
          float d[8], f[8];
          cd[j].widen(d);
          cx[j].widen(f);
          if (map.skip[j] > 0) {
            float v[8];
            load_affine(static_cast<const W*>(a.w), map.col[j], 1.0f, v);
#pragma unroll
            for (int i = 0; i < 8; ++i) d[i] *= v[i];
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) d[i] *= w[j][i];
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float xh = (f[i] - mu) * rs;
            d[i] = rs * (d[i] - c1 - xh * c2);
          }
          Chunk<T> o;
          o.narrow(d);
          o.store_stream(dx + r * a.lddx + map.col[j]);
        }
      }
    }
    if (AHEAD) {
#pragma unroll
      for (int j = 0; j < EC; ++j) cd[j] = nd[j], cx[j] = nx[j];
    }
  }
  if (!a.dw && !a.db) return;
  // the row groups' sums, group by group; each thread of the first group ends with its columns'
  if constexpr (ROWS > 1) {
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      __syncthreads();
#pragma unroll
      for (int j = 0; j < EC; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i)
          sums[(j * 8 + i) * 1024 + threadIdx.x] = which ? sb[j][i] : sw[j][i];
      __syncthreads();
      // G * EC * 8 column sums over 1024 threads
      constexpr int COLS = G * EC * 8;
      float total[(COLS + 1023) / 1024];
#pragma unroll
      for (int q = 0; q < (COLS + 1023) / 1024; ++q) {
        const int e = q * 1024 + threadIdx.x;
        total[q] = 0.0f;
        if (COLS % 1024 == 0 || e < COLS) {
          for (int g = 0; g < ROWS; ++g) total[q] += sums[(e / G) * 1024 + g * G + e % G];
        }
      }
      __syncthreads();
#pragma unroll
      for (int q = 0; q < (COLS + 1023) / 1024; ++q) {
        const int e = q * 1024 + threadIdx.x;
        if (COLS % 1024 == 0 || e < COLS) sums[e] = total[q];
      }
      __syncthreads();
      if (grp == 0) {
#pragma unroll
        for (int j = 0; j < EC; ++j)
#pragma unroll
          for (int i = 0; i < 8; ++i)
            (which ? sb : sw)[j][i] = sums[(j * 8 + i) * G + lane];
      }
    }
    if (grp != 0) return;
  }
  W* dw = static_cast<W*>(a.dw);
  W* db = static_cast<W*>(a.db);
  float* pw = part + (int64_t)blockIdx.x * 2 * Np;
#pragma unroll
  for (int j = 0; j < EC; ++j) {
    if (gridDim.x > 1 && map.skip[j] == 0) {   // a whole chunk: columns 8 n, 16-byte aligned
      f32x4* w4 = reinterpret_cast<f32x4*>(pw + map.col[j]);
      f32x4* b4 = reinterpret_cast<f32x4*>(pw + Np + map.col[j]);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        w4[i] = f32x4{sw[j][4 * i], sw[j][4 * i + 1], sw[j][4 * i + 2], sw[j][4 * i + 3]};
        b4[i] = f32x4{sb[j][4 * i], sb[j][4 * i + 1], sb[j][4 * i + 2], sb[j][4 * i + 3]};
      }
      continue;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (i < map.skip[j]) continue;
      const int64_t c = map.col[j] + i;
      if (gridDim.x > 1) {
        pw[c] = sw[j][i];
        pw[Np + c] = sb[j][i];
      } else {
        if (dw) dw[c] = from_f32<W>(a.accumulate ? to_f32(dw[c]) + sw[j][i] : sw[j][i]);
        if (db) db[c] = from_f32<W>(a.accumulate ? to_f32(db[c]) + sb[j][i] : sb[j][i]);
      }
    }
  }
}

// Sums the partial rows: Q groups of 4 columns to a workgroup, 256 / Q threads a group, each over
// every (256 / Q)-th partial row, then those in order.  Q = 4 gives narrow norms workgroups, 16
// reads whole lines of wide ones.
template <typename W, int Q>
__global__ __launch_bounds__(256) void norm_finalize_kernel(const float* part, int64_t nparts,
                                                            W* dw, W* db, int64_t N, int64_t Np,
                                                            int acc) {
  constexpr int P = 256 / Q;
  __shared__ f32x4 red[P][Q];
  const int q = threadIdx.x % Q, lane = threadIdx.x / Q;
  const int64_t c = (wide_block() * Q + q) * 4;   // column of the 2 Np
  f32x4 s = {0.0f, 0.0f, 0.0f, 0.0f};
  if (c < 2 * Np) {
#pragma unroll 4
    for (int64_t p = lane; p < nparts; p += P)
      s += *reinterpret_cast<const f32x4*>(part + p * 2 * Np + c);
  }
  red[lane][q] = s;
  __syncthreads();
  for (int n = P / 2; n > 0; n >>= 1) {
    if (lane < n) red[lane][q] += red[lane + n][q];
    __syncthreads();
  }
  if (threadIdx.x >= 4 * Q) return;
  const int64_t e = wide_block() * 4 * Q + threadIdx.x;
  const int64_t col = e < Np ? e : e - Np;
  W* dst = e < Np ? dw : db;
  if (e >= 2 * Np || col >= N || dst == nullptr) return;
  const float v = red[0][threadIdx.x >> 2][threadIdx.x & 3];
  dst[col] = from_f32<W>(acc ? to_f32(dst[col]) + v : v);
}

template <typename T, typename W>
static hipError_t norm_fwd_t(const NormArgs& a, hipStream_t stream) {
  const T* x = static_cast<const T*>(a.x);
  const W* w = static_cast<const W*>(a.w);
  const W* b = static_cast<const W*>(a.b);
  T* y = static_cast<T*>(a.y);
#define SWG_FWD(G, EC)                                                                        \
  SWG_TRY(SWG_LAUNCH((norm_fwd_kernel<T, W, G, EC>),                                          \
                     dim3(norm_fwd_grid(a.M, G > 256 ? 1 : 256 / G, G > 256 ? G : 256)),      \
                     dim3(G > 256 ? G : 256), 0, stream, x, a.ldx, w, b, y, a.ldy,            \
                     a.mean, a.rstd, a.M, a.N, a.eps))
  if (a.N < 8) {
    SWG_TRY(SWG_LAUNCH((norm_fwd_any_kernel<T, W, 64>), dim3(row_grid(a.M)), dim3(64), 0, stream,
                       x, a.ldx, w, b, y, a.ldy, a.mean, a.rstd, a.M, a.N, a.eps));
  } else if (a.N > 16384) {
    SWG_TRY(SWG_LAUNCH((norm_fwd_any_kernel<T, W, 512>), dim3(row_grid(a.M)), dim3(512), 0,
                       stream, x, a.ldx, w, b, y, a.ldy, a.mean, a.rstd, a.M, a.N, a.eps));
  } else if (a.N <= 64) SWG_FWD(8, 1);
  else if (a.N <= 128) SWG_FWD(16, 1);
  else if (a.N <= 256) SWG_FWD(32, 1);
  else if (a.N <= 512) SWG_FWD(64, 1);
  else if (a.N <= 1024) SWG_FWD(64, 2);
  else if (a.N <= 2048) SWG_FWD(256, 1);
  else if (a.N <= 4096) SWG_FWD(256, 2);
  else if (a.N <= 8192) SWG_FWD(512, 2);
  else SWG_FWD(1024, 2);
#undef SWG_FWD
  return hipSuccess;
}

template <typename T, typename W>
static hipError_t norm_bwd_t(const NormArgs& a, const NormPlan& p, float* part,
                             hipStream_t stream) {
  const T* dy = static_cast<const T*>(a.dy);
  const T* x = static_cast<const T*>(a.x);
  if (a.M > 0 && p.group == 0) {
    const W* w = static_cast<const W*>(a.w);
    T* dx = static_cast<T*>(a.dx);
    if (a.dx && a.N < 8)
      SWG_TRY(SWG_LAUNCH((norm_dx_any_kernel<T, W, 64>), dim3(row_grid(a.M)), dim3(64), 0, stream,
                         dy, a.lddy, x, a.ldx, w, a.mean, a.rstd, dx, a.lddx, a.M, a.N));
    else if (a.dx)
      SWG_TRY(SWG_LAUNCH((norm_dx_any_kernel<T, W, 512>), dim3(row_grid(a.M)), dim3(512), 0,
                         stream, dy, a.lddy, x, a.ldx, w, a.mean, a.rstd, dx, a.lddx, a.M, a.N));
    if (!a.dw && !a.db) return hipSuccess;
    SWG_TRY(SWG_LAUNCH((norm_cols_any_kernel<T>),
                       dim3((unsigned)ceil_div(a.N, 2048), (unsigned)p.parts), dim3(256), 0,
                       stream, dy, a.lddy, x, a.ldx, a.mean, a.rstd, part, a.M, a.N, p.np,
                       p.rows));
  } else if (a.M > 0) {
#define SWG_BWD(G, EC)                                                                  \
  case G * 16 + EC:                                                                     \
    SWG_TRY(SWG_LAUNCH((norm_bwd_kernel<T, W, G, EC>), dim3((unsigned)p.parts),         \
                       dim3(1024), 0, stream, a, part, p.np));                          \
    break
    switch (p.group * 16 + p.chunks) {
      SWG_BWD(8, 1);
      SWG_BWD(16, 1);
      SWG_BWD(32, 1);
      SWG_BWD(64, 1);
      SWG_BWD(128, 1);
      SWG_BWD(128, 2);
      SWG_BWD(256, 2);
      SWG_BWD(512, 2);
      SWG_BWD(1024, 2);
    }
#undef SWG_BWD
    if (p.parts == 1 || (!a.dw && !a.db)) return hipSuccess;
  } else if (!a.dw && !a.db) {
    return hipSuccess;
  }
  // M = 0: no partial rows, the empty sums
  const int64_t np = a.M > 0 ? p.np : ceil_div(a.N, 4) * 4;
  const int64_t parts = a.M > 0 ? p.parts : 0;
  if (np < 2048)
    SWG_TRY(SWG_LAUNCH((norm_finalize_kernel<W, 4>), dim3((unsigned)ceil_div(2 * np, 16)),
                       dim3(256), 0, stream, part, parts, static_cast<W*>(a.dw),
                       static_cast<W*>(a.db), a.N, np, a.accumulate));
  else
    SWG_TRY(SWG_LAUNCH((norm_finalize_kernel<W, 16>), wide_grid(ceil_div(2 * np, 64)),
                       dim3(256), 0, stream, part, parts, static_cast<W*>(a.dw),
                       static_cast<W*>(a.db), a.N, np, a.accumulate));
  return hipSuccess;
}

hipError_t launch_norm_fwd(int dtype, int wdtype, const NormArgs& a, hipStream_t stream) {
  if (dtype == 2) return norm_fwd_t<float, float>(a, stream);
  if (wdtype == 2)
    return dtype == 0 ? norm_fwd_t<bf16, float>(a, stream) : norm_fwd_t<fp16, float>(a, stream);
  return dtype == 0 ? norm_fwd_t<bf16, bf16>(a, stream) : norm_fwd_t<fp16, fp16>(a, stream);
}

hipError_t launch_norm_bwd(int dtype, int wdtype, const NormArgs& a, const NormPlan& p,
                           float* part, hipStream_t stream) {
  if (dtype == 2) return norm_bwd_t<float, float>(a, p, part, stream);
  if (wdtype == 2)
    return dtype == 0 ? norm_bwd_t<bf16, float>(a, p, part, stream)
                      : norm_bwd_t<fp16, float>(a, p, part, stream);
  return dtype == 0 ? norm_bwd_t<bf16, bf16>(a, p, part, stream)
                    : norm_bwd_t<fp16, fp16>(a, p, part, stream);
}

}  // namespace swg
