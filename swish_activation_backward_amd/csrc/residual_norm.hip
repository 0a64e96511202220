// Residual norm over the rows of [M, N]: the root mean square norm after a block, its gate, the
// residual sum and the norm before the next block, forward and backward.
//
//   u = y rs wp (or y),  rs = 1 / sqrt(sum y^2 / N + eps)
//   out = residual + scale gate u
//   norm = out rp wq,    rp = 1 / sqrt(sum out^2 / N + eps)
//
// Backward, from dout and dnorm, with xh = out rp, yh = y rs, h = dnorm wq:
//   D = dout + rp (h - xh c),  c = sum(h xh) / N          (the residual's gradient)
//   v = scale gate D wp,  dy = rs (v - yh t),  t = sum(v yh) / N
//   dwq = sum over rows of dnorm xh,  dwp = sum over rows of scale gate D yh
//   dgate = scale D u, summed over the row or over the rows where the gate was broadcast
// The row sums are formed at once, t from D's two parts:
//   sum D e = sum (dout + rp h) e - rp c sum xh e   for e = yh wp gate
//
// y, norm and a gate of the rows are of type T (bf16, fp16, fp32), residual and out of type R (T
// or fp32), wp, wq and a gate of the columns of T or fp32.  All arithmetic, sums and statistics are
// fp32; each output is rounded once (norm is formed from out before its rounding).
//
// Bound by memory: every input is read and every output written once.  Forward [220000, 512] bf16
// with a gate of the columns 167 us = 5.4 TB/s, one row of 4096 4.5 us (the loads of a row and two
// sums one after the other).  Backward, with the join of the column sums: [220000, 512] bf16 with a
// gate an element 317 us = 5.7 TB/s, [16384, 4096] bf16 under an fp32 stream 231 us = 5.2 TB/s,
// [8191, 1023] fp32 with a gate a row 48 us = 4.2 TB/s.
// Not so where the backward pass spills registers, with two chunks a thread: above 1024 columns with
// a gate an element (112 to 158 registers under an fp32 stream, 4 to 26 else; [16384, 4096] bf16
// under fp32 344 us = 4.3 TB/s, fp32 576 us = 3.7) or all of fp32 (13 to 18, 337 us = 4.8), and
// above 8192 columns in every form (83 to 155; [4096, 16384] 404 to 873 us = 2.0 to 2.6 TB/s).  The
// forward spills 10 to 19 above 8192 columns with a gate an element under fp32 (4.2 to 4.8 TB/s).
#include "launch.hpp"
#include "rows.hpp"

namespace swg {

// n weights from column c on as fp32, `absent` without weights
template <int n, typename T>
__device__ inline void load_weights(const void* w, bool wide, int64_t c, float absent, float* f) {
  if (!w) {
#pragma unroll
    for (int i = 0; i < n; ++i) f[i] = absent;
  } else if (wide) {
    load_part<n>(static_cast<const float*>(w) + c, f);
  } else {
    load_part<n>(static_cast<const T*>(w) + c, f);
  }
}

// wp times what of the gate varies along the row (e = yh times this)
template <int n, typename T>
__device__ inline void load_gated(const ResidualNormArgs& a, int64_t row, int64_t c, float* f) {
  load_weights<n, T>(a.post ? a.wp : nullptr, a.wide, c, 1.0f, f);
  if (a.kind == kGateChannel || a.kind == kGateFull) {
    float g[n];
    if (a.kind == kGateChannel) load_weights<n, T>(a.gate, a.wide, c, 1.0f, g);
    else load_part<n>(static_cast<const T*>(a.gate) + row * a.ldg + c, g);
#pragma unroll
    for (int i = 0; i < n; ++i) f[i] *= g[i];
  }
}

// scale times a gate of the row
template <typename T> __device__ inline float row_scale(const ResidualNormArgs& a, int64_t row) {
  if (a.kind != kGateRow) return a.scale;
  return a.scale * to_f32(static_cast<const T*>(a.gate)[row * a.ldg]);
}

// ------------------------------------------------------------------ rows of any length
// Forward three passes over a row, backward three launches with a thread a block of rows for the
// column sums: [1000, 40000] bf16 with a gate of the columns 93 and 323 us, [220000, 7] 117 and 581.
// `out` may be `residual`: each thread writes the elements that only it reads, after its last use
// of them.
template <typename T, typename R, int NT>
__global__ __launch_bounds__(NT) void rnorm_fwd_any_kernel(ResidualNormArgs a) {
  __shared__ float red[NT / 64];
  const float n_f = (float)a.N;
  for (int64_t r = blockIdx.x; r < a.M; r += gridDim.x) {
    const T* y = static_cast<const T*>(a.y) + r * a.ldy;
    const R* res = static_cast<const R*>(a.residual);
    if (res) res += r * a.ldr;
    float rs = 1.0f;
    if (a.post) {
      float s = 0.0f;
      each_part<NT>(a.N, [&](int64_t c, auto size) {
        constexpr int n = decltype(size)::value;
        float f[n];
        load_part<n>(y + c, f);
#pragma unroll
        for (int i = 0; i < n; ++i) s = __builtin_fmaf(f[i], f[i], s);
      });
      rs = inv_root(block_sum<NT>(s, red) / n_f + a.eps);
    }
    const float k = row_scale<T>(a, r);
    auto stream = [&](int64_t c, auto size, float* f) {   // the new residual stream
      constexpr int n = decltype(size)::value;
      float e[n], h[n];
      load_part<n>(y + c, f);
      load_gated<n, T>(a, r, c, e);
#pragma unroll
      for (int i = 0; i < n; ++i) h[i] = 0.0f;
      if (res) load_part<n>(res + c, h);
#pragma unroll
      for (int i = 0; i < n; ++i) f[i] = __builtin_fmaf(k * e[i], f[i] * rs, h[i]);
    };
    float rp = 0.0f;
    if (a.pre) {
      float s = 0.0f;
      each_part<NT>(a.N, [&](int64_t c, auto size) {
        constexpr int n = decltype(size)::value;
        float f[n];
        stream(c, size, f);
#pragma unroll
        for (int i = 0; i < n; ++i) s = __builtin_fmaf(f[i], f[i], s);
      });
      rp = inv_root(block_sum<NT>(s, red) / n_f + a.eps);
    }
    each_part<NT>(a.N, [&](int64_t c, auto size) {
      constexpr int n = decltype(size)::value;
      float f[n], w[n];
      stream(c, size, f);
      store_part<n>(static_cast<R*>(a.out) + r * a.ldo + c, f);
      if (a.pre) {
        load_weights<n, T>(a.wq, a.wide, c, 1.0f, w);
#pragma unroll
        for (int i = 0; i < n; ++i) f[i] *= rp * w[i];
        store_part<n>(static_cast<T*>(a.norm) + r * a.ldn + c, f);
      }
    });
    if (threadIdx.x == 0) {
      if (a.post && a.rstd_post) a.rstd_post[r] = rs;
      if (a.pre && a.rstd_pre) a.rstd_pre[r] = rp;
    }
  }
}

// The parts of dout, dnorm, out and y that a thread holds, as fp32 (0 where absent): d = dout,
// dn = dnorm, xh and yh.
template <int n, typename T, typename R> struct GradPart {
  float d[n], dn[n], xh[n], yh[n];
  __device__ inline GradPart(const ResidualNormArgs& a, int64_t r, int64_t c, float rs, float rp) {
#pragma unroll
    for (int i = 0; i < n; ++i) d[i] = dn[i] = xh[i] = 0.0f;
    if (a.dout) load_part<n>(static_cast<const R*>(a.dout) + r * a.lddo + c, d);
    if (a.dnorm) {
      load_part<n>(static_cast<const T*>(a.dnorm) + r * a.lddn + c, dn);
      load_part<n>(static_cast<const R*>(a.out) + r * a.ldo + c, xh);
#pragma unroll
      for (int i = 0; i < n; ++i) xh[i] *= rp;
    }
    load_part<n>(static_cast<const T*>(a.y) + r * a.ldy + c, yh);
#pragma unroll
    for (int i = 0; i < n; ++i) yh[i] *= rs;
  }
};

// stat[2 r] = c, stat[2 r + 1] = sum D yh wp gate / N
template <typename T, typename R, int NT>
__global__ __launch_bounds__(NT) void rnorm_stat_any_kernel(ResidualNormArgs a, float* stat) {
  __shared__ float red[NT / 64];
  for (int64_t r = blockIdx.x; r < a.M; r += gridDim.x) {
    const float rs = a.post ? a.rstd_post[r] : 1.0f, rp = a.dnorm ? a.rstd_pre[r] : 0.0f;
    float s0 = 0.0f, s1 = 0.0f, s2 = 0.0f;
    each_part<NT>(a.N, [&](int64_t c, auto size) {
      constexpr int n = decltype(size)::value;
      const GradPart<n, T, R> p(a, r, c, rs, rp);
      float w[n], e[n];
      load_weights<n, T>(a.wq, a.wide, c, 1.0f, w);
      load_gated<n, T>(a, r, c, e);
#pragma unroll
      for (int i = 0; i < n; ++i) {
        const float h = p.dn[i] * w[i], ye = p.yh[i] * e[i];
        s0 = __builtin_fmaf(h, p.xh[i], s0);
        s1 = __builtin_fmaf(__builtin_fmaf(rp, h, p.d[i]), ye, s1);
        s2 = __builtin_fmaf(p.xh[i], ye, s2);
      }
    });
    const float c = block_sum<NT>(s0, red) / (float)a.N;
    const float t1 = block_sum<NT>(s1, red), t2 = block_sum<NT>(s2, red);
    if (threadIdx.x == 0) {
      stat[2 * r] = c;
      stat[2 * r + 1] = __builtin_fmaf(-rp * c, t2, t1) / (float)a.N;
    }
  }
}

// One partial row [dnorm xh | gate D yh] of fp32 per block of rows; a thread takes 8 columns, or
// the up to 7 at the end.
template <typename T, typename R>
__global__ __launch_bounds__(256) void rnorm_cols_any_kernel(ResidualNormArgs a, const float* stat,
                                                             float* part, int64_t Np,
                                                             int64_t rows) {
  const int64_t c = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8;
  if (c >= a.N) return;
  const int64_t r0 = (int64_t)blockIdx.y * rows, r1 = r0 + rows < a.M ? r0 + rows : a.M;
  part += (int64_t)blockIdx.y * 2 * Np;
  auto columns = [&](int64_t col, auto size) {
    constexpr int n = decltype(size)::value;
    float sq[n], sp[n];
#pragma unroll
    for (int i = 0; i < n; ++i) sq[i] = sp[i] = 0.0f;
    for (int64_t r = r0; r < r1; ++r) {
      const float rs = a.post ? a.rstd_post[r] : 1.0f, rp = a.dnorm ? a.rstd_pre[r] : 0.0f;
      const GradPart<n, T, R> p(a, r, col, rs, rp);
      const float cr = stat[2 * r];
      float w[n], g[n];
      load_weights<n, T>(a.wq, a.wide, col, 1.0f, w);
#pragma unroll
      for (int i = 0; i < n; ++i) g[i] = 1.0f;
      if (a.kind == kGateFull) load_part<n>(static_cast<const T*>(a.gate) + r * a.ldg + col, g);
      const float gr = a.kind == kGateRow ? to_f32(static_cast<const T*>(a.gate)[r * a.ldg]) : 1.0f;
#pragma unroll
      for (int i = 0; i < n; ++i) {
        const float D = p.d[i] + rp * (p.dn[i] * w[i] - p.xh[i] * cr);
        sq[i] = __builtin_fmaf(p.dn[i], p.xh[i], sq[i]);
        sp[i] = __builtin_fmaf(g[i] * gr * D, p.yh[i], sp[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < n; ++i) {
      part[col + i] = sq[i];
      part[Np + col + i] = sp[i];
    }
  };
  if (a.N - c >= 8) {
    columns(c, std::integral_constant<int, 8>());
  } else {
    for (int64_t col = c; col < a.N; ++col) columns(col, std::integral_constant<int, 1>());
  }
}

// dy, dresidual and a row's or element's dgate; `dresidual` may be `dout`.
template <typename T, typename R, int NT>
__global__ __launch_bounds__(NT) void rnorm_apply_any_kernel(ResidualNormArgs a,
                                                             const float* stat) {
  for (int64_t r = blockIdx.x; r < a.M; r += gridDim.x) {
    const float rs = a.post ? a.rstd_post[r] : 1.0f, rp = a.dnorm ? a.rstd_pre[r] : 0.0f;
    const float cr = stat[2 * r], k = row_scale<T>(a, r);
    const float t = a.post ? stat[2 * r + 1] : 0.0f;
    each_part<NT>(a.N, [&](int64_t c, auto size) {
      constexpr int n = decltype(size)::value;
      const GradPart<n, T, R> p(a, r, c, rs, rp);
      float w[n], e[n], D[n], f[n];
      load_weights<n, T>(a.wq, a.wide, c, 1.0f, w);
      load_gated<n, T>(a, r, c, e);
#pragma unroll
      for (int i = 0; i < n; ++i) {
        D[i] = p.d[i] + rp * (p.dn[i] * w[i] - p.xh[i] * cr);
        f[i] = rs * k * (D[i] * e[i] - p.yh[i] * t);
      }
      if (a.dy) store_part<n>(static_cast<T*>(a.dy) + r * a.lddy + c, f);
      if (a.dgate && a.kind == kGateFull) {
        load_weights<n, T>(a.post ? a.wp : nullptr, a.wide, c, 1.0f, e);
#pragma unroll
        for (int i = 0; i < n; ++i) f[i] = a.scale * D[i] * (p.yh[i] * e[i]);
        store_part<n>(static_cast<T*>(a.dgate) + r * a.lddg + c, f);
      }
      if (a.dresidual) store_part<n>(static_cast<R*>(a.dresidual) + r * a.lddr + c, D);
    });
    if (a.dgate && a.kind == kGateRow && threadIdx.x == 0)
      static_cast<T*>(a.dgate)[r * a.lddg] =
          from_f32<T>(a.scale * (stat[2 * r + 1] * (float)a.N));
  }
}

// ------------------------------------------------------------------ rows in registers
// 8 <= N <= 16384 (RowMap): every row is read once.

// 8 elements of a row, all but the first `skip` if they must not be written twice
template <typename T>
__device__ inline void store_chunk(T* p, const float* f, int skip, bool once) {
  if (once && skip > 0) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i >= skip) p[i] = from_f32<T>(f[i]);
    return;
  }
  Chunk<T> c;
  c.narrow(f);
  c.store_stream(p);
}

// Forward.  Workgroups walk over the rows with the next row's loads in flight (2048 of 256 threads, of
// which the registers let 768 to 2048 run at once).  A row that is changed in place and whose end is held twice is written once: without a
// norm no barrier orders the first write before the second read.
template <typename T, typename R, bool FULL, int G, int EC>
__global__ __launch_bounds__(G > 256 ? G : 256) void rnorm_fwd_kernel(ResidualNormArgs a) {
  constexpr int ROWS = G > 256 ? 1 : 256 / G;
  __shared__ float red[2][G > 256 ? G / 64 : 4];
  const int lane = threadIdx.x % G, grp = row_group<G>(), wave0 = grp * (G / 64);
  const RowMap<G, EC> map(lane, a.N);
  const float inv_n = 1.0f / (float)a.N;
  const T* y = static_cast<const T*>(a.y);
  const R* res = static_cast<const R*>(a.residual);
  const T* gate = static_cast<const T*>(a.gate);
  // of one chunk the weights stay in registers, of more they are read again (from cache)
  constexpr bool HELD = EC == 1;
  float wp[HELD ? 8 : 1], wq[HELD ? 8 : 1];
  auto gated = [&](int64_t c, float* f) {
    load_weights<8, T>(a.post ? a.wp : nullptr, a.wide, c, 1.0f, f);
    if (a.kind == kGateChannel) {
      float g[8];
      load_weights<8, T>(a.gate, a.wide, c, 1.0f, g);
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] *= g[i];
    }
  };
  if constexpr (HELD) {
    gated(map.col[0], wp);
    load_weights<8, T>(a.pre ? a.wq : nullptr, a.wide, map.col[0], 1.0f, wq);
  }
  struct Row {
    Chunk<T> y[EC], g[FULL ? EC : 1];
    Chunk<R> r[EC];
  };
  auto load = [&](Row& d, int64_t row) {
#pragma unroll
    for (int j = 0; j < EC; ++j) {
      d.y[j].zero();
      d.r[j].zero();
      if constexpr (FULL) d.g[j].zero();
      if (map.has(j) && row < a.M) {
        d.y[j].load_stream(y + row * a.ldy + map.col[j]);
        if (res) d.r[j].load_stream(res + row * a.ldr + map.col[j]);
        if constexpr (FULL) d.g[j].load_stream(gate + row * a.ldg + map.col[j]);
      }
    }
  };
  const int64_t step = (int64_t)gridDim.x * ROWS;
  int64_t r = (int64_t)blockIdx.x * ROWS + grp;
  int half = 0;
  auto root = [&](float s) {
    s = row_sum<G>(s, red[half], wave0);
    half ^= 1;
    return inv_root(__builtin_fmaf(s, inv_n, a.eps));
  };
  Row cur, next;
  load(cur, r);
  // every thread of the workgroup makes the same number of passes (barriers)
  for (int64_t base = (int64_t)blockIdx.x * ROWS; base < a.M; base += step, r += step) {
    load(next, r + step);
    const bool live = r < a.M;
    const float k = live ? row_scale<T>(a, r) : 0.0f;
    float f[EC][8];
    auto square = [&]() {
      float s = 0.0f;
#pragma unroll
      for (int j = 0; j < EC; ++j) {
        float g[8], q = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) g[i] = f[j][i];
        drop(g, map.skip[j]);
#pragma unroll
        for (int i = 0; i < 8; ++i) q = __builtin_fmaf(g[i], g[i], q);
        s += q;
      }
      return s;
    };
#pragma unroll
    for (int j = 0; j < EC; ++j) cur.y[j].widen(f[j]);
    float rs = 1.0f, rp = 0.0f;
    if (a.post) rs = root(square());
#pragma unroll
    for (int j = 0; j < EC; ++j) {
      float e[8], h[8];
      if constexpr (HELD) {
#pragma unroll
        for (int i = 0; i < 8; ++i) e[i] = wp[i];
      } else {
        gated(map.col[j], e);
      }
      if constexpr (FULL) {
        cur.g[j].widen(h);
#pragma unroll
        for (int i = 0; i < 8; ++i) e[i] *= h[i];
      }
      cur.r[j].widen(h);
#pragma unroll
      for (int i = 0; i < 8; ++i) f[j][i] = __builtin_fmaf(k * e[i], f[j][i] * rs, h[i]);
    }
    if (a.pre) rp = root(square());
    if (live) {
#pragma unroll
      for (int j = 0; j < EC; ++j) {
        if (!map.has(j)) continue;
        store_chunk(static_cast<R*>(a.out) + r * a.ldo + map.col[j], f[j], map.skip[j],
                    a.in_place);
        if (a.pre) {
          float e[8];
          if constexpr (HELD) {
#pragma unroll
            for (int i = 0; i < 8; ++i) e[i] = wq[i];
          } else {
            load_weights<8, T>(a.wq, a.wide, map.col[j], 1.0f, e);
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) e[i] *= f[j][i] * rp;
          store_chunk(static_cast<T*>(a.norm) + r * a.ldn + map.col[j], e, map.skip[j], false);
        }
      }
      if (lane == 0) {
        if (a.post && a.rstd_post) a.rstd_post[r] = rs;
        if (a.pre && a.rstd_pre) a.rstd_pre[r] = rp;
      }
    }
    cur = next;
  }
}

// Backward.  A workgroup of NT threads walks its share of the rows, NT / G at a time; each thread
// keeps the sums dnorm xh and gate D yh of its own columns in registers, and the row groups add
// theirs through LDS at the end, in a fixed order, to one partial row.
template <typename T, typename R, bool FULL, int G, int EC>
__global__ __launch_bounds__(G > 512 ? 1024 : 512) void rnorm_bwd_kernel(ResidualNormArgs a,
                                                                        float* part, int64_t Np) {
  constexpr int NT = G > 512 ? 1024 : 512, ROWS = NT / G;
  __shared__ float red[2][3][NT / 64];
  __shared__ float sums[ROWS > 1 ? NT * EC * 8 : 1];
  const int lane = threadIdx.x % G, grp = row_group<G>(), wave0 = grp * (G / 64);
  const RowMap<G, EC> map(lane, a.N);
  constexpr bool HELD = NT == 512;   // weights in registers, the next row's loads ahead
  float wp[HELD ? EC : 1][8], wq[HELD ? EC : 1][8], sq[EC][8], sp[EC][8];
  auto gated = [&](int64_t c, float* f) {
    load_weights<8, T>(a.post ? a.wp : nullptr, a.wide, c, 1.0f, f);
    if (a.kind == kGateChannel) {
      float g[8];
      load_weights<8, T>(a.gate, a.wide, c, 1.0f, g);
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] *= g[i];
    }
  };
#pragma unroll
  for (int j = 0; j < EC; ++j) {
    if constexpr (HELD) {
      gated(map.col[j], wp[j]);
      load_weights<8, T>(a.wq, a.wide, map.col[j], 1.0f, wq[j]);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) sq[j][i] = sp[j][i] = 0.0f;
  }
  const float inv_n = 1.0f / (float)a.N;
  struct Row {
    Chunk<T> dn[EC], y[EC], g[FULL ? EC : 1];
    Chunk<R> d[EC], o[EC];
    float rs, rp, gr;
  };
  auto load = [&](Row& q, int64_t row) {
#pragma unroll
    for (int j = 0; j < EC; ++j) {
      q.dn[j].zero();
      q.y[j].zero();
      q.d[j].zero();
      q.o[j].zero();
      if constexpr (FULL) q.g[j].zero();
      if (map.has(j) && row < a.M) {
        const int c = map.col[j];
        if (a.dnorm) {
          q.dn[j].load_stream(static_cast<const T*>(a.dnorm) + row * a.lddn + c);
          q.o[j].load_stream(static_cast<const R*>(a.out) + row * a.ldo + c);
        }
        q.y[j].load_stream(static_cast<const T*>(a.y) + row * a.ldy + c);
        if (a.dout) q.d[j].load_stream(static_cast<const R*>(a.dout) + row * a.lddo + c);
        if constexpr (FULL)
          q.g[j].load_stream(static_cast<const T*>(a.gate) + row * a.ldg + c);
      }
    }
    const bool live = row < a.M;
    q.rs = live && a.post ? a.rstd_post[row] : 1.0f;
    q.rp = live && a.dnorm ? a.rstd_pre[row] : 0.0f;
    q.gr = live && a.kind == kGateRow ? to_f32(static_cast<const T*>(a.gate)[row * a.ldg]) : 1.0f;
  };
  const int64_t step = (int64_t)gridDim.x * ROWS;
  int64_t r = (int64_t)blockIdx.x * ROWS + grp;
  int half = 0;
  Row cur, next;
  if (HELD) load(cur, r);
  for (int64_t base = (int64_t)blockIdx.x * ROWS; base < a.M; base += step, r += step) {
    if (HELD) load(next, r + step);
    else load(cur, r);
    const bool live = r < a.M;
    const float rs = cur.rs, rp = cur.rp;
    // one chunk's values: d = dout, dn, xh, yh, w = wq, e = wp and the gate along the row
    struct Part {
      float d[8], dn[8], xh[8], yh[8], w[8], e[8], g[8];
    };
    auto chunk = [&](int j, Part& p) {
      cur.d[j].widen(p.d);
      cur.dn[j].widen(p.dn);
      cur.o[j].widen(p.xh);
      cur.y[j].widen(p.yh);
      if constexpr (HELD) {
#pragma unroll
        for (int i = 0; i < 8; ++i) p.w[i] = wq[j][i], p.e[i] = wp[j][i];
      } else {
        load_weights<8, T>(a.wq, a.wide, map.col[j], 1.0f, p.w);
        gated(map.col[j], p.e);
      }
      if constexpr (FULL) cur.g[j].widen(p.g);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        p.xh[i] *= rp;
        p.yh[i] *= rs;
        if constexpr (!FULL) p.g[i] = 1.0f;
      }
    };
    float s0 = 0.0f, s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int j = 0; j < EC; ++j) {
      Part p;
      chunk(j, p);
      float h[8], ye[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        h[i] = p.dn[i] * p.w[i];
        ye[i] = p.yh[i] * (p.e[i] * p.g[i]);
        sq[j][i] = __builtin_fmaf(p.dn[i], p.xh[i], sq[j][i]);
      }
      drop(h, map.skip[j]);
      drop(ye, map.skip[j]);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        s0 = __builtin_fmaf(h[i], p.xh[i], s0);
        s1 = __builtin_fmaf(__builtin_fmaf(rp, h[i], p.d[i]), ye[i], s1);
        s2 = __builtin_fmaf(p.xh[i], ye[i], s2);
      }
    }
    constexpr int L = G < 64 ? G : 64;
    s0 = lanes_sum<L>(s0);
    s1 = lanes_sum<L>(s1);
    s2 = lanes_sum<L>(s2);
    if constexpr (G > 64) {
      if ((threadIdx.x & 63) == 0) {
        red[half][0][threadIdx.x >> 6] = s0;
        red[half][1][threadIdx.x >> 6] = s1;
        red[half][2][threadIdx.x >> 6] = s2;
      }
      __syncthreads();
      s0 = s1 = s2 = 0.0f;
#pragma unroll
      for (int i = 0; i < G / 64; ++i) {
        s0 += red[half][0][wave0 + i];
        s1 += red[half][1][wave0 + i];
        s2 += red[half][2][wave0 + i];
      }
      half ^= 1;
    }
    const float c = s0 * inv_n, total = __builtin_fmaf(-rp * c, s2, s1);
    const float t = a.post ? total * inv_n : 0.0f;
    const float k = rs * a.scale * cur.gr;
#pragma unroll
    for (int j = 0; j < EC; ++j) {
      Part p;
      chunk(j, p);
      float D[8], f[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        D[i] = __builtin_fmaf(rp, p.dn[i] * p.w[i] - p.xh[i] * c, p.d[i]);
        sp[j][i] = __builtin_fmaf(D[i] * (p.g[i] * cur.gr), p.yh[i], sp[j][i]);
        f[i] = k * (D[i] * (p.e[i] * p.g[i]) - p.yh[i] * t);
      }
      if (!live || !map.has(j)) continue;
      if (a.dy)
        store_chunk(static_cast<T*>(a.dy) + r * a.lddy + map.col[j], f, map.skip[j], false);
      if (a.dresidual)
        store_chunk(static_cast<R*>(a.dresidual) + r * a.lddr + map.col[j], D, map.skip[j],
                    a.in_place);
      if constexpr (FULL) {
        if (a.dgate) {
#pragma unroll
          for (int i = 0; i < 8; ++i) f[i] = a.scale * D[i] * (p.yh[i] * p.e[i]);
          store_chunk(static_cast<T*>(a.dgate) + r * a.lddg + map.col[j], f, map.skip[j], false);
        }
      }
    }
    if (a.kind == kGateRow && a.dgate && live && lane == 0)
      static_cast<T*>(a.dgate)[r * a.lddg] = from_f32<T>(a.scale * total);
    if (HELD) cur = next;
  }
  if (part == nullptr) return;
  // the row groups' sums, group by group; each thread of the first group ends with its columns'
  if constexpr (ROWS > 1) {
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      __syncthreads();
#pragma unroll
      for (int j = 0; j < EC; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i)
          sums[(j * 8 + i) * NT + threadIdx.x] = which ? sp[j][i] : sq[j][i];
      __syncthreads();
      // G * EC * 8 column sums over NT threads
      constexpr int COLS = G * EC * 8, Q = (COLS + NT - 1) / NT;
      float total[Q];
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        const int e = q * NT + threadIdx.x;
        total[q] = 0.0f;
        if (COLS % NT == 0 || e < COLS) {
          for (int g = 0; g < ROWS; ++g) total[q] += sums[(e / G) * NT + g * G + e % G];
        }
      }
      __syncthreads();
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        const int e = q * NT + threadIdx.x;
        if (COLS % NT == 0 || e < COLS) sums[e] = total[q];
      }
      __syncthreads();
      if (grp == 0) {
#pragma unroll
        for (int j = 0; j < EC; ++j)
#pragma unroll
          for (int i = 0; i < 8; ++i) (which ? sp : sq)[j][i] = sums[(j * 8 + i) * G + lane];
      }
    }
    if (grp != 0) return;
  }
  float* pq = part + (int64_t)blockIdx.x * 2 * Np;
#pragma unroll
  for (int j = 0; j < EC; ++j) {
    if (map.skip[j] == 0) {   // a whole chunk: columns 8 n, 16-byte aligned
      f32x4* q4 = reinterpret_cast<f32x4*>(pq + map.col[j]);
      f32x4* p4 = reinterpret_cast<f32x4*>(pq + Np + map.col[j]);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        q4[i] = f32x4{sq[j][4 * i], sq[j][4 * i + 1], sq[j][4 * i + 2], sq[j][4 * i + 3]};
        p4[i] = f32x4{sp[j][4 * i], sp[j][4 * i + 1], sp[j][4 * i + 2], sp[j][4 * i + 3]};
      }
      continue;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (i < map.skip[j]) continue;
      pq[map.col[j] + i] = sq[j][i];
      pq[Np + map.col[j] + i] = sp[j][i];
    }
  }
}

// Sums the partial rows (16 groups of 4 columns to a workgroup, 16 threads a group) and forms the
// weights' gradients: dwq = S0, dwp = scale gate S1, dgate = scale wp S1 (a gate of the columns).
template <typename T>
__global__ __launch_bounds__(256) void rnorm_finalize_kernel(ResidualNormArgs a, const float* part,
                                                             int64_t nparts, int64_t Np) {
  constexpr int Q = 16, P = 256 / Q;
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
  if (e >= 2 * Np || col >= a.N) return;
  const float v = red[0][threadIdx.x >> 2][threadIdx.x & 3];
  auto put = [&](void* dst, float x) {
    if (!dst) return;
    if (a.wide) {
      float* p = static_cast<float*>(dst) + col;
      *p = a.accumulate ? *p + x : x;
    } else {
      T* p = static_cast<T*>(dst) + col;
      *p = from_f32<T>(a.accumulate ? to_f32(*p) + x : x);
    }
  };
  if (e < Np) {
    put(a.dwq, v);
    return;
  }
  const bool channel = a.kind == kGateChannel;
  float w, g = 1.0f;
  if (channel) load_weights<1, T>(a.gate, a.wide, col, 1.0f, &g);
  load_weights<1, T>(a.post ? a.wp : nullptr, a.wide, col, 1.0f, &w);
  put(a.dwp, a.scale * g * v);
  if (channel) put(a.dgate, a.scale * w * v);
}

template <typename T, typename R>
static hipError_t rnorm_fwd_t(const ResidualNormArgs& a, hipStream_t stream) {
#define SWG_FWD(G, EC)                                                                         \
  do {                                                                                         \
    const dim3 grid(norm_fwd_grid(a.M, G > 256 ? 1 : 256 / G, G > 256 ? G : 256));             \
    const dim3 block(G > 256 ? G : 256);                                                       \
    if (a.kind == kGateFull)                                                                   \
      SWG_TRY(SWG_LAUNCH((rnorm_fwd_kernel<T, R, true, G, EC>), grid, block, 0, stream, a));   \
    else                                                                                       \
      SWG_TRY(SWG_LAUNCH((rnorm_fwd_kernel<T, R, false, G, EC>), grid, block, 0, stream, a));  \
  } while (0)
  if (a.N < 8)
    SWG_TRY(SWG_LAUNCH((rnorm_fwd_any_kernel<T, R, 64>), dim3(row_grid(a.M)), dim3(64), 0, stream,
                       a));
  else if (a.N > 16384)
    SWG_TRY(SWG_LAUNCH((rnorm_fwd_any_kernel<T, R, 512>), dim3(row_grid(a.M)), dim3(512), 0,
                       stream, a));
  else if (a.N <= 64) SWG_FWD(8, 1);
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

template <typename T, typename R>
static hipError_t rnorm_bwd_t(const ResidualNormArgs& a, const ResidualNormPlan& p, float* ws,
                              hipStream_t stream) {
  const bool cols = a.dwp || a.dwq || (a.dgate && a.kind == kGateChannel);
  float* stat = ws;
  float* part = ws + p.stat_floats;
  if (a.M > 0 && p.group == 0) {
    const bool narrow = a.N < 8;
    if (narrow)
      SWG_TRY(SWG_LAUNCH((rnorm_stat_any_kernel<T, R, 64>), dim3(row_grid(a.M)), dim3(64), 0,
                         stream, a, stat));
    else
      SWG_TRY(SWG_LAUNCH((rnorm_stat_any_kernel<T, R, 512>), dim3(row_grid(a.M)), dim3(512), 0,
                         stream, a, stat));
    if (cols)
      SWG_TRY(SWG_LAUNCH((rnorm_cols_any_kernel<T, R>),
                         dim3((unsigned)ceil_div(a.N, 2048), (unsigned)p.parts), dim3(256), 0,
                         stream, a, stat, part, p.np, p.rows));
    if (a.dy || a.dresidual || (a.dgate && a.kind != kGateChannel)) {
      if (narrow)
        SWG_TRY(SWG_LAUNCH((rnorm_apply_any_kernel<T, R, 64>), dim3(row_grid(a.M)), dim3(64), 0,
                           stream, a, stat));
      else
        SWG_TRY(SWG_LAUNCH((rnorm_apply_any_kernel<T, R, 512>), dim3(row_grid(a.M)), dim3(512), 0,
                           stream, a, stat));
    }
  } else if (a.M > 0) {
    float* sums = cols ? part : nullptr;
#define SWG_BWD(G, EC)                                                                        \
  case G * 16 + EC: {                                                                         \
    const dim3 grid((unsigned)p.parts), block(G > 512 ? 1024 : 512);                          \
    if (a.kind == kGateFull)                                                                  \
      SWG_TRY(SWG_LAUNCH((rnorm_bwd_kernel<T, R, true, G, EC>), grid, block, 0, stream, a,    \
                         sums, p.np));                                                        \
    else                                                                                      \
      SWG_TRY(SWG_LAUNCH((rnorm_bwd_kernel<T, R, false, G, EC>), grid, block, 0, stream, a,   \
                         sums, p.np));                                                        \
    break;                                                                                    \
  }
    switch (p.group * 16 + p.chunks) {
      SWG_BWD(8, 1)
      SWG_BWD(16, 1)
      SWG_BWD(32, 1)
      SWG_BWD(64, 1)
      SWG_BWD(128, 1)
      SWG_BWD(128, 2)
      SWG_BWD(256, 2)
      SWG_BWD(512, 2)
      SWG_BWD(1024, 2)
    }
#undef SWG_BWD
  }
  if (!cols) return hipSuccess;
  // M = 0: no partial rows, the empty sums
  const int64_t np = ceil_div(a.N, 4) * 4, parts = a.M > 0 ? p.parts : 0;
  SWG_TRY(SWG_LAUNCH((rnorm_finalize_kernel<T>), wide_grid(ceil_div(2 * np, 64)), dim3(256), 0, stream,
                     a, part, parts, np));
  return hipSuccess;
}

hipError_t launch_residual_norm_fwd(int dtype, int rdtype, const ResidualNormArgs& a,
                                    hipStream_t stream) {
  if (dtype == 2) return rnorm_fwd_t<float, float>(a, stream);
  if (rdtype == 2)
    return dtype == 0 ? rnorm_fwd_t<bf16, float>(a, stream) : rnorm_fwd_t<fp16, float>(a, stream);
  return dtype == 0 ? rnorm_fwd_t<bf16, bf16>(a, stream) : rnorm_fwd_t<fp16, fp16>(a, stream);
}

hipError_t launch_residual_norm_bwd(int dtype, int rdtype, const ResidualNormArgs& a,
                                    const ResidualNormPlan& p, float* ws, hipStream_t stream) {
  if (dtype == 2) return rnorm_bwd_t<float, float>(a, p, ws, stream);
  if (rdtype == 2)
    return dtype == 0 ? rnorm_bwd_t<bf16, float>(a, p, ws, stream)
                      : rnorm_bwd_t<fp16, float>(a, p, ws, stream);
  return dtype == 0 ? rnorm_bwd_t<bf16, bf16>(a, p, ws, stream)
                    : rnorm_bwd_t<fp16, fp16>(a, p, ws, stream);
}

}  // namespace swg
