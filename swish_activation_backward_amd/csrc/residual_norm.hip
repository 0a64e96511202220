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

// Sums the partial rows (16 groups of 4 columns to a workgroup, 16 threads a group) and forms the
// weights' gradients: dwq = S0, dwp = scale gate S1, dgate = scale wp S1 (a gate of the columns).
template <typename T>
__global__ __launch_bounds__(256) void rnorm_finalize_kernel(ResidualNormArgs a, const float* part,
                                                             int64_t nparts, int64_t Np) {
  constexpr int Q = 16, P = 256 / Q;
  __shared__ f32x4 red[P][Q];
  const int q = threadIdx.x % Q, lane = threadIdx.x / Q;
  const int64_t c = ((int64_t)blockIdx.x * Q + q) * 4;   // column of the 2 Np
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
  const int64_t e = (int64_t)blockIdx.x * 4 * Q + threadIdx.x;
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

#define SWG_TRY(EXPR)                          \
  do {                                         \
    EXPR;                                      \
    const hipError_t e_ = hipGetLastError();   \
    if (e_ != hipSuccess) return e_;           \
  } while (0)

template <typename T, typename R>
static hipError_t rnorm_fwd_t(const ResidualNormArgs& a, hipStream_t stream) {
  if (a.N < 8)
    SWG_TRY(SWG_LAUNCH((rnorm_fwd_any_kernel<T, R, 64>), dim3(row_grid(a.M)), dim3(64), 0, stream,
                       a));
  else
    SWG_TRY(SWG_LAUNCH((rnorm_fwd_any_kernel<T, R, 512>), dim3(row_grid(a.M)), dim3(512), 0,
                       stream, a));
  return hipSuccess;
}

template <typename T, typename R>
static hipError_t rnorm_bwd_t(const ResidualNormArgs& a, const ResidualNormPlan& p, float* ws,
                              hipStream_t stream) {
  const bool cols = a.dwp || a.dwq || (a.dgate && a.kind == kGateChannel);
  float* stat = ws;
  float* part = ws + p.stat_floats;
  if (a.M > 0) {
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
  }
  if (!cols) return hipSuccess;
  // M = 0: no partial rows, the empty sums
  const int64_t np = ceil_div(a.N, 4) * 4, parts = a.M > 0 ? p.parts : 0;
  SWG_TRY(SWG_LAUNCH((rnorm_finalize_kernel<T>), dim3((unsigned)ceil_div(2 * np, 64)), dim3(256), 0,
                     stream, a, part, parts, np));
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
