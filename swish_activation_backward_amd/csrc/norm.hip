// Layer norm over the rows of [M, N], forward and backward.
//
//   mean = sum x / N,  var = sum (x - mean)^2 / N,  rstd = 1 / sqrt(var + eps)
//   xh = (x - mean) rstd,  y = xh w + b
//   dx = rstd (dy w - c1 - xh c2),  c1 = sum(dy w) / N,  c2 = sum(dy w xh) / N
//   dw = sum over rows of dy xh,  db = sum over rows of dy
//
// Tensors of bf16, fp16 or fp32 (T); w and b of the same type or fp32 (W).  All arithmetic
// and all sums are fp32; each output is rounded once.
#include "launch.hpp"
#include "rows.hpp"

namespace swg {

template <typename T, typename W>
__global__ __launch_bounds__(256) void norm_fwd_kernel(const T* x, int64_t ldx, const W* w,
                                                       const W* b, T* y, int64_t ldy,
                                                       float* mean, float* rstd, int64_t M,
                                                       int64_t N, float eps) {
  __shared__ float red[4];
  for (int64_t r = blockIdx.x; r < M; r += gridDim.x) {
  const T* xr = x + r * ldx;
  float s = 0.0f;
  for (int64_t c = threadIdx.x; c < N; c += 256) s += to_f32(xr[c]);
  const float mu = block_sum<256>(s, red) / (float)N;
  s = 0.0f;
  for (int64_t c = threadIdx.x; c < N; c += 256) {
    const float d = to_f32(xr[c]) - mu;
    s = __builtin_fmaf(d, d, s);
  }
  const float rs = 1.0f / __builtin_sqrtf(block_sum<256>(s, red) / (float)N + eps);
  for (int64_t c = threadIdx.x; c < N; c += 256) {
    float v = (to_f32(xr[c]) - mu) * rs;
    if (w) v *= to_f32(w[c]);
    if (b) v += to_f32(b[c]);
    y[r * ldy + c] = from_f32<T>(v);
  }
  if (threadIdx.x == 0) {
    if (mean) mean[r] = mu;
    if (rstd) rstd[r] = rs;
  }
  }
}

template <typename T, typename W>
__global__ __launch_bounds__(256) void norm_dx_kernel(const T* dy, int64_t lddy, const T* x,
                                                      int64_t ldx, const W* w,
                                                      const float* mean, const float* rstd,
                                                      T* dx, int64_t lddx, int64_t M,
                                                      int64_t N) {
  __shared__ float red[4];
  for (int64_t r = blockIdx.x; r < M; r += gridDim.x) {
  const float mu = mean[r], rs = rstd[r];
  float s1 = 0.0f, s2 = 0.0f;
  for (int64_t c = threadIdx.x; c < N; c += 256) {
    const float h = to_f32(dy[r * lddy + c]) * (w ? to_f32(w[c]) : 1.0f);
    s1 += h;
    s2 = __builtin_fmaf(h, (to_f32(x[r * ldx + c]) - mu) * rs, s2);
  }
  const float c1 = block_sum<256>(s1, red) / (float)N;
  const float c2 = block_sum<256>(s2, red) / (float)N;
  for (int64_t c = threadIdx.x; c < N; c += 256) {
    const float h = to_f32(dy[r * lddy + c]) * (w ? to_f32(w[c]) : 1.0f);
    const float xh = (to_f32(x[r * ldx + c]) - mu) * rs;
    dx[r * lddx + c] = from_f32<T>(rs * (h - c1 - xh * c2));
  }
  }
}

// one partial row [dw | db] of fp32 per block of rows
template <typename T>
__global__ __launch_bounds__(256) void norm_cols_kernel(const T* dy, int64_t lddy, const T* x,
                                                        int64_t ldx, const float* mean,
                                                        const float* rstd, float* part,
                                                        int64_t M, int64_t N, int64_t rows) {
  const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (c >= N) return;
  const int64_t r0 = (int64_t)blockIdx.y * rows, r1 = r0 + rows < M ? r0 + rows : M;
  float sw = 0.0f, sb = 0.0f;
  for (int64_t r = r0; r < r1; ++r) {
    const float d = to_f32(dy[r * lddy + c]);
    sw = __builtin_fmaf(d, (to_f32(x[r * ldx + c]) - mean[r]) * rstd[r], sw);
    sb += d;
  }
  part[(int64_t)blockIdx.y * 2 * N + c] = sw;
  part[(int64_t)blockIdx.y * 2 * N + N + c] = sb;
}

template <typename W>
__global__ __launch_bounds__(256) void norm_finalize_kernel(const float* part, int64_t nparts,
                                                            W* dw, W* db, int64_t N, int acc) {
  const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (c >= 2 * N) return;
  W* dst = c < N ? dw : db;
  if (dst == nullptr) return;
  dst += c < N ? c : c - N;
  float s = 0.0f;
  for (int64_t p = 0; p < nparts; ++p) s += part[p * 2 * N + c];
  *dst = from_f32<W>(acc ? to_f32(*dst) + s : s);
}

template <typename T, typename W>
static hipError_t norm_fwd_t(const NormArgs& a, hipStream_t stream) {
  SWG_LAUNCH((norm_fwd_kernel<T, W>), dim3(row_grid(a.M)), dim3(256), 0, stream,
             static_cast<const T*>(a.x), a.ldx, static_cast<const W*>(a.w),
             static_cast<const W*>(a.b), static_cast<T*>(a.y), a.ldy, a.mean, a.rstd, a.M, a.N,
             a.eps);
  return hipGetLastError();
}

template <typename T, typename W>
static hipError_t norm_bwd_t(const NormArgs& a, const NormPlan& p, float* part,
                             hipStream_t stream) {
  const T* dy = static_cast<const T*>(a.dy);
  const T* x = static_cast<const T*>(a.x);
  if (a.dx && a.M > 0) {
    SWG_LAUNCH((norm_dx_kernel<T, W>), dim3(row_grid(a.M)), dim3(256), 0, stream, dy, a.lddy, x,
               a.ldx, static_cast<const W*>(a.w), a.mean, a.rstd, static_cast<T*>(a.dx), a.lddx,
               a.M, a.N);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (!a.dw && !a.db) return hipSuccess;
  if (p.parts > 0) {   // M = 0: the empty sums
    SWG_LAUNCH((norm_cols_kernel<T>), dim3((unsigned)ceil_div(a.N, 256), (unsigned)p.parts),
               dim3(256), 0, stream, dy, a.lddy, x, a.ldx, a.mean, a.rstd, part, a.M, a.N,
               p.rows);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  SWG_LAUNCH((norm_finalize_kernel<W>), dim3((unsigned)ceil_div(2 * a.N, 256)), dim3(256), 0,
             stream, part, p.parts, static_cast<W*>(a.dw), static_cast<W*>(a.db), a.N,
             a.accumulate);
  return hipGetLastError();
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
