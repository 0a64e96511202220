// Linear layer with its epilogue: z = x W + b, y = act(z) + residual, and its gradients
// dz = dy act'(z), dx = dz W^T, dW (+)= x^T dz, db (+)= sum over rows of dz.
//
// All three products are C[p, q] = sum_r A(p, r) B(q, r); an operand lies with its contraction
// index contiguous (A[p ld + r]) or its rows (A[r ld + p]).
#include "product.hpp"

namespace swg {

#define SWG_TRY(EXPR)                          \
  do {                                         \
    EXPR;                                      \
    const hipError_t e_ = hipGetLastError();   \
    if (e_ != hipSuccess) return e_;           \
  } while (0)

// ------------------------------------------------------------------ products
template <typename T>
__global__ __launch_bounds__(256) void product_kernel(Product a, int64_t nq) {
  __shared__ float la[16][65], lb[16][65];
  const int64_t p0 = (int64_t)(blockIdx.x / nq) * 64, q0 = (int64_t)(blockIdx.x % nq) * 64;
  const int tp = threadIdx.x / 16, tq = threadIdx.x % 16;
  float acc[4][4] = {};
  auto at = [](const Operand& o, int64_t row, int64_t r) {
    return to_f32(static_cast<const T*>(o.p)[o.deep ? row * o.ld + r : r * o.ld + row]);
  };
  for (int64_t r0 = 0; r0 < a.R; r0 += 16) {
    __syncthreads();
    for (int e = threadIdx.x; e < 16 * 64; e += 256) {
      const int ra = a.a.deep ? e % 16 : e / 64, pa = a.a.deep ? e / 16 : e % 64;
      const int rb = a.b.deep ? e % 16 : e / 64, qb = a.b.deep ? e / 16 : e % 64;
      la[ra][pa] = r0 + ra < a.R && p0 + pa < a.P ? at(a.a, p0 + pa, r0 + ra) : 0.0f;
      lb[rb][qb] = r0 + rb < a.R && q0 + qb < a.Q ? at(a.b, q0 + qb, r0 + rb) : 0.0f;
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < 16; ++r)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          acc[i][j] = __builtin_fmaf(la[r][tp + 16 * i], lb[r][tq + 16 * j], acc[i][j]);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t p = p0 + tp + 16 * i, q = q0 + tq + 16 * j;
      if (p < a.P && q < a.Q) finish<1, T>(a, p, q, &acc[i][j]);
    }
}

template <typename T> static hipError_t product_t(const Product& a, hipStream_t stream) {
  const int64_t nq = ceil_div(a.Q, 64), tiles = ceil_div(a.P, 64) * nq;
  SWG_TRY(SWG_LAUNCH((product_kernel<T>), dim3((unsigned)tiles), dim3(256), 0, stream, a, nq));
  return hipSuccess;
}

hipError_t launch_product(int dtype, const Product& a, const ProductPlan& p, void* ws, int cus,
                          hipStream_t stream) {
  if (dtype != 2) return launch_product16(dtype, a, p, ws, cus, stream);
  return product_t<float>(a, stream);
}

// ------------------------------------------------------------------ dz and db
// dz = dy act'(z) rounded to T, the operand of both products; db sums its fp32 values: one partial
// row per block of rows, then those in order.  A thread takes 8 columns, or the up to 7 at the end.
template <typename T>
__global__ __launch_bounds__(256) void act_bwd_kernel(const T* dy, int64_t lddy, const T* z,
                                                      int64_t ldz, T* dz, int64_t lddz, float* part,
                                                      int64_t Np, int64_t M, int64_t N,
                                                      int64_t rows, int act, float beta) {
  const int64_t c = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8;
  if (c >= N) return;
  const int64_t r0 = (int64_t)blockIdx.y * rows, r1 = r0 + rows < M ? r0 + rows : M;
  auto columns = [&](int64_t col, auto size) {
    constexpr int n = decltype(size)::value;
    float s[n];
#pragma unroll
    for (int i = 0; i < n; ++i) s[i] = 0.0f;
    for (int64_t r = r0; r < r1; ++r) {
      float d[n], f[n];
      load_part<n>(dy + r * lddy + col, d);
      if (act != kActNone) {
        load_part<n>(z + r * ldz + col, f);
#pragma unroll
        for (int i = 0; i < n; ++i) d[i] *= activation_slope(act, beta, f[i]);
      }
      if (dz) store_part<n>(dz + r * lddz + col, d);
#pragma unroll
      for (int i = 0; i < n; ++i) s[i] += d[i];
    }
    if (part) {
#pragma unroll
      for (int i = 0; i < n; ++i) part[blockIdx.y * Np + col + i] = s[i];
    }
  };
  if (N - c >= 8) {
    columns(c, std::integral_constant<int, 8>());
    return;
  }
  for (int64_t col = c; col < N; ++col) columns(col, std::integral_constant<int, 1>());
  if (dz) {   // the rest of dz's rows takes part in dx's sums
    for (int64_t r = r0; r < r1; ++r)
      for (int64_t col = N; col < lddz; ++col) dz[r * lddz + col] = from_f32<T>(0.0f);
  }
}

template <typename T>
__global__ __launch_bounds__(256) void bias_finalize_kernel(const float* part, int64_t nparts,
                                                            T* db, int64_t N, int64_t Np,
                                                            bool accumulate) {
  const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (c >= N) return;
  float s = 0.0f;
  for (int64_t p = 0; p < nparts; ++p) s += part[p * Np + c];
  db[c] = from_f32<T>(accumulate ? to_f32(db[c]) + s : s);
}

template <typename T>
static hipError_t act_bwd_t(const ActBwdArgs& a, const ActBwdPlan& p, float* part,
                            hipStream_t stream) {
  if (a.M > 0)
    SWG_TRY(SWG_LAUNCH((act_bwd_kernel<T>), dim3((unsigned)ceil_div(a.N, 2048), (unsigned)p.parts),
                       dim3(256), 0, stream, static_cast<const T*>(a.dy), a.lddy,
                       static_cast<const T*>(a.z), a.ldz, static_cast<T*>(a.dz), a.lddz,
                       a.db ? part : nullptr, p.np, a.M, a.N, p.rows, a.act, a.beta));
  if (!a.db) return hipSuccess;
  SWG_TRY(SWG_LAUNCH((bias_finalize_kernel<T>), dim3((unsigned)ceil_div(a.N, 256)), dim3(256), 0,
                     stream, part, a.M > 0 ? p.parts : 0, static_cast<T*>(a.db), a.N, p.np,
                     a.accumulate));
  return hipSuccess;
}

hipError_t launch_act_bwd(int dtype, const ActBwdArgs& a, const ActBwdPlan& p, float* part,
                          hipStream_t stream) {
  if (dtype == 0) return act_bwd_t<bf16>(a, p, part, stream);
  if (dtype == 1) return act_bwd_t<fp16>(a, p, part, stream);
  return act_bwd_t<float>(a, p, part, stream);
}

}  // namespace swg
