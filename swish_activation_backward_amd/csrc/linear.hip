// Linear layer with its epilogue: z = x W + b, y = act(z) + residual, and its gradients
// dz = dy act'(z), dx = dz W^T, dW (+)= x^T dz, db (+)= sum over rows of dz.
//
// All three products are C[p, q] = sum_r A(p, r) B(q, r); an operand lies with its contraction
// index contiguous (A[p ld + r]) or its rows (A[r ld + p]).
#include "product.hpp"

namespace swg {

hipError_t launch_product(int dtype, const Product& a, const ProductPlan& p, void* ws, int cus,
                          hipStream_t stream) {
  if (p.few) return launch_product_few(dtype, a, stream);
  if (dtype != 2) return launch_product16(dtype, a, p, ws, cus, stream);
  return launch_product32(a, p, ws, stream);
}

// ------------------------------------------------------------------ dz and db
// dz = dy act'(z) rounded to T, the operand of both products; db sums its fp32 values: one partial
// row per block of rows, then those in order.  A workgroup takes 512 columns, 8 a thread (or the up
// to 7 at the end), 4 rows at once, and a thread has the loads of 4 of its rows in flight.  A pass of
// its own, since both products read dz, one of them across the rows.  Bound by memory: [16384,
// 14336] bf16 280 us = 5.0 TB/s, the sums' second kernel 5 us.
constexpr int kActTx = 64, kActTy = 4, kActFlight = 4;

template <typename T>
__global__ __launch_bounds__(256) void act_bwd_kernel(ActBwdArgs a, float* part, int64_t Np,
                                                      int64_t rows) {
  __shared__ float red[kActTy][kActTx][8];
  const int tx = threadIdx.x % kActTx, ty = threadIdx.x / kActTx;
  const int64_t c = ((int64_t)blockIdx.x * kActTx + tx) * 8;
  const int64_t r0 = (int64_t)blockIdx.y * rows, r1 = r0 + rows < a.M ? r0 + rows : a.M;
  const T* dy = static_cast<const T*>(a.dy);
  const T* z = static_cast<const T*>(a.z);
  T* dz = static_cast<T*>(a.dz);
  float s[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) s[i] = 0.0f;
  if (c < a.N && a.N >= 8) {
    // columns that are no multiple of 8 end with a chunk moved back to the row's end: its first
    // `skip` elements count in the chunk before
    const int64_t at = c + 8 <= a.N ? c : a.N - 8;
    const int skip = (int)(c - at);
    const int64_t pad = skip > 0 && dz ? (a.N + 7) / 8 * 8 : 0;
    for (int64_t r = r0 + ty; r < r1; r += kActTy * kActFlight) {
      Chunk<T> d[kActFlight], f[kActFlight];
#pragma unroll
      for (int k = 0; k < kActFlight; ++k) {
        const int64_t row = r + k * kActTy;
        d[k].zero();
        f[k].zero();
        if (row < r1) {
          d[k].load_stream(dy + row * a.lddy + at);
          if (a.act != kActNone) f[k].load_stream(z + row * a.ldz + at);
        }
      }
#pragma unroll
      for (int k = 0; k < kActFlight; ++k) {
        const int64_t row = r + k * kActTy;
        float g[8], v[8];
        d[k].widen(g);
        if (a.act != kActNone) {
          f[k].widen(v);
#pragma unroll
          for (int i = 0; i < 8; ++i) g[i] *= activation_slope(a.act, a.beta, v[i]);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) s[i] += g[i];
        if (dz && row < r1) {
          Chunk<T> o;
          o.narrow(g);
          o.store_stream(dz + row * a.lddz + at);
          // 0 up to a multiple of 8, which takes part in dx's sums
          for (int64_t e = a.N; e < pad; ++e) dz[row * a.lddz + e] = from_f32<T>(0.0f);
        }
      }
    }
    // to the places of columns c ..
    if (skip > 0) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = s[i];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        s[i] = 0.0f;
#pragma unroll
        for (int k = 0; k < 8; ++k) s[i] = k == i + skip ? v[k] : s[i];
      }
    }
  } else if (c < a.N) {   // fewer than 8 columns
    for (int64_t r = r0 + ty; r < r1; r += kActTy) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float g = 0.0f;
        if (i < a.N) {
          g = to_f32(dy[r * a.lddy + i]);
          if (a.act != kActNone) g *= activation_slope(a.act, a.beta, to_f32(z[r * a.ldz + i]));
        }
        s[i] += g;
        if (dz) dz[r * a.lddz + i] = from_f32<T>(g);
      }
    }
  }
  if (part == nullptr) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) red[ty][tx][i] = s[i];
  __syncthreads();
  for (int e = threadIdx.x; e < kActTx * 8; e += 256) {
    const int64_t col = (int64_t)blockIdx.x * kActTx * 8 + e;
    if (col >= a.N) break;
    const float* p = &red[0][0][0] + e;
    part[blockIdx.y * Np + col] = (p[0] + p[kActTx * 8]) + (p[2 * kActTx * 8] + p[3 * kActTx * 8]);
  }
}

// Sums the partial rows: 4 groups of 4 columns to a workgroup, 64 threads a group.
template <typename T>
__global__ __launch_bounds__(256) void bias_finalize_kernel(const float* part, int64_t nparts,
                                                            T* db, int64_t N, int64_t Np,
                                                            bool accumulate) {
  constexpr int Q = 4, P = 256 / Q;
  __shared__ f32x4 red[P][Q];
  const int q = threadIdx.x % Q, lane = threadIdx.x / Q;
  const int64_t c = ((int64_t)blockIdx.x * Q + q) * 4;
  f32x4 s = {0.0f, 0.0f, 0.0f, 0.0f};
  if (c < Np) {
#pragma unroll 4
    for (int64_t p = lane; p < nparts; p += P)
      s += *reinterpret_cast<const f32x4*>(part + p * Np + c);
  }
  red[lane][q] = s;
  __syncthreads();
  for (int n = P / 2; n > 0; n >>= 1) {
    if (lane < n) red[lane][q] += red[lane + n][q];
    __syncthreads();
  }
  const int64_t col = (int64_t)blockIdx.x * 4 * Q + threadIdx.x;
  if (threadIdx.x >= 4 * Q || col >= N) return;
  const float v = red[0][threadIdx.x >> 2][threadIdx.x & 3];
  db[col] = from_f32<T>(accumulate ? to_f32(db[col]) + v : v);
}

template <typename T>
static hipError_t act_bwd_t(const ActBwdArgs& a, const ActBwdPlan& p, float* part,
                            hipStream_t stream) {
  if (a.M > 0)
    SWG_TRY(SWG_LAUNCH((act_bwd_kernel<T>),
                       dim3((unsigned)ceil_div(a.N, 8 * kActTx), (unsigned)p.parts), dim3(256), 0,
                       stream, a, a.db ? part : nullptr, p.np, p.rows));
  if (!a.db) return hipSuccess;
  SWG_TRY(SWG_LAUNCH((bias_finalize_kernel<T>), dim3((unsigned)ceil_div(a.N, 16)), dim3(256), 0,
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
