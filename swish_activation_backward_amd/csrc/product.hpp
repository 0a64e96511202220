// The epilogue of the linear layer's products, shared by their kernels.
#pragma once

#include "activation.hpp"
#include "launch.hpp"
#include "rows.hpp"

namespace swg {

// n consecutive outputs (1 or 8) of row p from column q on, from their fp32 sums.
template <int n, typename T>
__device__ inline void finish(const Product& a, int64_t p, int64_t q, float* v) {
  float f[n];
  if (a.bias) {
    load_part<n>(static_cast<const T*>(a.bias) + q, f);
#pragma unroll
    for (int i = 0; i < n; ++i) v[i] += f[i];
  }
  if (a.z) store_part<n>(static_cast<T*>(a.z) + p * a.ldz + q, v);
  if (a.act != kActNone) {
#pragma unroll
    for (int i = 0; i < n; ++i) v[i] = activate(a.act, a.beta, v[i]);
  }
  T* out = static_cast<T*>(a.out) + p * a.ldo + q;
  if (a.residual || a.accumulate) {
    load_part<n>(a.accumulate ? out : static_cast<const T*>(a.residual) + p * a.ldr + q, f);
#pragma unroll
    for (int i = 0; i < n; ++i) v[i] += f[i];
  }
  store_part<n>(out, v);
}

// up to 8 of them
template <typename T>
__device__ inline void finish_chunk(const Product& a, int64_t p, int64_t q, float* v) {
  if (q + 8 <= a.Q) {
    finish<8, T>(a, p, q, v);
  } else {
    const int left = (int)(a.Q - q);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < left) finish<1, T>(a, p, q + i, v + i);
  }
}

}  // namespace swg
