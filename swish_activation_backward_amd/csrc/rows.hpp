// Device helpers of the row operators (layer norm, token log probabilities, distillation):
// reductions over a wave and a workgroup in a fixed order, and the keys that order logits.
#pragma once

#include "common.hpp"

namespace swg {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ inline float neg_inf() { return -__builtin_inff(); }

// Sum and maximum over the workgroup, the same value in every thread.  `red` holds at least
// blockDim.x / 64 floats and may be used again after the call.
__device__ inline float wave_sum(float v) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d);
  return v;
}

__device__ inline float wave_max(float v) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v = __builtin_fmaxf(v, __shfl_xor(v, d));
  return v;
}

template <int T> __device__ inline float block_sum(float v, float* red) {
  v = wave_sum(v);
  if constexpr (T > 64) {
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    v = red[0];
#pragma unroll
    for (int i = 1; i < T / 64; ++i) v += red[i];
  }
  return v;
}

template <int T> __device__ inline float block_max(float v, float* red) {
  v = wave_max(v);
  if constexpr (T > 64) {
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    v = red[0];
#pragma unroll
    for (int i = 1; i < T / 64; ++i) v = __builtin_fmaxf(v, red[i]);
  }
  return v;
}

// Order of a row's entries: larger value first, equal values by rising index.  The key of
// (value, index) is a 64-bit whole number that compares the same way: the value's bits made
// monotone in the high half (-0 counted as +0, NaN as -inf), the complement of the index in
// the low half.  Keys of one row are distinct, and 0 is below every key.
typedef unsigned long long u64;

__device__ inline uint32_t value_key(float v) {
  v = v == v ? v + 0.0f : neg_inf();
  const uint32_t b = __float_as_uint(v);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ inline float key_value(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}
__device__ inline u64 entry_key(float v, uint32_t index) {
  return ((u64)value_key(v) << 32) | (u64)(~index);
}
__device__ inline uint32_t key_index(u64 k) { return ~(uint32_t)k; }

}  // namespace swg
