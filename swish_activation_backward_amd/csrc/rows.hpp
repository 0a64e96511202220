// Device helpers of the row operators (layer norm, token log probabilities, distillation):
// reductions over a wave and a workgroup in a fixed order, and the keys that order logits.
#pragma once

#include "common.hpp"

namespace swg {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ inline float neg_inf() { return -__builtin_inff(); }

// 8 consecutive elements of a row at any element alignment: one 16-byte vector (16-bit types)
// or two (fp32).  Unaligned vector accesses are legal in global memory on this target.
typedef u32x4 u32x4_el2 __attribute__((aligned(2)));
typedef u32x4 u32x4_el4 __attribute__((aligned(4)));
template <typename T> struct ElVec { typedef u32x4_el2 type; };
template <> struct ElVec<float> { typedef u32x4_el4 type; };

template <typename T> struct Chunk {
  static constexpr int NV = sizeof(T) / 2;        // 16-byte vectors
  u32x4 v[NV];
  __device__ inline void load(const T* p) {
    const typename ElVec<T>::type* q = reinterpret_cast<const typename ElVec<T>::type*>(p);
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] = q[i];
  }
  __device__ inline void load_stream(const T* p) {
    const typename ElVec<T>::type* q = reinterpret_cast<const typename ElVec<T>::type*>(p);
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] = __builtin_nontemporal_load(q + i);
  }
  __device__ inline void store_stream(T* p) const {
    typename ElVec<T>::type* q = reinterpret_cast<typename ElVec<T>::type*>(p);
#pragma unroll
    for (int i = 0; i < NV; ++i) __builtin_nontemporal_store(v[i], q + i);
  }
  __device__ inline void zero() {
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] = u32x4{0, 0, 0, 0};
  }
  // the compiler no longer knows the contents, so that nothing computed from them stays in
  // registers for a later use
  __device__ inline void forget() {
#pragma unroll
    for (int i = 0; i < NV; ++i) asm volatile("" : "+v"(v[i]));
  }
  __device__ inline void widen(float* f) const {
#pragma unroll
    for (int i = 0; i < NV; ++i) Vec16<T>::widen(v[i], f + i * Vec16<T>::VEC);
  }
  __device__ inline void narrow(const float* f) {
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] = Vec16<T>::narrow(f + i * Vec16<T>::VEC);
  }
};

// Exchanges between the lanes of a wave without LDS: DPP within 16 lanes, the gfx950 row and
// half swaps across them.  After step n (n = 1, 2, 4, ...) every group of 2n lanes holds the
// value combined over the group, so the mirrored permutations serve as the xor of 4 and 8.
template <int CTRL> __device__ inline float dpp(float v) {
  return __uint_as_float(
      __builtin_amdgcn_update_dpp(0, __float_as_uint(v), CTRL, 0xf, 0xf, true));
}
struct AddOp {
  __device__ inline float operator()(float a, float b) const { return a + b; }
};
struct MaxOp {
  __device__ inline float operator()(float a, float b) const { return __builtin_fmaxf(a, b); }
};
template <int G, typename Op> __device__ inline float lanes_reduce(float v, Op op) {
  if constexpr (G >= 2) v = op(v, dpp<0xB1>(v));
  if constexpr (G >= 4) v = op(v, dpp<0x4E>(v));
  if constexpr (G >= 8) v = op(v, dpp<0x141>(v));
  if constexpr (G >= 16) v = op(v, dpp<0x140>(v));
  if constexpr (G >= 32) {
    const uint32_t u = __float_as_uint(v);
    const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    v = op(__uint_as_float(r[0]), __uint_as_float(r[1]));
  }
  if constexpr (G >= 64) {
    const uint32_t u = __float_as_uint(v);
    const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    v = op(__uint_as_float(r[0]), __uint_as_float(r[1]));
  }
  return v;
}
// Over groups of G <= 64 consecutive lanes, the same value in every lane of the group.
template <int G> __device__ inline float lanes_sum(float v) { return lanes_reduce<G>(v, AddOp()); }
template <int G> __device__ inline float lanes_max(float v) { return lanes_reduce<G>(v, MaxOp()); }

__device__ inline float wave_sum(float v) { return lanes_sum<64>(v); }
__device__ inline float wave_max(float v) { return lanes_max<64>(v); }

// Sum and maximum over the workgroup, the same value in every thread.  `red` holds at least
// blockDim.x / 64 floats and may be used again after the call.
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
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ inline float key_value(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}
__device__ inline u64 entry_key(float v, uint32_t index) {
  return ((u64)value_key(v) << 32) | (u64)(~index);
}
__device__ inline uint32_t key_index(u64 k) { return ~(uint32_t)k; }

}  // namespace swg
