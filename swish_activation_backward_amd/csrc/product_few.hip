// The linear layer's product for a few rows (a token's, or some users' at once) and a weight whose
// contraction index is contiguous: C[p, q] = sum over r of A(p, r) B(q, r), both deep, P <= 16.
//
// Bound by reading B once, and where that takes 10 us and less by the launches and the latencies, so
// that nothing is split over workgroups and joined: a workgroup takes 16 columns q over the whole
// contraction.  Its 16 waves take turns at runs of 128 contraction indices (64 of fp32), each lane
// loading straight into the operands of 16 x 16 matrix instructions (lane l: row l % 16, the 16 bytes
// of indices at l / 16 of every fourth), and their sums meet in LDS in the waves' order.  A comes
// from the caches.  Rows at any alignment.
//
// Measured, bf16, one row: 4096 x 4096 6.8 us = 4.9 TB/s (the tiles with their join 12.1), 1024 x
// 1024 3.2 us (9.1); 16 rows 10.2 (12.9) and 3.8 (9.6).  fp32, one row: 4096 x 14336 48 us = 4.9
// TB/s (78).  4 waves to a workgroup: 4096 x 4096 8.3 us; 32 columns to one, which halves the reads
// of A: 10.2 us, and from 8192 columns on 18 against 20 us at 16 rows and 15 against 14 at one.
#include "product.hpp"

namespace swg {

namespace {

constexpr int kFewWaves = 16;

template <typename T> struct Few;
template <> struct Few<bf16> {
  static constexpr int VEC = 8;   // contraction indices of a lane's 16 bytes
  __device__ static inline f32x4 mma(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  }
};
template <> struct Few<fp16> {
  static constexpr int VEC = 8;
  __device__ static inline f32x4 mma(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(fp16x8, a),
                                                  __builtin_bit_cast(fp16x8, b), c, 0, 0, 0);
  }
};
template <> struct Few<float> {
  static constexpr int VEC = 4;
  // four instructions of four indices: one of each lane's in turn
  __device__ static inline f32x4 mma(u32x4 a, u32x4 b, f32x4 c) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a[e]), __uint_as_float(b[e]), c, 0, 0,
                                               0);
    return c;
  }
};

// 16 bytes of a row from index r on; what lies past its end R is 0 and not read
template <typename T> __device__ inline u32x4 row_end(const T* row, int r, int R) {
  constexpr int V = Few<T>::VEC;
  if (r + V <= R) return *reinterpret_cast<const typename ElVec<T>::type*>(row + r);
  float f[V];
#pragma unroll
  for (int e = 0; e < V; ++e) f[e] = r + e < R ? to_f32(row[r + e]) : 0.0f;
  return Vec16<T>::narrow(f);
}

template <typename T>
__global__ __launch_bounds__(64 * kFewWaves) void few_kernel(Product g) {
  constexpr int V = Few<T>::VEC, STEP = 4 * V, UN = 4, RUN = UN * STEP, WAVES = kFewWaves;
  __shared__ float red[WAVES][16][17];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t q0 = (int64_t)blockIdx.x * 16;
  const int i = lane & 15, at = (lane >> 4) * V;
  const int R = (int)g.R;
  // rows that do not exist repeat the last one: what they give is dropped
  const T* a = static_cast<const T*>(g.a.p) + (i < g.P ? i : g.P - 1) * g.a.ld;
  const T* b = static_cast<const T*>(g.b.p) + (q0 + i < g.Q ? q0 + i : g.Q - 1) * g.b.ld;
  f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
  typedef typename ElVec<T>::type vec;
  const int whole = R / RUN * RUN;
  int r = wave * RUN;
  for (; r < whole; r += WAVES * RUN) {
    u32x4 fa[UN], fb[UN];
#pragma unroll
    for (int u = 0; u < UN; ++u)
      fb[u] = __builtin_nontemporal_load(reinterpret_cast<const vec*>(b + r + u * STEP + at));
#pragma unroll
    for (int u = 0; u < UN; ++u) fa[u] = *reinterpret_cast<const vec*>(a + r + u * STEP + at);
#pragma unroll
    for (int u = 0; u < UN; ++u) acc = Few<T>::mma(fa[u], fb[u], acc);
  }
  if (r == whole)   // the wave whose turn it is takes the rest
    for (int s = whole; s < R; s += STEP)
      acc = Few<T>::mma(row_end(a, s + at, R), row_end(b, s + at, R), acc);
  // register e of lane l: row 4 (l / 16) + e, column l % 16
#pragma unroll
  for (int e = 0; e < 4; ++e) red[wave][4 * (lane >> 4) + e][i] = acc[e];
  __syncthreads();
  const int p = threadIdx.x / 16, c = threadIdx.x % 16;
  if (p >= g.P || q0 + c >= g.Q) return;
  float v = red[0][p][c];
#pragma unroll
  for (int w = 1; w < WAVES; ++w) v += red[w][p][c];
  finish<1, T>(g, p, q0 + c, &v);
}

template <typename T> hipError_t few_t(const Product& g, hipStream_t stream) {
  const dim3 grid((unsigned)ceil_div(g.Q, 16)), block(64 * kFewWaves);
  SWG_LAUNCH(few_kernel<T>, grid, block, 0, stream, g);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_product_few(int dtype, const Product& g, hipStream_t stream) {
  if (dtype == 0) return few_t<bf16>(g, stream);
  if (dtype == 1) return few_t<fp16>(g, stream);
  return few_t<float>(g, stream);
}

}  // namespace swg
