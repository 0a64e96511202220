// The linear layer's product for a few rows (a token's, or some users' at once):
//   C[p, q] = sum over r of A(p, r) B(q, r),  A deep
// with B deep (its contraction index contiguous) and P <= 16, or B flat and P <= 4.
//
// Bound by reading B once, and where that takes 10 us and less by the launches and the latencies, so
// that nothing is split over workgroups and joined: a workgroup takes some columns q over the whole
// contraction, its 16 waves take turns along it, and their sums meet in LDS in the waves' order.  A
// comes from the caches.  Rows at any alignment.
//
// Deep: 16 columns; a wave takes runs of 128 contraction indices (64 of fp32), each lane loading
// straight into the operands of 16 x 16 matrix instructions (lane l: row l % 16, the 16 bytes of
// indices at l / 16 of every fourth).  Measured on the GPU with W in the last cache, where these
// sizes mostly stay, bf16, one row: 4096 x 4096 6.8 us = 4.9 TB/s (the tiles with their join 12.1),
// 1024 x 1024 3.2 us (9.1); 16 rows 10.2 (12.9) and 3.8 (9.6).  With W from memory, each kernel on its
// own, 4096 x 4096 takes 10.4 us (12.7 and 3.9) for one row, 12.6 (12.2 and 3.9) for 16.
// fp32, one row: 4096 x 14336 48 us = 4.9 TB/s (78).  4 waves to a workgroup: 4096 x 4096 8.3 us; 32
// columns to one, which halves the reads of A: 10.2 us, and from 8192 columns on 18 against 20 us at
// 16 rows and 15 against 14 at one.
//
// Flat: 32 columns (16 of fp32), whose rows are half a cache line each: long contractions lose by
// that (4096 x 4096 19.7 us, the tiles 12.7), short ones have no time for a second launch: 1024 x
// 1024 4.4 us (9.6), 1001 x 1003 5.7 (15.9, which lay the weight out again), 1024 x 4096 6.1 (10.6).
// 64 columns: 5.9, 8.4 and 5.9 us; 16: 4.4, 4.8 and 7.0.
#include "product.hpp"

namespace swg {

namespace {

constexpr int kFewWaves = 16, kFlatChunks = 4;

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

// ---- rows of B contiguous
// x[0 .. 8) of a row from index r on, 0 past its end
template <typename T> __device__ inline void row_of_8(const T* row, int64_t r, int64_t R, float* f) {
  if (r + 8 <= R) {
    Chunk<T> c;
    c.load(row + r);
    c.widen(f);
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = r + i < R ? to_f32(row[r + i]) : 0.0f;
}

// At most 4 rows of A, whose products do not fill a matrix instruction: a lane multiplies 16 bytes
// of 8 rows of B, 16 lanes side by side in the contraction (so that their sums add within the
// registers) times 4 in the columns; the 16 waves take turns at runs of 128 rows.
template <typename T, int P>
__global__ __launch_bounds__(64 * kFewWaves) void few_flat_kernel(Product g) {
  constexpr int V = Few<T>::VEC, G = 64 / kFlatChunks, RUN = 8 * G, COLS = kFlatChunks * V;
  typedef typename ElVec<T>::type vec;
  __shared__ float red[kFewWaves][P][COLS];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int grp = lane % G, chunk = lane / G;
  const int64_t q0 = (int64_t)blockIdx.x * COLS, q = q0 + chunk * V;
  // the last chunk of a row is moved back to its end
  const int64_t at = q + V <= g.Q ? q : g.Q - V;
  const T* b = static_cast<const T*>(g.b.p) + at;
  const T* a[P];
#pragma unroll
  for (int p = 0; p < P; ++p)
    a[p] = static_cast<const T*>(g.a.p) + (p < g.P ? p : g.P - 1) * g.a.ld;
  float acc[P][V];
#pragma unroll
  for (int p = 0; p < P; ++p)
#pragma unroll
    for (int i = 0; i < V; ++i) acc[p][i] = 0.0f;
  auto add = [&](const u32x4 (&w)[8], int64_t r) {
    float x[P][8];
#pragma unroll
    for (int p = 0; p < P; ++p) row_of_8(a[p], r, g.R, x[p]);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      float f[V];
      Vec16<T>::widen(w[k], f);
#pragma unroll
      for (int p = 0; p < P; ++p)
#pragma unroll
        for (int i = 0; i < V; ++i) acc[p][i] = __builtin_fmaf(x[p][k], f[i], acc[p][i]);
    }
  };
  const int64_t whole = g.R / RUN * RUN;
  int64_t r = wave * RUN;
  for (; r < whole; r += kFewWaves * RUN) {
    u32x4 w[8];
#pragma unroll
    for (int k = 0; k < 8; ++k)
      w[k] = __builtin_nontemporal_load(
          reinterpret_cast<const vec*>(b + (r + grp * 8 + k) * g.b.ld));
    add(w, r + grp * 8);
  }
  if (r == whole && whole < g.R) {
    u32x4 w[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      w[k] = u32x4{0, 0, 0, 0};
      const int64_t row = r + grp * 8 + k;
      if (row < g.R) w[k] = *reinterpret_cast<const vec*>(b + row * g.b.ld);
    }
    add(w, r + grp * 8);
  }
  // the row groups' sums, then the waves'
#pragma unroll
  for (int p = 0; p < P; ++p)
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float v = lanes_sum<G>(acc[p][i]);
      if (grp == 0) red[wave][p][chunk * V + i] = v;
    }
  __syncthreads();
  for (int e = threadIdx.x; e < P * COLS; e += 64 * kFewWaves) {
    const int p = e / COLS, c = e % COLS;
    if (p >= g.P || q0 + c >= g.Q) continue;
    // the place of column q0 + c: its chunk may have been moved
    const int64_t first = q0 + c / V * V;
    const int back = first + V <= g.Q ? 0 : (int)(first + V - g.Q);
    float v = red[0][p][c + back];
#pragma unroll
    for (int w = 1; w < kFewWaves; ++w) v += red[w][p][c + back];
    finish<1, T>(g, p, q0 + c, &v);
  }
}

template <typename T> hipError_t flat_t(const Product& g, hipStream_t stream) {
  const dim3 grid((unsigned)ceil_div(g.Q, kFlatChunks * Few<T>::VEC)), block(64 * kFewWaves);
  if (g.P == 1) SWG_LAUNCH((few_flat_kernel<T, 1>), grid, block, 0, stream, g);
  else if (g.P == 2) SWG_LAUNCH((few_flat_kernel<T, 2>), grid, block, 0, stream, g);
  else SWG_LAUNCH((few_flat_kernel<T, 4>), grid, block, 0, stream, g);
  return hipGetLastError();
}

template <typename T> hipError_t either(const Product& g, hipStream_t stream) {
  return g.b.deep ? few_t<T>(g, stream) : flat_t<T>(g, stream);
}

}  // namespace

hipError_t launch_product_few(int dtype, const Product& g, hipStream_t stream) {
  if (dtype == 0) return either<bf16>(g, stream);
  if (dtype == 1) return either<fp16>(g, stream);
  return either<float>(g, stream);
}

}  // namespace swg
