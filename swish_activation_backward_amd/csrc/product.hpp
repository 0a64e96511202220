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

// ---- pieces of work
constexpr int kDepth = 32;   // contraction indices of a stage

// A piece of work: a tile and a range of the contraction.
struct ProductItem {
  int split, p0, q0, begin, end, stages;
};

struct ProductGrid {     // tiles, group of tile rows, ranges of `len`, items
  uint32_t np, nq, group, tiles, items;
  int64_t len;
};

// Tiles run down `group` tile rows before they move on a column, so that those that run at once on
// an XCD (consecutive ones) share rows and columns alike.
template <int P, int ROUND>
__device__ inline ProductItem product_item(const ProductGrid& g, uint32_t L, bool live, int64_t R) {
  ProductItem t;
  const uint32_t l = live ? L : 0;
  const uint32_t split = l / g.tiles, tile = l % g.tiles;
  const uint32_t full = g.group * g.nq, band = tile / full, in = tile % full;
  const uint32_t first = band * g.group;
  const uint32_t rows = g.np - first < g.group ? g.np - first : g.group;
  const int64_t b = split * g.len, e = b + g.len < R ? b + g.len : R;
  t.split = __builtin_amdgcn_readfirstlane((int)split);
  t.p0 = __builtin_amdgcn_readfirstlane((int)(first + in % rows) * P);
  t.q0 = __builtin_amdgcn_readfirstlane((int)(in / rows) * P);
  t.begin = __builtin_amdgcn_readfirstlane((int)b);
  // nothing to fetch past the last item
  t.end = __builtin_amdgcn_readfirstlane(live ? (int)e : (int)b);
  // whole rounds (of the LDS ring), one at least
  int n = (int)((e - b + ROUND - 1) / ROUND) * (ROUND / kDepth);
  if (n < ROUND / kDepth) n = ROUND / kDepth;
  t.stages = __builtin_amdgcn_readfirstlane(n);
  return t;
}

inline ProductGrid product_grid(const ProductPlan& p) {
  ProductGrid g;
  g.np = (uint32_t)p.np;
  g.nq = (uint32_t)p.nq;
  g.group = 4;
  g.tiles = (uint32_t)(p.np * p.nq);
  g.items = (uint32_t)(p.np * p.nq * p.splits);
  g.len = p.len;
  return g;
}

// ---- the way out through LDS
// Float (row, column) of a block in the wave's part of LDS.  Rows 4 apart, which the two halves of
// a wave write at once, use different banks.
template <int W> __device__ inline int out_at(int row, int col) {
  return (row * W + col) ^ (((row >> 2) & 1) << 5);
}

// 32 x 32 sums of one MFMA tile into columns c0 .. of the block: out_at of their rows and columns,
// two lane addresses and constants
template <int W>
__device__ __attribute__((always_inline)) inline void put_tile(const f32x16 v, float* out, int lane, int c0) {
#pragma unroll
  for (int r = 0; r < 16; ++r)
    out[out_at<W>(8 * (r >> 2) + 4 * (lane >> 5) + (r & 3), c0 + (lane & 31))] = v[r];
}

// ---- joining partial sums
// out from the `splits` partial sums, in order; a thread takes 8 columns of a row.
template <typename T>
__global__ __launch_bounds__(256) void product_join_kernel(Product g, const float* part,
                                                           int64_t splits, int64_t ldp,
                                                           int64_t chunks) {
  const int64_t total = g.P * chunks, plane = g.P * ldp;
  for (int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x; e < total;
       e += (int64_t)gridDim.x * 256) {
    const int64_t p = e / chunks, q = (e % chunks) * 8;
    const float* src = part + p * ldp + q;
    f32x4 lo = *reinterpret_cast<const f32x4*>(src), hi = *reinterpret_cast<const f32x4*>(src + 4);
    for (int64_t s = 1; s < splits; ++s) {
      lo += *reinterpret_cast<const f32x4*>(src + s * plane);
      hi += *reinterpret_cast<const f32x4*>(src + s * plane + 4);
    }
    float v[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = lo[i], v[4 + i] = hi[i];
    finish_chunk<T>(g, p, q, v);
  }
}

inline unsigned stream_grid(int64_t items) {
  const int64_t n = ceil_div(items, 256);
  return (unsigned)(n < kMaxStreamBlocks ? n : kMaxStreamBlocks);
}

template <typename T>
inline hipError_t product_join(const Product& g, const ProductPlan& p, const float* part,
                               hipStream_t stream) {
  const int64_t chunks = ceil_div(g.Q, 8);
  SWG_LAUNCH((product_join_kernel<T>), dim3(stream_grid(g.P * chunks)), dim3(256), 0, stream, g,
             part, p.splits, p.ldp, chunks);
  return hipGetLastError();
}

}  // namespace swg
