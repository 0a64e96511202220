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

// A piece of work: a tile and a range of the contraction; `tile` counts from the launch's first.
struct ProductItem {
  int split, tile, p0, q0, begin, end, stages;
};

// Tiles of the output (rows, columns, tile rows of a band), those of a launch (from `first` on,
// `tiles` of them), and the ranges that the contraction is cut into for them.
struct ProductGrid {
  uint32_t np, nq, band, first, tiles, items;
  int64_t len;
};

// Tiles run down a band of tile rows before they move on a column, so that those that run at once on
// an XCD (consecutive ones) share rows and columns alike.
template <int P, int ROUND>
__device__ inline ProductItem product_item(const ProductGrid& g, uint32_t L, bool live, int64_t R) {
  ProductItem t;
  const uint32_t l = live ? L : 0;
  const uint32_t split = l / g.tiles, tile = l % g.tiles;
  const uint32_t full = g.band * g.nq, band = (g.first + tile) / full, in = (g.first + tile) % full;
  const uint32_t top = band * g.band;
  const uint32_t rows = g.np - top < g.band ? g.np - top : g.band;
  const int64_t b = split * g.len, e = b + g.len < R ? b + g.len : R;
  t.split = __builtin_amdgcn_readfirstlane((int)split);
  t.tile = __builtin_amdgcn_readfirstlane((int)tile);
  t.p0 = __builtin_amdgcn_readfirstlane((int)(top + in % rows) * P);
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

// The launch of the whole tiles, and of the others.
inline ProductGrid product_grid(const ProductPlan& p, bool whole) {
  ProductGrid g;
  g.np = (uint32_t)p.np;
  g.nq = (uint32_t)p.nq;
  g.band = 4;
  g.first = whole ? 0 : (uint32_t)p.whole;
  g.tiles = (uint32_t)(whole ? p.whole : p.np * p.nq - p.whole);
  g.items = whole ? g.tiles : g.tiles * (uint32_t)p.splits;
  g.len = whole ? p.splits * p.len : p.len;
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
// out from the sums [split][tile][P][P] of tiles of edge P, in order; a thread takes 8 columns of
// one of a tile's first `height` rows (fewer than P exist where there is one tile row).
template <typename T>
__global__ __launch_bounds__(256) void product_join_kernel(Product g, ProductGrid grid, uint32_t P,
                                                           uint32_t height, const float* part,
                                                           int splits) {
  const int64_t plane = (int64_t)grid.tiles * P * P;
  const uint32_t each = height * P / 8, total = grid.tiles * each;
  for (uint32_t e = blockIdx.x * 256 + threadIdx.x; e < total; e += gridDim.x * 256) {
    const uint32_t tile = e / each, in = e % each;
    const uint32_t full = grid.band * grid.nq, band = (grid.first + tile) / full;
    const uint32_t at = (grid.first + tile) % full, top = band * grid.band;
    const uint32_t rows = grid.np - top < grid.band ? grid.np - top : grid.band;
    const int64_t p = (int64_t)(top + at % rows) * P + in / (P / 8);
    const int64_t q = (int64_t)(at / rows) * P + in % (P / 8) * 8;
    if (p >= g.P || q >= g.Q) continue;
    const float* src = part + (int64_t)tile * P * P + in * 8;
    f32x4 lo = *reinterpret_cast<const f32x4*>(src), hi = *reinterpret_cast<const f32x4*>(src + 4);
    int s = 1;
    for (; s + 4 <= splits; s += 4) {   // the loads of four ranges in flight
      f32x4 v[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = *reinterpret_cast<const f32x4*>(src + (s + i) * plane);
        v[2 * i + 1] = *reinterpret_cast<const f32x4*>(src + (s + i) * plane + 4);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) lo += v[2 * i], hi += v[2 * i + 1];
    }
    for (; s < splits; ++s) {
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
inline hipError_t product_join(const Product& g, const ProductPlan& p, const ProductGrid& grid,
                               const float* part, hipStream_t stream) {
  const uint32_t P = (uint32_t)tile_edge(p.f);
  const uint32_t height = p.np == 1 ? (uint32_t)g.P : P;
  SWG_LAUNCH((product_join_kernel<T>), dim3(stream_grid((int64_t)grid.tiles * height * P / 8)),
             dim3(256), 0, stream, g, grid, P, height, part, (int)p.splits);
  return hipGetLastError();
}

// ---- operands laid out again
// rows [n][cols] again with rows of ld elements, zeros up to a multiple of 8; a thread takes 8
// columns
template <typename T>
__global__ __launch_bounds__(256) void pack_kernel(const T* src, int64_t lds, T* dst, int64_t ldd,
                                                   int64_t n, int64_t cols) {
  const int64_t chunks = (cols + 7) / 8, total = n * chunks;
  for (int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x; e < total;
       e += (int64_t)gridDim.x * 256) {
    const int64_t r = e / chunks, c = (e % chunks) * 8;
    Chunk<T> v;
    if (c + 8 <= cols) {
      v.load(src + r * lds + c);
    } else {
      float f[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = c + i < cols ? to_f32(src[r * lds + c + i]) : 0.0f;
      v.narrow(f);
    }
#pragma unroll
    for (int i = 0; i < Chunk<T>::NV; ++i)
      reinterpret_cast<u32x4*>(dst + r * ldd + c)[i] = v.v[i];
  }
}

// An operand again in the workspace with rows of 16-byte multiples
template <typename T>
inline hipError_t pack_operand(Operand& o, int64_t rows, int64_t R, void* to, hipStream_t stream) {
  const int64_t n = o.deep ? rows : R, cols = o.deep ? R : rows, ld = packed_ld(cols);
  SWG_LAUNCH((pack_kernel<T>), dim3(stream_grid(n * ceil_div(cols, 8))), dim3(256), 0, stream,
             static_cast<const T*>(o.p), o.ld, static_cast<T*>(to), ld, n, cols);
  o.p = to;
  o.ld = ld;
  return hipGetLastError();
}

}  // namespace swg
