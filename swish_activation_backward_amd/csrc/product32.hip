// The linear layer's products for fp32 tensors, on the fp32 matrix instructions
// (v_mfma_f32_32x32x2_f32: a lane supplies row l % 32 and contraction index l / 32):
//   C[p, q] = sum over r of A(p, r) B(q, r)
// with operands of any alignment, deep or flat (see product.hip).
//
// A workgroup of four waves (2 x 2) owns a tile of edge 64 F, each wave 32 F x 32 F outputs.  A
// stage of 32 contraction indices is loaded into registers while the two before it are multiplied,
// and written to the other of two LDS buffers: a deep operand as [row][32], of which a lane reads
// four consecutive indices at once, a flat one as [32][row].  Lane half h takes index 8 j + 4 h + s
// in step s of a group j, of both operands alike.
#include <type_traits>

#include "mma.hpp"
#include "product.hpp"

namespace swg {

namespace {

constexpr int kThreads = 256;

// One operand's part of a stage: V 16-byte vectors a thread.
template <bool DEEP, int F> struct Part {
  static constexpr int P = 64 * F, V = P * kDepth / 4 / kThreads;
  static constexpr int PITCH = DEEP ? kDepth + 4 : P + 4;
  static constexpr int FLOATS = DEEP ? P * PITCH : kDepth * PITCH;
  f32x4 v[V];

  // row and contraction index of vector h
  static __device__ inline int row(int h) {
    return DEEP ? threadIdx.x / 8 + 32 * h : (threadIdx.x % (P / 4)) * 4;
  }
  static __device__ inline int deep(int h) {
    return DEEP ? (threadIdx.x % 8) * 4 : threadIdx.x / (P / 4) + kThreads / (P / 4) * h;
  }

  // The vectors' places in memory, a stage further with every load.
  struct Source {
    const float* q[V];
    int rows[V];      // of the vector's rows, those that exist (deep: 1 or 0)
    int64_t step;
    int left;         // contraction indices
    __device__ inline Source(const float* src, int64_t ld, int64_t row0, int64_t rows_, int begin,
                             int end) {
      left = end - begin;
      step = DEEP ? kDepth : kDepth * ld;
#pragma unroll
      for (int h = 0; h < V; ++h) {
        const int64_t p = row0 + row(h), r = begin + deep(h);
        const int64_t n = rows_ - p, most = DEEP ? 1 : 4;
        rows[h] = (int)(n < 0 ? 0 : n < most ? n : most);
        q[h] = src + (DEEP ? p * ld + r : r * ld + p);
      }
    }
  };

  // 0 past the rows and the contraction's end, where nothing is read
  __device__ inline void load(Source& s) {
#pragma unroll
    for (int h = 0; h < V; ++h) {
      const int along = s.left - deep(h);
      const int n = DEEP ? (s.rows[h] ? along : 0) : (along > 0 ? s.rows[h] : 0);
      v[h] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      if (n >= 4) {
        const u32x4_el4 u = *reinterpret_cast<const u32x4_el4*>(s.q[h]);
        v[h] = __builtin_bit_cast(f32x4, u);
      } else if (n > 0) {
#pragma unroll
        for (int e = 0; e < 3; ++e)
          if (e < n) v[h][e] = s.q[h][e];
      }
      s.q[h] += s.step;
    }
    s.left -= kDepth;
  }
  __device__ inline void store(float* lds) const {
#pragma unroll
    for (int h = 0; h < V; ++h)
      *reinterpret_cast<f32x4*>(lds + (DEEP ? row(h) * PITCH + deep(h)
                                            : deep(h) * PITCH + row(h))) = v[h];
  }
  // the four steps' values of group j, of the row `at`
  static __device__ inline f32x4 read(const float* lds, int at, int j, int half) {
    const int r = 8 * j + 4 * half;
    if constexpr (DEEP) return *reinterpret_cast<const f32x4*>(lds + at * PITCH + r);
    f32x4 f;
#pragma unroll
    for (int s = 0; s < 4; ++s) f[s] = lds[(r + s) * PITCH + at];
    return f;
  }
};

template <bool AD, bool BD, int F>
__global__ __launch_bounds__(kThreads) void product32_kernel(Product g, ProductGrid grid,
                                                             float* part) {
  typedef Part<AD, F> A;
  typedef Part<BD, F> B;
  constexpr int P = 64 * F, WR = 32 * F, BUF = A::FLOATS + B::FLOATS;
  static_assert(BUF >= 2 * 1024, "the way out takes a block of 1024 floats a wave");
  __shared__ __attribute__((aligned(16))) float lds[2 * BUF];
  const int lane = threadIdx.x & 63, half = lane >> 5, col = lane & 31;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wp = wave / 2, wq = wave % 2;
  const ProductItem t = product_item<P, 2 * kDepth>(grid, (uint32_t)xcd_remap(blockIdx.x, gridDim.x),
                                                true, g.R);
  const float* pa = static_cast<const float*>(g.a.p);
  const float* pb = static_cast<const float*>(g.b.p);
  f32x16 acc[F][F];
#pragma unroll
  for (int i = 0; i < F; ++i)
#pragma unroll
    for (int j = 0; j < F; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
  // two stages in flight: a set of registers is loaded again as soon as it is written to LDS
  A a[2];
  B b[2];
  typename A::Source sa(pa, g.a.ld, t.p0, g.P, t.begin, t.end);
  typename B::Source sb(pb, g.b.ld, t.q0, g.Q, t.begin, t.end);
  auto load = [&](auto Set) {
    a[decltype(Set)::value].load(sa);
    b[decltype(Set)::value].load(sb);
  };
  auto step = [&](auto Set) {
    constexpr int set = decltype(Set)::value;   // of the next stage, odd or even
    const float* cur = lds + (set ^ 1) * BUF;
    float* other = lds + set * BUF;
#pragma unroll
    for (int j = 0; j < kDepth / 8; ++j) {
      f32x4 fa[F], fb[F];
#pragma unroll
      for (int i = 0; i < F; ++i) {
        fa[i] = A::read(cur, wp * WR + 32 * i + col, j, half);
        fb[i] = B::read(cur + A::FLOATS, wq * WR + 32 * i + col, j, half);
      }
#pragma unroll
      for (int s = 0; s < 4; ++s)
#pragma unroll
        for (int i = 0; i < F; ++i)
#pragma unroll
          for (int k = 0; k < F; ++k)
            acc[i][k] = __builtin_amdgcn_mfma_f32_32x32x2f32(fa[i][s], fb[k][s], acc[i][k], 0, 0, 0);
    }
    a[set].store(other);
    b[set].store(other + A::FLOATS);
    load(Set);
    __syncthreads();
  };
  constexpr std::integral_constant<int, 0> kEven{};
  constexpr std::integral_constant<int, 1> kOdd{};
  load(kEven);
  load(kOdd);
  a[0].store(lds);
  b[0].store(lds + A::FLOATS);
  load(kEven);
  __syncthreads();
  for (int st = 0; st < t.stages; st += 2) {   // an even number of stages
    step(kOdd);
    step(kEven);
  }
  // out, 32 x 32 sums of a wave at a time
  float* out = lds + wave * 1024;
  if (part) part += ((int64_t)t.split * grid.tiles + t.tile) * P * P;
#pragma unroll
  for (int i = 0; i < F; ++i)
#pragma unroll
    for (int k = 0; k < F; ++k) {
      put_tile<32>(acc[i][k], out, lane, 0);
      const int64_t p0 = (int64_t)t.p0 + wp * WR + 32 * i;
      const int64_t q = (int64_t)t.q0 + wq * WR + 32 * k + 8 * (lane % 4);
#pragma unroll 1
      for (int row = lane / 4; row < 32; row += 16) {
        const float* src = out + out_at<32>(row, 8 * (lane % 4));
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = src[e];
        const int64_t p = p0 + row;
        if (p >= g.P || q >= g.Q) continue;
        if (part) {
#pragma unroll
          for (int e = 0; e < 8; ++e) part[(p - t.p0) * P + (q - t.q0) + e] = v[e];
        } else {
          finish_chunk<float>(g, p, q, v);
        }
      }
    }
}

template <int F>
hipError_t layouts(const Product& g, const ProductGrid& grid, float* part, hipStream_t stream) {
  const dim3 blocks(grid.items), block(kThreads);
  if (g.a.deep && !g.b.deep)
    SWG_LAUNCH((product32_kernel<true, false, F>), blocks, block, 0, stream, g, grid, part);
  else if (g.a.deep)
    SWG_LAUNCH((product32_kernel<true, true, F>), blocks, block, 0, stream, g, grid, part);
  else
    SWG_LAUNCH((product32_kernel<false, false, F>), blocks, block, 0, stream, g, grid, part);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_product32(const Product& g, const ProductPlan& p, void* ws, hipStream_t stream) {
  auto run = [&](const ProductGrid& grid, float* part) {
    return p.f == 2 ? layouts<2>(g, grid, part, stream) : layouts<1>(g, grid, part, stream);
  };
  if (p.whole > 0) {
    const hipError_t e = run(product_grid(p, true), nullptr);
    if (e != hipSuccess || p.splits == 1) return e;
  }
  const ProductGrid rest = product_grid(p, false);
  float* part = reinterpret_cast<float*>(static_cast<char*>(ws) + p.part_at);
  const hipError_t e = run(rest, part);
  if (e != hipSuccess) return e;
  return product_join<float>(g, p, rest, part, stream);
}

}  // namespace swg
