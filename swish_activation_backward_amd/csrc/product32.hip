// The linear layer's products for fp32 tensors, on the fp32 matrix instructions
// (v_mfma_f32_32x32x2_f32: a lane supplies row l % 32 and contraction index l / 32):
//   C[p, q] = sum over r of A(p, r) B(q, r)
// with operands of any alignment, deep or flat (see product.hip).
//
// A workgroup of four waves (2 x 2) owns a tile of edge 64 F, each wave 32 F x 32 F outputs.  A
// stage of 32 contraction indices is loaded into registers while the two before it are multiplied,
// and written to the other of two LDS buffers as [row][32], of which a lane reads four consecutive
// indices at once; a flat operand is transposed on the way, 4 rows by 4 (2) indices a thread.  Lane
// half h takes index 8 j + 4 h + s in step s of a group j, of both operands alike.  Registers are
// held to two workgroups a CU (F = 2) or four, for which F = 2 with both operands flat spills 6.
//
// Bound by the matrix cores and the loads' and stores' instructions beside them: 4096 x 4096 x 4096
// 133 TF with both deep, 118 with one flat, 112 with both (97 with flat operands read from [32][row]
// and one workgroup a CU).  [1021, 1023] x 2047 backward: dx 47 us and its join 5, dW 53 to 61.
#include <type_traits>

#include "mma.hpp"
#include "product.hpp"

namespace swg {

namespace {

constexpr int kThreads = 256;
constexpr uint32_t kLaunchTiles = 1u << 22;

// One operand's part of a stage: V 16-byte vectors a thread.
template <bool DEEP, int F> struct Part {
  static constexpr int P = 64 * F, V = P * kDepth / 4 / kThreads;
  static constexpr int PITCH = kDepth + 4, FLOATS = P * PITCH;
  f32x4 v[V];

  // row and contraction index of vector h
  static __device__ inline int row(int h) {
    return DEEP ? threadIdx.x / 8 + 32 * h : (threadIdx.x % (P / 4)) * 4;
  }
  static __device__ inline int deep(int h) {
    return DEEP ? (threadIdx.x % 8) * 4 : threadIdx.x / (P / 4) * V + h;
  }

  // The vectors' places in memory, a stage further with every load.  Every load is executed, so that
  // the compiler can count those in flight: a vector that would end past the row's end (deep) or the
  // last row (flat) starts as much earlier and is shifted; one past the contraction's end is taken
  // from the operand's first row and dropped.  Rows that do not exist repeat an existing one: their
  // outputs are dropped.  Both extents are at least 4.
  struct Source {
    const float* first;
    const float* q[V];
    int64_t step;
    int r, end, shift;   // contraction index of the stage, its end, shift of a flat vector
    __device__ inline Source(const float* src, int64_t ld, int64_t row0, int64_t rows, int begin,
                             int end_) {
      first = src;
      r = begin;
      end = end_;
      step = kDepth * ld;
#pragma unroll
      for (int h = 0; h < V; ++h) {
        const int64_t p = row0 + row(h);
        if constexpr (DEEP) {
          q[h] = src + (p < rows ? p : rows - 1) * ld;
        } else {
          const int64_t at = p + 4 <= rows ? p : rows - 4;
          shift = (int)(p - at);
          q[h] = src + (int64_t)(begin + deep(h)) * ld + at;
        }
      }
    }
  };

  __device__ inline void load(Source& s) {
#pragma unroll
    for (int h = 0; h < V; ++h) {
      const float* p = s.q[h];
      if constexpr (DEEP) {
        const int c = s.r + deep(h);
        p += c + 4 <= s.end ? c : s.end - 4;
      } else {
        p = s.r + deep(h) < s.end ? p : s.first;
        s.q[h] += s.step;
      }
      const u32x4_el4 u = *reinterpret_cast<const u32x4_el4*>(p);
      v[h] = __builtin_bit_cast(f32x4, u);
    }
    s.r += kDepth;
  }
  // v[n ..], zeros behind
  static __device__ inline f32x4 shifted(f32x4 v, int n) {
    if (n & 1) v = f32x4{v[1], v[2], v[3], 0.0f};
    if (n & 2) v = f32x4{v[2], v[3], 0.0f, 0.0f};
    if (n & ~3) v = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    return v;
  }
  // of the stage from contraction index r on: what does not exist becomes 0
  __device__ inline void trim(const Source& s, int r) {
    const bool tail = r + kDepth > s.end;
#pragma unroll
    for (int h = 0; h < V; ++h) {
      if constexpr (DEEP) {
        const int c = r + deep(h);
        if (tail) v[h] = shifted(v[h], c + 4 <= s.end ? 0 : c + 4 - s.end);
      } else {
        if (s.shift) v[h] = shifted(v[h], s.shift);
        if (tail && r + deep(h) >= s.end) v[h] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      }
    }
  }
  // the place of group c of four contraction indices of a row; a flat operand's groups change places
  // with the row, since its lanes write rows four apart
  static __device__ inline int place(int row, int c) {
    return row * PITCH + 4 * (DEEP ? c : c ^ ((row >> 2) & 7));
  }
  __device__ inline void store(float* lds) const {
    if constexpr (DEEP) {
#pragma unroll
      for (int h = 0; h < V; ++h)
        *reinterpret_cast<f32x4*>(lds + place(row(h), deep(h) / 4)) = v[h];
    } else {   // V indices of each of four rows
      typedef float vec __attribute__((ext_vector_type(V)));
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        vec t;
#pragma unroll
        for (int h = 0; h < V; ++h) t[h] = v[h][e];
        *reinterpret_cast<vec*>(lds + place(row(0) + e, deep(0) / 4) + deep(0) % 4) = t;
      }
    }
  }
  // the four steps' values of group j, of the row `at`
  static __device__ inline f32x4 read(const float* lds, int at, int j, int half) {
    return *reinterpret_cast<const f32x4*>(lds + place(at, 2 * j + half));
  }
};

template <bool AD, bool BD, int F>
__global__ __launch_bounds__(kThreads, F == 2 ? 2 : 4) void product32_kernel(Product g, ProductGrid grid,
                                                             float* part, int pad_a, int pad_b) {
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
  // an operand that was laid out again has zeros up to an extent of pad_a (pad_b)
  auto extent = [](int64_t n, int pad) { return n < pad ? (int64_t)pad : n; };
  typename A::Source sa(pa, g.a.ld, t.p0, AD ? g.P : extent(g.P, pad_a), t.begin,
                        AD ? (int)extent(t.end, pad_a) : t.end);
  typename B::Source sb(pb, g.b.ld, t.q0, BD ? g.Q : extent(g.Q, pad_b), t.begin,
                        BD ? (int)extent(t.end, pad_b) : t.end);
  int r = t.begin;   // of the stage being multiplied
  auto load = [&](auto Set) {
    a[decltype(Set)::value].load(sa);
    b[decltype(Set)::value].load(sb);
  };
  auto step = [&](auto Set) {
    constexpr int set = decltype(Set)::value;   // of the next stage, odd or even
    const float* cur = lds + (set ^ 1) * BUF;
    float* other = lds + set * BUF;
    // all reads ahead of the products: between them each would be waited for
    f32x4 fa[kDepth / 8][F], fb[kDepth / 8][F];
#pragma unroll
    for (int j = 0; j < kDepth / 8; ++j)
#pragma unroll
      for (int i = 0; i < F; ++i) {
        fa[j][i] = A::read(cur, wp * WR + 32 * i + col, j, half);
        fb[j][i] = B::read(cur + A::FLOATS, wq * WR + 32 * i + col, j, half);
      }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int j = 0; j < kDepth / 8; ++j)
#pragma unroll
      for (int s = 0; s < 4; ++s)
#pragma unroll
        for (int i = 0; i < F; ++i)
#pragma unroll
          for (int k = 0; k < F; ++k)
            acc[i][k] =
                __builtin_amdgcn_mfma_f32_32x32x2f32(fa[j][i][s], fb[j][k][s], acc[i][k], 0, 0, 0);
    r += kDepth;
    a[set].trim(sa, r);
    b[set].trim(sb, r);
    a[set].store(other);
    b[set].store(other + A::FLOATS);
    load(Set);
    __syncthreads();
  };
  constexpr std::integral_constant<int, 0> kEven{};
  constexpr std::integral_constant<int, 1> kOdd{};
  if (g.R > 0) {
    load(kEven);
    load(kOdd);
    a[0].trim(sa, r);
    b[0].trim(sb, r);
    a[0].store(lds);
    b[0].store(lds + A::FLOATS);
    load(kEven);
    __syncthreads();
    for (int st = 0; st < t.stages; st += 2) {   // an even number of stages
      step(kOdd);
      step(kEven);
    }
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
hipError_t layouts(const Product& g, const ProductPlan& p, const ProductGrid& grid, float* part,
                   hipStream_t stream) {
  const dim3 blocks(grid.items), block(kThreads);
  const int a = p.pack_a ? 8 : 0, b = p.pack_b ? 8 : 0;
  if (g.a.deep && !g.b.deep)
    SWG_LAUNCH((product32_kernel<true, false, F>), blocks, block, 0, stream, g, grid, part, a, b);
  else if (g.a.deep)
    SWG_LAUNCH((product32_kernel<true, true, F>), blocks, block, 0, stream, g, grid, part, a, b);
  else
    SWG_LAUNCH((product32_kernel<false, false, F>), blocks, block, 0, stream, g, grid, part, a, b);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_product32(Product g, const ProductPlan& p, void* ws, hipStream_t stream) {
  char* w = static_cast<char*>(ws);
  hipError_t e = hipSuccess;
  if (p.pack_a) e = pack_operand<float>(g.a, g.P, g.R, w + p.pack_a_at, stream);
  if (e == hipSuccess && p.pack_b) e = pack_operand<float>(g.b, g.Q, g.R, w + p.pack_b_at, stream);
  if (e != hipSuccess) return e;
  auto run = [&](const ProductGrid& grid, float* part) {
    return p.f == 2 ? layouts<2>(g, p, grid, part, stream)
                    : layouts<1>(g, p, grid, part, stream);
  };
  if (p.whole > 0) {
    // a launch has less than 2^32 threads
    ProductGrid grid = product_grid(p, true);
    for (const uint32_t all = grid.tiles; grid.first < all; grid.first += kLaunchTiles) {
      grid.tiles = all - grid.first < kLaunchTiles ? all - grid.first : kLaunchTiles;
      grid.items = grid.tiles;
      e = run(grid, nullptr);
      if (e != hipSuccess) return e;
    }
    if (p.splits == 1) return hipSuccess;
  }
  const ProductGrid rest = product_grid(p, false);
  float* part = reinterpret_cast<float*>(w + p.part_at);
  e = run(rest, part);
  if (e != hipSuccess) return e;
  return product_join<float>(g, p, rest, part, stream);
}

}  // namespace swg
