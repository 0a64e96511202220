// The linear layer's products for 16-bit tensors on the matrix cores:
//   C[p, q] = sum over r of A(p, r) B(q, r)
// An operand lies "deep" (its contraction index contiguous) or "flat" (its rows contiguous):
//   y = x W:      x deep, W flat (deep where W is stored as its transpose)
//   dx = dz W^T:  dz deep, W deep (flat)
//   dW = x^T dz:  both flat
//
// A workgroup of four waves (2 x 2) owns a P x P tile of C, P = 64 F: F = 4, each wave 128 x 128
// outputs = 4 x 4 MFMA tiles of 32 x 32 in 256 accumulators, or F = 2, each wave 64 x 64.  The
// contraction advances in stages of 32 through a ring of four LDS slots that loads fill straight
// from memory; a stage is multiplied from registers while the next one's fragments are read from
// LDS and the stage after the next three is fetched.  A deep operand's stage is [P rows][32], read
// 16 bytes a lane; a flat one's [32][P], read with the transposing LDS read.  Workgroups are
// persistent and the ring streams across their tiles.
//
// A tile's sums pass through LDS (a part of its own, wave by wave) on their way out, so that the
// epilogue reads and writes rows of 16 bytes a lane and its code exists once: a wave's 256
// accumulators have fixed registers, and bias, activation and residual spelled out for each would
// not fit the instruction cache.
//
// Operands have rows of 16-byte multiples at 16-byte boundaries (others are laid out again first);
// what lies past their edges is fetched at offsets beyond the buffer window and arrives as zeros.
//
// Bound by the matrix cores, whose clock falls under their power: a stage of a 256-wide tile takes
// 0.75 (both flat) to 0.80 us, 0.535 where the operands are zeros; a tile's way out 12 to 15 us.  A
// stage of 128-wide tiles takes 0.28 to 0.40 us alone, 0.54 where two share a CU.  bf16, [16384,
// 4096] x 14336 with gelu_tanh and z kept 1550 to 1645 us by box = 1240 to 1170 TF; its backward 3320
// to 3450 us; [220000, 1024] x 512 with a residual 282 to 292 us = 818 to 790 TF (the ends weigh more).
// [1, 14336] x 4096 24 us and the join 5 with W from memory, 22 and 4 with W in the last cache; 32
// rows against a deep W [14336, 4096] 33 us = 3.6 TB/s and 5, or 22.5 and 4.
#include <type_traits>
#include <utility>

#include "mma.hpp"
#include "product.hpp"

namespace swg {

namespace {

constexpr int kThreads = 256;

// Functions that take the accumulators are inlined before anything else happens to them, and index
// them by constants.
#define SWG_INLINE __device__ __attribute__((always_inline)) inline

template <int F> struct Shape {
  static constexpr int P = 64 * F;                 // tile edge
  static constexpr int WR = 32 * F;                // rows and columns of a wave
  static constexpr int SIDE = P * kDepth;          // elements of one operand's stage
  static constexpr int SLOT = 2 * SIDE;
  static constexpr int LOADS = 2 * F;              // 1 KiB loads of a wave a stage
  static constexpr int OUTW = F == 4 ? 64 : 32;    // columns of the epilogue's 32-row blocks
  static constexpr int OUT = 32 * OUTW;            // floats of a wave's part of the epilogue
  static constexpr int WAVES = F == 4 ? 1 : 2;     // waves a SIMD (workgroups a CU)
};

// What a lane needs of one operand: its loads' offsets into a stage's window and the column (along
// the contiguous index) that each fetches, and its fragments' place in a slot.
template <bool DEEP, int F> struct Side;

template <int F> struct Side<true, F> {
  uint32_t voff[F];
  int col;
  int at[2];
  __device__ inline Side(int wave, int part, int lane, int64_t ld) {
    const int sw = (lane >> 4) & 3;   // xsw of the rows below: multiples of 16 do not change it
    col = ((lane & 3) ^ sw) * 8;
#pragma unroll
    for (int i = 0; i < F; ++i) {
      const int row = 16 * F * wave + 16 * i + (lane >> 2);
      voff[i] = (uint32_t)row * (uint32_t)(ld * 2) + (uint32_t)col * 2u;
    }
    const int r = part * Shape<F>::WR + (lane & 31);
#pragma unroll
    for (int kk = 0; kk < 2; ++kk)
      at[kk] = r * kDepth + (((2 * kk + (lane >> 5)) ^ xsw(r)) << 3);
  }
  template <typename T, int KK, int I>
  __device__ inline typename Mfma<T>::frag read(const uint16_t* slot) const {
    return *reinterpret_cast<const typename Mfma<T>::frag*>(slot + at[KK] + I * 32 * kDepth);
  }
  __device__ inline int column(int) const { return col; }
};

template <int F> struct Side<false, F> {
  static constexpr int P = Shape<F>::P;
  uint32_t voff[F];
  int col[2];
  int at[F];
  __device__ inline Side(int wave, int part, int lane, int64_t ld) {
    constexpr int RPL = 1024 / (2 * P), LPR = 64 / RPL;   // rows a load, lanes a row
#pragma unroll
    for (int i = 0; i < F; ++i) {
      const int row = 8 * wave + RPL * i + lane / LPR;
      const int c = ((lane % LPR) ^ wsw(row)) * 8;        // of two values: row % 4 repeats
      col[i & 1] = c;
      voff[i] = (uint32_t)row * (uint32_t)(ld * 2) + (uint32_t)c * 2u;
    }
    w_lane_offsets<F, P>(lane, part * (Shape<F>::WR / 8), at);
  }
  template <typename T, int KK, int I>
  __device__ inline typename Mfma<T>::frag read(const uint16_t* slot) const {
    return tr_frag<T, P>(slot + 16 * KK * P + at[I]);
  }
  __device__ inline int column(int i) const { return col[i & 1]; }
};

// Where an operand's next stage is fetched from: a window of rows (deep) or of contraction indices
// (flat), a scalar offset into it and how far it reaches beyond that.  A stage's fetch only steps
// it on: anything longer would hold up the matrix cores behind the barrier.
template <bool DEEP, int P> struct Cursor {
  uint64_t base;
  uint32_t bytes, soff, step;   // step: bytes of 32 contraction indices (flat)
  int left;                     // deep: contraction indices; flat: rows from the tile's first on
  int end;                      // flat: contraction indices

  template <typename T>
  __device__ inline void start(const T* p, int64_t ld, int row0, int64_t rows, int k, int last) {
    const int n = (int)(rows - row0 < P ? rows - row0 : P);
    const uint32_t row = (uint32_t)ld * 2u;
    int64_t at;
    if constexpr (DEEP) {
      at = (int64_t)row0 * ld;
      bytes = n > 0 ? (uint32_t)n * row : 0u;
      soff = (uint32_t)k * 2u;
      left = last - k;
    } else {
      at = (int64_t)k * ld;
      soff = (uint32_t)row0 * 2u;
      left = (int)(rows - row0);
      end = last - k;
      step = row * kDepth;
      bytes = flat_bytes(row);
    }
    base = (uint64_t)(uintptr_t)uniform_ptr(p + at);
    bytes = __builtin_amdgcn_readfirstlane(bytes);
    soff = __builtin_amdgcn_readfirstlane(soff);
  }
  __device__ inline uint32_t flat_bytes(uint32_t row) const {
    const int n = end < kDepth ? end : kDepth;
    return n > 0 ? (uint32_t)n * row : 0u;
  }
  __device__ inline void advance() {
    if constexpr (DEEP) {
      soff += kDepth * 2;
      left -= kDepth;
    } else {
      // past the end the window is empty and its base no longer matters
      base += step;
      end -= kDepth;
      bytes = flat_bytes(step / kDepth);
    }
  }
  __device__ inline __amdgpu_buffer_rsrc_t window() const {
    return make_rsrc((const void*)(uintptr_t)base, bytes);
  }
};

template <bool AD, bool BD, int P> struct Source {
  Cursor<AD, P> a;
  Cursor<BD, P> b;
};

template <typename T, int F> struct Frags {
  typename Mfma<T>::frag a[2][F], b[2][F];
};

// Load E (0 .. 2F - 1) of a stage to the wave's part of a slot: the first F of A, the others of B.
template <bool AD, bool BD, int F, int E>
__device__ inline void load(const Source<AD, BD, Shape<F>::P>& s, const uint16_t* dst,
                            const Side<AD, F>& a, const Side<BD, F>& b) {
  constexpr int i = E % F;
  // a wave's loads of an operand fill consecutive KiB of the slot
  if constexpr (E < F) {
    const uint32_t v = a.column(i) < s.a.left ? a.voff[i] : kOOB;
    dma16s<i * 1024>(s.a.window(), v, s.a.soff, dst);
  } else {
    const uint32_t v = b.column(i) < s.b.left ? b.voff[i] : kOOB;
    dma16s<Shape<F>::SIDE * 2 + i * 1024>(s.b.window(), v, s.b.soff, dst);
  }
}

template <bool AD, bool BD, int F, int... E>
__device__ inline void load_all(std::integer_sequence<int, E...>,
                                Source<AD, BD, Shape<F>::P>& s, const uint16_t* dst,
                                const Side<AD, F>& a, const Side<BD, F>& b) {
  (load<AD, BD, F, E>(s, dst, a, b), ...);
  s.a.advance();
  s.b.advance();
}

// Fragment G (0 .. 4F - 1) of a slot: contraction half G / 2F, then A's blocks, then B's.
template <typename T, bool AD, bool BD, int F, int G>
__device__ inline void read_one(const uint16_t* slot, const Side<AD, F>& a, const Side<BD, F>& b,
                                Frags<T, F>& f) {
  constexpr int kk = G / (2 * F), i = G % (2 * F);
  if constexpr (i < F) f.a[kk][i] = a.template read<T, kk, i>(slot);
  else f.b[kk][i - F] = b.template read<T, kk, i - F>(slot + Shape<F>::SIDE);
}

template <typename T, bool AD, bool BD, int F, int... G>
__device__ inline void read_all(std::integer_sequence<int, G...>, const uint16_t* slot,
                                const Side<AD, F>& a, const Side<BD, F>& b, Frags<T, F>& f) {
  (read_one<T, AD, BD, F, G>(slot, a, b, f), ...);
}

// MFMA Q of a stage: contraction half, row block, column block
template <typename T, int F, int Q>
SWG_INLINE void mma(f32x16 (&acc)[F][F], const Frags<T, F>& f) {
  constexpr int kk = Q / (F * F), i = (Q / F) % F, j = Q % F;
  acc[i][j] = Mfma<T>::mma(f.a[kk][i], f.b[kk][j], acc[i][j]);
}

// Clears an accumulator, in AGPRs from there on: no copies at the loop.
SWG_INLINE void clear_one(f32x16& v) {
  v = (f32x16)(0.0f);
  asm volatile("" : "+a"(v));
}
template <int F, int... I>
SWG_INLINE void clear(std::integer_sequence<int, I...>, f32x16 (&acc)[F][F]) {
  (clear_one(acc[I / F][I % F]), ...);
}

// Group G (0 .. 4F - 1) of a step: F / 2 MFMAs of the stage in f, a fragment of the next stage and,
// in odd groups, a load, kept in this order by the scheduling fence.  An operand's cursor steps on
// behind its last load.
template <typename T, bool AD, bool BD, int F, bool NEXT, int G>
SWG_INLINE void group(f32x16 (&acc)[F][F], const Frags<T, F>& f, Frags<T, F>& fn,
                      const uint16_t* next, Source<AD, BD, Shape<F>::P>& s,
                      const uint16_t* dst, const Side<AD, F>& a, const Side<BD, F>& b) {
  mma<T, F, G * (F / 2)>(acc, f);
  if constexpr (F == 4) mma<T, F, G * (F / 2) + 1>(acc, f);
  // the reads end a quarter early: a step begins with a wait for the last of them
  if constexpr (NEXT && G < 3 * F) {
    read_one<T, AD, BD, F, G * 4 / 3>(next, a, b, fn);
    if constexpr ((G + 1) * 4 / 3 - G * 4 / 3 == 2) read_one<T, AD, BD, F, G * 4 / 3 + 1>(next, a, b, fn);
  }
  if constexpr ((G & 1) != 0) load<AD, BD, F, (G >> 1)>(s, dst, a, b);
  if constexpr (G == 2 * F - 1) s.a.advance();
  if constexpr (G == 4 * F - 1) s.b.advance();
  __builtin_amdgcn_sched_barrier(0);
}

template <typename T, bool AD, bool BD, int F, bool NEXT, int... G>
SWG_INLINE void groups(std::integer_sequence<int, G...>, f32x16 (&acc)[F][F],
                       const Frags<T, F>& f, Frags<T, F>& fn, const uint16_t* next,
                       Source<AD, BD, Shape<F>::P>& s, const uint16_t* dst,
                       const Side<AD, F>& a, const Side<BD, F>& b) {
  (group<T, AD, BD, F, NEXT, G>(acc, f, fn, next, s, dst, a, b), ...);
}

// ---- epilogue
// Block B: MFMA tiles (B / 2, 2 (B % 2)) and the one to its right (F = 4), tile (B / 2, B % 2) (F = 2)
// The sums pass through an empty assembly of each block's own: the compiler would join the blocks'
// reads into one of a choice of accumulators, for which they would have to be in memory.
template <int B> SWG_INLINE f32x16 apart(f32x16 v) {
  asm volatile("; block %1" : "+a"(v) : "i"(B));
  return v;
}
template <int F, int B>
SWG_INLINE void put_block(const f32x16 (&acc)[F][F], float* out, int lane) {
  constexpr int W = Shape<F>::OUTW;
  if constexpr (F == 4) {
    put_tile<W>(apart<B>(acc[B / 2][2 * (B % 2)]), out, lane, 0);
    put_tile<W>(apart<B>(acc[B / 2][2 * (B % 2) + 1]), out, lane, 32);
  } else {
    put_tile<W>(apart<B>(acc[B / 2][B % 2]), out, lane, 0);
  }
}

template <int F>
SWG_INLINE void put_any(const f32x16 (&acc)[F][F], float* out, int lane, int blk) {
  switch (blk) {
    case 0: put_block<F, 0>(acc, out, lane); break;
    case 1: put_block<F, 1>(acc, out, lane); break;
    case 2: put_block<F, 2>(acc, out, lane); break;
    case 3: put_block<F, 3>(acc, out, lane); break;
    case 4: if constexpr (F == 4) put_block<F, 4>(acc, out, lane); break;
    case 5: if constexpr (F == 4) put_block<F, 5>(acc, out, lane); break;
    case 6: if constexpr (F == 4) put_block<F, 6>(acc, out, lane); break;
    default: if constexpr (F == 4) put_block<F, 7>(acc, out, lane); break;
  }
}

// A wave's rows of a tensor of the epilogue: a window over those that exist, and the lane's place.
struct Rows {
  __amdgpu_buffer_rsrc_t r;
  uint32_t at, row;   // bytes
  __device__ inline Rows(const void* base, int64_t ld, int es, int64_t p0, int64_t q0, int n, int row_,
                         int col) {
    row = (uint32_t)(ld * es);
    r = make_rsrc(uniform_ptr(static_cast<const char*>(base) + (p0 * ld + q0) * es),
                  base ? __builtin_amdgcn_readfirstlane(clamp_bytes(n, row)) : 0u);
    at = (uint32_t)row_ * row + (uint32_t)(col * es);
  }
  // `down` rows further
  __device__ inline uint32_t below(int down) const { return at + (uint32_t)down * row; }
};

// at column bytes `col`, which carries kOOB where the column does not exist
__device__ inline int column_at(uint32_t v, uint32_t col) {
  return (int)((v + (col & 0x7fffffffu)) | (col & kOOB));
}

// The wave's sums at (p0, q0) on their way out, a block of 32 rows after the other, in two forms.
// Where rows are of 16-byte multiples at 16-byte boundaries they go through buffer windows, which
// drop what lies past the edges, and what the epilogue reads (the residual, or the old contents) is
// loaded two blocks ahead.
template <typename T, int F>
SWG_INLINE void epilogue_whole(const f32x16 (&acc)[F][F], const Product& g, float* out,
                               int lane, int64_t p0, int64_t q0) {
  constexpr int W = Shape<F>::OUTW, LANES = W / 8, ROWS = 64 / LANES, PASSES = 32 / ROWS;
  asm volatile("" : "+v"(lane));   // keeps what follows from lane out of the main loop's registers
  const int row = lane / LANES, col = 8 * (lane % LANES);
  const int n = g.P - p0 < Shape<F>::WR ? (int)(g.P - p0) : Shape<F>::WR;
  const float* src = out + out_at<W>(row, col);   // rows ROWS further: ROWS W floats
  const void* read = g.accumulate ? g.out : g.residual;
  const Rows more(read, g.accumulate ? g.ldo : g.ldr, 2, p0, q0, n, row, col);
  const Rows to(g.out, g.ldo, 2, p0, q0, n, row, col), to_z(g.z, g.ldz, 2, p0, q0, n, row, col);
  u32x4 ahead[2][PASSES], bias[2];
  uint32_t cols[2];   // byte offsets of the blocks' left and right half, or none
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const bool has = q0 + W * h + col < g.Q;
    cols[h] = (uint32_t)(W * h * 2) | (has ? 0u : kOOB);
    bias[h] = u32x4{0, 0, 0, 0};
    if (g.bias && has) {
      Chunk<T> b;
      b.load(static_cast<const T*>(g.bias) + q0 + W * h + col);
      bias[h] = b.v[0];
    }
  }
  auto load = [&](int pair, auto S) {
    constexpr int side = decltype(S)::value;
    uint32_t at = more.below(32 * pair);
#pragma unroll
    for (int k = 0; k < PASSES; ++k) {
      ahead[side][k] =
          __builtin_amdgcn_raw_buffer_load_b128(more.r, column_at(at, cols[side]), 0, 2);
      at += ROWS * more.row;
    }
  };
#pragma unroll
  for (int k = 0; k < PASSES; ++k) ahead[0][k] = ahead[1][k] = u32x4{0, 0, 0, 0};
  if (read) {
    load(0, std::integral_constant<int, 0>());
    load(0, std::integral_constant<int, 1>());
  }
  auto finish_block = [&](int pair, auto S) {
    constexpr int side = decltype(S)::value;
    uint32_t at = to.below(32 * pair), at_z = to_z.below(32 * pair);
#pragma unroll
    for (int k = 0; k < PASSES; ++k) {
      float v[8], f[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = src[k * ROWS * W + i];
      Vec16<T>::widen(bias[side], f);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] += f[i];
      if (g.z)
        __builtin_amdgcn_raw_buffer_store_b128(Vec16<T>::narrow(v), to_z.r,
                                               column_at(at_z, cols[side]), 0, 2);
      if (g.act != kActNone) activate8(g.act, g.beta, v);
      Vec16<T>::widen(ahead[side][k], f);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] += f[i];
      __builtin_amdgcn_raw_buffer_store_b128(Vec16<T>::narrow(v), to.r,
                                             column_at(at, cols[side]), 0, 2);
      at += ROWS * to.row;
      at_z += ROWS * to_z.row;
    }
    if (read && pair + 1 < F) load(pair + 1, S);
  };
#pragma unroll 1
  for (int blk = 0; blk < 2 * F; ++blk) {
    put_any<F>(acc, out, lane, blk);
    if (blk & 1) finish_block(blk / 2, std::integral_constant<int, 1>());
    else finish_block(blk / 2, std::integral_constant<int, 0>());
  }
}

// The other form: a tile's partial sums (part: the wave's place in it), or outputs of any alignment.
template <typename T, int F>
SWG_INLINE void epilogue_any(const f32x16 (&acc)[F][F], const Product& g, float* part, float* out,
                             int lane, int64_t p0, int64_t q0) {
  constexpr int W = Shape<F>::OUTW, LANES = W / 8, ROWS = 64 / LANES;
  asm volatile("" : "+v"(lane));
#pragma unroll 1
  for (int blk = 0; blk < 2 * F; ++blk) {
    put_any<F>(acc, out, lane, blk);
    const int pb = 32 * (blk / 2), q = W * (blk % 2) + 8 * (lane % LANES);
#pragma unroll 1
    for (int row = lane / LANES; row < 32; row += ROWS) {
      const float* src = out + out_at<W>(row, 8 * (lane % LANES));
      const f32x4 lo = *reinterpret_cast<const f32x4*>(src);
      const f32x4 hi = *reinterpret_cast<const f32x4*>(src + 4);
      if (p0 + pb + row >= g.P || q0 + q >= g.Q) continue;
      if (part) {
        f32x4* dst = reinterpret_cast<f32x4*>(part + (pb + row) * Shape<F>::P + q);
        dst[0] = lo;
        dst[1] = hi;
      } else {
        float v[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = lo[i], v[4 + i] = hi[i];
        finish_chunk<T>(g, p0 + pb + row, q0 + q, v);
      }
    }
  }
}

template <typename T, bool AD, bool BD, int F, bool WHOLE>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(Shape<F>::WAVES, Shape<F>::WAVES)))
void product16_kernel(Product g, ProductGrid grid, float* part) {
  constexpr int P = Shape<F>::P, SLOT = Shape<F>::SLOT, LOADS = Shape<F>::LOADS;
  __shared__ __attribute__((aligned(1024))) uint16_t ring[4 * SLOT];
  __shared__ __attribute__((aligned(16))) float outs[4 * Shape<F>::OUT];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wp = wave / 2, wq = wave % 2;
  const Side<AD, F> sa(wave, wp, lane, g.a.ld);
  const Side<BD, F> sb(wave, wq, lane, g.b.ld);
  const T* pa = static_cast<const T*>(g.a.p);
  const T* pb = static_cast<const T*>(g.b.p);
  const uint32_t G = gridDim.x, first = (uint32_t)xcd_remap(blockIdx.x, G);
  const uint32_t mine = grid.items > first ? (grid.items - first + G - 1) / G : 0;
  uint16_t* const dst = ring + wave * F * 512;   // the wave's part of slot 0
  Source<AD, BD, P> src;                         // of the stages being fetched
  auto start = [&](const ProductItem& t) {
    src.a.start(pa, g.a.ld, t.p0, g.P, t.begin, t.end);
    src.b.start(pb, g.b.ld, t.q0, g.Q, t.begin, t.end);
  };
  // One step u: the fragments of the stage in slot u are in registers and the next three stages in
  // flight.  Once this wave's loads of the next stage have landed and its LDS reads are done, the
  // barrier says so of every wave: slot u may be filled again and slot u + 1 read.  Every step
  // issues the same number of loads, so that "landed" is "at most two stages outstanding".
#define SWG_STEP(u, NEXT)                                                                   \
  do {                                                                                      \
    __builtin_amdgcn_s_waitcnt(vmcnt_le(2 * LOADS));                                        \
    __builtin_amdgcn_s_waitcnt(kLgkmcnt0);                                                  \
    SWG_COMPILER_FENCE();                                                                   \
    __builtin_amdgcn_s_barrier();                                                           \
    SWG_COMPILER_FENCE();                                                                   \
    groups<T, AD, BD, F, (NEXT)>(std::make_integer_sequence<int, 4 * F>{}, acc,             \
                                 frags[(u) & 1], frags[((u) + 1) & 1],                      \
                                 ring + (((u) + 1) & 3) * SLOT, src, dst + (u) * SLOT, sa,  \
                                 sb);                                                       \
  } while (0)

  f32x16 acc[F][F];
  Frags<T, F> frags[2];
  ProductItem cur = product_item<P, 4 * kDepth>(grid, first, mine > 0, g.R);
  start(cur);
  constexpr std::make_integer_sequence<int, LOADS> kLoads{};
  load_all<AD, BD, F>(kLoads, src, dst, sa, sb);
  load_all<AD, BD, F>(kLoads, src, dst + SLOT, sa, sb);
  load_all<AD, BD, F>(kLoads, src, dst + 2 * SLOT, sa, sb);
  load_all<AD, BD, F>(kLoads, src, dst + 3 * SLOT, sa, sb);
  __builtin_amdgcn_s_waitcnt(vmcnt_le(3 * LOADS));
  SWG_COMPILER_FENCE();
  __builtin_amdgcn_s_barrier();
  SWG_COMPILER_FENCE();
  for (uint32_t j = 0; j < mine; ++j) {
    clear(std::make_integer_sequence<int, F * F>{}, acc);
    read_all<T, AD, BD, F>(std::make_integer_sequence<int, 4 * F>{}, ring, sa, sb, frags[0]);
    for (int t = 4; t < cur.stages; t += 4) {
      SWG_STEP(0, true);
      SWG_STEP(1, true);
      SWG_STEP(2, true);
      SWG_STEP(3, true);
    }
    const ProductItem nxt = product_item<P, 4 * kDepth>(grid, first + (j + 1) * G, j + 1 < mine, g.R);
    start(nxt);
    SWG_STEP(0, true);
    SWG_STEP(1, true);
    SWG_STEP(2, true);
    SWG_STEP(3, false);   // the next item's first stage is read after the epilogue
    const int64_t p0 = (int64_t)cur.p0 + wp * Shape<F>::WR, q0 = (int64_t)cur.q0 + wq * Shape<F>::WR;
    float* out = outs + wave * Shape<F>::OUT;
    if constexpr (WHOLE) {
      epilogue_whole<T, F>(acc, g, out, lane, p0, q0);
    } else {
      float* to = nullptr;
      if (part)
        to = part + ((int64_t)cur.split * grid.tiles + cur.tile) * P * P +
             wp * Shape<F>::WR * P + wq * Shape<F>::WR;
      epilogue_any<T, F>(acc, g, to, out, lane, p0, q0);
    }
    cur = nxt;
  }
#undef SWG_STEP
  __builtin_amdgcn_s_waitcnt(vmcnt_le(0));
}

// Whether what the epilogue touches lies in rows of 16-byte multiples with 32-bit window offsets.
bool rows_whole(const Product& g) {
  const int64_t most = int64_t(1) << 22;
  auto ok = [&](const void* p, int64_t ld) {
    return !p || ((uintptr_t)p % 16 == 0 && ld % 8 == 0 && ld < most);
  };
  return g.Q % 8 == 0 && ok(g.out, g.ldo) && ok(g.z, g.ldz) && ok(g.residual, g.ldr);
}

template <typename T, bool AD, bool BD, int F>
hipError_t tiles(const Product& g, const ProductGrid& grid, float* part, int cus,
                 hipStream_t stream) {
  const int64_t slots = (int64_t)cus * Shape<F>::WAVES;
  const dim3 n((unsigned)(grid.items < slots ? grid.items : slots)), block(kThreads);
  if (!part && rows_whole(g))
    SWG_LAUNCH((product16_kernel<T, AD, BD, F, true>), n, block, 0, stream, g, grid, part);
  else
    SWG_LAUNCH((product16_kernel<T, AD, BD, F, false>), n, block, 0, stream, g, grid, part);
  return hipGetLastError();
}

template <typename T>
hipError_t layouts(const Product& g, const ProductPlan& p, const ProductGrid& grid, float* part,
                   int cus, hipStream_t stream) {
  if (p.f == 4) {
    if (g.a.deep && !g.b.deep) return tiles<T, true, false, 4>(g, grid, part, cus, stream);
    if (g.a.deep) return tiles<T, true, true, 4>(g, grid, part, cus, stream);
    return tiles<T, false, false, 4>(g, grid, part, cus, stream);
  }
  if (g.a.deep && !g.b.deep) return tiles<T, true, false, 2>(g, grid, part, cus, stream);
  if (g.a.deep) return tiles<T, true, true, 2>(g, grid, part, cus, stream);
  return tiles<T, false, false, 2>(g, grid, part, cus, stream);
}

template <typename T>
hipError_t product16_t(Product g, const ProductPlan& p, void* ws, int cus, hipStream_t stream) {
  char* w = static_cast<char*>(ws);
  if (g.R == 0) {   // nothing is fetched
    g.a.p = g.b.p = nullptr;
    g.a.ld = g.b.ld = 8;
  }
  if (p.pack_a) {
    const hipError_t e = pack_operand<T>(g.a, g.P, g.R, w + p.pack_a_at, stream);
    if (e != hipSuccess) return e;
  }
  if (p.pack_b) {
    const hipError_t e = pack_operand<T>(g.b, g.Q, g.R, w + p.pack_b_at, stream);
    if (e != hipSuccess) return e;
  }
  if (p.whole > 0) {
    const hipError_t e = layouts<T>(g, p, product_grid(p, true), nullptr, cus, stream);
    if (e != hipSuccess || p.splits == 1) return e;
  }
  const ProductGrid rest = product_grid(p, false);
  float* part = reinterpret_cast<float*>(w + p.part_at);
  const hipError_t e = layouts<T>(g, p, rest, part, cus, stream);
  if (e != hipSuccess) return e;
  return product_join<T>(g, p, rest, part, stream);
}

}  // namespace

hipError_t launch_product16(int dtype, const Product& g, const ProductPlan& p, void* ws, int cus,
                            hipStream_t stream) {
  return dtype == 0 ? product16_t<bf16>(g, p, ws, cus, stream)
                    : product16_t<fp16>(g, p, ws, cus, stream);
}

}  // namespace swg
