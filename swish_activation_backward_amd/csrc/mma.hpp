// Device helpers of the matrix-core kernels (16-bit operands): the MFMA instructions, loads
// from memory straight to LDS, and the layouts of operand tiles in LDS.
#pragma once

#include "common.hpp"

namespace swg {

typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef short i16x8 __attribute__((ext_vector_type(8)));
#define LDS_AS __attribute__((address_space(3)))

template <typename T> struct Mfma;
template <> struct Mfma<bf16> {
  typedef bf16x8 frag;
  __device__ static inline f32x16 mma(frag a, frag b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
  }
};
template <> struct Mfma<fp16> {
  typedef fp16x8 frag;
  __device__ static inline f32x16 mma(frag a, frag b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
  }
};

// MFMA 32x32x16 layout: lane l supplies row (l % 32) and contraction elements
// 8 (l / 32) .. 8 (l / 32) + 7 of each operand; accumulator register r of lane l holds
// row 8 (r / 4) + 4 (l / 32) + (r % 4), column l % 32.

constexpr uint32_t kOOB = 0x80000000u;  // offset past every window: loads zeros

// s_waitcnt with only the vector-memory counter constrained (gfx9 encoding)
constexpr int vmcnt_le(int n) { return (n & 0xF) | (0x7 << 4) | (0xF << 8) | ((n >> 4) << 14); }
constexpr int kLgkmcnt0 = 0xC07F;   // s_waitcnt lgkmcnt(0), other counters free

__device__ inline __amdgpu_buffer_rsrc_t make_rsrc(const void* base, uint32_t bytes) {
  // raw buffer, no stride: offsets >= bytes return zero
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)bytes,
                                           0x00020000);
}
__device__ inline uint32_t clamp_bytes(int64_t rows, int64_t row_bytes) {
  return rows > 0 ? (uint32_t)(rows * row_bytes) : 0u;
}
// 16 bytes per lane from window `r` at soffset + voffset to LDS at dst + OFS + 16 * lane
// (dst must be wave-uniform).  The hardware range check applies to voffset (plus the
// instruction offset) against the window's size, not to soffset: a wave-uniform column or
// stage offset can go into soffset while the per-lane row term in voffset keeps rows past
// the window reading zeros.  Issued as inline asm: the loads' completion is tracked by
// the explicit vmcnt waits of the pipeline (the compiler's own tracking of LDS-DMA stores
// would add conservative waits that drain the ring).  The constant OFS is added to M0
// inside the asm so one scalar base serves all loads of a stage; a load to LDS needs one wait
// state behind the scalar unit's write of M0, which the compiler does not see to inside asm.
template <int OFS>
__device__ inline void dma16s(__amdgpu_buffer_rsrc_t r, uint32_t voff, uint32_t soff,
                              const uint16_t* dst) {
  const uint32_t lds = __builtin_amdgcn_readfirstlane(
      (uint32_t)(uintptr_t)(LDS_AS const void*)dst);
  asm volatile("s_add_u32 m0, %2, %3\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, %4 offen lds"
               :
               : "v"(voff), "s"(r), "s"(lds), "i"(OFS), "s"(soff)
               : "memory", "scc");   // s_add_u32 writes SCC
}
// Compiler-only fence: keeps LDS reads and writes on their side of a barrier without
// emitting the memory-model waits of __syncthreads (which would drain the ring).
#define SWG_COMPILER_FENCE() asm volatile("" ::: "memory")

// consecutive logical tiles -> same XCD
__device__ inline int64_t xcd_remap(int64_t b, int64_t nblocks) {
  const int64_t per = nblocks / 8;
  if (b >= per * 8) return b;
  return (b % 8) * per + b / 8;
}

// 64-bit pointer pinned to scalar registers (a buffer resource must be wave-uniform)
template <typename P>
__device__ inline P* uniform_ptr(P* p) {
  const uint64_t v = (uint64_t)(uintptr_t)p;
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
  return (P*)(uintptr_t)(((uint64_t)hi << 32) | lo);
}

// Rows of 32 contraction elements: a row is 4 chunks of 16 B.
// Chunk c of row r sits at position c ^ xsw(r), xsw(r) = (r / 4) % 4: within 16
// consecutive rows (one group of 16 lanes of a 16-byte read) the four rows that share a
// 64-byte bank window take four different chunks (measured: full LDS read rate, no bank
// conflict cycles).
__device__ inline int xsw(int r) { return (r >> 2) & 3; }

// Contraction rows of 128 or 256 elements of an operand's rows: chunk c of row m sits at position
// c ^ wsw(m).  A transposing read covers 4 rows x 32 bytes per 16 lanes (64 bytes for 32 lanes);
// wsw spreads them over distinct banks (rows are a multiple of 256 bytes apart).
__device__ inline int wsw(int m) {
  const int t = m & 3;
  return t == 0 ? 0 : t == 1 ? 6 : t == 2 ? 12 : 10;
}

// ds_read_b64_tr_b16: within each 16-lane group, lane s supplies 4 consecutive 16-bit
// elements E[s][0..3]; lane i receives E[4 j + i / 4][i % 4] for j = 0..3.  With lane s
// pointing at row m0 + s / 4, column c0 + 4 (s % 4), lane i gets column c0 + i of rows
// m0 .. m0 + 3: four consecutive contraction elements of one operand row.
__device__ inline i16x4 tr_read(const uint16_t* p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((LDS_AS i16x4*)p);
}

// Per-lane part of the transposing-read address of operand block i (rows 32 i .. of the
// wave's WR), in elements, for contraction rows 0..3 of a 16-row step, in a [k][P] tile
// whose wave part starts at chunk wchunk:
//   lane = 16 grp + s:  row 8 (grp / 2) + s / 4, column 32 i + 16 (grp % 2) + 4 (s % 4)
// with the column's chunk swizzled by wsw(row) (row % 4 = s / 4: the swizzle does not
// depend on the step, so every other term is a compile-time offset).
template <int F, int P>
__device__ inline void w_lane_offsets(int lane, int wchunk, int (&off)[F]) {
  const int grp = lane >> 4, s = lane & 15;
  const int q = 2 * (grp & 1) + ((s & 3) >> 1);    // chunk inside the 32-column block
  const int sw = wsw(s >> 2);
  const int row = 8 * (grp >> 1) + (s >> 2);
#pragma unroll
  for (int i = 0; i < F; ++i)
    off[i] = row * P + (((wchunk + 4 * i + q) ^ sw) << 3) + 4 * (s & 1);
}

// Transposing-read fragment of 16 contraction rows from a [k][RL] tile: p is this lane's
// address for contraction rows 0..3; rows 4..7 are 4 rows further.
template <typename T, int RL>
__device__ inline typename Mfma<T>::frag tr_frag(const uint16_t* p) {
  const i16x4 lo = tr_read(p);
  const i16x4 hi = tr_read(p + 4 * RL);
  const i16x8 v = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
  return __builtin_bit_cast(typename Mfma<T>::frag, v);
}

}  // namespace swg
