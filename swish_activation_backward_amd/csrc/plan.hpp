// Host-side launch planning, shared by the workspace-size queries and the launches so
// the two always agree.  Pure integer arithmetic: no HIP calls.
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace swg {

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

inline int elem_size(int dtype) { return dtype == 2 ? 4 : 2; }
inline int vec_of(int dtype) { return 16 / elem_size(dtype); }

// ---------------------------------------------------------------- b stage
// A workgroup of 256 threads owns a strip of TX vector-columns (TX a power of two
// <= 32; TY = 256 / TX rows per pass, each lane issuing the loads of kBRowsInFlight rows
// before it computes them).  The rows are cut into units of unit_rows = max(64,
// kBRowsInFlight * TY) rows, so a unit is whole passes; the workgroups of a strip
// ("walkers", grid.y of them) take the units round-robin (walker w: units w, w + walkers,
// ...), a static assignment that keeps the column sums run-to-run deterministic while
// every walker ends within one unit of the others.  Each walker leaves one fp32 partial
// row [2N] (dg sums, then dfc sums) in the workspace, which the finalize kernel sums in
// walker order.  Measured on MI355X at M = 220000, N = 1024 bf16 (inputs in HBM, finalize
// included): 32-wide strips, 8 rows in flight and 64-row units with 256 walkers per strip
// run 384 us; 64-wide strips, 4 rows and 32-row units ran 403-406 us; walker counts that
// are not a power of two (balanced to whole rounds) ran slower.
struct BPlan {
  int vec;             // elements per 16-byte access (1 when the scalar path is used)
  int rif;             // rows whose loads a lane issues before computing (vector path)
  int tx, ty;          // thread layout inside the 256-thread workgroup
  int64_t cv;          // vector columns per row = N / vec
  int64_t nstrips;     // ceil(cv / tx)
  int64_t unit_rows;   // rows per work unit (a multiple of the rows one pass covers)
  int64_t nunits;      // ceil(M / unit_rows)
  int64_t nwalk;       // walkers per strip (grid.y) = partial rows
  size_t ws_bytes;     // nwalk * 2N * sizeof(float)
};

constexpr int kBThreads = 256;
constexpr int kBMaxTx = 32;              // widest strip, in 16-byte vector columns
constexpr int64_t kBMinUnitRows = 64;    // smallest work unit
// Walkers per strip: of the smallest power of two that launches at least kBMinBlocks
// workgroups in all and the next two (each capped at the number of units), the one that
// minimises rounds x units per walker, where a round is kBSlots workgroups (one resident
// per CU of the MI355X: the vector kernel holds 300 VGPRs).  More walkers would also add
// partial rows for the finalize to read.  Counts that are not a power of two ran
// slower even when balanced (measured at N = 1024); at N = 14336 bf16 the rule gives 56
// strips x 32 walkers (seven full rounds of 8 units, 434 us) where 56 x 19 ran 474 us and
// 56 x 18 441-444 us.
constexpr int64_t kBSlots = 256;
// Size of the static partial-row array used by swiglu_bwd_b_noalloc (16 MiB: every shape
// up to N = 2^21 columns fits; at N = 1024 the plan needs 2 MiB, at N = 14336 3.5 MiB).
constexpr size_t kBScratchBytes = size_t(16) << 20;
constexpr int64_t kBMinBlocks = 1024;
constexpr int kBRowsInFlight = 8;        // rows whose loads a lane issues before computing
// Small batches (at most kBSmallBlocks workgroups with kBRowsInFlight rows per lane): the
// vector kernel holds 300 registers, so one workgroup per CU runs its single pass of
// loads, then its arithmetic, with nothing to overlap them.  There the plan takes
// kBSmallRows rows in flight (a kernel several workgroups of which share a CU), units of
// one pass and one walker per unit (at most kBSmallMaxBlocks workgroups).
constexpr int kBSmallRows = 4;
constexpr int64_t kBSmallBlocks = 4096;
constexpr int64_t kBSmallMaxBlocks = 4096;

inline BPlan plan_b(int64_t M, int64_t N, int dtype, bool vector_path) {
  BPlan p{};
  // the unit size and the walker count depend only on (M, N, dtype), never on pointer
  // alignment (the workspace query cannot see the pointers)
  const int vref = vec_of(dtype);
  const int64_t cv_ref = (N % vref == 0) ? N / vref : N;
  int tx_ref = 1;
  while (tx_ref < kBMaxTx && tx_ref < cv_ref) tx_ref <<= 1;
  const int64_t strips_ref = ceil_div(cv_ref, tx_ref);
  const int64_t pass_rows = (int64_t)kBRowsInFlight * (kBThreads / tx_ref);
  p.rif = kBRowsInFlight;
  p.unit_rows = pass_rows > kBMinUnitRows ? pass_rows : kBMinUnitRows;
  p.nunits = M > 0 ? ceil_div(M, p.unit_rows) : 0;
  int64_t nwalk = 1;
  if (p.nunits > 0 && strips_ref * p.nunits <= kBSmallBlocks) {
    p.rif = kBSmallRows;
    p.unit_rows = (int64_t)kBSmallRows * (kBThreads / tx_ref);
    p.nunits = ceil_div(M, p.unit_rows);
    const int64_t cap = kBSmallMaxBlocks / strips_ref;
    nwalk = p.nunits < cap ? p.nunits : (cap > 0 ? cap : 1);
  } else if (p.nunits > 0) {
    int64_t w0 = 1;   // smallest power of two reaching kBMinBlocks workgroups
    while (strips_ref * w0 < kBMinBlocks) w0 *= 2;
    int64_t best_cost = -1;
    for (int64_t w = w0; w <= 4 * w0; w *= 2) {
      const int64_t ww = w < p.nunits ? w : p.nunits;
      const int64_t cost = ceil_div(strips_ref * ww, kBSlots) * ceil_div(p.nunits, ww);
      if (best_cost < 0 || cost < best_cost) {
        best_cost = cost;
        nwalk = ww;
      }
      if (ww == p.nunits) break;
    }
  }
  p.nwalk = nwalk;
  p.ws_bytes = (M > 0 && N > 0) ? (size_t)p.nwalk * (size_t)(2 * N) * sizeof(float) : 0;

  p.vec = (vector_path && N % vref == 0) ? vref : 1;
  p.cv = N / p.vec;
  int tx = 1;
  while (tx < kBMaxTx && tx < p.cv) tx <<= 1;
  p.tx = tx;
  p.ty = kBThreads / tx;
  p.nstrips = ceil_div(p.cv, tx);
  return p;
}

// ---------------------------------------------------------------- GEMM tiles
// Both GEMMs use square output tiles of edge 64 F per workgroup of four waves: F = 4
// (256 x 256) or F = 2 (128 x 128), and a 32-deep contraction step per LDS stage (the
// x stage moves two stages per load).
constexpr int kTileP = 256;     // output rows per workgroup at F = 4
constexpr int kTileQ = 256;     // output cols per workgroup at F = 4
constexpr int kTileR = 32;      // contraction depth per LDS stage
constexpr int64_t kMaxGemmDim = int64_t(1) << 22;  // K, N limit of the GEMM stages
inline int64_t tile_edge(int f) { return 64 * (int64_t)f; }

// Tile choice.  256 x 256 tiles load half the operand bytes per flop of 128 x 128 tiles
// and run faster per flop; 128 x 128 tiles win when the large ones leave CUs idle (small
// batches) or, in the w stage, need many M splits whose fp32 partials cost a round trip
// through memory.  The planner takes the configuration with the smaller time estimate:
// rounds of work items over the CUs x pipeline stages per item x the time of one stage
// at that configuration, plus, for the w stage, the partials' write and read at the
// streaming rate and the reduce launch.  Stage times from kernel spans on MI355X (bf16,
// both tile sizes forced, M = 256 .. 220000 at K = 512, N = 1024 and four shapes with K, N
// up to 4096 and 14336): at 128 x 128 one workgroup per CU is bound by LDS traffic (the
// DMA writes plus the fragment reads of twice as many bytes per flop), so its stage takes
// 0.4-0.45 of a 256 x 256 stage for a quarter of the work.  The x stage at 128 x 128 runs
// two workgroups per CU when it has more tiles than CUs: a double stage then takes 1.15 us
// per workgroup (two progress at once), against 0.75 us for a workgroup alone.
constexpr int64_t kGemmSlots = 256;        // one persistent workgroup per CU of the MI355X
constexpr int64_t kXStageNs[2] = {1700, 750};   // x: one 64-deep double stage, F = 4 / F = 2
constexpr int64_t kXStageNsShared = 1150;       // x, F = 2, two workgroups per CU
constexpr int64_t kWStageNs[2] = {850, 320};    // w: one 32-deep stage, F = 4 / F = 2
constexpr int64_t kReduceLaunchNs = 2000;       // w_reduce launch and ramp
constexpr int64_t kStreamBytesPerNs = 5000;     // partials' round trip, ~5 TB/s
inline int64_t stage_ns(const int64_t (&t)[2], int f) { return f == 4 ? t[0] : t[1]; }

// x stage: output [M, K] in tiles of edge 64 F; every tile runs nds double stages.
struct XPlan {
  int f;
  int64_t nq, tiles;       // column tiles per row block, tiles
};

inline int64_t x_double_stages(int64_t N) {
  const int64_t sd = ceil_div(N, 2 * kTileR);
  return 2 * (sd < 2 ? 2 : sd);
}

inline XPlan plan_x_f(int64_t M, int64_t K, int f) {
  XPlan p{};
  p.f = f;
  p.nq = ceil_div(K, tile_edge(f));
  p.tiles = ceil_div(M, tile_edge(f)) * p.nq;
  return p;
}

inline int64_t x_time_ns(const XPlan& p, int64_t N, int64_t slots) {
  const int64_t nds = x_double_stages(N);
  if (p.f == 4) return ceil_div(p.tiles, slots) * nds * kXStageNs[0];
  if (p.tiles <= slots) return nds * kXStageNs[1];   // one workgroup per CU
  return ceil_div(p.tiles, 2 * slots) * nds * kXStageNsShared;
}

// force_f: 4 or 2 overrides the estimate (0: the planner's choice); likewise below.
inline XPlan plan_x(int64_t M, int64_t K, int64_t N, int force_f = 0) {
  if (force_f == 4 || force_f == 2) return plan_x_f(M, K, force_f);
  const XPlan big = plan_x_f(M, K, 4), small = plan_x_f(M, K, 2);
  return x_time_ns(small, N, kGemmSlots) < x_time_ns(big, N, kGemmSlots) ? small : big;
}

// w stage: output [K, 2N]; when it has too few tiles to fill the chip the batch
// dimension M is split into S ranges whose fp32 partials are summed in order.
struct WPlan {
  int f;                   // tile configuration
  int64_t tk, tn, tiles;   // tile grid over [K, 2N]: tn / 2 column tiles in dg, tn / 2 in dfc
  int64_t splits;          // S
  int64_t rows;            // rows of M per split (multiple of kTileR)
  size_t ws_bytes;         // S > 1: S * K * 2N * sizeof(float)
};

constexpr int64_t kWTargetBlocks = kGemmSlots;
constexpr int64_t kWMinRowsPerSplit = 512;

inline WPlan plan_w_f(int64_t M, int64_t K, int64_t N, int f) {
  WPlan p{};
  p.f = f;
  p.tk = ceil_div(K, tile_edge(f));
  p.tn = 2 * ceil_div(N, tile_edge(f));
  p.tiles = p.tk * p.tn;
  // splits that keep tiles x S within one round of workgroups
  int64_t s = p.tiles > 0 ? kWTargetBlocks / p.tiles : 1;
  const int64_t smax = M / kWMinRowsPerSplit;
  if (s > smax) s = smax;
  if (s < 1) s = 1;
  p.rows = ceil_div(ceil_div(M, s), kTileR) * kTileR;
  if (p.rows < kTileR) p.rows = kTileR;
  p.splits = M > 0 ? ceil_div(M, p.rows) : 1;
  if (p.splits < 1) p.splits = 1;
  p.ws_bytes = (p.splits > 1 && K > 0 && N > 0)
                   ? (size_t)p.splits * (size_t)K * (size_t)(2 * N) * sizeof(float)
                   : 0;
  return p;
}

inline int64_t w_time_ns(const WPlan& p) {
  const int64_t nst = 4 * ceil_div(p.rows, 4 * kTileR);   // whole ring rounds per item
  int64_t t = ceil_div(p.splits * p.tiles, kWTargetBlocks) * nst * stage_ns(kWStageNs, p.f);
  if (p.splits > 1) t += kReduceLaunchNs + 2 * (int64_t)p.ws_bytes / kStreamBytesPerNs;
  return t;
}

inline WPlan plan_w(int64_t M, int64_t K, int64_t N, int force_f = 0) {
  if (force_f == 4 || force_f == 2) return plan_w_f(M, K, N, force_f);
  const WPlan big = plan_w_f(M, K, N, 4), small = plan_w_f(M, K, N, 2);
  return w_time_ns(small) < w_time_ns(big) ? small : big;
}

// fused w + x pass: the grid is split between x-stage tiles (gx workgroups) and w-stage
// items (gw workgroups).  Both GEMMs have the same flop count, so half of the workgroups
// go to each; the w items are the dW tiles times S splits over 256-row chunks taken
// round-robin, S chosen so the w half of the grid is filled (and at least 512 rows per
// split, as in the w stage).  With 128 + 128 workgroups both halves advance through the
// rows of [dg | dfc] at the same rate.  Both halves use 128 x 128 tiles when the x stage
// has fewer 256 x 256 tiles than its half of the grid.
struct WXPlan {
  bool separate;                   // run the w stage and the x stage as two launches
  int f;                           // tile configuration of both halves
  int64_t nq, x_tiles, gx;         // x stage: column tiles per row block, tiles, workgroups
  int64_t tn, w_tiles, splits;     // w stage: tile grid, tiles, S
  int64_t w_items, gw;             // items (tiles x S), workgroups
  int64_t chunk_rows;              // 256
  size_t ws_bytes;                 // S > 1: S * K * 2N * sizeof(float); separate: plan_w's
};

constexpr int64_t kWXChunkRows = 256;
constexpr int64_t kWXWorkgroups = 256;

inline WXPlan plan_wx(int64_t M, int64_t K, int64_t N, int force_f = 0) {
  WXPlan p{};
  p.f = ceil_div(M, tile_edge(4)) * ceil_div(K, tile_edge(4)) < kWXWorkgroups / 2 ? 2 : 4;
  if (force_f == 4 || force_f == 2) p.f = force_f;
  const int64_t edge = tile_edge(p.f);
  p.nq = ceil_div(K, edge);
  p.x_tiles = ceil_div(M, edge) * p.nq;
  p.gx = p.x_tiles < kWXWorkgroups / 2 ? p.x_tiles : kWXWorkgroups / 2;
  if (p.gx < 1) p.gx = 1;
  p.tn = 2 * ceil_div(N, edge);
  p.w_tiles = ceil_div(K, edge) * p.tn;
  const int64_t target = kWXWorkgroups - p.gx;
  int64_t s = p.w_tiles > 0 ? target / p.w_tiles : 1;
  const int64_t smax = M / kWMinRowsPerSplit;
  if (s > smax) s = smax;
  if (s < 1) s = 1;
  p.splits = s;
  p.chunk_rows = kWXChunkRows;
  p.w_items = p.w_tiles * p.splits;
  p.gw = p.w_items < target ? p.w_items : target;
  if (p.gw < 1) p.gw = 1;
  p.ws_bytes = (p.splits > 1 && K > 0 && N > 0)
                   ? (size_t)p.splits * (size_t)K * (size_t)(2 * N) * sizeof(float)
                   : 0;
  // Without an M split the w items each walk all of M while the x tiles walk row blocks,
  // so the two halves never read the same rows at the same time; when each stage also
  // fills the GPU on its own (two rounds or more of each half), fusing gives no traffic
  // back and only shares the chip: measured 1.68 ms against 1.53 ms for w + x at
  // M = 4096, K = 4096, N = 14336, and 6.6 ms against 6.2 ms at M = 16384.  Those shapes
  // run the two stages as separate launches.
  p.separate = p.splits == 1 && p.x_tiles >= 2 * p.gx && p.w_items >= 2 * p.gw;
  if (p.separate) p.ws_bytes = plan_w(M, K, N, force_f).ws_bytes;
  return p;
}

// ---------------------------------------------------------------- row operators
// Workgroups of a launch over rows (each takes every gridDim.x-th row): a launch holds
// fewer than 2^32 work items.
inline unsigned row_grid(int64_t rows) {
  return (unsigned)(rows < (int64_t(1) << 20) ? rows : (int64_t(1) << 20));
}

// Workgroups of a norm's forward pass, `rows` rows at a time each: as many as a kernel of up to 64
// registers has resident at once, so that each walks over its rows with the next ones' loads in
// flight.
inline unsigned norm_fwd_grid(int64_t M, int rows, int threads) {
  const int64_t n = ceil_div(M, rows), all = 2048 * 256 / threads;
  return (unsigned)(n < all ? n : all);
}

// Layer norm's backward pass.  Rows of 8 to 16384 elements: `group` threads hold a row, `chunks`
// chunks of 8 elements each, and one workgroup of 1024 threads per CU leaves one fp32 partial
// row [dw | db] of 2 np in the workspace (none is needed for a single workgroup).  Other
// lengths (group = 0): the rows are cut into `parts` blocks of `rows` with one partial row
// each.  The finalize kernel sums the partial rows in a fixed order.
// One chunk a thread up to 1024 columns, two above: at [16384, 4096] fp16 two chunks (256
// threads a row) take 80 us and one (512 threads, half the rows between barriers) 84 us; at
// [8191, 1023] fp32 one takes 29.5 us and two (a wave a row, more registers) 30.7 us.
struct NormPlan {
  int group, chunks;
  int64_t rows;
  int64_t parts;
  int64_t np;
  size_t ws_bytes;
};

inline NormPlan plan_norm_bwd(int64_t M, int64_t N) {
  NormPlan p{};
  p.np = ceil_div(N, 4) * 4;
  if (N < 8 || N > 16384) {
    // one thread walks a block of narrow rows: many short blocks
    const int64_t least = N < 8 ? 16 : 64, blocks = N < 8 ? 8192 : 256;
    p.rows = M > blocks * least ? ceil_div(M, blocks) : least;
    p.parts = ceil_div(M, p.rows);
    p.ws_bytes = (size_t)p.parts * 2 * (size_t)p.np * sizeof(float);
    return p;
  }
  p.chunks = N <= 1024 ? 1 : 2;
  p.group = 8;
  while ((int64_t)p.group * 8 * p.chunks < N) p.group *= 2;
  const int64_t n = ceil_div(M, 1024 / p.group);
  p.parts = n < 256 ? n : 256;
  p.ws_bytes = (size_t)p.parts * 2 * (size_t)p.np * sizeof(float);
  return p;
}

// The residual norm's backward pass, as layer norm's: rows of 8 to 16384 elements are held by
// `group` threads of `chunks` chunks each, and a workgroup (512 threads, 1024 above 8192 columns)
// per CU leaves one fp32 partial row of 2 np.  Other lengths (group = 0) need two fp32 values a row
// before those, and their partial rows are of blocks of `rows` rows.
struct ResidualNormPlan {
  int group, chunks;
  int64_t rows;
  int64_t parts;
  int64_t np;
  int64_t stat_floats;
  size_t ws_bytes;
};

inline ResidualNormPlan plan_residual_norm_bwd(int64_t M, int64_t N) {
  ResidualNormPlan p{};
  p.np = ceil_div(N, 4) * 4;
  if (N < 8 || N > 16384) {
    // one thread walks a block of narrow rows: many short blocks
    const int64_t least = N < 8 ? 16 : 64, blocks = N < 8 ? 8192 : 256;
    p.rows = M > blocks * least ? ceil_div(M, blocks) : least;
    p.parts = ceil_div(M, p.rows);
    p.stat_floats = ceil_div(2 * M, 4) * 4;
  } else {
    p.chunks = N <= 1024 ? 1 : 2;
    p.group = 8;
    while ((int64_t)p.group * 8 * p.chunks < N) p.group *= 2;
    const int64_t n = ceil_div(M, p.group > 512 ? 1 : 512 / p.group);
    p.parts = n < 256 ? n : 256;
  }
  p.ws_bytes = (size_t)(p.stat_floats + p.parts * 2 * p.np) * sizeof(float);
  return p;
}

// The linear layer's dz and db: `parts` blocks of `rows` rows, one fp32 partial row of np each.
struct ActBwdPlan {
  int64_t rows, parts, np;
};

inline ActBwdPlan plan_act_bwd(int64_t M, int64_t N) {
  ActBwdPlan p{};
  p.np = ceil_div(N, 4) * 4;
  // about 2048 workgroups of 512 columns, 16 rows at least
  int64_t blocks = ceil_div(2048, ceil_div(N < 1 ? 1 : N, 512));
  if (blocks > 512) blocks = 512;
  p.rows = M > blocks * 16 ? ceil_div(M, blocks) : 16;
  p.parts = ceil_div(M, p.rows);
  return p;
}

// One product of the linear layer: output [P, Q], contraction R, in tiles of edge 64 f (f = 4 or 2
// for 16-bit tensors, 2 or 1 for fp32).  The first `whole` tiles, whole rounds over the CUs, are
// finished by one workgroup each; the contraction of the others is cut into `splits` ranges of
// `len`, so that they too fill the CUs, and the ranges' fp32 sums are joined in order.  16-bit
// operands that do not lie in rows of 16-byte multiples are laid out again (pack_a, pack_b) in the
// workspace before, and so are fp32 operands with fewer than four elements along their rows.
//
// The tile and the split are those of the smallest estimate: rounds of items over the CUs, times an
// item's stages (32 deep) and what it spends before and after them, plus the partial sums' trip
// through memory and the launches.  force_f: 4 or 2 overrides the tile (16-bit).
struct ProductPlan {
  bool few;                // the form for few rows, which takes nothing of the workspace
  int f;
  int64_t np, nq, whole;
  int64_t splits, len;
  bool pack_a, pack_b;
  size_t pack_a_at, pack_b_at, part_at;
  size_t ws_bytes;
};

// Row stride of an operand that is laid out again: whole 128-byte lines, so that the 64-byte
// pieces of its rows that a stage fetches lie in one line each.
inline int64_t packed_ld(int64_t cols) { return ceil_div(cols, 64) * 64; }

// In ns, by f: a stage's time on a CU that is busy, the least time from one stage of an item to the
// next (its loads' latency), an item's ends, and the items that can share a CU.
struct ProductCost {
  int f;
  int64_t busy, least, ends, share;
};
constexpr ProductCost kProduct16[2] = {{4, 800, 800, 12000, 1}, {2, 270, 300, 4000, 2}};
constexpr ProductCost kProduct32[2] = {{2, 1900, 1900, 4000, 2}, {1, 480, 700, 2000, 4}};
constexpr int64_t kJoinNs = 6000;     // the join's launch and, of whole rounds before, the split's

// `items` of `len` contraction indices each
inline int64_t product_items_ns(int64_t items, int64_t len, const ProductCost& c) {
  if (items <= 0) return 0;
  const int64_t stages = ceil_div(len, 4 * kTileR) * 4;
  int64_t share = ceil_div(items, kGemmSlots);
  if (share > c.share) share = c.share;
  const int64_t stage = c.busy * share > c.least ? c.busy * share : c.least;
  return ceil_div(items, kGemmSlots * share) * (stages * stage + c.ends);
}

// Whether few rows go by the form without a split.  Against a flat operand it pays while all waves of
// a workgroup take one turn, and while the half lines that it reads do not set the time (4096 x
// 4096: 19.7 us against 12.7; 1024 x 4096: 6.1 against 10.6).  Against a deep one it pays while its
// workgroup of 16 columns has read its rows (30 bytes a ns) before the tiles have all of the weight (4800 bytes a ns, and 7 us
// of launches), and, 16-bit, while reading the rows again for every 16 columns is cheap: at 4096 x
// 12288 it takes 20.3 us for one row against 24.2, 24.6 against 24.6 for 8, 29.4 against 25.0 for
// 16; at 14336 x 1024 17.6 against 13.6 for one.  The fp32 tiles are slower.
inline bool few_rows(int dtype, int64_t P, int64_t Q, int64_t R, bool a_deep, bool b_deep) {
  if (!a_deep || R <= 0) return false;
  if (!b_deep) return P <= 4 && Q >= 8 && R <= 2048 && Q * R <= int64_t(1) << 23;
  if (P > 16 || Q <= 0 || R > (1 << 20) || Q > (1 << 25))
    return false;
  const int64_t row = R * (dtype == 2 ? 4 : 2);
  if (16 * row > 210000 + Q * row / 160) return false;
  return dtype == 2 || Q * R * (16 + P) <= int64_t(1) << 30;
}

inline ProductPlan plan_product(int64_t P, int64_t Q, int64_t R, int dtype, bool pack_a,
                                bool a_deep, bool pack_b, bool b_deep, int force_f) {
  ProductPlan p{};
  p.splits = 1;
  p.len = 1;
  if ((dtype == 2 || force_f == 0) && few_rows(dtype, P, Q, R, a_deep, b_deep)) {
    p.few = true;
    return p;
  }
  int64_t best = -1;
  auto consider = [&](const ProductCost& c, int64_t whole, int64_t rest, int64_t s) {
    int64_t t = product_items_ns(whole, R, c) + product_items_ns(rest * s, ceil_div(R, s), c);
    const int64_t edge = tile_edge(c.f);
    if (s > 1) t += kJoinNs + s * rest * edge * edge * 8 / kStreamBytesPerNs;
    if (best >= 0 && t >= best) return;
    best = t;
    p.f = c.f;
    p.whole = s > 1 ? whole : whole + rest;
    p.splits = s;
  };
  for (const ProductCost& c : dtype == 2 ? kProduct32 : kProduct16) {
    if (dtype != 2 && force_f != 0 && c.f != force_f) continue;
    const int64_t tiles = ceil_div(P, tile_edge(c.f)) * ceil_div(Q, tile_edge(c.f));
    consider(c, tiles, 0, 1);
    for (int64_t share = 1; share <= c.share; share *= 2) {
      const int64_t slots = share * kGemmSlots, whole = tiles / slots * slots, rest = tiles - whole;
      if (rest == 0) continue;
      const int64_t most = slots / rest < R / 256 ? slots / rest : R / 256;
      // 2, 3, 4, 6, 8, 12, ... and the most: this runs in every call
      for (int64_t s = 2; s < most; s += s & (s - 1) ? s / 3 : s / 2) consider(c, whole, rest, s);
      if (most > 1) consider(c, whole, rest, most);
    }
  }
  p.len = ceil_div(ceil_div(R, p.splits), 4 * kTileR) * 4 * kTileR;
  if (R > 0) p.splits = ceil_div(R, p.len);
  if (p.len < 1) p.len = 1;
  p.np = ceil_div(P, tile_edge(p.f));
  p.nq = ceil_div(Q, tile_edge(p.f));
  const int64_t rest = p.np * p.nq - p.whole;
  if (p.splits == 1) p.whole += rest;
  // fp32 operands are read four elements at a time, from any address, and need as many
  if (dtype == 2) {
    pack_a = (a_deep ? R : P) < 4;
    pack_b = (b_deep ? R : Q) < 4;
  }
  const int64_t es = elem_size(dtype);
  auto packed = [es](int64_t rows, int64_t deep_len, bool deep) {
    const int64_t n = deep ? rows : deep_len, c = deep ? deep_len : rows;
    return (size_t)(n * packed_ld(c) * es);
  };
  if (R > 0 && pack_a) {
    p.pack_a = true;
    p.ws_bytes += packed(P, R, a_deep);
  }
  if (R > 0 && pack_b) {
    p.pack_b = true;
    p.pack_b_at = p.ws_bytes;
    p.ws_bytes += packed(Q, R, b_deep);
  }
  if (p.splits > 1) {
    p.part_at = p.ws_bytes;
    p.ws_bytes += (size_t)(p.splits * rest * tile_edge(p.f) * tile_edge(p.f)) * sizeof(float);
  }
  return p;
}

// Workspace of the linear layer's backward pass, from its start: dz (where there is an activation;
// rows of packed_ld), the partial rows of db, then, from a line's start on, what the products take
// one after the other.
struct LinearBwdPlan {
  ActBwdPlan act;
  int64_t lddz;
  size_t part_at;
  size_t product_at;
};

inline LinearBwdPlan plan_linear_bwd(int64_t M, int64_t N, int act, int dtype) {
  LinearBwdPlan p{};
  p.act = plan_act_bwd(M, N);
  p.lddz = packed_ld(N);
  p.part_at = act != 0 ? (size_t)(M * p.lddz * elem_size(dtype)) : 0;
  p.product_at = p.part_at + (size_t)(ceil_div(p.act.parts * p.act.np, 32) * 128);
  return p;
}

// Operators on logits [R, V]: a workgroup of `threads` reads a row, or one of `split` segments
// of `seg` chunks (8 elements) where the rows alone do not fill the GPU.  Segments are whole
// passes of 256 threads (64 bytes each); a split row leaves the segments' sums (12 bytes each)
// and, for its top entries, row_max group maxima (fp32, one to a thread and pass, from byte
// max_at on) in the workspace.
struct VocabPlan {
  int threads, split;
  int64_t seg;
  int64_t row_max;
  size_t max_at;
  size_t stat_at;    // of the distillation's two-kernel form, past ws_bytes of the forward
  size_t ws_bytes;
};

// The distillation loss with its gradient reads the logits once where a workgroup can hold a row
// in registers (64 to 256 KiB of them) and, for the longer rows, there are enough rows: one row
// of 131072 bf16 takes 23 us so and 13 us split over the two kernels, 128 of them 24 and 31 us;
// of 65536, 16 rows 15.6 and 14.6, 80 rows 16.9 and 17.8 us.  The two kernels hand 8 bytes a row
// on through the workspace.
inline bool distill_held(int64_t R, int64_t V, int dtype) {
  const int64_t v = V * (dtype == 2 ? 2 : 1);   // in 16-bit units
  return v <= 32768 || (v <= 131072 && R * 1024 >= v);
}

inline VocabPlan plan_vocab(int64_t R, int64_t V, int64_t top, int dtype) {
  VocabPlan p{};
  const int64_t pass = dtype == 2 ? 512 : 1024;   // chunks
  const int64_t passes = ceil_div(V, 8 * pass);
  int64_t split = R < 512 ? ceil_div(1024, R < 1 ? 1 : R) : 1;
  if (split > passes) split = passes;
  if (split > 64) split = 64;
  if (split < 1) split = 1;
  p.seg = ceil_div(passes, split) * pass;
  p.split = (int)ceil_div(passes * pass, p.seg);
  p.threads = V <= 4096 ? 64 : 256;
  p.row_max = passes * 256;
  if (p.split > 1) {
    p.max_at = (size_t)ceil_div(R * p.split * 12, 16) * 16;
    p.ws_bytes = p.max_at + (top > 0 ? (size_t)(R * p.row_max) * 4 : 0);
  }
  p.stat_at = (p.ws_bytes + 15) / 16 * 16;
  return p;
}

inline size_t distill_ws_bytes(const VocabPlan& p, int64_t R, int64_t V, int dtype) {
  return distill_held(R, V, dtype) ? p.ws_bytes : p.stat_at + (size_t)R * 8;
}

}  // namespace swg
