// Operators over rows of logits z [R, V]: token log probabilities with entropy and top
// alternatives, and distillation from a teacher's top logits, each with its gradient.
//
//   a = z / T,  lse = log sum exp a,  p = exp(a - lse)   (p = 0 where z = -inf)
//   logprob = a_t - lse,  H = - sum p (a - lse)
//   da_v = g (1[v = t] - p_v) - h p_v (a_v - lse + H),  dz = da / T
//
//   teacher entries (u_j, id_j), an id outside [0, V) is padding:
//   q = softmax of u / T over the entries,  Q = sum q (1, or 0 if no entry counts)
//   L = T^2 sum_j q_j (log q_j - a_{id_j} + lse)
//   dz_v = c T (Q p_v - sum_{j: id_j = v} q_j);  0 where c = 0
//
// A row of nothing but -inf has lse = -inf, p = 0, log probabilities -inf and H = 0.
#include "launch.hpp"
#include "rows.hpp"

namespace swg {

// ------------------------------------------------------------------ a row as chunks
// A row is read as up to 7 single elements that lead to a 16-byte boundary, chunks of 8
// elements, and up to 7 single elements.
struct RowCut {
  int head, tail;
  int64_t chunks;
  template <typename T> __device__ inline RowCut(const T* z, int64_t V) {
    const int over = (int)((reinterpret_cast<uintptr_t>(z) & 15) / sizeof(T));
    const int64_t h = over ? 16 / (int)sizeof(T) - over : 0;
    head = (int)(h < V ? h : V);
    chunks = (V - head) >> 3;
    tail = (int)((V - head) & 7);
  }
  // the element index of the single element thread t takes, or -1
  __device__ inline int single(int t, int64_t V, bool first, bool last) const {
    if (t < head) return first ? t : -1;
    if (t >= 8 && t < 8 + tail) return last ? (int)V - tail + (t - 8) : -1;
    return -1;
  }
};

template <typename T> struct Fill;   // a chunk's word of masked entries
template <> struct Fill<bf16> { static constexpr uint32_t kNegInf = 0xff80ff80u; };
template <> struct Fill<fp16> { static constexpr uint32_t kNegInf = 0xfc00fc00u; };
template <> struct Fill<float> { static constexpr uint32_t kNegInf = 0xff800000u; };

template <typename T> __device__ inline void fill_masked(Chunk<T>& c) {
  constexpr uint32_t v = Fill<T>::kNegInf;
#pragma unroll
  for (int i = 0; i < Chunk<T>::NV; ++i) c.v[i] = u32x4{v, v, v, v};
}

constexpr float kLowest = -3.4028234663852886e38f;

// Sums of a softmax over values z relative to a value m: s = sum 2^d, t = sum d 2^d for
// d = (z - m) c, c = log2(e) / T; m is at least the lowest finite number, so that differences
// stay defined over masked entries.  A masked entry has 2^d = 0; its d is bounded where it is
// multiplied.  A NaN or +inf makes s and t NaN.
struct Soft {
  float m, s, t;
};
__device__ inline float bound_d(float d) { return __builtin_fmaxf(d, -1000.0f); }

// the same sums relative to m >= a.m
__device__ inline void soft_move(Soft& a, float m, float c) {
  const float d = bound_d((a.m - m) * c);
  const float w = __builtin_amdgcn_exp2f(d);
  a.t = w * __builtin_fmaf(d, a.s, a.t);
  a.s *= w;
  a.m = m;
}

template <bool ENT> __device__ inline void soft_add(Soft& a, float z, float c) {
  const float d = (z - a.m) * c;
  const float e = __builtin_amdgcn_exp2f(d);
  a.s += e;
  if constexpr (ENT) a.t = __builtin_fmaf(bound_d(d), e, a.t);
}

// The running form, where an element costs one fma, one exponential, an addition and the fma
// of t: d = z c - b against a reference b that need not be the maximum.  b moves only when a
// chunk's largest d passes kLift, so that few waves ever branch; up to there an fp32 sum loses
// nothing.  m is the largest value (-inf for none; NaN does not count).
struct Run {
  float b, m, s, t;
};
constexpr float kLift = 4.0f;
// b is a rounded product, and the rounding, up to half a unit of its last place, remains in the d
// of the element it comes from: harmless while it is a few units, as the sums are relative to b
// as it is.  At -1e10 it reaches 512, where 2^d is infinite or 0.  So a value far below (a finite
// mask) takes no part in the reference: its chunk leaves b where it was, at least kNoRef = -2^28
// (2^d <= 2^8 there), and adds 0.  A row whose maximum has |m c| >= kRange = 2^26 (all of it
// masked, or T tiny) has its sums formed again in the differences z - m.
constexpr float kNoRef = -268435456.0f;
constexpr float kRange = 67108864.0f;
__device__ inline bool run_in_range(float m, float c) {
  return __builtin_fabsf(m * c) < kRange || __builtin_fabsf(m) == __builtin_inff();
}

__device__ inline void run_move(Run& a, float b) {
  const float d = bound_d(a.b - b);
  const float w = __builtin_amdgcn_exp2f(d);
  a.t = w * __builtin_fmaf(d, a.s, a.t);
  a.s *= w;
  a.b = b;
}

// The instructions themselves: the language's maximum first makes a signaling NaN of either
// operand quiet, one instruction each.
__device__ inline float max3(float x, float y, float z) {
  float r;
  asm("v_max3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(x), "v"(y), "v"(z));
  return r;
}
__device__ inline float max2(float x, float y) {
  float r;
  asm("v_max_f32 %0, %1, %2" : "=v"(r) : "v"(x), "v"(y));
  return r;
}
__device__ inline float max8(const float* f) {
  return max2(max3(max3(f[0], f[1], f[2]), f[3], f[4]), max3(f[5], f[6], f[7]));
}

// 8 elements, the largest of which is gm
template <bool ENT> __device__ inline void run_chunk(Run& a, const float* f, float gm, float c) {
  a.m = max2(a.m, gm);
  const float top = gm * c;
  if (top - a.b > kLift) run_move(a, top);
  const float t0 = a.t;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float d = __builtin_fmaf(f[i], c, -a.b);
    const float e = __builtin_amdgcn_exp2f(d);
    a.s += e;
    if constexpr (ENT) a.t = __builtin_fmaf(d, e, a.t);
  }
  if constexpr (ENT) {
    // masked entries, -inf times 0: the chunk's exponentials again, for the whole wave (1021 x
    // 50021 fp32, every 16th entry masked, so every wave and chunk: 49.9 us, unmasked 48.3)
    if (a.t != a.t) {
      a.t = t0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float d = __builtin_fmaf(f[i], c, -a.b);
        a.t = __builtin_fmaf(bound_d(d), __builtin_amdgcn_exp2f(d), a.t);
      }
    }
  }
}

__device__ inline void run_single(Run& a, float x, float c) {
  a.m = __builtin_fmaxf(a.m, x);
  const float top = x * c;
  if (top - a.b > kLift) run_move(a, top);
  // not top - b: the product's rounding, half a unit of the last place of top, would stay in d
  // here and not in the chunks' d
  const float d = __builtin_fmaf(x, c, -a.b), e = __builtin_amdgcn_exp2f(d);
  a.s += e;
  a.t = __builtin_fmaf(bound_d(d), e, a.t);
}

// over the workgroup, the same in every thread: one barrier.  `red` holds 4 floats a wave and
// may be used again after the next barrier.
template <int NT> __device__ inline void run_block(Run& a, float* red) {
  a.m = wave_max(a.m);
  run_move(a, wave_max(a.b));
  a.s = wave_sum(a.s);
  a.t = wave_sum(a.t);
  if constexpr (NT > 64) {
    f32x4* r = reinterpret_cast<f32x4*>(red);
    if ((threadIdx.x & 63) == 0) r[threadIdx.x >> 6] = f32x4{a.b, a.m, a.s, a.t};
    __syncthreads();
    if constexpr (NT > 256) {   // a lane takes a wave's
      const int lane = threadIdx.x & 15;
      const f32x4 v = lane < NT / 64 ? r[lane] : f32x4{kNoRef, neg_inf(), 0.0f, 0.0f};
      a = Run{v[0], lanes_max<16>(v[1]), v[2], v[3]};
      run_move(a, lanes_max<16>(a.b));
      a.s = lanes_sum<16>(a.s);
      a.t = lanes_sum<16>(a.t);
      return;
    }
    float b = kNoRef;
#pragma unroll
    for (int i = 0; i < NT / 64; ++i) {
      b = __builtin_fmaxf(b, r[i][0]);
      a.m = __builtin_fmaxf(a.m, r[i][1]);
    }
    a.s = a.t = 0.0f;
    a.b = b;
#pragma unroll
    for (int i = 0; i < NT / 64; ++i) {
      Run o{r[i][0], 0.0f, r[i][2], r[i][3]};
      run_move(o, b);
      a.s += o.s;
      a.t += o.t;
    }
  }
}

// relative to the maximum
__device__ inline Soft run_soft(const Run& a, float c) {
  if (a.m == neg_inf()) return Soft{kLowest, a.s, a.t};
  const float d = __builtin_fmaf(a.m, c, -a.b);
  const float w = __builtin_amdgcn_exp2f(-d);
  return Soft{a.m, a.s * w, __builtin_fmaf(-d, a.s, a.t) * w};
}

// What a row's sums give.  log p = (z - m) / T - ls.
struct RowStat {
  float m, ls, lse, entropy;
  bool empty;
};
__device__ inline RowStat row_stat(const Soft& a, float inv_t) {
  RowStat r;
  r.empty = a.s == 0.0f;
  r.m = a.m;
  r.ls = logf(a.s);
  r.lse = r.empty ? neg_inf() : __builtin_fmaf(a.m, inv_t, r.ls);
  r.entropy = r.empty ? 0.0f : r.ls - kLn2 * (a.t / a.s);
  return r;
}
__device__ inline float log_prob(const RowStat& r, float z, float inv_t) {
  return r.empty ? neg_inf() : (z - r.m) * inv_t - r.ls;
}

// ------------------------------------------------------------------ top entries
// A workgroup's selection of the k largest keys of a row.  While the row is read, the largest
// value of every group of chunks is kept (`gmax`).  A value that at least k group maxima
// reach bounds the k-th largest entry from below, and only the groups that reach it, about k
// of them, are read again: their entries from the bound on are the candidates, ordered at the
// end by counting.
//
// The bound comes from a histogram of the maxima, linear in the value between the smallest of
// the threads' largest maxima (there are at least k such threads) and the largest of all: one
// pass and a scan of 512 bins.  Where that leaves too many groups (equal or masked entries),
// it comes from a bisection of the keys, and where equal values leave no bound with few
// groups, the entries above it are candidates and, of those equal to it, the first ones by
// index, found by a scan of the row.  Where the chosen groups hold too many entries (rows in
// order), a bisection of their keys raises the bound.
constexpr int kSlack = 64;          // entries of a tile that may be candidates beyond k
constexpr int kBins = 512;
__host__ __device__ inline int top_groups(int k) { return k + k / 8 + 8; }
// a tile's, the best k so far and the row's single elements
__host__ __device__ inline int top_candidates(int k) { return 2 * k + kSlack + 16; }

// The thread's number as a value the compiler cannot compute ahead: what the selection derives
// from it would otherwise wait in registers through the stream of every row.
__device__ inline int late_thread() {
  int t = (int)threadIdx.x;
  asm volatile("" : "+v"(t));
  return t;
}

template <int NT> struct TopState {
  uint32_t* glist;   // chosen groups
  u64* cand;         // candidates
  u64* best;         // k, in order
  uint32_t* hist;    // kBins, and the partial ranks
  int* count;        // TopCount<NT>::N
  int k;
};
// [0] candidates, [1] chosen groups, [2] the least key of their maxima, then the waves' counts
// and bounds, twice
template <int NT> struct TopCount { static constexpr int N = 4 + 4 * (NT / 64); };

// the sum of the waves' counts; successive calls alternate `half`
template <int NT> __device__ inline int block_count(int wave_count, int* count, int& half) {
  if constexpr (NT == 64) return wave_count;
  int* c = count + 4 + half * (NT / 64);
  half ^= 1;
  if ((threadIdx.x & 63) == 0) c[threadIdx.x >> 6] = wave_count;
  __syncthreads();
  int n = c[0];
#pragma unroll
  for (int i = 1; i < NT / 64; ++i) n += c[i];
  return n;
}

// smallest and largest over the workgroup; a barrier
template <int NT> __device__ inline void block_bounds(float& lo, float& hi, int* count) {
  const int tid = late_thread();
  lo = -wave_max(-lo);
  hi = wave_max(hi);
  if constexpr (NT > 64) {
    float* c = reinterpret_cast<float*>(count + 4 + 2 * (NT / 64));
    if ((tid & 63) == 0) {
      c[(tid >> 6) * 2] = lo;
      c[(tid >> 6) * 2 + 1] = hi;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NT / 64; ++i) {
      lo = __builtin_fminf(lo, c[i * 2]);
      hi = __builtin_fmaxf(hi, c[i * 2 + 1]);
    }
  } else {
    __syncthreads();
  }
}

// Bins of the histogram: falling values, equal ones together.
struct Bins {
  float hi, scale;
  __device__ inline Bins(float lo, float hi_) : hi(hi_) {
    scale = (float)(kBins - 1) / (hi - lo);
  }
  // scale is 0 where hi - lo leaves fp32: values then have no bin
  __device__ inline bool usable(float lo) const {
    return lo > neg_inf() && lo < hi && hi < __builtin_inff() && scale > 0.0f &&
           scale < __builtin_inff();
  }
  __device__ inline float at(float v) const { return (hi - v) * scale; }
  __device__ inline void add(uint32_t* hist, float v) const {
    const int b = (int)at(v);
    atomicAdd(&hist[b < kBins ? b : kBins - 1], 1u);
  }
};

// From a complete histogram: the fewest first bins that hold k, as `limit` (a value v is in
// them if bins.at(v) < limit); returns how many they hold, 0 if all together hold fewer.  Every
// wave scans by itself, kBins / 64 bins to a lane.
__device__ inline int hist_bound(const uint32_t* hist, int k, float& limit) {
  const int tid = late_thread();
  constexpr int PER = kBins / 64;
  const int lane = tid & 63;
  int c[PER], sum = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    c[i] = (int)hist[lane * PER + i];
    sum += c[i];
  }
  int incl = sum;
  incl += __builtin_amdgcn_update_dpp(0, incl, 0x111, 0xf, 0xf, false);
  incl += __builtin_amdgcn_update_dpp(0, incl, 0x112, 0xf, 0xf, false);
  incl += __builtin_amdgcn_update_dpp(0, incl, 0x114, 0xf, 0xf, false);
  incl += __builtin_amdgcn_update_dpp(0, incl, 0x118, 0xf, 0xf, false);
  incl += __builtin_amdgcn_update_dpp(0, incl, 0x142, 0xa, 0xf, false);
  incl += __builtin_amdgcn_update_dpp(0, incl, 0x143, 0xc, 0xf, false);
  const u64 over = __ballot(incl >= k);
  if (over == 0) return 0;
  int run = incl - sum, bin = 0, reach = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    run += c[i];
    if (reach == 0 && run >= k) {
      reach = run;
      bin = lane * PER + i + 1;
    }
  }
  const int at = __builtin_ctzll(over);
  const int bins = __builtin_amdgcn_readlane(bin, at);
  limit = bins >= kBins ? __builtin_inff() : (float)bins;   // the last bin has no lower end
  return __builtin_amdgcn_readlane(reach, at);
}

// Bisects for a bound: `lo` such that at least k of n keys are >= lo and either no more than
// `most`, or lo + 1 is reached by fewer than k.  count_from(x) is the number of the wave's keys
// >= x.  Returns the count at lo.  The same in every thread; n >= k.
template <int NT, typename K, typename F>
__device__ inline int bisect(F count_from, int n, int k, int most, K hi, int* count, K& lo) {
  int half = 0, at_lo = n;
  lo = 0;
  __syncthreads();
  while (at_lo > most && hi - lo > 1) {
    const K mid = lo + (hi - lo) / 2;
    const int c = block_count<NT>(count_from(mid), count, half);
    if (c >= k) {
      lo = mid;
      at_lo = c;
    } else {
      hi = mid;
    }
  }
  __syncthreads();
  return at_lo;
}

// the k largest of the n candidates to `best`, in falling order; called after a barrier, ends
// with one.  The rank of a key is the number of larger ones: a wave takes 64 keys against a
// share of all of them.
template <int NT> __device__ inline void order_top(const TopState<NT>& w, int n) {
  const int tid = late_thread();
  constexpr int WAVES = NT / 64;
  const int lane = tid & 63, wave = tid >> 6;
  const int blocks = (n + 63) / 64;
  const int parts = blocks > 0 && blocks <= WAVES ? WAVES / blocks : 1;
  if (parts == 1) {
    for (int i = tid; i < n; i += NT) {
      const u64 key = w.cand[i];
      int rank = 0;
#pragma unroll 8
      for (int j = 0; j < n; ++j) rank += w.cand[j] > key;
      if (rank < w.k) w.best[rank] = key;
    }
  } else {
    const int len = (n + parts - 1) / parts;
    const int i = (wave % blocks) * 64 + lane, part = wave / blocks;
    u64 key = 0;
    if (part < parts && i < n) {
      key = w.cand[i];
      const int j1 = (part + 1) * len < n ? (part + 1) * len : n;
      int rank = 0;
#pragma unroll 8
      for (int j = part * len; j < j1; ++j) rank += w.cand[j] > key;
      w.hist[part * (blocks * 64) + i] = (uint32_t)rank;
    }
    __syncthreads();
    if (part == 0 && i < n) {
      int rank = 0;
      for (int q = 0; q < parts; ++q) rank += (int)w.hist[q * (blocks * 64) + i];
      if (rank < w.k) w.best[rank] = key;
    }
  }
  __syncthreads();
}

// the candidates of one tile: chunks [t0, t1) of `body`, whose first element is entry `first`
// of the row; groups of GU chunks, NT apart.  Element j NT + thread of `gmax` (LDS) is the maximum
// of the thread's group j, written by itself; the histogram is clear.  Group j exists while its
// first chunk does.
template <typename T, int NT, int U, int GU, int SLOTS>
__device__ inline void collect_tile(const TopState<NT>& w, const float* gmax, const T* body,
                                    int64_t first, int64_t t0, int64_t t1) {
  const int tid = late_thread();
  constexpr int NS = SLOTS / NT;
  const int k = w.k, most = top_groups(k);
  const int chunks = (int)(t1 - t0);
  auto exists = [&](int j) {
    return j * (NT * (GU == 1 ? 1 : U)) + tid < chunks;
  };
  // read from LDS where it is used: 16 of them in registers take a wave a SIMD
  auto gv = [&](int j) { return exists(j) ? gmax[j * NT + tid] : neg_inf(); };
  const int groups = GU == 1 ? chunks
                             : chunks / (NT * U) * NT +
                                   (chunks % (NT * U) < NT ? chunks % (NT * U) : NT);
  float least = __builtin_inff(), largest = neg_inf();
#pragma unroll 4
  for (int j = 0; j < NS; ++j) {
    const float v = gv(j);
    largest = max2(largest, v);
    if (exists(j)) least = __builtin_fminf(least, v);
  }
  // between the smallest of the threads' largest maxima (of all where k is above NT) and the
  // largest lie at least k; threads with nothing but masked entries do not count
  float hi = largest, lo = k <= NT ? largest : least;
  if (lo == neg_inf()) lo = __builtin_inff();
  if (tid == 0) {
    w.count[1] = 0;
    w.count[2] = -1;
  }
  block_bounds<NT>(lo, hi, w.count);
  const int before = w.count[0];
  const Bins bins(lo, hi);
  uint32_t bound = 0;   // least key of the groups
  float limit = __builtin_inff();
  bool by_value = false, ties = false;
  if (groups > most) {
    int reach = 0;
    if (bins.usable(lo)) {
#pragma unroll 4
      for (int j = 0; j < NS; ++j) {
        const float v = gv(j);
        if (exists(j) && v >= lo) bins.add(w.hist, v);
      }
      __syncthreads();
      reach = hist_bound(w.hist, k, limit);
    }
    by_value = reach >= k && reach <= most;
    if (!by_value) {
      reach = bisect<NT, uint32_t>([&](uint32_t x) {
        int c = 0;
#pragma unroll 1
        for (int j = 0; j < NS; ++j) c += __popcll(__ballot(exists(j) && value_key(gv(j)) >= x));
        return c;
      }, groups, k, most, value_key(hi) + 1, w.count, bound);
      ties = reach > most;   // too many groups at the bound itself
      bound = bound == 0 ? value_key(neg_inf()) : bound;
    }
  }
#pragma unroll 2
  for (int j = 0; j < NS; ++j) {
    const float v = gv(j);
    if (!exists(j)) break;
    if (by_value ? v >= lo && bins.at(v) < limit : value_key(v) >= bound + ties) {
      w.glist[atomicAdd(&w.count[1], 1)] = (uint32_t)(j * NT + tid);
      if (by_value) atomicMin(reinterpret_cast<uint32_t*>(&w.count[2]), value_key(v));
    }
  }
  __syncthreads();
  // an entry is a candidate from the bound on, with ties from the next value on; a NaN ranks with
  // -inf: it passes, or with ties comes in the scan
  const float cut = key_value(by_value ? (uint32_t)w.count[2]
                                       : groups > most ? bound : value_key(neg_inf()));
  const float next = ties ? key_value(value_key(cut) + 1) : cut;
  auto passes = [&](float v) { return !(v < next); };
  const int chosen = w.count[1];
  auto each_chunk = [&](auto use) {   // of the chosen groups
    for (int i = tid; i < chosen * GU; i += NT) {
      const int g = (int)w.glist[i / GU], u = i % GU;
      const int q = GU == 1 ? g : (g / NT) * (NT * U) + u * NT + g % NT;
      if (q >= chunks) continue;
      Chunk<T> c;
      c.load(body + (t0 + q) * 8);
      float f[8];
      c.widen(f);
      use(f, (uint32_t)(first + (t0 + q) * 8));
    }
  };
  const int room = before + k + kSlack;
  u64 lowest = 0;
  for (;;) {
    each_chunk([&](const float* f, uint32_t id) {
      uint32_t hits = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) hits |= (uint32_t)passes(f[e]) << e;
      if (ties || lowest != 0) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if ((ties && f[e] != f[e]) || entry_key(f[e], id + e) < lowest) hits &= ~(1u << e);
      }
      if (hits == 0) return;
      int at = atomicAdd(&w.count[0], __popc(hits));
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (hits >> e & 1) {
          if (at < room) w.cand[at] = entry_key(f[e], id + e);
          ++at;
        }
      }
    });
    __syncthreads();
    const int have = w.count[0];
    if (have <= room) break;
    bisect<NT, u64>([&](u64 x) {
      int c = 0;
      each_chunk([&](const float* f, uint32_t id) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          c += passes(f[e]) && !(ties && f[e] != f[e]) && entry_key(f[e], id + e) >= x;
      });
      return (int)lanes_sum<64>((float)c);
    }, have - before, k, k + kSlack, ~0ull, w.count, lowest);
    if (tid == 0) w.count[0] = before;
    __syncthreads();
  }
  if (!ties) return;
  // the first k - (those above) entries equal to the bound, chunk by chunk in the row's order
  int need = k - (w.count[0] - before);
  int half = 0;
  for (int64_t base = t0; base < t1 && need > 0; base += NT) {
    const int64_t q = base + tid;
    float f[8];
    int equal = 0;
    if (q < t1) {
      Chunk<T> c;
      c.load(body + q * 8);
      c.widen(f);
#pragma unroll
      for (int e = 0; e < 8; ++e) equal += value_key(f[e]) == bound;
    }
    // the number before this thread's, in the wave and then over the waves
    int incl = equal;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_up(incl, d);
      if ((tid & 63) >= d) incl += o;
    }
    const int wave_total = __shfl(incl, 63);
    const int total = block_count<NT>(wave_total, w.count, half);
    int rank = incl - equal;
    if constexpr (NT > 64) {
      const int* c = w.count + 4 + (half ^ 1) * (NT / 64);
      for (int i = 0; i < (tid >> 6); ++i) rank += c[i];
    }
    if (q < t1 && equal) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (value_key(f[e]) == bound) {
          if (rank < need)
            w.cand[atomicAdd(&w.count[0], 1)] = entry_key(f[e], (uint32_t)(first + q * 8 + e));
          ++rank;
        }
      }
    }
    need -= total;
  }
  __syncthreads();
}

// the n = min(k, candidates) best become the only candidates, and the histogram is clear
template <int NT> __device__ inline void keep_best(const TopState<NT>& w) {
  const int n = w.count[0] < w.k ? w.count[0] : w.k;
  for (int i = threadIdx.x; i < n; i += NT) w.cand[i] = w.best[i];
  for (int i = threadIdx.x; i < kBins; i += NT) w.hist[i] = 0;
  __syncthreads();
  if (threadIdx.x == 0) w.count[0] = n;
}

// ------------------------------------------------------------------ the teacher's entries
__device__ inline float teacher_value(const VocabArgs& a, int64_t r, int64_t j, int64_t id) {
  if (id < 0 || id >= a.V) return neg_inf();
  const int64_t i = r * a.k + j;
  float u;
  if (a.teacher_dtype == 0) u = to_f32(static_cast<const bf16*>(a.teacher)[i]);
  else if (a.teacher_dtype == 1) u = to_f32(static_cast<const fp16*>(a.teacher)[i]);
  else u = static_cast<const float*>(a.teacher)[i];
  return u;
}

// An entry as the thread that reads it keeps it: id (-1: does not count) and u.
struct Entry {
  int64_t id;
  float u;
};
__device__ inline Entry load_entry(const VocabArgs& a, int64_t r, int64_t j) {
  Entry e{-1, neg_inf()};
  if (j < a.k) {
    e.id = a.ids[r * a.k + j];
    e.u = teacher_value(a, r, j, e.id);
    if (e.id < 0 || e.id >= a.V) e.id = -1;
  }
  return e;
}

// softmax over the entries: log q = d - lus, d = (u - um) / T, from the differences, which neither
// overflow at the type's lowest value nor lose digits beside a large one.  `mine` is the thread's
// first entry, entry threadIdx.x, whose u becomes its d; those from NT on are read again.
struct Teacher {
  float um, us, lus;
};
__device__ inline float teacher_d(const Teacher& t, const VocabArgs& a, float u) {
  return (u - t.um) * a.inv_t;
}
template <int NT>
__device__ inline Teacher teacher_softmax(const VocabArgs& a, int64_t r, Entry& mine,
                                          float* red) {
  Teacher t;
  float m = mine.u;
  for (int64_t j = threadIdx.x + NT; j < a.k; j += NT)
    m = __builtin_fmaxf(m, load_entry(a, r, j).u);
  m = block_max<NT>(m, red);
  t.um = m == neg_inf() ? 0.0f : m;
  mine.u = teacher_d(t, a, mine.u);
  float s = expf(mine.u);
  for (int64_t j = threadIdx.x + NT; j < a.k; j += NT)
    s += expf(teacher_d(t, a, load_entry(a, r, j).u));
  t.us = block_sum<NT>(s, red);
  t.lus = logf(t.us);
  return t;
}

// q (log q - log p) of one entry
__device__ inline float kl_term(const Teacher& t, const RowStat& st, float d, float z,
                                float inv_t) {
  const float q = expf(d) / t.us;
  if (t.us == 0.0f || q == 0.0f) return 0.0f;
  return q * (d - t.lus - log_prob(st, z, inv_t));
}

// ------------------------------------------------------------------ forward
enum { kLogprobs = 0, kDistill = 1 };

constexpr int64_t kIgnored = -2;

// The results of one row from its sums and, in falling order, its k best keys (null for none).
template <typename T, int NT, int MODE>
__device__ inline void finish_row(const VocabArgs& a, int64_t r, const Soft& sum,
                                  const u64* best, Entry mine, float z_mine, float* red) {
  const T* z = static_cast<const T*>(a.z) + r * a.ld;
  const RowStat st = row_stat(sum, a.inv_t);
  if constexpr (MODE == kLogprobs) {
    if (threadIdx.x == 0) {
      if (a.lse) a.lse[r] = st.lse;
      if (a.entropy) a.entropy[r] = st.entropy;
      if (a.target) {
        float lp = __builtin_nanf("");
        if (mine.id == kIgnored) lp = 0.0f;
        else if (mine.id >= 0) lp = log_prob(st, z_mine, a.inv_t);
        a.logprob[r] = lp;
      }
    }
    for (int j = threadIdx.x; j < (int)a.top; j += NT) {
      const u64 key = best[j];
      a.top_id[r * a.top + j] = key_index(key);
      a.top_logprob[r * a.top + j] = log_prob(st, key_value((uint32_t)(key >> 32)), a.inv_t);
    }
  } else {
    const Teacher t = teacher_softmax<NT>(a, r, mine, red);
    float kl = mine.id >= 0 ? kl_term(t, st, mine.u, z_mine, a.inv_t) : 0.0f;
    for (int64_t j = threadIdx.x + NT; j < a.k; j += NT) {
      const Entry e = load_entry(a, r, j);
      if (e.id >= 0) kl += kl_term(t, st, teacher_d(t, a, e.u), to_f32(z[e.id]), a.inv_t);
    }
    kl = block_sum<NT>(kl, red);
    if (threadIdx.x == 0) {
      a.loss[r] = a.t * a.t * kl;
      if (a.lse) a.lse[r] = st.lse;
      if (a.stat) {
        a.stat[2 * r] = st.empty ? 0.0f : st.m;
        a.stat[2 * r + 1] = st.empty ? 0.0f : st.ls;
      }
    }
  }
}

// what a thread reads of a row ahead of the stream: the target (-1 outside the vocabulary,
// kIgnored), or its first teacher entry
template <int MODE> __device__ inline Entry row_entry(const VocabArgs& a, int64_t r) {
  if constexpr (MODE == kLogprobs) {
    Entry e{-1, neg_inf()};
    if (a.target && threadIdx.x == 0) {
      const int64_t id = a.target[r];
      if (id >= 0 && id < a.V) e.id = id;
      if (id == a.ignore) e.id = kIgnored;
    }
    return e;
  } else {
    return load_entry(a, r, threadIdx.x);
  }
}

extern __shared__ __attribute__((aligned(16))) char swg_vocab_lds[];

// U chunks a thread and pass (64 bytes in flight), the next pass loaded before the present one
// is worked on.
template <typename T> struct Pass { static constexpr int U = sizeof(T) == 2 ? 4 : 2; };

// The thread's chunk of those that start at p, an address that all threads share: it stays in
// scalar registers and the thread adds 32 bits.
template <typename T> __device__ inline const T* lane_at(const T* p) {
  return reinterpret_cast<const T*>(reinterpret_cast<const char*>(p) +
                                    threadIdx.x * (uint32_t)(8 * sizeof(T)));
}
template <typename T> __device__ inline T* lane_at(T* p) {
  return const_cast<T*>(lane_at<T>(static_cast<const T*>(p)));
}

// What a workgroup does about the top entries: nothing, their selection, or, where it has a
// segment of the row only, leaving the group maxima to join_kernel.
enum { kNoTop = 0, kTop = 1, kTopLater = 2 };

// a tile's LDS beside the group maxima
__device__ inline void top_lds_layout(u64* lds, int k, u64*& cand, u64*& best, uint32_t*& hist,
                                      uint32_t*& glist) {
  cand = lds;
  best = cand + top_candidates(k);
  hist = reinterpret_cast<uint32_t*>(best + k);
  glist = hist + kBins;
}
static size_t top_lds_bytes(int k) {
  return sizeof(u64) * (size_t)(top_candidates(k) + k) +
         sizeof(uint32_t) * (size_t)(kBins + top_groups(k));
}

// A row's passes are NT U chunks each and its tiles, over which top entries are selected at a
// time, SLOTS groups of GU chunks.
template <typename T, int NT, int GU, int SLOTS> struct RowShape {
  static constexpr int U = Pass<T>::U;
  static constexpr int64_t PASS = NT * U;
  static constexpr int ITERS = SLOTS * GU / (NT * U);   // passes of a tile
  static constexpr int64_t TILE = ITERS * PASS;
};

// The thread's group maxima over chunks [t0, t1) of `body`, in their places from `out` on, by
// comparisons that pass over NaN.
template <typename T, int NT, int U, int GU>
__device__ inline void remake_groups(float* out, const T* body, int64_t t0, int64_t t1) {
  const int tid = late_thread(), chunks = (int)(t1 - t0);
#pragma unroll 1
  for (int base = 0; base < chunks; base += NT * U) {
    float group = neg_inf();
#pragma unroll 1
    for (int u = 0; u < U; ++u) {
      float gm = neg_inf();
      const int q = base + u * NT + tid;
      if (q < chunks) {
        Chunk<T> c;
        c.load(body + (t0 + q) * 8);
        float f[8];
        c.widen(f);
#pragma unroll
        for (int i = 0; i < 8; ++i) gm = f[i] > gm ? f[i] : gm;
      }
      if constexpr (GU == 1) out[q] = gm;
      group = gm > group ? gm : group;
    }
    if constexpr (GU > 1) out[base / U + tid] = group;
  }
}

// One row, or one segment of it (blockIdx.y of gridDim.y, `seg` chunks each, whole passes), by a
// workgroup of NT threads.  A segment leaves its sums in the workspace; join_kernel finishes the
// row.
//
// 4096 x 131072 bf16 (1.07 GB): 166 us = 6.5 TB/s without top entries, bound by memory with the
// arithmetic (36 issue cycles an element and wave, 16 of them the exponential) at three quarters
// of that; 200 us with 64.  The selection is latency: barriers, a second read of the chosen
// groups (130 MB of the pass's 1203 MB read), and their order, about 10 us a row behind 30 us of
// stream, so five rows share a CU (256 threads a row; two rows of 512 threads take 223 us, four of
// 256 204 us).  The 96 registers that five rows leave hold bf16; fp16 spills 12 bytes a lane (20
// with 64 threads) and takes 204 us.  1021 x 50021 fp32 with 5: 48 us = 4.2 TB/s.  Keeping the k
// best by insertion or by repeated maxima instead reads the row k times: 36.8 ms.
template <typename T, int NT, int GU, int SLOTS, int MODE, int TOP, bool ENT>
__global__ __launch_bounds__(NT, 5) void rows_kernel(VocabArgs a, int64_t seg, Soft* part,
                                                     float* part_max, int64_t row_max) {
  using Shape = RowShape<T, NT, GU, SLOTS>;
  constexpr int U = Shape::U;
  constexpr int64_t PASS = Shape::PASS, TILE = Shape::TILE;
  __shared__ __attribute__((aligned(16))) float red[NT / 64 * 4];
  __shared__ int count[TopCount<NT>::N];
  __shared__ float gmax[TOP == kTop ? SLOTS : 1];
  TopState<NT> w;
  const int k = (int)a.top;
  if constexpr (TOP == kTop) {
    w.k = k;
    w.count = count;
    top_lds_layout(reinterpret_cast<u64*>(swg_vocab_lds), k, w.cand, w.best, w.hist, w.glist);
  }
  const float c = a.inv_t * kLog2e;
  const int split = (int)gridDim.y, part_i = (int)blockIdx.y;
  for (int64_t r = blockIdx.x; r < a.R; r += gridDim.x) {
    const T* z = static_cast<const T*>(a.z) + r * a.ld;
    const RowCut cut(z, a.V);
    const T* body = z + cut.head;
    const int64_t c0 = part_i * seg, c1 = c0 + seg < cut.chunks ? c0 + seg : cut.chunks;
    const int lone = cut.single(threadIdx.x, a.V, part_i == 0, part_i == split - 1);
    Entry mine{-1, neg_inf()};
    if (split == 1) mine = row_entry<MODE>(a, r);
    float z_lone = lone >= 0 ? to_f32(z[lone]) : neg_inf();
    // one pass: U chunks of the thread, from `base` on, before t1
    auto load = [&](Chunk<T>* ch, int64_t base, int64_t t1) {
      const T* p = body + base * 8;
      const int64_t left = t1 - base;
      if (left >= PASS) {
#pragma unroll
        for (int u = 0; u < U; ++u) ch[u].load_stream(lane_at<T>(p + u * NT * 8));
      } else {
        const int n = (int)left;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          fill_masked(ch[u]);
          if ((int)threadIdx.x < n - u * NT) ch[u].load_stream(lane_at<T>(p + u * NT * 8));
        }
      }
    };
    Chunk<T> cur[U], next[U];
    load(cur, c0, TOP == kTop && c0 + TILE < c1 ? c0 + TILE : c1);
    const float z_mine = mine.id >= 0 ? to_f32(z[mine.id]) : 0.0f;

    __syncthreads();   // LDS of the row before
    if constexpr (TOP == kTop) {
      if (threadIdx.x == 0) count[0] = 0;
      for (int i = threadIdx.x; i < kBins; i += NT) w.hist[i] = 0;
      __syncthreads();
    }
    Run sum{kNoRef, neg_inf(), 0.0f, 0.0f};
    if (lone >= 0) {
      run_single(sum, z_lone, c);
      if constexpr (TOP == kTop)
        w.cand[atomicAdd(&count[0], 1)] = entry_key(z_lone, (uint32_t)lone);
    }
    for (int64_t t0 = c0; t0 < c1; t0 += TILE) {
      const int64_t t1 = TOP == kTop && t0 + TILE < c1 ? t0 + TILE : c1;
      float* out_max = nullptr;
      if constexpr (TOP == kTop) out_max = gmax + threadIdx.x;
      if constexpr (TOP == kTopLater)
        out_max = part_max + r * row_max + t0 / GU + threadIdx.x;
      for (int64_t base = t0; base < t1; base += PASS) {
        load(next, base + PASS, t1);
        float group = neg_inf();
#pragma unroll
        for (int u = 0; u < U; ++u) {
          float f[8];
          cur[u].widen(f);
          float gm = max8(f);
          if constexpr (TOP != kNoTop) {
            // 8 NaN come out as NaN; what others may hide is looked for behind the loop
            if (gm != gm) {
              gm = neg_inf();
#pragma unroll
              for (int i = 0; i < 8; ++i) gm = f[i] > gm ? f[i] : gm;
            }
            if constexpr (GU == 1) out_max[u * NT] = gm;
            group = max2(group, gm);
          }
          run_chunk<ENT>(sum, f, gm, c);
        }
        if constexpr (TOP != kNoTop) {
          if constexpr (GU > 1) out_max[0] = group;
          out_max += GU > 1 ? NT : PASS;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) cur[u] = next[u];
      }
      if constexpr (TOP != kNoTop) {
        // A NaN may have hidden others of its chunk from max8 (the maximum with a signaling NaN is
        // NaN, the next one drops it).  It is in the thread's sum, and the groups are formed again.
        if (sum.s != sum.s) {
          float* out = TOP == kTop ? gmax : part_max + r * row_max + t0 / GU;
          remake_groups<T, NT, U, GU>(out, body, t0, t1);
        }
      }
      if constexpr (TOP == kTop) {
        collect_tile<T, NT, U, GU, SLOTS>(w, gmax, body, cut.head, t0, t1);
        order_top<NT>(w, count[0]);
        if (t1 < c1) {   // the best so far are the next tile's first candidates
          keep_best<NT>(w);
          load(cur, t1, t1 + TILE < c1 ? t1 + TILE : c1);
        }
      } else {
        break;
      }
    }
    run_block<NT>(sum, red);
    Soft soft;
    if (run_in_range(sum.m, c)) {
      soft = run_soft(sum, c);
    } else {
      soft = Soft{sum.m, 0.0f, 0.0f};
      if (lone >= 0) soft_add<ENT>(soft, z_lone, c);
      for (int64_t q = c0 + threadIdx.x; q < c1; q += NT) {
        Chunk<T> ch;
        ch.load(body + q * 8);
        float f[8];
        ch.widen(f);
#pragma unroll
        for (int i = 0; i < 8; ++i) soft_add<ENT>(soft, f[i], c);
      }
      __syncthreads();
      soft.s = block_sum<NT>(soft.s, red);
      soft.t = block_sum<NT>(soft.t, red);
    }
    if (split > 1) {
      if (threadIdx.x == 0) part[r * split + part_i] = soft;
    } else {
      if constexpr (TOP == kTop) {
        if (c1 == 0) {   // a row of single elements
          __syncthreads();
          order_top<NT>(w, count[0]);
        }
      }
      finish_row<T, NT, MODE>(a, r, soft, TOP == kTop ? w.best : nullptr, mine, z_mine, red);
    }
  }
}

// Joins a row's segments (at most 64) and selects its top entries from the group maxima they
// left (`row_max` a row).  One row of 131072 bf16 with 20 entries: 4.4 us for the segments and
// 12 us here, most of it code that is fetched for the first time and waits for four loads in a
// row; with a selection in each segment and the join of their best 27 us together.
template <typename T, int GU, int SLOTS, int MODE, int TOP>
__global__ __launch_bounds__(256, 4) void join_kernel(VocabArgs a, int split, const Soft* part,
                                                      const float* part_max, int64_t row_max) {
  constexpr int NT = 256;
  constexpr int64_t TILE = RowShape<T, NT, GU, SLOTS>::TILE;
  __shared__ __attribute__((aligned(16))) float red[NT / 64 * 4];
  __shared__ int count[TopCount<NT>::N];
  __shared__ float gmax[TOP == kTop ? SLOTS : 1];
  const float c = a.inv_t * kLog2e;
  TopState<NT> w;
  const int k = (int)a.top;
  if constexpr (TOP == kTop) {
    w.k = k;
    w.count = count;
    top_lds_layout(reinterpret_cast<u64*>(swg_vocab_lds), k, w.cand, w.best, w.hist, w.glist);
  }
  for (int64_t r = blockIdx.x; r < a.R; r += gridDim.x) {
    const T* z = static_cast<const T*>(a.z) + r * a.ld;
    const Entry mine = row_entry<MODE>(a, r);
    const int lane = threadIdx.x & 63;   // every wave joins the sums by itself
    Soft soft{kLowest, 0.0f, 0.0f};
    if (lane < split) soft = part[r * split + lane];
    float z_mine = 0.0f;
    if constexpr (TOP == kTop) {
      constexpr int U = Pass<T>::U;
      const RowCut cut(z, a.V);
      const int lone = cut.single(threadIdx.x, a.V, true, true);
      const float* maxima = part_max + r * row_max;
      const float z_lone = lone >= 0 ? to_f32(z[lone]) : 0.0f;
      // the thread's own groups; past the row's end the workspace holds them up to row_max only
      auto fetch = [&](int64_t t0) {
        const float* from = maxima + t0 / GU;
        const int n = (int)(row_max - t0 / GU < SLOTS ? row_max - t0 / GU : SLOTS);
#pragma unroll 4
        for (int i = threadIdx.x; i < n; i += NT) gmax[i] = from[i];
      };
      fetch(0);
      if (mine.id >= 0) z_mine = to_f32(z[mine.id]);
      __syncthreads();   // LDS of the row before
      if (threadIdx.x == 0) count[0] = 0;
      for (int i = threadIdx.x; i < kBins; i += NT) w.hist[i] = 0;
      __syncthreads();
      if (lone >= 0) w.cand[atomicAdd(&count[0], 1)] = entry_key(z_lone, (uint32_t)lone);
      for (int64_t t0 = 0;;) {   // a split row has chunks
        const int64_t t1 = t0 + TILE < cut.chunks ? t0 + TILE : cut.chunks;
        collect_tile<T, NT, U, GU, SLOTS>(w, gmax, z + cut.head, cut.head, t0, t1);
        order_top<NT>(w, count[0]);
        if (t1 >= cut.chunks) break;
        keep_best<NT>(w);
        t0 = t1;
        fetch(t0);
      }
    } else {
      if (mine.id >= 0) z_mine = to_f32(z[mine.id]);
    }
    soft_move(soft, wave_max(soft.m), c);
    soft.s = wave_sum(soft.s);
    soft.t = wave_sum(soft.t);
    finish_row<T, NT, MODE>(a, r, soft, TOP == kTop ? w.best : nullptr, mine, z_mine, red);
  }
}

// ------------------------------------------------------------------ gradients
// The columns that hold more than their probability take part twice: the target is formed in
// the thread that owns its chunk; the teacher's entries are formed apart, from logits that were
// read before anything was written (the call may overwrite them), and stored over what the
// stream wrote once that has arrived.  An entry's column takes off the shares of all entries
// with its id, in their order, so repeated ids write equal values.
struct TeacherLds {
  int* id;       // k; -1 does not count
  float* share;  // q
  float* z;      // the logit at id
};
__device__ inline TeacherLds teacher_lds(int64_t k) {
  TeacherLds t;
  t.id = reinterpret_cast<int*>(swg_vocab_lds);
  t.share = reinterpret_cast<float*>(t.id + k);
  t.z = t.share + k;
  return t;
}
static size_t teacher_lds_bytes(int64_t k) { return (size_t)k * 12; }

// fills it (not yet visible to other threads), with the logits of entries in [from, to); `mine`
// and z_mine are the thread's first entry
template <typename T, int NT>
__device__ inline void teacher_fill(const TeacherLds& l, const VocabArgs& a, int64_t r,
                                    const T* z, const Teacher& t, const Entry& mine,
                                    float z_mine, int64_t from, int64_t to) {
  Entry e = mine;
  float x = z_mine;
  for (int64_t j = threadIdx.x; j < a.k; j += NT) {
    if (j >= NT) {
      e = load_entry(a, r, j);
      e.u = teacher_d(t, a, e.u);
      x = e.id >= from && e.id < to ? to_f32(z[e.id]) : 0.0f;
    }
    const bool counts = e.id >= 0 && t.us != 0.0f;
    l.id[j] = counts ? (int)e.id : -1;
    l.share[j] = counts ? expf(e.u) / t.us : 0.0f;
    l.z[j] = x;
  }
}

// stores the entries with columns in [from, to); prob gives a logit's probability
template <typename T, int NT, typename F>
__device__ inline void teacher_store(const TeacherLds& l, const VocabArgs& a, T* dz,
                                     int64_t from, int64_t to, float scale, F prob) {
  const int k = (int)a.k;
  // the stream's stores have arrived before one of them is overwritten
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
  for (int j = threadIdx.x; j < k; j += NT) {
    const int id = l.id[j];
    if (id < from || id >= to || id < 0) continue;
    float q = 0.0f;
#pragma unroll 8
    for (int i = 0; i < k; ++i) q += l.id[i] == id ? l.share[i] : 0.0f;
    dz[id] = from_f32<T>(scale * (prob(l.z[j]) - q));
  }
}

// A workgroup forms one of `split` segments of a row, `seg` chunks each.  Bound by memory:
// [2048, 65536] bf16 log probabilities, 537 MB, 89 us = 6.0 TB/s; [2047, 50021] bf16 with 32
// teacher entries into rows that start anywhere, 410 MB, 86 us = 4.8 TB/s (82 us where both
// rows start at lines; temporal stores 77 us; 102 us without the passes' start at a line and the
// loads ahead, 2.9 ms with a search of the entries for every column).
template <typename T, int NT, int MODE>
__global__ __launch_bounds__(NT) void grad_kernel(VocabArgs a, int split, int64_t seg) {
  constexpr int U = Pass<T>::U;
  __shared__ float red[NT / 64];
  // a wave's chunks of a pass follow each other
  const int first = (int)(threadIdx.x >> 6) * (64 * U) + (int)(threadIdx.x & 63);
  const TeacherLds lds = teacher_lds(MODE == kDistill ? a.k : 0);
  for (int64_t item = blockIdx.x; item < a.R * split; item += gridDim.x) {
    const int64_t r = item / split, part_i = item % split;
    const T* z = static_cast<const T*>(a.z) + r * a.ld;
    T* dz = static_cast<T*>(a.dz) + r * a.lddz;
    const RowCut cut(dz, a.V);
    const T* body = z + cut.head;
    T* out = dz + cut.head;
    const int64_t c0 = part_i * seg < cut.chunks ? part_i * seg : cut.chunks;
    const int64_t c1 = c0 + seg < cut.chunks ? c0 + seg : cut.chunks;
    const int lone = cut.single(threadIdx.x, a.V, part_i == 0, part_i == split - 1);
    const float z_lone = lone >= 0 ? to_f32(z[lone]) : 0.0f;
    Entry mine{-1, neg_inf()};
    if constexpr (MODE == kDistill) mine = load_entry(a, r, threadIdx.x);
    // log p = (z - m) / T - ls; with only lse, which rounds ls off beside a large m / T, m = 0
    const bool has_stat = MODE == kDistill && a.stat != nullptr;
    const float m = has_stat ? a.stat[2 * r] : 0.0f;
    const float ls_in = has_stat ? a.stat[2 * r + 1] : a.lse_in[r];
    // the segment's columns
    const int64_t from = part_i == 0 ? 0 : cut.head + c0 * 8;
    const int64_t to = part_i == split - 1 ? a.V : cut.head + c1 * 8;
    auto load = [&](Chunk<T>* ch, int64_t base) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t q = base + first + u * 64;
        if (q >= c0 && q < c1) ch[u].load_stream(body + q * 8);
      }
    };
    // passes start at a 128-byte line of the output: waves that share one cost 6 % at rows of
    // 50024 bf16 (73.8 and 78.3 us).  Not so in fp32: 1024 x 65536, where rows start at lines
    // anyway, takes 153 us with the offset and 122 without (107 with temporal stores)
    const int64_t start =
        c0 - (int64_t)((reinterpret_cast<uintptr_t>(out + c0 * 8) & 127) / (8 * sizeof(T)));
    Chunk<T> ch[U], next[U];
    load(ch, start);
    const float ls = ls_in == neg_inf() ? 0.0f : ls_in;   // a row of masked entries: p = 0

    float scale = 0.0f, gain = 0.0f, A = 0.0f, g = 0.0f, h = 0.0f, H = 0.0f;
    int64_t id = -1;
    if constexpr (MODE == kLogprobs) {
      const int64_t t = a.target ? a.target[r] : a.ignore;
      if (a.target && t != a.ignore) {
        g = a.dlogprob[r];
        if (t < 0 || t >= a.V) g = __builtin_nanf("");
        else id = t;
      }
      if (a.dentropy) {
        h = a.dentropy[r];
        H = a.entropy_in[r];
      }
      A = __builtin_fmaf(h, H, g);
      gain = -a.inv_t;
    } else {
      const float wgt = a.dloss[r];
      if (wgt == 0.0f) {
        Chunk<T> zero;
        zero.zero();
        for (int64_t q = c0 + threadIdx.x; q < c1; q += NT) zero.store_stream(out + q * 8);
        if (lone >= 0) dz[lone] = from_f32<T>(0.0f);
        continue;
      }
      scale = wgt * a.t;
      const bool here = mine.id >= from && mine.id < to;
      const float z_mine = here ? to_f32(z[mine.id]) : 0.0f;
      const Teacher t = teacher_softmax<NT>(a, r, mine, red);   // with barriers
      gain = t.us == 0.0f ? 0.0f : scale;
      teacher_fill<T, NT>(lds, a, r, z, t, mine, z_mine, from, to);
      __syncthreads();   // all entries' logits are read
    }
    // log p: at most 0, also where lse is too coarse beside a large |x| / T, so that p stays a
    // probability.  A NaN stays one.
    auto value = [&](float x) {
      return __builtin_elementwise_minimum(__builtin_fmaf(x - m, a.inv_t, -ls), 0.0f);
    };
    auto prob = [&](float x) { return __builtin_amdgcn_exp2f(value(x) * kLog2e); };
    auto at_target = [&](float x) {
      // g (1 - p) is of the size of g: the division by T in fp64 leaves one rounding to fp32
      // where the product with 1/T would leave three
      const float lp = value(x), p = prob(x);
      const double ent = p != 0.0f ? (double)(h * p * (lp + H)) : 0.0;
      return (float)(((double)g * (1.0 - (double)p) - ent) / (double)a.t);
    };
    auto plain = [&](float x) {
      if constexpr (MODE == kLogprobs)
        return prob(x) * __builtin_fmaf(h, __builtin_fmaxf(value(x), -200.0f), A) * gain;
      else
        return gain * prob(x);
    };
    if (lone >= 0) {
      float d = plain(z_lone);
      if (MODE == kLogprobs && lone == id && g != 0.0f) d = at_target(z_lone);
      dz[lone] = from_f32<T>(d);
    }
    for (int64_t base = start; base < c1; base += NT * U) {
      load(next, base + NT * U);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t q = base + first + u * 64;
        if (q < c0 || q >= c1) continue;
        float f[8], d[8];
        ch[u].widen(f);
#pragma unroll
        for (int i = 0; i < 8; ++i) d[i] = plain(f[i]);
        if constexpr (MODE == kLogprobs) {
          const int64_t col = cut.head + q * 8;
          if (id >= col && id < col + 8 && g != 0.0f) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (id == col + i) d[i] = at_target(f[i]);
          }
        }
        Chunk<T> o;
        o.narrow(d);
        o.store_stream(out + q * 8);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) ch[u] = next[u];
    }
    if constexpr (MODE == kDistill) {
      teacher_store<T, NT>(lds, a, dz, from, to, scale, prob);
      __syncthreads();   // LDS of the next item
    }
  }
}

__device__ inline float uniform(float v) {
  return __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(v)));
}

// ------------------------------------------------------------------ distillation in one pass
// Loss, lse and gradient of a row that a workgroup holds in registers, D chunks a thread: the
// logits are read once.  4096 x 131072 bf16 with 64 teacher entries (2.15 GB): 457 us = 4.7 TB/s,
// against 532 us for the two kernels that read them twice.  A row of that length takes a CU's
// registers (1024 threads, 16 chunks each, beside 64 registers for the rest, 12 bytes a lane
// spilled), so its load, its sums and its stores follow each other, and memory rests while the
// sums are formed; loading the next row behind the stores, or forming its sums there as well, came
// to 455 and 494 us (a wait for a load waits for the stores before it too).  Rows of half the length share a CU:
// 2500 x 65536 137 us = 4.8 TB/s, 177 us for the two kernels.
template <typename T, int NT, int D, int WAVES>
__global__ __launch_bounds__(NT, WAVES) void distill_kernel(VocabArgs a) {
  __shared__ __attribute__((aligned(16))) float red[NT / 64 * 4];
  const TeacherLds lds = teacher_lds(a.k);
  const float c = a.inv_t * kLog2e;
  for (int64_t r = blockIdx.x; r < a.R; r += gridDim.x) {
    const T* z = static_cast<const T*>(a.z) + r * a.ld;
    T* dz = static_cast<T*>(a.dz) + r * a.lddz;
    const RowCut cut(z, a.V);   // by the logits: the sums do not depend on where dz lies
    const T* body = z + cut.head;
    T* out = dz + cut.head;
    const int lone = cut.single(threadIdx.x, a.V, true, true);
    Entry mine = load_entry(a, r, threadIdx.x);
    // waited for ahead of the row's loads: 4096 x 131072 takes 469 us where the wait comes behind
    // them, 457 so; shorter rows are 2 to 4 % faster without
    if constexpr (NT == 1024) asm volatile("" : "+v"(mine.u));
    const float wgt = a.dloss[r];
    const float z_lone = lone >= 0 ? to_f32(z[lone]) : 0.0f;
    // chunk u of the thread, if the row has it
    const int chunks = (int)cut.chunks;
    auto has = [&](int u) { return (int)threadIdx.x < chunks - u * NT; };
    Chunk<T> ch[D];
#pragma unroll
    for (int u = 0; u < D; ++u) {
      fill_masked(ch[u]);
      if (has(u))
        ch[u].load_stream(lane_at<T>(body + u * NT * 8));
    }
    const float z_mine = mine.id >= 0 ? to_f32(z[mine.id]) : 0.0f;
    Teacher t = teacher_softmax<NT>(a, r, mine, red);
    t = Teacher{uniform(t.um), uniform(t.us), uniform(t.lus)};
    teacher_fill<T, NT>(lds, a, r, z, t, mine, z_mine, 0, a.V);
    __syncthreads();

    Run sum{kNoRef, neg_inf(), 0.0f, 0.0f};
    if (lone >= 0) run_single(sum, z_lone, c);
#pragma unroll
    for (int u = 0; u < D; ++u) {
      float f[8];
      ch[u].widen(f);
      run_chunk<false>(sum, f, max8(f), c);
      // one chunk after the other, and widened again where it is used again: the fp32 values of
      // many chunks do not fit the registers
      ch[u].forget();
      __builtin_amdgcn_sched_barrier(0);
    }
    run_block<NT>(sum, red);   // all of the row is read
    Soft soft;
    if (run_in_range(sum.m, c)) {
      soft = run_soft(sum, c);
    } else {
      soft = Soft{sum.m, 0.0f, 0.0f};
      if (lone >= 0) soft_add<false>(soft, z_lone, c);
#pragma unroll
      for (int u = 0; u < D; ++u) {
        float f[8];
        ch[u].widen(f);
#pragma unroll
        for (int i = 0; i < 8; ++i) soft_add<false>(soft, f[i], c);
        ch[u].forget();
        __builtin_amdgcn_sched_barrier(0);
      }
      __syncthreads();
      soft.s = block_sum<NT>(soft.s, red);
    }
    // the same in every lane: scalar registers
    soft.m = uniform(soft.m);
    soft.s = uniform(soft.s);
    const RowStat st = row_stat(soft, a.inv_t);
    float kl = 0.0f;
    for (int j = threadIdx.x; j < (int)a.k; j += NT)
      if (lds.id[j] >= 0)
        kl += kl_term(t, st, j < NT ? mine.u : teacher_d(t, a, load_entry(a, r, j).u), lds.z[j],
                      a.inv_t);
    if constexpr (NT > 64) __syncthreads();
    kl = block_sum<NT>(kl, red);
    if (threadIdx.x == 0) {
      a.loss[r] = a.t * a.t * kl;
      a.lse[r] = st.lse;
    }
    if (wgt == 0.0f) {
      Chunk<T> zero;
      zero.zero();
      for (int q = threadIdx.x; q < chunks; q += NT) zero.store_stream(out + (int64_t)q * 8);
      if (lone >= 0) dz[lone] = from_f32<T>(0.0f);
    } else {
      const float scale = uniform(wgt * a.t);
      const float over = uniform(st.empty ? 0.0f : 1.0f / soft.s);   // p = over 2^((z - m) c)
      const float gain = uniform(t.us == 0.0f ? 0.0f : scale * over);
      auto power = [&](float x) { return __builtin_amdgcn_exp2f((x - soft.m) * c); };
      if (lone >= 0) dz[lone] = from_f32<T>(gain * power(z_lone));
#pragma unroll
      for (int u = 0; u < D; ++u) {
        if (has(u)) {
          float f[8];
          ch[u].widen(f);
#pragma unroll
          for (int i = 0; i < 8; ++i) f[i] = gain * power(f[i]);
          Chunk<T> o;
          o.narrow(f);
          o.store_stream(lane_at<T>(out + u * NT * 8));
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      teacher_store<T, NT>(lds, a, dz, 0, a.V, scale, [&](float x) { return over * power(x); });
    }
    __syncthreads();   // LDS of the next row
  }
}

// ------------------------------------------------------------------ launches
template <typename T, int MODE, bool ENT>
static hipError_t forward_rows(const VocabArgs& a, const VocabPlan& p, void* ws,
                               hipStream_t stream) {
  constexpr int U = Pass<T>::U;
  Soft* part = static_cast<Soft*>(ws);
  float* part_max = reinterpret_cast<float*>(static_cast<char*>(ws) + p.max_at);
  const int k = (int)a.top;
  const size_t lds = k > 0 ? top_lds_bytes(k) : 0;
  const dim3 grid(row_grid(a.R), (unsigned)p.split);
#define SWG_ROWS(NT, GU, SLOTS, TOP)                                                           \
  SWG_LAUNCH((rows_kernel<T, NT, GU, SLOTS, MODE, TOP, ENT>), grid, dim3(NT),                  \
             TOP == kTop ? lds : 0, stream, a, p.seg, part, part_max, p.row_max)
  const bool top = MODE == kLogprobs && k > 0;
  constexpr int kT = MODE == kLogprobs ? kTop : kNoTop;   // distillation has no top entries
  constexpr int kL = MODE == kLogprobs ? kTopLater : kNoTop;
  if (p.split > 1) {
    if (top) SWG_ROWS(256, U, 4096, kL);
    else SWG_ROWS(256, U, 4096, kNoTop);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (top)
      SWG_LAUNCH((join_kernel<T, U, 4096, MODE, kT>), dim3(row_grid(a.R)), dim3(256), lds, stream,
                 a, p.split, part, part_max, p.row_max);
    else
      SWG_LAUNCH((join_kernel<T, U, 4096, MODE, kNoTop>), dim3(row_grid(a.R)), dim3(256), 0,
                 stream, a, p.split, part, part_max, p.row_max);
  } else if (p.threads == 64) {
    if (top) SWG_ROWS(64, 1, 512, kT);
    else SWG_ROWS(64, 1, 512, kNoTop);
  } else if (!top) {
    SWG_ROWS(256, U, 4096, kNoTop);
  } else if constexpr (MODE == kLogprobs) {
    if (a.V <= 32768) SWG_ROWS(256, 1, 4096, kT);
    else SWG_ROWS(256, U, 4096, kT);
  }
#undef SWG_ROWS
  return hipGetLastError();
}

template <typename T, int MODE>
static hipError_t gradient_rows(const VocabArgs& a, hipStream_t stream) {
  const size_t lds = MODE == kDistill ? teacher_lds_bytes(a.k) : 0;
  // Segments of about 16384 elements, 32768 where each prepares the teacher's entries, down to
  // 8192 where rows are few.  [2048, 65536] bf16 log probabilities take 90 us with 16384 and 95
  // with 32768 (fewer workgroups to even out), [2047, 50021] with 32 teacher entries 92 and 88.
  int64_t split = ceil_div(a.V, MODE == kDistill ? 32768 : 16384);
  const int64_t want = ceil_div(2048, a.R), most = ceil_div(a.V, 8192);
  if (split < want) split = want < most ? want : most;
  const int64_t seg = ceil_div(ceil_div(a.V, 8), split * 64) * 64;   // whole lines
  const dim3 grid(row_grid(a.R * split));
  if (a.V <= 2048)
    SWG_LAUNCH((grad_kernel<T, 64, MODE>), grid, dim3(64), lds, stream, a, (int)split, seg);
  else
    SWG_LAUNCH((grad_kernel<T, 256, MODE>), grid, dim3(256), lds, stream, a, (int)split, seg);
  return hipGetLastError();
}

// the one-pass kernel for rows that fit a workgroup's registers, where there are enough of them;
// otherwise `held` becomes false
template <typename T>
static hipError_t distill_rows(const VocabArgs& a, hipStream_t stream, bool& held) {
  const size_t lds = teacher_lds_bytes(a.k);
  const int64_t v = a.V * (int64_t)sizeof(T) / 2;   // in units of 16 bits
  held = true;
#define SWG_HELD(NT, D, WAVES)                                                               \
  SWG_LAUNCH((distill_kernel<T, NT, D * 2 / (int)sizeof(T), WAVES>), dim3(row_grid(a.R)),    \
             dim3(NT), lds, stream, a)
  if (a.stat) held = false;
  else if (v <= 2048) SWG_HELD(64, 4, 4);
  else if (v <= 8192) SWG_HELD(256, 4, 4);
  else if (v <= 16384) SWG_HELD(256, 8, 4);
  else if (v <= 32768) SWG_HELD(512, 8, 4);
  else if (v <= 65536) SWG_HELD(512, 16, 4);
  else SWG_HELD(1024, 16, 4);
#undef SWG_HELD
  return hipGetLastError();
}

hipError_t launch_logprobs(int dtype, const VocabArgs& a, const VocabPlan& p, void* ws,
                           hipStream_t stream) {
  if (dtype == 0) return forward_rows<bf16, kLogprobs, true>(a, p, ws, stream);
  if (dtype == 1) return forward_rows<fp16, kLogprobs, true>(a, p, ws, stream);
  return forward_rows<float, kLogprobs, true>(a, p, ws, stream);
}
hipError_t launch_logprobs_bwd(int dtype, const VocabArgs& a, hipStream_t stream) {
  if (dtype == 0) return gradient_rows<bf16, kLogprobs>(a, stream);
  if (dtype == 1) return gradient_rows<fp16, kLogprobs>(a, stream);
  return gradient_rows<float, kLogprobs>(a, stream);
}
hipError_t launch_distill_fwd(int dtype, const VocabArgs& a, const VocabPlan& p, void* ws,
                              hipStream_t stream) {
  if (dtype == 0) return forward_rows<bf16, kDistill, false>(a, p, ws, stream);
  if (dtype == 1) return forward_rows<fp16, kDistill, false>(a, p, ws, stream);
  return forward_rows<float, kDistill, false>(a, p, ws, stream);
}
hipError_t launch_distill_bwd(int dtype, const VocabArgs& a, hipStream_t stream) {
  if (dtype == 0) return gradient_rows<bf16, kDistill>(a, stream);
  if (dtype == 1) return gradient_rows<fp16, kDistill>(a, stream);
  return gradient_rows<float, kDistill>(a, stream);
}
hipError_t launch_distill_fwd_bwd(int dtype, const VocabArgs& a, const VocabPlan& p, void* ws,
                                  hipStream_t stream) {
  bool held;
  hipError_t e = dtype == 0   ? distill_rows<bf16>(a, stream, held)
                 : dtype == 1 ? distill_rows<fp16>(a, stream, held)
                              : distill_rows<float>(a, stream, held);
  if (held || e != hipSuccess) return e;
  e = launch_distill_fwd(dtype, a, p, ws, stream);
  if (e != hipSuccess) return e;
  VocabArgs b = a;
  b.lse_in = a.lse;
  return launch_distill_bwd(dtype, b, stream);
}

}  // namespace swg
