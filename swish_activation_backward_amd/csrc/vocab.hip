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
  __device__ inline int64_t single(int t, int64_t V, bool first, bool last) const {
    if (t < head) return first ? t : -1;
    if (t >= 8 && t < 8 + tail) return last ? V - tail + (t - 8) : -1;
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

// A running softmax over values z: m the largest (at least the lowest finite number, so that
// differences stay defined over masked entries), s = sum 2^d, t = sum d 2^d for d = (z - m) c,
// c = log2(e) / T.  A masked entry has 2^d = 0; its d is bounded where it is multiplied.  A
// NaN or +inf makes s and t NaN.
struct Soft {
  float m, s, t;
};
__device__ inline float bound_d(float d) { return __builtin_fmaxf(d, -1000.0f); }

// the same sums relative to a maximum m >= a.m
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

template <int NT> __device__ inline void soft_block(Soft& a, float c, float* red) {
  const float m = block_max<NT>(a.m, red);
  soft_move(a, m, c);
  a.s = block_sum<NT>(a.s, red);
  a.t = block_sum<NT>(a.t, red);
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
// value of every group of chunks is kept (`gkeys`).  A value that at least k group maxima
// reach bounds the k-th largest entry from below, and only the groups that reach it, about k
// of them, are read again: their entries from the bound on are the candidates, ordered at the
// end by counting.  Where equal values leave no bound with few groups, the entries above it
// are candidates and, of those equal to it, the first ones by index, found by a scan.
constexpr int kSlack = 64;          // keys a selection may leave beyond k before the ordering
__host__ __device__ inline int top_groups(int k) { return k + k / 4 + 8; }
__host__ __device__ inline int top_candidates(int k, int group) {
  return top_groups(k) * group + 2 * k + 16;
}

template <int NT> struct TopState {
  uint32_t* gkeys;   // one per group of the tile
  uint32_t* glist;   // chosen groups
  u64* cand;         // candidates
  u64* sel;          // k + kSlack
  u64* best;         // k, in order
  int* count;        // [0] candidates, [1] groups, [2..] counts of the waves, twice
  int k;
};

// the number of threads' flags over the workgroup; successive calls alternate `half`
template <int NT> __device__ inline int block_count(int wave_count, int* count, int& half) {
  if constexpr (NT == 64) return wave_count;
  int* c = count + 2 + half * (NT / 64);
  half ^= 1;
  if ((threadIdx.x & 63) == 0) c[threadIdx.x >> 6] = wave_count;
  __syncthreads();
  int n = c[0];
#pragma unroll
  for (int i = 1; i < NT / 64; ++i) n += c[i];
  return n;
}

// Bisects for a bound: `lo` such that at least k of the n keys are >= lo and either no more
// than `most`, or lo + 1 is reached by fewer than k.  Returns the count at lo.  The same in
// every thread; n >= k.
template <int NT, typename K>
__device__ inline int bisect(const K* keys, int n, int k, int most, K hi, int* count, K& lo) {
  int half = 0, at_lo = n;
  lo = 0;
  while (at_lo > most && hi - lo > 1) {
    const K mid = lo + (hi - lo) / 2;
    int c = 0;
    for (int i = threadIdx.x & ~63; i < n; i += NT) {
      const int j = i + (threadIdx.x & 63);
      c += __popcll(__ballot(j < n && keys[j] >= mid));
    }
    c = block_count<NT>(c, count, half);
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

// the k largest of the n candidates to `best`, in falling order; the rest of best becomes 0
template <int NT> __device__ inline void order_top(const TopState<NT>& w, int n) {
  const u64* from = w.cand;
  if (n > w.k + kSlack) {
    u64 lo;
    n = bisect<NT, u64>(w.cand, n, w.k, w.k + kSlack, ~0ull, w.count, lo);
    const int all = w.count[0];
    if (threadIdx.x == 0) w.count[1] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < all; i += NT) {
      const u64 key = w.cand[i];
      if (key >= lo) w.sel[atomicAdd(&w.count[1], 1)] = key;
    }
    __syncthreads();
    from = w.sel;
  }
  for (int i = threadIdx.x; i < w.k; i += NT)
    if (i >= n) w.best[i] = 0;
  for (int i = threadIdx.x; i < n; i += NT) {
    const u64 key = from[i];
    int rank = 0;
    for (int j = 0; j < n; ++j) rank += from[j] > key;
    if (rank < w.k) w.best[rank] = key;
  }
  __syncthreads();
}

// the candidates of one tile: chunks [t0, t1) of `body`, whose first element is entry `first`
// of the row; groups of GU chunks, NT apart
template <typename T, int NT, int U, int GU>
__device__ inline void collect_tile(const TopState<NT>& w, const T* body, int64_t first,
                                    int64_t t0, int64_t t1, int slots) {
  const int k = w.k, most = top_groups(k);
  __syncthreads();   // the group keys are written
  uint32_t top = 0;
  int groups = 0;
  for (int i = threadIdx.x; i < slots; i += NT) {
    const uint32_t g = w.gkeys[i];
    top = g > top ? g : top;
    groups += g != 0;
  }
  // bounds of the bisection: all groups, and the largest key
  float* red = reinterpret_cast<float*>(w.sel);
  groups = (int)block_sum<NT>((float)groups, red);
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) {
    const uint32_t o = __shfl_xor(top, d);
    top = o > top ? o : top;
  }
  if constexpr (NT > 64) {
    uint32_t* r = reinterpret_cast<uint32_t*>(w.sel) + 64;
    if ((threadIdx.x & 63) == 0) r[threadIdx.x >> 6] = top;
    __syncthreads();
    for (int i = 0; i < NT / 64; ++i) top = r[i] > top ? r[i] : top;
  }
  uint32_t bound = 0;
  int reach = groups;
  if (groups > most)
    reach = bisect<NT, uint32_t>(w.gkeys, slots, k, most, top + 1, w.count, bound);
  const bool ties = reach > most;             // too many groups at the bound itself
  const uint32_t from = ties ? bound + 1 : (bound ? bound : 1);
  if (threadIdx.x == 0) w.count[1] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < slots; i += NT)
    if (w.gkeys[i] >= from) w.glist[atomicAdd(&w.count[1], 1)] = (uint32_t)i;
  __syncthreads();
  const int chosen = w.count[1], before = w.count[0];
  for (int i = threadIdx.x; i < chosen * GU; i += NT) {
    const int g = (int)w.glist[i / GU], u = i % GU;
    const int64_t q = GU == 1 ? t0 + g : t0 + (int64_t)(g / NT) * (NT * U) + u * NT + g % NT;
    if (q >= t1) continue;
    Chunk<T> c;
    c.load(body + q * 8);
    float f[8];
    c.widen(f);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (value_key(f[e]) >= from)
        w.cand[atomicAdd(&w.count[0], 1)] = entry_key(f[e], (uint32_t)(first + q * 8 + e));
    }
  }
  __syncthreads();
  if (!ties) return;
  // the first k - (those above) entries equal to the bound, chunk by chunk in the row's order
  int need = k - (w.count[0] - before), half = 0;
  for (int64_t base = t0; base < t1 && need > 0; base += NT) {
    const int64_t q = base + threadIdx.x;
    float f[8];
    int mine = 0;
    if (q < t1) {
      Chunk<T> c;
      c.load(body + q * 8);
      c.widen(f);
#pragma unroll
      for (int e = 0; e < 8; ++e) mine += value_key(f[e]) == bound;
    }
    // the number before this thread's, in the wave and then over the waves
    int incl = mine;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_up(incl, d);
      if ((int)(threadIdx.x & 63) >= d) incl += o;
    }
    const int wave_total = __shfl(incl, 63);
    const int total = block_count<NT>(wave_total, w.count, half);
    int rank = incl - mine;
    if constexpr (NT > 64) {
      const int* c = w.count + 2 + (half ^ 1) * (NT / 64);
      for (int i = 0; i < (int)(threadIdx.x >> 6); ++i) rank += c[i];
    }
    if (q < t1 && mine) {
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

// ------------------------------------------------------------------ the teacher's entries
__device__ inline float teacher_value(const VocabArgs& a, int64_t r, int64_t j, int64_t id) {
  if (id < 0 || id >= a.V) return neg_inf();
  const int64_t i = r * a.k + j;
  float u;
  if (a.teacher_dtype == 0) u = to_f32(static_cast<const bf16*>(a.teacher)[i]);
  else if (a.teacher_dtype == 1) u = to_f32(static_cast<const fp16*>(a.teacher)[i]);
  else u = static_cast<const float*>(a.teacher)[i];
  return u * a.inv_t;
}

// An entry as the thread that reads it keeps it: id (-1: does not count) and u / T.
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

// softmax over the entries: log q = u - um - lus.  `mine` is the thread's first entry, entry
// threadIdx.x; those from NT on are read again.
struct Teacher {
  float um, us, lus;
};
template <int NT>
__device__ inline Teacher teacher_softmax(const VocabArgs& a, int64_t r, const Entry& mine,
                                          float* red) {
  Teacher t;
  float m = mine.u;
  for (int64_t j = threadIdx.x + NT; j < a.k; j += NT)
    m = __builtin_fmaxf(m, load_entry(a, r, j).u);
  m = block_max<NT>(m, red);
  t.um = m == neg_inf() ? 0.0f : m;
  float s = expf(mine.u - t.um);
  for (int64_t j = threadIdx.x + NT; j < a.k; j += NT) s += expf(load_entry(a, r, j).u - t.um);
  t.us = block_sum<NT>(s, red);
  t.lus = logf(t.us);
  return t;
}

// q (log q - log p) of one entry
__device__ inline float kl_term(const Teacher& t, const RowStat& st, float u, float z,
                                float inv_t) {
  const float lq = u - t.um, q = expf(lq) / t.us;
  if (t.us == 0.0f || q == 0.0f) return 0.0f;
  return q * (lq - t.lus - log_prob(st, z, inv_t));
}

// ------------------------------------------------------------------ forward
enum { kLogprobs = 0, kDistill = 1 };

// The results of one row from its sums and, in falling order, its k best keys (null for none).
template <typename T, int NT, int MODE>
__device__ inline void finish_row(const VocabArgs& a, int64_t r, const Soft& sum,
                                  const u64* best, const Entry& mine, float z_mine, float* red) {
  const T* z = static_cast<const T*>(a.z) + r * a.ld;
  const RowStat st = row_stat(sum, a.inv_t);
  if constexpr (MODE == kLogprobs) {
    if (threadIdx.x == 0) {
      if (a.lse) a.lse[r] = st.lse;
      if (a.entropy) a.entropy[r] = st.entropy;
      if (a.target) {
        // mine.id: the target, -1 where it lies outside the vocabulary
        float lp = __builtin_nanf("");
        if (a.target[r] == a.ignore) lp = 0.0f;
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
      if (e.id >= 0) kl += kl_term(t, st, e.u, to_f32(z[e.id]), a.inv_t);
    }
    kl = block_sum<NT>(kl, red);
    if (threadIdx.x == 0) {
      a.loss[r] = a.t * a.t * kl;
      if (a.lse) a.lse[r] = st.lse;
    }
  }
}

// what a thread reads of a row ahead of the stream: the target, or its first teacher entry
template <typename T, int MODE>
__device__ inline Entry row_entry(const VocabArgs& a, int64_t r, float& z_mine) {
  Entry e{-1, neg_inf()};
  z_mine = 0.0f;
  if constexpr (MODE == kLogprobs) {
    if (a.target && threadIdx.x == 0) {
      const int64_t id = a.target[r];
      if (id >= 0 && id < a.V) e.id = id;
    }
  } else {
    e = load_entry(a, r, threadIdx.x);
  }
  if (e.id >= 0) z_mine = to_f32(static_cast<const T*>(a.z)[r * a.ld + e.id]);
  return e;
}

extern __shared__ __attribute__((aligned(16))) char swg_vocab_lds[];

// U chunks a thread and pass (64 bytes in flight), the next pass loaded before the present one
// is worked on.
template <typename T> struct Pass { static constexpr int U = sizeof(T) == 2 ? 4 : 2; };

// One row, or one of `split` segments of it, by a workgroup of NT threads.  A segment leaves
// its sums and its k best keys in the workspace; join_kernel finishes the row.
template <typename T, int NT, int GU, int SLOTS, int MODE, bool TOP, bool ENT>
__global__ __launch_bounds__(NT) void rows_kernel(VocabArgs a, int split, int64_t seg,
                                                  Soft* part, u64* part_keys) {
  constexpr int U = Pass<T>::U;
  constexpr int ITERS = SLOTS * GU / (NT * U);   // passes of a tile
  __shared__ float red[NT / 64];
  __shared__ int count[2 + 2 * (NT / 64)];
  TopState<NT> w;
  const int k = (int)a.top;
  if constexpr (TOP) {
    w.k = k;
    w.cand = reinterpret_cast<u64*>(swg_vocab_lds);
    w.sel = w.cand + top_candidates(k, GU * 8);
    w.best = w.sel + k + kSlack;
    w.gkeys = reinterpret_cast<uint32_t*>(w.best + k);
    w.glist = w.gkeys + SLOTS;
    w.count = count;
  }
  const float c = a.inv_t * kLog2e;
  for (int64_t item = blockIdx.x; item < a.R * split; item += gridDim.x) {
    const int64_t r = item / split, part_i = item % split;
    const T* z = static_cast<const T*>(a.z) + r * a.ld;
    const RowCut cut(z, a.V);
    const T* body = z + cut.head;
    const int64_t c0 = part_i * seg, c1 = c0 + seg < cut.chunks ? c0 + seg : cut.chunks;
    float z_mine = 0.0f;
    Entry mine{-1, neg_inf()};
    if (split == 1) mine = row_entry<T, MODE>(a, r, z_mine);
    if constexpr (TOP) {
      __syncthreads();
      if (threadIdx.x == 0) count[0] = 0;
      __syncthreads();
    }
    Soft sum{kLowest, 0.0f, 0.0f};
    {
      const int64_t i = cut.single(threadIdx.x, a.V, part_i == 0, part_i == split - 1);
      if (i >= 0) {
        const float x = to_f32(z[i]);
        sum.m = __builtin_fmaxf(sum.m, x);
        soft_add<ENT>(sum, x, c);
        if constexpr (TOP) w.cand[atomicAdd(&count[0], 1)] = entry_key(x, (uint32_t)i);
      }
    }
    // one pass: U chunks of the thread, from `base` on
    auto load = [&](Chunk<T>* ch, int64_t base) {
      if (base + NT * U <= c1) {
#pragma unroll
        for (int u = 0; u < U; ++u)
          ch[u].load_stream(body + (base + u * NT + threadIdx.x) * 8);
      } else {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int64_t q = base + u * NT + threadIdx.x;
          fill_masked(ch[u]);
          if (q < c1) ch[u].load_stream(body + q * 8);
        }
      }
    };
    Chunk<T> cur[U], next[U];
    load(cur, c0);
    for (int64_t t0 = c0; t0 < c1; t0 += (int64_t)ITERS * NT * U) {
      const int64_t t1 = TOP && t0 + ITERS * NT * U < c1 ? t0 + ITERS * NT * U : c1;
      int it = 0;
      for (int64_t base = t0; base < t1; base += NT * U, ++it) {
        load(next, base + NT * U);
        float f[U][8], gm[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          cur[u].widen(f[u]);
          gm[u] = __builtin_fmaxf(
              __builtin_fmaxf(__builtin_fmaxf(f[u][0], f[u][1]),
                              __builtin_fmaxf(f[u][2], f[u][3])),
              __builtin_fmaxf(__builtin_fmaxf(f[u][4], f[u][5]),
                              __builtin_fmaxf(f[u][6], f[u][7])));
        }
        float m = gm[0];
#pragma unroll
        for (int u = 1; u < U; ++u) m = __builtin_fmaxf(m, gm[u]);
        if constexpr (TOP) {
          if constexpr (GU == 1) {
#pragma unroll
            for (int u = 0; u < U; ++u)
              w.gkeys[(it * U + u) * NT + threadIdx.x] =
                  base + u * NT + threadIdx.x < t1 ? value_key(gm[u]) : 0;
          } else {
            w.gkeys[it * NT + threadIdx.x] = base + threadIdx.x < t1 ? value_key(m) : 0;
          }
        }
        soft_move(sum, __builtin_fmaxf(sum.m, m), c);
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int i = 0; i < 8; ++i) soft_add<ENT>(sum, f[u][i], c);
#pragma unroll
        for (int u = 0; u < U; ++u) cur[u] = next[u];
      }
      if constexpr (TOP) {
        collect_tile<T, NT, U, GU>(w, body, cut.head, t0, t1, it * (GU == 1 ? U : 1) * NT);
        if (t1 < c1) {   // the best so far are the next tile's first candidates
          order_top<NT>(w, count[0]);
          const int n = count[0] < k ? count[0] : k;
          for (int i = threadIdx.x; i < n; i += NT) w.cand[i] = w.best[i];
          __syncthreads();
          if (threadIdx.x == 0) count[0] = n;
        }
      }
      if constexpr (!TOP) break;
    }
    soft_block<NT>(sum, c, red);
    if constexpr (TOP) {
      __syncthreads();
      order_top<NT>(w, count[0]);
    }
    if (split == 1) {
      finish_row<T, NT, MODE>(a, r, sum, TOP ? w.best : nullptr, mine, z_mine, red);
    } else {
      if (threadIdx.x == 0) part[item] = sum;
      if constexpr (TOP) {
        for (int i = threadIdx.x; i < k; i += NT) part_keys[item * k + i] = w.best[i];
      }
    }
  }
}

// Joins a row's segments (at most 64).
template <typename T, int MODE>
__global__ __launch_bounds__(256) void join_kernel(VocabArgs a, int split, const Soft* part,
                                                   const u64* part_keys) {
  constexpr int NT = 256;
  __shared__ float red[NT / 64];
  __shared__ int count[2 + 2 * (NT / 64)];
  const float c = a.inv_t * kLog2e;
  const int k = (int)a.top, n = k * split;
  TopState<NT> w;
  w.k = k;
  w.cand = reinterpret_cast<u64*>(swg_vocab_lds);
  w.sel = w.cand + n;
  w.best = w.sel + k + kSlack;
  w.gkeys = w.glist = nullptr;
  w.count = count;
  for (int64_t r = blockIdx.x; r < a.R; r += gridDim.x) {
    float z_mine;
    const Entry mine = row_entry<T, MODE>(a, r, z_mine);
    Soft sum{kLowest, 0.0f, 0.0f};
    if ((int)threadIdx.x < split) sum = part[r * split + threadIdx.x];
    if (k > 0) {
      for (int i = threadIdx.x; i < n; i += NT) w.cand[i] = part_keys[r * n + i];
      if (threadIdx.x == 0) count[0] = n;
    }
    soft_block<NT>(sum, c, red);
    if (k > 0) {
      __syncthreads();
      order_top<NT>(w, n);
    }
    finish_row<T, NT, MODE>(a, r, sum, k > 0 ? w.best : nullptr, mine, z_mine, red);
    __syncthreads();
  }
}

// ------------------------------------------------------------------ gradients
// A workgroup forms up to kGradChunks chunks of a row.  The columns that hold more than their
// probability (the target, the teacher's entries) are formed with it in the thread that owns
// them, so the call may overwrite the logits.  The teacher's entries hang in lists by chunk
// (`first`, `next`); a thread goes through its chunk's list in the order of the entries, so
// repeated ids add up in a fixed order.
constexpr int kGradChunks = 2048;

template <typename T, int NT, int MODE>
__global__ __launch_bounds__(NT) void grad_kernel(VocabArgs a, int split) {
  constexpr int U = Pass<T>::U;
  __shared__ float red[NT / 64];
  // lists, one per chunk and one for the single elements
  int* first = reinterpret_cast<int*>(swg_vocab_lds);
  int* next = first + kGradChunks + 8;
  int* column = next + a.k;
  float* share = reinterpret_cast<float*>(column + a.k);
  for (int64_t item = blockIdx.x; item < a.R * split; item += gridDim.x) {
    const int64_t r = item / split, part_i = item % split;
    const T* z = static_cast<const T*>(a.z) + r * a.ld;
    T* dz = static_cast<T*>(a.dz) + r * a.lddz;
    const RowCut cut(z, a.V);
    const T* body = z + cut.head;
    T* out = dz + cut.head;
    const int64_t c0 = part_i * kGradChunks;
    const int64_t c1 = c0 + kGradChunks < cut.chunks ? c0 + kGradChunks : cut.chunks;
    const int64_t lone = cut.single(threadIdx.x, a.V, part_i == 0, part_i == split - 1);
    const float lse_in = a.lse_in[r];
    const float lse = lse_in == neg_inf() ? 0.0f : lse_in;   // a row of masked entries: p = 0

    float scale = 0.0f, A = 0.0f, g = 0.0f, h = 0.0f, H = 0.0f, Q = 0.0f;
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
      scale = -a.inv_t;
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
      __syncthreads();   // the lists' readers of the last item are done
      for (int i = threadIdx.x; i < kGradChunks + 8; i += NT) first[i] = -1;
      const Entry mine = load_entry(a, r, threadIdx.x);
      const Teacher t = teacher_softmax<NT>(a, r, mine, red);
      Q = t.us == 0.0f ? 0.0f : 1.0f;
      __syncthreads();
      Entry e = mine;
      for (int64_t j = threadIdx.x; j < a.k; j += NT) {
        if (j >= NT) e = load_entry(a, r, j);
        if (e.id < 0 || t.us == 0.0f) continue;
        const int64_t col = e.id - cut.head, ch = col >> 3;
        int list;
        if (col < 0 || ch >= cut.chunks) list = kGradChunks;   // single elements
        else if (ch >= c0 && ch < c1) list = (int)(ch - c0);
        else continue;
        column[j] = (int)e.id;
        share[j] = expf(e.u - t.um) / t.us;
        next[j] = atomicExch(&first[list], (int)j);
      }
      __syncthreads();
    }
    // the teacher's share of column `col` of a list
    auto teacher_share = [&](int list_first, int col) {
      float q = 0.0f;
      for (int last = -1;;) {
        int best = 0x7fffffff;
        for (int j = list_first; j >= 0; j = next[j])
          if (column[j] == col && j > last && j < best) best = j;
        if (best == 0x7fffffff) return q;
        q += share[best];
        last = best;
      }
    };
    auto value = [&](float x) {   // log p
      return __builtin_fmaf(x, a.inv_t, -lse);
    };
    auto at_target = [&](float x) {
      // g (1 - p) is of the size of g: the division by T in fp64 leaves one rounding to fp32
      // where the product with 1/T would leave three
      const float lp = value(x), p = __builtin_amdgcn_exp2f(lp * kLog2e);
      const double ent = p != 0.0f ? (double)(h * p * (lp + H)) : 0.0;
      return (float)(((double)g * (1.0 - (double)p) - ent) / (double)a.t);
    };
    auto plain = [&](float x) {
      const float lp = value(x), p = __builtin_amdgcn_exp2f(lp * kLog2e);
      if constexpr (MODE == kLogprobs)
        return p * __builtin_fmaf(h, __builtin_fmaxf(lp, -200.0f), A) * scale;
      else
        return scale * (Q * p);
    };
    if (lone >= 0) {
      const float x = to_f32(z[lone]);
      float d;
      if constexpr (MODE == kLogprobs) {
        d = lone == id && g != 0.0f ? at_target(x) : plain(x);
      } else {
        const float p = __builtin_amdgcn_exp2f(value(x) * kLog2e);
        d = scale * (Q * p - teacher_share(first[kGradChunks], (int)lone));
      }
      dz[lone] = from_f32<T>(d);
    }
    for (int64_t base = c0; base < c1; base += NT * U) {
      Chunk<T> ch[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t q = base + u * NT + threadIdx.x;
        if (q < c1) ch[u].load_stream(body + q * 8);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t q = base + u * NT + threadIdx.x;
        if (q >= c1) continue;
        float f[8], d[8];
        ch[u].widen(f);
#pragma unroll
        for (int i = 0; i < 8; ++i) d[i] = plain(f[i]);
        const int64_t col = cut.head + q * 8;
        if constexpr (MODE == kLogprobs) {
          if (id >= col && id < col + 8 && g != 0.0f) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (id == col + i) d[i] = at_target(f[i]);
          }
        } else {
          const int list = first[q - c0];
          if (list >= 0) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float p = __builtin_amdgcn_exp2f(value(f[i]) * kLog2e);
              d[i] = scale * (Q * p - teacher_share(list, (int)(col + i)));
            }
          }
        }
        ch[u].narrow(d);
        ch[u].store_stream(out + q * 8);
      }
    }
  }
}

// ------------------------------------------------------------------ launches
static size_t top_lds(int k, int group, int slots) {
  return sizeof(u64) * (size_t)(top_candidates(k, group) + 2 * k + kSlack) +
         sizeof(uint32_t) * (size_t)(slots + top_groups(k));
}

template <typename T, int MODE, bool ENT>
static hipError_t forward_rows(const VocabArgs& a, const VocabPlan& p, void* ws,
                               hipStream_t stream) {
  Soft* part = static_cast<Soft*>(ws);
  u64* keys = reinterpret_cast<u64*>(static_cast<char*>(ws) + p.keys_at);
  const int k = (int)a.top;
#define SWG_ROWS(NT, GU, SLOTS)                                                              \
  do {                                                                                       \
    if (k > 0) {                                                                             \
      if constexpr (MODE == kLogprobs)                                                       \
        SWG_LAUNCH((rows_kernel<T, NT, GU, SLOTS, MODE, true, ENT>),                         \
                   dim3(row_grid(a.R * p.split)), dim3(NT), top_lds(k, GU * 8, SLOTS),       \
                   stream, a, p.split, p.seg, part, keys);                                   \
    } else {                                                                                 \
      SWG_LAUNCH((rows_kernel<T, NT, GU, SLOTS, MODE, false, ENT>),                          \
                 dim3(row_grid(a.R * p.split)), dim3(NT), 0, stream, a, p.split, p.seg, part, \
                 keys);                                                                      \
    }                                                                                        \
  } while (0)
  constexpr int U = Pass<T>::U;
  if (p.threads == 64) SWG_ROWS(64, 1, 512);
  else if (p.threads == 256) SWG_ROWS(256, 1, 4096);
  else SWG_ROWS(512, U, (16384 / U));
#undef SWG_ROWS
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.split == 1) return e;
  const size_t lds = k > 0 ? sizeof(u64) * (size_t)(k * p.split + 2 * k + kSlack) : 0;
  SWG_LAUNCH((join_kernel<T, MODE>), dim3(row_grid(a.R)), dim3(256), lds, stream, a, p.split,
             part, keys);
  return hipGetLastError();
}

template <typename T, int MODE>
static hipError_t gradient_rows(const VocabArgs& a, hipStream_t stream) {
  const size_t lds =
      MODE == kDistill ? sizeof(int) * (size_t)(kGradChunks + 8 + 3 * a.k) : sizeof(int);
  const int split = (int)ceil_div(a.V, (int64_t)kGradChunks * 8);
  if (a.V <= 2048)
    SWG_LAUNCH((grad_kernel<T, 64, MODE>), dim3(row_grid(a.R * split)), dim3(64), lds, stream, a,
               split);
  else
    SWG_LAUNCH((grad_kernel<T, 256, MODE>), dim3(row_grid(a.R * split)), dim3(256), lds, stream,
               a, split);
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
  const hipError_t e = launch_distill_fwd(dtype, a, p, ws, stream);
  if (e != hipSuccess) return e;
  VocabArgs b = a;
  b.lse_in = a.lse;
  return launch_distill_bwd(dtype, b, stream);
}

}  // namespace swg
