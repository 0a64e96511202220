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

// m = max a, s = sum exp(a - m), both in every thread; m = 0 for a row of only -inf (s = 0)
template <typename T>
__device__ inline void row_softmax(const T* z, int64_t V, float inv_t, float* red, float& m,
                                   float& s) {
  float v = neg_inf();
  for (int64_t c = threadIdx.x; c < V; c += 256) v = __builtin_fmaxf(v, to_f32(z[c]) * inv_t);
  m = block_max<256>(v, red);
  if (m == neg_inf()) m = 0.0f;
  v = 0.0f;
  for (int64_t c = threadIdx.x; c < V; c += 256) v += expf(to_f32(z[c]) * inv_t - m);
  s = block_sum<256>(v, red);
}

__device__ inline u64 block_max_key(u64 k, u64* red) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) {
    const u64 o = __shfl_xor(k, d);
    k = o > k ? o : k;
  }
  __syncthreads();
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = k;
  __syncthreads();
  k = red[0];
  for (int i = 1; i < 4; ++i) k = red[i] > k ? red[i] : k;
  return k;
}

template <typename T>
__global__ __launch_bounds__(256) void logprobs_kernel(VocabArgs a) {
  __shared__ float red[4];
  __shared__ u64 kred[4];
  for (int64_t r = blockIdx.x; r < a.R; r += gridDim.x) {
    const T* z = static_cast<const T*>(a.z) + r * a.ld;
    float m, s;
    row_softmax(z, a.V, a.inv_t, red, m, s);
    float t = 0.0f;
    for (int64_t c = threadIdx.x; c < a.V; c += 256) {
      const float d = to_f32(z[c]) * a.inv_t - m;
      if (d != neg_inf()) t = __builtin_fmaf(d, expf(d), t);
    }
    t = block_sum<256>(t, red);
    const float ls = logf(s);
    if (threadIdx.x == 0) {
      if (a.lse) a.lse[r] = s == 0.0f ? neg_inf() : m + ls;
      if (a.entropy) a.entropy[r] = s == 0.0f ? 0.0f : ls - t / s;
      if (a.target) {
        const int64_t id = a.target[r];
        float lp = __builtin_nanf("");
        if (id == a.ignore) lp = 0.0f;
        else if (id >= 0 && id < a.V)
          lp = s == 0.0f ? neg_inf() : to_f32(z[id]) * a.inv_t - m - ls;
        a.logprob[r] = lp;
      }
    }
    u64 below = ~0ull;
    for (int64_t j = 0; j < a.top; ++j) {
      u64 best = 0;
      for (int64_t c = threadIdx.x; c < a.V; c += 256) {
        const u64 k = entry_key(to_f32(z[c]), (uint32_t)c);
        if (k < below && k > best) best = k;
      }
      below = block_max_key(best, kred);
      if (threadIdx.x == 0) {
        const uint32_t id = key_index(below);
        a.top_id[r * a.top + j] = id;
        a.top_logprob[r * a.top + j] =
            s == 0.0f ? neg_inf() : to_f32(z[id]) * a.inv_t - m - ls;
      }
    }
  }
}

template <typename T>
__global__ __launch_bounds__(256) void logprobs_bwd_kernel(VocabArgs a) {
  for (int64_t r = blockIdx.x; r < a.R; r += gridDim.x) {
    const T* z = static_cast<const T*>(a.z) + r * a.ld;
    T* dz = static_cast<T*>(a.dz) + r * a.lddz;
    const float lse = a.lse_in[r];
    const int64_t id = a.target ? a.target[r] : a.ignore;
    float g = a.dlogprob && (!a.target || id != a.ignore) ? a.dlogprob[r] : 0.0f;
    if (a.target && id != a.ignore && (id < 0 || id >= a.V)) g = __builtin_nanf("");
    const float h = a.dentropy ? a.dentropy[r] : 0.0f;
    const float H = a.dentropy ? a.entropy_in[r] : 0.0f;
    for (int64_t c = threadIdx.x; c < a.V; c += 256) {
      const float x = to_f32(z[c]);
      float d = 0.0f;
      const float lp = x * a.inv_t - lse;
      const float p = x == neg_inf() ? 0.0f : expf(lp);
      d = -g * p;
      if (p != 0.0f) d -= h * p * (lp + H);
      d *= a.inv_t;
      // the target's g (1 - p) is of the size of g: the division by T in fp64 leaves one
      // rounding to fp32 where the product with 1/T would leave three
      if (c == id && g != 0.0f) {
        const double ent = p != 0.0f ? (double)(h * p * (lp + H)) : 0.0;
        d = (float)(((double)g * (1.0 - (double)p) - ent) / (double)a.t);
      }
      dz[c] = from_f32<T>(d);
    }
  }
}

__device__ inline float teacher_value(const VocabArgs& a, int64_t r, int64_t j) {
  const int64_t i = r * a.k + j;
  const int64_t id = a.ids[i];
  if (id < 0 || id >= a.V) return neg_inf();
  float u;
  if (a.teacher_dtype == 0) u = to_f32(static_cast<const bf16*>(a.teacher)[i]);
  else if (a.teacher_dtype == 1) u = to_f32(static_cast<const fp16*>(a.teacher)[i]);
  else u = static_cast<const float*>(a.teacher)[i];
  return u * a.inv_t;
}

template <typename T>
__global__ __launch_bounds__(256) void distill_fwd_kernel(VocabArgs a) {
  __shared__ float red[4];
  for (int64_t r = blockIdx.x; r < a.R; r += gridDim.x) {
    const T* z = static_cast<const T*>(a.z) + r * a.ld;
    float m, s;
    row_softmax(z, a.V, a.inv_t, red, m, s);
    const float ls = logf(s);
    float um = neg_inf();
    for (int64_t j = threadIdx.x; j < a.k; j += 256)
      um = __builtin_fmaxf(um, teacher_value(a, r, j));
    um = block_max<256>(um, red);
    if (um == neg_inf()) um = 0.0f;
    float us = 0.0f;
    for (int64_t j = threadIdx.x; j < a.k; j += 256) us += expf(teacher_value(a, r, j) - um);
    us = block_sum<256>(us, red);
    const float lus = logf(us);
    float kl = 0.0f;
    for (int64_t j = threadIdx.x; j < a.k; j += 256) {
      const float lq = teacher_value(a, r, j) - um;
      const float q = expf(lq) / us;
      if (us != 0.0f && q != 0.0f) {
        const float lp =
            s == 0.0f ? neg_inf() : to_f32(z[a.ids[r * a.k + j]]) * a.inv_t - m - ls;
        kl += q * (lq - lus - lp);
      }
    }
    kl = block_sum<256>(kl, red);
    if (threadIdx.x == 0) {
      a.loss[r] = a.t * a.t * kl;
      if (a.lse) a.lse[r] = s == 0.0f ? neg_inf() : m + ls;
    }
  }
}

template <typename T>
__global__ __launch_bounds__(256) void distill_bwd_kernel(VocabArgs a) {
  __shared__ float red[4];
  for (int64_t r = blockIdx.x; r < a.R; r += gridDim.x) {
    const T* z = static_cast<const T*>(a.z) + r * a.ld;
    T* dz = static_cast<T*>(a.dz) + r * a.lddz;
    const float w = a.dloss[r];
    if (w == 0.0f) {
      for (int64_t c = threadIdx.x; c < a.V; c += 256) dz[c] = from_f32<T>(0.0f);
      continue;
    }
    const float lse = a.lse_in[r];
    float um = neg_inf();
    for (int64_t j = threadIdx.x; j < a.k; j += 256)
      um = __builtin_fmaxf(um, teacher_value(a, r, j));
    um = block_max<256>(um, red);
    if (um == neg_inf()) um = 0.0f;
    float us = 0.0f;
    for (int64_t j = threadIdx.x; j < a.k; j += 256) us += expf(teacher_value(a, r, j) - um);
    us = block_sum<256>(us, red);
    const float Q = us == 0.0f ? 0.0f : 1.0f;
    // each thread forms its own columns: the teacher's share of a column is summed in entry
    // order, so repeated ids add up in a fixed order
    for (int64_t c = threadIdx.x; c < a.V; c += 256) {
      const float x = to_f32(z[c]);
      const float p = x == neg_inf() ? 0.0f : expf(x * a.inv_t - lse);
      float q = 0.0f;
      for (int64_t j = 0; j < a.k; ++j)
        if (a.ids[r * a.k + j] == c && us != 0.0f) q += expf(teacher_value(a, r, j) - um) / us;
      dz[c] = from_f32<T>(w * a.t * (Q * p - q));
    }
  }
}

#define SWG_VOCAB_DISPATCH(KERNEL)                                                          \
  switch (dtype) {                                                                          \
    case 0: SWG_LAUNCH((KERNEL<bf16>), dim3(row_grid(a.R)), dim3(256), 0, stream, a); break; \
    case 1: SWG_LAUNCH((KERNEL<fp16>), dim3(row_grid(a.R)), dim3(256), 0, stream, a); break; \
    default: SWG_LAUNCH((KERNEL<float>), dim3(row_grid(a.R)), dim3(256), 0, stream, a);      \
  }                                                                                         \
  return hipGetLastError();

hipError_t launch_logprobs(int dtype, const VocabArgs& a, void* ws, hipStream_t stream) {
  SWG_VOCAB_DISPATCH(logprobs_kernel)
}
hipError_t launch_logprobs_bwd(int dtype, const VocabArgs& a, hipStream_t stream) {
  SWG_VOCAB_DISPATCH(logprobs_bwd_kernel)
}
hipError_t launch_distill_fwd(int dtype, const VocabArgs& a, void* ws, hipStream_t stream) {
  SWG_VOCAB_DISPATCH(distill_fwd_kernel)
}
hipError_t launch_distill_bwd(int dtype, const VocabArgs& a, hipStream_t stream) {
  SWG_VOCAB_DISPATCH(distill_bwd_kernel)
}
hipError_t launch_distill_fwd_bwd(int dtype, const VocabArgs& a, void* ws, hipStream_t stream) {
  const hipError_t e = launch_distill_fwd(dtype, a, ws, stream);
  if (e != hipSuccess) return e;
  VocabArgs b = a;
  b.lse_in = a.lse;
  return launch_distill_bwd(dtype, b, stream);
}

}  // namespace swg
