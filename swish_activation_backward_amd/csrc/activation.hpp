// Activations of the linear layer's epilogue and their slopes, in fp32.
#pragma once

#include "common.hpp"
#include "launch.hpp"

namespace swg {

constexpr float kInvSqrt2Pi = 0.3989422804014327f;
// the tanh form of gelu is z sigma(2 a), 2 a = kTanh1 z + kTanh3 z^3
constexpr float kTanh1 = 1.5957691216057308f;
constexpr float kTanh3 = 0.07135481627159929f;

// Phi(z), the normal distribution function, and e = exp(-z^2 / 2).  The tail beyond |z| is
// e t p(t) for t = 1 / (1 + 0.3 x), x = |z| / sqrt(2), where t p(t) is half the scaled complementary
// error function exp(x^2) erfc(x): p of degree 8 by weighted least squares on 0 <= x <= 14, 4e-8
// off relatively.  With the roundings of its evaluation Phi is within 3e-7 (measured 2.7e-7, next to
// 0).  Relative to itself the tail loses with z^2, as the exponent is rounded twice: within
// (32 + 1.25 z^2) 2^-24 (measured 5.6e-7 from -2 to 0, 9.4e-7 to -4, 3.2e-6 to -8, 7.7e-6 to -12.5).
__device__ inline float normal_cdf(float z, float* e) {
  const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.21213204f, __builtin_fabsf(z), 1.0f));
  float p = -0.06330819f;
  p = __builtin_fmaf(p, t, 0.23591267f);
  p = __builtin_fmaf(p, t, -0.24234506f);
  p = __builtin_fmaf(p, t, 0.25852355f);
  p = __builtin_fmaf(p, t, -0.03702401f);
  p = __builtin_fmaf(p, t, 0.10319236f);
  p = __builtin_fmaf(p, t, 0.07523449f);
  p = __builtin_fmaf(p, t, 0.08521185f);
  p = __builtin_fmaf(p, t, 0.08460238f);
  *e = __builtin_amdgcn_exp2f(-0.7213475204444817f * z * z);
  const float h = p * t * *e;
  return z < 0.0f ? h : 1.0f - h;
}

__device__ inline float activate(int act, float beta, float z) {
  switch (act) {
    case kActRelu: return z < 0.0f ? 0.0f : z;   // NaN stays
    case kActSwish: return z * sigmoid_only(beta * z);
    case kActGelu: {
      float e;
      return z * normal_cdf(z, &e);
    }
    case kActGeluTanh: return z * sigmoid_only(z * __builtin_fmaf(kTanh3 * z, z, kTanh1));
    default: return z;
  }
}

// 8 values: one test of the kind
__device__ inline void activate8(int act, float beta, float* v) {
#define SWG_EACH(EXPR)                                \
  _Pragma("unroll") for (int i = 0; i < 8; ++i) {     \
    const float z = v[i];                             \
    v[i] = (EXPR);                                    \
  }                                                   \
  break
  switch (act) {
    case kActRelu: SWG_EACH(activate(kActRelu, beta, z));
    case kActSwish: SWG_EACH(activate(kActSwish, beta, z));
    case kActGelu: SWG_EACH(activate(kActGelu, beta, z));
    case kActGeluTanh: SWG_EACH(activate(kActGeluTanh, beta, z));
    default: break;
  }
#undef SWG_EACH
}

// v held within most on either side, in one instruction; a NaN, which is not kept, comes out of the
// other term of the slopes below
__device__ inline float held(float v, float most) {
  return __builtin_amdgcn_fmed3f(v, -most, most);
}

// A z of +-infinity, as a 16-bit z beyond its type is kept, has the slope of large z: what vanishes
// there multiplies an argument that is held where it is 0 in fp32 anyway.
__device__ inline float activation_slope(int act, float beta, float z) {
  switch (act) {
    case kActRelu: return z > 0.0f ? 1.0f : z != z ? z : 0.0f;
    case kActSwish: {
      const float t = beta * z;
      const SigmoidParts p = sigmoid_parts(t);         // sigma (1 - sigma) is 0 from |t| = 104 on
      return __builtin_fmaf(held(t, 128.0f), p.s1ms, p.s);
    }
    case kActHalf: return z != z ? z : 0.5f;
    case kActGelu: {
      float e;                                         // 0 from |z| = 14.5 on
      const float cdf = normal_cdf(z, &e);
      return __builtin_fmaf(held(z, 16.0f), kInvSqrt2Pi * e, cdf);
    }
    case kActGeluTanh: {
      const float c = held(z, 16.0f);                  // sigma (1 - sigma) is 0 from |z| = 12 on
      const SigmoidParts p = sigmoid_parts(z * __builtin_fmaf(kTanh3 * z, z, kTanh1));
      return __builtin_fmaf(c * __builtin_fmaf(3.0f * kTanh3 * c, c, kTanh1), p.s1ms, p.s);
    }
    default: return 1.0f;
  }
}

}  // namespace swg
