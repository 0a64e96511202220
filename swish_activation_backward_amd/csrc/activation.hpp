// Activations of the linear layer's epilogue and their slopes, in fp32.
#pragma once

#include "common.hpp"
#include "launch.hpp"

namespace swg {

constexpr float kSqrtHalf = 0.7071067811865476f;
constexpr float kInvSqrt2Pi = 0.3989422804014327f;
// the tanh form of gelu is z sigma(2 a), 2 a = kTanh1 z + kTanh3 z^3
constexpr float kTanh1 = 1.5957691216057308f;
constexpr float kTanh3 = 0.07135481627159929f;

__device__ inline float activate(int act, float beta, float z) {
  switch (act) {
    case kActRelu: return z < 0.0f ? 0.0f : z;   // NaN stays
    case kActSwish: return z * sigmoid_only(beta * z);
    case kActGelu: return 0.5f * z * erfcf(-z * kSqrtHalf);
    case kActGeluTanh: return z * sigmoid_only(z * __builtin_fmaf(kTanh3 * z, z, kTanh1));
    default: return z;
  }
}

__device__ inline float activation_slope(int act, float beta, float z) {
  switch (act) {
    case kActRelu: return z > 0.0f ? 1.0f : z != z ? z : 0.0f;
    case kActSwish: return swish_factor(beta * z);
    case kActGelu: {
      const float pdf = kInvSqrt2Pi * __builtin_amdgcn_exp2f(-0.7213475204444817f * z * z);
      return __builtin_fmaf(z, pdf, 0.5f * erfcf(-z * kSqrtHalf));
    }
    case kActGeluTanh: {
      // sigma (1 - sigma) is 0 in fp32 from |z| = 12 on: the powers of z stay finite
      const float c = __builtin_fminf(__builtin_fmaxf(z, -16.0f), 16.0f);
      const SigmoidParts p = sigmoid_parts(z * __builtin_fmaf(kTanh3 * z, z, kTanh1));
      return __builtin_fmaf(c * __builtin_fmaf(3.0f * kTanh3 * c, c, kTanh1), p.s1ms, p.s);
    }
    default: return 1.0f;
  }
}

}  // namespace swg
