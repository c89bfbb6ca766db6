// i8_act.h -- the activations (GEMMQ_ACT_*) on the device.
#pragma once

#include <float.h>

#include "i8_block.h"
#include "i8_common.h"

namespace gemmq {
namespace i8 {

// SiLU and tanh's GELU are both z sigma(z (c0 + c1 z^2)): (1 + tanh a) / 2 = sigma(2 a),
// 2 a = sqrt(8 / pi) (z + 0.044715 z^3); ReLU and none max(z, c0), with 0 or -inf, that
// keeps a NaN.  The kernels' unrolled epilogues hold each form once, SiLU one of its own: it
// is what most gates have, and takes two thirds of the other's instructions (the gated pair
// of 2048 x 12288 over 4096 208 -> 204 us).
struct Act {
  enum Form { kMax, kSilu, kSigmoid, kErf } form;
  float c0, c1;
};

__device__ __forceinline__ Act act_of(int act) {
  switch (act) {
    case GEMMQ_ACT_SILU: return {Act::kSilu, 1.0f, 0.0f};
    case GEMMQ_ACT_GELU_TANH: return {Act::kSigmoid, 1.5957691216057308f, 0.07135481282637043f};
    case GEMMQ_ACT_GELU: return {Act::kErf, 0.0f, 0.0f};
    case GEMMQ_ACT_RELU: return {Act::kMax, 0.0f, 0.0f};
    default: return {Act::kMax, -__builtin_inff(), 0.0f};
  }
}

__device__ __forceinline__ float sigmoid(float arg) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(arg * -kLog2e));
}
// sigma(z (c0 + c1 z^2)); past |z| = 10^15 its sign is all that counts, and z^2 is held
// there so that 0 * infinity does not come up
__device__ __forceinline__ float sigmoid_of(const Act& a, float z) {
  return sigmoid(z * fmaf(a.c1, fminf(z * z, 1e30f), a.c0));
}
// the normal distribution's function, (1 + erf(z / sqrt 2)) / 2
__device__ __forceinline__ float normal_of(float z) {
  return fmaf(0.5f, erff(z * 0.7071067811865476f), 0.5f);
}

// At an infinite z (a sum past f32, or z kept in f16, which ends at 65504) act and its slope are
// their limits: the factor z of sigma(z) = 0 is held at the lowest f32, where 0 * infinity would
// come up.  A NaN is kept by the other factor.
__device__ __forceinline__ float above_lowest(float z) { return fmaxf(z, -FLT_MAX); }

// act(z) for each of z[0..N)
template <int N>
__device__ __forceinline__ void activate(const Act& a, float (&z)[N]) {
  if (a.form == Act::kSilu) {
#pragma unroll
    for (int e = 0; e < N; ++e) z[e] = above_lowest(z[e]) * sigmoid(z[e]);
  } else if (a.form == Act::kSigmoid) {
#pragma unroll
    for (int e = 0; e < N; ++e) z[e] = above_lowest(z[e]) * sigmoid_of(a, z[e]);
  } else if (a.form == Act::kErf) {
#pragma unroll
    for (int e = 0; e < N; ++e) z[e] = above_lowest(z[e]) * normal_of(z[e]);
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e) z[e] = z[e] < a.c0 ? a.c0 : z[e];
  }
}

// act(z) and its derivative: with p = sigma(arg), p + z p (1 - p) arg'; Phi + z phi; and
// ReLU's is 0 at 0
__device__ __forceinline__ void activate_slope(const Act& a, float z, float& value, float& slope) {
  if (a.form == Act::kSilu || a.form == Act::kSigmoid) {
    const float p = sigmoid_of(a, z);
    value = above_lowest(z) * p;
    slope = fmaf(fminf(value, FLT_MAX) * (1.0f - p), fmaf(3.0f * a.c1, fminf(z * z, 1e30f), a.c0), p);
  } else if (a.form == Act::kErf) {
    const float p = normal_of(z);
    const float density = 0.3989422804014327f * __builtin_amdgcn_exp2f(z * z * (-0.5f * kLog2e));
    value = above_lowest(z) * p;
    slope = fmaf(fminf(above_lowest(z), FLT_MAX), density, p);
  } else {
    value = z < a.c0 ? a.c0 : z;
    slope = a.c0 == 0.0f && z <= 0.0f ? 0.0f : 1.0f;
  }
}

}  // namespace i8
}  // namespace gemmq
