// The gate functions of the single-token steps and of the gated linear
// recurrence, with their derivatives, in fp32 (see gdr.h for the definitions).
#pragma once

#include "../gdr_device.h"

namespace gdr {

// log2(1 + e) for e in [0, 1].  u = 1 + e is rounded; c = e - (u - 1) is what the
// rounding lost, exactly, and log2(u + c) = log2(u) + c log2(e) / u with u near 1
// wherever c matters: without it a small e would keep no relative accuracy.
__device__ __forceinline__ float log2_1p(float e) {
  const float u = 1.f + e;
  return fmaf(e - (u - 1.f), kLog2e, __builtin_amdgcn_logf(u));
}

// 1 - 2^l given a = 2^l: near l = 0 by the series of 1 - e^x, x = l ln 2 (next term
// x^7 / 5040)
__device__ __forceinline__ float one_minus_exp2(float l, float a) {
  const float x = l * 0.6931471805599453f;
  const float series = -x * (1.f + x * (0.5f + x * (1.f / 6.f + x * (1.f / 24.f + x * (1.f / 120.f + x * (1.f / 720.f))))));
  return fabsf(l) < 0.36f ? series : 1.f - a;
}

// Base-2 log decay of the per-channel gates (lambda log2(e), so that the decay is
// one bare exponential) from z2 = (raw gate + bias) log2(e).
//   FN 0: -eA softplus(z);  FN 1: gs sigmoid(eA z)
template <int FN>
__device__ __forceinline__ float gate_log2(float z2, float eA, float gs) {
  if constexpr (FN == 0) return -eA * (fmaxf(z2, 0.f) + log2_1p(fast_exp2(-fabsf(z2))));
  else return gs * kLog2e * __builtin_amdgcn_rcpf(1.f + fast_exp2(-eA * z2));
}

// The same with the slope d lambda / d z.  Where the gate saturates (z infinite) the
// slope is finite, so a gate that is shut or open for good gives zero gradients and
// no NaN.
template <int FN>
__device__ __forceinline__ void gate_log2_grad(float z2, float eA, float gs, float& l2, float& dz) {
  if constexpr (FN == 0) {
    const float e = fast_exp2(-fabsf(z2));
    const float r = __builtin_amdgcn_rcpf(1.f + e);
    l2 = -eA * (fmaxf(z2, 0.f) + log2_1p(e));
    dz = -eA * (z2 >= 0.f ? r : e * r);
  } else {
    const float w2 = eA * z2;
    const float e = fast_exp2(-fabsf(w2));
    const float r = __builtin_amdgcn_rcpf(1.f + e);
    l2 = gs * kLog2e * (w2 >= 0.f ? r : e * r);
    dz = gs * eA * (e * r * r);
  }
}

}  // namespace gdr
