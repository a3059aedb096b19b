// The gate functions of the single-token steps and of the gated linear
// recurrence, with their derivatives, in fp32 (see gdr.h for the definitions).
#pragma once

#include "gdr_device.h"

namespace gdr {

// exp for the storage type: the hardware exponential of x log2(e) (rounding the
// product costs |x| 2^-24 relative, nothing beside a bf16 result) or expf
template <typename TIO> __device__ __forceinline__ float exp_io(float x);
template <> __device__ __forceinline__ float exp_io<bf16>(float x) { return __expf(x); }
template <> __device__ __forceinline__ float exp_io<float>(float x) { return expf(x); }

// log(1 + e) for e in [0, 1]: the hardware log of a rounded 1 + e loses the
// relative accuracy of a small e, so there the series (next term e^6 / 6 < 2e-8 e)
__device__ __forceinline__ float log1p01(float e) {
  const float series = e * (1.f + e * (-0.5f + e * (1.f / 3.f + e * (-0.25f + e * 0.2f))));
  return e < 0.04f ? series : __logf(1.f + e);
}

// 1 - exp(l) given a = exp(l): near l = 0 by the series (next term l^7 / 5040)
__device__ __forceinline__ float one_minus_exp(float l, float a) {
  const float series = -l * (1.f + l * (0.5f + l * (1.f / 6.f + l * (1.f / 24.f + l * (1.f / 120.f + l * (1.f / 720.f))))));
  return fabsf(l) < 0.25f ? series : 1.f - a;
}

// Log decay of the per-channel gates from the raw gate plus bias z.
//   FN 0: -eA softplus(z);  FN 1: gs sigmoid(eA z)
template <typename TIO, int FN>
__device__ __forceinline__ float gate_log(float z, float eA, float gs) {
  if constexpr (FN == 0) {
    return -eA * (fmaxf(z, 0.f) + log1p01(exp_io<TIO>(-fabsf(z))));
  } else {
    return gs / (1.f + exp_io<TIO>(-eA * z));
  }
}

// The same with d lambda / d z and d lambda / d A_log.  Where the sigmoid or the
// decay saturates (z infinite) the slopes are finite, so a gate that is shut or
// open for good gives zero gradients and no NaN.
template <typename TIO, int FN>
__device__ __forceinline__ void gate_log_grad(float z, float eA, float gs, float& lam, float& dz, float& dA) {
  if constexpr (FN == 0) {
    const float e = exp_io<TIO>(-fabsf(z));
    const float r = 1.f / (1.f + e);
    lam = -eA * (fmaxf(z, 0.f) + log1p01(e));
    dz = -eA * (z >= 0.f ? r : e * r);
    dA = fmaxf(lam, -3.0e38f);
  } else {
    const float w = eA * z;
    const float e = exp_io<TIO>(-fabsf(w));
    const float r = 1.f / (1.f + e);
    const float slope = gs * e * r * r;
    lam = gs * (w >= 0.f ? r : e * r);
    dz = slope * eA;
    dA = slope * fminf(fmaxf(w, -200.f), 200.f);
  }
}

}  // namespace gdr
