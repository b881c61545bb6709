// Epilogue arithmetic of the matrix products: activation, gate and residual in
// fp32, one rounding at the store.
#pragma once
#include <cuda_bf16.h>

#include "common.cuh"
#include "linear.h"
#include "mcs.h"

namespace mcs {

// The gates of SiLU and of the tanh form of GELU are logistic functions, z /
// (1 + exp(-t)): no cancellation for negative z, and exp overflowing to
// infinity gives the right limit 0. GELU's erf form uses erfc for the same reason.
__device__ __forceinline__ float activate(int act, float z) {
  if (act == MCS_ACT_NONE) return z;
  if (act == MCS_ACT_GELU_ERF) return 0.5f * z * erfcf(z * -0.70710678f);
  // sqrt(8 / pi) = 1.5957691216
  const float t = act == MCS_ACT_SILU ? z : 1.5957691216f * (z + 0.044715f * z * z * z);
  return __fdividef(z, 1.f + __expf(-t));
}

// One output element from its sum (any alignment).
template <typename T>
__device__ __forceinline__ void finish_one(const LinearParams& p, int m, int o, float acc) {
  if (p.bias) acc += to_f32(static_cast<const T*>(p.bias)[o]);
  acc = activate(p.act, acc);
  if (p.gate) acc *= to_f32(static_cast<const T*>(p.gate)[size_t(m / p.N) * p.O + o]);
  const size_t at = size_t(m) * p.O + o;
  if (p.residual) acc += to_f32(static_cast<const T*>(p.residual)[at]);
  static_cast<T*>(p.y)[at] = from_f32<T>(acc);
}

}  // namespace mcs
