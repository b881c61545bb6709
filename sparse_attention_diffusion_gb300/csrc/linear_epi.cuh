// Epilogue arithmetic of the matrix products: activation, gate and residual in
// fp32, one rounding at the store.
#pragma once
#include <cuda_bf16.h>

#include "common.cuh"
#include "linear.h"
#include "mcs.h"

namespace mcs {

// The gates of SiLU and of the tanh form of GELU are logistic functions, z / (1 + exp(-t)), taken
// as z exp(t) / (1 + exp(t)) for negative t: no cancellation, no overflow, and a denominator
// between 1 and 2, which the fast division needs. GELU's erf form uses erfc for the same reason.
// bf16 outputs take the fast exponential (2 + 1.2 |t| ulp, below 2^-16 wherever the result is in
// bf16's normal range) and division. fp32 outputs take expf (2 ulp), of t / 2 and squared, so that
// it stays in the normal range as long as the result does, and the division to nearest.
template <bool kF32>
__device__ __forceinline__ float logistic_gate(float z, float t) {
  if constexpr (kF32) {
    const float h = expf(-0.5f * fabsf(t));
    return (t < 0.f ? z * h * h : z) / (1.f + h * h);
  } else {
    const float e = __expf(-fabsf(t));
    return __fdividef(t < 0.f ? z * e : z, 1.f + e);
  }
}
template <int kAct, bool kF32 = false, int n>
__device__ __forceinline__ void activate(float (&v)[n]) {
#pragma unroll
  for (int i = 0; i < n; ++i) {
    if constexpr (kAct == MCS_ACT_GELU_TANH)  // sqrt(8 / pi) = 1.5957691216
      v[i] = logistic_gate<kF32>(v[i], 1.5957691216f * (v[i] + 0.044715f * v[i] * v[i] * v[i]));
    else if constexpr (kAct == MCS_ACT_SILU)
      v[i] = logistic_gate<kF32>(v[i], v[i]);
    else if constexpr (kAct == MCS_ACT_GELU_ERF)
      v[i] = 0.5f * v[i] * erfcf(v[i] * -0.70710678f);
  }
}

// One output element from its sum (any alignment).
template <int kAct, typename T>
__device__ __forceinline__ void finish_one(const LinearParams& p, int m, int o, float acc) {
  if (p.bias) acc += to_f32(static_cast<const T*>(p.bias)[o]);
  float v[1] = {acc};
  activate<kAct, sizeof(T) == 4>(v);
  acc = v[0];
  if (p.gate) acc *= to_f32(static_cast<const T*>(p.gate)[size_t(m / p.N) * p.O + o]);
  const size_t at = size_t(m) * p.O + o;
  if (p.residual) acc += to_f32(static_cast<const T*>(p.residual)[at]);
  static_cast<T*>(p.y)[at] = from_f32<T>(acc);
}

// Eight bf16 values of a 16-byte word.
__device__ __forceinline__ void unpack8(const uint4& w, float (&v)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) v[2 * i] = __uint_as_float(u[i] << 16), v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
}
// Four consecutive bf16 outputs of one row from their sums; bias4 holds the bias
// there (ignored where absent). Needs O % 4 == 0.
__device__ __forceinline__ void unpack4(const uint2& w, float (&v)[4]) {
  v[0] = __uint_as_float(w.x << 16), v[1] = __uint_as_float(w.x & 0xffff0000u);
  v[2] = __uint_as_float(w.y << 16), v[3] = __uint_as_float(w.y & 0xffff0000u);
}
template <int kAct>
__device__ __forceinline__ void finish_four(const LinearParams& p, int m, int o, float (&v)[4], const uint2& bias4) {
  float t[4];
  const size_t at = size_t(m) * p.O + o;
  if (p.bias) {
    unpack4(bias4, t);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] += t[i];
  }
  activate<kAct>(v);
  if (p.gate) {
    unpack4(*reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p.gate) + size_t(m / p.N) * p.O + o), t);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] *= t[i];
  }
  if (p.residual) {
    unpack4(*reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p.residual) + at), t);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] += t[i];
  }
  const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
  *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.y) + at) =
      make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}

// Four consecutive fp32 outputs of one row from their sums (any alignment).
template <int kAct>
__device__ __forceinline__ void finish_row4(const LinearParams& p, int m, int o, float (&v)[4]) {
  if (p.O % 4 != 0 || o + 4 > p.O) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (o + i < p.O) finish_one<kAct, float>(p, m, o + i, v[i]);
    return;
  }
  auto at4 = [](const void* q, size_t i) { return *reinterpret_cast<const float4*>(static_cast<const float*>(q) + i); };
  const size_t at = size_t(m) * p.O + o;
  if (p.bias) {
    const float4 t = at4(p.bias, o);
    v[0] += t.x, v[1] += t.y, v[2] += t.z, v[3] += t.w;
  }
  activate<kAct, true>(v);
  if (p.gate) {
    const float4 t = at4(p.gate, size_t(m / p.N) * p.O + o);
    v[0] *= t.x, v[1] *= t.y, v[2] *= t.z, v[3] *= t.w;
  }
  if (p.residual) {
    const float4 t = at4(p.residual, at);
    v[0] += t.x, v[1] += t.y, v[2] += t.z, v[3] += t.w;
  }
  *reinterpret_cast<float4*>(static_cast<float*>(p.y) + at) = make_float4(v[0], v[1], v[2], v[3]);
}

}  // namespace mcs
