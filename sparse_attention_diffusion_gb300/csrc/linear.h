// Host-side interface of the matrix product with bias, activation, gate and
// residual: y = residual + gate_b * act(x w^T + bias).
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

namespace mcs {

// How many 64-column steps one tensor-core accumulator takes. The tensor core adds by truncation
// (on this GPU two bits below the sum's last one are kept, measured), so errors have the sums'
// sign and grow with their number: a step of 16 columns costs up to 5.25 * 2^-23 of the running
// sum, half a last bit on average. Up to kOneAccSteps (1,536 columns) a row has one accumulator;
// a longer one takes one for every kAccSteps (1,024 columns), and they are added in fp32 registers,
// to nearest. Against one accumulator for any length that costs about half a microsecond a call
// (452 x 4,096 -> 5,120 18.1 -> 18.8 us, 2,048 x 8,192 -> 2,048 42.1 -> 42.8 us; 1,024 x 2,048 ->
// 1,536 9.4 -> 10.2 us, which is why shorter rows are left whole), and at 5,120 columns 0.08 % of
// the bf16 outputs instead of 0.28 % differ from the rounded fp32 sum's.
constexpr int kOneAccSteps = 24;
constexpr int kAccSteps = 16;
inline int acc_count(int steps) { return steps <= kOneAccSteps ? 1 : (steps + kAccSteps - 1) / kAccSteps; }

struct LinearParams {
  const void* x;         // [B, N, K], or [B, heads, N, K / heads]
  const void* w;         // [O, K]
  const void* bias;      // [O] or null
  const void* gate;      // [B, O] or null
  const void* residual;  // [M, O] or null
  void* y;               // [M, O]
  int B, N, M;           // M = B * N rows
  int K, O;
  int heads;             // 0: token-major x
  int act;               // mcs_act
  uint32_t* status;
};
// What a product runs as: the kernel (mcs_linear_kernel), columns (pairs) or rows of x (few) of a tile, K slices,
// and accumulators a slice takes one after another.
struct LinearPlan {
  int kernel, tile, slices, accumulators;
};
LinearPlan plan_linear_tc(const LinearParams& p, int num_sms);
LinearPlan plan_linear_f32(const LinearParams& p, int num_sms);
cudaError_t linear_tc(const LinearParams& p, int num_sms, cudaStream_t s);
// fp32: rows by the CUDA cores (up to eight) or the tensor cores in bf16 parts.
cudaError_t linear_f32(const LinearParams& p, int num_sms, cudaStream_t s);
cudaError_t linear_split(const LinearParams& p, int splits, cudaStream_t s);

}  // namespace mcs
