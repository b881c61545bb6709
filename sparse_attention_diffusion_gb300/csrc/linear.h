// Host-side interface of the matrix product with bias, activation, gate and
// residual: y = residual + gate_b * act(x w^T + bias).
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

namespace mcs {

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
cudaError_t linear_tc(const LinearParams& p, int num_sms, cudaStream_t s);
// fp32: rows by the CUDA cores (up to eight) or the tensor cores in bf16 parts.
cudaError_t linear_f32(const LinearParams& p, int num_sms, cudaStream_t s);
cudaError_t linear_split(const LinearParams& p, int num_sms, cudaStream_t s);

}  // namespace mcs
