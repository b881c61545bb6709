// fp32 matrix product with epilogue in SIMT arithmetic: 64 x 64 output tiles,
// K in steps of 16 through shared memory, 4 x 4 outputs per thread.
#include "launch.cuh"
#include "linear.h"
#include "linear_epi.cuh"

namespace mcs {
namespace {

constexpr int kT = 64, kBK = 16;

// Address of x[row m][k] for either layout (k a multiple of 4 stays inside a head).
__device__ __forceinline__ const float* x_at(const LinearParams& p, int m, int k) {
  const float* x = static_cast<const float*>(p.x);
  if (p.heads == 0) return x + size_t(m) * p.K + k;
  const int d = p.K / p.heads, b = m / p.N, n = m % p.N;
  return x + ((size_t(b) * p.heads + k / d) * p.N + n) * d + k % d;
}

template <int kAct>
__global__ void __launch_bounds__(256) linear_simt_kernel(const LinearParams p) {
  __shared__ float xs[kBK][kT + 4], wsm[kBK][kT + 4];
  const int tid = threadIdx.x, tx = tid % 16, ty = tid / 16;
  const int m0 = blockIdx.x * kT, o0 = blockIdx.y * kT;
  const int lr = tid / 4, lk = (tid % 4) * 4;  // this thread's row and first k of the loads
  grid_inputs_ready();
  grid_let_next_start();
  float acc[4][4] = {};
  for (int k0 = 0; k0 < p.K; k0 += kBK) {
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
    if (k0 + lk < p.K) {
      if (m0 + lr < p.M) a = *reinterpret_cast<const float4*>(x_at(p, m0 + lr, k0 + lk));
      if (o0 + lr < p.O)
        b = *reinterpret_cast<const float4*>(static_cast<const float*>(p.w) + size_t(o0 + lr) * p.K + k0 + lk);
    }
    __syncthreads();
    xs[lk][lr] = a.x, xs[lk + 1][lr] = a.y, xs[lk + 2][lr] = a.z, xs[lk + 3][lr] = a.w;
    wsm[lk][lr] = b.x, wsm[lk + 1][lr] = b.y, wsm[lk + 2][lr] = b.z, wsm[lk + 3][lr] = b.w;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kBK; ++k) {
      float av[4], bv[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) av[i] = xs[k][ty * 4 + i], bv[i] = wsm[k][tx * 4 + i];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] += av[i] * bv[j];
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int m = m0 + ty * 4 + i, o = o0 + tx * 4 + j;
      if (m < p.M && o < p.O) finish_one<kAct, float>(p, m, o, acc[i][j]);
    }
}

}  // namespace

cudaError_t linear_simt(const LinearParams& p, int num_sms, cudaStream_t s) {
  (void)num_sms;
  const dim3 grid((p.M + kT - 1) / kT, (p.O + kT - 1) / kT);
  switch (p.act) {
    case MCS_ACT_GELU_TANH: return launch_overlapped(linear_simt_kernel<MCS_ACT_GELU_TANH>, grid, 256, 0, s, 0, p);
    case MCS_ACT_GELU_ERF: return launch_overlapped(linear_simt_kernel<MCS_ACT_GELU_ERF>, grid, 256, 0, s, 0, p);
    case MCS_ACT_SILU: return launch_overlapped(linear_simt_kernel<MCS_ACT_SILU>, grid, 256, 0, s, 0, p);
    default: return launch_overlapped(linear_simt_kernel<MCS_ACT_NONE>, grid, 256, 0, s, 0, p);
  }
}

}  // namespace mcs
