// fp32 matrix product with epilogue for up to eight rows, on the CUDA cores: each
// warp streams two rows of w against up to four rows of x, two products a packed
// FMA; reading w bounds it (1 x 5,120 -> 5,120 27 us = 0.58 of the copy bandwidth).
#include "launch.cuh"
#include "linear.h"
#include "linear_epi.cuh"
#include "linear_few.h"
#include "ptx.cuh"

namespace mcs {
namespace {

constexpr int kThreads = 256;

// x as rows of any layout: element (row, k) at row_base + (k >> shift) * head + (k & mask).
struct XView {
  long long head;  // elements between heads of a row
  int mask, shift;
};
__device__ __forceinline__ const float* x_row(const LinearParams& p, int m) {
  const float* x = static_cast<const float*>(p.x);
  if (p.heads == 0) return x + size_t(m) * p.K;
  const int b = m / p.N, n = m - b * p.N;
  return x + (size_t(b) * p.heads * p.N + n) * (p.K / p.heads);
}

// Few rows: a warp takes kOut rows of w and kRows rows of x, lanes along K;
// kUnroll 16-byte pieces of each row of w are in flight per lane.
template <int kRows, int kOut, int kUnroll, int kAct>
__global__ void __launch_bounds__(kThreads) linear_f32_few_kernel(const LinearParams p, const XView xv) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int o0 = (blockIdx.x * (kThreads / 32) + warp) * kOut, m0 = blockIdx.y * kRows;
  grid_inputs_ready();
  grid_let_next_start();
  if (o0 >= p.O) return;
  const int rows = min(kRows, p.M - m0), outs = min(kOut, p.O - o0);
  const float* w = static_cast<const float*>(p.w) + size_t(o0) * p.K;
  const float* xr[kRows];
#pragma unroll
  for (int m = 0; m < kRows; ++m) xr[m] = x_row(p, m0 + min(m, rows - 1));
  uint64_t acc[kRows][kOut];
#pragma unroll
  for (int m = 0; m < kRows; ++m)
#pragma unroll
    for (int o = 0; o < kOut; ++o) acc[m][o] = f2_pack(0.f, 0.f);
#pragma unroll kUnroll
  for (int k = lane * 4; k < p.K; k += 128) {
    float4 wv[kOut];
#pragma unroll
    for (int o = 0; o < kOut; ++o)
      wv[o] = *reinterpret_cast<const float4*>(w + size_t(min(o, outs - 1)) * p.K + k);
    const long long at = (k >> xv.shift) * xv.head + (k & xv.mask);
#pragma unroll
    for (int m = 0; m < kRows; ++m) {
      if (m < rows) {
        const float4 x = *reinterpret_cast<const float4*>(xr[m] + at);
        const uint64_t x0 = f2_pack(x.x, x.y), x1 = f2_pack(x.z, x.w);
#pragma unroll
        for (int o = 0; o < kOut; ++o)
          acc[m][o] = f2_fma(x1, f2_pack(wv[o].z, wv[o].w), f2_fma(x0, f2_pack(wv[o].x, wv[o].y), acc[m][o]));
      }
    }
  }
#pragma unroll
  for (int m = 0; m < kRows; ++m) {
    float v[kOut];
#pragma unroll
    for (int o = 0; o < kOut; ++o) {
      float a, b;
      f2_unpack(acc[m][o], a, b);
      v[o] = a + b;
#pragma unroll
      for (int s = 16; s > 0; s >>= 1) v[o] += __shfl_xor_sync(0xffffffffu, v[o], s);
    }
    if (m < rows && lane < outs) {
      float mine = v[0];
#pragma unroll
      for (int o = 1; o < kOut; ++o) mine = lane == o ? v[o] : mine;
      finish_one<kAct, float>(p, m0 + m, o0 + lane, mine);
    }
  }
}

template <int kAct>
cudaError_t launch(const LinearParams& p, cudaStream_t s) {
  XView xv{0, INT32_MAX, 31};
  if (p.heads > 0) {
    const int d = p.K / p.heads;
    xv = {static_cast<long long>(p.N) * d, d - 1, d == 64 ? 6 : 7};
  }
  if (p.M <= 2)
    return launch_overlapped(linear_f32_few_kernel<2, 2, 4, kAct>, dim3((p.O + 15) / 16), kThreads, 0, s, 0, p, xv);
  // five to eight rows read w twice, the second time mostly from L2
  return launch_overlapped(linear_f32_few_kernel<4, 2, 4, kAct>, dim3((p.O + 15) / 16, (p.M + 3) / 4), kThreads, 0, s, 0,
                           p, xv);
}

}  // namespace

LinearPlan plan_linear_f32(const LinearParams& p, int num_sms) {
  if (p.M <= 8) return {MCS_LINEAR_F32_ROWS, p.M <= 2 ? 2 : 4, 1, 1};
  // K slices of 128 x 128 tiles: the shortest estimate of waves x (steps of 32 columns of about 1,150 clocks + way in and out)
  const int nk = (p.K + 31) / 32;
  const long long row_tiles = p.heads > 0 ? static_cast<long long>((p.N + 127) / 128) * p.B : (p.M + 127) / 128;
  const long long tiles = row_tiles * ((p.O + 127) / 128);
  long long best = 0;
  int slices = 1;
  for (int splits = 1; splits <= 8 && splits <= nk; splits *= 2) {
    const int slots = few_slots(splits, num_sms);
    const long long cost = (tiles * splits + slots - 1) / slots *
                           (static_cast<long long>((nk + splits - 1) / splits) * 1150 + 6000 + (splits > 1 ? 3000 : 0));
    if (best == 0 || cost < best) best = cost, slices = splits;
  }
  return {MCS_LINEAR_F32_PARTS, 128, slices, (nk + slices - 1) / slices};
}

cudaError_t linear_f32(const LinearParams& p, int num_sms, cudaStream_t s) {
  const LinearPlan plan = plan_linear_f32(p, num_sms);
  if (plan.kernel == MCS_LINEAR_F32_PARTS) return linear_split(p, plan.slices, s);
  switch (p.act) {
    case MCS_ACT_GELU_TANH: return launch<MCS_ACT_GELU_TANH>(p, s);
    case MCS_ACT_GELU_ERF: return launch<MCS_ACT_GELU_ERF>(p, s);
    case MCS_ACT_SILU: return launch<MCS_ACT_SILU>(p, s);
    default: return launch<MCS_ACT_NONE>(p, s);
  }
}

}  // namespace mcs
