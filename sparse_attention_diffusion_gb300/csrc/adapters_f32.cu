// Projections with low-rank adapters, fp32: h = scale_a x down_a^T and then h up_a^T on the CUDA cores, for the
// fp32 product's epilogue to add to its sums. Both read and compute R / in of what the product does.
#include "adapters.h"
#include "common.cuh"
#include "launch.cuh"
#include "linear.h"
#include "ptx.cuh"
#include "status.cuh"

namespace mcs {
namespace {

// z = h up_a^T, 0 in rows without an adapter: 64 x 64 outputs a block, 4 x 4 a thread, 16 columns of R at a time.
constexpr int kTile = 64, kStep = 16, kLd = kStep + 4;
__global__ void __launch_bounds__(256) adapters_f32_up_kernel(const LinearParams p, const AdapterParams a, const float* h, float* z) {
  __shared__ __align__(16) float hs[kTile][kLd], us[kTile][kLd];
  const int tid = threadIdx.x, lane = tid & 31, ty = tid >> 4, tx = tid & 15;
  const long long m0 = static_cast<long long>(blockIdx.x) * kTile;
  const int o0 = blockIdx.y * kTile;
  grid_inputs_ready();
  grid_let_next_start();
  const int m1 = int(min(static_cast<long long>(p.M), m0 + kTile));
  float acc[4][4] = {};
  for (int s = max(0, segment_at(a.start, a.S, int(m0), lane)); s < a.S; ++s) {
    if (a.start[s] >= m1) break;
    int ra, rb;
    segment_rows(a.start, s, p.M, ra, rb);
    const int lo = max(ra, int(m0)), hi = min(rb, m1);
    if (lo >= hi) continue;
    const int ad = a.which[s];
    if (ad < 0 || ad >= a.count) continue;
    const float* up = static_cast<const float*>(a.up) + static_cast<size_t>(ad) * p.O * a.R;
    const int first = int(m0) + ty * 4;
    for (int r0 = 0; r0 < a.R; r0 += kStep) {
      __syncthreads();
      {
        const int row = tid / 4, c = r0 + tid % 4 * 4, m = int(m0) + row, o = o0 + row;  // R is a multiple of 4
        const float4 none = make_float4(0.f, 0.f, 0.f, 0.f);
        *reinterpret_cast<float4*>(&hs[row][tid % 4 * 4]) =
            m >= lo && m < hi && c < a.R ? *reinterpret_cast<const float4*>(h + static_cast<size_t>(m) * a.R + c) : none;
        *reinterpret_cast<float4*>(&us[row][tid % 4 * 4]) =
            o < p.O && c < a.R ? *reinterpret_cast<const float4*>(up + static_cast<size_t>(o) * a.R + c) : none;
      }
      __syncthreads();
      if (first + 4 <= lo || first >= hi) continue;  // none of this thread's rows
#pragma unroll
      for (int k = 0; k < kStep; k += 4) {
        float4 u[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) u[j] = *reinterpret_cast<const float4*>(&us[tx + 16 * j][k]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (first + i < lo || first + i >= hi) continue;  // 0 times what is not finite
          const float4 w = *reinterpret_cast<const float4*>(&hs[ty * 4 + i][k]);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            acc[i][j] = fmaf(w.w, u[j].w, fmaf(w.z, u[j].z, fmaf(w.y, u[j].y, fmaf(w.x, u[j].x, acc[i][j]))));
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const long long m = m0 + ty * 4 + i;
    if (m >= p.M) break;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int o = o0 + tx + 16 * j;
      if (o < p.O) z[static_cast<size_t>(m) * p.O + o] = acc[i][j];
    }
  }
}

// The same where few rows share an adapter: a block takes a row and 256 outputs, a thread an output, whose row of `up`
// it reads by itself.
__global__ void __launch_bounds__(256) adapters_f32_up_rows_kernel(const LinearParams p, const AdapterParams a, const float* h, const int32_t* of_row, float* z) {
  const int o = blockIdx.y * 256 + threadIdx.x, m = blockIdx.x;
  grid_inputs_ready();
  grid_let_next_start();
  if (o >= p.O) return;
  const int ad = of_row[m];
  float acc = 0.f;
  if (ad >= 0) {
    const float4* x = reinterpret_cast<const float4*>(h + static_cast<size_t>(m) * a.R);
    const float4* u = reinterpret_cast<const float4*>(static_cast<const float*>(a.up) + (static_cast<size_t>(ad) * p.O + o) * a.R);
#pragma unroll 4
    for (int r = 0; r < a.R / 4; ++r) {
      const float4 v = x[r], w = __ldg(u + r);
      acc = fmaf(v.w, w.w, fmaf(v.z, w.z, fmaf(v.y, w.y, fmaf(v.x, w.x, acc))));
    }
  }
  z[static_cast<size_t>(m) * p.O + o] = acc;
}

}  // namespace

cudaError_t linear_adapters_f32(const LinearParams& p, const AdapterParams& a, int num_sms, cudaStream_t s) {
  float* h = static_cast<float*>(a.ws);
  float* z = h + (size_t(p.M) * a.R + 63) / 64 * 64;
  int32_t* of_row = reinterpret_cast<int32_t*>(z + (size_t(p.M) * p.O + 63) / 64 * 64);
  cudaError_t e = adapters_down_rows(p, a, false, h, of_row, s);
  if (e != cudaSuccess) return e;
  // a tile of 64 rows goes through its segments one by one (70 rows with adapters of their own: 88 us in all, 31 row by row)
  if (p.M <= 4ll * a.S)
    e = launch_overlapped(adapters_f32_up_rows_kernel, dim3(unsigned(p.M), (p.O + 255) / 256), 256, 0, s, 0, p, a, h, of_row, z);
  else
    e = launch_overlapped(adapters_f32_up_kernel, dim3((unsigned(p.M) + kTile - 1) / kTile, (p.O + kTile - 1) / kTile), 256, 0, s, 0, p, a, h, z);
  if (e != cudaSuccess) return e;
  LinearParams with = p;
  with.add = z;
  return linear_f32(with, num_sms, s);
}

}  // namespace mcs
