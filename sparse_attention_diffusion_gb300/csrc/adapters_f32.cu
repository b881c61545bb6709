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

// h: a block takes 4 rows and 8 columns, its four warps a quarter of K each, lanes along K; rows of several
// segments are worked off one segment after another.
constexpr int kRows = 4, kCols = 8, kWarps = 4;
__global__ void __launch_bounds__(32 * kWarps) adapters_f32_down_kernel(const LinearParams p, const AdapterParams a, float* h) {
  __shared__ float part[kWarps][kRows * kCols];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long m0 = static_cast<long long>(blockIdx.x) * kRows;
  const int c0 = blockIdx.y * kCols;
  grid_inputs_ready();
  grid_let_next_start();
  if (blockIdx.y == 0 && warp == 0) {
    for (long long s = static_cast<long long>(blockIdx.x) * 32 + lane; s < a.S; s += static_cast<long long>(gridDim.x) * 32) {
      int x, y;
      if (!segment_rows(a.start, int(s), p.M, x, y) || a.which[s] >= a.count) raise_status(p.status, kStatusBounds);
    }
    __syncwarp();
  }
  const int m1 = int(min(static_cast<long long>(p.M), m0 + kRows));
  const float* x[kRows];  // row m's columns, by head if they lie so
  const int hd = p.heads > 0 ? p.K / p.heads : p.K;
  const long long head = static_cast<long long>(p.N) * hd;  // from one head's column to the next head's
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    const int m = min(int(m0) + r, p.M - 1), b = m / p.N;
    x[r] = static_cast<const float*>(p.x) + (p.heads > 0 ? b * p.heads * head + static_cast<long long>(m - b * p.N) * hd
                                                         : static_cast<long long>(m) * p.K);
  }
  for (int s = max(0, segment_at(a.start, a.S, int(m0), lane)); s < a.S; ++s) {
    if (a.start[s] >= m1) break;
    int ra, rb;
    segment_rows(a.start, s, p.M, ra, rb);
    const int lo = max(ra, int(m0)), hi = min(rb, m1);
    if (lo >= hi) continue;
    const int ad = a.which[s];
    if (ad < 0 || ad >= a.count) continue;
    const float* down = static_cast<const float*>(a.down) + static_cast<size_t>(ad) * a.R * p.K;
    uint64_t sum[kRows][kCols] = {};
    for (int k = (warp * 32 + lane) * 4; k < p.K; k += 128 * kWarps) {
      const int q = k / hd;
      ulonglong2 xv[kRows];
#pragma unroll
      for (int r = 0; r < kRows; ++r) xv[r] = *reinterpret_cast<const ulonglong2*>(x[r] + (p.heads > 0 ? q * head + (k - q * hd) : k));
#pragma unroll
      for (int c = 0; c < kCols; ++c) {
        if (c0 + c >= a.R) break;
        const ulonglong2 dv = *reinterpret_cast<const ulonglong2*>(down + static_cast<size_t>(c0 + c) * p.K + k);
#pragma unroll
        for (int r = 0; r < kRows; ++r) sum[r][c] = f2_fma(xv[r].y, dv.y, f2_fma(xv[r].x, dv.x, sum[r][c]));
      }
    }
    __syncthreads();  // the last segment's sums have been read
#pragma unroll
    for (int r = 0; r < kRows; ++r)
#pragma unroll
      for (int c = 0; c < kCols; ++c) {
        float e, o;
        f2_unpack(sum[r][c], e, o);
        e += o;
#pragma unroll
        for (int w = 16; w > 0; w >>= 1) e += __shfl_xor_sync(0xffffffffu, e, w);
        if (lane == 0) part[warp][r * kCols + c] = e;
      }
    __syncthreads();
    if (warp == 0) {
      const int r = lane / kCols, c = lane % kCols, m = int(m0) + r;
      float e = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) e += part[w][lane];
      if (m >= lo && m < hi && c0 + c < a.R) h[static_cast<size_t>(m) * a.R + c0 + c] = a.scale[ad] * e;
    }
  }
}

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

}  // namespace

cudaError_t linear_adapters_f32(const LinearParams& p, const AdapterParams& a, int num_sms, cudaStream_t s) {
  float* h = static_cast<float*>(a.ws);
  float* z = h + (size_t(p.M) * a.R + 63) / 64 * 64;
  const dim3 down((unsigned(p.M) + kRows - 1) / kRows, (a.R + kCols - 1) / kCols);
  const dim3 up((unsigned(p.M) + kTile - 1) / kTile, (p.O + kTile - 1) / kTile);
  cudaError_t e = launch_overlapped(adapters_f32_down_kernel, down, 32 * kWarps, 0, s, 0, p, a, h);
  if (e == cudaSuccess) e = launch_overlapped(adapters_f32_up_kernel, up, 256, 0, s, 0, p, a, h, z);
  if (e != cudaSuccess) return e;
  LinearParams with = p;
  with.add = z;
  return linear_f32(with, num_sms, s);
}

}  // namespace mcs
