// Projections with low-rank adapters, fp32: h = scale_a x down_a^T and then z = h up_a^T on the CUDA cores, for the
// fp32 product's epilogue to add to its sums. They compute R / in and R / out of what the product does; the first reads all of x,
// the second writes as much as the product, which reads it back: 4 M in + 8 M out bytes beside the product's 4 M (in + out).
#include "adapters.h"
#include "common.cuh"
#include "launch.cuh"
#include "linear.h"
#include "ptx.cuh"
#include "status.cuh"

namespace mcs {
namespace {

// h = scale_a x down_a^T where many rows share an adapter: 64 rows and kCols columns of h a block, 4 x kCols / 16 a thread, 32 columns
// of x at a time, the next ones on their way meanwhile. Where tiles are few a cluster of `splits` blocks shares K and adds its sums
// through distributed shared memory, ranks in order.
template <int kCols>
__global__ void __launch_bounds__(256) adapters_f32_down_kernel(const LinearParams p, const AdapterParams a, float* h, const int hd, const int splits) {
  constexpr int kRows = 64, kK = 32, kPitch = kK + 4, kJ = kCols / 16;
  __shared__ __align__(16) float xs[kRows][kPitch], ds[kCols][kPitch], part[kRows][kCols + 1];
  const int tid = threadIdx.x, lane = tid & 31, ty = tid >> 4, tx = tid & 15;
  const int tile = blockIdx.x / splits, rank = blockIdx.x - tile * splits;  // of the cluster {splits, 1, 1}
  const long long m0 = static_cast<long long>(tile) * kRows;
  const int nk = (p.K + kK - 1) / kK;
  const int k_beg = int(static_cast<long long>(nk) * rank / splits) * kK, k_end = min(p.K, int(static_cast<long long>(nk) * (rank + 1) / splits) * kK);
  const int c0 = blockIdx.y * kCols;
  grid_inputs_ready();
  grid_let_next_start();
  if (blockIdx.y == 0 && tid < 32) {
    for (long long s = static_cast<long long>(blockIdx.x) * 32 + lane; s < a.S; s += static_cast<long long>(gridDim.x) * 32) {
      int x, y;
      if (!segment_rows(a.start, int(s), p.M, x, y) || a.which[s] >= a.count) raise_status(p.status, kStatusBounds);
    }
  }
  const int m1 = int(min(static_cast<long long>(p.M), m0 + kRows));
  const int row = tid >> 3, q4 = (tid & 7) * 4;  // loads: rows `row` and `row` + 32, four columns from q4 on
  const long long head = static_cast<long long>(p.N) * hd;  // from one head's column to the next head's
  const float* x[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int m = min(int(m0) + row + 32 * i, p.M - 1), b = m / p.N;
    x[i] = static_cast<const float*>(p.x) + (p.heads > 0 ? b * p.heads * head + static_cast<long long>(m - b * p.N) * hd
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
    const float4 none = make_float4(0.f, 0.f, 0.f, 0.f);
    float4 xv[2], dv[2];
    auto fetch = [&](int k0) {
      const int k = k0 + q4, q = p.heads > 0 ? k / hd : 0;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        xv[i] = k < k_end ? *reinterpret_cast<const float4*>(x[i] + (q * head + (k - q * hd))) : none;
        const int c = row + 32 * i;
        dv[i] = k < k_end && c < kCols && c0 + c < a.R ? __ldg(reinterpret_cast<const float4*>(down + static_cast<size_t>(c0 + c) * p.K + k)) : none;
      }
    };
    float acc[4][kJ] = {};
    fetch(k_beg);
    for (int k0 = k_beg; k0 < k_end; k0 += kK) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        *reinterpret_cast<float4*>(&xs[row + 32 * i][q4]) = xv[i];
        if (row + 32 * i < kCols) *reinterpret_cast<float4*>(&ds[row + 32 * i][q4]) = dv[i];
      }
      __syncthreads();
      if (k0 + kK < k_end) fetch(k0 + kK);
#pragma unroll
      for (int k = 0; k < kK; k += 4) {
        float4 u[kJ];
#pragma unroll
        for (int j = 0; j < kJ; ++j) u[j] = *reinterpret_cast<const float4*>(&ds[tx + 16 * j][k]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4 w = *reinterpret_cast<const float4*>(&xs[ty * 4 + i][k]);
#pragma unroll
          for (int j = 0; j < kJ; ++j)
            acc[i][j] = fmaf(w.w, u[j].w, fmaf(w.z, u[j].z, fmaf(w.y, u[j].y, fmaf(w.x, u[j].x, acc[i][j]))));
        }
      }
    }
    const float sc = a.scale[ad];
    if (splits > 1) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < kJ; ++j) part[ty * 4 + i][tx + 16 * j] = acc[i][j];
      cluster_sync();
      for (int e = rank * 256 + tid; e < kRows * kCols; e += splits * 256) {
        const int r = e / kCols, c = e % kCols, m = int(m0) + r;
        float sum = 0.f;
        for (int q = 0; q < splits; ++q) {
          float f;
          asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(f) : "r"(cluster_map(smem_u32(&part[r][c]), q)) : "memory");
          sum += f;
        }
        if (m >= lo && m < hi && c0 + c < a.R) h[static_cast<size_t>(m) * a.R + c0 + c] = sc * sum;
      }
      cluster_sync();  // the sums have been read
      continue;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int m = int(m0) + ty * 4 + i;
      if (m < lo || m >= hi) continue;
#pragma unroll
      for (int j = 0; j < kJ; ++j)
        if (const int c = c0 + tx + 16 * j; c < a.R) h[static_cast<size_t>(m) * a.R + c] = sc * acc[i][j];
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
  const long long M = p.M, S = a.S;
  // Second step row by row, whose threads read `up` again for every row: 70 rows with adapters of their own 31 us in all, 88 by
  // tiles of 64 rows, which go through their segments one by one; 300 rows of 30 segments to 300 outputs 15 and 23.
  const bool single = M <= 4 * S || (M <= 16 * S && M * p.O * a.R <= (16ll << 20));
  // First step by tiles: rows that share adapters, and enough of them, the fewer the higher the rank, as four rows at a time read
  // `down` again for every four (two segments, to 512 outputs, in all, by tiles and four rows at a time: 2,100 x 1,536, rank 16, 44 and 43
  // us, 2,000 x 1,536, rank 32, 55 and 57; rank 64: 1,400 rows 66 and 72, 1,600 68 and 76, of 4,096 columns 136 and 136; rank 128: 700
  // rows of 4,096 columns 124 and 122, 1,000 126 and 148; rank 256: 300 and 400 rows of 4,096 columns 135 and 132, 145 and 157; 74,156 x
  // 128 -> 16, rank 72: 158 and 1,182).
  const bool tiles = !single && M >= 32 * S && (M >= 2048 || M * a.R >= 2048 * 48);
  cudaError_t e;
  if (tiles) {
    auto go = [&](auto kern, int cols) {
      const long long rows = (M + 63) / 64, across = (a.R + cols - 1) / cols;
      // slices until there are eight blocks an SM, of four steps at least (2,482 x 3,200, rank 40: 330 us in all with one, 94 with
      // eight; 5,658 x 3,720, rank 48: 484 with one, 213 with four blocks an SM, 189 with eight)
      int splits = 1;
      while (splits < 8 && rows * across * splits * 2 <= 8ll * num_sms && p.K >= splits * 2 * 4 * 32) splits *= 2;
      return launch_overlapped(kern, dim3(unsigned(rows * splits), unsigned(across)), 256, 0, s, unsigned(splits), p, a, h,
                               p.heads > 0 ? p.K / p.heads : p.K, splits);
    };
    e = a.R <= 16 ? go(adapters_f32_down_kernel<16>, 16) : a.R <= 32 ? go(adapters_f32_down_kernel<32>, 32) : go(adapters_f32_down_kernel<64>, 64);
  } else {
    e = adapters_down_rows(p, a, false, h, of_row, s);
  }
  if (e != cudaSuccess) return e;
  if (single)
    e = launch_overlapped(adapters_f32_up_rows_kernel, dim3(unsigned(p.M), (p.O + 255) / 256), 256, 0, s, 0, p, a, h, of_row, z);
  else
    e = launch_overlapped(adapters_f32_up_kernel, dim3((unsigned(p.M) + kTile - 1) / kTile, (p.O + kTile - 1) / kTile), 256, 0, s, 0, p, a, h, z);
  if (e != cudaSuccess) return e;
  LinearParams with = p;
  with.add = z;
  return linear_f32(with, num_sms, s);
}

}  // namespace mcs
