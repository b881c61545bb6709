// First step of projections with low-rank adapters on the CUDA cores: h = scale_a x down_a^T in fp32, for fp32 and for
// bf16 rows of which few share an adapter. Reading the adapters bounds it there.
#include "adapters.h"
#include "common.cuh"
#include "launch.cuh"
#include "linear.h"
#include "linear_epi.cuh"
#include "ptx.cuh"
#include "status.cuh"

namespace mcs {
namespace {

constexpr int kCols = 8;

// Elements of a 16-byte load as packed fp32 pairs.
template <typename T>
struct Pairs {
  static constexpr int n = 16 / sizeof(T) / 2;
  uint64_t v[n];
};
__device__ __forceinline__ Pairs<float> pairs16(const float* p) {
  const ulonglong2 w = *reinterpret_cast<const ulonglong2*>(p);
  return {{w.x, w.y}};
}
__device__ __forceinline__ Pairs<__nv_bfloat16> pairs16(const __nv_bfloat16* p) {
  float f[8];
  unpack8(*reinterpret_cast<const uint4*>(p), f);
  return {{f2_pack(f[0], f[1]), f2_pack(f[2], f[3]), f2_pack(f[4], f[5]), f2_pack(f[6], f[7])}};
}

// A block takes kRows rows and 8 columns of h, its warps a share of K each, lanes along K; rows of several
// segments are worked off one segment after another.
template <typename T, int kRows, int kWarps>
__global__ void __launch_bounds__(32 * kWarps) adapters_rows_kernel(const LinearParams p, const AdapterParams a, float* h, int32_t* of_row) {
  __shared__ float part[kWarps][kRows * kCols];
  constexpr int kV = 16 / sizeof(T);
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
  const T* x[kRows];  // row m's columns, by head if they lie so
  const int hd = p.heads > 0 ? p.K / p.heads : p.K;
  const long long head = static_cast<long long>(p.N) * hd;  // from one head's column to the next head's
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    const int m = min(int(m0) + r, p.M - 1), b = m / p.N;
    x[r] = static_cast<const T*>(p.x) + (p.heads > 0 ? b * p.heads * head + static_cast<long long>(m - b * p.N) * hd
                                                     : static_cast<long long>(m) * p.K);
  }
  int mine = -1;  // warp 0 of the first columns' blocks: the adapter of row m0 + lane
  for (int s = max(0, segment_at(a.start, a.S, int(m0), lane)); s < a.S; ++s) {
    if (a.start[s] >= m1) break;
    int ra, rb;
    segment_rows(a.start, s, p.M, ra, rb);
    const int lo = max(ra, int(m0)), hi = min(rb, m1);
    if (lo >= hi) continue;
    const int ad = a.which[s];
    if (ad < 0 || ad >= a.count) continue;
    if (int(m0) + lane >= lo && int(m0) + lane < hi) mine = ad;
    const T* down = static_cast<const T*>(a.down) + static_cast<size_t>(ad) * a.R * p.K;
    uint64_t sum[kRows][kCols] = {};
#pragma unroll 2
    for (int k = (warp * 32 + lane) * kV; k < p.K; k += 32 * kV * kWarps) {
      const int q = p.heads > 0 ? k / hd : 0;
      Pairs<T> xv[kRows];
#pragma unroll
      for (int r = 0; r < kRows; ++r) xv[r] = pairs16(x[r] + (q * head + (k - q * hd)));
#pragma unroll
      for (int c = 0; c < kCols; ++c) {  // columns past the last are not written
        const Pairs<T> dv = pairs16(down + static_cast<size_t>(min(c0 + c, a.R - 1)) * p.K + k);
#pragma unroll
        for (int r = 0; r < kRows; ++r)
#pragma unroll
          for (int i = 0; i < Pairs<T>::n; ++i) sum[r][c] = f2_fma(xv[r].v[i], dv.v[i], sum[r][c]);
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
    if (warp == 0 && lane < kRows * kCols) {
      const int r = lane / kCols, c = lane % kCols, m = int(m0) + r;
      float e = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) e += part[w][lane];
      if (m >= lo && m < hi && c0 + c < a.R) h[static_cast<size_t>(m) * a.R + c0 + c] = a.scale[ad] * e;
    }
  }
  if (of_row != nullptr && blockIdx.y == 0 && warp == 0 && lane < kRows && m0 + lane < p.M) of_row[m0 + lane] = mine;
}

}  // namespace

cudaError_t adapters_down_rows(const LinearParams& p, const AdapterParams& a, bool bf16, float* h, int32_t* of_row, cudaStream_t s) {
  auto go = [&](auto kern, int rows, int warps) {
    const dim3 grid((unsigned(p.M) + rows - 1) / rows, (a.R + kCols - 1) / kCols);
    return launch_overlapped(kern, grid, 32 * warps, 0, s, 0, p, a, h, of_row);
  };
  // a row a block where no two rows share a segment to speak of
  const bool single = p.M <= 2ll * a.S;
  if (bf16) return single ? go(adapters_rows_kernel<__nv_bfloat16, 1, 8>, 1, 8) : go(adapters_rows_kernel<__nv_bfloat16, 4, 4>, 4, 4);
  return single ? go(adapters_rows_kernel<float, 1, 8>, 1, 8) : go(adapters_rows_kernel<float, 4, 4>, 4, 4);
}

}  // namespace mcs
