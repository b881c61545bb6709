// Host-side interface of projections with a low-rank adapter for each segment of rows,
//   y = residual + gate_b * act(x w^T + bias + scale_a (x down_a^T) up_a^T),  a = which[segment of the row],
// and what the kernels of its two steps share.
//
// bf16: a first kernel takes h = scale_a x down_a^T (fp32 sums) and keeps it as two bf16 parts, h = hi + lo to 2^-17,
// in slabs: one for every row tile of the product and every segment in it, zero in the rows that are not the
// segment's. The product then takes a few more k steps a segment, hi up_a^T and lo up_a^T, into the same
// accumulators. slot(tile, segment) = tile + segment is another number for every pair that meets: walking along
// the rows, one of the two rises at every step. Slabs of pairs that do not meet are neither written nor read.
#pragma once
#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "divisor.h"
#include "linear.h"

namespace mcs {

constexpr int kAdapterPieces = 64;  // shares in which an adapter's `up` is looked over (below)

struct AdapterParams {
  const void* down;       // [count, R, K]
  const void* up;         // [count, O, R]
  const float* scale;     // [count]
  const int32_t* start;   // [S + 1]
  const int32_t* which;   // [S]
  int count, R, S;
  void* ws;
};

// Row tiles of the product: sections of `rows` rows each, `tiles` tiles of `height` rows a section.
struct RowTiles {
  int rows, tiles, sections, height;
  Divisor by_rows, by_height, by_tiles;
  RowTiles() = default;
  RowTiles(int r, int s, int h) : rows(r), tiles((r + h - 1) / h), sections(s), height(h), by_rows(r), by_height(h), by_tiles(tiles) {}
#ifdef __CUDACC__
  // The tile of a row, 0 .. rows * sections (that one: the number of tiles).
  __device__ __forceinline__ int of(int row) const {
    const int sec = by_rows.div(row);
    return sec * tiles + by_height.div(row - sec * rows);
  }
  // First row of a tile, and the row behind its last.
  __device__ __forceinline__ int first(int t) const {
    const int sec = by_tiles.div(t);
    return sec * rows + (t - sec * tiles) * height;
  }
  __device__ __forceinline__ int end(int t) const {
    const int sec = by_tiles.div(t);
    return min(sec * rows + (t - sec * tiles + 1) * height, (sec + 1) * rows);
  }
#endif
};

// What the kernels read of the adapters. A zero row of a slab times an element of `up` that is not finite would be
// NaN in another request's row. So the first kernel also looks through the adapters' `up`, each in shares,
// and leaves a byte a share: such an adapter takes one step instead, NaN in its own rows times zeros, which a copy from
// behind w's columns brings (w's own columns may hold infinities, and other requests' rows are 0 in that step).
struct AdapterView {
  const int32_t* start;
  const int32_t* which;
  const uint8_t* odd;     // [S][kAdapterPieces] share of `up` that is not finite
  int count, R, S, M;
  int halves_splits;      // blocks of the first kernel a slab (each takes a share of `up`)
  int more_shares;        // blocks a segment that take nothing else
  RowTiles tiles;
  Divisor by_one;
};
// How a product takes its adapters: as more k steps from the slabs, or, where few rows share one, on the CUDA cores while
// the sums leave, from h as it is: h [M][R] and every row's adapter (negative: none) lie in the workspace then.
enum { kNoAdapters = 0, kAdapterSteps = 1, kAdapterRows = 2 };
template <int kAdapt>
struct AdapterArgs {};
template <>
struct AdapterArgs<kAdapterSteps> {
  CUtensorMap h;      // slabs [2 slot + part][height][R]
  CUtensorMap mask;   // [slot][height][8]: NaN in the segment's rows
  CUtensorMap up;     // [count][O][R]
  AdapterView v;
};
template <>
struct AdapterArgs<kAdapterRows> {
  const float* h;         // [M][R]
  const int32_t* of_row;  // [M]
  const __nv_bfloat16* up;
  int R;
};

size_t adapters_workspace_bytes(const LinearParams& p, const AdapterParams& a, bool bf16);
// First step, bf16: slabs for `t`'s tiles; fills the view and the maps (boxes of `box` slab rows and `wbox` rows of up).
// free_sms: those that the product leaves, which runs beside it.
cudaError_t adapters_down_tc(const LinearParams& p, const AdapterParams& a, const RowTiles& t, int box, int wbox, int num_sms,
                             int free_sms, AdapterArgs<kAdapterSteps>* args, cudaStream_t s);
// First step with rows of their own: h and every row's adapter (of_row may be null).
cudaError_t adapters_down_rows(const LinearParams& p, const AdapterParams& a, bool bf16, float* h, int32_t* of_row, cudaStream_t s);
cudaError_t linear_adapters_tc(const LinearParams& p, const AdapterParams& a, int num_sms, cudaStream_t s);
cudaError_t linear_adapters_f32(const LinearParams& p, const AdapterParams& a, int num_sms, cudaStream_t s);

#ifdef __CUDACC__
// The last s with start[s] <= row, or -1. One warp.
__device__ __forceinline__ int segment_at(const int32_t* start, int S, int row, int lane) {
  int lo = 0, n = S;
  while (true) {
    const int jump = (n + 31) >> 5, at = lane * jump;
    const int c = __popc(__ballot_sync(0xffffffffu, at < n && start[lo + at] <= row));
    if (c == 0) return lo == 0 ? -1 : lo;
    lo += (c - 1) * jump;
    n = min(jump, n - (c - 1) * jump);
    if (jump == 1) return lo;
  }
}
// Rows of segment s, empty where its bounds fall or leave the rows.
__device__ __forceinline__ bool segment_rows(const int32_t* start, int s, int M, int& a, int& b) {
  a = start[s], b = start[s + 1];
  if (a >= 0 && b >= a && b <= M) return true;
  a = b = 0;
  return false;
}
// Shares in which the `up` of a segment over rows a .. b - 1 (not none) is looked over.
__device__ __forceinline__ int up_shares(const AdapterView& v, int a, int b) {
  return min(kAdapterPieces, (v.tiles.of(b - 1) - v.tiles.of(a) + 1) * v.halves_splits + v.more_shares);
}
// Calls f(segment, adapter, odd) for every segment with an adapter in rows row0 .. row1 - 1; one warp, all lanes.
template <typename F>
__device__ __forceinline__ void for_segments(const AdapterView& v, int row0, int row1, int lane, F f) {
  int base = max(0, segment_at(v.start, v.S, row0, lane));
  while (true) {
    const int s = base + lane;
    int a = INT32_MAX, b = 0, ad = -1;
    bool behind = true, odd = false;
    if (s < v.S) {
      behind = v.start[s] >= row1;
      segment_rows(v.start, s, v.M, a, b);
      if (max(a, row0) < min(b, row1)) {
        ad = v.which[s];
        if (ad >= v.count) ad = -1;
        if (ad >= 0) {
          const int n = up_shares(v, a, b);
          const uint4* at = reinterpret_cast<const uint4*>(v.odd + size_t(s) * kAdapterPieces);
          for (int q = 0; q * 16 < n; ++q) {
            const uint4 w = at[q];
            const uint32_t word[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int live = n - (q * 16 + i * 4);  // bytes of this word that are shares
              if (live > 0) odd |= (live >= 4 ? word[i] : word[i] & ((1u << (8 * live)) - 1)) != 0;
            }
          }
        }
      }
    }
    uint32_t todo = __ballot_sync(0xffffffffu, ad >= 0);
    const bool end = __any_sync(0xffffffffu, behind);
    while (todo) {
      const int l = __ffs(todo) - 1;
      todo &= todo - 1;
      f(base + l, __shfl_sync(0xffffffffu, ad, l), __shfl_sync(0xffffffffu, int(odd), l) != 0);
    }
    if (end) return;
    base += 32;
  }
}
#endif

}  // namespace mcs
