// Host-side interface of the rotary-position and query/key norm kernels.
#pragma once
#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "divisor.h"

namespace mcs {

// A rope as the kernels use it: pairs per axis, grid lengths and table offsets
// (in (cos, sin) entries).
struct RopeGeom {
  int axes;
  int pairs[3];
  int len[3];
  int toff[3];
  int npairs;   // pairs that turn
  int first;    // first grid token
  int ngrid;    // grid tokens
  Divisor by[3];  // by len
};

struct RopeTableParams {
  RopeGeom g;
  double start[3], scale[3], theta;
  float2* table;
};
cudaError_t rope_table(const RopeTableParams& p, cudaStream_t s);

struct ViewStrides {
  long long b, h, n;  // elements
};

// Streams 0 and 1 are rotated (and normed); stream 2 is copied. A stream whose
// src is null is absent.
struct RotateParams {
  const void* src[3];
  void* dst[3];
  ViewStrides in, out;
  const void* w[2];        // norm weights or null (1)
  float eps;
  const float2* table;
  const int32_t* pos;      // [B, N, axes] or null (grid)
  float sin_sign;          // -1: inverse rotation
  RopeGeom g;
  int B, H, N;
  int heads_per_block;     // set by the launcher
  uint32_t* status;
};
// Rotation alone (norm = false) or norm + rotation + copy of stream 2.
cudaError_t rotate(bool bf16, int d, bool half_style, bool norm, RotateParams p, int num_sms, cudaStream_t s);

// Gradient of norm + rotation. x: forward inputs (view `in`); dy: contiguous
// [B,H,N,d]; dx: written with the view `in`; dw: fp32 [d] or null; partial: fp32
// [blocks][2][d] scratch.
struct NormBwdParams {
  const void* x[2];
  const void* dy[3];
  void* dx[3];
  ViewStrides in;
  const void* w[2];
  float* dw[2];
  float* partial;
  float eps;
  const float2* table;
  const int32_t* pos;
  RopeGeom g;
  int B, H, N;
  int heads_per_unit;      // set by the launcher, with the divisors by its chunks and tiles
  Divisor by_chunks, by_tiles;
  uint32_t* status;
};
// Upper bound of the blocks (rows of `partial`) a backward launch uses.
constexpr int kNormBwdMaxBlocks = 1216;
cudaError_t qk_norm_rope_bwd(bool bf16, int d, bool half_style, const NormBwdParams& p, int num_sms, cudaStream_t s);

}  // namespace mcs
