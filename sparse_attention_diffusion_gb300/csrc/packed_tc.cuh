// What the two bf16 kernels of attention over packed sequences share.
#pragma once
#include "packed.h"
#include "ptx.cuh"
#include "tc_common.cuh"
#include "tma.cuh"

namespace mcs {
namespace {

struct PackedWalk {
  Divisor by_tq, by_chunk, by_one;
};

__device__ __forceinline__ bool finite_bf16x2(uint32_t w) {
  return (w & 0x7f80u) != 0x7f80u && (w & 0x7f800000u) != 0x7f800000u;
}
// Both halves, what is not finite as 0.
__device__ __forceinline__ uint32_t finite_part(uint32_t w) {
  if ((w & 0x7f80u) == 0x7f80u) w &= 0xffff0000u;
  if ((w & 0x7f800000u) == 0x7f800000u) w &= 0x0000ffffu;
  return w;
}

// Rows some .. none - 1 of a V tile, which some tokens do not see, with what is not finite as 0, and rows from none
// on, which nobody sees, as 0. Whether there was such an element. Warp `part` of kParts, 16 bytes a lane.
template <int D, int kParts = 1>
__device__ __forceinline__ bool settle_v(uint32_t v, int some, int none, int part, int lane) {
  constexpr int kRowLanes = D / 8, kRows = kParts * 32 / kRowLanes;
  const int ch = lane % kRowLanes, row0 = part * (32 / kRowLanes) + lane / kRowLanes;
  bool found = false;
#pragma unroll 4
  for (int r = some + row0; r < none; r += kRows) {
    const uint32_t at = v + sw128_off(r, ch);
    uint4 w;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w) : "r"(at) : "memory");
    if (!(finite_bf16x2(w.x) && finite_bf16x2(w.y) && finite_bf16x2(w.z) && finite_bf16x2(w.w))) {
      found = true;
      asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(finite_part(w.x)), "r"(finite_part(w.y)),
                   "r"(finite_part(w.z)), "r"(finite_part(w.w))
                   : "memory");
    }
  }
  for (int r = none + row0; r < 128; r += kRows)
    asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(v + sw128_off(r, ch)), "r"(0) : "memory");
  return found;
}

// Scores of keys from nvalid on as -inf, in tensor memory, where a loop can go through the columns: masks of the 128 registers
// of a row would be a third of the softmax's code, and the kernels' instructions already miss their cache.
__device__ __forceinline__ void mask_scores(uint32_t tS, int nvalid) {
#pragma unroll 1
  for (int q = 0; q < 128; q += 32) {
    if (!__any_sync(0xffffffffu, nvalid < q + 32)) continue;
    uint32_t r[32];
    tmem_ld32(tS + q, r);
#pragma unroll
    for (int i = 0; i < 32; ++i) r[i] = nvalid - q > i ? r[i] : __float_as_uint(-INFINITY);
    tmem_st32(tS + q, r);
  }
}

// Tiled map over a [heads, tokens, d] bf16 view, box = 64 columns x box_heads x box_tokens, 128-byte swizzle.
bool make_view_map(CUtensorMap* m, const void* base, int heads, int tokens, int d, const PackedStrides& s, int box_heads, int box_tokens) {
  auto enc = tensor_map_encoder();
  if (enc == nullptr) return false;
  const cuuint64_t dims[3] = {cuuint64_t(d), cuuint64_t(heads), cuuint64_t(tokens)};
  // the stride of a dimension of one is never used
  const cuuint64_t strides[2] = {cuuint64_t(heads > 1 ? s.head : d) * 2, cuuint64_t(tokens > 1 ? s.token : d) * 2};
  const cuuint32_t box[3] = {64, cuuint32_t(box_heads), cuuint32_t(box_tokens)};
  const cuuint32_t estr[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

PackedWalk walk_of(const PackedParams& p) { return {Divisor(p.tq), Divisor(p.chunk > 0 ? p.chunk : 1), Divisor(1)}; }

}  // namespace
}  // namespace mcs
