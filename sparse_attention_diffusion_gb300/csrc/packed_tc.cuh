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

// Whether one of two bf16 numbers is infinite or NaN: adding 1 to an exponent of ones carries into the sign's place.
__device__ __forceinline__ uint32_t odd_bf16x2(uint32_t w) { return ((w & 0x7f807f80u) + 0x00800080u) & 0x80008000u; }
// Both, what is not finite as 0.
__device__ __forceinline__ uint32_t finite_part(uint32_t w) {
  const uint32_t o = odd_bf16x2(w);
  return w & ~((o >> 15 & 0x00010001u) * 0xffffu);
}
// Rows some .. none - 1 of a V tile, which some tokens do not see, with what is not finite as 0, and rows from none
// on, which nobody sees, as 0. Whether there was such an element. Warp `part` of kParts, 16 bytes a lane.
template <int D, int kParts = 1>
__device__ __forceinline__ bool settle_v(uint32_t v, int some, int none, int part, int lane) {
  constexpr int kRowLanes = D / 8, kRows = kParts * 32 / kRowLanes;
  const int ch = lane % kRowLanes, row0 = part * (32 / kRowLanes) + lane / kRowLanes;
  bool found = false;
#pragma unroll 1
  for (int r0 = some + row0; r0 < none; r0 += 4 * kRows) {
    uint4 w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)  // rows from `none` on are overwritten below, where they are looked at here
      asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(w[i].x), "=r"(w[i].y), "=r"(w[i].z), "=r"(w[i].w)
                   : "r"(v + sw128_off(min(r0 + i * kRows, 127), ch))
                   : "memory");
    uint32_t odd = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) odd |= odd_bf16x2(w[i].x) | odd_bf16x2(w[i].y) | odd_bf16x2(w[i].z) | odd_bf16x2(w[i].w);
    if (odd == 0) continue;
#pragma unroll 1
    for (int r = r0; r < min(none, r0 + 4 * kRows); r += kRows) {
      const uint32_t at = v + sw128_off(r, ch);
      uint4 x;
      asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "r"(at) : "memory");
      found |= (odd_bf16x2(x.x) | odd_bf16x2(x.y) | odd_bf16x2(x.z) | odd_bf16x2(x.w)) != 0;
      asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(finite_part(x.x)), "r"(finite_part(x.y)),
                   "r"(finite_part(x.z)), "r"(finite_part(x.w))
                   : "memory");
    }
  }
#pragma unroll 4
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

// Adds to the outputs of a row that lie in a patch row (128 bytes, 16-byte pieces swizzled by `sw`: 32 fp32 sums or 64 bf16
// outputs, of the columns from `col` on) the elements of V that were left out of the products because they are not finite
// and not all rows see them: of the keys all_see .. lim - 1 of the item. An infinity or a NaN stays one, whatever finite numbers
// are added, divided or rounded.
template <bool kF32>
__device__ __forceinline__ void add_unseen(uint32_t patch_row, int sw, const PackedParams& p, const PackedItem& it, int col, int all_see, int lim) {
  const __nv_bfloat16* v = static_cast<const __nv_bfloat16*>(p.v) + static_cast<long long>(it.hk) * p.vs.head + col;
#pragma unroll 1
  for (int j = all_see; j < lim; ++j) {
#pragma unroll 1
    for (int i = 0; i < (kF32 ? 32 : 64); ++i) {
      const float f = __bfloat162float(v[static_cast<long long>(it.k0 + j) * p.vs.token + i]);
      if (isfinite(f)) continue;
      const int byte = i * (kF32 ? 4 : 2);
      const uint32_t at = patch_row + (((byte >> 4) ^ (sw & 7)) << 4) + (byte & 15);
      if constexpr (kF32) {
        float o;
        asm volatile("ld.shared.f32 %0, [%1];" : "=f"(o) : "r"(at) : "memory");
        asm volatile("st.shared.f32 [%0], %1;" ::"r"(at), "f"(o + f) : "memory");
      } else {
        uint16_t o;
        asm volatile("ld.shared.u16 %0, [%1];" : "=h"(o) : "r"(at) : "memory");
        const __nv_bfloat16 sum = __float2bfloat16_rn(__bfloat162float(__ushort_as_bfloat16(o)) + f);
        asm volatile("st.shared.u16 [%0], %1;" ::"r"(at), "h"(__bfloat16_as_ushort(sum)) : "memory");
      }
    }
  }
}

// The items of one block: its own, then those of blocks that have not started yet, which it asks the hardware for, one
// request ahead. One warp; `bar` has a count of one, `slot` is 16 aligned bytes of shared memory.
struct PackedBlocks {
  uint64_t* bar;
  uint32_t slot, answers = 0;
  bool own = true;
  PackedLane sequence;
  __device__ __forceinline__ PackedBlocks(const PackedParams& p, const PackedWalk& wk, int lane, uint64_t* b, uint32_t s) : bar(b), slot(s) {
    ask();
    if (p.S <= 32) sequence = packed_lane(p, wk.by_tq, wk.by_chunk, lane);
  }
  __device__ __forceinline__ void ask() {
    if (elect_one()) {
      mbar_arrive_expect_tx(bar, 16);
      steal_block(slot, bar);
    }
    __syncwarp();
  }
  // The next item that has something to do (tiles -1: none is left). False if a wait ran out.
  __device__ __forceinline__ bool next(const PackedParams& p, const PackedWalk& wk, int lane, PackedItem& it) {
    while (true) {
      int i = int(blockIdx.x);
      if (!own) {
        if (!warp_all(mbar_wait_short(bar, answers++ & 1))) return false;
        i = stolen_block(slot);
        if (i < 0) {
          it.tiles = -1;
          return true;
        }
        fence_proxy_async_smem();  // the answer has been read; the next one may overwrite it
        __syncwarp();
        ask();
      }
      own = false;
      if (const long long s = static_cast<long long>(i) * 32 + lane; s < p.S) {  // there are more items than sequences
        int a, b, c, d;
        if (!packed_sequence(p, int(s), a, b, c, d)) raise_status(p.status, kStatusBounds);
      }
      __syncwarp();
      if (packed_item(p, wk.by_tq, wk.by_chunk, sequence, i, lane, &it)) return true;
    }
  }
};

// The same for kernels whose blocks are numbered up to kBanks: after its own item a block takes the next one of a counter in the
// workspace (dealt out in advance, nine chunks of 5,000 tokens and less over 90,000 keys and less took 3.2 ms instead of 2.8).
struct PackedCounted {
  long long at = blockIdx.x;
  PackedLane sequence;
  __device__ __forceinline__ PackedCounted(const PackedParams& p, const PackedWalk& wk, int lane, uint64_t*, uint32_t) {
    if (p.S <= 32) sequence = packed_lane(p, wk.by_tq, wk.by_chunk, lane);
  }
  __device__ __forceinline__ bool next(const PackedParams& p, const PackedWalk& wk, int lane, PackedItem& it) {
    while (true) {
      const long long i = at;
      if (i >= p.items) {
        it.tiles = -1;
        return true;
      }
      uint32_t taken = 0;
      if (lane == 0) taken = atomicAdd(p.taken, 1u);
      at = static_cast<long long>(gridDim.x) + __shfl_sync(0xffffffffu, taken, 0);
      if (const long long s = i * 32 + lane; s < p.S) {  // there are more items than sequences
        int a, b, c, d;
        if (!packed_sequence(p, int(s), a, b, c, d)) raise_status(p.status, kStatusBounds);
      }
      __syncwarp();
      if (packed_item(p, wk.by_tq, wk.by_chunk, sequence, i, lane, &it)) return true;
    }
  }
};

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
