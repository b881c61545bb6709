// bf16 matrix product with bias, activation, gate and residual in its epilogue
// on the tcgen05 tensor cores:
//   y[m, o] = residual[m, o] + gate[b, o] * act(sum_k x[m, k] w[o, k] + bias[o])
//
// One CTA per 128 x 128 output tile; K in steps of 64 through a ring of TMA
// stages; the accumulator in tensor memory. x may be the attention's output
// [B, heads, N, d]: its tensor map has the heads as the third dimension, so a
// k step is 64 columns of one head and no transposed copy exists.
#include "attn_tc.h"
#include "common.cuh"
#include "linear.h"
#include "linear_epi.cuh"
#include "ptx.cuh"
#include "tc_common.cuh"
#include "tma.cuh"

namespace mcs {
namespace {

constexpr int kStages = 5;
constexpr int kTileThreads = 192;
constexpr int kStageBytes = 2 * kRegion;
constexpr int kBarOff = kStages * kStageBytes;
constexpr int kSmemAlloc = kBarOff + 256 + 1024;

// How the rows of x are cut into tiles: `groups` sections of `rows` rows each
// (one section for token-major x, one per batch for head-major x).
struct RowTiling {
  int rows, tiles;  // rows of a section, tiles of a section
  int head_dim;     // 0: token-major
};

__global__ void __launch_bounds__(kTileThreads, 1)
    linear_tc_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w,
                     const LinearParams p, const RowTiling rt) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kBarOff);
  uint64_t* empty = full + kStages;
  uint64_t* done = empty + kStages;
  uint64_t* drain = done + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int sec = blockIdx.x / rt.tiles, row0 = (blockIdx.x % rt.tiles) * 128, o0 = blockIdx.y * 128;
  const int nk = (p.K + 63) / 64;
  uint32_t* st = p.status;
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) mbar_init(full + s, 1), mbar_init(empty + s, 1);
    mbar_init(done, 1);
    mbar_init(drain, 1);
    fence_mbar_init();
  }
  if (warp == 4) {
    tmem_alloc(tmem_slot, 128);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 5) {
    if (lane == 0) {
      bool ok = true;
      int armed = 0;
      for (int i = 0; i < nk; ++i) {
        const int s = i % kStages;
        if (!(ok = mbar_wait(empty + s, ((i / kStages) & 1) ^ 1, st))) break;
        mbar_arrive_expect_tx(full + s, kStageBytes);
        const int k = i * 64;
        const int c = rt.head_dim ? k % rt.head_dim : k;
        const int z = rt.head_dim ? sec * p.heads + k / rt.head_dim : 0;
        tma_load_3d(sbase + s * kStageBytes, &map_x, c, row0, z, smem_u32(full + s));
        tma_load_3d(sbase + s * kStageBytes + kRegion, &map_w, k, o0, 0, smem_u32(full + s));
        armed = i + 1;
      }
      if (!ok) raise_status(st, kStatusTimeout);
      for (int i = armed > kStages ? armed - kStages : 0; i < armed; ++i)
        mbar_wait(full + i % kStages, (i / kStages) & 1, st);
    }
    __syncwarp();
  } else if (warp == 4) {
    if (lane == 0) {
      constexpr uint32_t kIdesc = idesc_bf16_f32(128, 128, 0, 0);
      bool ok = true, issued = false;
      for (int i = 0; i < nk; ++i) {
        const int s = i % kStages;
        if (!(ok = mbar_wait(full + s, (i / kStages) & 1, st))) break;
        tc_fence_after();
        issued = true;
        const uint32_t a = desc_lo_kmajor(sbase + s * kStageBytes);
        const uint32_t b = desc_lo_kmajor(sbase + s * kStageBytes + kRegion);
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
          tc_mma_ss_lo(tmem, a + kstep_kmajor(ks), b + kstep_kmajor(ks), kIdesc, (i > 0 || ks > 0) ? 1u : 0u);
        tc_commit(empty + s);
      }
      if (ok) {
        tc_commit(done);
      } else {
        raise_status(st, kStatusTimeout);
        if (issued) {
          tc_commit(drain);
          mbar_wait(drain, 0, st);
        }
      }
    }
    __syncwarp();
  } else {
    const bool ok = warp_all(mbar_wait(done, 0, st));
    if (!ok && tid == 0) raise_status(st, kStatusTimeout);
    tc_fence_after();
    const int n = row0 + tid;
    const bool live = ok && n < rt.rows;
    const int m = sec * rt.rows + n;
#pragma unroll 1
    for (int c = 0; c < 128; c += 32) {
      uint32_t r[32];
      tmem_ld32(tmem + (uint32_t(warp * 32) << 16) + c, r);
      if (live) {
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (o0 + c + i < p.O) finish_one<__nv_bfloat16>(p, m, o0 + c + i, __uint_as_float(r[i]));
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 4) {
    tc_fence_after();
    tmem_dealloc(tmem, 128);
  }
}

}  // namespace

cudaError_t linear_tc(const LinearParams& p, int num_sms, cudaStream_t s) {
  (void)num_sms;
  RowTiling rt{};
  CUtensorMap mx, mw;
  bool ok;
  int sections = 1;
  if (p.heads > 0) {
    rt.head_dim = p.K / p.heads;
    rt.rows = p.N;
    sections = p.B;
    ok = make_tile_map(&mx, p.x, uint64_t(p.B) * p.heads, p.N, rt.head_dim, 128);
  } else {
    rt.rows = p.M;
    ok = make_tile_map(&mx, p.x, 1, p.M, p.K, 128);
  }
  ok = ok && make_tile_map(&mw, p.w, 1, p.O, p.K, 128);
  if (!ok) return cudaErrorInvalidValue;
  rt.tiles = (rt.rows + 127) / 128;
  cudaError_t e = cudaFuncSetAttribute(linear_tc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemAlloc);
  if (e != cudaSuccess) return e;
  const dim3 grid(rt.tiles * sections, (p.O + 127) / 128);
  linear_tc_kernel<<<grid, kTileThreads, kSmemAlloc, s>>>(mx, mw, p, rt);
  note_launches(1);
  return cudaGetLastError();
}

}  // namespace mcs
