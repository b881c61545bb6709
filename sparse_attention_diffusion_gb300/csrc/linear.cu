// bf16 matrix product with bias, activation, gate and residual in its epilogue
// on the tcgen05 tensor cores:
//   y[m, o] = residual[m, o] + gate[b, o] * act(sum_k x[m, k] w[o, k] + bias[o])
//
// x may be the attention's output [B, heads, N, d]: its tensor map has the heads
// as the third dimension, so a k step is 64 columns of one head and no transposed
// copy exists.
//
// Many rows: a persistent kernel of CTA pairs (cta_group::2). A pair owns a tile
// of 256 rows x up to 256 outputs: each CTA loads 128 rows of x and half of the
// tile's rows of w, so every operand byte in shared memory feeds two tensor
// cores, which halves the shared-memory and L2 traffic of w against one-CTA
// tiles. 384 threads:
//   warp 0       TMA producer (both CTAs, each its own half), six 64-column stages
//   warp 1       MMA issuer (even CTA only, for both)
//   warp 2       tensor-memory allocation
//   warps 4-11   epilogue: 32 x 32 pieces of the accumulator through a swizzled
//                shared-memory patch, so that bias, gate, residual and the store
//                run along rows, 64 contiguous bytes a row
// The accumulator is double-buffered in tensor memory (2 x 256 columns), so a
// tile's epilogue runs under the next tile's products. Tiles are walked in bands
// of eight row tiles, column by column, which keeps the band's x rows and the
// current columns of w in L2.
#include "attn_tc.h"
#include "common.cuh"
#include "linear.h"
#include "linear_epi.cuh"
#include "ptx.cuh"
#include "tc_common.cuh"
#include "tma.cuh"

namespace mcs {
namespace {

constexpr int kStages = 6;
constexpr int kThreads = 384;
constexpr int kEpiWarps = 8;
constexpr int kHalfTile = 128 * 128;  // bytes of 128 rows x 64 columns
constexpr int kStageBytes = 2 * kHalfTile;
constexpr int kPatchOff = kStages * kStageBytes;
constexpr int kPatch = 32 * 32 * 4;
constexpr int kBarOff = kPatchOff + kEpiWarps * kPatch;
constexpr int kSmemAlloc = kBarOff + 256 + 1024;
constexpr int kBand = 8;

// How the rows of x are cut into tiles: sections of `rows` rows each (one
// section for token-major x, one per batch for head-major x), `tiles` tiles of
// 256 rows a section; columns in `cols` tiles of `bn` outputs.
struct Tiling {
  int rows, tiles, sections;
  int head_dim;  // 0: token-major
  int bn, cols;
  int total;
};
struct Tile {
  int sec, row0, o0;
};
__device__ __forceinline__ Tile tile_at(const Tiling& t, int i) {
  const int nrt = t.tiles * t.sections;
  const int band = i / (kBand * t.cols), rem = i - band * kBand * t.cols;
  const int rows = min(kBand, nrt - band * kBand);
  const int col = rem / rows, rt = band * kBand + rem % rows;
  return {rt / t.tiles, (rt % t.tiles) * 256, col * t.bn};
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    linear_pair_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w,
                       const LinearParams p, const Tiling tl) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kBarOff);  // even CTA: both CTAs' copies of a stage landed
  uint64_t* empty = full + kStages;                              // each CTA: the MMAs of a stage are done
  uint64_t* acc_full = empty + kStages;                          // [2] each CTA: accumulator written
  uint64_t* acc_empty = acc_full + 2;                            // [2] even CTA: accumulator read by both CTAs
  uint64_t* drain = acc_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = int(cluster_rank());
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const int nk = (p.K + 63) / 64;
  uint32_t* st = p.status;
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) mbar_init(full + s, 1), mbar_init(empty + s, 1);
    for (int b = 0; b < 2; ++b) mbar_init(acc_full + b, 1), mbar_init(acc_empty + b, 2 * kEpiWarps);
    mbar_init(drain, 1);
    fence_mbar_init();
  }
  __syncthreads();
  if (warp == 2) {
    tmem_alloc_pair(tmem_slot, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0) {
    if (lane == 0) {
      const int bn2 = tl.bn / 2;
      bool ok = true;
      int u = 0;  // stage uses so far
      for (int t = pair; t < tl.total && ok; t += pairs) {
        const Tile ti = tile_at(tl, t);
        for (int i = 0; i < nk; ++i, ++u) {
          const int s = u % kStages;
          if (!(ok = mbar_wait(empty + s, ((u / kStages) & 1) ^ 1, st))) break;
          if (rank == 0) mbar_arrive_expect_tx(full + s, 2 * (kHalfTile + bn2 * 128));
          const uint32_t bar = cluster_map(smem_u32(full + s), 0);
          const int k = i * 64;
          const int c = tl.head_dim ? k % tl.head_dim : k;
          const int z = tl.head_dim ? ti.sec * p.heads + k / tl.head_dim : 0;
          tma_load_3d_pair(sbase + s * kStageBytes, &map_x, c, ti.row0 + rank * 128, z, bar);
          tma_load_3d_pair(sbase + s * kStageBytes + kHalfTile, &map_w, k, ti.o0 + rank * bn2, 0, bar);
        }
      }
      if (!ok) raise_status(st, kStatusTimeout);
      // let the armed copies of both CTAs land before the pair can exit
      if (rank == 0)
        for (int v = u > kStages ? u - kStages : 0; v < u; ++v) mbar_drain(full + v % kStages, (v / kStages) & 1);
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      const uint32_t idesc = idesc_bf16_f32(256, 0, 0, 0) | (uint32_t(tl.bn >> 3) << 17);
      bool ok = true, issued = false;
      int u = 0, it = 0;
      for (int t = pair; t < tl.total && ok; t += pairs, ++it) {
        const int b = it & 1;
        if (!(ok = mbar_wait(acc_empty + b, ((it >> 1) & 1) ^ 1, st))) break;
        for (int i = 0; i < nk; ++i, ++u) {
          const int s = u % kStages;
          if (!(ok = mbar_wait(full + s, (u / kStages) & 1, st))) break;
          tc_fence_after();
          issued = true;
          const uint32_t a = desc_lo_kmajor(sbase + s * kStageBytes);
          const uint32_t w = desc_lo_kmajor(sbase + s * kStageBytes + kHalfTile);
#pragma unroll
          for (int ks = 0; ks < 4; ++ks)
            tc_mma_ss_lo_pair(tmem + b * 256, a + kstep_kmajor(ks), w + kstep_kmajor(ks), idesc,
                              (i > 0 || ks > 0) ? 1u : 0u);
          tc_commit_pair(empty + s);
        }
        if (ok) tc_commit_pair(acc_full + b);
      }
      if (!ok) {
        raise_status(st, kStatusTimeout);
        if (issued) {
          tc_commit_pair(drain);
          mbar_drain(drain, 0);
        }
      }
    }
    __syncwarp();
  } else if (warp >= 4) {
    const int e = warp - 4, quarter = e & 3, half = e >> 2;
    const uint32_t patch = sbase + kPatchOff + e * kPatch;
    const uint32_t lane_off = uint32_t(quarter * 32) << 16;
    const int prow = lane >> 2, pcol = (lane & 3) * 8;  // this lane's row (of eight) and columns when reading back
    const bool vec = p.O % 8 == 0;
    bool ok = true;
    int it = 0;
    for (int t = pair; t < tl.total; t += pairs, ++it) {
      const int b = it & 1;
      ok = warp_all(mbar_wait(acc_full + b, (it >> 1) & 1, st));
      if (!ok) break;
      tc_fence_after();
      const Tile ti = tile_at(tl, t);
      const int n0 = ti.row0 + rank * 128 + quarter * 32;
      const int m0 = ti.sec * tl.rows + n0;
      const int nchunks = tl.bn / 32;
      if (half >= nchunks) {  // nothing of this accumulator for this warp
        tc_fence_before();
        if (lane == 0) mbar_arrive_cluster(cluster_map(smem_u32(acc_empty + b), 0));
      }
      for (int cc = half; cc < nchunks; cc += 2) {
        const int o = ti.o0 + cc * 32 + pcol;
        uint4 bias8{}, res8[4] = {};
        if (vec && o < p.O) {
          if (p.bias) bias8 = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.bias) + o);
          if (p.residual) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (n0 + i * 8 + prow < tl.rows)
                res8[i] = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.residual) +
                                                          size_t(m0 + i * 8 + prow) * p.O + o);
          }
        }
        uint32_t r[32];
        tmem_ld32(tmem + lane_off + b * 256 + cc * 32, r);
        if (cc + 2 >= nchunks) {  // last read of this accumulator by this warp
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(cluster_map(smem_u32(acc_empty + b), 0));
        }
#pragma unroll
        for (int q = 0; q < 8; ++q)
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(patch + lane * 128 + ((q ^ (lane & 7)) << 4)),
                       "r"(r[4 * q]), "r"(r[4 * q + 1]), "r"(r[4 * q + 2]), "r"(r[4 * q + 3])
                       : "memory");
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int row = i * 8 + prow;
          float v[8];
#pragma unroll
          for (int h = 0; h < 2; ++h)
            asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                         : "=f"(v[4 * h]), "=f"(v[4 * h + 1]), "=f"(v[4 * h + 2]), "=f"(v[4 * h + 3])
                         : "r"(patch + row * 128 + (((pcol / 4 + h) ^ (row & 7)) << 4))
                         : "memory");
          if (n0 + row < tl.rows) {
            if (vec) {
              if (o < p.O) finish_eight(p, m0 + row, o, v, bias8, res8[i]);
            } else {
              for (int j = 0; j < 8; ++j)
                if (o + j < p.O) finish_one<__nv_bfloat16>(p, m0 + row, o + j, v[j]);
            }
          }
        }
        __syncwarp();
      }
    }
    if (!ok && lane == 0) raise_status(st, kStatusTimeout);
  }
  tc_fence_before();
  cluster_sync();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

cudaError_t launch_pair(const LinearParams& p, int num_sms, cudaStream_t s) {
  Tiling t{};
  CUtensorMap mx, mw;
  bool ok;
  if (p.heads > 0) {
    t.head_dim = p.K / p.heads;
    t.rows = p.N;
    t.sections = p.B;
    ok = make_tile_map(&mx, p.x, uint64_t(p.B) * p.heads, p.N, t.head_dim, 128);
  } else {
    t.rows = p.M;
    t.sections = 1;
    ok = make_tile_map(&mx, p.x, 1, p.M, p.K, 128);
  }
  t.tiles = (t.rows + 255) / 256;
  t.cols = (p.O + 255) / 256;
  t.bn = ((p.O + t.cols - 1) / t.cols + 31) / 32 * 32;  // equal column tiles, in steps of 32
  t.cols = (p.O + t.bn - 1) / t.bn;
  const long long total = static_cast<long long>(t.tiles) * t.sections * t.cols;
  if (total > INT32_MAX - 1024) return cudaErrorInvalidValue;
  t.total = int(total);
  ok = ok && make_tile_map(&mw, p.w, 1, p.O, p.K, t.bn / 2);
  if (!ok) return cudaErrorInvalidValue;
  cudaError_t e = cudaFuncSetAttribute(linear_pair_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemAlloc);
  if (e != cudaSuccess) return e;
  const int pairs = t.total < num_sms / 2 ? t.total : num_sms / 2;
  linear_pair_kernel<<<2 * pairs, kThreads, kSmemAlloc, s>>>(mx, mw, p, t);
  note_launches(1);
  return cudaGetLastError();
}

}  // namespace

cudaError_t linear_tc(const LinearParams& p, int num_sms, cudaStream_t s) { return launch_pair(p, num_sms, s); }

}  // namespace mcs
