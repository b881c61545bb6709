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
//   warp 0       TMA producer (both CTAs, each its own half), six or more 64-column
//                stages
//   warp 1       MMA issuer (even CTA only, for both)
//   warp 2       tensor-memory allocation
//   warps 4-11   epilogue: 32 x 32 pieces of the accumulator, a row per lane; the
//                residual arrives in a swizzled shared-memory patch by TMA one
//                piece ahead, the result leaves through the same patch by TMA, so
//                no lane touches rows of x's or y's stride (outputs whose row is
//                no multiple of 16 bytes go through the patch in fp32 and leave by
//                plain stores along the row)
// The accumulator is double-buffered in tensor memory (2 x 256 columns), so a
// tile's epilogue runs under the next tile's products. A long row takes several
// accumulators (linear.h), which the epilogue's warps sum in registers meanwhile: 128 of
// them a thread, for which the other warps hand registers over (without that some are
// spilled, and reloads from local memory beside the copies held the next tile up: 75,600 x
// 5,120 -> 5,120 with gated residual 2.50 ms instead of 2.33). Tiles are walked in bands
// of eight row tiles, column by column, which keeps the band's x rows and the
// current columns of w in L2.
//
// Measured: 32,768 x 1,536 -> 4,608 outputs 237 us alone (1,954 TFLOP/s, tensor pipe
// 93 % active) and 276 us back to back under the power cap (1,680); 75,600 x 5,120 ->
// 5,120 from heads with gated residual 2.34 ms (1,696). A k step of 256 columns needs
// 64 bytes per clock and SM of operands, about what an SM takes in (62 measured), so
// the tensor pipe and the operand port run out together; tiles of 128 x 128 on single
// CTAs (twice the bytes per FLOP), without epilogue overlap, took 2,423 us and 10.9 ms.
#pragma once
#include "adapters.h"
#include "attn_tc.h"
#include "common.cuh"
#include "divisor.h"
#include "linear.h"
#include "linear_epi.cuh"
#include "launch.cuh"
#include "linear_few.h"
#include "ptx.cuh"
#include "tc_common.cuh"
#include "tma.cuh"

namespace mcs {
namespace {

constexpr int kMaxStages = 9;
constexpr int kThreads = 384;
constexpr int kEpiWarps = 8;
// Registers a thread of the long-row kernels: all warps start with kLaunchRegs; the control warps' go to the
// epilogue's, which hold 128 sums.
constexpr int kLaunchRegs = 168, kControlRegs = 56, kEpiRegs = 224;
static_assert(128 * kControlRegs + 32 * kEpiWarps * kEpiRegs <= kThreads * kLaunchRegs, "an increase would wait forever");
constexpr int kHalfTile = 128 * 128;      // bytes of 128 rows x 64 columns
constexpr int kRing = 6 * 2 * kHalfTile;  // six stages of the widest tile, more of narrower ones
constexpr int kPatchOff = kRing;
constexpr int kPatch = 32 * 32 * 4;       // two bf16 pieces, or one in fp32
constexpr int kBarOff = kPatchOff + kEpiWarps * kPatch;
constexpr int kSmemAlloc = kBarOff + 512 + 1024;
constexpr int kBand = 8;

// How the rows of x are cut into tiles: sections of `rows` rows each (one
// section for token-major x, one per batch for head-major x), `tiles` tiles of
// 256 rows a section; columns in `cols` tiles of `bn` outputs.
struct Tiling {
  int rows, tiles, sections;
  int col_mask, head_shift;  // column k of x is column k & col_mask of head k >> head_shift (token-major: one head)
  int bn, cols;
  int stages, stage_bytes;
  int total;
  Divisor by_band, by_tail, by_tiles, by_batch;  // by kBand * cols, the last band's rows, tiles, rows of a batch
};
struct Tile {
  int sec, row0, o0;
};
__device__ __forceinline__ Tile tile_at(const Tiling& t, int i) {
  const int band = t.by_band.div(i), rem = i - band * kBand * t.cols;
  const int rows = min(kBand, t.tiles * t.sections - band * kBand);
  const int col = rows == kBand ? rem / kBand : t.by_tail.div(rem);
  const int rt = band * kBand + rem - col * rows, sec = t.by_tiles.div(rt);
  return {sec, (rt - sec * t.tiles) * 256, col * t.bn};
}

// The number of a tile's row tile, over all sections.
__device__ __forceinline__ int row_tile(const Tiling& t, int i) {
  const int band = t.by_band.div(i), rem = i - band * kBand * t.cols;
  const int rows = min(kBand, t.tiles * t.sections - band * kBand);
  return band * kBand + rem - (rows == kBand ? rem / kBand : t.by_tail.div(rem)) * rows;
}

// Values o .. o + 31 of a bf16 row of `len`, a multiple of 8 (16-byte aligned at o); 0 past its end.
struct Words32 {
  uint4 w[4];
};
__device__ __forceinline__ Words32 row32(const __nv_bfloat16* row, int o, int len) {
  Words32 r;
#pragma unroll
  for (int q = 0; q < 4; ++q) r.w[q] = o + 8 * q < len ? *reinterpret_cast<const uint4*>(row + o + 8 * q) : uint4{};
  return r;
}
// Adds 32 columns of tensor memory to fp32 sums.
__device__ __forceinline__ void add_tmem32(uint32_t at, float (&v)[32]) {
  uint32_t r[32];
  tmem_ld32(at, r);
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] += __uint_as_float(r[i]);
}
__device__ __forceinline__ void get_tmem32(uint32_t at, float (&v)[32]) {
  uint32_t r[32];
  tmem_ld32(at, r);
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void put_tmem32(uint32_t at, const float (&v)[32]) {  // complete after tmem_wait_st
  uint32_t r[32];
#pragma unroll
  for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(v[i]);
  tmem_st32_nowait(at, r);
}
// Address of a 16-byte piece of a patch row (rows of 64 bytes; with 128-byte rows and one
// ring stage less for the room, the epilogue took the same time and the products longer).
__device__ __forceinline__ uint32_t piece_at(uint32_t patch, int row, int q) {
  return patch + row * 64 + ((q ^ ((row >> 1) & 3)) << 4);
}

// A 32 x 32 piece of outputs whose rows are no multiple of 16 bytes: through the
// patch in fp32, then along rows, one output a lane (two where the rows allow
// 4-byte stores).
template <int kAct>
__device__ __forceinline__ void store_odd(const LinearParams& p, int rows, int sec, int n0, int o, uint32_t patch,
                                          int lane, const float (&r)[32]) {
#pragma unroll
  for (int q = 0; q < 8; ++q)
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(patch + lane * 128 + ((q ^ (lane & 7)) << 4)),
                 "f"(r[4 * q]), "f"(r[4 * q + 1]), "f"(r[4 * q + 2]), "f"(r[4 * q + 3])
                 : "memory");
  __syncwarp();
  auto sum = [&](int row, int c) {
    float f;
    asm volatile("ld.shared.f32 %0, [%1];"
                 : "=f"(f)
                 : "r"(patch + row * 128 + (((c >> 2) ^ (row & 7)) << 4) + (c & 3) * 4));
    return f;
  };
  const __nv_bfloat16* bias = static_cast<const __nv_bfloat16*>(p.bias);
  const __nv_bfloat16* gate = static_cast<const __nv_bfloat16*>(p.gate);
  const __nv_bfloat16* res = static_cast<const __nv_bfloat16*>(p.residual);
  __nv_bfloat16* y = static_cast<__nv_bfloat16*>(p.y);
  const int live = min(32, rows - n0), cols = min(32, p.O - o);
  if (p.O % 2 == 0) {
    const int c = (lane & 15) * 2;
    if (c < cols) {  // cols is even
      const float2 bs = bias ? __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(bias + o + c)) : make_float2(0, 0);
#pragma unroll 4
      for (int row = lane >> 4; row < live; row += 2) {
        const int m = sec * rows + n0 + row;
        const size_t at = size_t(m) * p.O + o + c;
        float v[2] = {sum(row, c) + bs.x, sum(row, c + 1) + bs.y};
        activate<kAct>(v);
        if (gate) {
          const float2 g = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(gate + size_t(m / p.N) * p.O + o + c));
          v[0] *= g.x, v[1] *= g.y;
        }
        if (res) {
          const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(res + at));
          v[0] += f.x, v[1] += f.y;
        }
        *reinterpret_cast<uint32_t*>(y + at) = pack_bf16x2(v[0], v[1]);
      }
    }
  } else if (lane < cols) {
    const float bs = bias ? __bfloat162float(bias[o + lane]) : 0.f;
#pragma unroll 4
    for (int row = 0; row < live; ++row) {
      const int m = sec * rows + n0 + row;
      const size_t at = size_t(m) * p.O + o + lane;
      float v[1] = {sum(row, lane) + bs};
      activate<kAct>(v);
      if (gate) v[0] *= __bfloat162float(gate[size_t(m / p.N) * p.O + o + lane]);
      if (res) v[0] += __bfloat162float(res[at]);
      y[at] = __float2bfloat16_rn(v[0]);
    }
  }
  __syncwarp();
}

// kPieces: 0 for rows of one accumulator; otherwise the pieces of 32 columns that a warp sums in registers, 3 or 4
// (tiles of up to 192 and 256 columns). kBack: how long rows leave. With one tile a pair the sums go back to tensor
// memory, which keeps the way out's code short (452 x 4,096 -> 5,120 18.8 us against 19.9); with more tiles that
// would keep the next tile's second accumulator waiting (75,600 x 5,120 -> 5,120 with gated residual 2.42 ms against
// 2.33).
// kAdapt: the segments of a tile with an adapter add their k steps after those of w, into the row's last accumulator
// (adapters.h); the producers leave a word a stage that says how many 16-column products it takes and whether it is
// the tile's last. Only they wait for the kernel before, which makes the slabs, and only when they come to them; x and w are
// there (launch.cuh, the second kernel of a pair).
template <int kAct, int kPieces, bool kBack, int kAdapt>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    linear_pair_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w,
                       const __grid_constant__ CUtensorMap map_y, const __grid_constant__ CUtensorMap map_r,
                       const __grid_constant__ AdapterArgs<kAdapt> ad, const LinearParams p, const Tiling tl) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kBarOff);  // even CTA: both CTAs' copies of a stage landed
  uint64_t* empty = full + kMaxStages;                           // each CTA: the MMAs of a stage are done
  uint64_t* acc_full = empty + kMaxStages;                       // [2] each CTA: accumulator written
  uint64_t* acc_empty = acc_full + 2;                            // [2] even CTA: accumulator read by both CTAs
  uint64_t* drain = acc_empty + 2;
  uint64_t* res_full = drain + 1;                                // [epilogue warp][2] residual piece landed
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(res_full + 2 * kEpiWarps);
  [[maybe_unused]] volatile uint32_t* stage_info = tmem_slot + 1;  // [kMaxStages]
  constexpr bool kLong = kPieces > 0;
  const int tid = threadIdx.x, warp = warp_uniform(tid >> 5), lane = tid & 31;
  const int rank = blockIdx.x & 1;  // of the cluster {2, 1, 1}
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const int nk = (p.K + 63) / 64;
  uint32_t* st = p.status;
  if (tid == 32) {
    tma_prefetch_map(&map_x);
    tma_prefetch_map(&map_w);
    if (p.O % 8 == 0) tma_prefetch_map(&map_y);
    if (p.O % 8 == 0 && p.residual) tma_prefetch_map(&map_r);
  }
  if (tid == 0) {
    for (int s = 0; s < tl.stages; ++s) mbar_init(full + s, 1), mbar_init(empty + s, 1);
    for (int b = 0; b < 2; ++b) mbar_init(acc_full + b, 1), mbar_init(acc_empty + b, 2 * kEpiWarps);
    mbar_init(drain, 1);
    for (int e = 0; e < 2 * kEpiWarps; ++e) mbar_init(res_full + e, 1);
    fence_mbar_init();
  }
  if (warp == 2) {
    tmem_alloc_pair(tmem_slot, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = warp_uniform(*tmem_slot);
  if constexpr (!kAdapt) {
    grid_inputs_ready();
    grid_let_next_start();
  }

  if (warp < 4) {
    if constexpr (kLong) registers_down<kControlRegs>();
    if (warp == 0) {
      const int bn2 = tl.bn / 2;
      const uint32_t bytes = uint32_t(2 * (kHalfTile + bn2 * 128));
      bool ok = true;
      int s = 0;
      uint32_t phase = 0;
      for (int t = pair; t < tl.total && ok; t += pairs) {
        const Tile ti = tile_at(tl, t);
        const int xrow = ti.row0 + rank * 128, wrow = ti.o0 + rank * bn2, z0 = ti.sec * p.heads;
        // one stage: 64 columns of two maps, `info` for the MMA warp
        auto load = [&](const CUtensorMap* ma, int ca, int ra, int za, const CUtensorMap* mb, int cb, int zb, uint32_t info) {
          if (!(ok = warp_all(mbar_wait(empty + s, phase ^ 1, st)))) return;
          const uint32_t bar = cluster_map(smem_u32(full + s), 0);
          const uint32_t dst = sbase + s * tl.stage_bytes;
          if (elect_one()) {
            if (kAdapt && rank == 0) stage_info[s] = info;
            if (rank == 0) mbar_arrive_expect_tx(full + s, bytes);
            tma_load_3d_pair(dst, ma, ca, ra, za, bar);
            tma_load_3d_pair(dst + kHalfTile, mb, cb, wrow, zb, bar);
          }
          __syncwarp();
          if (++s == tl.stages) s = 0, phase ^= 1;
        };
        if constexpr (kAdapt) {
          const int rt = row_tile(tl, t), row0 = ad.v.tiles.first(rt), row1 = ad.v.tiles.end(rt);
          const int chunks = (ad.v.R + 63) / 64;
          int more = 0;
          for (int i = 0; i < nk && ok; ++i) {
            const int k = i * 64;
            if (i == nk - 1) {
              if (t == pair) {
                grid_inputs_ready();
                grid_let_next_start();
              }
              for_segments(ad.v, row0, row1, lane, [&](int, int, bool odd) { more += odd ? 1 : 2 * chunks; });
            }
            load(&map_x, k & tl.col_mask, xrow, z0 + (k >> tl.head_shift), &map_w, k, 0, 4 | (more == 0 && i == nk - 1 ? 8 : 0));
          }
          for_segments(ad.v, row0, row1, lane, [&](int seg, int which, bool odd) {
            if (odd) {
              --more;
              if (ok) load(&ad.mask, 0, rank * 128, rt + seg, &map_w, nk * 64, 0, 1 | (more == 0 ? 8 : 0));  // zeros behind w's columns
              return;
            }
            for (int c = 0; c < 2 * chunks; ++c) {
              const int col = (c >> 1) * 64;
              --more;
              if (ok) load(&ad.h, col, rank * 128, 2 * (rt + seg) + (c & 1), &ad.up, col, which, (min(64, ad.v.R - col) + 15) / 16 | (more == 0 ? 8 : 0));
            }
          });
        } else {
          for (int i = 0; i < nk && ok; ++i) {
            const int k = i * 64;
            load(&map_x, k & tl.col_mask, xrow, z0 + (k >> tl.head_shift), &map_w, k, 0, 0);
          }
        }
      }
      if (!ok) {
        if (lane == 0) raise_status(st, kStatusTimeout);
        settle_copies();  // normally the MMAs have consumed every copy before the pair exits
      }
      __syncwarp();
    } else if (warp == 1) {
      if (rank == 0) {
        const uint32_t idesc = idesc_bf16_f32(256, 0, 0, 0) | (uint32_t(tl.bn >> 3) << 17);
        bool ok = true, issued = false;
        int s = 0, it = 0, b = 0;  // ring stage, accumulators begun, the current one's buffer
        uint32_t phase = 0;
        for (int t = pair; t < tl.total && ok; t += pairs) {
          for (int i = 0; kAdapt || i < nk; ++i) {
            const bool extra = kAdapt && i >= nk;  // into the accumulator that is there
            const int step = extra ? 1 : kLong ? i % kAccSteps : i;
            if (step == 0) {
              b = it & 1;
              if (!(ok = warp_all(mbar_wait(acc_empty + b, ((it++ >> 1) & 1) ^ 1, st)))) break;
            }
            if (!(ok = warp_all(mbar_wait(full + s, phase, st)))) break;
            tc_fence_after();
            issued = true;
            const uint32_t info = kAdapt ? warp_uniform(stage_info[s]) : 4u;
            const bool last = kAdapt ? (info & 8) != 0 : i == nk - 1;
            const uint32_t a = desc_lo_kmajor(sbase + s * tl.stage_bytes);
            const uint32_t w = desc_lo_kmajor(sbase + s * tl.stage_bytes + kHalfTile);
            if (elect_one()) {
#pragma unroll
              for (int ks = 0; ks < 4; ++ks)
                if (!kAdapt || ks < int(info & 7))
                  tc_mma_ss_lo_pair(tmem + b * 256, a + kstep_kmajor(ks), w + kstep_kmajor(ks), idesc,
                                    (step > 0 || ks > 0) ? 1u : 0u);
              tc_commit_pair(empty + s);
              if ((kLong && !extra && step == kAccSteps - 1 && i < nk - 1) || last) tc_commit_pair(acc_full + b);
            }
            __syncwarp();
            if (++s == tl.stages) s = 0, phase ^= 1;
            if (last) break;
          }
        }
        if (!ok) {
          if (lane == 0) raise_status(st, kStatusTimeout);
          if (issued) {
            if (elect_one()) tc_commit_pair(drain);
            __syncwarp();
            mbar_drain(drain, 0);
          }
          settle_copies();
        }
      }
      __syncwarp();
    }
  } else {
    if constexpr (kLong) registers_up<kEpiRegs>();
    const int e = warp - 4, quarter = e & 3, half = e >> 2;
    const uint32_t patch = sbase + kPatchOff + e * kPatch;
    const uint32_t lane_off = uint32_t(quarter * 32) << 16;
    const int nchunks = tl.bn / 32;
    const bool vec = p.O % 8 == 0, add = vec && p.residual != nullptr;
    const __nv_bfloat16 *bias = static_cast<const __nv_bfloat16*>(p.bias), *gate = static_cast<const __nv_bfloat16*>(p.gate);
    uint64_t* rbar = res_full + 2 * e;
    bool ok = true;
    int it = 0, buf = 0;      // tile and patch buffer
    uint32_t rphase = 0;      // bit b: parity of the next residual piece in buffer b
    uint32_t awaited = 0;     // bit b: a residual piece is on its way to buffer b
    // starts the copy of the residual piece (tile t, chunk cc) into buffer b, whose last store has to be read out
    auto fetch = [&](const Tile& ti, int cc, int b) {
      const int n0 = ti.row0 + rank * 128 + quarter * 32, o = ti.o0 + cc * 32;
      if (n0 >= tl.rows || o >= p.O) return;
      if (elect_one()) {
        bulk_wait_read<0>();
        mbar_arrive_expect_tx(rbar + b, kPatch / 2);
        tma_load_3d(patch + b * (kPatch / 2), &map_r, o, n0, ti.sec, smem_u32(rbar + b));
      }
      __syncwarp();
      awaited |= 1u << b;
    };
    if (add && pair < tl.total && half < nchunks) fetch(tile_at(tl, pair), half, 0);
    for (int t = pair; t < tl.total; t += pairs, ++it) {
      [[maybe_unused]] float sum[kLong ? kPieces : 1][32];
      if constexpr (kLong) {
        // The accumulators of the row are summed in registers. With kBack the sums go back over the last one, from
        // where they leave as those of a short row do; otherwise its columns are the next tile's at once, and the
        // pieces move up in registers.
        for (int i = 0;; i += kAccSteps, ++it) {
          const int b = it & 1;
          const bool last = i + kAccSteps >= nk;
          if (!(ok = warp_all(mbar_wait(acc_full + b, (it >> 1) & 1, st)))) break;
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < kPieces; ++c) {
            if (half + 2 * c >= nchunks) continue;
            const uint32_t at = tmem + lane_off + b * 256 + (half + 2 * c) * 32;
            if (i == 0) get_tmem32(at, sum[c]);
            else add_tmem32(at, sum[c]);
            if (kBack && last) put_tmem32(at, sum[c]);
          }
          if (kBack && last) {
            tmem_wait_st();
            break;
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster_relaxed(cluster_map(smem_u32(acc_empty + b), 0));
          if (last) break;
        }
        if (!ok) break;
      }
      const int b = it & 1;
      constexpr bool kHeld = !kLong || kBack;  // the accumulator is still to be read
      if (half >= nchunks) {             // nothing of it for this warp
        if (!kLong && !(ok = warp_all(mbar_wait(acc_full + b, (it >> 1) & 1, st)))) break;
        if (kHeld && lane == 0) mbar_arrive_cluster_relaxed(cluster_map(smem_u32(acc_empty + b), 0));
        continue;
      }
      const Tile ti = tile_at(tl, t);
      const int n0 = ti.row0 + rank * 128 + quarter * 32;
      const int n = n0 + lane, m = ti.sec * tl.rows + n;  // this lane's row
      const __nv_bfloat16* grow = gate ? gate + size_t(n < tl.rows ? tl.by_batch.div(m) : 0) * p.O : nullptr;
      Words32 bw, gw;  // the current piece's bias and gate
      auto read_rows = [&](int cc) {
        const int o = ti.o0 + cc * 32;
        if (vec && bias) bw = row32(bias, o, p.O);
        if (vec && grow) gw = row32(grow, o, p.O);
      };
      read_rows(half);
#pragma unroll 1
      for (int cc = half; cc < nchunks; cc += 2) {
        const int o = ti.o0 + cc * 32;
        const bool live = n0 < tl.rows && o < p.O;  // the piece has outputs
        if (add) {  // the next piece's residual, while this one is worked on
          if (cc + 2 < nchunks) fetch(ti, cc + 2, buf ^ 1);
          else if (t + pairs < tl.total) fetch(tile_at(tl, t + pairs), half, buf ^ 1);
        }
        if (!kLong && cc == half && !(ok = warp_all(mbar_wait(acc_full + b, (it >> 1) & 1, st)))) break;
        tc_fence_after();
        float v[32];
        if constexpr (kHeld) {
          get_tmem32(tmem + lane_off + b * 256 + cc * 32, v);
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            v[i] = sum[0][i];
#pragma unroll
            for (int c = 1; c < kPieces; ++c) sum[c - 1][i] = sum[c][i];
          }
        }
        if (kHeld && cc + 2 >= nchunks) {  // last read of this accumulator by this warp
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster_relaxed(cluster_map(smem_u32(acc_empty + b), 0));
        }
        if (!vec) {
          if (live) store_odd<kAct>(p, tl.rows, ti.sec, n0, o, patch, lane, v);
          continue;
        }
        if (!live) {  // pieces take the two buffers in turn, each with its bulk group, an empty one here
          if (elect_one()) bulk_commit();
          __syncwarp();
          buf ^= 1;
          continue;
        }
        if (bias) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            float t8[8];
            unpack8(bw.w[q], t8);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[8 * q + i] += t8[i];
          }
        }
        activate<kAct>(v);
        if (grow) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            float t8[8];
            unpack8(gw.w[q], t8);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[8 * q + i] *= t8[i];
          }
        }
        if (cc + 2 < nchunks) read_rows(cc + 2);  // arrive while this piece leaves
        const uint32_t piece = patch + buf * (kPatch / 2);
        if (add) {
          if (!(ok = warp_all(mbar_wait(rbar + buf, (rphase >> buf) & 1, st)))) break;
          rphase ^= 1u << buf;
          awaited &= ~(1u << buf);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint4 w;
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
                         : "r"(piece_at(piece, lane, q)));
            float t8[8];
            unpack8(w, t8);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[8 * q + i] += t8[i];
          }
        } else {
          if (elect_one()) bulk_wait_read<1>();  // the store before the last one used this buffer
          __syncwarp();
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) w[i] = pack_bf16x2(v[8 * q + 2 * i], v[8 * q + 2 * i + 1]);
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(piece_at(piece, lane, q)), "r"(w[0]), "r"(w[1]),
                       "r"(w[2]), "r"(w[3])
                       : "memory");
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (elect_one()) {
          tma_store_3d(&map_y, piece, o, n0, ti.sec);
          bulk_commit();
        }
        __syncwarp();
        buf ^= 1;
      }
      if (!ok) break;
    }
    if (!ok && awaited) settle_copies();
    if (elect_one()) bulk_wait_all();
    __syncwarp();
    if (!ok && lane == 0) raise_status(st, kStatusTimeout);
  }
  tc_fence_before();
  cluster_sync();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

template <int kAct, int kAdapt>
cudaError_t start_pair(const CUtensorMap& mx, const CUtensorMap& mw, const CUtensorMap& my, const CUtensorMap& mr,
                       const AdapterArgs<kAdapt>& ad, const LinearParams& p, const Tiling& t, int pairs, cudaStream_t s) {
  auto start = [&](auto kern, cudaError_t e) {
    return e != cudaSuccess ? e : launch_overlapped(kern, dim3(2 * pairs), kThreads, kSmemAlloc, s, 0, mx, mw, my, mr, ad, p, t);
  };
  if (p.K <= 64 * kOneAccSteps)
    return start(linear_pair_kernel<kAct, 0, false, kAdapt>, allow_smem<linear_pair_kernel<kAct, 0, false, kAdapt>>(kSmemAlloc));
  const bool one = t.total <= pairs;
  if (t.bn <= 192)
    return one ? start(linear_pair_kernel<kAct, 3, true, kAdapt>, allow_smem_and_regs<linear_pair_kernel<kAct, 3, true, kAdapt>>(kSmemAlloc, kLaunchRegs))
               : start(linear_pair_kernel<kAct, 3, false, kAdapt>, allow_smem_and_regs<linear_pair_kernel<kAct, 3, false, kAdapt>>(kSmemAlloc, kLaunchRegs));
  return one ? start(linear_pair_kernel<kAct, 4, true, kAdapt>, allow_smem_and_regs<linear_pair_kernel<kAct, 4, true, kAdapt>>(kSmemAlloc, kLaunchRegs))
             : start(linear_pair_kernel<kAct, 4, false, kAdapt>, allow_smem_and_regs<linear_pair_kernel<kAct, 4, false, kAdapt>>(kSmemAlloc, kLaunchRegs));
}

// adapters: null without adapters.
template <int kAdapt>
cudaError_t launch_pair(const LinearParams& p, int bn, const AdapterParams* adapters, int num_sms, cudaStream_t s) {
  Tiling t{};
  CUtensorMap mx, mw, my{}, mr{};
  bool ok;
  if (p.heads > 0) {
    const int d = p.K / p.heads;
    t.head_shift = d == 64 ? 6 : 7;
    t.col_mask = d - 1;
    t.rows = p.N;
    t.sections = p.B;
    ok = make_tile_map(&mx, p.x, uint64_t(p.B) * p.heads, p.N, d, 128);
  } else {
    t.head_shift = 31;
    t.col_mask = INT32_MAX;
    t.rows = p.M;
    t.sections = 1;
    ok = make_tile_map(&mx, p.x, 1, p.M, p.K, 128);
  }
  t.tiles = (t.rows + 255) / 256;
  t.bn = bn;
  t.cols = (p.O + t.bn - 1) / t.bn;
  t.stage_bytes = kHalfTile + t.bn / 2 * 128;
  t.stages = kRing / t.stage_bytes < kMaxStages ? kRing / t.stage_bytes : kMaxStages;
  const long long total = static_cast<long long>(t.tiles) * t.sections * t.cols;
  if (total > INT32_MAX - 1024) return cudaErrorInvalidValue;
  t.total = int(total);
  const int tail = t.tiles * t.sections % kBand;
  t.by_band = Divisor(kBand * t.cols);
  t.by_tail = Divisor(tail > 0 ? tail : kBand);
  t.by_tiles = Divisor(t.tiles);
  t.by_batch = Divisor(p.N);
  ok = ok && make_tile_map(&mw, p.w, 1, p.O, p.K, t.bn / 2);
  if (p.O % 8 == 0) {  // otherwise the epilogue does not use them
    ok = ok && make_patch_map(&my, p.y, t.sections, t.rows, p.O);
    if (p.residual) ok = ok && make_patch_map(&mr, p.residual, t.sections, t.rows, p.O);
  }
  if (!ok) return cudaErrorInvalidValue;
  const int pairs = t.total < num_sms / 2 ? t.total : num_sms / 2;
  AdapterArgs<kAdapt> ad{};
  if constexpr (kAdapt) {
    const cudaError_t e = adapters_down_tc(p, *adapters, RowTiles(t.rows, t.sections, 256), 128, t.bn / 2, num_sms, num_sms - 2 * pairs, &ad, s);
    if (e != cudaSuccess) return e;
  }
  switch (p.act) {
    case MCS_ACT_GELU_TANH: return start_pair<MCS_ACT_GELU_TANH>(mx, mw, my, mr, ad, p, t, pairs, s);
    case MCS_ACT_GELU_ERF: return start_pair<MCS_ACT_GELU_ERF>(mx, mw, my, mr, ad, p, t, pairs, s);
    case MCS_ACT_SILU: return start_pair<MCS_ACT_SILU>(mx, mw, my, mr, ad, p, t, pairs, s);
    default: return start_pair<MCS_ACT_NONE>(mx, mw, my, mr, ad, p, t, pairs, s);
  }
}

}  // namespace
}  // namespace mcs
