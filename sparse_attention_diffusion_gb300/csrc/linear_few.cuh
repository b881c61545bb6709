// bf16 matrix product with epilogue for few rows of x (a step's modulation
// vectors, a short text): reading w once is the bound, and the output tiles alone
// do not fill the GPU. The operands are exchanged, so that the 128 lanes of the
// tensor core take 128 rows of w (outputs) and the rows of x (tokens, 16 to 256
// of them) are the MMA's N; K is cut into S slices, one per CTA of a cluster.
// Each CTA streams its slice of w through a ring of TMA stages into fp32
// accumulators [128 outputs x tokens] in tensor memory (one for up to 1,536 columns,
// linear.h) and leaves their sum in its shared memory; after a cluster barrier every
// CTA adds a share of the tokens over the S partial sums (distributed shared memory,
// ranks in order, so that equal calls give equal bits) and applies the epilogue. No
// workspace, one launch.
// Measured: 2 rows x 5,120 -> 30,720 outputs (315 MB of w) 49 us = 0.95 of the copy
// bandwidth; back to back, 1 x 5,120 -> 5,120 13 us with three slices (18 with one),
// 64 x 1,536 -> 1,536 6.3 us, 200 x 5,120 -> 1,000 10 us with four slices (19 with one).
// 192 threads: warp 0 TMA producer, warp 1 MMA issuer and tensor-memory
// allocation, warps 2-5 the accumulator's way out; all six the final sum.
#pragma once
#include "adapters.h"
#include "attn_tc.h"
#include "common.cuh"
#include "linear.h"
#include "linear_epi.cuh"
#include "launch.cuh"
#include "linear_few.h"
#include "ptx.cuh"
#include "tc_common.cuh"
#include "tma.cuh"

namespace mcs {
namespace {

constexpr int kThreads = 192, kWarps = kThreads / 32;
constexpr int kWTile = 128 * 128;  // bytes of 128 rows of w x 64 columns
// barriers, the tensor-memory slot and with adapters a word a stage, after the ring
template <int kAdapt>
constexpr int kBarBytes = kAdapt == kAdapterSteps ? 320 : 256;
constexpr int kMaxStages = 12;

struct FewArgs {
  int rows, tiles, sections;  // rows of a section of x, its token tiles
  int col_mask, head_shift;   // column k of x is column k & col_mask of head k >> head_shift (token-major: one head)
  int bn, stages, splits;
  int accs, acc_cols;         // accumulators of the longest slice, their columns in tensor memory
  uint32_t tmem_cols;
};

// A 32-bit word of shared memory as the CTA of rank r holds it.
__device__ __forceinline__ uint32_t peer_word(uint32_t addr, int r, int splits) {
  uint32_t v;
  if (splits == 1) asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  else asm volatile("ld.shared::cluster.b32 %0, [%1];" : "=r"(v) : "r"(cluster_map(addr, r)) : "memory");
  return v;
}

// Adds a row's adapter to four of its sums: 16 bytes of `up` a load, a warp's lanes along the outputs.
__device__ __forceinline__ void add_adapter(const AdapterArgs<kAdapterRows>& ad, const LinearParams& p, int m, int o, float (&v)[4]) {
  const int a = ad.of_row[m];
  if (a < 0) return;
  const float4* h = reinterpret_cast<const float4*>(ad.h + size_t(m) * ad.R);
  const __nv_bfloat16* up = ad.up + (size_t(a) * p.O + o) * ad.R;
#pragma unroll 2
  for (int r = 0; r < ad.R; r += 8) {
    const float4 x = h[r / 4], y = h[r / 4 + 1];
    uint4 w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = o + i < p.O ? __ldg(reinterpret_cast<const uint4*>(up + size_t(i) * ad.R + r)) : uint4{};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float u[8];
      unpack8(w[i], u);
      v[i] = fmaf(x.x, u[0], fmaf(x.y, u[1], fmaf(x.z, u[2], fmaf(x.w, u[3], v[i]))));
      v[i] = fmaf(y.x, u[4], fmaf(y.y, u[5], fmaf(y.z, u[6], fmaf(y.w, u[7], v[i]))));
    }
  }
}

// This CTA's share of the outputs: tokens rank, rank + splits, ... over its warps,
// kTok of them and kRanks partial accumulators at a time, ranks added in order.
template <int kAct, int kTok, int kRanks, int kAdapt>
__device__ __forceinline__ void final_sums(const LinearParams& p, const FewArgs& a, const AdapterArgs<kAdapt>& ad, uint32_t sbase, int rank, int warp,
                                           int lane, int m0, int ntok, int o0) {
  const int o = o0 + lane * 4;
  const bool vec = p.O % 4 == 0;
  uint2 bias4{};
  if (vec && p.bias && o < p.O) bias4 = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p.bias) + o);
  const int stride = a.splits * kWarps;
  for (int c0 = rank + a.splits * warp; c0 < ntok; c0 += kTok * stride) {
    float v[kTok][4] = {};
    for (int r0 = 0; r0 < a.splits; r0 += kRanks) {
      float f[kTok][kRanks][4];
#pragma unroll
      for (int t = 0; t < kTok; ++t)
#pragma unroll
        for (int r = 0; r < kRanks; ++r) {
          f[t][r][0] = f[t][r][1] = f[t][r][2] = f[t][r][3] = 0.f;
          if (c0 + t * stride >= ntok || r0 + r >= a.splits) continue;
          const uint32_t at = sbase + uint32_t((c0 + t * stride) * 128 + lane * 4) * 4;
          if constexpr (kRanks == 1)
            asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                         : "=f"(f[t][r][0]), "=f"(f[t][r][1]), "=f"(f[t][r][2]), "=f"(f[t][r][3])
                         : "r"(at));
          else
            asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                         : "=f"(f[t][r][0]), "=f"(f[t][r][1]), "=f"(f[t][r][2]), "=f"(f[t][r][3])
                         : "r"(cluster_map(at, r0 + r)));
        }
#pragma unroll
      for (int t = 0; t < kTok; ++t)
#pragma unroll
        for (int r = 0; r < kRanks; ++r)  // those past the cluster add zero
#pragma unroll
          for (int i = 0; i < 4; ++i) v[t][i] += f[t][r][i];
    }
    if constexpr (kAdapt == kAdapterRows) {
#pragma unroll
      for (int t = 0; t < kTok; ++t)
        if (c0 + t * stride < ntok) add_adapter(ad, p, m0 + c0 + t * stride, o, v[t]);
    }
#pragma unroll
    for (int t = 0; t < kTok; ++t) {
      const int c = c0 + t * stride;
      if (c >= ntok) break;
      if (vec) {
        if (o < p.O) finish_four<kAct>(p, m0 + c, o, v[t], bias4);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (o + i < p.O) finish_one<kAct, __nv_bfloat16>(p, m0 + c, o + i, v[t][i]);
      }
    }
  }
}

// kTurns: two accumulators take turns and their sums are kept in registers; otherwise all stay until the end.
// kAdapt: with kAdapterSteps the segments of a tile with an adapter add their k steps, shared among the slices, after
// those of w, into a slice's last accumulator (adapters.h); with kAdapterRows a row's adapter is added to its sums on
// their way out. Only what reads h waits for the kernel before, which makes it; x and w are there (launch.cuh, the second
// kernel of a pair).
template <int kAct, bool kTurns, int kAdapt>
__global__ void __launch_bounds__(kThreads, 2)
    linear_few_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w,
                      const __grid_constant__ AdapterArgs<kAdapt> ad, const LinearParams p, const FewArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const int stage_bytes = kWTile + a.bn * 128;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + a.stages * stage_bytes);
  uint64_t* empty = full + kMaxStages;
  uint64_t* acc_full = empty + kMaxStages;  // [2] accumulator written (the first: all of them, if they stay)
  uint64_t* acc_empty = acc_full + 2;       // [2] accumulator read
  uint64_t* drain = acc_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile uint32_t* failed = tmem_slot + 1;  // a wait of this CTA ran out
  [[maybe_unused]] volatile uint32_t* stage_info = tmem_slot + 2;  // [kMaxStages]: 16-column products of the stage, 8: the last one
  const int tid = threadIdx.x, warp = warp_uniform(tid >> 5), lane = tid & 31;
  const int tt = blockIdx.x / a.splits, rank = blockIdx.x % a.splits;  // of the cluster {splits, 1, 1}
  const int sec = tt / a.tiles, tok0 = (tt % a.tiles) * a.bn, o0 = blockIdx.y * 128;
  const int nk = (p.K + 63) / 64;
  const int k_beg = int(static_cast<long long>(nk) * rank / a.splits);
  const int k_end = int(static_cast<long long>(nk) * (rank + 1) / a.splits);
  const int per_acc = a.accs > 1 ? kAccSteps : kOneAccSteps;  // k steps; a.accs: of the longest slice
  const int accs = (k_end - k_beg + per_acc - 1) / per_acc;
  uint32_t* st = p.status;
  if (tid == 64) {
    tma_prefetch_map(&map_w);
    tma_prefetch_map(&map_x);
  }
  if (tid == 0) {
    for (int s = 0; s < a.stages; ++s) mbar_init(full + s, 1), mbar_init(empty + s, 1);
    for (int b = 0; b < 2; ++b) mbar_init(acc_full + b, 1), mbar_init(acc_empty + b, 4);
    mbar_init(drain, 1);
    *failed = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, a.tmem_cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = warp_uniform(*tmem_slot);
  if constexpr (kAdapt == kNoAdapters) {
    grid_inputs_ready();
    grid_let_next_start();
  }

  bool ok = true;
  if (warp == 0) {
    int s = 0;
    uint32_t phase = 0;
    const int z0 = sec * p.heads;
    auto load = [&](const CUtensorMap* mw, int cw, int zw, const CUtensorMap* mx, int cx, int rx, int zx, uint32_t info) {
      if (!(ok = warp_all(mbar_wait(empty + s, phase ^ 1, st)))) return;
      const uint32_t dst = sbase + s * stage_bytes;
      if (elect_one()) {
        if (kAdapt == kAdapterSteps) stage_info[s] = info;
        mbar_arrive_expect_tx(full + s, stage_bytes);
        tma_load_3d(dst, mw, cw, o0, zw, smem_u32(full + s));
        tma_load_3d(dst + kWTile, mx, cx, rx, zx, smem_u32(full + s));
      }
      __syncwarp();
      if (++s == a.stages) s = 0, phase ^= 1;
    };
    if constexpr (kAdapt == kAdapterSteps) {
      const int row0 = ad.v.tiles.first(tt), row1 = ad.v.tiles.end(tt), chunks = (ad.v.R + 63) / 64;
      for (int i = k_beg; i < k_end - 1 && ok; ++i) {  // the last one when it is known whether more follow
        const int k = i * 64;
        load(&map_w, k, 0, &map_x, k & a.col_mask, tok0, z0 + (k >> a.head_shift), 4);
      }
      grid_inputs_ready();
      grid_let_next_start();
      int steps = 0;  // of all slices
      for_segments(ad.v, row0, row1, lane, [&](int, int, bool odd) { steps += odd ? 1 : 2 * chunks; });
      const int beg = int(static_cast<long long>(steps) * rank / a.splits), end = int(static_cast<long long>(steps) * (rank + 1) / a.splits);
      if (ok) {
        const int k = (k_end - 1) * 64;
        load(&map_w, k, 0, &map_x, k & a.col_mask, tok0, z0 + (k >> a.head_shift), 4 | (beg == end ? 8 : 0));
      }
      int n = 0;
      for_segments(ad.v, row0, row1, lane, [&](int seg, int which, bool odd) {
        for (int c = 0; c < (odd ? 1 : 2 * chunks); ++c, ++n) {
          if (n < beg || n >= end || !ok) continue;
          const uint32_t last = n == end - 1 ? 8 : 0;
          const int col = (c >> 1) * 64;
          if (odd) load(&map_w, nk * 64, 0, &ad.mask, 0, 0, tt + seg, 1 | last);  // zeros behind w's columns
          else load(&ad.up, col, which, &ad.h, col, 0, 2 * (tt + seg) + (c & 1), (min(64, ad.v.R - col) + 15) / 16 | last);
        }
      });
    } else {
      for (int i = k_beg; i < k_end && ok; ++i) {
        const int k = i * 64;
        load(&map_w, k, 0, &map_x, k & a.col_mask, tok0, z0 + (k >> a.head_shift), 0);
      }
    }
    if (!ok) {
      if (lane == 0) {
        *failed = 1;
        raise_status(st, kStatusTimeout);
      }
      settle_copies();  // normally the MMAs have consumed every copy before the CTA exits
    }
    __syncwarp();
  } else if (warp == 1) {
    const uint32_t idesc = idesc_bf16_f32(128, 0, 0, 0) | (uint32_t(a.bn >> 3) << 17);
    bool issued = false;
    int s = 0;
    uint32_t phase = 0;
    int step = 0, c = 0;  // k steps in the accumulator c
    constexpr bool kSteps = kAdapt == kAdapterSteps;
    for (int i = k_beg; kSteps || i < k_end; ++i) {
      const bool extra = kSteps && i >= k_end;  // into the accumulator that is there
      const int b = kTurns ? c & 1 : c;
      if (kTurns && step == 0 && !extra && !(ok = warp_all(mbar_wait(acc_empty + b, ((c >> 1) & 1) ^ 1, st)))) break;
      if (!(ok = warp_all(mbar_wait(full + s, phase, st)))) break;
      tc_fence_after();
      issued = true;
      const uint32_t info = kSteps ? warp_uniform(stage_info[s]) : 4u;
      const bool last = kSteps ? (info & 8) != 0 : i == k_end - 1;
      const uint32_t w = desc_lo_kmajor(sbase + s * stage_bytes);
      const uint32_t x = desc_lo_kmajor(sbase + s * stage_bytes + kWTile);
      if (elect_one()) {
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
          if (!kSteps || ks < int(info & 7))
            tc_mma_ss_lo(tmem + b * a.acc_cols, w + kstep_kmajor(ks), x + kstep_kmajor(ks), idesc,
                         (step > 0 || ks > 0 || extra) ? 1u : 0u);
        tc_commit(empty + s);
        if (last || (kTurns && !extra && step == per_acc - 1 && i < k_end - 1)) tc_commit(acc_full + (kTurns ? b : 0));
      }
      __syncwarp();
      if (++s == a.stages) s = 0, phase ^= 1;
      if (last) break;
      if (i < k_end - 1 && ++step == per_acc) step = 0, ++c;
    }
    if (!ok) {
      if (lane == 0) {
        *failed = 1;
        raise_status(st, kStatusTimeout);
      }
      if (issued) {
        if (elect_one()) tc_commit(drain);
        __syncwarp();
        mbar_drain(drain, 0);
      }
      settle_copies();
    }
    __syncwarp();
  } else {
    if constexpr (kAdapt == kAdapterRows) {  // the rows' adapters come to the L2 cache while the products run
      grid_inputs_ready();
      const int live = min(128, p.O - o0), lines = (live * ad.R * 2 + 127) / 128;
      for (int c = rank + a.splits * (warp - 2); c < min(a.bn, a.rows - tok0); c += 4 * a.splits) {
        const int which = ad.of_row[sec * a.rows + tok0 + c];
        if (which < 0) continue;
        const char* up = reinterpret_cast<const char*>(ad.up + (size_t(which) * p.O + o0) * ad.R);
        for (int i = lane; i < lines; i += 32) asm volatile("prefetch.global.L2 [%0];" ::"l"(up + min(i * 128, live * ad.R * 2 - 1)));
      }
      __syncwarp();
    }
    const int quarter = warp & 3;
    const uint32_t acc = tmem + (uint32_t(quarter * 32) << 16);
    float* part = reinterpret_cast<float*>(smem) + quarter * 32 + lane;
    auto add = [](uint32_t (&v)[32], const uint32_t (&r)[32]) {
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) + __uint_as_float(r[i]));
    };
    // every MMA has read its stages once the last accumulator is complete, so the ring is free then
    auto leave = [&](const uint32_t (&v)[32], int c) {
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (c + i < a.bn) part[(c + i) * 128] = __uint_as_float(v[i]);
    };
    if constexpr (kTurns) {
      uint32_t sum[4][32];  // this output's sums of 32 tokens each
      for (int n = 0; n < accs; ++n) {
        const int b = n & 1;
        if (!(ok = warp_all(mbar_wait(acc_full + b, (n >> 1) & 1, st)))) break;
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          if (c * 32 >= a.bn) continue;
          if (n == 0) {
            tmem_ld32(acc + c * 32, sum[c]);
          } else {
            uint32_t r[32];
            tmem_ld32(acc + b * a.acc_cols + c * 32, r);
            add(sum[c], r);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(acc_empty + b);
      }
      if (ok) {
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (c * 32 < a.bn) leave(sum[c], c * 32);
      }
    } else if ((ok = warp_all(mbar_wait(acc_full, 0, st)))) {
      tc_fence_after();
      for (int c = 0; c < a.bn; c += 32) {
        uint32_t v[32];
        tmem_ld32(acc + c, v);
        for (int n = 1; n < accs; ++n) {
          uint32_t r[32];
          tmem_ld32(acc + n * a.acc_cols + c, r);
          add(v, r);
        }
        leave(v, c);
      }
    }
    if (!ok && lane == 0) {
      *failed = 1;
      raise_status(st, kStatusTimeout);
    }
  }
  tc_fence_before();
  // partial accumulators complete in every CTA of the cluster (all threads of all of them come here)
  if (a.splits > 1) cluster_sync();
  else __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, a.tmem_cols);
  }
  if constexpr (kAdapt == kAdapterRows) {
    grid_inputs_ready();
    grid_let_next_start();
  }
  // sums with a failed CTA's share are not written anywhere
  ok = true;
  for (int r = 0; r < a.splits; ++r) ok = ok && peer_word(smem_u32(tmem_slot + 1), r, a.splits) == 0;
  const int ntok = min(a.bn, a.rows - tok0);
  // several reads in flight: a remote one takes several hundred clocks
  if (ok) {
    if (a.splits == 1) final_sums<kAct, 4, 1>(p, a, ad, sbase, rank, warp, lane, sec * a.rows + tok0, ntok, o0);
    else final_sums<kAct, 2, 4>(p, a, ad, sbase, rank, warp, lane, sec * a.rows + tok0, ntok, o0);
  }
  if (a.splits > 1) cluster_sync();  // the other CTAs may still be reading this one's sums
}

template <int kAct, bool kTurns, int kAdapt>
cudaError_t start_few_act(const CUtensorMap& mx, const CUtensorMap& mw, const AdapterArgs<kAdapt>& ad, const LinearParams& p,
                      const FewArgs& a, dim3 grid, size_t smem, cudaStream_t s) {
  const cudaError_t e = allow_smem<linear_few_kernel<kAct, kTurns, kAdapt>>(226 * 1024);
  if (e != cudaSuccess) return e;
  return launch_overlapped(linear_few_kernel<kAct, kTurns, kAdapt>, grid, kThreads, smem, s, unsigned(a.splits), mx, mw, ad, p, a);
}
template <bool kTurns, int kAdapt>
cudaError_t start_few(const CUtensorMap& mx, const CUtensorMap& mw, const AdapterArgs<kAdapt>& ad, const LinearParams& p,
                      const FewArgs& a, dim3 grid, size_t smem, cudaStream_t s) {
  switch (p.act) {
    case MCS_ACT_GELU_TANH: return start_few_act<MCS_ACT_GELU_TANH, kTurns>(mx, mw, ad, p, a, grid, smem, s);
    case MCS_ACT_GELU_ERF: return start_few_act<MCS_ACT_GELU_ERF, kTurns>(mx, mw, ad, p, a, grid, smem, s);
    case MCS_ACT_SILU: return start_few_act<MCS_ACT_SILU, kTurns>(mx, mw, ad, p, a, grid, smem, s);
    default: return start_few_act<MCS_ACT_NONE, kTurns>(mx, mw, ad, p, a, grid, smem, s);
  }
}


// adapters: null without adapters.
template <int kAdapt>
cudaError_t launch_few(const LinearParams& p, const FewPlan& plan, const AdapterParams* adapters, int num_sms, cudaStream_t s) {
  FewArgs a{};
  CUtensorMap mx, mw;
  bool ok;
  if (p.heads > 0) {
    const int d = p.K / p.heads;
    a.head_shift = d == 64 ? 6 : 7;
    a.col_mask = d - 1;
    a.rows = p.N;
    a.sections = p.B;
    ok = make_tile_map(&mx, p.x, uint64_t(p.B) * p.heads, p.N, d, plan.bn);
  } else {
    a.head_shift = 31;
    a.col_mask = INT32_MAX;
    a.rows = p.M;
    a.sections = 1;
    ok = make_tile_map(&mx, p.x, 1, p.M, p.K, plan.bn);
  }
  ok = ok && make_tile_map(&mw, p.w, 1, p.O, p.K, 128);
  if (!ok) return cudaErrorInvalidValue;
  a.bn = plan.bn;
  a.splits = plan.splits;
  a.tiles = (a.rows + a.bn - 1) / a.bn;
  const int steps = ((p.K + 63) / 64 + a.splits - 1) / a.splits;
  a.accs = acc_count(steps);
  a.acc_cols = few_acc_cols(a.bn);
  a.tmem_cols = 32;
  while (int(a.tmem_cols) < few_accs(a.bn, steps) * a.acc_cols) a.tmem_cols *= 2;
  // the ring takes an SM's shared memory when every CTA has an SM to itself, half of it otherwise; it ends
  // up holding the partial accumulator
  const int stage = kWTile + a.bn * 128;
  const long long ctas = static_cast<long long>(a.splits) * a.tiles * a.sections * ((p.O + 127) / 128);
  const bool half = ctas > few_slots(a.splits, num_sms) && few_two_per_sm(a.bn, steps);
  a.stages = (half ? kFewHalfSm : 226 * 1024 - kBarBytes<kAdapt> - 1024) / stage;
  if (a.stages > kMaxStages) a.stages = kMaxStages;
  const size_t smem = size_t(a.stages) * stage + kBarBytes<kAdapt> + 1024;
  AdapterArgs<kAdapt> ad{};
  if constexpr (kAdapt == kAdapterSteps) {
    const cudaError_t e = adapters_down_tc(p, *adapters, RowTiles(a.rows, a.sections, a.bn), a.bn, 128, num_sms, int(ctas < num_sms ? num_sms - ctas : 0), &ad, s);
    if (e != cudaSuccess) return e;
  }
  if constexpr (kAdapt == kAdapterRows) {
    float* h = static_cast<float*>(adapters->ws);
    int32_t* of_row = reinterpret_cast<int32_t*>(h + size_t(p.M) * adapters->R);
    const cudaError_t e = adapters_down_rows(p, *adapters, true, h, of_row, s);
    if (e != cudaSuccess) return e;
    ad = {h, of_row, static_cast<const __nv_bfloat16*>(adapters->up), adapters->R};
  }
  const dim3 grid(unsigned(a.splits) * a.tiles * a.sections, (p.O + 127) / 128);
  return few_turns(a.bn, steps) ? start_few<true>(mx, mw, ad, p, a, grid, smem, s)
                                : start_few<false>(mx, mw, ad, p, a, grid, smem, s);
}


}  // namespace
}  // namespace mcs
