// Softmax attention over packed sequences, bf16, two tiles of 128 query rows at a time: sequences of more than one tile.
// Formula, items, masks and what lies in masked places as in packed_attn.cu.
//
// One tile alone leaves the tensor core idle while its softmax runs, and the other way round: 1,850 clocks a tile of 128 x
// 128 scores of which the products take 1,024. Here two tiles, A and B, share every K and V tile and take turns: while A's
// softmax runs, B's P V and next S do. A block an item, of which one an SM runs and takes over the items of blocks that
// have not started (cluster launch control), so that items of unlike length spread by themselves; 512 threads:
//   warps 0-3, 4-7  softmax of A and of B, a thread per row
//   warps 8-11      the rows' way out, of A and then of B, while the softmax is at the next item
//   warp 12         finds the items and loads by TMA: the queries of A and of B, and one ring of K_0, V_0, K_1, V_1, ...
//   warps 13, 14    the products of A and of B: S_0; then for every tile P_j V_j and S_{j+1}, in strict turns: without
//                   them A and B fall into step, both softmaxes and then both products (3,200 clocks a pair of tiles)
//   warp 15         makes V tiles that hold masked keys harmless and lets the products go
// A wait takes a product warp 200 to 300 clocks beside eight softmax warps even where nothing is to be waited for, as much
// as the products in the queue hide. So warp 15 looks after everything that a step needs (keys, values, a free O) and
// arrives together with the softmax's threads, and the turn is handed over before the last products are taken in. From one
// warp, A's step and then B's, 32,768 causal tokens took 2,255 us. P handed over
// in two halves was slower (2,450 us instead of 2,260), and the last tile's maximum as a first guess, checked
// afterwards, no faster (2,270).
// Tensor memory: S_A, S_B, O_A, O_B of 128 columns each, P_j written over S_j (a row per lane, so a thread overwrites only
// what it has read); the products of one warp run in order, so S_{j+1} cannot meet P_j.
// A sees fewer keys than B under a causal mask and leaves its last tiles out. Softmax warps take the registers that the
// others hand over (128 at launch; 184, 96 on the way out, 48).
//
// The compiler spills 36 to 40 bytes a thread in the kernel without cuts, 12 to 16 with, 148 to 186 in the one for long sums: the way
// out keeps eight 64-bit addresses in its 96 registers.
//
// Measured: 32,768 causal tokens of 12 heads on 4, d = 128: 2,160 to 2,190 us, 1,505 to 1,525 TFLOP/s at 1,910 to 1,940 MHz
// (0.86 to 0.87 of the sustained rate of plain products); three full sequences of 7,716, 4,031 and 1,626 tokens, 12 heads: 338
// us, 1,426 TFLOP/s, tensor pipe 64 % active; 16 causal prompts of 6 to 839 tokens, 32 heads on 8: 50 us, pipe 26 %. There the instructions count: with 62 KB of them, unrolled masks and
// 40 for every wait, a quarter of the fetches missed the instruction cache and the same prompts took 99 us.
#include <algorithm>
#include <type_traits>

#include "attn_common.cuh"
#include "common.cuh"
#include "launch.cuh"
#include "packed.h"
#include "packed_tc.cuh"
#include "ptx.cuh"
#include "tc_common.cuh"
#include "tma.cuh"

namespace mcs {
namespace {

constexpr int kThreads = 512;
constexpr int kLaunchRegs = 128, kControlRegs = 48, kOutRegs = 96, kSoftmaxRegs = 184;
static_assert(128 * kControlRegs + 128 * kOutRegs + 256 * kSoftmaxRegs <= kThreads * kLaunchRegs, "an increase would wait forever");
constexpr int kItems = 4;   // items found ahead
constexpr int kFlags = 8;   // items whose V flags are kept (warp 15 is at most kItems ahead of the way out)
// Waits that last as long as an item: of the way out for its sums, and of a chain without rows in it for the next. An item
// of 2^30 keys is 2^23 tiles of 1.7 us, 14 s.
constexpr uint64_t kItemLimitNs = 30ull * 1000ull * 1000ull * 1000ull;
constexpr int kPatch = 32 * 128;  // a warp's rows x 128 bytes on their way out

template <int D, bool kLong>
struct Cfg {
  static constexpr int kStages = (D == 128) ? 4 : 8;  // K and V tiles
  static constexpr int kTile = (D / 64) * kRegion;
  static constexpr int kQ = 0;                        // [2]
  static constexpr int kRing = 2 * kTile;
  static constexpr int kOut = kRing + kStages * kTile;
  static constexpr int kStats = kOut + 4 * kPatch;    // (maximum, sum) of A's and B's rows
  static constexpr int kBar = kStats + 2 * 128 * 8;
  static constexpr int kNumBars = 2 * kStages + 2 * 7 + 2 * kItems + 5;
  static constexpr int kSteal = (kBar + kNumBars * 8 + 15) / 16 * 16;  // the answer to a request for a block
  static constexpr int kMisc = kSteal + 16;
  static constexpr int kItem = (kMisc + 16 + kFlags * 4 + 15) / 16 * 16;
  static constexpr int kScale = kItem + kItems * int(sizeof(PackedItem));  // [2][128] the bank's factor (kLong)
  static constexpr int kBytes = kScale + (kLong ? 2 * 128 * 4 : 0);
  static constexpr int kAlloc = kBytes + 1024;
  static constexpr uint32_t kColS = 0, kColO = 256;  // of A; B's lie 128 behind
};
static_assert(Cfg<128, true>::kAlloc <= 227 * 1024 && Cfg<64, true>::kAlloc <= 227 * 1024, "shared memory");

// A chain's sums of a row, added to its bank, whose own sums are taken times `keep`. first: it holds nothing yet.
template <int D>
__device__ __forceinline__ void empty_sums(uint32_t tO, float4* bank, float keep, bool first) {
#pragma unroll 1
  for (int q = 0; q < D / 32; ++q) {
    uint32_t o[32];
    tmem_ld32(tO + q * 32, o);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float4 b = first ? make_float4(0.f, 0.f, 0.f, 0.f) : bank[q * 8 + i];
      b.x = (isfinite(b.x) ? b.x * keep : b.x) + __uint_as_float(o[4 * i]);
      b.y = (isfinite(b.y) ? b.y * keep : b.y) + __uint_as_float(o[4 * i + 1]);
      b.z = (isfinite(b.z) ? b.z * keep : b.z) + __uint_as_float(o[4 * i + 2]);
      b.w = (isfinite(b.w) ? b.w * keep : b.w) + __uint_as_float(o[4 * i + 3]);
      bank[q * 8 + i] = b;
    }
  }
}

// kCut: an item's keys are one piece of its sequence's, its sums leave in fp32 for packed_join.
// kLong: items may have more than 2^18 keys. Every kSumTiles tiles the softmax's threads add their rows' sums to the block's bank in
// global memory (P V of the tile before is done when they hold the scores) and the next P V begins anew; the sums of weights
// go with them, in registers. The way out adds the bank before it gives O back, so the next item cannot meet it.
template <int D, bool kCut, bool kLong>
__global__ void __launch_bounds__(kThreads, 1)
    packed_pair_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                       const __grid_constant__ CUtensorMap map_v, const PackedParams p, const PackedWalk wk) {
  static_assert(!(kCut && kLong), "pieces are short");
  using L = Cfg<D, kLong>;
  constexpr int R = L::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::kBar);  // K or V tile landed
  uint64_t* empty = full + R;         // its products of A and of B are done
  uint64_t* q_full = empty + R;       // [2] and so on: of A and of B
  uint64_t* q_empty = q_full + 2;
  uint64_t* s_go = q_empty + 2;       // queries and first keys are there
  uint64_t* s_full = s_go + 2;
  uint64_t* p_full = s_full + 2;      // P written (128 threads), and all else that P V and the next S need (warp 15)
  uint64_t* o_full = p_full + 2;
  uint64_t* o_free = o_full + 2;
  uint64_t* it_full = o_free + 2;     // [kItems]
  uint64_t* it_empty = it_full + kItems;
  uint64_t* turn = it_empty + kItems;  // [2] products of a tile issued, or left out
  uint64_t* drain = turn + 2;          // [2]
  uint64_t* steal = drain + 2;
  const uint32_t steal_slot = sbase + L::kSteal;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kMisc);
  volatile uint32_t* odd = tmem_slot + 4;  // [kFlags] the item's V held something that is not finite and not seen by all
  float2* stats = reinterpret_cast<float2*>(smem + L::kStats);
  [[maybe_unused]] float* bank_scale = reinterpret_cast<float*>(smem + L::kScale);
  // a row of a chain in this block's bank
  [[maybe_unused]] auto bank_row = [&](int c, int row) {
    return reinterpret_cast<float4*>(p.part_o + ((static_cast<size_t>(blockIdx.x) * 2 + c) * 128 + row) * D);
  };
  PackedItem* items = reinterpret_cast<PackedItem*>(smem + L::kItem);

  const int tid = threadIdx.x, warp = warp_uniform(tid >> 5), lane = tid & 31;
  uint32_t* st = p.status;
  if (tid == 0) {
    for (int s = 0; s < R; ++s) mbar_init(full + s, 1), mbar_init(empty + s, 2);
    for (int c = 0; c < 2; ++c) {
      mbar_init(q_full + c, 1), mbar_init(q_empty + c, 1), mbar_init(s_go + c, 1), mbar_init(turn + c, 1), mbar_init(drain + c, 1), mbar_init(s_full + c, 1);
      mbar_init(p_full + c, 129), mbar_init(o_full + c, 130), mbar_init(o_free + c, 128);
    }
    mbar_init(steal, 1);
    for (int b = 0; b < kItems; ++b) mbar_init(it_full + b, 1), mbar_init(it_empty + b, 8 + 4 + 3);
    fence_mbar_init();
  }
  if (warp == 12 && lane == 0) tma_prefetch_map(&map_q), tma_prefetch_map(&map_k), tma_prefetch_map(&map_v);
  if (warp == 13) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = warp_uniform(*tmem_slot);
  grid_inputs_ready();
  grid_let_next_start();
  const int half = p.tq / 2;  // tokens of a tile

  // The next item for a role; its slot is given back at once. n: items taken so far.
  auto take = [&](int n, PackedItem& it) -> bool {
    const int b = n % kItems;
    if (!warp_all(mbar_wait_short<kItemLimitNs>(it_full + b, uint32_t(n / kItems) & 1))) return false;
    it = items[b];
    __syncwarp();
    if (lane == 0) mbar_arrive(it_empty + b);
    return true;
  };
  // Key tiles of A (c = 0) or B; 0 where it has no tokens or they see nothing.
  auto tiles_of = [&](const PackedItem& it, int c) -> int {
    const int n = min(it.ntok - c * half, half);
    return n <= 0 ? 0 : (visible_keys(it, p.causal, c * half + n - 1) + 127) >> 7;
  };

  if (warp >= 12) {
    registers_down<kControlRegs>();
    if (warp == 12) {
      // ---------------------------------------------------------- items and copies
      bool ok = true;
      int n = 0, cnt = 0, live0 = 0, live1 = 0;  // items, K and V tiles, items of A and B so far
      auto load = [&](const CUtensorMap* map, const PackedItem& it, int j) -> bool {
        const int s = cnt % R;
        if (!warp_all(mbar_wait_short(empty + s, (uint32_t(cnt / R) & 1) ^ 1))) return false;
        if (elect_one()) {
          mbar_arrive_expect_tx(full + s, L::kTile);
#pragma unroll
          for (int rg = 0; rg < D / 64; ++rg)
            tma_load_3d(sbase + L::kRing + s * L::kTile + rg * kRegion, map, rg * 64, it.hk, it.k0 + j * 128, smem_u32(full + s));
        }
        __syncwarp();
        ++cnt;
        return true;
      };
      std::conditional_t<kLong, PackedCounted, PackedBlocks> blocks(p, wk, lane, steal, steal_slot);
      PackedItem it{}, following{};  // the first turn finds an item and loads nothing
      for (bool begun = false;; it = following, begun = true) {
        if (begun) {
          const int b = n % kItems;
          if (!(ok = warp_all(mbar_wait_short(it_empty + b, (uint32_t(n / kItems) & 1) ^ 1)))) break;
          if (lane == 0) {
            items[b] = it;
            mbar_arrive(it_full + b);
          }
          __syncwarp();
          ++n;
          if (it.tiles < 0) break;
        }
        for (int x = 0; x < max(2 * it.tiles, 2); ++x) {  // K_0, queries, the item after this one, V_0, K_1, V_1, ...
          if (x < 2 * it.tiles) {
            if (!(ok = load(x & 1 ? &map_v : &map_k, it, x >> 1))) break;
          }
          if (x > 0) continue;
#pragma unroll 1
          for (int c = 0; c < 2 && ok && it.tiles > 0; ++c) {
            if (tiles_of(it, c) == 0) continue;
            const int nth = c ? live1++ : live0++;
            if (!(ok = warp_all(mbar_wait_short(q_empty + c, (uint32_t(nth) & 1) ^ 1)))) break;
            if (elect_one()) {
              mbar_arrive_expect_tx(q_full + c, uint32_t(half * p.g * 128 * (D / 64)));
#pragma unroll
              for (int rg = 0; rg < D / 64; ++rg)
                tma_load_3d(sbase + L::kQ + c * L::kTile + rg * kRegion, &map_q, rg * 64, it.hk * p.g, it.q0 + c * half, smem_u32(q_full + c));
            }
            __syncwarp();
          }
          if (!ok) break;
          if (!(ok = blocks.next(p, wk, lane, following))) break;
        }
        if (!ok) break;
      }
      if (!ok) {
        if (lane == 0) raise_status(st, kStatusTimeout);
        settle_copies();  // normally the products have consumed every copy before the CTA exits
      }
      __syncwarp();
    } else if (warp <= 14) {
      // ---------------------------------------------------------- products of A (warp 13) and of B (warp 14)
      const int c = warp - 13;
      constexpr uint32_t kIdescQK = idesc_bf16_f32(128, 128, 0, 0);
      constexpr uint32_t kIdescPV = idesc_bf16_f32(128, D, 0, 1);
      const uint32_t tO = tmem + L::kColO + c * 128, tS = tmem + L::kColS + c * 128;
      const uint32_t qlo = desc_lo_kmajor(sbase + L::kQ + c * L::kTile);
      bool ok = true, issued = false;
      uint32_t tile = 0, done = 0, live = 0;  // K/V tiles so far, those of this chain, its items
      for (int n = 0; ok; ++n) {
        PackedItem it;
        if (!(ok = take(n, it))) break;
        if (it.tiles < 0) break;
        const int T = tiles_of(it, c);
        // S_0; then P_j V_j and S_{j+1}
        for (int j = -1; j < it.tiles; ++j) {
          if (j < 0 && T == 0) continue;
          const uint32_t xv = 2 * (tile + j) + 1, sv = xv % R, xk = xv + 1, sk = xk % R;
          if (j >= 0) {
            // the other one's products of the tile before (A: of B; B: of A, this tile) have been issued
            if (!(ok = warp_all(mbar_wait_short(turn + (c ^ 1), (tile + j + (c ^ 1)) & 1)))) break;
            if (j >= T) {  // a tile that only B takes: its keys and values are let go when they have come
              ok = warp_all(mbar_wait_short(full + (xv - 1) % R, ((xv - 1) / R) & 1)) && warp_all(mbar_wait_short(full + sv, (xv / R) & 1));
              if (!ok) break;
              if (lane == 0) mbar_arrive(empty + (xv - 1) % R), mbar_arrive(empty + sv), mbar_arrive(turn + c);
              __syncwarp();
              continue;
            }
          }
          if (!(ok = warp_all(mbar_wait_short((j < 0 ? s_go : p_full) + c, j < 0 ? live & 1 : (done + j) & 1)))) break;
          tc_fence_after();
          issued = true;
          const uint32_t vlo = desc_lo_mnmajor(sbase + L::kRing + sv * L::kTile), klo = desc_lo_kmajor(sbase + L::kRing + sk * L::kTile);
          if (elect_one()) {
            if (j >= 0) {
#pragma unroll
              for (int ks = 0; ks < 8; ++ks)
                tc_mma_ts_lo(tO, tS + ks * 8, vlo + kstep_mnmajor(ks), kIdescPV, ((kLong ? j % kSumTiles : j) > 0 || ks > 0) ? 1u : 0u);
              tc_commit(empty + sv);
              // The other one's turn: it takes 300 clocks to begin, two S products are in the queue by then (with all
              // of them 345 us instead of 344 for three clips, from P V on 345).
              if (j + 1 >= T) mbar_arrive(turn + c);
              if (j == T - 1) {
                tc_commit(o_full + c);
                mbar_arrive(o_full + c);  // passes on the flag of V
              }
            }
            if (j + 1 < T) {
#pragma unroll
              for (int ks = 0; ks < D / 16; ++ks) {
                tc_mma_ss_lo(tS, qlo + kstep_kmajor(ks), klo + kstep_kmajor(ks), kIdescQK, ks > 0 ? 1u : 0u);
                if (j >= 0 && ks == 1) mbar_arrive(turn + c);
              }
              tc_commit(s_full + c);
              tc_commit(empty + sk);
              if (j + 2 == T) tc_commit(q_empty + c);
            }
          }
          __syncwarp();
        }
        if (!ok) break;
        tile += it.tiles;
        done += T, live += T > 0;
      }
      if (!ok) {
        if (lane == 0) raise_status(st, kStatusTimeout);
        if (issued) {
          if (elect_one()) tc_commit(drain + c);
          __syncwarp();
          mbar_drain(drain + c, 0);
        }
      }
      __syncwarp();
    } else {
      // ---------------------------------------------------------- V tiles, and what lets the products go
      bool ok = true;
      int tile = 0, done0 = 0, done1 = 0, live0 = 0, live1 = 0;
      auto landed = [&](int x) { return warp_all(mbar_wait_short(full + x % R, uint32_t(x / R) & 1)); };
      for (int n = 0; ok; ++n) {
        PackedItem it;
        if (!(ok = take(n, it))) break;
        if (it.tiles < 0) break;
        const int T0 = tiles_of(it, 0), T1 = tiles_of(it, 1);
        const int all_see = visible_keys(it, p.causal, 0);
        bool found = false;
        if (lane == 0) odd[n % kFlags] = 0;
        if (it.tiles > 0 && !(ok = landed(2 * tile))) break;
#pragma unroll 1
        for (int x = -2; x < 2 * it.tiles && ok; ++x) {
          const int j = x >> 1, c = x & 1, T = c ? T1 : T0, live = c ? live1 : live0;
          if (j >= 0 && c == 0) {
            const int v = 2 * (tile + j) + 1;
            if (!(ok = landed(v))) break;
            if ((j + 1) * 128 > all_see) {
              found |= settle_v<D>(sbase + L::kRing + v % R * L::kTile, max(0, all_see - j * 128), min(128, it.nkeys - j * 128), 0, lane);
              fence_proxy_async_smem();
              if (__any_sync(0xffffffffu, found) && lane == 0) odd[n % kFlags] = 1;
              __syncwarp();
            }
            if (j + 1 < it.tiles && !(ok = landed(v + 1))) break;
          }
          if (j >= T || T == 0) continue;
          if (j < 0) {
            ok = warp_all(mbar_wait_short(q_full + c, uint32_t(live) & 1));
          } else {
            if (j == 0) ok = warp_all(mbar_wait_short(o_free + c, (uint32_t(live) & 1) ^ 1));
            // one arrival a phase: the last tile's has to be complete
            if (ok) ok = warp_all(mbar_wait_short(p_full + c, (uint32_t((c ? done1 : done0) + j) & 1) ^ 1));
          }
          if (ok && lane == 0) mbar_arrive((j < 0 ? s_go : p_full) + c);
        }
        tile += it.tiles;
        done0 += T0, done1 += T1, live0 += T0 > 0, live1 += T1 > 0;
      }
      if (!ok && lane == 0) raise_status(st, kStatusTimeout);
      __syncwarp();
    }
  } else if (warp >= 8) {
    registers_down<kOutRegs>();
    // ------------------------------------------------------------ the way out
    const int w4 = warp & 3, row = w4 * 32 + lane;
    const int tt = p.by_group.div(row), hh = row - tt * p.g;  // this row's token of a tile and head of the group
    bool ok = true;
    int live0 = 0, live1 = 0;
    const uint32_t patch = sbase + L::kOut + w4 * kPatch;
    // where this lane's pieces of a tile's rows go: made once, an address is some 30 instructions
    [[maybe_unused]] long long row_at[8];
    if constexpr (!kCut) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int r = w4 * 32 + i * 4 + (lane >> 3), rt = p.by_group.div(r);
        row_at[i] = (r - rt * p.g) * p.os.head + rt * p.os.token + (lane & 7) * 8;
      }
    }
    for (int n = 0; ok; ++n) {
      PackedItem it;
      if (!(ok = take(n, it))) break;
      if (it.tiles < 0) break;
      const int all_see = visible_keys(it, p.causal, 0);
#pragma unroll 1
      for (int c = 0; c < 2; ++c) {
        const int ntok = min(it.ntok - c * half, half);
        if (ntok <= 0) continue;
        const bool some = tiles_of(it, c) > 0;  // otherwise no row sees anything
        const uint32_t tO = tmem + L::kColO + c * 128 + (uint32_t(w4 * 32) << 16);
        float2 ml = make_float2(-INFINITY, 0.f);
        if (some) {
          if (!(ok = warp_all(mbar_wait_short<kItemLimitNs>(o_full + c, uint32_t(c ? live1++ : live0++) & 1)))) break;
          tc_fence_after();
          ml = stats[c * 128 + row];
        }
        const bool mine = tt < ntok;
        const int rows = min(32, ntok * p.g - w4 * 32);  // of this warp
        if (rows > 0) {
          const float l = ml.y, inv = kCut ? 1.f : l == 0.f ? 0.f : 1.f / l;  // rows that see nothing give 0
          // elements of V that are not finite and that only some rows see (left out of the products)
          const bool extra = some && all_see < it.nkeys && odd[n % kFlags] != 0;
          const int lim = visible_keys(it, p.causal, c * half + tt);
          constexpr int kPass = kCut ? 32 : 64;  // columns of 128 bytes of a row
          __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.o) + static_cast<long long>(it.hk) * p.g * p.os.head +
                               static_cast<long long>(it.q0 + c * half) * p.os.token;
          const long long part = it.part + c * half * p.g + w4 * 32;  // this warp's first row of the partial sums
#pragma unroll 1
          for (int q = 0; q < D / kPass; ++q) {
#pragma unroll 1
            for (int x = 0; x < kPass / 32; ++x) {  // 32 columns
              uint32_t u[32];
              if (some) {  // rows that see nothing have sums of 0
                tmem_ld32(tO + q * kPass + x * 32, u);
              } else {
#pragma unroll
                for (int i = 0; i < 32; ++i) u[i] = 0;
              }
              if (kLong && some && tiles_of(it, c) > kSumTiles) {
                const float4* bank = bank_row(c, row) + q * (kPass / 4) + x * 8;
                const float f = bank_scale[c * 128 + row];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                  float4 b;  // one after the other: all eight at once would not fit the registers
                  asm volatile("ld.global.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(b.x), "=f"(b.y), "=f"(b.z), "=f"(b.w) : "l"(bank + i) : "memory");
                  u[4 * i] = __float_as_uint(__uint_as_float(u[4 * i]) + (isfinite(b.x) ? b.x * f : b.x));
                  u[4 * i + 1] = __float_as_uint(__uint_as_float(u[4 * i + 1]) + (isfinite(b.y) ? b.y * f : b.y));
                  u[4 * i + 2] = __float_as_uint(__uint_as_float(u[4 * i + 2]) + (isfinite(b.z) ? b.z * f : b.z));
                  u[4 * i + 3] = __float_as_uint(__uint_as_float(u[4 * i + 3]) + (isfinite(b.w) ? b.w * f : b.w));
                }
              }
              if constexpr (!kCut) {
#pragma unroll
                for (int i = 0; i < 16; ++i) u[i] = pack_bf16x2(__uint_as_float(u[2 * i]) * inv, __uint_as_float(u[2 * i + 1]) * inv);
              }
#pragma unroll
              for (int i = 0; i < (kCut ? 8 : 4); ++i)
                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(patch + lane * 128 + (((x * 4 + i) ^ (lane & 7)) << 4)),
                             "r"(u[4 * i]), "r"(u[4 * i + 1]), "r"(u[4 * i + 2]), "r"(u[4 * i + 3])
                             : "memory");
            }
            if (q == D / kPass - 1 && some) {  // the sums have been read
              tc_fence_before();
              mbar_arrive(o_free + c);
            }
            if (extra && mine) add_unseen<kCut>(patch + lane * 128, lane, p, it, q * kPass, all_see, lim);
            __syncwarp();
            // along rows: eight lanes a row, four rows in flight
#pragma unroll
            for (int i0 = 0; i0 < 8; i0 += 4) {
              uint4 w[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int r = (i0 + i) * 4 + (lane >> 3);
                asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(w[i].x), "=r"(w[i].y), "=r"(w[i].z), "=r"(w[i].w)
                             : "r"(patch + r * 128 + (((lane & 7) ^ (r & 7)) << 4))
                             : "memory");
              }
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int r = (i0 + i) * 4 + (lane >> 3);
                if (r >= rows) break;
                if constexpr (kCut) {
                  *reinterpret_cast<uint4*>(p.part_o + (part + r) * D + q * kPass + (lane & 7) * 4) = w[i];
                } else {
                  *reinterpret_cast<uint4*>(out + row_at[i0 + i] + q * kPass) = w[i];
                }
              }
            }
            __syncwarp();
          }
          if (kCut && mine) p.part_ml[part + lane] = ml;
          if (!kCut && mine && p.lse != nullptr)
            p.lse[static_cast<long long>(it.hk * p.g + hh) * p.Tq + it.q0 + c * half + tt] = l == 0.f ? -INFINITY : (ml.x + __log2f(l)) * kLn2;
        } else if (some) {
          tc_fence_before();
          mbar_arrive(o_free + c);
        }
      }
    }
    if (!ok && lane == 0) raise_status(st, kStatusTimeout);
    __syncwarp();
  } else {
    registers_up<kSoftmaxRegs>();
    // ------------------------------------------------------------ softmax
    const int c = warp >> 2, w4 = warp & 3;
    const int row = tid & 127;
    const int tt = p.by_group.div(row), t = c * half + tt;  // this row's token of the tile, of the item
    const uint32_t lane_off = uint32_t(w4 * 32) << 16;
    const uint32_t tS = tmem + L::kColS + c * 128 + lane_off, tO = tmem + L::kColO + c * 128 + lane_off;
    const float sl2 = p.scale_log2;
    bool ok = true;
    int tile = 0, live = 0;  // of this chain
    for (int n = 0; ok; ++n) {
      PackedItem it;
      if (!(ok = take(n, it))) break;
      if (it.tiles < 0) break;
      const int ntok = min(it.ntok - c * half, half);
      if (ntok <= 0) continue;
      const int T = tiles_of(it, c);
      const bool mine = tt < ntok;  // ntok <= half, so a row past the tile's last is nobody's
      const int lim = mine ? visible_keys(it, p.causal, t) : it.nkeys;
      const bool busy = w4 * 32 < ntok * p.g;
      float m = -INFINITY, l = 0.f;
      [[maybe_unused]] float bank_m = -INFINITY, bank_l = 0.f;
      for (int j = 0; j < T; ++j, ++tile) {
        if (!(ok = warp_all(mbar_wait_short(s_full + c, uint32_t(tile) & 1)))) break;
        tc_fence_after();
        if (kLong && busy && j > 0 && j % kSumTiles == 0) {
          const float keep = bank_m == m ? 1.f : ex2_approx(bank_m - m);
          empty_sums<D>(tO, bank_row(c, row), keep, j == kSumTiles);
          bank_l = bank_l * keep + l;
          bank_m = m, l = 0.f;
        }
        uint32_t pk[64];
        bool need = false;
        float alpha = 1.f;
        if (busy) {
          const int nvalid = lim - j * 128;
          if (__any_sync(0xffffffffu, nvalid < 128)) mask_scores(tS, nvalid);
          uint32_t r[128];
          tmem_ld128(tS, r);
          float mp[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) mp[i] = __uint_as_float(r[i]);
#pragma unroll
          for (int i = 8; i < 128; i += 2) mp[(i >> 1) & 7] = fmax3(mp[(i >> 1) & 7], __uint_as_float(r[i]), __uint_as_float(r[i + 1]));
          const float mx = fmax3(fmax3(mp[0], mp[1], mp[2]), fmax3(mp[3], mp[4], mp[5]), fmaxf(mp[6], mp[7]));
          const float m_new = fmaxf(m, mx * sl2);
          need = m_new > m + 8.f;  // the sums are scaled anew only where the maximum grew by more than 2^8
          const float m_use = need ? m_new : m;
          alpha = need ? ex2_approx(m - m_new) : 1.f;
          const float neg_m = m_use == -INFINITY ? 0.f : -m_use;
          const uint64_t sl2x2 = f2_pack(sl2, sl2), negmx2 = f2_pack(neg_m, neg_m);
          uint64_t ls2[2] = {f2_pack(0.f, 0.f), f2_pack(0.f, 0.f)};
#pragma unroll
          for (int i = 0; i < 64; ++i) {
            float x0, x1;
            f2_unpack(f2_fma(f2_pack(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1])), sl2x2, negmx2), x0, x1);
            const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
            ls2[i & 1] = f2_add(ls2[i & 1], f2_pack(p0, p1));
            pk[i] = pack_bf16x2(p0, p1);
          }
          float la, lb;
          f2_unpack(f2_add(ls2[0], ls2[1]), la, lb);
          l = l * alpha + (la + lb);
          m = m_use;
          // the last tile's P V is done: S came behind it
          if (__any_sync(0xffffffffu, need && j > 0)) {
#pragma unroll 1
            for (int q = 0; q < D / 32; ++q) {
              uint32_t o[32];
              tmem_ld32(tO + q * 32, o);
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
              tmem_st32(tO + q * 32, o);
            }
          }
          tmem_st64(tS, pk);
        }
        tc_fence_before();
        mbar_arrive(p_full + c);
      }
      if (!ok) break;
      if (T == 0) continue;
      // the last item's rows have been read
      if (!(ok = warp_all(mbar_wait_short(o_free + c, (uint32_t(live) & 1) ^ 1)))) break;
      ++live;
      if (kLong && T > kSumTiles) {
        const float f = bank_m == m ? 1.f : ex2_approx(bank_m - m);
        l += bank_l * f;
        bank_scale[c * 128 + row] = f;
      }
      stats[c * 128 + row] = make_float2(m, l);
      mbar_arrive(o_full + c);
    }
    if (!ok && lane == 0) raise_status(st, kStatusTimeout);
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 13) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Sets the items' counter to 0 once the kernels before are done with the workspace.
__global__ void packed_none_taken_kernel(uint32_t* taken) {
  grid_inputs_ready();
  grid_let_next_start();
  *taken = 0;
}

template <int D, bool kCut, bool kLong = false>
cudaError_t launch_two(const PackedParams& p, cudaStream_t s) {
  CUtensorMap mq, mk, mv;
  if (!(make_view_map(&mq, p.q, p.H, p.Tq, D, p.qs, p.g, p.tq / 2) && make_view_map(&mk, p.k, p.Hk, p.Tk, D, p.ks, 1, 128) &&
        make_view_map(&mv, p.v, p.Hk, p.Tk, D, p.vs, 1, 128)))
    return cudaErrorInvalidValue;
  constexpr int kSmem = Cfg<D, kLong>::kAlloc;
  if constexpr (kLong) {
    const cudaError_t e = launch_overlapped(packed_none_taken_kernel, dim3(1), 1, 0, s, 0, p.taken);
    if (e != cudaSuccess) return e;
  }
  const cudaError_t e = allow_smem_and_regs<packed_pair_kernel<D, kCut, kLong>>(kSmem, kLaunchRegs);
  if (e != cudaSuccess) return e;
  const long long blocks = kLong ? std::min(p.banks, p.sms) : p.items;
  return launch_overlapped(packed_pair_kernel<D, kCut, kLong>, dim3(unsigned(blocks)), kThreads, kSmem, s, 0, mq, mk, mv, p, walk_of(p));
}

}  // namespace

cudaError_t packed_attn_pair(const PackedParams& p, cudaStream_t s) {
  if (p.banks > 0) return p.d == 128 ? launch_two<128, false, true>(p, s) : launch_two<64, false, true>(p, s);
  if (p.chunk == 0) return p.d == 128 ? launch_two<128, false>(p, s) : launch_two<64, false>(p, s);
  const cudaError_t e = p.d == 128 ? launch_two<128, true>(p, s) : launch_two<64, true>(p, s);
  return e != cudaSuccess ? e : packed_join(p, true, s);
}

}  // namespace mcs
