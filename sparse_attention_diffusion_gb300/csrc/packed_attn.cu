// Softmax attention over packed sequences on the tcgen05 tensor cores, bf16:
//   o_i = sum_j softmax_j(scale q_i . k_j) v_j,  lse_i = log sum_j exp(scale q_i . k_j)
// over the keys j of query i's own sequence that it sees (with a causal mask the last of its nq queries
// sees all nk keys and each one before it one key less), grouped heads, lengths read on the device.
//
// A block an item of packed.h, of which one an SM runs and takes over the items of blocks that have not started (cluster
// launch control), so that items of unlike length spread by themselves; 224 threads:
//   warp 5    finds the items (four ahead) and loads by TMA: the item's queries as one box of g heads x
//             tq tokens, then rings of K and V tiles of 128 keys, K one tile ahead of V;
//   warp 4    tensor-memory allocation, S_j = Q K_j^T into two buffers;
//   warp 6    makes V tiles that hold masked keys harmless (below), O += P_j V_j, P from tensor memory;
//   warps 0-3 softmax, a thread per row, and the row's way out.
// Tensor memory: S0 [0,128), S1 [128,256), O [256,256+D), P [384,448) columns.
// The next item's queries, keys and first two S run under the last P V and the way out.
//
// Masked keys: their scores become -inf by selection, whatever they are, so P is 0. But 0 times an infinity or a NaN
// is NaN, and behind a sequence's last key lie another request's values. So in the tiles that hold a key some row
// does not see, warp 6 (which waits for P meanwhile) overwrites rows past the item's keys with zeros, and replaces
// what is not finite in the rows that only some tokens see by zero; rows that do see such an element add it on their way out
// (an infinity or a NaN stays one whatever finite numbers are added).
//
// Cut sequences (chunk > 0): an item is one chunk of a sequence's keys, its sums leave as fp32 with the row's
// maximum and sum, and a second launch joins them. A sequence of one chunk leaves at once.
//
// This kernel is for sequences of one tile, single tokens over kept keys above all; longer ones go two tiles at a time
// (packed_pair.cu). Measured: 64 tokens over 88 to 16,343 keys of 8 heads, d = 128: 263 to 266 us = 6.74 to 6.81 TB/s, as fast as
// the measured copy (302 us with items dealt out in advance and larger pieces); one token over 4,000 keys 11.5 to 11.9 us.
#include <algorithm>
#include <cfloat>

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

constexpr int kThreads = 224;
constexpr int kItems = 4;   // items found ahead
constexpr int kFlags = 2;   // items whose V flags are kept: warp 6 is one item ahead of the way out at most

template <int D, bool kQuarters>
struct Cfg {
  static constexpr int kStages = (D == 128) ? 3 : 6;
  static constexpr int kTile = (D / 64) * kRegion;
  static constexpr int kQ = 0;
  static constexpr int kK = kQ + kTile;
  static constexpr int kV = kK + kStages * kTile;
  static constexpr int kBar = kV + kStages * kTile;
  static constexpr int kNumBars = 4 * kStages + 2 + 2 + 2 + 2 + 2 + 2 * kItems + 2 + 1 + 1;
  static constexpr int kSteal = (kBar + kNumBars * 8 + 15) / 16 * 16;  // the answer to a request for a block
  static constexpr int kMisc = kSteal + 16;  // tensor-memory slot, flags, items
  static constexpr int kItem = (kMisc + 16 + kFlags * 4 + 15) / 16 * 16;
  static constexpr int kJoin = (kItem + kItems * int(sizeof(PackedItem)) + 127) / 128 * 128;  // 32 columns of four warps' sums,
  static constexpr int kJoinMl = kJoin + 4 * 32 * 128;                                         // their maxima and sums of weights
  static constexpr int kBytes = kQuarters ? kJoinMl + 4 * 32 * 8 : kJoin;
  static constexpr int kAlloc = kBytes + 1024;
  static constexpr uint32_t kColS = 0, kColO = 256, kColP = 384;
};
static_assert(Cfg<128, false>::kAlloc <= 227 * 1024 && Cfg<64, true>::kAlloc <= 227 * 1024, "shared memory");

// kQuarters: items of 32 rows at most, which lie four times in the tile, 32 rows apart: every softmax warp has all of them
// and takes a quarter of a tile's keys, P being 0 for the others', and the four sums meet on the way out. One warp's softmax
// of 128 keys (2,100 clocks a tile with its waits) bounded tokens of d = 64, whose tiles take 1,500 from HBM: 64 over
// 16,384 keys and less of 8 heads 189 us with a softmax warp for all keys, 141 with four (0.94 of the copy bandwidth). With d = 128
// a tile takes twice as long, and there is no shared memory for the sums.
template <int D, bool kQuarters>
__global__ void __launch_bounds__(kThreads, 1)
    packed_attn_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                       const __grid_constant__ CUtensorMap map_v, const PackedParams p, const PackedWalk wk) {
  using L = Cfg<D, kQuarters>;
  constexpr int S = L::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + L::kBar);
  uint64_t* k_empty = k_full + S;
  uint64_t* v_full = k_empty + S;
  uint64_t* v_empty = v_full + S;
  uint64_t* s_full = v_empty + S;       // [2]
  uint64_t* s_free = s_full + 2;        // [2]
  uint64_t* p_full = s_free + 2;
  uint64_t* p_empty = p_full + 1;
  uint64_t* q_full = p_empty + 1;
  uint64_t* q_empty = q_full + 1;
  uint64_t* o_full = q_empty + 1;
  uint64_t* o_free = o_full + 1;
  uint64_t* it_full = o_free + 1;       // [kItems]
  uint64_t* it_empty = it_full + kItems;
  uint64_t* drain = it_empty + kItems;  // [2]
  uint64_t* steal = drain + 2;
  uint64_t* join = steal + 1;           // the softmax warps meet (kQuarters)
  const uint32_t steal_slot = sbase + L::kSteal;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kMisc);
  volatile uint32_t* odd = tmem_slot + 4;  // [kFlags] the item's V held something that is not finite and not seen by all
  PackedItem* items = reinterpret_cast<PackedItem*>(smem + L::kItem);

  const int tid = threadIdx.x, warp = warp_uniform(tid >> 5), lane = tid & 31;
  uint32_t* st = p.status;
  if (tid == 0) {
    for (int s = 0; s < S; ++s) mbar_init(k_full + s, 1), mbar_init(k_empty + s, 1), mbar_init(v_full + s, 1), mbar_init(v_empty + s, 1);
    for (int b = 0; b < 2; ++b) mbar_init(s_full + b, 1), mbar_init(s_free + b, 128), mbar_init(drain + b, 1);
    mbar_init(p_full, 128), mbar_init(p_empty, 1);
    mbar_init(q_full, 1), mbar_init(q_empty, 1), mbar_init(steal, 1), mbar_init(join, 128);
    mbar_init(o_full, 2), mbar_init(o_free, 128);  // o_full: the products and the flag of V
    for (int b = 0; b < kItems; ++b) mbar_init(it_full + b, 1), mbar_init(it_empty + b, 4 + 2);
    fence_mbar_init();
  }
  if (warp == 5 && lane == 0) tma_prefetch_map(&map_q), tma_prefetch_map(&map_k), tma_prefetch_map(&map_v);
  if (warp == 4) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = warp_uniform(*tmem_slot);
  const uint32_t tS = tmem + L::kColS, tO = tmem + L::kColO, tP = tmem + L::kColP;
  grid_inputs_ready();
  grid_let_next_start();

  // The next item for a role; its slot is given back at once. n: items taken so far.
  auto take = [&](int n, PackedItem& it) -> bool {
    const int b = n % kItems;
    const bool ok = warp_all(mbar_wait_short(it_full + b, uint32_t(n / kItems) & 1));
    if (!ok) return false;
    it = items[b];
    __syncwarp();
    if (lane == 0) mbar_arrive(it_empty + b);
    return true;
  };

  if (warp == 5) {
    // ------------------------------------------------------------ items and copies
    bool ok = true;
    int n = 0, live = 0, kn = 0, vn = 0;  // items, those with keys, K and V tiles so far
    auto load = [&](uint64_t* full, uint64_t* empty, int base, const CUtensorMap* map, int& cnt, const PackedItem& it, int j) -> bool {
      const int s = cnt % S;
      if (!warp_all(mbar_wait_short(empty + s, (uint32_t(cnt / S) & 1) ^ 1))) return false;
      if (elect_one()) {
        mbar_arrive_expect_tx(full + s, L::kTile);
#pragma unroll
        for (int rg = 0; rg < D / 64; ++rg)
          tma_load_3d(sbase + base + s * L::kTile + rg * kRegion, map, rg * 64, it.hk, it.k0 + j * 128, smem_u32(full + s));
      }
      __syncwarp();
      ++cnt;
      return true;
    };
    PackedBlocks blocks(p, wk, lane, steal, steal_slot);
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
      // K_0, queries, K_1, V_0; the item after this one; K_2, V_1, ...: the first keys do not wait for the queries'
      // place, which the last item's S products still read
      const int loads = 2 * it.tiles, found_at = min(loads, 3);
      for (int x = 0; x <= loads && ok; ++x) {
        if (x == found_at && !(ok = blocks.next(p, wk, lane, following))) break;
        if (x == loads) break;
        // in turn K_0, then K_{j+1} and V_j, at last V
        const bool is_v = x == loads - 1 || (x > 0 && (x & 1) == 0);
        const int j = is_v ? (x == loads - 1 ? it.tiles - 1 : x / 2 - 1) : (x + 1) / 2;
        if (!(ok = is_v ? load(v_full, v_empty, L::kV, &map_v, vn, it, j) : load(k_full, k_empty, L::kK, &map_k, kn, it, j))) break;
        if (x > 0) continue;
        if (!(ok = warp_all(mbar_wait_short(q_empty, (uint32_t(live) & 1) ^ 1)))) break;
        if (elect_one()) {
          constexpr int kCopies = kQuarters ? 4 : 1;
          mbar_arrive_expect_tx(q_full, uint32_t(p.rows * 128 * (D / 64) * kCopies));
#pragma unroll
          for (int rg = 0; rg < D / 64 * kCopies; ++rg)
            tma_load_3d(sbase + L::kQ + rg / kCopies * kRegion + rg % kCopies * 32 * 128, &map_q, rg / kCopies * 64, it.hk * p.g, it.q0,
                        smem_u32(q_full));
        }
        __syncwarp();
        ++live;
      }
      if (!ok) break;
    }
    if (!ok) {
      if (lane == 0) raise_status(st, kStatusTimeout);
      settle_copies();  // normally the MMAs have consumed every copy before the CTA exits
    }
    __syncwarp();
  } else if (warp == 4 || warp == 6) {
    // ------------------------------------------------------------ MMA issuers
    constexpr uint32_t kIdescQK = idesc_bf16_f32(128, 128, 0, 0);
    constexpr uint32_t kIdescPV = idesc_bf16_f32(128, D, 0, 1);
    bool ok = true, issued = false;
    int tile = 0, live = 0;
    for (int n = 0; ok; ++n) {
      PackedItem it;
      if (!(ok = take(n, it))) break;
      if (it.tiles < 0) break;
      if (it.tiles == 0) continue;
      if (warp == 4) {
        if (!(ok = warp_all(mbar_wait_short(q_full, uint32_t(live) & 1)))) break;
        const uint32_t qlo = desc_lo_kmajor(sbase + L::kQ);
        for (int j = 0; j < it.tiles; ++j, ++tile) {
          const int s = tile % S, b = tile & 1;
          ok = warp_all(mbar_wait_short(k_full + s, uint32_t(tile / S) & 1) &&
                        mbar_wait_short(s_free + b, (uint32_t(tile >> 1) & 1) ^ 1));
          if (!ok) break;
          tc_fence_after();
          issued = true;
          const uint32_t klo = desc_lo_kmajor(sbase + L::kK + s * L::kTile);
          if (elect_one()) {
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks)
              tc_mma_ss_lo(tS + b * 128, qlo + kstep_kmajor(ks), klo + kstep_kmajor(ks), kIdescQK, ks > 0 ? 1u : 0u);
            tc_commit(s_full + b);
            tc_commit(k_empty + s);
            if (j == it.tiles - 1) tc_commit(q_empty);
          }
          __syncwarp();
        }
      } else {
        const int all_see = visible_keys(it, p.causal, 0);
        bool found = false;
        for (int j = 0; j < it.tiles; ++j, ++tile) {
          const int s = tile % S;
          if (!(ok = warp_all(mbar_wait_short(v_full + s, uint32_t(tile / S) & 1)))) break;
          if ((j + 1) * 128 > all_see) {
            found |= settle_v<D>(sbase + L::kV + s * L::kTile, max(0, all_see - j * 128), min(128, it.nkeys - j * 128), 0, lane);
            fence_proxy_async_smem();
            __syncwarp();
          }
          if (j == 0) ok = warp_all(mbar_wait_short(o_free, (uint32_t(live) & 1) ^ 1));
          if (ok) ok = warp_all(mbar_wait_short(p_full, uint32_t(tile) & 1));
          if (!ok) break;
          tc_fence_after();
          issued = true;
          const uint32_t vlo = desc_lo_mnmajor(sbase + L::kV + s * L::kTile);
          if (elect_one()) {
#pragma unroll
            for (int ks = 0; ks < 8; ++ks)
              tc_mma_ts_lo(tO, tP + ks * 8, vlo + kstep_mnmajor(ks), kIdescPV, (j > 0 || ks > 0) ? 1u : 0u);
            tc_commit(p_empty);
            tc_commit(v_empty + s);
            if (j == it.tiles - 1) tc_commit(o_full);
          }
          __syncwarp();
        }
        if (!ok) break;
        found = __any_sync(0xffffffffu, found);
        if (lane == 0) {
          odd[n % kFlags] = found;
          mbar_arrive(o_full);
        }
      }
      ++live;
    }
    if (!ok) {
      if (lane == 0) raise_status(st, kStatusTimeout);
      uint64_t* d = drain + (warp == 6 ? 1 : 0);
      if (issued) {
        if (elect_one()) tc_commit(d);
        __syncwarp();
        mbar_drain(d, 0);
      }
    }
    __syncwarp();
  } else if constexpr (kQuarters) {
    // ------------------------------------------------------------ softmax of a quarter of the keys, and the way out
    const int t = p.by_group.div(lane), hh = lane - t * p.g;  // this row's token of the item and head of the group
    const uint32_t lane_off = uint32_t(warp * 32) << 16;
    const uint32_t tSw = tS + lane_off + warp * 32, tOw = tO + lane_off;
    const float sl2 = p.scale_log2;
    uint8_t* sums = smem + L::kJoin;
    float2* ml = reinterpret_cast<float2*>(smem + L::kJoinMl);
    bool ok = true;
    int tile = 0, live = 0;
    uint32_t met = 0;
    auto meet = [&]() -> bool {
      mbar_arrive(join);
      return warp_all(mbar_wait_short(join, met++ & 1));
    };
    {
      uint32_t zero[64];
#pragma unroll
      for (int c = 0; c < 64; ++c) zero[c] = 0;
      tmem_st64(tP + lane_off, zero);  // the other warps' keys, for good
    }
    for (int n = 0; ok; ++n) {
      PackedItem it;
      if (!(ok = take(n, it))) break;
      if (it.tiles < 0) break;
      const bool mine = t < it.ntok && lane < p.rows;
      const int lim = mine ? visible_keys(it, p.causal, t) : it.nkeys;
      float m = -INFINITY, l = 0.f;
      for (int j = 0; j < it.tiles; ++j, ++tile) {
        const int b = tile & 1;
        if (!(ok = warp_all(mbar_wait_short(s_full + b, uint32_t(tile >> 1) & 1)))) break;
        tc_fence_after();
        uint32_t r[32], pk[16];
        tmem_ld32(tSw + b * 128, r);
        tc_fence_before();
        mbar_arrive(s_free + b);
        const int nvalid = lim - j * 128 - warp * 32;
        if (__any_sync(0xffffffffu, nvalid < 32)) {
#pragma unroll
          for (int i = 0; i < 32; ++i) r[i] = i < nvalid ? r[i] : __float_as_uint(-INFINITY);
        }
        float mp[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) mp[i] = __uint_as_float(r[i]);
#pragma unroll
        for (int c = 4; c < 32; c += 2) mp[(c >> 1) & 3] = fmax3(mp[(c >> 1) & 3], __uint_as_float(r[c]), __uint_as_float(r[c + 1]));
        const float m_new = fmaxf(m, fmax3(fmaxf(mp[0], mp[1]), mp[2], mp[3]) * sl2);
        const bool need = m_new > m + 8.f;  // as below
        const float m_use = need ? m_new : m;
        const float alpha = need ? ex2_approx(m - m_new) : 1.f;
        const float neg_m = m_use == -INFINITY ? 0.f : -m_use;
        const uint64_t sl2x2 = f2_pack(sl2, sl2), negmx2 = f2_pack(neg_m, neg_m);
        uint64_t ls2[2] = {f2_pack(0.f, 0.f), f2_pack(0.f, 0.f)};
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          float x0, x1;
          f2_unpack(f2_fma(f2_pack(__uint_as_float(r[2 * c]), __uint_as_float(r[2 * c + 1])), sl2x2, negmx2), x0, x1);
          const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
          ls2[c & 1] = f2_add(ls2[c & 1], f2_pack(p0, p1));
          pk[c] = pack_bf16x2(p0, p1);
        }
        float la, lb;
        f2_unpack(f2_add(ls2[0], ls2[1]), la, lb);
        l = l * alpha + (la + lb);
        m = m_use;
        if (!(ok = warp_all(mbar_wait_short(p_empty, (uint32_t(tile) & 1) ^ 1)))) break;  // the last tile's P V is done
        tc_fence_after();
        if (__any_sync(0xffffffffu, need && j > 0)) {
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            uint32_t o[32];
            tmem_ld32(tOw + c * 32, o);
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
            tmem_st32(tOw + c * 32, o);
          }
        }
        tmem_st16(tP + lane_off + warp * 16, pk);
        tc_fence_before();
        mbar_arrive(p_full);
      }
      if (!ok) break;
      if (it.tiles > 0) {
        if (!(ok = warp_all(mbar_wait_short(o_full, uint32_t(live) & 1)))) break;
        ++live;
        tc_fence_after();
      }
      // 32 columns at a time: a warp leaves its sums of them, and adds the four warps' of eight
      const bool cut = !it.whole, extra = it.tiles > 0 && odd[n % kFlags] != 0;
      const int h = it.hk * p.g + hh, all_see = visible_keys(it, p.causal, 0);
      float M = -INFINITY, total = 0.f, f[4] = {};
      uint32_t far = 0;  // warps whose weight is 0 in fp32: only their infinities and NaN stay
      ml[tid] = make_float2(m, l);
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        if (it.tiles > 0) {
          uint32_t u[32];
          tmem_ld32(tOw + c * 32, u);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            *reinterpret_cast<uint4*>(sums + tid * 128 + ((i ^ (lane & 7)) << 4)) = make_uint4(u[4 * i], u[4 * i + 1], u[4 * i + 2], u[4 * i + 3]);
        }
        if (!(ok = meet())) break;
        if (c == 0) {  // weights of the four as in packed_join_kernel
          float2 x[4];
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            x[w] = ml[w * 32 + lane];
            M = fmaxf(M, x[w].x);
          }
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            f[w] = x[w].y == 0.f ? 0.f : x[w].x == -INFINITY ? 1.f : ex2_approx(x[w].x - M);
            total += x[w].y * f[w];
            if (x[w].y != 0.f && f[w] == 0.f) far |= 1 << w;
          }
        }
        if (mine) {
          const int col = c * 32 + warp * 8;
          float o[8] = {};
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            if (f[w] == 0.f) continue;  // no key, and what the sums hold then does not count, or far below the others
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float4 v = *reinterpret_cast<const float4*>(sums + (w * 32 + lane) * 128 + (((warp * 2 + i) ^ (lane & 7)) << 4));
              o[4 * i] = fmaf(f[w], v.x, o[4 * i]), o[4 * i + 1] = fmaf(f[w], v.y, o[4 * i + 1]);
              o[4 * i + 2] = fmaf(f[w], v.z, o[4 * i + 2]), o[4 * i + 3] = fmaf(f[w], v.w, o[4 * i + 3]);
            }
          }
#pragma unroll 1
          for (uint32_t left = far; left != 0; left &= left - 1) {
            const uint8_t* row = sums + ((__ffs(left) - 1) * 32 + lane) * 128;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float v = *reinterpret_cast<const float*>(row + (((warp * 2 + i / 4) ^ (lane & 7)) << 4) + i % 4 * 4);
              o[i] += isfinite(v) ? 0.f : v;
            }
          }
          const float inv = cut ? 1.f : total == 0.f ? 0.f : 1.f / total;  // rows that see nothing give 0
          bool lost = false;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            o[i] *= inv;
            lost |= !isfinite(o[i]);
          }
          // Elements of V that are not finite: those that only some rows see were left out of the products, and those that all
          // see are NaN in the sums of the warps whose P is 0 there. Their sum is what the row gives, if its weights are numbers.
          if (isfinite(total) && total != 0.f && (lost || extra)) {
            const __nv_bfloat16* vc = static_cast<const __nv_bfloat16*>(p.v) + static_cast<long long>(it.hk) * p.vs.head + col;
            float e[8] = {};
#pragma unroll 1
            for (int j = lost ? 0 : all_see; j < lim; ++j) {
              const uint4 v = *reinterpret_cast<const uint4*>(vc + static_cast<long long>(it.k0 + j) * p.vs.token);
              if ((odd_bf16x2(v.x) | odd_bf16x2(v.y) | odd_bf16x2(v.z) | odd_bf16x2(v.w)) == 0) continue;
              const uint32_t w4[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const float y = __uint_as_float(i & 1 ? w4[i >> 1] & 0xffff0000u : w4[i >> 1] << 16);
                if (!isfinite(y)) e[i] += y;
              }
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (!isfinite(e[i])) o[i] = e[i];
          }
          if (cut) {
            float* prow = p.part_o + (it.part + lane) * D + col;
            *reinterpret_cast<float4*>(prow) = make_float4(o[0], o[1], o[2], o[3]);
            *reinterpret_cast<float4*>(prow + 4) = make_float4(o[4], o[5], o[6], o[7]);
          } else {
            __nv_bfloat16* orow = static_cast<__nv_bfloat16*>(p.o) + (static_cast<long long>(h) * p.os.head + static_cast<long long>(it.q0 + t) * p.os.token) + col;
            *reinterpret_cast<uint4*>(orow) = make_uint4(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]), pack_bf16x2(o[4], o[5]), pack_bf16x2(o[6], o[7]));
          }
        }
        if (!(ok = meet())) break;  // the place is free again
      }
      if (!ok) break;
      if (mine && warp == 0) {
        if (cut) p.part_ml[it.part + lane] = make_float2(M, total);
        else if (p.lse != nullptr)
          p.lse[static_cast<long long>(h) * p.Tq + it.q0 + t] = total == 0.f ? -INFINITY : ((M == -INFINITY ? 0.f : M) + __log2f(total)) * kLn2;
      }
      if (it.tiles > 0) {
        tc_fence_before();
        mbar_arrive(o_free);
      }
    }
    if (!ok && lane == 0) raise_status(st, kStatusTimeout);
    __syncwarp();
  } else {
    // ------------------------------------------------------------ softmax and the way out
    const int row = tid;
    const int t = p.by_group.div(row), hh = row - t * p.g;  // this row's token of the tile and head of the group
    const uint32_t lane_off = uint32_t(warp * 32) << 16;
    const float sl2 = p.scale_log2;
    bool ok = true;
    int tile = 0, live = 0;
    for (int n = 0; ok; ++n) {
      PackedItem it;
      if (!(ok = take(n, it))) break;
      if (it.tiles < 0) break;
      const bool mine = t < it.ntok && row < p.rows;
      const int lim = mine ? visible_keys(it, p.causal, t) : it.nkeys;
      const bool busy = warp * 32 < it.ntok * p.g;  // the warp has rows (those of single tokens lie in the first ones)
      float m = -INFINITY, l = 0.f;
      for (int j = 0; j < it.tiles; ++j, ++tile) {
        const int b = tile & 1;
        if (!(ok = warp_all(mbar_wait_short(s_full + b, uint32_t(tile >> 1) & 1)))) break;
        tc_fence_after();
        uint32_t pk[64];
        bool need = false;
        float alpha = 1.f;
        if (busy) {
          const int nvalid = lim - j * 128;
          if (__any_sync(0xffffffffu, nvalid < 128)) mask_scores(tS + lane_off + b * 128, nvalid);
          uint32_t r[128];
          tmem_ld128(tS + lane_off + b * 128, r);
          tc_fence_before();
          mbar_arrive(s_free + b);
          float mp[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) mp[i] = __uint_as_float(r[i]);
#pragma unroll
          for (int c = 8; c < 128; c += 2) mp[(c >> 1) & 7] = fmax3(mp[(c >> 1) & 7], __uint_as_float(r[c]), __uint_as_float(r[c + 1]));
          const float mx = fmax3(fmax3(mp[0], mp[1], mp[2]), fmax3(mp[3], mp[4], mp[5]), fmaxf(mp[6], mp[7]));
          const float m_new = fmaxf(m, mx * sl2);
          need = m_new > m + 8.f;  // the sums are scaled anew only where the maximum grew by more than 2^8
          const float m_use = need ? m_new : m;
          alpha = need ? ex2_approx(m - m_new) : 1.f;
          const float neg_m = m_use == -INFINITY ? 0.f : -m_use;
          const uint64_t sl2x2 = f2_pack(sl2, sl2), negmx2 = f2_pack(neg_m, neg_m);
          uint64_t ls2[2] = {f2_pack(0.f, 0.f), f2_pack(0.f, 0.f)};
#pragma unroll
          for (int c = 0; c < 64; ++c) {
            float x0, x1;
            f2_unpack(f2_fma(f2_pack(__uint_as_float(r[2 * c]), __uint_as_float(r[2 * c + 1])), sl2x2, negmx2), x0, x1);
            const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
            ls2[c & 1] = f2_add(ls2[c & 1], f2_pack(p0, p1));
            pk[c] = pack_bf16x2(p0, p1);
          }
          float la, lb;
          f2_unpack(f2_add(ls2[0], ls2[1]), la, lb);
          l = l * alpha + (la + lb);
          m = m_use;
        } else {
          tc_fence_before();
          mbar_arrive(s_free + b);
        }
        if (!(ok = warp_all(mbar_wait_short(p_empty, (uint32_t(tile) & 1) ^ 1)))) break;  // the last tile's P V is done
        if (busy) {
          tc_fence_after();
          if (__any_sync(0xffffffffu, need && j > 0)) {
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              uint32_t o[32];
              tmem_ld32(tO + lane_off + c * 32, o);
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
              tmem_st32(tO + lane_off + c * 32, o);
            }
          }
          tmem_st64(tP + lane_off, pk);
        }
        tc_fence_before();
        mbar_arrive(p_full);
      }
      if (!ok) break;
      if (it.tiles > 0) {
        if (!(ok = warp_all(mbar_wait_short(o_full, uint32_t(live) & 1)))) break;
        ++live;
        tc_fence_after();
      }
      if (busy) {
        const int h = it.hk * p.g + hh;
        const bool cut = !it.whole;
        const float inv = cut ? 1.f : l == 0.f ? 0.f : 1.f / l;  // rows that see nothing give 0
        // elements of V that are not finite and that only some rows see (left out of the products)
        const bool extra = it.tiles > 0 && odd[n % kFlags] != 0;
        const int all_see = visible_keys(it, p.causal, 0);
        __nv_bfloat16* orow = static_cast<__nv_bfloat16*>(p.o) + (static_cast<long long>(h) * p.os.head + static_cast<long long>(it.q0 + t) * p.os.token);
        float* prow = cut ? p.part_o + (it.part + row) * D : nullptr;
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t u[32];
          float o[32];
          if (it.tiles > 0) {
            tmem_ld32(tO + lane_off + c * 32, u);
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = l == 0.f ? 0.f : __uint_as_float(u[i]) * inv;
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = 0.f;
          }
          if (!mine) continue;
          if (extra) {
            const __nv_bfloat16* vb = static_cast<const __nv_bfloat16*>(p.v) + static_cast<long long>(it.hk) * p.vs.head + c * 32;
            for (int j = all_see; j < lim; ++j) {
              const __nv_bfloat16* vr = vb + static_cast<long long>(it.k0 + j) * p.vs.token;
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                const float f = __bfloat162float(vr[i]);
                if (!isfinite(f)) o[i] += f;
              }
            }
          }
          if (cut) {
#pragma unroll
            for (int i = 0; i < 32; i += 4) *reinterpret_cast<float4*>(prow + c * 32 + i) = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
          } else {
#pragma unroll
            for (int i = 0; i < 32; i += 8) {
              uint4 w;
              w.x = pack_bf16x2(o[i], o[i + 1]);
              w.y = pack_bf16x2(o[i + 2], o[i + 3]);
              w.z = pack_bf16x2(o[i + 4], o[i + 5]);
              w.w = pack_bf16x2(o[i + 6], o[i + 7]);
              *reinterpret_cast<uint4*>(orow + c * 32 + i) = w;
            }
          }
        }
        if (mine && cut) p.part_ml[it.part + row] = make_float2(m, l);
        if (mine && !cut && p.lse != nullptr)
          p.lse[static_cast<long long>(h) * p.Tq + it.q0 + t] = l == 0.f ? -INFINITY : (m + __log2f(l)) * kLn2;
      }
      if (it.tiles > 0) {
        tc_fence_before();
        mbar_arrive(o_free);
      }
    }
    if (!ok && lane == 0) raise_status(st, kStatusTimeout);
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 4) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the chunks of a row: a block or more per token, a warp per head and turn. With M the largest of the chunks' maxima m_c,
//   o = sum_c 2^(m_c - M) O_c / sum_c 2^(m_c - M) l_c.
// Latency bounds it: lengths, maxima and sums are read one behind the other. Registers for a fourth block an SM are not spared
// (one token over 4,000 keys 12.9 us in both launches with four, 11.9 with three), and few instructions lie between the loads
// (four sums a turn 11.4 us, eight 11.9, sixteen 12.9).
template <int D, typename T>
__global__ void __launch_bounds__(256, 3) packed_join_kernel(const PackedParams p, const PackedWalk wk) {
  // The lengths are read before the wait for the pieces (launch.cuh, the second kernel of a pair). Every block waits, those
  // without work too, as the next call may overwrite the workspace once this grid is done.
  const int lane = threadIdx.x & 31, tok = blockIdx.x;
  const int s = packed_find(p.q_start, p.S, wk.by_one, 0, tok, lane);
  int q0 = 0, nq = 0, k0 = 0, nk = 0;
  const bool mine = s >= 0 && packed_sequence(p, s, q0, nq, k0, nk) && tok >= q0 && tok < q0 + nq;
  grid_inputs_ready();
  grid_let_next_start();
  if (!mine) return;
  const int i = tok - q0, iq = wk.by_tq.div(i), last = min((iq + 1) * p.tq, nq);
  const int seen = p.causal ? max(0, min(nk, last + nk - nq)) : nk;
  if (!p.pair && seen > 0 && seen <= p.chunk) return;  // one piece, which has left by itself
  const int chunks = wk.by_chunk.div(seen + p.chunk - 1), slot = wk.by_chunk.div(k0) + s;
  for (int h = blockIdx.y * 8 + (threadIdx.x >> 5); h < p.H; h += 8 * gridDim.y) {
    const int hk = p.by_group.div(h), hh = h - hk * p.g;
    const long long row = (i - iq * p.tq) * p.g + hh;
    auto at = [&](int c) { return ((static_cast<long long>(slot + c) * p.tiles + iq) * p.Hk + hk) * p.part_rows + row; };
    constexpr int kE = D / 32;
    float M = -INFINITY, l = 0.f, o[kE] = {};
    auto read = [&](int c, float (&v)[kE]) {
      const float* po = p.part_o + at(c) * D + lane * kE;
      if constexpr (kE == 4) {
        const float4 x = *reinterpret_cast<const float4*>(po);
        v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
      } else {
        const float2 x = *reinterpret_cast<const float2*>(po);
        v[0] = x.x, v[1] = x.y;
      }
    };
    for (int c0 = 0; c0 < chunks; c0 += 32) {
      const float2 ml = c0 + lane < chunks ? p.part_ml[at(c0 + lane)] : make_float2(-INFINITY, 0.f);
      constexpr int kFirst = 4;  // sums that are on their way while the maxima are compared
      float first[kFirst][kE];
  #pragma unroll
      for (int c = 0; c < kFirst; ++c)
        if (c0 + c < chunks) read(c0 + c, first[c]);
      float top = ml.x;
  #pragma unroll
      for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
      const float Mn = fmaxf(M, top), keep = M == -INFINITY ? 0.f : exp2f(M - Mn);
      // a chunk without a visible key has sum 0; one of NaN scores has maximum -inf but a sum that is NaN
      // (one whose weight leaves fp32's normal range adds nothing but its infinities and NaN, below)
      float f = ml.y == 0.f ? 0.f : ml.x == -INFINITY ? 1.f : exp2f(ml.x - Mn);
      uint32_t far = __ballot_sync(0xffffffffu, ml.y != 0.f && f < FLT_MIN);
      f = f < FLT_MIN ? 0.f : f;
      float sum = ml.y * f;
  #pragma unroll
      for (int x = 16; x > 0; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
      l = l * keep + sum;
  #pragma unroll
      for (int e = 0; e < kE; ++e) o[e] *= isfinite(o[e]) ? keep : 1.f;
      auto add = [&](int c, const float (&v)[kE]) {
        const float fc = __shfl_sync(0xffffffffu, f, c);
        if (fc != 0.f) {
  #pragma unroll
          for (int e = 0; e < kE; ++e) o[e] = fmaf(fc, v[e], o[e]);
        }
      };
      const int n = min(32, chunks - c0);
  #pragma unroll
      for (int c = 0; c < kFirst; ++c)
        if (c < n) add(c, first[c]);
  #pragma unroll 4
      for (int c = kFirst; c < n; ++c) {
        float v[kE];
        read(c0 + c, v);
        add(c, v);
      }
  #pragma unroll 1
      for (; far != 0; far &= far - 1) {
        float v[kE];
        read(c0 + __ffs(far) - 1, v);
  #pragma unroll
        for (int e = 0; e < kE; ++e) o[e] += isfinite(v[e]) ? 0.f : v[e];
      }
      M = Mn;
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    T* orow = static_cast<T*>(p.o) + (static_cast<long long>(h) * p.os.head + static_cast<long long>(tok) * p.os.token) + lane * kE;
  #pragma unroll
    for (int e = 0; e < kE; ++e) o[e] = l == 0.f ? 0.f : o[e] * inv;
    if constexpr (sizeof(T) == 2) {
      if constexpr (kE == 4) *reinterpret_cast<uint2*>(orow) = make_uint2(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]));
      else *reinterpret_cast<uint32_t*>(orow) = pack_bf16x2(o[0], o[1]);
    } else {
      if constexpr (kE == 4) *reinterpret_cast<float4*>(orow) = make_float4(o[0], o[1], o[2], o[3]);
      else *reinterpret_cast<float2*>(orow) = make_float2(o[0], o[1]);
    }
    if (p.lse != nullptr && lane == 0)
      p.lse[static_cast<long long>(h) * p.Tq + tok] = l == 0.f ? -INFINITY : (M == -INFINITY ? 0.f : M) * kLn2 + logf(l);
  }
}

template <int D, bool kQuarters>
cudaError_t launch_tc(const PackedParams& p, cudaStream_t s) {
  CUtensorMap mq, mk, mv;
  if (!(make_view_map(&mq, p.q, p.H, p.Tq, D, p.qs, p.g, p.tq) && make_view_map(&mk, p.k, p.Hk, p.Tk, D, p.ks, 1, 128) &&
        make_view_map(&mv, p.v, p.Hk, p.Tk, D, p.vs, 1, 128)))
    return cudaErrorInvalidValue;
  const cudaError_t e = allow_smem<packed_attn_kernel<D, kQuarters>>(Cfg<D, kQuarters>::kAlloc);
  if (e != cudaSuccess) return e;
  return launch_overlapped(packed_attn_kernel<D, kQuarters>, dim3(unsigned(p.items)), kThreads, Cfg<D, kQuarters>::kAlloc, s, 0, mq, mk, mv, p, walk_of(p));
}

}  // namespace

// Tiles and chunks. A tile takes as many tokens as fit in 128 rows (32: see kQuarters); on the CUDA cores in 64, or in 16 where
// a sequence has no more or the tiles of 64 are fewer than the SMs (77 tokens of 2 x 2 heads 13.9 us with 64 rows, 9.9 with 16).
// Sequences are cut where the tiles alone do not fill the GPU and a sequence has many keys. Where a sequence is one tile every
// SM gets eight pieces (64 tokens over 16,384 keys and less 288 us with four, 268 with eight, 265 with sixteen; but 128 over
// 2,000 keys and less 83 us with eight, 93 with sixteen, eight over 30,000 and less 74 and 101), unless they would be shorter than
// eight tiles: then one round of pieces, or pieces of eight tiles (16 tokens over 4,000 keys and less of 16 heads, d = 64, 34 us in pieces
// of two tiles, 24 so; three over 20,000 and less of 8 heads, d = 128, 22 and 17; the CUDA cores
// rather have the short ones: 32 tokens over 4,000 keys and less of 4 heads 185 us so, 145 without, 64 over 2,000 of 8 heads 314 and
// 302, though four over 9,000, d = 64, 33 and 36). Otherwise two an SM, as every tile
// of a sequence leaves its sums (seven chunks of 300 tokens and less: 49 us with one, 45 with two, 53 with four, 65 with eight).
// Sequences of more than one tile go two tiles at a time.
// The plan is made without a device (its workspace is asked for on the host) and so for the SMs of a whole one; with fewer the pieces are
// smaller than they need be.
// On the tensor cores no piece has more than kSumKeys, and sequences of one tile that may be longer than twice as many are cut too.
// The rules know the keys of all sequences together, not the longest: one of 16,384 keys among 64 whose others have 64 is not cut (122 us,
// of which its bytes take 12), nor are eight tokens over 100,000 keys beside a prompt of 4,096 (1,440 us; alone 477 and 135).
bool plan_packed(PackedParams* p, bool bf16, int longest) {
  constexpr int kSms = 152;
  p->g = p->H / p->Hk;
  int rows = bf16 ? 128 : 64;
  if (!bf16 && p->g <= 16) {
    const long long tiles64 = static_cast<long long>(p->Tq) / (64 / p->g) + p->S;
    if (static_cast<long long>(p->max_q) * p->g <= 16 || tiles64 * p->Hk < kSms) rows = 16;
  }
  p->quarters = bf16 && p->d == 64 && static_cast<long long>(p->max_q) * p->g <= 32;
  if (p->quarters) rows = 32;
  p->tq = rows / p->g;
  p->pair = bf16 && p->max_q > p->tq;
  if (p->pair) p->tq *= 2;
  p->by_group = Divisor(p->g);
  p->by_heads = Divisor(p->Hk);
  const long long tiles = (static_cast<long long>(p->max_q) + p->tq - 1) / p->tq;
  long long slots = static_cast<long long>(p->Tq) / p->tq + p->S;
  // tiles of all sequences together: not more than the slots, nor than the longest's of each
  const long long most = p->S * tiles < slots ? p->S * tiles : slots;
  const long long keys = static_cast<long long>(p->Tk) / p->S;
  p->chunk = 0;
  p->tiles = 1;
  const int piece = bf16 ? 128 : 64;
  if (keys >= 4 * piece && tiles <= 64 && (most * p->Hk < 2 * kSms || (tiles == 1 && most * p->Hk < 8 * kSms))) {
    const long long work = most * keys * p->Hk, each = tiles == 1 ? 8 : 2;
    long long chunk = (work / (each * kSms) + piece - 1) / piece * piece;
    // short pieces: rather one round of the SMs than eight
    const long long round = (work / kSms + piece - 1) / piece * piece;
    if (bf16 && tiles == 1) chunk = std::max(chunk, std::min(round, 8ll * piece));
    if (chunk < 2 * piece) chunk = 2 * piece;
    p->chunk = int(chunk < (1 << 30) ? chunk : (1 << 30));
    if (bf16) p->chunk = std::min(p->chunk, kSumKeys);
  } else if (bf16 && !p->pair && longest > 2 * kSumKeys) {
    p->chunk = kSumKeys;
  }
  if (p->chunk > 0) {
    p->tiles = int(tiles);
    slots = p->Tk / p->chunk + p->S;
    p->by_tiles = Divisor(p->tiles);
  }
  p->rows = p->tq * p->g;
  p->part_rows = std::min(p->tq, p->max_q) * p->g;
  p->items = slots * p->tiles * p->Hk;
  if (p->items >= (1ll << 31) - 65536) return false;
  p->banks = p->pair && p->chunk == 0 && longest > 2 * kSumKeys ? int(std::min<long long>(p->items, kBanks)) : 0;
  p->slots = int(slots);
  p->by_slots = Divisor(p->slots);
  return true;
}

size_t packed_workspace_bytes(const PackedParams& p) {
  if (p.chunk == 0) return p.banks > 0 ? kTakenBytes + size_t(p.banks) * 256 * p.d * 4 : 16;
  return size_t(p.items) * p.part_rows * (size_t(p.d) * 4 + 8);
}

cudaError_t packed_attn_tc(const PackedParams& p, cudaStream_t s) {
  if (p.pair) return packed_attn_pair(p, s);
  const cudaError_t e = p.d == 128 ? launch_tc<128, false>(p, s) : p.quarters ? launch_tc<64, true>(p, s) : launch_tc<64, false>(p, s);
  return e != cudaSuccess || p.chunk == 0 ? e : packed_join(p, true, s);
}

cudaError_t packed_join(const PackedParams& p, bool bf16, cudaStream_t s) {
  // as many blocks a token as fill the GPU twice, a turn of eight heads each at least
  const int turns = (p.H + 7) / 8, want = (2 * p.sms + p.Tq - 1) / p.Tq, each = want < turns ? want : turns;
  auto go = [&](auto kern) { return launch_overlapped(kern, dim3(unsigned(p.Tq), unsigned(each)), 256, 0, s, 0, p, walk_of(p)); };
  if (bf16) return p.d == 128 ? go(packed_join_kernel<128, __nv_bfloat16>) : go(packed_join_kernel<64, __nv_bfloat16>);
  return p.d == 128 ? go(packed_join_kernel<128, float>) : go(packed_join_kernel<64, float>);
}

}  // namespace mcs
