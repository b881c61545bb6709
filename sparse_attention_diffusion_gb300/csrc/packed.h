// Host-side interface of attention over packed sequences, and the walk over its work that
// the bf16 and fp32 kernels share.
//
// Sequence s holds queries q_start[s] .. q_start[s + 1] - 1 and keys k_start[s] .. k_start[s + 1] - 1.
// A tile is `rows` rows of one key head: `tq` tokens with the `g` query heads that read that
// head, row = token * g + head, so that a group's heads share every key that is loaded, in long
// prompts and for single tokens alike. The offsets live on the device, so the tiles are found there
// without a planning launch: slot(s, i) = start[s] / unit + s + i is another number for every tile i
// (or chunk i of keys) of every sequence s, all below start[S] / unit + S, and s is found again
// by a search over start[s] / unit + s, which rises strictly. Slots that no tile takes are skipped. Up to 32 sequences
// need no search: a warp's lanes hold them.
#pragma once
#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "divisor.h"

namespace mcs {

// The tensor core adds into its fp32 sums by truncation, a step of 16 keys after another: the sums of 2^20 keys with equal weights came
// out 0.5 % too small, of 2^22 2.6 %. So no sum takes more than 2^18 keys: pieces of sequences have 2^17 at most, and a kernel that
// may meet longer sequences whole empties its sums every kSumTiles tiles into fp32 memory of its block (a bank), adding to nearest.
constexpr int kSumKeys = 1 << 17, kSumTiles = kSumKeys / 128;
constexpr int kBanks = 152;  // blocks that may have one
constexpr int kTakenBytes = 256;  // before the banks: the items' counter

struct PackedStrides {
  long long head, token;  // elements
};
struct PackedParams {
  const void* q;
  const void* k;
  const void* v;
  void* o;
  float* lse;             // [H, Tq] or null
  const int32_t* q_start; // [S + 1]
  const int32_t* k_start;
  PackedStrides qs, ks, vs, os;
  int S, Tq, Tk, H, Hk, g, d;
  int causal, max_q;
  float scale_log2;       // scale * log2(e)
  int tq, rows;           // tokens and rows (tq * g) of a tile (of two tiles: pair)
  int part_rows;          // rows of a tile that can hold a token, for which there are partial sums
  int pair;               // bf16, two tiles of 128 rows an item
  int quarters;           // bf16, d = 64, items of 32 rows at most: every softmax warp a quarter of the keys
  int chunk;              // keys of a piece of a sequence, 0: sequences are not cut
  int tiles;              // with chunk > 0: query tiles of the longest sequence
  int banks;              // blocks that need a bank each: [bank][2][128 rows][d] in part_o; 0: none
  long long items;        // slots of all heads (and tiles)
  Divisor by_heads, by_tiles, by_group, by_slots;
  int slots;
  float* part_o;          // with chunk > 0: [slot][tile][Hk][part_rows][d] sums, not divided
  float2* part_ml;        // [slot][tile][Hk][part_rows] (maximum in log2 units, sum)
  uint32_t* taken;        // with banks: items that blocks have taken after their own
  uint32_t* status;
  int sms;                // of the device
};

// Fills the tiles, chunks and item counts for sequences of up to `longest` keys; false where they do not fit in 31 bits.
bool plan_packed(PackedParams* p, bool bf16, int longest);
size_t packed_workspace_bytes(const PackedParams& p);
cudaError_t packed_attn_tc(const PackedParams& p, cudaStream_t s);
cudaError_t packed_attn_pair(const PackedParams& p, cudaStream_t s);
cudaError_t packed_attn_f32(const PackedParams& p, cudaStream_t s);
cudaError_t packed_join(const PackedParams& p, bool bf16, cudaStream_t s);

#ifdef __CUDACC__
// A tile (or its share of a sequence's keys) as the kernels work it off.
struct PackedItem {
  int q0, ntok;   // first token in the packed queries, tokens
  int k0, nkeys;  // first key, keys that any of its rows sees
  int lim;        // keys that its first token sees, from k0 on (not clamped); all see nkeys without a mask
  int hk;         // key head
  int tiles;      // of 128 keys; -1: no more items
  int whole;      // it has all keys that its rows see
  long long part; // row in the partial sums
};
// Keys from the item's first that token t of it sees.
__device__ __forceinline__ int visible_keys(const PackedItem& it, int causal, int t) {
  return causal ? max(0, min(it.nkeys, it.lim + t)) : it.nkeys;
}

// The sequence whose slots hold `slot`: the last s with start[s] / unit + s * step <= slot, or -1. One warp.
__device__ __forceinline__ int packed_find(const int32_t* start, int S, Divisor unit, int step, int slot, int lane) {
  int lo = 0, n = S;
  while (true) {
    const int jump = (n + 31) >> 5;
    const int at = lane * jump;
    const bool ok = at < n && unit.div(max(0, start[lo + at])) + (lo + at) * step <= slot;
    const int c = __popc(__ballot_sync(0xffffffffu, ok));
    if (c == 0) return lo == 0 ? -1 : lo;
    lo += (c - 1) * jump;
    n = min(jump, n - (c - 1) * jump);
    if (jump == 1) return lo;
  }
}
__device__ __forceinline__ bool packed_sequence(const PackedParams& p, int s, int& a, int& nq, int& k0, int& nk) {
  a = p.q_start[s], k0 = p.k_start[s];
  const int qe = p.q_start[s + 1], ke = p.k_start[s + 1];
  const bool ok = a >= 0 && qe >= a && qe <= p.Tq && k0 >= 0 && ke >= k0 && ke <= p.Tk && qe - a <= p.max_q;
  nq = ok ? qe - a : 0, nk = ok ? ke - k0 : 0;
  return ok;
}
// Up to 32 sequences lie in a warp's lanes, the ones with the most keys first in the walk, so that blocks end with short
// items: three clips of 20,000 tokens and less, in the order they came in, left the SMs idle for a fifth of the time.
struct PackedLane {
  int q0, nq, k0, nk;
  long long first, count;  // items before this sequence's, and its own
};
__device__ __forceinline__ PackedLane packed_lane(const PackedParams& p, const Divisor& by_tq, const Divisor& by_chunk, int lane) {
  PackedLane s{};
  if (lane < p.S) packed_sequence(p, lane, s.q0, s.nq, s.k0, s.nk);
  s.count = static_cast<long long>(by_tq.div(s.nq + p.tq - 1)) * p.Hk * (p.chunk > 0 ? by_chunk.div(s.nk + p.chunk - 1) : 1);
#pragma unroll 1
  for (int l = 0; l < p.S; ++l) {
    const int nk = __shfl_sync(0xffffffffu, s.nk, l);
    const long long n = __shfl_sync(0xffffffffu, s.count, l);
    if (nk > s.nk || (nk == s.nk && l < lane)) s.first += n;
  }
  return s;
}
// Item i of the walk; false if nothing is to be done for it. One warp.
__device__ __forceinline__ bool packed_item(const PackedParams& p, const Divisor& by_tq, const Divisor& by_chunk, const PackedLane& mine,
                                            long long i, int lane, PackedItem* it) {
  int slot, iq = 0, nq, nk, k0, q0, c = 0;
  const Divisor& unit = p.chunk > 0 ? by_chunk : by_tq;
  if (p.S <= 32) {
    const uint32_t has = __ballot_sync(0xffffffffu, i >= mine.first && i < mine.first + mine.count);
    if (has == 0) return false;
    const int s = __ffs(has) - 1;
    q0 = __shfl_sync(0xffffffffu, mine.q0, s), nq = __shfl_sync(0xffffffffu, mine.nq, s);
    k0 = __shfl_sync(0xffffffffu, mine.k0, s), nk = __shfl_sync(0xffffffffu, mine.nk, s);
    const int r = int(i - __shfl_sync(0xffffffffu, mine.first, s)), ntiles = by_tq.div(nq + p.tq - 1);
    if (p.chunk > 0) {  // heads fastest: neighbours in memory are read at the same time
      const int j = p.by_heads.div(r);
      it->hk = r - j * p.Hk;
      c = j / ntiles;
      iq = j - c * ntiles;
      slot = unit.div(k0) + s + c;
    } else {  // tiles fastest: they read the same keys; those that see the most first
      it->hk = r / ntiles;
      iq = ntiles - 1 - (r - it->hk * ntiles);
      slot = 0;
    }
  } else {
    if (p.chunk > 0) {
      const int j = p.by_heads.div(int(i));
      it->hk = int(i) - j * p.Hk;
      slot = p.by_tiles.div(j);
      iq = j - slot * p.tiles;
    } else {
      it->hk = p.by_slots.div(int(i));
      slot = int(i) - it->hk * p.slots;
    }
    const int32_t* start = p.chunk > 0 ? p.k_start : p.q_start;
    const int s = packed_find(start, p.S, unit, 1, slot, lane);
    if (s < 0 || !packed_sequence(p, s, q0, nq, k0, nk)) return false;
    const int ntiles = by_tq.div(nq + p.tq - 1), n = slot - (unit.div(start[s]) + s);
    if (n < 0) return false;  // only where the bounds do not rise
    if (p.chunk > 0) c = n;
    else iq = ntiles - 1 - n;
    if (iq < 0 || iq >= ntiles) return false;
  }
  const int t0 = iq * p.tq;
  it->ntok = min(p.tq, nq - t0);
  it->q0 = q0 + t0;
  const int seen = p.causal ? max(0, min(nk, t0 + it->ntok + nk - nq)) : nk;  // by the last token
  const long long k_first = static_cast<long long>(c) * p.chunk;
  if (p.chunk > 0 && k_first >= seen) return false;
  it->k0 = k0 + int(k_first);
  it->nkeys = p.chunk > 0 ? min(p.chunk, seen - int(k_first)) : seen;
  it->whole = it->nkeys == seen;
  it->lim = t0 + 1 + nk - nq - int(k_first);
  it->tiles = (it->nkeys + 127) >> 7;
  it->part = ((static_cast<long long>(slot) * p.tiles + iq) * p.Hk + it->hk) * p.part_rows;
  return true;
}
#endif

}  // namespace mcs
