// First step of projections with low-rank adapters, bf16: h = scale_a x down_a^T for every segment's rows on the
// tensor cores, as slabs for the product (adapters.h).
//
// A cluster of 1 to 8 CTAs takes 128 rows of one slab, each CTA a slice of K: 64-column steps of the segment's rows of
// x (boxes of 32 rows, only those that hold rows of the segment) and of down_a through a ring of TMA stages into one
// fp32 accumulator [128 rows x R] in tensor memory, whose sums the cluster joins through distributed shared memory,
// ranks in order. 192 threads: warp 0 copies, warp 1 MMAs, warps 2-5 look over their share of up_a meanwhile and
// then bring the accumulator out, all six add and write. Reading x once bounds it: 75,600 x 5,120 with rank 32 in 115 us
// = 6.7 TB/s, 32,768 x 1,536 with rank 64 in 25 us.
#include <algorithm>

#include "adapters.h"
#include "attn_tc.h"
#include "common.cuh"
#include "launch.cuh"
#include "linear_few.h"
#include "ptx.cuh"
#include "tc_common.cuh"
#include "tma.cuh"

namespace mcs {
namespace {

constexpr int kThreads = 192;
constexpr int kXTile = 128 * 128;
constexpr int kMaxStages = 8;
constexpr int kBarBytes = 256;

struct DownArgs {
  AdapterView v;
  const __nv_bfloat16* up;
  const float* scale;
  __nv_bfloat16* slab;
  __nv_bfloat16* mask;
  uint8_t* odd;
  long long up_elems;     // of one adapter
  int K, heads, col_mask, head_shift;
  int halves, splits, rn; // 128-row halves of a slab; R rounded up to the MMA's 16 columns
  int units;              // halves of all slabs; the clusters behind them only look over `up`
  int stages;
  uint32_t tmem_cols;
  uint32_t* status;
};

__device__ __forceinline__ bool not_finite(const uint4& w) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
  bool r = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) r |= (u[i] & 0x7f80u) == 0x7f80u || (u[i] & 0x7f800000u) == 0x7f800000u;
  return r;
}

__global__ void __launch_bounds__(kThreads, 2)
    adapters_down_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_d, const DownArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const int stage_bytes = kXTile + a.rn * 128;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + a.stages * stage_bytes);
  uint64_t* empty = full + kMaxStages;
  uint64_t* done = empty + kMaxStages;
  uint64_t* drain = done + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile uint32_t* failed = tmem_slot + 1;
  const int tid = threadIdx.x, warp = warp_uniform(tid >> 5), lane = tid & 31;
  const int unit = blockIdx.x / a.splits, rank = blockIdx.x - unit * a.splits;  // of the cluster {splits, 1, 1}
  const int slot = unit / a.halves, half = unit - slot * a.halves;
  uint32_t* st = a.status;
  const AdapterView& v = a.v;
  if (tid == 0) {
    for (int s = 0; s < a.stages; ++s) mbar_init(full + s, 1), mbar_init(empty + s, 1);
    mbar_init(done, 1), mbar_init(drain, 1);
    *failed = 0;
    fence_mbar_init();
    tma_prefetch_map(&map_x), tma_prefetch_map(&map_d);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, a.tmem_cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = warp_uniform(*tmem_slot);
  grid_inputs_ready();
  grid_let_next_start();

  if (warp == 0) {  // bad bounds and adapters are flagged, each by one block
    for (long long s = static_cast<long long>(blockIdx.x) * 32 + lane; s < v.S; s += static_cast<long long>(gridDim.x) * 32) {
      int x, y;
      if (!segment_rows(v.start, int(s), v.M, x, y) || v.which[s] >= v.count) raise_status(st, kStatusBounds);
    }
    __syncwarp();
  }
  // The segment of this slot: the last whose first slot is not above it; every warp finds it for itself.
  int seg = -1, ad = -1, rt = 0, ra = 0, rb = 0, r0 = 0, r1 = 0;
  if (unit < a.units) {
    int lo = 0, n = v.S;
    while (true) {
      const int jump = (n + 31) >> 5, at = lane * jump;
      const bool ok = at < n && v.tiles.of(max(0, min(v.start[lo + at], v.M))) + lo + at <= slot;
      const int c = __popc(__ballot_sync(0xffffffffu, ok));
      if (c == 0) break;
      lo += (c - 1) * jump;
      n = min(jump, n - (c - 1) * jump);
      if (jump == 1) {
        seg = lo;
        break;
      }
    }
  }
  bool live = seg >= 0 && segment_rows(v.start, seg, v.M, ra, rb) && ra < rb;
  if (live) {
    rt = slot - seg;
    live = rt >= v.tiles.of(ra) && rt <= v.tiles.of(rb - 1);
    ad = v.which[seg];
    live = live && ad >= 0 && ad < v.count;
  }
  int share = live ? ((rt - v.tiles.of(ra)) * a.halves + half) * a.splits + rank : -1;  // of the adapter's `up`
  if (unit >= a.units) {
    const int more = v.more_shares / a.splits;  // clusters a segment
    seg = (unit - a.units) / more;
    if (segment_rows(v.start, seg, v.M, ra, rb) && ra < rb) {
      ad = v.which[seg];
      if (ad >= 0 && ad < v.count)
        share = (v.tiles.of(rb - 1) - v.tiles.of(ra) + 1) * v.halves_splits + (unit - a.units - seg * more) * a.splits + rank;
    }
  }
  // rows of this half of the slab that are the segment's, counted from the half's first row
  const int height = min(128, v.tiles.height - half * 128);
  if (live) {
    const int first = v.tiles.first(rt) + half * 128;
    r0 = max(0, min(ra - first, height));
    r1 = max(0, min(min(rb, v.tiles.end(rt)) - first, height));
    if (r1 < r0) r1 = r0;
  }
  const bool rows = live && r1 > r0;
  const int nk = (a.K + 63) / 64;
  const int k_beg = int(static_cast<long long>(nk) * rank / a.splits), k_end = int(static_cast<long long>(nk) * (rank + 1) / a.splits);

  bool ok = true;
  if (warp == 0 && rows) {
    const int sec = v.tiles.by_tiles.div(rt), row = (rt - sec * v.tiles.tiles) * v.tiles.height + half * 128, z0 = sec * a.heads;
    const int b0 = r0 / 32, b1 = (r1 + 31) / 32;  // boxes of 32 rows
    const uint32_t bytes = uint32_t((b1 - b0) * 32 * 128 + a.rn * 128);
    int s = 0;
    uint32_t phase = 0;
    for (int i = k_beg; i < k_end; ++i) {
      if (!(ok = warp_all(mbar_wait(empty + s, phase ^ 1, st)))) break;
      const int k = i * 64;
      const uint32_t dst = sbase + s * stage_bytes;
      if (elect_one()) {
        mbar_arrive_expect_tx(full + s, bytes);
        tma_load_3d(dst + kXTile, &map_d, k, 0, ad, smem_u32(full + s));
        for (int b = b0; b < b1; ++b)
          tma_load_3d(dst + b * 32 * 128, &map_x, k & a.col_mask, row + b * 32, z0 + (k >> a.head_shift), smem_u32(full + s));
      }
      __syncwarp();
      if (++s == a.stages) s = 0, phase ^= 1;
    }
    if (!ok) {
      if (lane == 0) {
        *failed = 1;
        raise_status(st, kStatusTimeout);
      }
      settle_copies();  // normally the MMAs have consumed every copy before the CTA exits
    }
    __syncwarp();
  } else if (warp == 1 && rows) {
    const uint32_t idesc = idesc_bf16_f32(128, 0, 0, 0) | (uint32_t(a.rn >> 3) << 17);
    int s = 0;
    uint32_t phase = 0;
    bool issued = false;
    for (int i = k_beg; i < k_end; ++i) {
      if (!(ok = warp_all(mbar_wait(full + s, phase, st)))) break;
      tc_fence_after();
      issued = true;
      const uint32_t x = desc_lo_kmajor(sbase + s * stage_bytes), d = desc_lo_kmajor(sbase + s * stage_bytes + kXTile);
      if (elect_one()) {
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
          tc_mma_ss_lo(tmem, x + kstep_kmajor(ks), d + kstep_kmajor(ks), idesc, (i > k_beg || ks > 0) ? 1u : 0u);
        tc_commit(empty + s);
        if (i == k_end - 1) tc_commit(done);
      }
      __syncwarp();
      if (++s == a.stages) s = 0, phase ^= 1;
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
    }
    __syncwarp();
  } else if (warp >= 2) {
    if (const int shares = share >= 0 ? up_shares(v, ra, rb) : 0; share >= 0 && share < shares) {
      const long long words = a.up_elems / 8;  // R is a multiple of 8
      const long long w0 = words * share / shares, w1 = words * (share + 1) / shares;
      const uint4* up = reinterpret_cast<const uint4*>(a.up + size_t(ad) * a.up_elems);
      bool odd = false;
      // sixteen reads in flight
      for (long long w = w0 + tid - 64; w < w1; w += 16 * 128) {
        uint4 x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = w + i * 128 < w1 ? __ldg(up + w + i * 128) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < 16; ++i) odd |= not_finite(x[i]);
      }
      // warps 2 to 5 meet on their own barrier
      uint32_t any;
      asm volatile("{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n bar.red.or.pred q, 1, 128, p;\n selp.u32 %0, 1, 0, q;\n}\n"
                   : "=r"(any)
                   : "r"(uint32_t(odd))
                   : "memory");
      if (tid == 64) a.odd[size_t(seg) * kAdapterPieces + share] = uint8_t(any);
    }
    if (rows) {
      if ((ok = warp_all(mbar_wait(done, 0, st)))) {
        tc_fence_after();
        // every stage has been read: the sums take the ring's place, [column][128 rows]
        const int quarter = warp & 3;
        float* part = reinterpret_cast<float*>(smem) + quarter * 32 + lane;
        for (int c = 0; c < a.rn; c += 16) {
          uint32_t r[16];
          tmem_ld16(tmem + (uint32_t(quarter * 32) << 16) + c, r);
#pragma unroll
          for (int i = 0; i < 16; ++i) part[(c + i) * 128] = __uint_as_float(r[i]);
        }
      } else if (lane == 0) {
        *failed = 1;
        raise_status(st, kStatusTimeout);
      }
    }
  }
  tc_fence_before();
  if (a.splits > 1) cluster_sync();
  else __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, a.tmem_cols);
  }
  if (live) {
    ok = true;
    for (int r = 0; r < a.splits && a.splits > 1; ++r) {
      uint32_t f;
      asm volatile("ld.shared::cluster.b32 %0, [%1];" : "=r"(f) : "r"(cluster_map(smem_u32(tmem_slot + 1), r)) : "memory");
      ok = ok && f == 0;
    }
    ok = ok && *failed == 0;
    // this CTA's share: 8 columns of a row a thread, rows fastest; a failed cluster leaves its slab as it was
    const int pieces = v.R / 8, todo = pieces * height;
    const float sc = a.scale[ad];
    const size_t slab = (static_cast<size_t>(slot) * 2 * v.tiles.height + half * 128) * v.R;
    const size_t part_elems = static_cast<size_t>(v.tiles.height) * v.R;
    for (int e = rank * kThreads + tid; ok && e < todo; e += a.splits * kThreads) {
      const int c8 = e / height, row = e - c8 * height;
      float h[8] = {};
      if (row >= r0 && row < r1) {
        for (int r = 0; r < a.splits; ++r) {
          const uint32_t at = sbase + uint32_t((c8 * 8) * 128 + row) * 4;
          const uint32_t from = a.splits > 1 ? cluster_map(at, r) : at;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            float f;
            if (a.splits > 1) asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(f) : "r"(from + i * 512) : "memory");
            else asm volatile("ld.shared.f32 %0, [%1];" : "=f"(f) : "r"(from + i * 512) : "memory");
            h[i] += f;
          }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] *= sc;  // only here: a scale that is not finite stays in its rows
      }
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float x = h[2 * i], y = h[2 * i + 1];
        hi[i] = pack_bf16x2(x, y);
        const float xh = __uint_as_float(hi[i] << 16), yh = __uint_as_float(hi[i] & 0xffff0000u);
        lo[i] = pack_bf16x2(isfinite(xh) ? x - xh : 0.f, isfinite(yh) ? y - yh : 0.f);
      }
      __nv_bfloat16* dst = a.slab + slab + static_cast<size_t>(row) * v.R + c8 * 8;
      *reinterpret_cast<uint4*>(dst) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
      *reinterpret_cast<uint4*>(dst + part_elems) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
    if (rank == 0 && tid < height) {
      const uint32_t nan = tid >= r0 && tid < r1 ? 0x7fffu : 0u;
      *reinterpret_cast<uint4*>(a.mask + (static_cast<size_t>(slot) * v.tiles.height + half * 128 + tid) * 8) = make_uint4(nan, 0, 0, 0);
    }
  }
  if (a.splits > 1) cluster_sync();  // the other CTAs may still be reading this one's sums
}

size_t align256(size_t n) { return (n + 255) & ~size_t(255); }

}  // namespace

// bf16: slabs, masks and the bytes of `up`'s shares, for row tiles of any height up to 256 (h and the rows' adapters are
// smaller): which kernel and tile a product takes depends on the device, and this is asked for without one. fp32: h, the adapters' part of the sums and the
// rows' adapters.
size_t adapters_workspace_bytes(const LinearParams& p, const AdapterParams& a, bool bf16) {
  if (!bf16) return align256(size_t(p.M) * a.R * 4) + align256(size_t(p.M) * p.O * 4) + align256(size_t(p.M) * 4);
  const size_t sections = p.heads > 0 ? p.B : 1;
  const size_t rows = size_t(p.M) + (sections + a.S) * 256;  // of all slabs
  return align256(rows * 2 * a.R * 2) + align256(rows * 8 * 2) + align256(size_t(a.S) * kAdapterPieces);
}

cudaError_t adapters_down_tc(const LinearParams& p, const AdapterParams& a, const RowTiles& t, int box, int wbox, int num_sms,
                             int free_sms, AdapterArgs<kAdapterSteps>* args, cudaStream_t s) {
  DownArgs d{};
  const size_t slots = size_t(t.tiles) * t.sections + a.S, rows = slots * t.height;
  d.halves = (t.height + 127) / 128;
  d.rn = (a.R + 15) / 16 * 16;
  d.K = p.K;
  d.heads = p.heads;
  // K slices of four steps at least; slots that hold nothing leave at once. Beside a product that leaves SMs free (its blocks take
  // an SM each and would wait for these) two blocks on each of those: 452 x 4,096 -> 5,120 with two adapters 27 us with
  // eight slices, 25 with four or two. Where two slices have no room there, the product waits for the sums anyway, and two blocks
  // on every SM bring them soonest (512 x 4,096 -> 9,472 with two adapters of rank 256 220 us with one slice, 68 with
  // more, 52 with the blocks below).
  const int nk = (p.K + 63) / 64;
  const long long units = static_cast<long long>(slots) * d.halves;
  const bool beside = units * 2 <= 2ll * free_sms;
  const long long most = 2ll * (beside ? free_sms : num_sms);
  d.splits = 1;
  while (d.splits < 8 && units * d.splits * 2 <= most && nk >= d.splits * 2 * 4) d.splits *= 2;
  // Clusters that only look over `up`, as many a segment as give shares of 16 KB, where the SMs have room (beside a product one on
  // each, as blocks go to empty SMs first, unless the shares are long without them: 512 x 4,096 -> 8,960, rank 32, 38 us with two and
  // 31 with one, 256 x 1,536 -> 8,960, rank 128, 26 us with two and 36 with none).
  const long long up_bytes = static_cast<long long>(p.O) * a.R * 2;
  const long long room = (beside && up_bytes / (d.halves * d.splits) < 160 * 1024 ? free_sms : most) - units * d.splits;
  const long long want = std::min<long long>(kAdapterPieces, up_bytes >> 14) - d.halves * d.splits;
  const int more = int(std::max(0ll, std::min(want / d.splits, room / (static_cast<long long>(a.S) * d.splits))));
  d.units = int(units);
  const long long grid = (units + static_cast<long long>(more) * a.S) * d.splits;
  if (grid > INT32_MAX) return cudaErrorInvalidValue;
  const int stage = kXTile + d.rn * 128;
  const int per_rank = (nk + d.splits - 1) / d.splits;
  d.stages = std::min({kMaxStages, (108 * 1024) / stage, std::max(2, per_rank)});
  while (d.stages * stage < d.rn * 512) ++d.stages;  // the ring ends up holding the sums
  d.tmem_cols = 32;
  while (int(d.tmem_cols) < d.rn) d.tmem_cols *= 2;
  char* ws = static_cast<char*>(a.ws);
  const size_t rows_all = size_t(p.M) + (size_t(t.sections) + a.S) * 256;
  d.slab = reinterpret_cast<__nv_bfloat16*>(ws);
  d.mask = reinterpret_cast<__nv_bfloat16*>(ws + align256(rows_all * 2 * a.R * 2));
  d.odd = reinterpret_cast<uint8_t*>(ws + align256(rows_all * 2 * a.R * 2) + align256(rows_all * 8 * 2));
  if (rows > rows_all) return cudaErrorInvalidValue;
  d.v = {a.start, a.which, d.odd, a.count, a.R, a.S, p.M, d.halves * d.splits, more * d.splits, t, Divisor(1)};
  d.up = static_cast<const __nv_bfloat16*>(a.up);
  d.up_elems = static_cast<long long>(p.O) * a.R;
  d.scale = a.scale;
  d.status = p.status;
  CUtensorMap mx, md;
  bool ok;
  if (p.heads > 0) {
    const int hd = p.K / p.heads;
    d.head_shift = hd == 64 ? 6 : 7;
    d.col_mask = hd - 1;
    ok = make_tile_map(&mx, p.x, uint64_t(p.B) * p.heads, p.N, hd, 32);
  } else {
    d.head_shift = 31;
    d.col_mask = INT32_MAX;
    ok = make_tile_map(&mx, p.x, 1, p.M, p.K, 32);
  }
  ok = ok && make_tile_map(&md, a.down, a.count, a.R, p.K, d.rn) && make_tile_map(&args->h, d.slab, 2 * slots, t.height, a.R, box) &&
       make_tile_map(&args->mask, d.mask, slots, t.height, 8, box) && make_tile_map(&args->up, a.up, a.count, p.O, a.R, wbox);
  if (!ok) return cudaErrorInvalidValue;
  args->v = d.v;
  const size_t smem = size_t(d.stages) * stage + kBarBytes + 1024;
  const cudaError_t e = allow_smem<adapters_down_kernel>(226 * 1024);
  if (e != cudaSuccess) return e;
  return launch_overlapped(adapters_down_kernel, dim3(unsigned(grid)), kThreads, smem, s, unsigned(d.splits), mx, md, d);
}

}  // namespace mcs
