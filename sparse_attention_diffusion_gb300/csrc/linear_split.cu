// fp32 matrix product with epilogue on the bf16 tensor cores, with fp32's accuracy.
//
// Every fp32 number is the exact sum of three bf16 parts, h + m + l: it is rounded to
// bf16, then twice what is left (exact subtractions; two numbers a conversion), which takes
// as many instructions as cutting the bits off. Of the nine products of parts the six
// largest are summed; |m| < 2^-8 |x| and |l| <= 2^-17 |x| leave at most 1.01 * 2^-24 |x w|
// out, of either sign (parts cut off left out up to 2^-20, always towards 0). A number
// keeps bits down to 2^-133 only, bf16's last. The tensor core adds into its fp32
// accumulator by truncation (measured on this GPU: two bits below the sum's last one
// are kept), which over a long K would shrink the sum by 2^-24 a step or more. So an
// accumulator takes 32 columns of K only, small products first, and the epilogue's
// threads add it to fp32 sums in registers, rounding to nearest.
//
// One CTA per 128 x 128 tile, 576 threads:
//   warp 0        TMA producer: fp32 tiles of 32 columns, four stages
//   warp 1        tensor-memory allocation and MMA issue: 12 MMAs a step
//   warps 2-9     cut the fp32 tiles into parts, in the layout the MMA reads: those of x
//                 go to tensor memory (the MMA's A operand), those of w to shared memory,
//                 rows of 128 bytes with h and m of the 32 columns and a second tile for l
//   warps 10-17   sums: two threads a row, 64 columns each
// Accumulators and parts are double-buffered. Shared memory's bandwidth bounds a step:
// 32 KB in, 32 KB read, 24 KB of parts written and 48 KB read by the MMAs, 1,088 clocks
// at 128 bytes each, against 768 of MMAs (with the parts of x in shared memory too,
// 1,664 clocks; 4,096 x 5,120 x 5,120 took 1.22 ms).
// Few tiles are cut along K over the CTAs of a cluster, which join their sums through
// distributed shared memory, ranks in order, so that equal calls give equal bits.
// Outputs that come out infinite or NaN are summed again on the CUDA cores.
//
// Measured: 4,096 x 5,120 -> 5,120 outputs 0.85 ms (252 TFLOP/s; 1,140 clocks a step;
// the CUDA cores' 128 x 128 tiles of packed FMAs took 3.89 ms), 1,024 x 1,536 -> 1,536 33
// us, 300 x 3,200 -> 320 15 us in eight slices; relative error of the result 0.5e-7 to
// 1.4e-7 over K = 4 .. 5,120 (fp32 FMAs in order: 0.4e-7 to 13e-7).
#include "attn_tc.h"
#include "common.cuh"
#include "launch.cuh"
#include "linear.h"
#include "linear_epi.cuh"
#include "ptx.cuh"
#include "tc_common.cuh"
#include "tma.cuh"

namespace mcs {
namespace {

constexpr int kThreads = 576, kWarps = kThreads / 32;
constexpr int kCutWarps = 8, kSumWarps = 8;
constexpr int kBK = 32;
constexpr int kTile = 128 * 128;            // bytes of a 128-row tile of 128-byte rows
constexpr int kRawStages = 4;
constexpr int kRaw = 2 * kTile;             // fp32 stage: x, w
constexpr int kParts = 2 * kTile;           // bf16 stage: w h|m, w l
constexpr int kPartsOff = kRawStages * kRaw;
constexpr int kBarOff = kPartsOff + 2 * kParts;
constexpr int kSmemAlloc = kBarOff + 256 + 1024;
constexpr uint32_t kColX = 256;             // tensor memory: accumulators [0, 256), parts of x [256, 384)
constexpr int kSumLd = 132;                 // floats a row of the final sums takes in shared memory
static_assert(128 * kSumLd * 4 <= kBarOff, "the sums fit over the stages");

struct SplitArgs {
  int rows, tiles;            // rows of a section of x (as in the bf16 kernels), its row tiles
  int col_mask, head_shift;
  int splits;
};

// Cuts eight fp32 numbers into their parts: 16 bytes of h, m and l.
__device__ __forceinline__ void cut8(const float4& a, const float4& b, uint4& h, uint4& m, uint4& l) {
  const float x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  uint32_t hw[4], mw[4], lw[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float u = x[2 * i], v = x[2 * i + 1];
    hw[i] = pack_bf16x2(u, v);
    u -= __uint_as_float(hw[i] << 16), v -= __uint_as_float(hw[i] & 0xffff0000u);
    mw[i] = pack_bf16x2(u, v);
    u -= __uint_as_float(mw[i] << 16), v -= __uint_as_float(mw[i] & 0xffff0000u);
    lw[i] = pack_bf16x2(u, v);
  }
  h = make_uint4(hw[0], hw[1], hw[2], hw[3]);
  m = make_uint4(mw[0], mw[1], mw[2], mw[3]);
  l = make_uint4(lw[0], lw[1], lw[2], lw[3]);
}
__device__ __forceinline__ float4 lds4(uint32_t at) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ void sts4(uint32_t at, const uint4& v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// A row's four sums of a lane, joined over the K slices (ranks in order).
__device__ __forceinline__ void joined_sums(const SplitArgs& a, uint32_t sbase, int r, int lane, float (&v)[4]) {
  const uint32_t at = sbase + (r * kSumLd + lane * 4) * 4;
  v[0] = v[1] = v[2] = v[3] = 0.f;
  if (a.splits == 1) {
    const float4 f = lds4(at);
    v[0] = f.x, v[1] = f.y, v[2] = f.z, v[3] = f.w;
  } else {
    float f[4][4];
    for (int c0 = 0; c0 < a.splits; c0 += 4) {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        f[c][0] = f[c][1] = f[c][2] = f[c][3] = 0.f;
        if (c0 + c < a.splits)
          asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                       : "=f"(f[c][0]), "=f"(f[c][1]), "=f"(f[c][2]), "=f"(f[c][3])
                       : "r"(cluster_map(at, c0 + c)));
      }
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] += f[c][i];
    }
  }
}

// Not finite if one of the four is not (or if they are very large).
__device__ __forceinline__ float sum4(const float (&v)[4]) { return (v[0] + v[1]) + (v[2] + v[3]); }

// The outputs whose sum over the parts is not finite, summed again in fp32 on the CUDA cores: an infinite element
// has no parts (infinity less infinity), nor has one that bf16 rounds to infinity (3.39e38 and more); here they
// give what their products and sums are. A function of its own, with the parameters left in constant memory, so
// that the ordinary way out keeps its registers (20,000 x 200 -> 1,000 86 -> 88 us with it, 92 inline; 4,096 x
// 5,120 -> 5,120 874 -> 880 us).
template <int kAct>
__device__ __noinline__ void finish_not_finite(const LinearParams& p, const SplitArgs& a, uint32_t sbase, int sec, int row0,
                                               int live, int o0, int rank, int warp, int lane) {
  const int d = p.heads > 0 ? p.K / p.heads : p.K, o = o0 + lane * 4;
  const size_t head = size_t(a.rows) * d;
  for (int r = rank + a.splits * warp; r < live; r += a.splits * kWarps) {
    float v[4];
    joined_sums(a, sbase, r, lane, v);
    const bool bad = o < p.O && !isfinite(sum4(v));
    const float* x = static_cast<const float*>(p.x) + size_t(sec) * (p.heads > 0 ? p.heads : 1) * head + size_t(row0 + r) * d;
    for (uint32_t left = __ballot_sync(0xffffffffu, bad); left != 0; left &= left - 1) {
      const int owner = __ffs(left) - 1, first = o0 + owner * 4;  // the warp sums the four outputs of one lane
      const float* w[4];
      float t[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = static_cast<const float*>(p.w) + size_t(min(first + i, p.O - 1)) * p.K;
#pragma unroll 2
      for (int k0 = 0; k0 < p.K; k0 += 128) {
        const int k = k0 + lane * 4;
        if (k < p.K) {
          const float4 f = *reinterpret_cast<const float4*>(x + (k >> a.head_shift) * head + (k & a.col_mask));
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float4 g = *reinterpret_cast<const float4*>(w[i] + k);
            t[i] = fmaf(f.w, g.w, fmaf(f.z, g.z, fmaf(f.y, g.y, fmaf(f.x, g.x, t[i]))));
          }
        }
        // NaN stays, so a NaN in x ends its row here
        if (__any_sync(0xffffffffu, isnan(t[0]) && isnan(t[1]) && isnan(t[2]) && isnan(t[3]))) break;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int n = 16; n > 0; n >>= 1) t[i] += __shfl_xor_sync(0xffffffffu, t[i], n);
        if (lane == owner && !isfinite(v[i])) v[i] = t[i];
      }
    }
    if (bad) finish_row4<kAct>(p, sec * a.rows + row0 + r, o, v);
  }
}

template <int kAct>
__global__ void __launch_bounds__(kThreads, 1)
    linear_split_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w,
                        const __grid_constant__ LinearParams p, const __grid_constant__ SplitArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  uint64_t* raw_full = reinterpret_cast<uint64_t*>(smem + kBarOff);  // [kRawStages], like raw_empty; the others [2]
  uint64_t* raw_empty = raw_full + kRawStages;
  uint64_t* parts_full = raw_empty + kRawStages;
  uint64_t* parts_empty = parts_full + 2;
  uint64_t* acc_full = parts_empty + 2;
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* drain = acc_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  uint32_t* failed = tmem_slot + 1;  // a wait of this CTA ran out
  const int tid = threadIdx.x, warp = warp_uniform(tid >> 5), lane = tid & 31;
  const int rt = blockIdx.x / a.splits, rank = blockIdx.x % a.splits;  // of the cluster {splits, 1, 1}
  const int sec = rt / a.tiles, row0 = (rt % a.tiles) * 128, o0 = blockIdx.y * 128;
  const int nk = (p.K + kBK - 1) / kBK;
  const int k_beg = int(static_cast<long long>(nk) * rank / a.splits);
  const int steps = int(static_cast<long long>(nk) * (rank + 1) / a.splits) - k_beg;
  uint32_t* st = p.status;
  if (tid == 64) {
    tma_prefetch_map(&map_x);
    tma_prefetch_map(&map_w);
  }
  if (tid == 0) {
    for (int b = 0; b < kRawStages; ++b) {
      mbar_init(raw_full + b, 1);
      mbar_init(raw_empty + b, kCutWarps);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(parts_full + b, kCutWarps);
      mbar_init(parts_empty + b, 1);
      mbar_init(acc_full + b, 1);
      mbar_init(acc_empty + b, kSumWarps);
    }
    mbar_init(drain, 1);
    *reinterpret_cast<volatile uint32_t*>(failed) = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = warp_uniform(*tmem_slot);
  grid_inputs_ready();
  grid_let_next_start();

  bool ok = true;
  float2 sum[32];  // sum warps: this thread's 64 columns
  if (warp == 0) {
    const int z0 = sec * p.heads;
    for (int i = 0; i < steps; ++i) {
      const int s = i % kRawStages;
      if (!(ok = warp_all(mbar_wait(raw_empty + s, ((i / kRawStages) & 1) ^ 1, st)))) break;
      const int k = (k_beg + i) * kBK;
      const uint32_t dst = sbase + s * kRaw;
      if (elect_one()) {
        mbar_arrive_expect_tx(raw_full + s, kRaw);
        tma_load_3d(dst, &map_x, k & a.col_mask, row0, z0 + (k >> a.head_shift), smem_u32(raw_full + s));
        tma_load_3d(dst + kTile, &map_w, k, o0, 0, smem_u32(raw_full + s));
      }
      __syncwarp();
    }
    if (!ok) settle_copies();  // normally the cutting warps have read every copy before the CTA exits
  } else if (warp == 1) {
    constexpr uint32_t kIdesc = idesc_bf16_f32(128, 128, 0, 0);
    bool issued = false;
    for (int i = 0; i < steps; ++i) {
      const int s = i & 1;
      const uint32_t phase = (i >> 1) & 1;
      ok = warp_all(mbar_wait(parts_full + s, phase, st)) && warp_all(mbar_wait(acc_empty + s, phase ^ 1, st));
      if (!ok) break;
      tc_fence_after();
      issued = true;
      const uint32_t base = sbase + kPartsOff + s * kParts;
      const uint32_t whm = desc_lo_kmajor(base), wl = desc_lo_kmajor(base + kTile);
      const uint32_t xh = tmem + kColX + s * 64, xm = xh + 16, xl = xh + 32;
      if (elect_one()) {
        const uint32_t d = tmem + s * 128;
#pragma unroll
        for (int ks = 0; ks < 2; ++ks)  // m m
          tc_mma_ts_lo(d, xm + ks * 8, whm + kstep_kmajor(2 + ks), kIdesc, ks > 0 ? 1u : 0u);
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) tc_mma_ts_lo(d, xh + ks * 8, wl + kstep_kmajor(ks), kIdesc, 1u);       // h l
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) tc_mma_ts_lo(d, xl + ks * 8, whm + kstep_kmajor(ks), kIdesc, 1u);      // l h
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) tc_mma_ts_lo(d, xh + ks * 8, whm + kstep_kmajor(2 + ks), kIdesc, 1u);  // h m
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) tc_mma_ts_lo(d, xm + ks * 8, whm + kstep_kmajor(ks), kIdesc, 1u);      // m h
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) tc_mma_ts_lo(d, xh + ks * 8, whm + kstep_kmajor(ks), kIdesc, 1u);      // h h
        tc_commit(parts_empty + s);
        tc_commit(acc_full + s);
      }
      __syncwarp();
    }
    if (!ok && issued) {
      if (elect_one()) tc_commit(drain);
      __syncwarp();
      mbar_drain(drain, 0);
    }
  } else if (warp < 2 + kCutWarps) {
    // a unit is eight numbers of a row: 16 bytes of each part; a warp takes the 32 rows of its tensor-memory
    // lanes and two of the four units of a row, of x and of w
    const int quarter = warp & 3, row = quarter * 32 + lane, j0 = ((warp - 2) >> 2) * 2;
    for (int i = 0; i < steps; ++i) {
      const int s = i & 1, rs = i % kRawStages;
      ok = warp_all(mbar_wait(raw_full + rs, (i / kRawStages) & 1, st)) &&
           warp_all(mbar_wait(parts_empty + s, ((i >> 1) & 1) ^ 1, st));
      if (!ok) break;
      tc_fence_after();
      const uint32_t src = sbase + rs * kRaw + row * 128;
      uint4 h[2], m[2], l[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int j = j0 + u;
        cut8(lds4(src + (((2 * j) ^ (row & 7)) << 4)), lds4(src + (((2 * j + 1) ^ (row & 7)) << 4)), h[u], m[u], l[u]);
      }
      const uint32_t xt = tmem + (uint32_t(quarter * 32) << 16) + kColX + s * 64 + j0 * 4;
      tmem_st8_nowait(xt, h[0], h[1]);
      tmem_st8_nowait(xt + 16, m[0], m[1]);
      tmem_st8_nowait(xt + 32, l[0], l[1]);
      const uint32_t dst = sbase + kPartsOff + s * kParts + row * 128;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int j = j0 + u;
        uint4 wh, wm, wl;
        cut8(lds4(src + kTile + (((2 * j) ^ (row & 7)) << 4)), lds4(src + kTile + (((2 * j + 1) ^ (row & 7)) << 4)), wh, wm, wl);
        sts4(dst + ((j ^ (row & 7)) << 4), wh);
        sts4(dst + (((4 + j) ^ (row & 7)) << 4), wm);
        sts4(dst + kTile + ((j ^ (row & 7)) << 4), wl);
      }
      tmem_wait_st();
      tc_fence_before();
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(parts_full + s);
        mbar_arrive(raw_empty + rs);
      }
    }
  } else {
    const int quarter = warp & 3, half = (warp - 2 - kCutWarps) >> 2;
#pragma unroll
    for (int i = 0; i < 32; ++i) sum[i] = make_float2(0.f, 0.f);
    for (int i = 0; i < steps; ++i) {
      const int s = i & 1;
      if (!(ok = warp_all(mbar_wait(acc_full + s, (i >> 1) & 1, st)))) break;
      tc_fence_after();
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t r[32];
        tmem_ld32(tmem + (uint32_t(quarter * 32) << 16) + s * 128 + half * 64 + c * 32, r);
#pragma unroll
        for (int q = 0; q < 16; ++q) {
          float2& v = sum[c * 16 + q];
          const uint64_t t =
              f2_add(f2_pack(v.x, v.y), f2_pack(__uint_as_float(r[2 * q]), __uint_as_float(r[2 * q + 1])));
          f2_unpack(t, v.x, v.y);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(acc_empty + s);
    }
  }
  if (!ok && lane == 0) {
    *reinterpret_cast<volatile uint32_t*>(failed) = 1;
    raise_status(st, kStatusTimeout);
  }
  // all MMAs are done once the sum warps are (the last accumulator's commit covers them): the stages are free
  __syncthreads();
  if (warp >= 2 + kCutWarps) {
    const int quarter = warp & 3, half = (warp - 2 - kCutWarps) >> 2;
    const uint32_t at = sbase + ((quarter * 32 + lane) * kSumLd + half * 64) * 4;
#pragma unroll
    for (int q = 0; q < 16; ++q)
      sts4(at + q * 16, make_uint4(__float_as_uint(sum[2 * q].x), __float_as_uint(sum[2 * q].y),
                                   __float_as_uint(sum[2 * q + 1].x), __float_as_uint(sum[2 * q + 1].y)));
  }
  tc_fence_before();
  if (a.splits > 1) cluster_sync();
  else __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  // sums with a failed CTA's share are not written anywhere
  ok = true;
  for (int r = 0; r < a.splits; ++r) {
    uint32_t f;
    if (a.splits == 1) asm volatile("ld.shared.b32 %0, [%1];" : "=r"(f) : "r"(smem_u32(failed)) : "memory");
    else asm volatile("ld.shared::cluster.b32 %0, [%1];" : "=r"(f) : "r"(cluster_map(smem_u32(failed), r)) : "memory");
    ok = ok && f == 0;
  }
  const int live = min(128, a.rows - row0), o = o0 + lane * 4;
  bool again = false;
#pragma unroll 1
  for (int r = rank + a.splits * warp; ok && r < live; r += a.splits * kWarps) {
    float v[4];
    joined_sums(a, sbase, r, lane, v);
    if (isfinite(sum4(v))) finish_row4<kAct>(p, sec * a.rows + row0 + r, o, v);
    else again = true;
  }
  if (__any_sync(0xffffffffu, again)) finish_not_finite<kAct>(p, a, sbase, sec, row0, live, o0, rank, warp, lane);
  if (a.splits > 1) cluster_sync();  // the other CTAs may still be reading this one's sums
}

template <int kAct>
cudaError_t start(const CUtensorMap& mx, const CUtensorMap& mw, const LinearParams& p, const SplitArgs& a, dim3 grid,
                  cudaStream_t s) {
  const cudaError_t e = allow_smem<linear_split_kernel<kAct>>(kSmemAlloc);
  if (e != cudaSuccess) return e;
  return launch_overlapped(linear_split_kernel<kAct>, grid, kThreads, kSmemAlloc, s, unsigned(a.splits), mx, mw, p, a);
}

}  // namespace

cudaError_t linear_split(const LinearParams& p, int splits, cudaStream_t s) {
  SplitArgs a{};
  CUtensorMap mx, mw;
  bool ok;
  int sections = 1;
  if (p.heads > 0) {
    const int d = p.K / p.heads;
    a.head_shift = d == 64 ? 6 : 7;
    a.col_mask = d - 1;
    a.rows = p.N;
    sections = p.B;
    ok = make_tile_map_f32(&mx, p.x, uint64_t(p.B) * p.heads, p.N, d, 128);
  } else {
    a.head_shift = 31;
    a.col_mask = INT32_MAX;
    a.rows = p.M;
    ok = make_tile_map_f32(&mx, p.x, 1, p.M, p.K, 128);
  }
  if (!(ok && make_tile_map_f32(&mw, p.w, 1, p.O, p.K, 128))) return cudaErrorInvalidValue;
  a.tiles = (a.rows + 127) / 128;
  a.splits = splits;
  const long long gx = static_cast<long long>(a.splits) * a.tiles * sections;
  if (gx > INT32_MAX) return cudaErrorInvalidValue;
  const dim3 grid(unsigned(gx), (p.O + 127) / 128);
  switch (p.act) {
    case MCS_ACT_GELU_TANH: return start<MCS_ACT_GELU_TANH>(mx, mw, p, a, grid, s);
    case MCS_ACT_GELU_ERF: return start<MCS_ACT_GELU_ERF>(mx, mw, p, a, grid, s);
    case MCS_ACT_SILU: return start<MCS_ACT_SILU>(mx, mw, p, a, grid, s);
    default: return start<MCS_ACT_NONE>(mx, mw, p, a, grid, s);
  }
}

}  // namespace mcs
