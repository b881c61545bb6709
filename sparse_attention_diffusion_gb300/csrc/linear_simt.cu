// fp32 matrix product with epilogue in SIMT arithmetic.
//
// Tiles: 128 x 128 outputs per CTA (8 x 8 a thread) or 64 x 64 (4 x 4 a thread),
// K in steps of 16 through two shared-memory buffers, the next step's loads in
// flight in registers meanwhile. Two outputs go through one packed FMA, which
// halves the instructions to issue and leaves the issue slots to the shared-memory
// reads; the fp32 pipe bounds the large tile. Few 64 x 64 tiles are cut along K
// over the CTAs of a cluster, which add their partial tiles through distributed
// shared memory, ranks in order, so that equal calls give equal bits.
//
// Measured: 4,096 x 5,120 -> 5,120 outputs 3.89 ms = 55 TFLOP/s (FMA pipe 73 % active
// while the tiles last; scalar FMAs 4.62 ms), 1,024 x 1,536 -> 1,536 155 us, 300 x 3,200
// -> 320 32 us in eight slices.
//
// Up to eight rows: each warp streams two rows of w against up to four rows of x;
// reading w bounds it (1 x 5,120 -> 5,120 27 us = 0.58 of the copy bandwidth).
#include "launch.cuh"
#include "linear.h"
#include "linear_epi.cuh"
#include "ptx.cuh"

namespace mcs {
namespace {

constexpr int kThreads = 256, kBK = 16;

// x as rows of any layout: element (row, k) at row_base + (k >> shift) * head + (k & mask).
struct XView {
  long long head;  // elements between heads of a row
  int mask, shift;
};
__device__ __forceinline__ const float* x_row(const LinearParams& p, int m) {
  const float* x = static_cast<const float*>(p.x);
  if (p.heads == 0) return x + size_t(m) * p.K;
  const int b = m / p.N, n = m - b * p.N;
  return x + (size_t(b) * p.heads * p.N + n) * (p.K / p.heads);
}

// Four consecutive outputs of one row from their sums.
template <int kAct>
__device__ __forceinline__ void finish_row4(const LinearParams& p, int m, int o, float (&v)[4]) {
  if (p.O % 4 != 0 || o + 4 > p.O) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (o + i < p.O) finish_one<kAct, float>(p, m, o + i, v[i]);
    return;
  }
  auto at4 = [](const void* q, size_t i) { return *reinterpret_cast<const float4*>(static_cast<const float*>(q) + i); };
  const size_t at = size_t(m) * p.O + o;
  if (p.bias) {
    const float4 t = at4(p.bias, o);
    v[0] += t.x, v[1] += t.y, v[2] += t.z, v[3] += t.w;
  }
  activate<kAct>(v);
  if (p.gate) {
    const float4 t = at4(p.gate, size_t(m / p.N) * p.O + o);
    v[0] *= t.x, v[1] *= t.y, v[2] *= t.z, v[3] *= t.w;
  }
  if (p.residual) {
    const float4 t = at4(p.residual, at);
    v[0] += t.x, v[1] += t.y, v[2] += t.z, v[3] += t.w;
  }
  *reinterpret_cast<float4*>(static_cast<float*>(p.y) + at) = make_float4(v[0], v[1], v[2], v[3]);
}

// Q: 16-row groups of four a thread holds in each direction (2: 128 x 128, 1: 64 x 64).
template <int Q, int kAct>
__global__ void __launch_bounds__(kThreads, Q == 2 ? 2 : 5) linear_simt_kernel(const LinearParams p, const XView xv, const int splits) {
  constexpr int kT = 64 * Q, kLd = kT + 4;
  __shared__ __align__(16) float sm[2][2][kBK][kLd];  // [buffer][x, w][k][row]
  const int tid = threadIdx.x, tx = tid % 16, ty = tid / 16;
  const int rank = blockIdx.x % splits, m0 = int(blockIdx.x / splits) * kT, o0 = blockIdx.y * kT;
  const int lr = tid / 4, lk = (tid % 4) * 4;  // this thread's row (of 64) and first k of the loads
  const int nk = (p.K + kBK - 1) / kBK;
  const int k_beg = int(static_cast<long long>(nk) * rank / splits), k_end = int(static_cast<long long>(nk) * (rank + 1) / splits);
  grid_inputs_ready();
  grid_let_next_start();
  const float* xr[Q];
  const float* wr[Q];
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    const int m = m0 + q * 64 + lr, o = o0 + q * 64 + lr;
    xr[q] = m < p.M ? x_row(p, m) : nullptr;
    wr[q] = o < p.O ? static_cast<const float*>(p.w) + size_t(o) * p.K : nullptr;
  }
  float4 la[Q], lb[Q];
  auto load = [&](int step) {
    const int k = step * kBK + lk;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      la[q] = lb[q] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (k < p.K) {
        if (xr[q]) la[q] = *reinterpret_cast<const float4*>(xr[q] + (k >> xv.shift) * xv.head + (k & xv.mask));
        if (wr[q]) lb[q] = *reinterpret_cast<const float4*>(wr[q] + k);
      }
    }
  };
  auto store = [&](int buf) {
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const int r = q * 64 + lr;
      sm[buf][0][lk][r] = la[q].x, sm[buf][0][lk + 1][r] = la[q].y, sm[buf][0][lk + 2][r] = la[q].z,
      sm[buf][0][lk + 3][r] = la[q].w;
      sm[buf][1][lk][r] = lb[q].x, sm[buf][1][lk + 1][r] = lb[q].y, sm[buf][1][lk + 2][r] = lb[q].z,
      sm[buf][1][lk + 3][r] = lb[q].w;
    }
  };
  uint64_t acc[4 * Q][2 * Q];  // row q*4+i, outputs two by two
#pragma unroll
  for (int i = 0; i < 4 * Q; ++i)
#pragma unroll
    for (int j = 0; j < 2 * Q; ++j) acc[i][j] = f2_pack(0.f, 0.f);
  load(k_beg);
  store(0);
  __syncthreads();
  for (int s = k_beg; s < k_end; ++s) {
    const int buf = (s - k_beg) & 1;
    if (s + 1 < k_end) load(s + 1);
#pragma unroll
    for (int k = 0; k < kBK; ++k) {
      uint64_t b[2 * Q];
      float a[4 * Q];
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        const float4 av = *reinterpret_cast<const float4*>(&sm[buf][0][k][q * 64 + ty * 4]);
        const float4 bv = *reinterpret_cast<const float4*>(&sm[buf][1][k][q * 64 + tx * 4]);
        a[4 * q] = av.x, a[4 * q + 1] = av.y, a[4 * q + 2] = av.z, a[4 * q + 3] = av.w;
        b[2 * q] = f2_pack(bv.x, bv.y), b[2 * q + 1] = f2_pack(bv.z, bv.w);
      }
#pragma unroll
      for (int i = 0; i < 4 * Q; ++i) {
        const uint64_t aa = f2_pack(a[i], a[i]);
#pragma unroll
        for (int j = 0; j < 2 * Q; ++j) acc[i][j] = f2_fma(aa, b[j], acc[i][j]);
      }
    }
    if (s + 1 < k_end) store(buf ^ 1);
    __syncthreads();
  }
  if (Q > 1 || splits == 1) {
#pragma unroll
    for (int i = 0; i < 4 * Q; ++i) {
      const int m = m0 + (i / 4) * 64 + ty * 4 + i % 4;
      if (m >= p.M) continue;
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        float v[4];
        f2_unpack(acc[i][2 * q], v[0], v[1]);
        f2_unpack(acc[i][2 * q + 1], v[2], v[3]);
        finish_row4<kAct>(p, m, o0 + q * 64 + tx * 4, v);
      }
    }
    return;
  }
  // partial tiles [64][64] over the buffers, then this CTA's share of the rows
  float* part = &sm[0][0][0][0];
  static_assert(sizeof(sm) >= 64 * 64 * 4, "the buffers hold a partial tile");
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float4 f;
    f2_unpack(acc[i][0], f.x, f.y);
    f2_unpack(acc[i][1], f.z, f.w);
    *reinterpret_cast<float4*>(part + (ty * 4 + i) * 64 + tx * 4) = f;
  }
  cluster_sync();
  for (int r = rank + splits * ty; r < 64 && m0 + r < p.M; r += splits * 16) {
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    for (int c = 0; c < splits; ++c) {
      float f[4];
      asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                   : "=f"(f[0]), "=f"(f[1]), "=f"(f[2]), "=f"(f[3])
                   : "r"(cluster_map(smem_u32(part + r * 64 + tx * 4), c)));
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] += f[i];
    }
    finish_row4<kAct>(p, m0 + r, o0 + tx * 4, v);
  }
  cluster_sync();  // the other CTAs may still be reading this one's tile
}

// Few rows: a warp takes kOut rows of w and kRows rows of x, lanes along K;
// kUnroll 16-byte pieces of each row of w are in flight per lane.
template <int kRows, int kOut, int kUnroll, int kAct>
__global__ void __launch_bounds__(kThreads) linear_simt_few_kernel(const LinearParams p, const XView xv) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int o0 = (blockIdx.x * (kThreads / 32) + warp) * kOut, m0 = blockIdx.y * kRows;
  grid_inputs_ready();
  grid_let_next_start();
  if (o0 >= p.O) return;
  const int rows = min(kRows, p.M - m0), outs = min(kOut, p.O - o0);
  const float* w = static_cast<const float*>(p.w) + size_t(o0) * p.K;
  const float* xr[kRows];
#pragma unroll
  for (int m = 0; m < kRows; ++m) xr[m] = x_row(p, m0 + min(m, rows - 1));
  uint64_t acc[kRows][kOut];
#pragma unroll
  for (int m = 0; m < kRows; ++m)
#pragma unroll
    for (int o = 0; o < kOut; ++o) acc[m][o] = f2_pack(0.f, 0.f);
#pragma unroll kUnroll
  for (int k = lane * 4; k < p.K; k += 128) {
    float4 wv[kOut];
#pragma unroll
    for (int o = 0; o < kOut; ++o)
      wv[o] = *reinterpret_cast<const float4*>(w + size_t(min(o, outs - 1)) * p.K + k);
    const long long at = (k >> xv.shift) * xv.head + (k & xv.mask);
#pragma unroll
    for (int m = 0; m < kRows; ++m) {
      if (m < rows) {
        const float4 x = *reinterpret_cast<const float4*>(xr[m] + at);
        const uint64_t x0 = f2_pack(x.x, x.y), x1 = f2_pack(x.z, x.w);
#pragma unroll
        for (int o = 0; o < kOut; ++o)
          acc[m][o] = f2_fma(x1, f2_pack(wv[o].z, wv[o].w), f2_fma(x0, f2_pack(wv[o].x, wv[o].y), acc[m][o]));
      }
    }
  }
#pragma unroll
  for (int m = 0; m < kRows; ++m) {
    float v[kOut];
#pragma unroll
    for (int o = 0; o < kOut; ++o) {
      float a, b;
      f2_unpack(acc[m][o], a, b);
      v[o] = a + b;
#pragma unroll
      for (int s = 16; s > 0; s >>= 1) v[o] += __shfl_xor_sync(0xffffffffu, v[o], s);
    }
    if (m < rows && lane < outs) {
      float mine = v[0];
#pragma unroll
      for (int o = 1; o < kOut; ++o) mine = lane == o ? v[o] : mine;
      finish_one<kAct, float>(p, m0 + m, o0 + lane, mine);
    }
  }
}

template <int kAct>
cudaError_t launch(const LinearParams& p, int num_sms, cudaStream_t s) {
  XView xv{0, INT32_MAX, 31};
  if (p.heads > 0) {
    const int d = p.K / p.heads;
    xv = {static_cast<long long>(p.N) * d, d - 1, d == 64 ? 6 : 7};
  }
  if (p.M <= 2)
    return launch_overlapped(linear_simt_few_kernel<2, 2, 4, kAct>, dim3((p.O + 15) / 16), kThreads, 0, s, 0, p, xv);
  if (p.M <= 8)  // five to eight rows read w twice, the second time mostly from L2
    return launch_overlapped(linear_simt_few_kernel<4, 2, 4, kAct>, dim3((p.O + 15) / 16, (p.M + 3) / 4), kThreads, 0, s,
                             0, p, xv);
  // a 64 x 64 tile is a quarter of the work of a 128 x 128 one at about 0.35 of its rate; a 128 x 128 tile
  // alone on an SM reaches about 0.67 of what two of them do
  const long long big = static_cast<long long>((p.M + 127) / 128) * ((p.O + 127) / 128);
  const long long small = static_cast<long long>((p.M + 63) / 64) * ((p.O + 63) / 64);
  const double big_time = 4.0 * double((big + num_sms - 1) / num_sms) / (big > num_sms ? 1.0 : 0.67);
  const double small_time = double((small + num_sms - 1) / num_sms) / 0.35;
  if (big_time <= small_time) {
    const dim3 grid((p.M + 127) / 128, (p.O + 127) / 128);
    return launch_overlapped(linear_simt_kernel<2, kAct>, grid, kThreads, 0, s, 0, p, xv, 1);
  }
  // K slices, each of at least eight steps, while the SMs have about two CTAs (of the five that fit)
  const int nk = (p.K + kBK - 1) / kBK;
  int splits = 1;
  while (splits < 8 && small * splits * 4 <= 5ll * num_sms && nk >= 16 * splits) splits *= 2;
  const dim3 grid(unsigned((p.M + 63) / 64) * splits, (p.O + 63) / 64);
  return launch_overlapped(linear_simt_kernel<1, kAct>, grid, kThreads, 0, s, unsigned(splits), p, xv, splits);
}

}  // namespace

cudaError_t linear_simt(const LinearParams& p, int num_sms, cudaStream_t s) {
  switch (p.act) {
    case MCS_ACT_GELU_TANH: return launch<MCS_ACT_GELU_TANH>(p, num_sms, s);
    case MCS_ACT_GELU_ERF: return launch<MCS_ACT_GELU_ERF>(p, num_sms, s);
    case MCS_ACT_SILU: return launch<MCS_ACT_SILU>(p, num_sms, s);
    default: return launch<MCS_ACT_NONE>(p, num_sms, s);
  }
}

}  // namespace mcs
