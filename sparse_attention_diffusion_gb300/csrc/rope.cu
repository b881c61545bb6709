// Rotary positions with several axes, and the norms of queries and keys for
// each head with the rotation in the same pass (forward and backward).
//
//   y = R(n) (x * rstd * w),  rstd = 1 / sqrt(mean(x^2) + eps)
//
// with R(n) turning the head's element pairs by the token's angles. Everything
// here reads its rows once and writes them once: HBM bounds it, the table of
// cosines and sines (a few hundred KB at most on a video grid) stays in L1/L2.
// The angles come from a table because a position far from the origin needs
// 64-bit angles, which are too slow to make for every token.
//
// A row (one token of one head, d elements) is held by D * sizeof(T) / 16 lanes
// of one warp, 16 bytes a lane; a lane always holds both elements of a pair, so
// the rotation needs no exchange, and the norm only the shuffle sum over the
// row's lanes. The lanes of a row keep their token's cosines and sines in
// registers and walk over its heads.
//
// Measured against the copy bandwidth of 6,783 GB/s (bf16, d = 128): rotation of 40 heads x
// 75,600 tokens 224 us (1.02 of it), norm + rotation + repacking of its q, k, v 680 us
// (1.01), of 12 heads x 32,768 tokens 93 us (0.96); gradient of the latter 134 us (0.89)
// and of the former 0.93 ms (0.99).
#include "rope.h"

#include "common.cuh"
#include "kernels.h"
#include "launch.cuh"
#include "ptx.cuh"
#include "status.cuh"

namespace mcs {
namespace {

constexpr int kThreads = 256;

template <typename T, int D>
struct Row {
  static constexpr int E = 16 / int(sizeof(T));  // elements a lane
  static constexpr int L = D / E;                // lanes a row
  static constexpr int NP = E / 2;               // pairs a lane
  static constexpr int kTokens = kThreads / L;   // rows a block holds at once
};

// 16 bytes of a row as loaded: interleaved pairs are one 16-byte piece, halves
// are 8 bytes of the first half and the matching 8 bytes of the second.
struct Raw {
  uint32_t w[4];
};

template <typename T, int D, bool kHalf>
__device__ __forceinline__ Raw load_raw(const T* row, int lane) {
  Raw r;
  if constexpr (kHalf) {
    const uint2 a = *reinterpret_cast<const uint2*>(row + lane * Row<T, D>::NP);
    const uint2 b = *reinterpret_cast<const uint2*>(row + D / 2 + lane * Row<T, D>::NP);
    r.w[0] = a.x, r.w[1] = a.y, r.w[2] = b.x, r.w[3] = b.y;
  } else {
    const uint4 a = *reinterpret_cast<const uint4*>(row + lane * Row<T, D>::E);
    r.w[0] = a.x, r.w[1] = a.y, r.w[2] = a.z, r.w[3] = a.w;
  }
  return r;
}
template <typename T, int D, bool kHalf>
__device__ __forceinline__ void store_raw(T* row, int lane, const Raw& r) {
  if constexpr (kHalf) {
    *reinterpret_cast<uint2*>(row + lane * Row<T, D>::NP) = make_uint2(r.w[0], r.w[1]);
    *reinterpret_cast<uint2*>(row + D / 2 + lane * Row<T, D>::NP) = make_uint2(r.w[2], r.w[3]);
  } else {
    *reinterpret_cast<uint4*>(row + lane * Row<T, D>::E) = make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
  }
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Raw words <-> the lane's pairs (a[j], b[j]).
template <typename T, bool kHalf, int NP>
__device__ __forceinline__ void unpack(const Raw& r, float (&a)[NP], float (&b)[NP]) {
  if constexpr (sizeof(T) == 2) {
    if constexpr (kHalf) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        a[2 * i] = bf16_lo(r.w[i]), a[2 * i + 1] = bf16_hi(r.w[i]);
        b[2 * i] = bf16_lo(r.w[2 + i]), b[2 * i + 1] = bf16_hi(r.w[2 + i]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) a[j] = bf16_lo(r.w[j]), b[j] = bf16_hi(r.w[j]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      a[j] = __uint_as_float(r.w[kHalf ? j : 2 * j]);
      b[j] = __uint_as_float(r.w[kHalf ? 2 + j : 2 * j + 1]);
    }
  }
}
template <typename T, bool kHalf, int NP>
__device__ __forceinline__ Raw pack(const float (&a)[NP], const float (&b)[NP]) {
  Raw r;
  if constexpr (sizeof(T) == 2) {
    if constexpr (kHalf) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        r.w[i] = bf16_pair(a[2 * i], a[2 * i + 1]);
        r.w[2 + i] = bf16_pair(b[2 * i], b[2 * i + 1]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) r.w[j] = bf16_pair(a[j], b[j]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      r.w[kHalf ? j : 2 * j] = __float_as_uint(a[j]);
      r.w[kHalf ? 2 + j : 2 * j + 1] = __float_as_uint(b[j]);
    }
  }
  return r;
}

// The same with two pairs per 64-bit register: (a[2i], a[2i + 1]), (b[2i], b[2i + 1]).
template <typename T, bool kHalf, int N2>
__device__ __forceinline__ void unpack2(const Raw& r, uint64_t (&a)[N2], uint64_t (&b)[N2]) {
  float x[2 * N2], y[2 * N2];
  unpack<T, kHalf, 2 * N2>(r, x, y);
#pragma unroll
  for (int i = 0; i < N2; ++i) a[i] = f2_pack(x[2 * i], x[2 * i + 1]), b[i] = f2_pack(y[2 * i], y[2 * i + 1]);
}
template <typename T, bool kHalf, int N2>
__device__ __forceinline__ Raw pack2(const uint64_t (&a)[N2], const uint64_t (&b)[N2]) {
  float x[2 * N2], y[2 * N2];
#pragma unroll
  for (int i = 0; i < N2; ++i) f2_unpack(a[i], x[2 * i], x[2 * i + 1]), f2_unpack(b[i], y[2 * i], y[2 * i + 1]);
  return pack<T, kHalf, 2 * N2>(x, y);
}

// Cosines and sines of the pairs lane * NP .. + NP - 1 of token n of batch b.
// Returns false when a listed position is out of range (nothing is read then).
template <int NP>
__device__ __forceinline__ bool load_angles(const RopeGeom& g, const float2* table, const int32_t* pos, int b, int N,
                                            int n, int lane, float (&c)[NP], float (&s)[NP]) {
  int p[3] = {0, 0, 0};
  bool turns = true;
  if (pos != nullptr) {
    const int32_t* row = pos + (size_t(b) * N + n) * g.axes;
    for (int a = 0; a < g.axes; ++a) {
      p[a] = row[a];
      if (p[a] < 0 || p[a] >= g.len[a]) return false;
    }
  } else {
    int i = n - g.first;
    turns = i >= 0 && i < g.ngrid;
    if (turns) {
      for (int a = g.axes - 1; a > 0; --a) {
        const int q = g.by[a].div(i);
        p[a] = i - q * g.len[a];
        i = q;
      }
      p[0] = i;
    }
  }
#pragma unroll
  for (int j = 0; j < NP; ++j) {
    c[j] = 1.f, s[j] = 0.f;
    int pr = lane * NP + j;
    if (turns && pr < g.npairs) {
      int a = 0;
      while (pr >= g.pairs[a]) pr -= g.pairs[a++];
      const float2 t = __ldg(table + g.toff[a] + p[a] * g.pairs[a] + pr);
      c[j] = t.x, s[j] = t.y;
    }
  }
  return true;
}

template <int L>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The lane's norm weights in pair order (1 where absent).
template <typename T, int D, bool kHalf, int NP>
__device__ __forceinline__ void load_weights(const void* w, int lane, float (&a)[NP], float (&b)[NP]) {
#pragma unroll
  for (int j = 0; j < NP; ++j) a[j] = b[j] = 1.f;
  if (w != nullptr) unpack<T, kHalf, NP>(load_raw<T, D, kHalf>(static_cast<const T*>(w), lane), a, b);
}

__global__ void rope_table_kernel(const RopeTableParams p) {
  const int a = blockIdx.y;
  const long long total = static_cast<long long>(p.g.len[a]) * p.g.pairs[a];
  for (long long i = blockIdx.x * static_cast<long long>(blockDim.x) + threadIdx.x; i < total;
       i += static_cast<long long>(gridDim.x) * blockDim.x) {
    const int pos = int(i / p.g.pairs[a]), j = int(i % p.g.pairs[a]);
    const double f = pow(p.theta, -double(j) / p.g.pairs[a]);
    double sn, cs;
    sincos((p.start[a] + pos) * p.scale[a] * f, &sn, &cs);
    p.table[p.g.toff[a] + i] = make_float2(float(cs), float(sn));
  }
}

// Heads whose rows one lane has in flight at once.
constexpr int kUnroll = 4;

template <typename T, int D, bool kHalf, bool kNorm>
__global__ void __launch_bounds__(kThreads) rotate_kernel(const RotateParams p) {
  using R = Row<T, D>;
  constexpr int NP = R::NP;
  const int lane = threadIdx.x % R::L;
  const int n = blockIdx.x * R::kTokens + threadIdx.x / R::L, b = blockIdx.z;
  const int h_beg = blockIdx.y * p.heads_per_block, h_end = min(p.H, h_beg + p.heads_per_block);
  float c[NP], s[NP];
  bool live = n < p.N;
  grid_inputs_ready();
  grid_let_next_start();
  if (live && !load_angles<NP>(p.g, p.table, p.pos, b, p.N, n, lane, c, s)) {
    live = false;
    raise_status(p.status, kStatusBounds);
  }
  if (!live) {
#pragma unroll
    for (int j = 0; j < NP; ++j) c[j] = s[j] = 0.f;
  }
#pragma unroll
  for (int j = 0; j < NP; ++j) s[j] *= p.sin_sign;
  const long long in_off = b * p.in.b + n * p.in.n, out_off = b * p.out.b + n * p.out.n;
#pragma unroll
  for (int st = 0; st < (kNorm ? 3 : 1); ++st) {
    if (p.src[st] == nullptr) continue;
    const T* src = static_cast<const T*>(p.src[st]) + in_off;
    T* dst = static_cast<T*>(p.dst[st]) + out_off;
    float wa[NP], wb[NP];
    if constexpr (kNorm) {
      if (st < 2) load_weights<T, D, kHalf, NP>(p.w[st], lane, wa, wb);
    }
    for (int h0 = h_beg; h0 < h_end; h0 += kUnroll) {
      Raw r[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        r[u] = Raw{};
        if (live && h0 + u < h_end) r[u] = load_raw<T, D, kHalf>(src + (h0 + u) * p.in.h, lane);
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        if (st < 2) {
          float x[NP], y[NP];
          unpack<T, kHalf, NP>(r[u], x, y);
          if constexpr (kNorm) {
            float ss = 0.f;
#pragma unroll
            for (int j = 0; j < NP; ++j) ss += x[j] * x[j] + y[j] * y[j];
            const float rstd = rsqrtf(row_sum<R::L>(ss) * (1.f / D) + p.eps);
#pragma unroll
            for (int j = 0; j < NP; ++j) x[j] *= rstd * wa[j], y[j] *= rstd * wb[j];
          }
          float xr[NP], yr[NP];
#pragma unroll
          for (int j = 0; j < NP; ++j) {
            xr[j] = x[j] * c[j] - y[j] * s[j];
            yr[j] = x[j] * s[j] + y[j] * c[j];
          }
          r[u] = pack<T, kHalf, NP>(xr, yr);
        }
        if (live && h0 + u < h_end) store_raw<T, D, kHalf>(dst + (h0 + u) * p.out.h, lane, r[u]);
      }
    }
  }
}

// Gradient of norm + rotation. The work is a list of units, a unit being one
// stream's (q, k or the copy of v) heads_per_unit heads of one token tile, with
// the tokens' angles in registers; blocks take every gridDim.x-th unit, stream
// after stream. A lane's share of dw (its own pairs, all its tokens and heads)
// stays in registers until the block's units of that stream are done, is summed
// over the block's rows through shared memory, and goes to partial[block];
// norm_bwd_reduce_kernel adds the blocks in order.
//
// With g = R^T dy and xhat = rstd x: dw += g xhat and dx = rstd (g w - xhat mean(g w xhat)).
// The row is scaled by rstd before anything is multiplied with it, so that no factor leaves
// fp32's range for rows of any length: one whose squares overflow has rstd = 0 and gives 0.
// (Both row sums taken together over the unscaled row give infinities and NaN for long rows and
// lose the projection where dot rstd^2 underflows.) Instructions bound this (two row sums and
// the conversions beside 48 bytes a lane), so pairs of pairs go through packed fp32 operations.
// Heads in flight per lane, at three blocks an SM; and whether the lengths of all of them are
// summed before the first gradient (480p layer, 12 heads of 128, bf16: four heads 138 us, with all
// lengths first 172; as halves, whose rows are two loads, two heads 156, three 177 and four 175,
// three with all lengths first 145, four 173; fp32, 2 x 6 heads of 128 x 16,687 tokens: 152, all
// lengths first 149).
template <bool kHalf>
constexpr int kBwdUnroll = kHalf ? 3 : 4;
constexpr int kBwdBlocksPerSm = 3;

template <typename T, int D, bool kHalf>
__global__ void __launch_bounds__(kThreads, kBwdBlocksPerSm) norm_bwd_kernel(const NormBwdParams p) {
  using R = Row<T, D>;
  constexpr int NP = R::NP, U = kBwdUnroll<kHalf>;
  constexpr bool kTogether = kHalf || sizeof(T) == 4;
  __shared__ float red[R::kTokens][D];
  const int lane = threadIdx.x % R::L, row = threadIdx.x / R::L;
  const int tiles = (p.N + R::kTokens - 1) / R::kTokens;
  const int chunks = (p.H + p.heads_per_unit - 1) / p.heads_per_unit;
  const int units = tiles * p.B * chunks;  // of a stream; fewer than 2^31 rows
  int u = blockIdx.x;                      // counted from the current stream's first unit
  grid_inputs_ready();
  grid_let_next_start();
#pragma unroll 1
  for (int st = 0; st < 3; ++st) {
    if (p.dy[st] == nullptr) continue;
    constexpr int N2 = NP / 2;
    uint64_t da[N2], db[N2], wa[N2], wb[N2];  // two pairs each
    {
      float a[NP], b[NP];
      load_weights<T, D, kHalf, NP>(st < 2 ? p.w[st] : nullptr, lane, a, b);
#pragma unroll
      for (int j = 0; j < N2; ++j) {
        wa[j] = f2_pack(a[2 * j], a[2 * j + 1]), wb[j] = f2_pack(b[2 * j], b[2 * j + 1]);
        da[j] = db[j] = f2_pack(0.f, 0.f);
      }
    }
    for (; u < units; u += gridDim.x) {
      const int bt = p.by_chunks.div(u), b = p.by_tiles.div(bt), n = (bt - b * tiles) * R::kTokens + row;
      const int h_beg = (u - bt * chunks) * p.heads_per_unit, h_end = min(p.H, h_beg + p.heads_per_unit);
      float c[NP], s[NP];
      bool live = n < p.N;
      if (live && !load_angles<NP>(p.g, p.table, p.pos, b, p.N, n, lane, c, s)) {
        live = false;
        raise_status(p.status, kStatusBounds);
      }
      if (!live) {
#pragma unroll
        for (int j = 0; j < NP; ++j) c[j] = s[j] = 0.f;
      }
      uint64_t c2[N2], s2[N2], n2[N2];
#pragma unroll
      for (int j = 0; j < N2; ++j) {
        c2[j] = f2_pack(c[2 * j], c[2 * j + 1]), s2[j] = f2_pack(s[2 * j], s[2 * j + 1]);
        n2[j] = f2_pack(-s[2 * j], -s[2 * j + 1]);
      }
      const long long off = b * p.in.b + n * p.in.n;
      const T* dy = static_cast<const T*>(p.dy[st]) + (static_cast<long long>(b) * p.H * p.N + n) * D;
      const T* px = st < 2 ? static_cast<const T*>(p.x[st]) + off : nullptr;
      T* dx = static_cast<T*>(p.dx[st]) + off;
      for (int h0 = h_beg; h0 < h_end; h0 += U) {
        Raw ry[U], rx[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
          ry[i] = rx[i] = Raw{};
          if (live && h0 + i < h_end) {
            ry[i] = load_raw<T, D, kHalf>(dy + static_cast<long long>(h0 + i) * p.N * D, lane);
            if (st < 2) rx[i] = load_raw<T, D, kHalf>(px + (h0 + i) * p.in.h, lane);
          }
        }
        auto squares = [&](const Raw& r) {
          uint64_t x[N2], y[N2], ss = f2_pack(0.f, 0.f);
          unpack2<T, kHalf, N2>(r, x, y);
#pragma unroll
          for (int j = 0; j < N2; ++j) ss = f2_fma(y[j], y[j], f2_fma(x[j], x[j], ss));
          float s0, s1;
          f2_unpack(ss, s0, s1);
          return s0 + s1;
        };
        [[maybe_unused]] float lengths[U];
        if constexpr (kTogether) {
          if (st < 2) {
#pragma unroll
            for (int i = 0; i < U; ++i) lengths[i] = squares(rx[i]);
#pragma unroll
            for (int i = 0; i < U; ++i) lengths[i] = row_sum<R::L>(lengths[i]);
          }
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
          if (st < 2) {
            const float rstd = rsqrtf((kTogether ? lengths[i] : row_sum<R::L>(squares(rx[i]))) * (1.f / D) + p.eps);
            uint64_t x[N2], y[N2], ga[N2], gb[N2], dot = f2_pack(0.f, 0.f);
            unpack2<T, kHalf, N2>(rx[i], x, y);
            unpack2<T, kHalf, N2>(ry[i], ga, gb);
            const uint64_t r2 = f2_pack(rstd, rstd);
#pragma unroll
            for (int j = 0; j < N2; ++j) {
              x[j] = f2_mul(x[j], r2), y[j] = f2_mul(y[j], r2);
              const uint64_t g = ga[j];
              ga[j] = f2_fma(gb[j], s2[j], f2_mul(g, c2[j]));
              gb[j] = f2_fma(g, n2[j], f2_mul(gb[j], c2[j]));
              da[j] = f2_fma(ga[j], x[j], da[j]), db[j] = f2_fma(gb[j], y[j], db[j]);
              ga[j] = f2_mul(ga[j], wa[j]), gb[j] = f2_mul(gb[j], wb[j]);
              dot = f2_fma(gb[j], y[j], f2_fma(ga[j], x[j], dot));
            }
            float s0, s1;
            f2_unpack(dot, s0, s1);
            const float m = -row_sum<R::L>(s0 + s1) * (1.f / D);
            const uint64_t m2 = f2_pack(m, m);
#pragma unroll
            for (int j = 0; j < N2; ++j) {
              ga[j] = f2_mul(r2, f2_fma(m2, x[j], ga[j]));
              gb[j] = f2_mul(r2, f2_fma(m2, y[j], gb[j]));
            }
            ry[i] = pack2<T, kHalf, N2>(ga, gb);
          }
          if (live && h0 + i < h_end) store_raw<T, D, kHalf>(dx + (h0 + i) * p.in.h, lane, ry[i]);
        }
      }
    }
    u -= units;
    if (st < 2 && p.dw[st] != nullptr) {
#pragma unroll
      for (int j = 0; j < NP; ++j) {
        const int pr = lane * NP + j;
        float lo, hi;
        f2_unpack(da[j / 2], lo, hi);
        red[row][kHalf ? pr : 2 * pr] = j & 1 ? hi : lo;
        f2_unpack(db[j / 2], lo, hi);
        red[row][kHalf ? D / 2 + pr : 2 * pr + 1] = j & 1 ? hi : lo;
      }
      __syncthreads();
      if (threadIdx.x < D) {
        float v = 0.f;
        for (int i = 0; i < R::kTokens; ++i) v += red[i][threadIdx.x];
        p.partial[(size_t(blockIdx.x) * 2 + st) * D + threadIdx.x] = v;
      }
      __syncthreads();
    }
  }
}

// dw[st][e] = sum over blocks of partial[block][st][e], in a fixed order: a block
// takes 32 elements, a warp every 32nd row with eight rows in flight, then the
// warps' sums in order.
__global__ void __launch_bounds__(1024) norm_bwd_reduce_kernel(const float* partial, int nblk, int D, float* dwq,
                                                               float* dwk) {
  __shared__ float red[32][33];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, st = blockIdx.y, e = blockIdx.x * 32 + lane;
  float* dw = st == 0 ? dwq : dwk;
  grid_inputs_ready();
  grid_let_next_start();
  if (dw == nullptr) return;
  const float* src = partial + st * D + e;
  float v = 0.f;
  for (int i = warp; i < nblk; i += 32 * 8) {
    float f[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) f[u] = i + 32 * u < nblk ? src[size_t(i + 32 * u) * 2 * D] : 0.f;
#pragma unroll
    for (int u = 0; u < 8; ++u) v += f[u];
  }
  red[warp][lane] = v;
  __syncthreads();
  if (warp == 0) {
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) t += red[i][lane];
    dw[e] = t;
  }
}

template <typename T, int D, bool kHalf, bool kNorm>
cudaError_t launch_rotate(RotateParams p, int num_sms, cudaStream_t s) {
  using R = Row<T, D>;
  const int tiles = (p.N + R::kTokens - 1) / R::kTokens;
  // heads a block: the fewest rounds of blocks over the SMs (five fit on each), a block costing its
  // groups of heads plus about half a group for the token's angles
  const long long rows = static_cast<long long>(tiles) * p.B, slots = 5ll * num_sms;
  const int groups = (p.H + kUnroll - 1) / kUnroll;
  long long best = 0;
  for (int c = 1; c <= groups; ++c) {
    const int per = (groups + c - 1) / c;
    const long long cost = (rows * ((groups + per - 1) / per) + slots - 1) / slots * (2 * per + 1);
    if (best == 0 || cost < best) best = cost, p.heads_per_block = per * kUnroll;
  }
  if (p.heads_per_block > p.H) p.heads_per_block = p.H;
  const dim3 grid(tiles, (p.H + p.heads_per_block - 1) / p.heads_per_block, p.B);
  return launch_overlapped(rotate_kernel<T, D, kHalf, kNorm>, grid, kThreads, 0, s, 0, p);
}

template <typename T, int D, bool kHalf>
cudaError_t launch_bwd(NormBwdParams p, int num_sms, cudaStream_t s) {
  using R = Row<T, D>;
  const long long tiles = static_cast<long long>((p.N + R::kTokens - 1) / R::kTokens) * p.B;
  long long blocks = static_cast<long long>(kBwdBlocksPerSm) * num_sms;
  if (blocks > kNormBwdMaxBlocks) blocks = kNormBwdMaxBlocks;
  // heads a unit: the fewest rounds of units over the blocks, a unit costing its heads plus about
  // two more for the token's angles
  int streams = 0;
  for (int i = 0; i < 3; ++i) streams += p.dy[i] != nullptr;
  constexpr int kU = kBwdUnroll<kHalf>;
  const int groups = (p.H + kU - 1) / kU;
  long long best = 0, units = 0;
  for (int c = 1; c <= groups; ++c) {
    const int heads = (groups + c - 1) / c * kU;
    const long long n = tiles * ((p.H + heads - 1) / heads) * streams;
    const long long cost = (n + blocks - 1) / blocks * (heads + 2);
    if (best == 0 || cost < best) best = cost, units = n, p.heads_per_unit = heads;
  }
  if (p.heads_per_unit > p.H) p.heads_per_unit = p.H;
  if (blocks > units) blocks = units;
  p.by_chunks = Divisor((p.H + p.heads_per_unit - 1) / p.heads_per_unit);
  p.by_tiles = Divisor((p.N + R::kTokens - 1) / R::kTokens);
  const cudaError_t e = launch_overlapped(norm_bwd_kernel<T, D, kHalf>, dim3(unsigned(blocks)), kThreads, 0, s, 0, p);
  if (e != cudaSuccess || (p.dw[0] == nullptr && p.dw[1] == nullptr)) return e;
  return launch_overlapped(norm_bwd_reduce_kernel, dim3(D / 32, 2), 1024, 0, s, 0, p.partial, int(blocks), D, p.dw[0], p.dw[1]);
}

template <typename T, int D>
cudaError_t rotate_td(bool half_style, bool norm, const RotateParams& p, int num_sms, cudaStream_t s) {
  if (half_style)
    return norm ? launch_rotate<T, D, true, true>(p, num_sms, s) : launch_rotate<T, D, true, false>(p, num_sms, s);
  return norm ? launch_rotate<T, D, false, true>(p, num_sms, s) : launch_rotate<T, D, false, false>(p, num_sms, s);
}
template <typename T, int D>
cudaError_t bwd_td(bool half_style, const NormBwdParams& p, int num_sms, cudaStream_t s) {
  return half_style ? launch_bwd<T, D, true>(p, num_sms, s) : launch_bwd<T, D, false>(p, num_sms, s);
}

}  // namespace

cudaError_t rope_table(const RopeTableParams& p, cudaStream_t s) {
  long long most = 0;
  for (int a = 0; a < p.g.axes; ++a) {
    const long long n = static_cast<long long>(p.g.len[a]) * p.g.pairs[a];
    if (n > most) most = n;
  }
  const long long blocks = (most + 127) / 128;
  const dim3 grid(unsigned(blocks < 4096 ? blocks : 4096), p.g.axes);
  rope_table_kernel<<<grid, 128, 0, s>>>(p);
  note_launches(1);
  return cudaGetLastError();
}

cudaError_t rotate(bool bf16, int d, bool half_style, bool norm, RotateParams p, int num_sms, cudaStream_t s) {
  if (bf16)
    return d == 128 ? rotate_td<__nv_bfloat16, 128>(half_style, norm, p, num_sms, s)
                    : rotate_td<__nv_bfloat16, 64>(half_style, norm, p, num_sms, s);
  return d == 128 ? rotate_td<float, 128>(half_style, norm, p, num_sms, s)
                  : rotate_td<float, 64>(half_style, norm, p, num_sms, s);
}

cudaError_t qk_norm_rope_bwd(bool bf16, int d, bool half_style, const NormBwdParams& p, int num_sms, cudaStream_t s) {
  if (bf16)
    return d == 128 ? bwd_td<__nv_bfloat16, 128>(half_style, p, num_sms, s)
                    : bwd_td<__nv_bfloat16, 64>(half_style, p, num_sms, s);
  return d == 128 ? bwd_td<float, 128>(half_style, p, num_sms, s) : bwd_td<float, 64>(half_style, p, num_sms, s);
}

}  // namespace mcs
