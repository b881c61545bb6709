// Softmax attention over packed sequences on the CUDA cores, fp32. (Products of three bf16 parts on the tensor cores, as the
// fp32 matrix product takes them, are as exact; they are not made here.) The items of packed.h with 64 rows a tile,
// a block each; 16 rows where those are too few for the GPU.
//
// 256 threads as 16 x 16: a thread has 4 rows (or one) x 4 keys of the scores and as many x D / 16 columns of the sums, in packed
// pairs (scores: two columns of the head side by side; sums: two outputs). Keys and values take turns in one buffer of
// 64 rows, so that two blocks share an SM and one loads while the other multiplies. A step of four head columns
// reads 12 shared-memory wavefronts for 64 multiplications a lane (16 clocks); the multiplications bound it.
// Masked keys as in the bf16 kernel: scores by selection, V that not all rows see with what is not finite as 0.
// Measured: one full sequence of 4,096 tokens, 8 heads, d = 128: 1.91 ms, 36 TFLOP/s (0.45 of the pipe); four causal ones of
// 1,200 tokens and less, 20 heads on 4: 253 us; 77 tokens of 4 heads on 2: 9.1 us; 32 single tokens over 4,000 keys and less of 4
// heads, 16 heads, d = 128: 145 us, a fifth of the copy bandwidth, as a block waits for each tile (all of a tile's loads in
// flight at once: 166 us with four. Four blocks an SM instead of two: 129, but three tokens each over 2,531 keys of 9 heads
// 192 instead of 127).
#include "common.cuh"
#include "launch.cuh"
#include "packed.h"
#include "ptx.cuh"
#include "status.cuh"

namespace mcs {
namespace {

constexpr int kKeys = 64, kThreads = 256;
template <int D, int kR>  // kR: rows of a thread
struct Cfg {
  static constexpr int kRowsTile = 16 * kR;
  static constexpr int kLd = D + 4;     // floats of a row: 16 rows' 16-byte pieces lie in different banks
  static constexpr int kLdP = kKeys + 4;
  static constexpr int kBytes = (kRowsTile * kLd + kKeys * kLd + kRowsTile * kLdP) * 4;
};
struct Walk {
  Divisor by_tq, by_chunk;
};

template <int D, int kR>
__global__ void __launch_bounds__(kThreads, 2) packed_attn_f32_kernel(const PackedParams p, const Walk wk) {
  using L = Cfg<D, kR>;
  constexpr int kRowsTile = L::kRowsTile;
  constexpr int kC = D / 64;  // 16-byte pieces of a row of sums a thread has
  extern __shared__ __align__(16) float sm[];
  float* qs = sm;
  float* kv = qs + kRowsTile * L::kLd;
  float* ps = kv + kKeys * L::kLd;
  __shared__ PackedItem item;
  __shared__ int go, odd;
  const int tid = threadIdx.x, lane = tid & 31, ty = tid >> 4, tx = tid & 15;
  grid_inputs_ready();
  grid_let_next_start();
  if (tid < 32) {
    for (long long s = static_cast<long long>(blockIdx.x) * 32 + lane; s < p.S; s += static_cast<long long>(gridDim.x) * 32) {
      int a, b, c, d;
      if (!packed_sequence(p, int(s), a, b, c, d)) raise_status(p.status, kStatusBounds);
    }
    __syncwarp();
    PackedItem it{};
    const PackedLane sequence = p.S <= 32 ? packed_lane(p, wk.by_tq, wk.by_chunk, lane) : PackedLane{};
    const bool found = packed_item(p, wk.by_tq, wk.by_chunk, sequence, blockIdx.x, lane, &it);
    if (lane == 0) item = it, go = found, odd = 0;
  }
  __syncthreads();
  if (!go) return;
  const PackedItem it = item;
  const int all_see = visible_keys(it, p.causal, 0);

  for (int e = tid; e < kRowsTile * D / 4; e += kThreads) {
    const int r = e / (D / 4), c = e % (D / 4), t = p.by_group.div(r), h = it.hk * p.g + r - t * p.g;
    float4 w = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r < p.rows && t < it.ntok)
      w = reinterpret_cast<const float4*>(static_cast<const float*>(p.q) + h * p.qs.head + (it.q0 + t) * p.qs.token)[c];
    *reinterpret_cast<float4*>(qs + r * L::kLd + c * 4) = w;
  }
  int lim[kR];
  float m[kR], l[kR];
  uint64_t o[kR][kC * 2];
#pragma unroll
  for (int i = 0; i < kR; ++i) {
    const int r = ty * kR + i, t = p.by_group.div(r);
    lim[i] = r < p.rows && t < it.ntok ? visible_keys(it, p.causal, t) : 0;
    m[i] = -INFINITY, l[i] = 0.f;
#pragma unroll
    for (int c = 0; c < kC * 2; ++c) o[i][c] = f2_pack(0.f, 0.f);
  }
  const float* kb = static_cast<const float*>(p.k) + it.hk * p.ks.head + it.k0 * p.ks.token;
  const float* vb = static_cast<const float*>(p.v) + it.hk * p.vs.head + it.k0 * p.vs.token;
  for (int j0 = 0; j0 < it.nkeys; j0 += kKeys) {
    __syncthreads();  // the last tile's values have been read
#pragma unroll 8
    for (int e = tid; e < kKeys * D / 4; e += kThreads) {
      const int r = e / (D / 4), c = e % (D / 4);
      float4 w = make_float4(0.f, 0.f, 0.f, 0.f);
      if (j0 + r < it.nkeys) w = reinterpret_cast<const float4*>(kb + (j0 + r) * p.ks.token)[c];
      *reinterpret_cast<float4*>(kv + r * L::kLd + c * 4) = w;
    }
    __syncthreads();
    uint64_t s2[kR][4];
#pragma unroll
    for (int i = 0; i < kR; ++i)
#pragma unroll
      for (int n = 0; n < 4; ++n) s2[i][n] = f2_pack(0.f, 0.f);
#pragma unroll 4
    for (int k = 0; k < D; k += 4) {
      ulonglong2 a[kR], b[4];
#pragma unroll
      for (int i = 0; i < kR; ++i) a[i] = *reinterpret_cast<const ulonglong2*>(qs + (ty * kR + i) * L::kLd + k);
#pragma unroll
      for (int n = 0; n < 4; ++n) b[n] = *reinterpret_cast<const ulonglong2*>(kv + (tx + 16 * n) * L::kLd + k);
#pragma unroll
      for (int i = 0; i < kR; ++i)
#pragma unroll
        for (int n = 0; n < 4; ++n) s2[i][n] = f2_fma(a[i].y, b[n].y, f2_fma(a[i].x, b[n].x, s2[i][n]));
    }
    __syncthreads();  // the keys have been read: the values take their place
    bool found = false;
#pragma unroll 8
    for (int e = tid; e < kKeys * D / 4; e += kThreads) {
      const int r = e / (D / 4), c = e % (D / 4);
      float4 w = make_float4(0.f, 0.f, 0.f, 0.f);
      if (j0 + r < it.nkeys) w = reinterpret_cast<const float4*>(vb + (j0 + r) * p.vs.token)[c];
      if (j0 + r >= all_see && !(isfinite(w.x) && isfinite(w.y) && isfinite(w.z) && isfinite(w.w))) {
        found = true;
        w = make_float4(isfinite(w.x) ? w.x : 0.f, isfinite(w.y) ? w.y : 0.f, isfinite(w.z) ? w.z : 0.f, isfinite(w.w) ? w.w : 0.f);
      }
      *reinterpret_cast<float4*>(kv + r * L::kLd + c * 4) = w;
    }
    if (found) odd = 1;
#pragma unroll
    for (int i = 0; i < kR; ++i) {
      float s[4], top = -INFINITY;
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        float lo, hi;
        f2_unpack(s2[i][n], lo, hi);
        s[n] = j0 + tx + 16 * n < lim[i] ? (lo + hi) * p.scale_log2 : -INFINITY;
        top = fmaxf(top, s[n]);
      }
#pragma unroll
      for (int x = 8; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
      const float m_new = fmaxf(m[i], top), base = m_new == -INFINITY ? 0.f : m_new;
      const float alpha = m[i] == -INFINITY ? 0.f : exp2f(m[i] - m_new);
      float sum = 0.f;
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        const float e = exp2f(s[n] - base);
        sum += e;
        ps[(ty * kR + i) * L::kLdP + tx + 16 * n] = e;
      }
#pragma unroll
      for (int x = 8; x > 0; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
      l[i] = l[i] * (l[i] == 0.f ? 0.f : m[i] == -INFINITY ? 1.f : alpha) + sum;  // a sum of NaN scores stays
      m[i] = m_new;
      const uint64_t f = f2_pack(alpha, alpha);
#pragma unroll
      for (int c = 0; c < kC * 2; ++c) o[i][c] = f2_mul(o[i][c], f);
    }
    __syncthreads();
#pragma unroll 2
    for (int j = 0; j < kKeys; j += 4) {
      float4 w[kR];
#pragma unroll
      for (int i = 0; i < kR; ++i) w[i] = *reinterpret_cast<const float4*>(ps + (ty * kR + i) * L::kLdP + j);
#pragma unroll
      for (int jj = 0; jj < 4; ++jj) {
        ulonglong2 v[kC];
#pragma unroll
        for (int c = 0; c < kC; ++c) v[c] = *reinterpret_cast<const ulonglong2*>(kv + (j + jj) * L::kLd + tx * 4 + 64 * c);
#pragma unroll
        for (int i = 0; i < kR; ++i) {
          const float e = jj == 0 ? w[i].x : jj == 1 ? w[i].y : jj == 2 ? w[i].z : w[i].w;
          const uint64_t e2 = f2_pack(e, e);
#pragma unroll
          for (int c = 0; c < kC; ++c) {
            o[i][2 * c] = f2_fma(e2, v[c].x, o[i][2 * c]);
            o[i][2 * c + 1] = f2_fma(e2, v[c].y, o[i][2 * c + 1]);
          }
        }
      }
    }
  }
  __syncthreads();
  const bool extra = odd != 0;
#pragma unroll
  for (int i = 0; i < kR; ++i) {
    const int r = ty * kR + i, t = p.by_group.div(r), h = it.hk * p.g + r - t * p.g;
    if (r >= p.rows || t >= it.ntok) continue;
    const bool cut = !it.whole;
    const float inv = cut ? 1.f : 1.f / l[i];
    float v[kC * 4];
#pragma unroll
    for (int c = 0; c < kC * 2; ++c) f2_unpack(o[i][c], v[2 * c], v[2 * c + 1]);
#pragma unroll
    for (int c = 0; c < kC * 4; ++c) v[c] = l[i] == 0.f ? 0.f : v[c] * inv;
    if (extra) {  // elements that are not finite and that only some rows see
      for (int j = all_see; j < lim[i]; ++j)
#pragma unroll
        for (int c = 0; c < kC * 4; ++c) {
          const float f = vb[j * p.vs.token + tx * 4 + 64 * (c / 4) + c % 4];
          if (!isfinite(f)) v[c] += f;
        }
    }
    float* out = cut ? p.part_o + (it.part + r) * D : static_cast<float*>(p.o) + h * p.os.head + (it.q0 + t) * p.os.token;
#pragma unroll
    for (int c = 0; c < kC; ++c)
      *reinterpret_cast<float4*>(out + tx * 4 + 64 * c) = make_float4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
    if (tx != 0) continue;
    if (cut) p.part_ml[it.part + r] = make_float2(m[i], l[i]);
    else if (p.lse != nullptr)
      p.lse[static_cast<long long>(h) * p.Tq + it.q0 + t] = l[i] == 0.f ? -INFINITY : (m[i] == -INFINITY ? 0.f : m[i]) * kLn2 + logf(l[i]);
  }
}

template <int D, int kR>
cudaError_t launch_f32(const PackedParams& p, cudaStream_t s) {
  const cudaError_t e = allow_smem<packed_attn_f32_kernel<D, kR>>(Cfg<D, kR>::kBytes);
  if (e != cudaSuccess) return e;
  const Walk wk{Divisor(p.tq), Divisor(p.chunk > 0 ? p.chunk : 1)};
  return launch_overlapped(packed_attn_f32_kernel<D, kR>, dim3(unsigned(p.items)), kThreads, Cfg<D, kR>::kBytes, s, 0, p, wk);
}

}  // namespace

cudaError_t packed_attn_f32(const PackedParams& p, cudaStream_t s) {
  const cudaError_t e = p.rows > 16 ? (p.d == 128 ? launch_f32<128, 4>(p, s) : launch_f32<64, 4>(p, s))
                                    : (p.d == 128 ? launch_f32<128, 1>(p, s) : launch_f32<64, 1>(p, s));
  return e != cudaSuccess || p.chunk == 0 ? e : packed_join(p, false, s);
}

}  // namespace mcs
