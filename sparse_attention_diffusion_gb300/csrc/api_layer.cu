// C ABI of the operators around the attention call (rotary positions, query/key
// norms, projections; declared in include/mcs.h): argument validation and
// dispatch. No C++ exception and no device allocation here.
#include <cmath>
#include <cstdint>

#include "mcs.h"
#include "api_checks.h"
#include "api_internal.h"
#include "common.cuh"
#include "linear.h"
#include "rope.h"

namespace {

using mcs::aligned16;
using mcs::aligned16_or_null;
using mcs::from_cuda;
using mcs::overlap;
using mcs::Range;
using mcs::range;

// Checks a rope by itself and fills the kernels' geometry; entries: table pairs.
mcs_status check_rope(const mcs_rope* r, mcs::RopeGeom* g, long long* entries) {
  if (r == nullptr || r->axes < 1 || r->axes > 3 || r->first < 0) return MCS_ERR_INVALID_ARG;
  if (r->style != MCS_ROPE_INTERLEAVED && r->style != MCS_ROPE_HALF) return MCS_ERR_UNSUPPORTED;
  if (!std::isfinite(r->theta) || r->theta <= 0.0) return MCS_ERR_INVALID_ARG;
  *g = mcs::RopeGeom{};
  long long off = 0, grid = 1;
  g->axes = r->axes;
  for (int a = 0; a < r->axes; ++a) {
    if (r->dims[a] < 2 || r->dims[a] % 2 != 0 || r->dims[a] > 128) return MCS_ERR_UNSUPPORTED;
    if (r->len[a] < 1) return MCS_ERR_INVALID_ARG;
    if (!std::isfinite(r->start[a]) || !std::isfinite(r->scale[a])) return MCS_ERR_INVALID_ARG;
    // the largest angle: theta^(-2 j / dims) lies between 1 and 1 / theta
    const double f = r->theta < 1.0 ? 1.0 / r->theta : 1.0;
    if (!std::isfinite((std::fabs(r->start[a]) + r->len[a]) * std::fabs(r->scale[a]) * f)) return MCS_ERR_INVALID_ARG;
    g->pairs[a] = r->dims[a] / 2;
    g->len[a] = r->len[a];
    g->by[a] = mcs::Divisor(r->len[a]);
    g->toff[a] = int(off);
    g->npairs += g->pairs[a];
    off += static_cast<long long>(r->len[a]) * g->pairs[a];
    if (off >= (1ll << 31)) return MCS_ERR_UNSUPPORTED;
    if (grid < (1ll << 31)) grid *= r->len[a];  // saturates above any token count
  }
  g->first = r->first;
  g->ngrid = grid < (1ll << 31) ? int(grid) : INT32_MAX;
  *entries = off;
  return MCS_OK;
}

// The rope against the problem it is applied to.
mcs_status check_rope_use(const mcs_desc* desc, const mcs_rope* r, const float* table, const int32_t* pos,
                          mcs::RopeGeom* g) {
  mcs_status st = mcs::validate_desc(desc);
  if (st != MCS_OK) return st;
  long long entries = 0;
  if ((st = check_rope(r, g, &entries)) != MCS_OK) return st;
  if (2 * g->npairs > desc->d) return MCS_ERR_UNSUPPORTED;
  if (r->style == MCS_ROPE_HALF && 2 * g->npairs != desc->d) return MCS_ERR_UNSUPPORTED;
  if (!aligned16(table) || !aligned16_or_null(pos)) return MCS_ERR_INVALID_ARG;
  if (pos == nullptr && static_cast<long long>(g->first) + g->ngrid > desc->N) return MCS_ERR_INVALID_ARG;
  return MCS_OK;
}

// Strides of a [B,H,N,d] view in elements; false unless each one that counts is
// a non-negative multiple of 16 bytes and, for a written view, rows are apart.
bool view(const mcs_desc* desc, const mcs_strides* s, bool written, mcs::ViewStrides* o) {
  const long long d = desc->d, es = desc->dtype == MCS_BF16 ? 2 : 4;
  if (s == nullptr) {
    *o = {static_cast<long long>(desc->H) * desc->N * d, static_cast<long long>(desc->N) * d, d};
    return true;
  }
  *o = {desc->B > 1 ? s->batch : 0, desc->H > 1 ? s->head : 0, desc->N > 1 ? s->token : 0};
  long long st[3] = {o->b, o->h, o->n}, sz[3] = {desc->B, desc->H, desc->N};
  for (int i = 0; i < 3; ++i)
    if (st[i] < 0 || st[i] * es % 16 != 0 || st[i] > (1ll << 40)) return false;
  if (!written) return true;
  for (int i = 0; i < 2; ++i)  // ascending by stride
    for (int j = 0; j < 2 - i; ++j)
      if (st[j] > st[j + 1]) {
        const long long a = st[j], b = sz[j];
        st[j] = st[j + 1], sz[j] = sz[j + 1], st[j + 1] = a, sz[j + 1] = b;
      }
  long long extent = d;
  for (int i = 0; i < 3; ++i) {
    if (sz[i] == 1) continue;
    if (st[i] < extent) return false;
    extent = st[i] * (sz[i] - 1) + extent;
  }
  return true;
}

// From a view's first element to its last.
Range range(const mcs_desc* d, const void* p, const mcs::ViewStrides& v) {
  const long long n = (d->B - 1) * v.b + (d->H - 1) * v.h + (d->N - 1) * v.n + d->d;
  return {static_cast<const char*>(p), n * (d->dtype == MCS_BF16 ? 2 : 4)};
}
bool contiguous(const mcs_desc* d, const mcs::ViewStrides& v) {
  return (d->B == 1 || v.b == static_cast<long long>(d->H) * d->N * d->d) &&
         (d->H == 1 || v.h == static_cast<long long>(d->N) * d->d) && (d->N == 1 || v.n == d->d);
}

}  // namespace

namespace mcs {

// The checks of a product's description; fills its sizes.
mcs_status check_linear(const mcs_linear_desc* desc, mcs::LinearParams* p) {
  if (desc == nullptr) return MCS_ERR_INVALID_ARG;
  if (desc->B < 1 || desc->N < 1 || desc->in < 1 || desc->out < 1 || desc->heads < 0) return MCS_ERR_INVALID_ARG;
  if (desc->dtype != MCS_F32 && desc->dtype != MCS_BF16) return MCS_ERR_UNSUPPORTED;
  if (desc->act < MCS_ACT_NONE || desc->act > MCS_ACT_SILU) return MCS_ERR_UNSUPPORTED;
  const bool bf16 = desc->dtype == MCS_BF16;
  const long long rows = static_cast<long long>(desc->B) * desc->N;
  if (desc->in > (1 << 20) || desc->out > (1 << 20) || rows >= (1ll << 31) - 256) return MCS_ERR_UNSUPPORTED;
  if (desc->in % (bf16 ? 8 : 4) != 0) return MCS_ERR_UNSUPPORTED;
  if (desc->heads > 0 && desc->in != 64ll * desc->heads && desc->in != 128ll * desc->heads) return MCS_ERR_UNSUPPORTED;
  if (static_cast<long long>(desc->B) * (desc->heads > 0 ? desc->heads : 1) >= (1ll << 31)) return MCS_ERR_UNSUPPORTED;
  p->B = desc->B;
  p->N = desc->N;
  p->M = int(rows);
  p->K = desc->in;
  p->O = desc->out;
  p->heads = desc->heads;
  p->act = desc->act;
  return MCS_OK;
}

}  // namespace mcs

extern "C" {

size_t mcs_rope_table_size(const mcs_rope* rope) {
  mcs::RopeGeom g;
  long long entries = 0;
  if (check_rope(rope, &g, &entries) != MCS_OK) return 0;
  return size_t(entries) * sizeof(float2);
}

mcs_status mcs_rope_table(const mcs_rope* rope, float* table, mcs_stream stream) {
  mcs::RopeTableParams p{};
  long long entries = 0;
  const mcs_status st = check_rope(rope, &p.g, &entries);
  if (st != MCS_OK) return st;
  if (!aligned16(table)) return MCS_ERR_INVALID_ARG;
  for (int a = 0; a < rope->axes; ++a) p.start[a] = rope->start[a], p.scale[a] = rope->scale[a];
  p.theta = rope->theta;
  p.table = reinterpret_cast<float2*>(table);
  return from_cuda(mcs::rope_table(p, reinterpret_cast<cudaStream_t>(stream)));
}

mcs_status mcs_rope_apply(const mcs_desc* desc, const mcs_rope* rope, const float* table, const int32_t* pos,
                          const void* x, const mcs_strides* xs, void* out, const mcs_strides* os, int inverse,
                          mcs_stream stream) {
  mcs::RotateParams p{};
  mcs_status st = check_rope_use(desc, rope, table, pos, &p.g);
  if (st != MCS_OK) return st;
  if (!aligned16(x) || !aligned16(out)) return MCS_ERR_INVALID_ARG;
  if (!view(desc, xs, false, &p.in) || !view(desc, os, true, &p.out)) return MCS_ERR_INVALID_ARG;
  if (x == out && (p.in.b != p.out.b || p.in.h != p.out.h || p.in.n != p.out.n)) return MCS_ERR_INVALID_ARG;
  int sms = 0;
  if ((st = mcs::current_device(&p.status, &sms)) != MCS_OK) return st;
  p.src[0] = x;
  p.dst[0] = out;
  p.table = reinterpret_cast<const float2*>(table);
  p.pos = pos;
  p.sin_sign = inverse ? -1.f : 1.f;
  p.B = desc->B, p.H = desc->H, p.N = desc->N;
  return from_cuda(mcs::rotate(desc->dtype == MCS_BF16, desc->d, rope->style == MCS_ROPE_HALF, false, p, sms,
                               reinterpret_cast<cudaStream_t>(stream)));
}

mcs_status mcs_qk_norm_rope(const mcs_desc* desc, const mcs_rope* rope, const float* table, const int32_t* pos,
                            const void* q, const void* k, const void* v, const mcs_strides* in, const void* wq,
                            const void* wk, float eps, void* q_out, void* k_out, void* v_out, mcs_stream stream) {
  mcs::RotateParams p{};
  mcs_status st = check_rope_use(desc, rope, table, pos, &p.g);
  if (st != MCS_OK) return st;
  const void* src[3] = {q, k, v};
  void* dst[3] = {q_out, k_out, v_out};
  if (q == nullptr && k == nullptr && v == nullptr) return MCS_ERR_INVALID_ARG;
  for (int i = 0; i < 3; ++i) {
    if ((src[i] == nullptr) != (dst[i] == nullptr)) return MCS_ERR_INVALID_ARG;
    if (!aligned16_or_null(src[i]) || !aligned16_or_null(dst[i])) return MCS_ERR_INVALID_ARG;
    p.src[i] = src[i];
    p.dst[i] = dst[i];
  }
  if (!aligned16_or_null(wq) || !aligned16_or_null(wk)) return MCS_ERR_INVALID_ARG;
  if (!std::isfinite(eps) || eps <= 0.f) return MCS_ERR_INVALID_ARG;
  if (!view(desc, in, false, &p.in) || !view(desc, nullptr, true, &p.out)) return MCS_ERR_INVALID_ARG;
  for (int i = 0; i < 3; ++i) {  // an output may only be its own input, row by row
    const Range out = range(desc, dst[i], p.out);
    for (int j = 0; j < 3; ++j) {
      if (j < i && overlap(out, range(desc, dst[j], p.out))) return MCS_ERR_INVALID_ARG;
      if (i == j && src[j] == dst[i] && contiguous(desc, p.in)) continue;
      if (overlap(out, range(desc, src[j], p.in))) return MCS_ERR_INVALID_ARG;
    }
  }
  int sms = 0;
  if ((st = mcs::current_device(&p.status, &sms)) != MCS_OK) return st;
  p.w[0] = wq;
  p.w[1] = wk;
  p.eps = eps;
  p.table = reinterpret_cast<const float2*>(table);
  p.pos = pos;
  p.sin_sign = 1.f;
  p.B = desc->B, p.H = desc->H, p.N = desc->N;
  return from_cuda(mcs::rotate(desc->dtype == MCS_BF16, desc->d, rope->style == MCS_ROPE_HALF, true, p, sms,
                               reinterpret_cast<cudaStream_t>(stream)));
}

size_t mcs_qk_norm_rope_bwd_workspace_size(const mcs_desc* desc) {
  if (mcs::validate_desc(desc) != MCS_OK) return 0;
  return size_t(mcs::kNormBwdMaxBlocks) * 2 * desc->d * sizeof(float);
}

mcs_status mcs_qk_norm_rope_bwd(const mcs_desc* desc, const mcs_rope* rope, const float* table, const int32_t* pos,
                                const void* q, const void* k, const mcs_strides* in, const void* wq, const void* wk,
                                float eps, const void* dq_out, const void* dk_out, const void* dv_out, void* dq,
                                void* dk, void* dv, float* dwq, float* dwk, void* ws, size_t ws_bytes,
                                mcs_stream stream) {
  mcs::NormBwdParams p{};
  mcs_status st = check_rope_use(desc, rope, table, pos, &p.g);
  if (st != MCS_OK) return st;
  const void* dy[3] = {dq_out, dk_out, dv_out};
  void* dx[3] = {dq, dk, dv};
  const void* x[2] = {q, k};
  const void* w[2] = {wq, wk};
  float* dw[2] = {dwq, dwk};
  if (dq_out == nullptr && dk_out == nullptr && dv_out == nullptr) return MCS_ERR_INVALID_ARG;
  for (int i = 0; i < 3; ++i) {
    if ((dy[i] == nullptr) != (dx[i] == nullptr)) return MCS_ERR_INVALID_ARG;
    if (!aligned16_or_null(dy[i]) || !aligned16_or_null(dx[i])) return MCS_ERR_INVALID_ARG;
    p.dy[i] = dy[i];
    p.dx[i] = dx[i];
    if (i == 2) break;
    if ((dy[i] == nullptr) != (x[i] == nullptr) || !aligned16_or_null(x[i])) return MCS_ERR_INVALID_ARG;
    if (dy[i] == nullptr && dw[i] != nullptr) return MCS_ERR_INVALID_ARG;
    if (!aligned16_or_null(w[i]) || !aligned16_or_null(dw[i])) return MCS_ERR_INVALID_ARG;
    p.x[i] = x[i];
    p.w[i] = w[i];
    p.dw[i] = dw[i];
  }
  if (!std::isfinite(eps) || eps <= 0.f) return MCS_ERR_INVALID_ARG;
  if (!view(desc, in, true, &p.in)) return MCS_ERR_INVALID_ARG;
  if (!aligned16(ws) || ws_bytes < mcs_qk_norm_rope_bwd_workspace_size(desc)) return MCS_ERR_WORKSPACE;
  mcs::ViewStrides block;
  view(desc, nullptr, true, &block);
  if (dwq != nullptr && dwq == dwk) return MCS_ERR_INVALID_ARG;
  for (int i = 0; i < 3; ++i) {  // a gradient may only take the place of its own stream's tensors, row by row
    if (dx[i] == nullptr) continue;
    for (int j = 0; j < 3; ++j) {
      if (i != j && (dx[i] == dx[j] || (j < 2 && dx[i] == x[j]))) return MCS_ERR_INVALID_ARG;
      if (i == j && dx[i] == dy[j] && contiguous(desc, p.in)) continue;
      if (overlap(range(desc, dx[i], p.in), range(desc, dy[j], block))) return MCS_ERR_INVALID_ARG;
    }
  }
  int sms = 0;
  if ((st = mcs::current_device(&p.status, &sms)) != MCS_OK) return st;
  p.partial = static_cast<float*>(ws);
  p.eps = eps;
  p.table = reinterpret_cast<const float2*>(table);
  p.pos = pos;
  p.B = desc->B, p.H = desc->H, p.N = desc->N;
  return from_cuda(mcs::qk_norm_rope_bwd(desc->dtype == MCS_BF16, desc->d, rope->style == MCS_ROPE_HALF, p, sms,
                                         reinterpret_cast<cudaStream_t>(stream)));
}

mcs_status mcs_linear(const mcs_linear_desc* desc, const void* x, const void* w, const void* bias, const void* gate,
                      const void* residual, void* y, mcs_stream stream) {
  mcs::LinearParams p{};
  mcs_status st = mcs::check_linear(desc, &p);
  if (st != MCS_OK) return st;
  if (!aligned16(x) || !aligned16(w) || !aligned16(y)) return MCS_ERR_INVALID_ARG;
  if (!aligned16_or_null(bias) || !aligned16_or_null(gate) || !aligned16_or_null(residual)) return MCS_ERR_INVALID_ARG;
  const bool bf16 = desc->dtype == MCS_BF16;
  const long long es = bf16 ? 2 : 4, out = desc->out, rows = p.M;
  const Range written = range(y, rows * out * es);
  if (overlap(written, range(x, rows * desc->in * es)) || overlap(written, range(w, out * desc->in * es)) ||
      overlap(written, range(bias, out * es)) || overlap(written, range(gate, desc->B * out * es)))
    return MCS_ERR_INVALID_ARG;
  if (residual != y && overlap(written, range(residual, rows * out * es))) return MCS_ERR_INVALID_ARG;
  int sms = 0;
  if ((st = mcs::current_device(&p.status, &sms)) != MCS_OK) return st;
  p.x = x;
  p.w = w;
  p.bias = bias;
  p.gate = gate;
  p.residual = residual;
  p.y = y;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return from_cuda(bf16 ? mcs::linear_tc(p, sms, s) : mcs::linear_f32(p, sms, s));
}

mcs_status mcs_linear_plan(const mcs_linear_desc* desc, int with_residual, int num_sms, mcs_linear_choice* choice) {
  mcs::LinearParams p{};
  const mcs_status st = mcs::check_linear(desc, &p);
  if (st != MCS_OK) return st;
  if (num_sms < 8 || num_sms > 1024 || choice == nullptr) return MCS_ERR_INVALID_ARG;
  p.residual = with_residual ? choice : nullptr;  // only whether there is one
  const mcs::LinearPlan plan = desc->dtype == MCS_BF16 ? mcs::plan_linear_tc(p, num_sms) : mcs::plan_linear_f32(p, num_sms);
  *choice = {plan.kernel, plan.tile, plan.slices, plan.accumulators};
  return MCS_OK;
}

}  // extern "C"
