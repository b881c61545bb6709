// C ABI of attention over packed sequences (declared in include/mcs.h): argument
// validation and dispatch. No C++ exception and no device allocation here.
#include <cmath>
#include <cstdint>

#include "mcs.h"
#include "api_checks.h"
#include "api_internal.h"
#include "common.cuh"
#include "packed.h"

namespace {

using mcs::aligned16;
using mcs::from_cuda;
using mcs::overlap;
using mcs::Range;

// The checks of a description; fills its sizes and the plan. own_keys: every sequence's keys are as many as its queries.
mcs_status check_packed(const mcs_packed_desc* d, mcs::PackedParams* p, bool own_keys) {
  if (d == nullptr) return MCS_ERR_INVALID_ARG;
  if (d->S < 1 || d->Tq < 1 || d->Tk < 1 || d->H < 1 || d->Hk < 1 || d->H % d->Hk != 0) return MCS_ERR_INVALID_ARG;
  if (d->max_q < 0 || !std::isfinite(d->scale)) return MCS_ERR_INVALID_ARG;
  if (d->dtype != MCS_F32 && d->dtype != MCS_BF16) return MCS_ERR_UNSUPPORTED;
  if ((d->d != 64 && d->d != 128) || d->H / d->Hk > 64) return MCS_ERR_UNSUPPORTED;
  constexpr int kMost = 1 << 30;
  if (d->S > kMost || d->Tq > kMost || d->Tk > kMost || d->H > (1 << 20)) return MCS_ERR_UNSUPPORTED;
  p->S = d->S, p->Tq = d->Tq, p->Tk = d->Tk, p->H = d->H, p->Hk = d->Hk, p->d = d->d;
  p->causal = d->causal != 0;
  p->max_q = d->max_q > 0 && d->max_q < d->Tq ? d->max_q : d->Tq;
  p->scale_log2 = (d->scale > 0.f ? d->scale : 1.f / std::sqrt(float(d->d))) * mcs::kLog2e;
  if (!std::isfinite(p->scale_log2)) return MCS_ERR_INVALID_ARG;  // a score of 0 would become NaN
  return mcs::plan_packed(p, d->dtype == MCS_BF16, own_keys && p->max_q < p->Tk ? p->max_q : p->Tk) ? MCS_OK : MCS_ERR_UNSUPPORTED;
}

// Strides of a [heads, tokens, d] view in elements (NULL: contiguous); false unless rows are apart and each stride
// that counts is a multiple of 16 bytes. bytes: from the first element to the last.
bool view(const mcs_strides* s, long long heads, long long tokens, long long d, int es, mcs::PackedStrides* o, long long* bytes) {
  *o = {heads > 1 ? (s ? s->head : tokens * d) : 0, tokens > 1 ? (s ? s->token : d) : 0};
  for (const long long st : {o->head, o->token})
    if (st < 0 || st * es % 16 != 0 || st > (1ll << 38)) return false;
  const bool head_first = tokens > 1 && (heads == 1 || o->token <= o->head);  // tokens inside a head
  const long long inner = head_first ? o->token : o->head, ni = head_first ? tokens : heads;
  const long long outer = head_first ? o->head : o->token, no = head_first ? heads : tokens;
  if (ni > 1 && inner < d) return false;
  const long long extent = (ni - 1) * inner + d;
  if (no > 1 && outer < extent) return false;
  *bytes = ((no - 1) * outer + extent) * es;
  return true;
}

}  // namespace

extern "C" {

size_t mcs_packed_attn_workspace_size(const mcs_packed_desc* desc) {
  mcs::PackedParams p{};
  return check_packed(desc, &p, false) == MCS_OK ? mcs::packed_workspace_bytes(p) : 0;
}

mcs_status mcs_packed_attn(const mcs_packed_desc* desc, const void* q, const mcs_strides* qs, const void* k,
                           const mcs_strides* ks, const void* v, const mcs_strides* vs, const int32_t* q_start,
                           const int32_t* k_start, void* o, const mcs_strides* os, float* lse, void* ws, size_t ws_bytes,
                           mcs_stream stream) {
  mcs::PackedParams p{};
  mcs_status st = check_packed(desc, &p, q_start == k_start);
  if (st != MCS_OK) return st;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !mcs::aligned16_or_null(lse)) return MCS_ERR_INVALID_ARG;
  if (!aligned16(q_start) || !aligned16(k_start)) return MCS_ERR_INVALID_ARG;
  const bool bf16 = desc->dtype == MCS_BF16;
  const int es = bf16 ? 2 : 4;
  long long nq = 0, nk = 0, nv = 0, no = 0;
  if (!view(qs, p.H, p.Tq, p.d, es, &p.qs, &nq) || !view(ks, p.Hk, p.Tk, p.d, es, &p.ks, &nk) ||
      !view(vs, p.Hk, p.Tk, p.d, es, &p.vs, &nv) || !view(os, p.H, p.Tq, p.d, es, &p.os, &no))
    return MCS_ERR_INVALID_ARG;
  const size_t need = mcs::packed_workspace_bytes(p);
  if (!aligned16(ws) || ws_bytes < need) return MCS_ERR_WORKSPACE;
  // what is written: the output, the log-sum-exp and the workspace
  const Range in[] = {mcs::range(q, nq), mcs::range(k, nk), mcs::range(v, nv), mcs::range(q_start, 4ll * p.S + 4),
                      mcs::range(k_start, 4ll * p.S + 4)};
  const Range out[] = {mcs::range(o, no), mcs::range(lse, 4ll * p.H * p.Tq), mcs::range(ws, static_cast<long long>(need))};
  for (int i = 0; i < 3; ++i) {
    for (const Range& r : in)
      if (overlap(out[i], r)) return MCS_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (overlap(out[i], out[j])) return MCS_ERR_INVALID_ARG;
  }
  if ((st = mcs::current_device(&p.status, &p.sms)) != MCS_OK) return st;
  p.q = q, p.k = k, p.v = v, p.o = o, p.lse = lse;
  p.q_start = q_start, p.k_start = k_start;
  p.taken = static_cast<uint32_t*>(ws);
  p.part_o = static_cast<float*>(ws) + (p.banks > 0 ? mcs::kTakenBytes / 4 : 0);
  p.part_ml = reinterpret_cast<float2*>(p.part_o + size_t(p.items) * p.part_rows * p.d);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return from_cuda(bf16 ? mcs::packed_attn_tc(p, s) : mcs::packed_attn_f32(p, s));
}

}  // extern "C"
