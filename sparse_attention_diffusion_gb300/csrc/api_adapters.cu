// C ABI of projections with low-rank adapters (declared in include/mcs.h): argument
// validation and dispatch. No C++ exception and no device allocation here.
#include <cstdint>

#include "mcs.h"
#include "adapters.h"
#include "api_checks.h"
#include "api_internal.h"
#include "common.cuh"
#include "linear.h"

namespace {

using mcs::aligned16;
using mcs::aligned16_or_null;
using mcs::overlap;
using mcs::Range;

mcs_status check_adapters(const mcs_linear_desc* desc, const mcs_adapters* ad, mcs::LinearParams* p, mcs::AdapterParams* a) {
  const mcs_status st = mcs::check_linear(desc, p);
  if (st != MCS_OK) return st;
  if (ad == nullptr || ad->count < 1 || ad->rank < 1 || ad->segments < 1) return MCS_ERR_INVALID_ARG;
  if (ad->rank > 256 || ad->rank % (desc->dtype == MCS_BF16 ? 8 : 4) != 0) return MCS_ERR_UNSUPPORTED;
  if (ad->count > (1 << 20) || ad->segments > (1 << 20)) return MCS_ERR_UNSUPPORTED;
  a->count = ad->count;
  a->R = ad->rank;
  a->S = ad->segments;
  return MCS_OK;
}

}  // namespace

extern "C" {

size_t mcs_linear_adapters_workspace_size(const mcs_linear_desc* desc, const mcs_adapters* adapters) {
  mcs::LinearParams p{};
  mcs::AdapterParams a{};
  if (check_adapters(desc, adapters, &p, &a) != MCS_OK) return 0;
  return mcs::adapters_workspace_bytes(p, a, desc->dtype == MCS_BF16);
}

mcs_status mcs_linear_adapters(const mcs_linear_desc* desc, const mcs_adapters* adapters, const void* x, const void* w,
                               const void* bias, const void* gate, const void* residual, const void* down, const void* up,
                               const float* scale, const int32_t* start, const int32_t* which, void* y, void* ws,
                               size_t ws_bytes, mcs_stream stream) {
  mcs::LinearParams p{};
  mcs::AdapterParams a{};
  mcs_status st = check_adapters(desc, adapters, &p, &a);
  if (st != MCS_OK) return st;
  if (!aligned16(x) || !aligned16(w) || !aligned16(y) || !aligned16(down) || !aligned16(up)) return MCS_ERR_INVALID_ARG;
  if (!aligned16_or_null(bias) || !aligned16_or_null(gate) || !aligned16_or_null(residual)) return MCS_ERR_INVALID_ARG;
  if (!aligned16(scale) || !aligned16(start) || !aligned16(which)) return MCS_ERR_INVALID_ARG;
  const bool bf16 = desc->dtype == MCS_BF16;
  const size_t need = mcs::adapters_workspace_bytes(p, a, bf16);
  if (!aligned16(ws) || ws_bytes < need) return MCS_ERR_WORKSPACE;
  const long long es = bf16 ? 2 : 4, in = desc->in, out = desc->out, rows = p.M;
  const Range read[] = {mcs::range(x, rows * in * es), mcs::range(w, out * in * es), mcs::range(bias, out * es),
                        mcs::range(gate, desc->B * out * es), mcs::range(down, static_cast<long long>(a.count) * a.R * in * es),
                        mcs::range(up, static_cast<long long>(a.count) * a.R * out * es), mcs::range(scale, 4ll * a.count),
                        mcs::range(start, 4ll * a.S + 4), mcs::range(which, 4ll * a.S)};
  const Range res = mcs::range(residual, rows * out * es), dst = mcs::range(y, rows * out * es),
              scratch = mcs::range(ws, static_cast<long long>(need));
  for (const Range& r : read)
    if (overlap(dst, r) || overlap(scratch, r)) return MCS_ERR_INVALID_ARG;
  if (overlap(scratch, dst) || overlap(scratch, res) || (residual != y && overlap(dst, res))) return MCS_ERR_INVALID_ARG;
  int sms = 0;
  if ((st = mcs::current_device(&p.status, &sms)) != MCS_OK) return st;
  p.x = x;
  p.w = w;
  p.bias = bias;
  p.gate = gate;
  p.residual = residual;
  p.y = y;
  a.down = down;
  a.up = up;
  a.scale = scale;
  a.start = start;
  a.which = which;
  a.ws = ws;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return mcs::from_cuda(bf16 ? mcs::linear_adapters_tc(p, a, sms, s) : mcs::linear_adapters_f32(p, a, sms, s));
}

}  // extern "C"
