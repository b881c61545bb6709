// Host-side interface of the few-rows matrix product.
#pragma once
#include <cuda_runtime.h>

#include "linear.h"

namespace mcs {

struct FewPlan {
  int bn;      // tokens per tile: a multiple of 16, 16 .. 256
  int splits;  // K slices = CTAs of a cluster, 1 .. 8
};
// CTAs that run at once, one per SM: clusters of more than two leave SMs of a GPU
// processing cluster over (144 CTAs in clusters of three took two waves on 152 SMs).
inline int few_slots(int splits, int num_sms) {
  if (splits <= 2) return num_sms;
  const int clusters = int(0.85 * num_sms) / splits;
  return (clusters > 0 ? clusters : 1) * splits;
}
// Tensor memory: an accumulator's columns, and how many accumulators a slice of `steps` k steps holds at once. All
// of them stay until the end where they fit in half of the tensor memory; otherwise, up to 128 tokens, two take turns
// and their sums are kept in registers.
inline int few_acc_cols(int bn) { return (bn + 31) / 32 * 32; }
inline bool few_turns(int bn, int steps) {
  return bn <= 128 && acc_count(steps) * few_acc_cols(bn) > 256;
}
inline int few_accs(int bn, int steps) { return few_turns(bn, steps) ? 2 : acc_count(steps); }
inline bool few_fits(int bn, int steps) { return few_accs(bn, steps) * few_acc_cols(bn) <= 512; }
// Half of an SM's shared memory holds three stages (16 KB of w and bn x 128 bytes of x each) and the bn x 512
// bytes of the partial accumulator, and half of its tensor memory the accumulators.
constexpr int kFewHalfSm = 112 * 1024 - 1280;
inline bool few_two_per_sm(int bn, int steps) {
  const int stage = 16384 + bn * 128;
  return kFewHalfSm / stage >= 3 && kFewHalfSm / stage * stage >= bn * 512 && few_accs(bn, steps) * few_acc_cols(bn) <= 256;
}
cudaError_t linear_few(const LinearParams& p, const FewPlan& plan, int num_sms, cudaStream_t s);

}  // namespace mcs
