// The few-rows matrix product without adapters.
#include "linear_few.cuh"

namespace mcs {

cudaError_t linear_few(const LinearParams& p, const FewPlan& plan, int num_sms, cudaStream_t s) {
  return launch_few<kNoAdapters>(p, plan, nullptr, num_sms, s);
}

}  // namespace mcs
