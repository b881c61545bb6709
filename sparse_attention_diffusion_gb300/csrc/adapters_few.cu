// The few-rows matrix product with adapters, and which kernel a product with adapters takes.
#include "linear_few.cuh"

namespace mcs {

cudaError_t linear_adapters_pair(const LinearParams& p, int bn, const AdapterParams& a, int num_sms, cudaStream_t s);

cudaError_t linear_adapters_tc(const LinearParams& p, const AdapterParams& a, int num_sms, cudaStream_t s) {
  const LinearPlan plan = plan_linear_tc(p, num_sms);
  return plan.kernel == MCS_LINEAR_FEW ? launch_few<true>(p, {plan.tile, plan.slices}, &a, num_sms, s)
                                       : linear_adapters_pair(p, plan.tile, a, num_sms, s);
}

}  // namespace mcs
