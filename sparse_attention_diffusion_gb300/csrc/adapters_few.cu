// The few-rows matrix product with adapters, and which kernel a product with adapters takes.
#include "linear_few.cuh"

namespace mcs {

cudaError_t linear_adapters_pair(const LinearParams& p, int bn, const AdapterParams& a, int num_sms, cudaStream_t s);

// Few rows: a segment's k steps cost some 400 clocks for 64 columns of either part of h, whatever its rows; on the CUDA
// cores a row costs its block 128 x R elements of `up` (4 R clocks at what an SM reads from L2). So segments of less
// than 800 / 4 R rows on average go there (64 rows with adapters of their own of rank 16 to 4,096 x 4,096: 36 us by k steps,
// 18.6 on the CUDA cores).
cudaError_t linear_adapters_tc(const LinearParams& p, const AdapterParams& a, int num_sms, cudaStream_t s) {
  const LinearPlan plan = plan_linear_tc(p, num_sms);
  if (plan.kernel != MCS_LINEAR_FEW) return linear_adapters_pair(p, plan.tile, a, num_sms, s);
  const bool rows = static_cast<long long>(p.M) * a.R <= 200ll * ((a.R + 63) / 64) * a.S;
  return rows ? launch_few<kAdapterRows>(p, {plan.tile, plan.slices}, &a, num_sms, s)
              : launch_few<kAdapterSteps>(p, {plan.tile, plan.slices}, &a, num_sms, s);
}

}  // namespace mcs
