// The matrix product on CTA pairs with adapters.
#include "linear_pair.cuh"

namespace mcs {

cudaError_t linear_adapters_pair(const LinearParams& p, int bn, const AdapterParams& a, int num_sms, cudaStream_t s) {
  return launch_pair<kAdapterSteps>(p, bn, &a, num_sms, s);
}

}  // namespace mcs
