// Launch of the d = 64 and 128 backward kernels with a score rule (fa_bwd_sq.cuh).
#include "fa_bwd_sq.cuh"

namespace fa {

cudaError_t launch_bwd_sq_rule(int kind, int d, bool bf16, const CUtensorMap& q, const CUtensorMap& k,
                               const CUtensorMap& v, const CUtensorMap& dout, const BwdRuleArgs& a,
                               cudaStream_t stream) {
  switch (kind) {
    case kRuleMask: return launch_sq_r<kRuleMask>(d, bf16, q, k, v, dout, a, stream);
    case kRuleBias: return launch_sq_r<kRuleBias>(d, bf16, q, k, v, dout, a, stream);
    case kRuleCap: return launch_sq_r<kRuleCap>(d, bf16, q, k, v, dout, a, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace fa
