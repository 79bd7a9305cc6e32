// Launch of the forward kernel with a score rule (the kernel is in fa_fwd.cuh, the rules
// in fa_rule.cuh).
#include "fa_fwd.cuh"

namespace fa {

cudaError_t launch_fwd_rule(int kind, int d, bool bf16, int rows, const CUtensorMap& q, const CUtensorMap& k,
                            const CUtensorMap& v, const CUtensorMap& o, const FwdRuleArgs& a, cudaStream_t stream) {
  switch (kind) {
    case kRuleMask: return launch_fwd_r<kRuleMask>(d, bf16, rows, q, k, v, o, a, stream);
    case kRuleBias: return launch_fwd_r<kRuleBias>(d, bf16, rows, q, k, v, o, a, stream);
    case kRuleCap: return launch_fwd_r<kRuleCap>(d, bf16, rows, q, k, v, o, a, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace fa
