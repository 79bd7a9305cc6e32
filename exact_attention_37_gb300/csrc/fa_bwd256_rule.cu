// Launch of the d = 256 backward kernel with a score rule (fa_bwd256.cuh).
#include "fa_bwd256.cuh"

namespace fa {
namespace {

template <int RULE>
cudaError_t launch_r(bool bf16, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                     const CUtensorMap& dout, const BwdRuleArgs& a, cudaStream_t stream) {
  return bf16 ? launch_256<true, RULE>(q, k, v, dout, a, stream) : launch_256<false, RULE>(q, k, v, dout, a, stream);
}

}  // namespace

cudaError_t launch_bwd_256_rule(int kind, bool bf16, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                                const CUtensorMap& dout, const BwdRuleArgs& a, cudaStream_t stream) {
  switch (kind) {
    case kRuleMask: return launch_r<kRuleMask>(bf16, q, k, v, dout, a, stream);
    case kRuleBias: return launch_r<kRuleBias>(bf16, q, k, v, dout, a, stream);
    case kRuleCap: return launch_r<kRuleCap>(bf16, q, k, v, dout, a, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace fa
