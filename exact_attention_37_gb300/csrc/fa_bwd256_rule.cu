// The d = 256 backward kernel with a score rule of one kind, FA_RULE_KIND (the kernel is
// in fa_bwd256.cuh, the rules in fa_rule.cuh); compiled once for each kind.
#include "fa_bwd256.cuh"

namespace fa {

template <>
cudaError_t launch_bwd_256_rule_kind<FA_RULE_KIND>(bool bf16, const CUtensorMap& q, const CUtensorMap& k,
                                                   const CUtensorMap& v, const CUtensorMap& dout, const BwdRuleArgs& a,
                                                   cudaStream_t stream) {
  return bf16 ? launch_256<true, FA_RULE_KIND>(q, k, v, dout, a, stream)
              : launch_256<false, FA_RULE_KIND>(q, k, v, dout, a, stream);
}

}  // namespace fa
