// The d = 64 and 128 backward kernels with a score rule of one kind, FA_RULE_KIND (the
// kernels are in fa_bwd_sq.cuh, the rules in fa_rule.cuh); compiled once for each kind.
#include "fa_bwd_sq.cuh"

namespace fa {

template <>
cudaError_t launch_bwd_sq_rule_kind<FA_RULE_KIND>(int d, bool bf16, const CUtensorMap& q, const CUtensorMap& k,
                                                  const CUtensorMap& v, const CUtensorMap& dout, const BwdRuleArgs& a,
                                                  cudaStream_t stream) {
  return launch_sq_r<FA_RULE_KIND>(d, bf16, q, k, v, dout, a, stream);
}

}  // namespace fa
