// The forward kernel with a score rule of one kind, FA_RULE_KIND (the kernel is in
// fa_fwd.cuh, the rules in fa_rule.cuh); compiled once for each kind.
#include "fa_fwd.cuh"

namespace fa {

template <>
cudaError_t launch_fwd_rule_kind<FA_RULE_KIND>(int d, bool bf16, int rows, const CUtensorMap& q, const CUtensorMap& k,
                                               const CUtensorMap& v, const CUtensorMap& o, const FwdRuleArgs& a,
                                               cudaStream_t stream) {
  return launch_fwd_r<FA_RULE_KIND>(d, bf16, rows, q, k, v, o, a, stream);
}

}  // namespace fa
