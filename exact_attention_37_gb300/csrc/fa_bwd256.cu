// Launch of the d = 256 backward kernel of plain attention (fa_bwd256.cuh).
#include "fa_bwd256.cuh"

namespace fa {

cudaError_t launch_bwd_main_256(bool bf16, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                                const CUtensorMap& dout, const BwdArgs& a, cudaStream_t stream) {
  return bf16 ? launch_256<true, kRuleOff>(q, k, v, dout, a, stream)
              : launch_256<false, kRuleOff>(q, k, v, dout, a, stream);
}

}  // namespace fa
