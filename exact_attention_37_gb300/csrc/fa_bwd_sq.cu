// Launch of the d = 64 and 128 backward kernels of plain attention (fa_bwd_sq.cuh).
#include "fa_bwd_sq.cuh"

namespace fa {

cudaError_t launch_bwd_main_sq(int d, bool bf16, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                               const CUtensorMap& dout, const BwdArgs& a, cudaStream_t stream) {
  return launch_sq_r<kRuleOff>(d, bf16, q, k, v, dout, a, stream);
}

}  // namespace fa
