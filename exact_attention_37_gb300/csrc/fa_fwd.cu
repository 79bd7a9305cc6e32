// Launch of the forward kernel of plain attention (the kernel is in fa_fwd.cuh).
#include "fa_fwd.cuh"

namespace fa {

int fwd_rows_per_cta(int d, long long BH, int N, int num_sms) {
  if (d == 256) return kBM;
  const long long ctas = BH * (((long long)N + 2 * kBM - 1) / (2 * kBM));
  return ctas < num_sms ? kBM : 2 * kBM;
}

cudaError_t launch_fwd(int d, bool bf16, int rows, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                       const CUtensorMap& o, const FwdArgs& a, cudaStream_t stream) {
  return launch_fwd_r<kRuleOff>(d, bf16, rows, q, k, v, o, a, stream);
}

}  // namespace fa
