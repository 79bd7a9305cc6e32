// Instances of the kernel for trees with many rows (fa_kv4_wide.cuh).
#include "fa_kv4_wide.cuh"

namespace fa {

cudaError_t launch_kv4_wide(const Kv4TreeArgs& a, int d, bool bf16, long long room, int num_sms, cudaStream_t stream) {
  switch (d) {
    case 64:
      return bf16 ? launch_wide_t<64, true>(a, room, num_sms, stream) : launch_wide_t<64, false>(a, room, num_sms, stream);
    case 128:
      return bf16 ? launch_wide_t<128, true>(a, room, num_sms, stream) : launch_wide_t<128, false>(a, room, num_sms, stream);
    case 256:
      return bf16 ? launch_wide_t<256, true>(a, room, num_sms, stream) : launch_wide_t<256, false>(a, room, num_sms, stream);
    default:
      return cudaErrorInvalidValue;
  }
}

}  // namespace fa
