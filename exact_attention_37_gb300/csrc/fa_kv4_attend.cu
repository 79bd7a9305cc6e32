// Attention of the last tokens of each sequence over its paged 4-bit cache: the kernels of
// fa_kv4_attend.cuh without a tree.
#include "fa_kv4_attend.cuh"

namespace fa {

int kv4_unit_cols(int d, int cols) {
  if (cols <= 8) return 8;
  return cols <= 16 || d > 64 ? 16 : 32;
}

cudaError_t launch_kv4_attend(Kv4AttendArgs a, int d, bool bf16, long long tokens_bound, int num_sms,
                              cudaStream_t stream) {
  return launch_units(a, d, bf16, tokens_bound, num_sms, stream);
}

}  // namespace fa
