// Attention of a tree of drafted tokens of each sequence over its paged 4-bit cache: the
// kernels of fa_kv4_attend.cuh with a tree.
#include "fa_kv4_attend.cuh"

namespace fa {

cudaError_t launch_kv4_tree(Kv4TreeArgs a, int d, bool bf16, long long tokens_bound, int num_sms, cudaStream_t stream) {
  return launch_units(a, d, bf16, tokens_bound, num_sms, stream);
}

}  // namespace fa
