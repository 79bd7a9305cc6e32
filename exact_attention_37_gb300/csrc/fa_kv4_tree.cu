// Attention of a tree of drafted tokens of each sequence over its paged 4-bit cache: the
// kernels of fa_kv4_attend.cuh with a tree, and the choice between them and the kernel for many
// rows (fa_kv4_wide.cuh).
#include "fa_kv4_attend.cuh"

namespace fa {

bool kv4_tree_wide(int d, int cols) { return cols > kv4_unit_cols(d, cols) && cols <= 1 << 20; }

cudaError_t launch_kv4_tree(Kv4TreeArgs a, int d, bool bf16, long long tokens_bound, int num_sms, cudaStream_t stream) {
  if (kv4_tree_wide(d, a.cols)) {
    const long long room = (long long)a.pool.max_pages << a.pool.page_shift;
    return launch_kv4_wide(a, d, bf16, room, num_sms, stream);
  }
  return launch_units(a, d, bf16, tokens_bound, num_sms, stream);
}

}  // namespace fa
