// Attention of a tree of drafted tokens of each sequence over its paged 4-bit cache: the
// kernels of fa_kv4_attend.cuh with a tree, and the choice between them and the kernel for many
// rows (fa_kv4_wide.cuh).
#include "fa_kv4_attend.cuh"

namespace fa {

// (what it can take: rows for more than one unit of the other kernel's)
bool kv4_tree_wide(int d, int cols) { return cols > kv4_unit_cols(d, cols) && cols <= 1 << 20; }

namespace {
// Whether the kernel for many rows is the faster one.  It unpacks a key/value head's tokens once for up
// to 128 rows, where the other does so for each 16 (d = 64: 32) of them; but its tiles take blocks of
// their own, and a unit costs it 6 us beside them.  With x units of the other and room for n tokens a
// sequence, measured in bf16 at 1 to 64 sequences, 8 to 32 drafted tokens for groups of 4 or 8 query heads
// and 128 to 30000 tokens (us, other / this):
//   d 128  x 16 (1 sequence)   8000: 23 / 32    30000: 42 / 41
//          x 32                2000: 15 / 20     4000: 28 / 23    30000: 72 / 34
//          x 128 (8)            300: 18 / 20     1000: 29 / 23    30000: 117 / 70
//          x 256                128: 15 / 16      300: 33 / 20     8000: 107 / 39
//          x 1024 (32)          128: 70 / 22     2000: 168 / 52    8000: 332 / 87
//   d 256  x 16                2000: 20 / 27     8000: 38 / 33
//          x 32                2000: 22 / 28     4000: 49 / 31
//          x 256                128: 23 / 34      300: 52 / 36     8000: 191 / 70
//   d 64   x 16                2000: 16 / 17     4000: 22 / 21    30000: 49 / 31
//          x 32                 517: 15 / 14     4000: 31 / 20
// The other has all of its units under way at once while x is small, hence the square.
bool wide_is_faster(const Kv4TreeArgs& a, int d, long long room) {
  const int unit = kv4_unit_cols(d, a.cols);
  const double x = (double)a.B * a.pool.H_kv * ((a.cols + unit - 1) / unit), work = x * room * (d == 64 ? 8 : 1);
  return work >= 3 << 14 && x * work >= 1 << 22;
}
}  // namespace

// (the parts of either kernel fit behind part_o and part_ml: 2 kKv4MaxCtas units of up to 32 columns are
// 2 kWideMaxCtas of kWideRows)
static_assert(kKv4MaxCtas * 32 <= kWideMaxCtas * kWideRows, "parts");
cudaError_t launch_kv4_tree(Kv4TreeArgs a, int d, bool bf16, long long tokens_bound, int num_sms, cudaStream_t stream) {
  const long long room = (long long)a.pool.max_pages << a.pool.page_shift;
  if (kv4_tree_wide(d, a.cols) && wide_is_faster(a, d, room)) return launch_kv4_wide(a, d, bf16, room, num_sms, stream);
  return launch_units(a, d, bf16, tokens_bound, num_sms, stream);
}

}  // namespace fa
