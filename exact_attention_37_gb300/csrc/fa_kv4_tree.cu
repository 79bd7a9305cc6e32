// Attention of a tree of drafted tokens of each sequence over its paged 4-bit cache: the
// kernels of fa_kv4_attend.cuh with a tree, and the choice between them and the kernel for many
// rows (fa_kv4_wide.cuh).
#include "fa_kv4_attend.cuh"

namespace fa {

// (what it can take: rows for more than one unit of the other kernel's)
bool kv4_tree_wide(int d, int cols) { return cols > kv4_unit_cols(d, cols) && cols <= 1 << 20; }

// Whether the kernel for many rows takes a call: where it is the faster one.  It unpacks a key/value head's
// tokens once for up to 128 rows, where the other does so for each 16 (d = 64: 32) of them; but it has one
// block an SM, and a unit of 128 rows costs it 6 us beside its tokens.  With x units of the other and y of this
// one, and room for n tokens a sequence:
//   Where the other runs as clusters that are all on the GPU at once (cluster_ctas), it is the faster one, but
//   for short sequences at d 64 and 256.  Else this one is, from some number of units on, or from fewer of
//   them when the tokens are many: x^3 n / y is what a regression of the times gives.  It needs four times as
//   much where a sequence's rows end in a tile of up to 32 (at d 64 and 128 four copies, whose parts the join
//   takes one after the other).
// Measured (us, other / this; the table's room is the longest sequence's):
//   d 64    n 64      x 64   14.0 / 11.6                           d 128   n 64      x 64   12.7 / 13.8    x 512  34.2 / 22.6
//           n 320     x 64   15.2 / 16.7    x 128  21.5 / 16.8             n 320     x 16   11.1 / 15.7
//           n 1024    x 2    12.7 / 13.5                                   n 1024    x 32   12.5 / 19.7    x 512  68.9 / 37.7
//           n 2560    x 24   24.0 / 16.7                                   n 2560    x 12   16.9 / 29.3    x 48   27.1 / 20.3
//           n 24000   x 3    22.4 / 37.0    x 12   38.0 / 27.8             n 12032   x 16   26.8 / 33.8    x 32   36.9 / 27.2
//           n 300032  x 3    73.1 / 51.1                                   n 300032  x 3    62.5 / 77.6    x 6   105.7 / 55.9
//   d 256   n 64      x 32   17.7 / 12.9                           d 256   n 2560    x 12   24.1 / 32.0    x 24   42.9 / 29.3
//           n 320     x 32   17.0 / 18.0                                   n 30016   x 4    32.5 / 57.6    x 64  133.3 / 88.3
//           n 832     x 28   18.1 / 23.5                                   n 100032  x 4    57.1 / 73.6
//           n 1024    x 64   35.8 / 24.9                                   n 300032  x 12  215.5 / 151.6
// Over 3712 sizes (1 to 200 sequences, 1 to 16 key/value heads, 17 to 2048 rows, room for 32 to 300032
// tokens, bf16 and fp16) it takes a kernel that is more than 10 % the slower one at 65; the worst is 24.8 us for
// 18.4 (d 128, 60 units of 3 sequences with 150 rows, 1536 tokens).
bool kv4_tree_many_rows(int B, int H_kv, int cols, int d, long long room, int num_sms) {
  if (!kv4_tree_wide(d, cols)) return false;
  const int unit = kv4_unit_cols(d, cols);
  const long long x = (long long)B * H_kv * ((cols + unit - 1) / unit), y = (long long)B * H_kv * ((cols + kWideRows - 1) / kWideRows);
  if (cluster_ctas(d, unit / 8, x, x * ((room + 127) / 128 * 128), num_sms) > 0) return d != 128 && room <= 256;
  const int last = cols % kWideRows;
  const bool few = d < 256 && cols > kWideRows && last > 0 && last <= 32;
  const double need = d == 64 ? 4 << 20 : d == 128 ? 16 << 20 : 12 << 20;
  return x >= (d == 128 ? 24 : 16) || (double)x * x * x * room >= need * (few ? 4 : 1) * y;
}

// (the parts of either kernel fit behind part_o and part_ml: 2 kKv4MaxCtas units of up to 32 columns are
// 2 kWideMaxCtas of kWideRows)
static_assert(kKv4MaxCtas * 32 <= kWideMaxCtas * kWideRows, "parts");
cudaError_t launch_kv4_tree(Kv4TreeArgs a, int d, bool bf16, long long tokens_bound, int num_sms, cudaStream_t stream) {
  const long long room = (long long)a.pool.max_pages << a.pool.page_shift;
  if (kv4_tree_many_rows(a.B, a.pool.H_kv, a.cols, d, room, num_sms)) return launch_kv4_wide(a, d, bf16, room, num_sms, stream);
  return launch_units(a, d, bf16, tokens_bound, num_sms, stream);
}

}  // namespace fa
