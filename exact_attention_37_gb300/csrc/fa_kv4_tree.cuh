// Trees of drafted tokens, as the kernels of attention over the 4-bit cache read them.
#pragma once
#include "fa_kv4.h"

namespace fa {

// Drafted tokens of a sequence; its cached prefix ends in front of them.
__device__ __forceinline__ int draft_count(const Kv4TreeArgs& a, int b) {
  return a.tree.count ? min(max(a.tree.count[b], 0), a.N_q) : a.N_q;
}
// Follows a drafted token's parents up to the prefix: which drafted tokens it sees (its ancestors
// and itself) and how deep it is, -1 for a row that is no token of the tree.
__device__ __forceinline__ int tree_row(const Kv4TreeArgs& a, int b, int count, int prefix, int i, uint64_t (&see)[2]) {
  const int32_t* parents = a.tree.parents + (size_t)b * a.N_q;
  see[0] = see[1] = 0;
  if (i >= count || prefix + i < 0) return -1;
  for (int p = i, depth = 0;; ++depth) {
    if (p < 64) see[0] |= 1ull << p; else see[1] |= 1ull << (p - 64);
    const int up = parents[p];
    if (up == -1) return depth;
    if (up < -1 || up >= p || prefix + up < 0) {  // no chain to the prefix
      see[0] = see[1] = 0;
      return -1;
    }
    p = up;
  }
}
// Which of 64 tokens from `first` on, counted from the prefix's end, a row sees: all of the prefix.
__device__ __forceinline__ uint64_t tree_window(const uint64_t (&see)[2], int first) {
  if (first <= -64) return ~0ull;
  if (first < 0) return (see[0] << -first) | ((1ull << -first) - 1);
  if (first == 0) return see[0];
  if (first < 64) return (see[0] >> first) | (see[1] << (64 - first));
  return first < 128 ? see[1] >> (first - 64) : 0;
}
// The drafted tokens of a unit's sequence in shared memory.
struct TreeRows {
  uint64_t see[kKv4MaxDraft][2];
  int depth[kKv4MaxDraft];
};
// Fills them, a thread a row.
__device__ __forceinline__ void tree_rows(const Kv4TreeArgs& a, int b, int count, int prefix, TreeRows& rows, int i) {
  if (i >= a.N_q) return;
  uint64_t see[2];
  rows.depth[i] = tree_row(a, b, count, prefix, i, see);
  rows.see[i][0] = see[0], rows.see[i][1] = see[1];
}
// A (scale, low) of the cache that is not finite.
template <bool BF16>
__device__ __forceinline__ bool not_finite(uint32_t par) {
  constexpr uint32_t kExp = BF16 ? 0x7F80u : 0x7C00u;
  return (par & kExp) == kExp || ((par >> 16) & kExp) == kExp;
}

}  // namespace fa
