// The paged 4-bit key/value cache: its layout, shared by the kernels and the host.
//
// A pool has num_pages pages of page_size token rows for each key/value head:
//   codes  [num_pages, H_kv, page_size, d / 2] bytes; byte i of a row holds channel 2 i in
//          its low half and channel 2 i + 1 in its high half
//   params [num_pages, H_kv, page_size, d / 32, 2] 16-bit: (scale, low) of each group of 32
//          channels
// and channel c of a row stands for T(low + scale * code), one rounding to the cache's type.
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

#include "fa_internal.h"

namespace fa {

constexpr int kKv4Group = 32;  // channels that share a scale and a low value

// The page at place `at` of a sequence's part of the page table, or -1 where it is none of
// the pool's.
__host__ __device__ inline int kv4_page(const int32_t* table_row, int num_pages, long long at) {
  const int page = table_row[at];
  return page < 0 || page >= num_pages ? -1 : page;
}

// Row of token `pos` of a sequence inside a pool seen as [num_pages, page_size] rows, or -1
// where the page table does not lead to one (a negative position, one past the table, a
// page outside the pool).
__host__ __device__ inline long long kv4_row(const int32_t* table_row, int max_pages, int page_shift, int num_pages,
                                             long long pos) {
  if (pos < 0) return -1;
  const long long p = pos >> page_shift;
  if (p >= max_pages) return -1;
  const int page = kv4_page(table_row, num_pages, p);
  if (page < 0) return -1;
  return ((long long)page << page_shift) + (pos & ((1ll << page_shift) - 1));
}

// Offset, in rows, of a head's row: pages are [H_kv, page_size] rows.
__host__ __device__ inline long long kv4_head_row(long long row, int page_shift, int H_kv, int h) {
  const long long page = row >> page_shift;
  return ((page * H_kv + h) << page_shift) + (row & ((1ll << page_shift) - 1));
}

struct Kv4Pool {
  uint8_t* codes[2];   // keys, values
  uint32_t* params[2]; // (scale, low) pairs
  const int32_t* table;
  int num_pages, page_shift, max_pages, H_kv;
  uint32_t* err;
};

cudaError_t launch_kv4_append(const Kv4Pool& c, int d, bool bf16, const void* k, const void* v, const int32_t* start,
                              const int32_t* count, int B, int N, int num_sms, cudaStream_t stream);
cudaError_t launch_kv4_read(const Kv4Pool& c, int d, bool bf16, const int32_t* start, const int32_t* lengths, void* k,
                            void* v, int B, int N, int num_sms, cudaStream_t stream);

struct Kv4AttendArgs {
  Kv4Pool pool;
  const void* q;
  const int32_t* lengths;
  void* o;
  float* lse;
  float* part_o;         // [2, CTAs, columns of a unit, d]: of the units that a CTA's stretch cuts
  float* part_ml;        // [2, CTAs, columns of a unit, 2]
  int B, H, N_q, group;
  int cols, col_tiles;   // group * N_q columns in tiles of 8 NT
  int ctas, early;       // early: neighbours in the stream may overlap
  int causal, cap;
  float scale_log2;
  RuleArgs rule;         // cap and slopes
};
// A tree of drafted tokens: the last tokens of each sequence, one query row each.
struct Kv4Tree {
  const int32_t* parents;  // [B, N_q]
  const int32_t* count;    // [B], or null: N_q each
};
struct Kv4TreeArgs : Kv4AttendArgs {
  Kv4Tree tree;
};
constexpr int kKv4MaxDraft = 128;  // drafted tokens of a sequence
constexpr int kWideRows = 128;     // rows of a tile of the kernel for many of them
constexpr int kWideMaxCtas = 160;  // one an SM
constexpr int kKv4MaxBatch = 4096;
constexpr int kKv4MaxCtas = 640;  // 4 an SM of 160
constexpr int kKv4MaxCluster = 8;
// Columns (query heads times query rows) of one unit of work.
int kv4_unit_cols(int d, int cols);
// tokens_bound: tokens of all units, at most.
cudaError_t launch_kv4_attend(Kv4AttendArgs a, int d, bool bf16, long long tokens_bound, int num_sms, cudaStream_t stream);
// The same for trees of drafted tokens.  With more rows than one unit's columns (kv4_tree_wide)
// the kernel for many rows may take them, and the parts have room for its kWideMaxCtas CTAs:
// part_o [2, kWideMaxCtas, d, kWideRows], part_ml [2, kWideMaxCtas, kWideRows, 2].
bool kv4_tree_wide(int d, int cols);
bool kv4_tree_many_rows(int B, int H_kv, int cols, int d, long long room, int num_sms);
cudaError_t launch_kv4_wide(const Kv4TreeArgs& a, int d, bool bf16, long long room, int num_sms, cudaStream_t stream);
cudaError_t launch_kv4_tree(Kv4TreeArgs a, int d, bool bf16, long long tokens_bound, int num_sms, cudaStream_t stream);

}  // namespace fa
