// Page tables made on the GPU, and rows moved inside the cache.
#pragma once
#include "fa_kv4.h"

namespace fa {

struct Kv4PlanArgs {
  int32_t* table;          // [B, max_pages]
  int32_t* held;           // [B]
  int32_t* free;           // [num_free]: a stack
  int32_t* free_count;
  const int32_t* start;
  const int32_t* count;
  const int32_t* parents;  // [B, N] or null
  int32_t* out_count;      // [B]
  int32_t* lengths;        // [B]
  int64_t* slots;          // [B, N]
  int32_t* positions;      // [B, N]
  int B, N, max_pages, num_free, page_shift;
};
cudaError_t launch_kv4_plan(const Kv4PlanArgs& a, int num_sms, cudaStream_t stream);

cudaError_t launch_kv4_keep(const Kv4Pool& c, int d, const int32_t* start, const int32_t* path, const int32_t* kept,
                            int B, int N, cudaStream_t stream);

}  // namespace fa
