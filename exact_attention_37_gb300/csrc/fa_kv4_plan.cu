// Page tables that grow and shrink with their requests, and accepted rows of a draft moved
// together (fa_kv4_plan, fa_kv4_keep; the header has the definitions).
//
// The plan is integer arithmetic on a few kilobytes, so it is bound by latency: one launch of
// one cluster, whose CTAs each scan all requests (a read of 12 B bytes) and then share the
// pages that move and the new tokens' slots; a barrier of the cluster stands between steps that
// read what others write.  A page's sequence is found by bisection in the scan's sums, so that
// long and short sequences weigh by their pages.  Slots and positions of many tokens (B N from
// kSplit on) are a second launch over the whole GPU.
//
// The keep moves whole rows: a CTA takes one head's keys or values of one sequence, has all of
// its rows in registers before it writes the first, and so may write where it read.
//
// Measured (one GB300, kernels alone in a graph): a plan of 256 sequences with one token 6.5 us together with
// the copy of its state, of 64 trees of 24 tokens 9, of 64 prompts of up to 8192 tokens 14 (two launches: 6.4
// MB of slots and positions); most of it is starts, barriers and chains of dependent loads (0.2 instructions a
// clock).  A keep of 64 sequences of up to 16 rows (8 heads, d 128) 2.8, of 120 of up to 61 (4 heads, d 256)
// 4.8; looking the rows' places up once for a block first did not help (3.2 and 4.7).
#include <algorithm>
#include <climits>
#include <type_traits>

#include "fa_kv4_plan.h"
#include "ptx.cuh"

namespace fa {
namespace {

constexpr int kThreads = 512;
constexpr int kCluster = 4;
constexpr long long kSplit = 1 << 14;

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\nbarrier.cluster.wait.acquire;" ::: "memory");
}

// A request as the plan sees it.
struct Request {
  long long start;
  int count, had, want;  // tokens, pages; want: kTooMany where the table has no room
};
constexpr int kTooMany = INT_MAX;
__device__ __forceinline__ Request request_of(const Kv4PlanArgs& a, int b) {
  Request r;
  r.start = max(a.start[b], 0);
  r.count = min(max(a.count[b], 0), a.N);
  r.had = min(max(a.held[b], 0), a.max_pages);
  const long long want = (r.start + r.count + (1 << a.page_shift) - 1) >> a.page_shift;
  r.want = want > a.max_pages ? kTooMany : (int)want;
  return r;
}
__device__ __forceinline__ int back_of(const Request& r) { return max(r.had - r.want, 0); }
__device__ __forceinline__ int more_of(const Request& r) { return r.want == kTooMany ? 0 : max(r.want - r.had, 0); }

// The slot of token `pos` of a sequence, -1 where it has no page.
__device__ __forceinline__ long long slot_of(const Kv4PlanArgs& a, int b, long long pos) {
  const int page = __ldcg(a.table + (size_t)b * a.max_pages + (pos >> a.page_shift));
  return page < 0 ? -1 : ((long long)page << a.page_shift) + (pos & ((1 << a.page_shift) - 1));
}

// Slots and positions of a sequence's drafted tokens, by one warp: the depth of a token is found
// by following parents twice as far each time.
struct Chain {
  int up, depth;  // an ancestor (-1: none left) and its distance; negative for ever where the chain is broken
};
__device__ __forceinline__ void fill_draft(const Kv4PlanArgs& a, int b, long long start, int count, Chain* chain) {
  const int lane = threadIdx.x & 31;
  constexpr int kPer = kKv4MaxDraft / 32;
  for (int i = lane; i < a.N; i += 32) {
    const int p = a.parents[(size_t)b * a.N + i];
    chain[i] = p < -1 || p >= i || i >= count ? Chain{-1, INT_MIN / 2} : Chain{p, p < 0 ? 0 : 1};
  }
  __syncwarp();
  for (int far = 1; far < a.N; far *= 2) {
    Chain next[kPer];
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int i = lane + 32 * k;
      if (i < a.N) {
        next[k] = chain[i];
        if (next[k].up >= 0) {
          const Chain u = chain[next[k].up];
          next[k] = Chain{u.up, max(next[k].depth + u.depth, INT_MIN / 2)};
        }
      }
    }
    __syncwarp();
#pragma unroll
    for (int k = 0; k < kPer; ++k)
      if (lane + 32 * k < a.N) chain[lane + 32 * k] = next[k];
    __syncwarp();
  }
  for (int i = lane; i < a.N; i += 32) {
    const size_t e = (size_t)b * a.N + i;
    a.slots[e] = i < count ? slot_of(a, b, start + i) : -1;
    a.positions[e] = chain[i].depth < 0 ? -1 : (int)(start + chain[i].depth);
  }
  __syncwarp();
}
// The same of B N tokens in a row, `first` and every `step`-th behind it.
__device__ __forceinline__ void fill_rows(const Kv4PlanArgs& a, long long first, long long step) {
  for (long long e = first; e < (long long)a.B * a.N; e += step) {
    const int b = (int)(e / a.N), i = (int)(e - (long long)b * a.N);
    const bool real = i < __ldcg(a.out_count + b);
    const long long pos = (long long)max(a.start[b], 0) + i;
    a.slots[e] = real ? slot_of(a, b, pos) : -1;
    a.positions[e] = real ? (int)pos : -1;
  }
}
__device__ __forceinline__ void fill(const Kv4PlanArgs& a, int cta, int ctas, Chain (*chains)[kKv4MaxDraft]) {
  if (a.parents) {
    const int warp = threadIdx.x >> 5, warps = kThreads / 32;
    for (int b = cta * warps + warp; b < a.B; b += ctas * warps)
      fill_draft(a, b, max(a.start[b], 0), __ldcg(a.out_count + b), chains[warp]);
  } else {
    fill_rows(a, (long long)cta * kThreads + threadIdx.x, (long long)ctas * kThreads);
  }
}

template <bool FILL>
__global__ void __launch_bounds__(kThreads) kv4_plan_kernel(const Kv4PlanArgs a) {
  extern __shared__ long long sums[];  // [B] pages given back, [B] pages wanted, of the sequences up to each
  __shared__ long long warp_sum[2][kThreads / 32];
  __shared__ Chain chains[FILL ? kThreads / 32 : 1][kKv4MaxDraft];
  long long* back_to = sums;
  long long* more_to = sums + a.B;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int cta = blockIdx.x, ctas = gridDim.x;
  grid_dep_launch();
  grid_dep_wait();
  // ---- sums over the sequences
  const int per = (a.B + kThreads - 1) / kThreads, b0 = min((int)threadIdx.x * per, a.B), b1 = min(b0 + per, a.B);
  long long back = 0, more = 0;
  for (int b = b0; b < b1; ++b) {
    const Request r = request_of(a, b);
    back += back_of(r), more += more_of(r);
    back_to[b] = back, more_to[b] = more;
  }
  long long x = back, y = more;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, x, off), v = __shfl_up_sync(0xffffffffu, y, off);
    if (lane >= off) x += u, y += v;
  }
  if (lane == 31) warp_sum[0][warp] = x, warp_sum[1][warp] = y;
  __syncthreads();
  x -= back, y -= more;
  for (int w = 0; w < warp; ++w) x += warp_sum[0][w], y += warp_sum[1][w];
  for (int b = b0; b < b1; ++b) back_to[b] += x, more_to[b] += y;
  __syncthreads();
  const long long backs = a.B ? back_to[a.B - 1] : 0;
  const int had_free = min(max(*a.free_count, 0), a.num_free);
  const long long n = min(had_free + backs, (long long)a.num_free);  // pages on the stack before growth
  // ---- which requests are served: those up to the first whose pages are not there
  long long mine = 0;  // pages that the served ones of this thread's sequences take up to
  int counts[8], wants[8];
  const bool write = cta == 0;
  auto served = [&](const Request& r, int b) { return r.want != kTooMany && (more_of(r) == 0 || more_to[b] <= n); };
  for (int b = b0; b < b1; ++b) {
    const Request r = request_of(a, b);
    const bool ok = served(r, b);
    if (ok && more_of(r) > 0) mine = more_to[b];
    counts[b - b0] = ok ? r.count : 0;
    wants[b - b0] = ok ? r.want : r.had;
  }
#pragma unroll
  for (int off = 16; off; off >>= 1) mine = max(mine, __shfl_xor_sync(0xffffffffu, mine, off));
  __syncthreads();  // warp_sum has been read
  if (lane == 0) warp_sum[0][warp] = mine;
  __syncthreads();
  long long taken = 0;
  for (int w = 0; w < kThreads / 32; ++w) taken = max(taken, warp_sum[0][w]);
  // (every CTA has read held and the free count here)
  cluster_sync();
  // ---- pages that are given back: the last sequence's first, each sequence's last page first
  for (long long r = (long long)cta * kThreads + threadIdx.x; r < backs; r += (long long)ctas * kThreads) {
    const long long from_front = backs - 1 - r;
    int lo = 0, hi = a.B - 1;  // the first sequence with back_to > from_front
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (back_to[mid] > from_front) hi = mid; else lo = mid + 1;
    }
    const int before = lo ? (int)(from_front - back_to[lo - 1]) : (int)from_front;
    const long long tokens = (long long)max(a.start[lo], 0) + min(max(a.count[lo], 0), a.N);
    const int place = (int)((tokens + (1 << a.page_shift) - 1) >> a.page_shift) + before;
    int32_t* at = a.table + (size_t)lo * a.max_pages + place;
    if (had_free + r < a.num_free) a.free[had_free + r] = *at;
    *at = -1;
  }
  if (backs > 0 && taken > 0) cluster_sync();
  // ---- growth: the stack's pages from the top, in the order of the sequences
  for (long long k = (long long)cta * kThreads + threadIdx.x; k < taken; k += (long long)ctas * kThreads) {
    int lo = 0, hi = a.B - 1;  // the first sequence with more_to > k
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (more_to[mid] > k) hi = mid; else lo = mid + 1;
    }
    const int had = min(max(a.held[lo], 0), a.max_pages);
    const long long place = had + k - (lo ? more_to[lo - 1] : 0);
    a.table[(size_t)lo * a.max_pages + place] = __ldcg(a.free + (n - 1 - k));
  }
  if (write)
    for (int b = b0; b < b1; ++b) {
      a.out_count[b] = counts[b - b0];
      a.lengths[b] = (int)min((long long)max(a.start[b], 0) + counts[b - b0], (long long)INT_MAX);
    }
  cluster_sync();  // held has been read; the table is as it will be
  if (write) {
    for (int b = b0; b < b1; ++b) a.held[b] = wants[b - b0];
    if (threadIdx.x == 0) *a.free_count = (int)(n - taken);
  }
  if constexpr (FILL) fill(a, cta, ctas, chains);
}

__global__ void __launch_bounds__(kThreads) kv4_fill_kernel(const Kv4PlanArgs a) {
  __shared__ Chain chains[kThreads / 32][kKv4MaxDraft];
  grid_dep_launch();
  grid_dep_wait();
  fill(a, blockIdx.x, gridDim.x, chains);
}

// ---------------------------------------------------------------- accepted rows
constexpr int kKeepUnits = 5;  // pieces of rows a thread has in registers

template <int D>
struct KeepRow {
  // A row's codes and parameters in equal pieces: 8 bytes at d = 64, 16 above.
  using Piece = std::conditional_t<D == 64, uint2, uint4>;
  static constexpr int kCodes = D / 2 / sizeof(Piece), kParams = D / 8 / sizeof(Piece), kPieces = kCodes + kParams;
};

template <int D>
__global__ void kv4_keep_kernel(const Kv4Pool c, const int32_t* start, const int32_t* path, const int32_t* kept, int N) {
  using R = KeepRow<D>;
  using Piece = typename R::Piece;
  grid_dep_launch();
  grid_dep_wait();
  const int which = blockIdx.x & 1, h = (blockIdx.x >> 1) % c.H_kv, b = (blockIdx.x >> 1) / c.H_kv;
  const int rows = min(max(kept[b], 0), N);
  const long long first = start[b];
  const int32_t* table = c.table + (size_t)b * c.max_pages;
  Piece* codes = reinterpret_cast<Piece*>(c.codes[which]);
  Piece* params = reinterpret_cast<Piece*>(c.params[which]);
  auto row_of = [&](long long pos) { return kv4_row(table, c.max_pages, c.page_shift, c.num_pages, pos); };
  auto piece = [&](long long row, int e) -> Piece* {
    const long long hr = kv4_head_row(row, c.page_shift, c.H_kv, h);
    return e < R::kCodes ? codes + hr * R::kCodes + e : params + hr * R::kParams + (e - R::kCodes);
  };
  Piece held[kKeepUnits];
  Piece* to[kKeepUnits];
#pragma unroll
  for (int u = 0; u < kKeepUnits; ++u) {
    const int i = threadIdx.x + u * blockDim.x, j = i / R::kPieces, e = i % R::kPieces;
    to[u] = nullptr;
    if (j >= rows) continue;
    const int p = path[(size_t)b * N + j];
    const long long src = p < 0 || p >= N ? -1 : row_of(first + p), dst = row_of(first + j);
    if (src < 0 || dst < 0) {
      if (e == 0) record_check(c.err, kDbgPage, (uint32_t)(src < 0 ? first + p : first + j));
      continue;
    }
    held[u] = *piece(src, e);
    if (p != j) to[u] = piece(dst, e);
  }
  __syncthreads();  // every row is in registers
#pragma unroll
  for (int u = 0; u < kKeepUnits; ++u)
    if (to[u]) *to[u] = held[u];
}

template <int D>
cudaError_t keep_t(const Kv4Pool& c, const int32_t* start, const int32_t* path, const int32_t* kept, int B, int N, cudaStream_t s) {
  const int pieces = N * KeepRow<D>::kPieces, threads = ((pieces + kKeepUnits - 1) / kKeepUnits + 31) / 32 * 32;
  return launch_dependent(kv4_keep_kernel<D>, (unsigned)(2ll * B * c.H_kv), (unsigned)threads, 0, s, c, start, path, kept, N);
}

}  // namespace

cudaError_t launch_kv4_plan(const Kv4PlanArgs& a, int num_sms, cudaStream_t stream) {
  static_assert(kKv4MaxBatch <= 8 * kThreads, "a thread's sequences");
  const bool split = (long long)a.B * a.N >= kSplit;
  auto kern = split ? kv4_plan_kernel<false> : kv4_plan_kernel<true>;
  cudaError_t e = cudaSuccess;
  // (past 48 KB with the static part the limit is raised, to one value for every batch; the call is a
  // microsecond of the host's time)
  if (a.B > 1024) e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 16 * kKv4MaxBatch);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(kCluster);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = 16 * (size_t)a.B;
  cfg.stream = stream;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = kCluster;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, kern, a);
  if (e != cudaSuccess || !split) return e;
  const long long blocks = a.parents ? (a.B + kThreads / 32 - 1) / (kThreads / 32) : ((long long)a.B * a.N + 4 * kThreads - 1) / (4 * kThreads);
  return launch_dependent(kv4_fill_kernel, (unsigned)std::min<long long>(blocks, 4LL * num_sms), kThreads, 0, stream, a);
}

cudaError_t launch_kv4_keep(const Kv4Pool& c, int d, const int32_t* start, const int32_t* path, const int32_t* kept,
                            int B, int N, cudaStream_t s) {
  switch (d) {
    case 64:
      return keep_t<64>(c, start, path, kept, B, N, s);
    case 128:
      return keep_t<128>(c, start, path, kept, B, N, s);
    case 256:
      return keep_t<256>(c, start, path, kept, B, N, s);
    default:
      return cudaErrorInvalidValue;
  }
}

}  // namespace fa
