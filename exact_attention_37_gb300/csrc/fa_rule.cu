// Host side of the score rules, the document plan and the backward pre-pass with a rule.
//
// Document ids are any integers in any order, so which 128 x 128 blocks hold a visible
// pair is found on the device.  One pass over the ids writes them padded to whole blocks
// (-1 for every negative id and past the end) with a summary of each block.  A second one
// writes, for every block of rows, the list of the blocks it meets (those whose id ranges
// overlap and that the causal mask or the prefix reaches), and for every row the range of
// the other side that has its id, by bisection, when those ids are in order.  A list may
// name a block whose pairs are all hidden: the kernels hide by range, or id by id in
// blocks of unordered ids, so a list only has to name enough.  Both passes together take
// 5 us at B2 N8192 (with the launches; the lists' blocks are read by every head, so they
// are made once a call).  At B2 H16 N8192 d128 a causal mask takes 430 us as a mask, 447 as
// one document's ids, and documents of 900 rows on average 155.
#include <algorithm>
#include <climits>
#include <type_traits>

#include "fa_internal.h"
#include "fa_rule.cuh"
#include "ptx.cuh"

namespace fa {
namespace {

constexpr int kBlkRows = 128;
constexpr int kPlanWarps = 4;

size_t up(size_t x) { return (x + 255) / 256 * 256; }

// A block's ids: smallest and largest id >= 0, whether it has padding, the first and last
// row that is none, how many are none, and whether an id is followed by a smaller one
// (the row behind the block included).
struct BlockIds {
  int lo, hi, neg, first, last, count, falls, unused;
};

__global__ void __launch_bounds__(32 * kPlanWarps)
    rule_ids_kernel(const int* q_doc, const int* k_doc, int* q_ids, int* k_ids, BlockIds* q_sum, BlockIds* k_sum, int B,
                    int N, int Nk, int nqb, int nkb) {
  grid_dep_launch();
  grid_dep_wait();
  const int per = nqb + nkb;
  const long long w = (long long)blockIdx.x * kPlanWarps + (threadIdx.x >> 5);
  if (w >= (long long)B * per) return;
  const int lane = threadIdx.x & 31;
  const int b = (int)(w / per), x = (int)(w % per);
  const bool is_q = x < nqb;
  const int blk = is_q ? x : x - nqb, n = is_q ? N : Nk, nb = is_q ? nqb : nkb;
  const int* src = (is_q ? q_doc : k_doc) + (size_t)b * n;
  int* dst = (is_q ? q_ids : k_ids) + ((size_t)b * nb + blk) * kBlkRows;
  int lo = INT_MAX, hi = -1, first = INT_MAX, last = -1, count = 0;
  bool neg = false, falls = false;
#pragma unroll
  for (int i = lane; i < kBlkRows; i += 32) {
    const int row = blk * kBlkRows + i;
    int id = -1;
    if (row < n) {
      id = max(src[row], -1);
      neg |= id < 0;
      if (id >= 0 && row + 1 < n) {
        const int next = src[row + 1];
        falls |= next >= 0 && next < id;
      }
    } else {
      neg |= !is_q;  // keys past the end must be hidden; rows past the end are never written
    }
    dst[i] = id;
    if (id >= 0) lo = min(lo, id), hi = max(hi, id), first = min(first, row), last = max(last, row), ++count;
  }
  constexpr unsigned kAll = 0xffffffffu;
  lo = __reduce_min_sync(kAll, lo);
  hi = __reduce_max_sync(kAll, hi);
  first = __reduce_min_sync(kAll, first);
  last = __reduce_max_sync(kAll, last);
  count = __reduce_add_sync(kAll, count);
  const bool any_neg = __any_sync(kAll, neg), any_falls = __any_sync(kAll, falls);
  if (lane == 0)
    (is_q ? q_sum : k_sum)[(size_t)b * nb + blk] = BlockIds{lo, hi, any_neg ? 1 : 0, first, last, count, any_falls ? 1 : 0, 0};
}

// The rows [first, last] of a side that are no padding, when its ids do not decrease and
// no padding lies between them; first > last when it has no such row.
struct Ordered {
  bool yes;
  int first, last;
};
__device__ Ordered ordered_ids(const BlockIds* sum, int nb) {
  constexpr unsigned kAll = 0xffffffffu;
  int first = INT_MAX, last = -1, count = 0;
  bool falls = false;
  for (int i = threadIdx.x & 31; i < nb; i += 32) {
    const BlockIds s = sum[i];
    first = min(first, s.first), last = max(last, s.last), count += s.count, falls |= s.falls != 0;
  }
  first = __reduce_min_sync(kAll, first);
  last = __reduce_max_sync(kAll, last);
  count = __reduce_add_sync(kAll, count);
  Ordered o;
  o.yes = !__any_sync(kAll, falls) && (count == 0 || count == last - first + 1);
  o.first = first;
  o.last = last;
  return o;
}
// First row of ids [first, last + 1) whose id is >= v.
__device__ __forceinline__ int lower_bound(const int* ids, int first, int last, int v) {
  int lo = first, hi = last + 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (ids[mid] < v) lo = mid + 1; else hi = mid;
  }
  return lo;
}

struct PlanArgs {
  const int *q_ids, *k_ids, *prefix;
  const BlockIds *q_sum, *k_sum;
  int *q_lo, *q_hi, *k_lo, *k_hi;
  int *q_list, *q_count, *k_list, *k_count;
  int B, N, Nk, nqb, nkb, nql, q_blocks, nkl, q_list_stride, k_list_stride, causal, k_ranges;
};

// One warp a list (the key blocks of a group of query rows, or the query blocks of a key
// block), and one warp for the ranges of 32 rows.
__global__ void __launch_bounds__(32 * kPlanWarps) rule_list_kernel(const PlanArgs p) {
  grid_dep_launch();
  grid_dep_wait();
  const int q_warps = p.nqb * (kBlkRows / 32), k_warps = p.k_ranges ? p.nkb * (kBlkRows / 32) : 0;
  const int per = p.nql + p.nkl + q_warps + k_warps;
  const long long w = (long long)blockIdx.x * kPlanWarps + (threadIdx.x >> 5);
  if (w >= (long long)p.B * per) return;
  const int lane = threadIdx.x & 31;
  const int b = (int)(w / per);
  int x = (int)(w % per);
  const BlockIds* q_sum = p.q_sum + (size_t)b * p.nqb;
  const BlockIds* k_sum = p.k_sum + (size_t)b * p.nkb;
  if (x >= p.nql + p.nkl) {  // ranges
    x -= p.nql + p.nkl;
    const bool is_q = x < q_warps;
    const int row = (is_q ? x : x - q_warps) * 32 + lane;
    const Ordered o = is_q ? ordered_ids(k_sum, p.nkb) : ordered_ids(q_sum, p.nqb);
    const size_t q_at = (size_t)b * p.nqb * kBlkRows, k_at = (size_t)b * p.nkb * kBlkRows;
    const int id = is_q ? p.q_ids[q_at + row] : p.k_ids[k_at + row];
    const int* other = is_q ? p.k_ids + k_at : p.q_ids + q_at;
    int lo = 0, hi = INT_MAX;
    if (id < 0 || (o.yes && o.first > o.last)) {
      hi = 0;
    } else if (o.yes) {
      lo = lower_bound(other, o.first, o.last, id);
      hi = id == INT_MAX ? o.last + 1 : lower_bound(other, lo, o.last, id + 1);
    }
    (is_q ? p.q_lo + q_at : p.k_lo + k_at)[row] = lo;
    (is_q ? p.q_hi + q_at : p.k_hi + k_at)[row] = hi;
    return;
  }
  const bool is_q = x < p.nql;
  const int own = is_q ? x : x - p.nql;
  const int koff = p.Nk - p.N;
  const int pre = p.prefix ? max(0, min(p.prefix[b], p.Nk)) : 0;
  const bool one_by_one = is_q ? !ordered_ids(k_sum, p.nkb).yes : !ordered_ids(q_sum, p.nqb).yes;
  int my_lo = INT_MAX, my_hi = -1;
  const int rows = (is_q ? p.q_blocks : 1) * kBlkRows;
  if (is_q) {
    for (int i = own * p.q_blocks; i < min(p.nqb, (own + 1) * p.q_blocks); ++i)
      my_lo = min(my_lo, q_sum[i].lo), my_hi = max(my_hi, q_sum[i].hi);
  } else {
    my_lo = k_sum[own].lo, my_hi = k_sum[own].hi;
  }
  const int other_n = is_q ? p.nkb : p.nqb;
  int* out = is_q ? p.q_list + ((size_t)b * p.nql + own) * p.q_list_stride
                  : p.k_list + ((size_t)b * p.nkl + own) * p.k_list_stride;
  int count = 0;
  for (int base = 0; base < other_n; base += 32) {
    const int o = base + lane;
    int entry = -1;
    if (o < other_n) {
      const BlockIds& s = is_q ? k_sum[o] : q_sum[o];
      const int q_last = min((is_q ? own * rows + rows : o * kBlkRows + kBlkRows), p.N) - 1;
      const int k_first = (is_q ? o : own) * kBlkRows;
      const bool reach = !p.causal || k_first <= q_last + koff || k_first < pre;
      if (reach && max(my_lo, s.lo) <= min(my_hi, s.hi))
        entry = (o << kListShift) | (one_by_one ? kListIds : 0) | (s.neg ? kListClean : 0);
    }
    const unsigned m = __ballot_sync(0xffffffffu, entry >= 0);
    if (entry >= 0) out[count + __popc(m & ((1u << lane) - 1u))] = entry;
    count += __popc(m);
  }
  if (lane == 0) (is_q ? p.q_count + (size_t)b * p.nql : p.k_count + (size_t)b * p.nkl)[own] = count;
}

// The backward pre-pass with a rule: D and L log2 e padded per head as in the plain
// pre-pass, and rows that see nothing (L = -inf) or are padding get L = +inf, D = 0, so
// that every P of theirs is 0 and nothing of their O and dO is used.
struct Words8 {
  uint32_t w[8];
};
// 32 bytes that no other thread reads: one load where the address allows it.
template <bool WIDE>
__device__ __forceinline__ Words8 load32(const uint16_t* p) {
  Words8 r;
  if constexpr (WIDE) {
    asm volatile("ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3]), "=r"(r.w[4]), "=r"(r.w[5]), "=r"(r.w[6]),
                   "=r"(r.w[7])
                 : "l"(p));
  } else {
    const uint4 a = reinterpret_cast<const uint4*>(p)[0], b = reinterpret_cast<const uint4*>(p)[1];
    r = Words8{{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
  }
  return r;
}

// Bound by reading O and dO.  Two steps of 32-byte loads in flight and 8 blocks an SM
// measured best (B2 H16 N8192 d128, the pre-pass among launches that do nothing else: 8 us
// less than 16-byte loads, 16 blocks an SM; four steps in flight 10 us more).
template <int D, bool BF16, bool WIDE>
__global__ void __launch_bounds__(256) rule_pre_kernel(const BwdArgs args, const int* q_doc, long long slots) {
  grid_dep_launch();
  grid_dep_wait();
  constexpr int kLpr = D / 16;     // lanes per row, 32 bytes of O and of dO each
  constexpr int kRpw = 32 / kLpr;  // rows per warp step
  constexpr int kSteps = 2;        // warp steps in flight
  const int lane = threadIdx.x & 31;
  const int sub = lane / kLpr, part = lane % kLpr;
  const uint32_t warp0 = (blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const uint32_t nwarps = (gridDim.x * blockDim.x) >> 5;
  const uint16_t* o = reinterpret_cast<const uint16_t*>(args.o);
  const uint16_t* g = reinterpret_cast<const uint16_t*>(args.dout);
  const long long steps = (slots + kRpw - 1) / kRpw;
  for (long long st0 = warp0; st0 < steps; st0 += (long long)kSteps * nwarps) {
    Words8 ov[kSteps], gv[kSteps];
    long long slot[kSteps];
    float l[kSteps];
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
      const long long st = st0 + (long long)k * nwarps;
      slot[k] = st * kRpw + sub;
      const uint32_t head = (uint32_t)(slot[k] / args.Npad);
      const int i = (int)(slot[k] - (long long)head * args.Npad);
      l[k] = -INFINITY;
#pragma unroll
      for (int w = 0; w < 8; ++w) ov[k].w[w] = gv[k].w[w] = 0u;
      if (st < steps && slot[k] < slots && i < args.N) {
        const size_t row = (size_t)head * args.N + i;
        l[k] = args.lse[row];
        if (q_doc && q_doc[(size_t)(head / args.H) * args.N + i] < 0) l[k] = -INFINITY;
        ov[k] = load32<WIDE>(o + row * D + part * 16);
        gv[k] = load32<WIDE>(g + row * D + part * 16);
      }
    }
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
      // two sums of 8 columns, added last: the order of the plain pre-pass, so that the same
      // O and dO give the same D
      float half[2] = {0.f, 0.f};
#pragma unroll
      for (int w = 0; w < 8; ++w) {
        float& acc = half[w >> 2];
        acc = fmaf(widen16<BF16>((uint16_t)(ov[k].w[w] & 0xFFFFu)), widen16<BF16>((uint16_t)(gv[k].w[w] & 0xFFFFu)), acc);
        acc = fmaf(widen16<BF16>((uint16_t)(ov[k].w[w] >> 16)), widen16<BF16>((uint16_t)(gv[k].w[w] >> 16)), acc);
      }
#pragma unroll
      for (int off = kLpr / 2; off > 0; off >>= 1) {
        half[0] += __shfl_xor_sync(0xffffffffu, half[0], off);
        half[1] += __shfl_xor_sync(0xffffffffu, half[1], off);
      }
      const float acc = half[0] + half[1];
      if (st0 + (long long)k * nwarps < steps && slot[k] < slots && part == 0) {
        const bool none = l[k] == -INFINITY;
        args.lse_log2[slot[k]] = none ? INFINITY : l[k] * kLog2eF;
        args.delta[slot[k]] = none ? 0.f : acc;
      }
    }
  }
}

template <int D, bool BF16>
cudaError_t launch_pre(const BwdArgs& a, const int* q_doc, cudaStream_t stream) {
  int dev = 0, sms = 0;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  const long long slots = (long long)a.BH * a.Npad;
  const long long want = (slots * D / 512 + 7) / 8;  // warp steps / warps per block
  const int grid = (int)std::max<long long>(1, std::min<long long>(want, (long long)std::max(sms, 1) * 8));
  const bool wide = ((reinterpret_cast<uintptr_t>(a.o) | reinterpret_cast<uintptr_t>(a.dout)) & 31u) == 0;
  auto kern = wide ? rule_pre_kernel<D, BF16, true> : rule_pre_kernel<D, BF16, false>;
  return launch_dependent(kern, grid, 256, 0, stream, a, q_doc, slots);
}

}  // namespace

int rule_kind(const RuleArgs& r) {
  return (r.slopes ? kRuleBias : 0) | (r.cap2 > 0.f ? kRuleCap : 0) | (r.list ? kRuleDocs : 0);
}

RulePlan rule_plan(int B, int N, int Nk, int q_rows, bool kv_lists) {
  RulePlan p{};
  const size_t nqb = ((size_t)N + kBlkRows - 1) / kBlkRows, nkb = ((size_t)Nk + kBlkRows - 1) / kBlkRows;
  p.q_stride = (int)(nqb * kBlkRows);
  p.k_stride = (int)(nkb * kBlkRows);
  p.nql = (int)(((size_t)N + q_rows - 1) / q_rows);
  p.nkl = kv_lists ? (int)nkb : 0;
  p.q_list_stride = (int)nkb;
  p.k_list_stride = (int)nqb;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t o = at;
    at += up(bytes);
    return o;
  };
  p.q_ids = take((size_t)B * p.q_stride * 4);
  p.k_ids = take((size_t)B * p.k_stride * 4);
  p.q_lo = take((size_t)B * p.q_stride * 4);
  p.q_hi = take((size_t)B * p.q_stride * 4);
  p.k_lo = take(kv_lists ? (size_t)B * p.k_stride * 4 : 0);
  p.k_hi = take(kv_lists ? (size_t)B * p.k_stride * 4 : 0);
  p.q_sum = take((size_t)B * nqb * sizeof(BlockIds));
  p.k_sum = take((size_t)B * nkb * sizeof(BlockIds));
  p.q_count = take((size_t)B * p.nql * 4);
  p.k_count = take((size_t)B * p.nkl * 4);
  p.q_list = take((size_t)B * p.nql * p.q_list_stride * 4);
  p.k_list = take((size_t)B * p.nkl * p.k_list_stride * 4);
  p.bytes = at;
  return p;
}

cudaError_t launch_rule_plan(const RulePlan& p, char* ws, const int* q_doc, const int* k_doc, const int* prefix, int B,
                             int N, int Nk, int q_rows, int causal, cudaStream_t stream) {
  const int nqb = p.q_stride / kBlkRows, nkb = p.k_stride / kBlkRows;
  auto* q_sum = reinterpret_cast<BlockIds*>(ws + p.q_sum);
  auto* k_sum = reinterpret_cast<BlockIds*>(ws + p.k_sum);
  auto ints = [&](size_t o) { return reinterpret_cast<int*>(ws + o); };
  const long long w1 = (long long)B * (nqb + nkb);
  cudaError_t e = launch_dependent(rule_ids_kernel, (unsigned)((w1 + kPlanWarps - 1) / kPlanWarps), 32 * kPlanWarps, 0, stream,
                                   q_doc, k_doc, ints(p.q_ids), ints(p.k_ids), q_sum, k_sum, B, N, Nk, nqb, nkb);
  if (e != cudaSuccess) return e;
  PlanArgs a{};
  a.q_ids = ints(p.q_ids), a.k_ids = ints(p.k_ids), a.prefix = prefix;
  a.q_sum = q_sum, a.k_sum = k_sum;
  a.q_lo = ints(p.q_lo), a.q_hi = ints(p.q_hi), a.k_lo = ints(p.k_lo), a.k_hi = ints(p.k_hi);
  a.q_list = ints(p.q_list), a.q_count = ints(p.q_count), a.k_list = ints(p.k_list), a.k_count = ints(p.k_count);
  a.B = B, a.N = N, a.Nk = Nk, a.nqb = nqb, a.nkb = nkb, a.nql = p.nql, a.q_blocks = q_rows / kBlkRows, a.nkl = p.nkl;
  a.q_list_stride = p.q_list_stride, a.k_list_stride = p.k_list_stride, a.causal = causal, a.k_ranges = p.nkl > 0;
  const long long w2 = (long long)B * (p.nql + p.nkl + (nqb + (a.k_ranges ? nkb : 0)) * (kBlkRows / 32));
  return launch_dependent(rule_list_kernel, (unsigned)((w2 + kPlanWarps - 1) / kPlanWarps), 32 * kPlanWarps, 0, stream, a);
}

void rule_plan_args(RuleArgs& r, const RulePlan& p, char* ws) {
  auto ints = [&](size_t o) { return reinterpret_cast<int*>(ws + o); };
  r.q_ids = ints(p.q_ids);
  r.k_ids = ints(p.k_ids);
  r.q_lo = ints(p.q_lo);
  r.q_hi = ints(p.q_hi);
  r.k_lo = ints(p.k_lo);
  r.k_hi = ints(p.k_hi);
  r.list = ints(p.q_list);
  r.count = ints(p.q_count);
  r.q_stride = p.q_stride;
  r.k_stride = p.k_stride;
  r.list_stride = p.q_list_stride;
}

// Calls f(std::integral_constant<int, kind>).
template <class F>
static cudaError_t by_kind(int kind, F f) {
  switch (kind) {
    case 0: return f(std::integral_constant<int, 0>());
    case 1: return f(std::integral_constant<int, 1>());
    case 2: return f(std::integral_constant<int, 2>());
    case 3: return f(std::integral_constant<int, 3>());
    case 4: return f(std::integral_constant<int, 4>());
    case 5: return f(std::integral_constant<int, 5>());
    case 6: return f(std::integral_constant<int, 6>());
    case 7: return f(std::integral_constant<int, 7>());
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t launch_fwd_rule(int kind, int d, bool bf16, int rows, const CUtensorMap& q, const CUtensorMap& k,
                            const CUtensorMap& v, const CUtensorMap& o, const FwdRuleArgs& a, cudaStream_t stream) {
  return by_kind(kind, [&](auto n) { return launch_fwd_rule_kind<decltype(n)::value>(d, bf16, rows, q, k, v, o, a, stream); });
}

cudaError_t launch_bwd_rule(int kind, int d, bool bf16, const CUtensorMap& q, const CUtensorMap& k,
                            const CUtensorMap& v, const CUtensorMap& dout, const BwdRuleArgs& a, const int* q_doc,
                            cudaStream_t stream) {
  cudaError_t e;
  switch (d) {
    case 64: e = bf16 ? launch_pre<64, true>(a, q_doc, stream) : launch_pre<64, false>(a, q_doc, stream); break;
    case 128: e = bf16 ? launch_pre<128, true>(a, q_doc, stream) : launch_pre<128, false>(a, q_doc, stream); break;
    case 256: e = bf16 ? launch_pre<256, true>(a, q_doc, stream) : launch_pre<256, false>(a, q_doc, stream); break;
    default: return cudaErrorInvalidValue;
  }
  if (e != cudaSuccess) return e;
  return by_kind(kind, [&](auto n) {
    constexpr int kKind = decltype(n)::value;
    return d == 256 ? launch_bwd_256_rule_kind<kKind>(bf16, q, k, v, dout, a, stream)
                    : launch_bwd_sq_rule_kind<kKind>(d, bf16, q, k, v, dout, a, stream);
  });
}

}  // namespace fa
