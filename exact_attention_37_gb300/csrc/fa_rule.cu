// Host side of the score rules, the document plan and the backward pre-pass with a rule.
//
// Document ids are any integers in any order, so which 128 x 128 blocks hold a visible
// pair is found on the device: one pass over the ids writes them padded to whole blocks
// (-1 for every negative id and past the end) with each block's smallest and largest id,
// and a second one writes, for every block of rows, the list of the blocks it meets:
// those whose id ranges overlap and that the causal mask or the prefix reaches.  A list
// may name a block whose pairs are all hidden (ranges overlap, ids differ): the kernels
// hide pair by pair in every block that is not marked as seen in full, so a list only
// has to name enough.
#include <algorithm>
#include <climits>

#include "fa_internal.h"
#include "fa_rule.cuh"
#include "ptx.cuh"

namespace fa {
namespace {

constexpr int kBlkRows = 128;
constexpr int kPlanWarps = 4;

size_t up(size_t x) { return (x + 255) / 256 * 256; }

// Smallest and largest id >= 0 of a block, and whether it has padding.
struct BlockIds {
  int lo, hi, neg, unused;
};

__global__ void __launch_bounds__(32 * kPlanWarps)
    rule_ids_kernel(const int* q_doc, const int* k_doc, int* q_ids, int* k_ids, BlockIds* q_sum, BlockIds* k_sum, int B,
                    int N, int Nk, int nqb, int nkb) {
  const int per = nqb + nkb;
  const long long w = (long long)blockIdx.x * kPlanWarps + (threadIdx.x >> 5);
  if (w >= (long long)B * per) return;
  const int lane = threadIdx.x & 31;
  const int b = (int)(w / per), x = (int)(w % per);
  const bool is_q = x < nqb;
  const int blk = is_q ? x : x - nqb, n = is_q ? N : Nk, nb = is_q ? nqb : nkb;
  const int* src = (is_q ? q_doc : k_doc) + (size_t)b * n;
  int* dst = (is_q ? q_ids : k_ids) + ((size_t)b * nb + blk) * kBlkRows;
  int lo = INT_MAX, hi = -1;
  bool neg = false;
#pragma unroll
  for (int i = lane; i < kBlkRows; i += 32) {
    const int row = blk * kBlkRows + i;
    int id = -1;
    if (row < n) {
      id = max(src[row], -1);
      neg |= id < 0;
    } else {
      neg |= !is_q;  // keys past the end must be hidden; rows past the end are never written
    }
    dst[i] = id;
    if (id >= 0) lo = min(lo, id), hi = max(hi, id);
  }
  lo = __reduce_min_sync(0xffffffffu, lo);
  hi = __reduce_max_sync(0xffffffffu, hi);
  const bool any = __any_sync(0xffffffffu, neg);
  if (lane == 0) (is_q ? q_sum : k_sum)[(size_t)b * nb + blk] = BlockIds{lo, hi, any ? 1 : 0, 0};
}

// One warp a list: the key blocks of a group of query rows, or (kv lists) the query
// blocks of a key block.
__global__ void __launch_bounds__(32 * kPlanWarps)
    rule_list_kernel(const BlockIds* q_sum, const BlockIds* k_sum, int* q_list, int* q_count, int* k_list, int* k_count,
                     const int* prefix, int B, int N, int Nk, int nqb, int nkb, int nql, int q_blocks, int nkl,
                     int q_list_stride, int k_list_stride, int causal) {
  const int per = nql + nkl;
  const long long w = (long long)blockIdx.x * kPlanWarps + (threadIdx.x >> 5);
  if (w >= (long long)B * per) return;
  const int lane = threadIdx.x & 31;
  const int b = (int)(w / per), x = (int)(w % per);
  const bool is_q = x < nql;
  const int own = is_q ? x : x - nql;
  const int koff = Nk - N;
  const int pre = prefix ? max(0, min(prefix[b], Nk)) : 0;
  auto load_q = [&](int g, int blocks) {  // summary of `blocks` query blocks from g * blocks on
    BlockIds s{INT_MAX, -1, 0, 0};
    for (int i = g * blocks; i < min(nqb, (g + 1) * blocks); ++i) {
      const BlockIds t = q_sum[(size_t)b * nqb + i];
      s.lo = min(s.lo, t.lo), s.hi = max(s.hi, t.hi), s.neg |= t.neg;
    }
    return s;
  };
  const BlockIds mine = is_q ? load_q(own, q_blocks) : k_sum[(size_t)b * nkb + own];
  const int other_n = is_q ? nkb : nqb;
  int* out = is_q ? q_list + ((size_t)b * nql + own) * q_list_stride : k_list + ((size_t)b * nkl + own) * k_list_stride;
  int count = 0;
  for (int base = 0; base < other_n; base += 32) {
    const int o = base + lane;
    int entry = -1;
    if (o < other_n) {
      const BlockIds oth = is_q ? k_sum[(size_t)b * nkb + o] : load_q(o, 1);
      const BlockIds &qs = is_q ? mine : oth, &ks = is_q ? oth : mine;
      const int rows = is_q ? q_blocks * kBlkRows : kBlkRows;
      const int q_first = (is_q ? own : o) * rows, q_last = min(q_first + rows, N) - 1;
      const int k_first = (is_q ? o : own) * kBlkRows, k_last = k_first + kBlkRows - 1;
      const bool reach = !causal || k_first <= q_last + koff || k_first < pre;
      if (reach && max(qs.lo, ks.lo) <= min(qs.hi, ks.hi)) {
        const bool all = qs.lo == qs.hi && ks.lo == ks.hi && qs.lo == ks.lo && !qs.neg && !ks.neg;
        const bool open = !causal || k_last <= q_first + koff || k_last < pre;
        entry = (o << kListShift) | (all && open ? 0 : kListPartial) | (oth.neg ? kListClean : 0);
      }
    }
    const unsigned m = __ballot_sync(0xffffffffu, entry >= 0);
    if (entry >= 0) out[count + __popc(m & ((1u << lane) - 1u))] = entry;
    count += __popc(m);
  }
  if (lane == 0) (is_q ? q_count : k_count)[(size_t)b * (is_q ? nql : nkl) + own] = count;
}

// The backward pre-pass with a rule: D and L log2 e padded per head as in the plain
// pre-pass, and rows that see nothing (L = -inf) or are padding get L = +inf, D = 0, so
// that every P of theirs is 0 and nothing of their O and dO is used.
template <int D, bool BF16>
__global__ void __launch_bounds__(256) rule_pre_kernel(const BwdArgs args, const int* q_doc, long long slots) {
  constexpr int kLpr = D / 8;      // lanes per row, 16 bytes of O and of dO each
  constexpr int kRpw = 32 / kLpr;  // rows per warp step
  const int lane = threadIdx.x & 31;
  const int sub = lane / kLpr, part = lane % kLpr;
  const long long warp0 = ((long long)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const long long nwarps = ((long long)gridDim.x * blockDim.x) >> 5;
  const uint16_t* o = reinterpret_cast<const uint16_t*>(args.o);
  const uint16_t* g = reinterpret_cast<const uint16_t*>(args.dout);
  const long long steps = (slots + kRpw - 1) / kRpw;
  for (long long st0 = warp0; st0 < steps; st0 += 2 * nwarps) {
    uint4 ov[2], gv[2];
    long long slot[2];
    float l[2];
    bool live[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const long long st = st0 + k * nwarps;
      slot[k] = st * kRpw + sub;
      const long long head = slot[k] / args.Npad;
      const int i = (int)(slot[k] - head * args.Npad);
      live[k] = st < steps && slot[k] < slots && i < args.N;
      l[k] = -INFINITY;
      ov[k] = gv[k] = make_uint4(0, 0, 0, 0);
      if (live[k]) {
        const size_t row = (size_t)head * args.N + i;
        l[k] = args.lse[row];
        if (q_doc && q_doc[(size_t)(head / args.H) * args.N + i] < 0) l[k] = -INFINITY;
        ov[k] = *reinterpret_cast<const uint4*>(o + row * D + part * 8);
        gv[k] = *reinterpret_cast<const uint4*>(g + row * D + part * 8);
      }
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint32_t ow[4] = {ov[k].x, ov[k].y, ov[k].z, ov[k].w};
      const uint32_t gw[4] = {gv[k].x, gv[k].y, gv[k].z, gv[k].w};
      float acc = 0.f;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        acc = fmaf(widen16<BF16>((uint16_t)(ow[w] & 0xFFFFu)), widen16<BF16>((uint16_t)(gw[w] & 0xFFFFu)), acc);
        acc = fmaf(widen16<BF16>((uint16_t)(ow[w] >> 16)), widen16<BF16>((uint16_t)(gw[w] >> 16)), acc);
      }
#pragma unroll
      for (int off = kLpr / 2; off > 0; off >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, off);
      if (st0 + k * nwarps < steps && slot[k] < slots && part == 0) {
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
  const long long want = (slots * D / 256 + 7) / 8;  // warp steps / warps per block
  const int grid = (int)std::max<long long>(1, std::min<long long>(want, (long long)std::max(sms, 1) * 16));
  rule_pre_kernel<D, BF16><<<grid, 256, 0, stream>>>(a, q_doc, slots);
  return cudaGetLastError();
}

}  // namespace

int rule_kind(const RuleArgs& r, bool cap) { return cap ? kRuleCap : r.slopes ? kRuleBias : kRuleMask; }

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
  const long long w1 = (long long)B * (nqb + nkb), w2 = (long long)B * (p.nql + p.nkl);
  rule_ids_kernel<<<(unsigned)((w1 + kPlanWarps - 1) / kPlanWarps), 32 * kPlanWarps, 0, stream>>>(
      q_doc, k_doc, ints(p.q_ids), ints(p.k_ids), q_sum, k_sum, B, N, Nk, nqb, nkb);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  rule_list_kernel<<<(unsigned)((w2 + kPlanWarps - 1) / kPlanWarps), 32 * kPlanWarps, 0, stream>>>(
      q_sum, k_sum, ints(p.q_list), ints(p.q_count), ints(p.k_list), ints(p.k_count), prefix, B, N, Nk, nqb, nkb, p.nql,
      q_rows / kBlkRows, p.nkl, p.q_list_stride, p.k_list_stride, causal);
  return cudaGetLastError();
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
  return d == 256 ? launch_bwd_256_rule(kind, bf16, q, k, v, dout, a, stream)
                  : launch_bwd_sq_rule(kind, d, bf16, q, k, v, dout, a, stream);
}

}  // namespace fa
