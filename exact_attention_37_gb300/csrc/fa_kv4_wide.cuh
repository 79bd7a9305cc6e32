// A tree of drafted tokens over the paged 4-bit cache when it has many rows (query heads of a
// group times drafted tokens): each cached token is read and turned into values once for 128 rows.
//
// The kernels of fa_kv4_attend.cuh turn codes into the register operands of narrow products, 16
// rows at a time, and read the cache again for every 16.  Here the values of a tile of T tokens
// are written to shared memory once and the fifth-generation tensor cores take them from there:
//   S = Q K^T  [128 rows x T tokens],  O += P V  [128 rows x d],  P from tensor memory.
// One CTA an SM, whose warps hand items (a tile's keys, a tile's values) along rings:
//   loader    bulk copies of codes and parameters of whole runs of pages into the raw ring;
//   8 warps   codes to 16-bit values, into the value ring as the operands want them (128-byte
//             swizzle); also the unit's rows of Q;
//   issuer    S(0) S(1) | P(j) V(j), S(j + 2) | ...: S(j + 2) takes the columns of P(j);
//   softmax   a thread a row.  At d = 64 and 128 two warpgroups take turns at the tiles, each with
//             an O of its own in tensor memory (lanes are rows, so either can read both), so that
//             the exponentials of one tile overlap the other's wait; at d = 256, where tensor
//             memory holds one O, one warpgroup.
// Eight channels lie in the order 0 4 1 5 2 6 3 7, as the codes' bits come out, in K and Q (the
// order of a contraction does not matter) and in V, whose columns are put right when O is stored.
//
// Rows are those of the sequence's drafted tokens (count, not N_q), tiles of all units are dealt to
// the CTAs in equal stretches, and parts of units that a stretch cuts are joined by a second kernel
// in CTA order.
#pragma once
#include <algorithm>
#include <climits>

#include "fa_kv4.cuh"
#include "fa_kv4_tree.cuh"
#include "fa_rule.cuh"
#include "ptx.cuh"

namespace fa {
namespace {

template <int D>
struct Wide {
  static constexpr int kTok = D == 256 ? 64 : 128;       // tokens of a tile
  static constexpr int kChains = D == 256 ? 1 : 2;       // softmax warpgroups
  static constexpr int kPanels = D / 64;
  static constexpr uint32_t kPanel = kTok * 128;         // a panel of 64 channels of a tile
  static constexpr uint32_t kQPanel = kWideRows * 128;
  static constexpr uint32_t kItem = kPanels * kPanel;    // a tile's keys or values
  static constexpr int kItems = 4;
  static constexpr int kRow = D / 2, kPar = D / 8;       // bytes of a row's codes, parameters
  static constexpr uint32_t kRaw = kTok * (kRow + kPar);
  static constexpr int kRaws = D == 256 ? 3 : D == 128 ? 6 : 8;
  static constexpr int kGroups = D / kKv4Group;
  // warps
  static constexpr int kSoftmax = 4 * kChains, kUnpack = 8;
  static constexpr int kWarpIssue = kSoftmax + kUnpack, kWarpLoad = kWarpIssue + 1;
  static constexpr int kThreads = 32 * (kWarpLoad + 1);
  // shared memory
  static constexpr uint32_t kQ = 0;
  static constexpr uint32_t kValues = kQ + kPanels * kQPanel;
  static constexpr uint32_t kRawRing = kValues + kItems * kItem;
  static constexpr uint32_t kBar = kRawRing + kRaws * kRaw;
  static constexpr int kRawFull = 0, kRawEmpty = kRawFull + kRaws, kFull = kRawEmpty + kRaws, kEmpty = kFull + kItems,
                       kSFull = kEmpty + kItems, kPFull = kSFull + 2, kODone = kPFull + 2, kQFull = kODone + 2,
                       kQEmpty = kQFull + 1, kUnitDone = kQEmpty + 1, kMlFull = kUnitDone + 1, kOFree = kMlFull + 1,
                       kDrain = kOFree + 1, kBars = kDrain + 1;
  static constexpr uint32_t kHave = kBar + 8 * kBars;              // runs of each raw slot that have a page
  static constexpr uint32_t kBad = kHave + 4 * kRaws;              // [4 units][groups][4]: drafted values that are not finite
  static constexpr uint32_t kMl = (kBad + 64 * kGroups + 15) / 16 * 16;  // [2][rows]: (m, l) of the chains
  static constexpr uint32_t kTmemSlot = kMl + 2 * kWideRows * 8;
  static constexpr uint32_t kBytes = kTmemSlot + 16;
  static constexpr uint32_t kAlloc = kBytes + 1024;
  static_assert(kAlloc <= 232448, "shared memory budget");
  // tensor memory columns
  static constexpr uint32_t s_col(int b) { return (uint32_t)kTok * b; }
  static constexpr uint32_t o_col(int c) { return 2u * kTok + (uint32_t)D * c; }
  static_assert(2 * kTok + kChains * D <= 512, "tensor memory budget");
};

// What a sequence has: cached tokens, drafted ones, tiles of its rows, tiles of its tokens.
struct WideSeq {
  int len, count, row_tiles, tiles;
};
template <int TOK>
__device__ __forceinline__ WideSeq wide_seq(const Kv4TreeArgs& a, int b) {
  WideSeq s;
  s.len = (int)min((long long)max(a.lengths[b], 0), (long long)a.pool.max_pages << a.pool.page_shift);
  s.count = draft_count(a, b);
  s.row_tiles = (a.group * s.count + kWideRows - 1) / kWideRows;
  s.tiles = (s.len + TOK - 1) / TOK;
  return s;
}
template <int TOK>
__device__ __forceinline__ int wide_work(const Kv4TreeArgs& a, int b) {
  const WideSeq s = wide_seq<TOK>(a, b);
  return s.tiles * s.row_tiles * a.pool.H_kv;
}

// The tiles of a stretch, unit by unit: all roles of a CTA walk through it alike.
template <int TOK>
struct WideWalk {
  int x, x_end;       // tiles, counted over all units
  int b, before;      // the sequence of tile x, tiles of the sequences in front of it
  int b_of;           // the sequence that `seq` is of
  WideSeq seq;
  int unit, p0, p1;   // of the sequence: unit, first and last + 1 tile of it in this stretch
  __device__ __forceinline__ bool next(const Kv4TreeArgs& a) {
    if (x >= x_end) return false;
    for (;;) {
      if (b_of != b) seq = wide_seq<TOK>(a, b), b_of = b;
      const int work = seq.tiles * seq.row_tiles * a.pool.H_kv;
      if (x < before + work) break;
      before += work;
      ++b;
    }
    unit = (x - before) / seq.tiles;
    p0 = x - before - unit * seq.tiles;
    p1 = min(seq.tiles, p0 + x_end - x);
    x += p1 - p0;
    return true;
  }
  __device__ __forceinline__ bool whole() const { return p0 == 0 && p1 == seq.tiles; }
  __device__ __forceinline__ int h_kv() const { return unit / seq.row_tiles; }
  __device__ __forceinline__ int row0() const { return unit % seq.row_tiles * kWideRows; }
};

// The stretch of this CTA: of all sequences' tiles, [c T / G, (c + 1) T / G) for CTA c of G; and the
// sequence in which it begins.  Returns T.  Every thread of the block calls it.
template <int TOK>
__device__ __forceinline__ int wide_begin(const Kv4TreeArgs& a, WideWalk<TOK>& walk) {
  __shared__ int sums[32], found[2];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int per = (a.B + blockDim.x - 1) / blockDim.x, b0 = threadIdx.x * per, b1 = min(b0 + per, a.B);
  int mine = 0;
  for (int b = b0; b < b1; ++b) mine += wide_work<TOK>(a, b);
  int upto = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, upto, off);
    if (lane >= off) upto += y;
  }
  if (lane == 31) sums[warp] = upto;
  __syncthreads();
  int before = upto - mine, total = 0;
  for (int w = 0; w < (int)(blockDim.x >> 5); ++w) {
    before += w < warp ? sums[w] : 0;
    total += sums[w];
  }
  const int G = min(a.ctas, total);
  walk.x = walk.x_end = 0;
  if ((int)blockIdx.x < G) {
    walk.x = (int)((long long)blockIdx.x * total / G);
    walk.x_end = (int)(((long long)blockIdx.x + 1) * total / G);
  }
  if (walk.x >= before && walk.x < before + mine) {
    int b = b0;
    for (int w; walk.x >= before + (w = wide_work<TOK>(a, b)); ++b) before += w;
    found[0] = b, found[1] = before;
  }
  __syncthreads();
  walk.b = found[0], walk.before = found[1];
  walk.b_of = -1;
  return total;
}
// Where a CTA's stretch begins, for the join: the sequence and its unit, the tile of the unit (0: it
// begins there, or the CTA has none), all tiles.
struct WideCut {
  int b, unit, p0, total;
};
// O = 0 and L = -inf for rows that no tile has: those behind a sequence's count, all of one
// without a token.
template <int D, int TOK>
__device__ __forceinline__ void wide_no_rows(const Kv4TreeArgs& a) {
  for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
    const WideSeq s = wide_seq<TOK>(a, b);
    const int from = s.tiles > 0 ? s.count : 0, none = a.N_q - from;
    for (int i = threadIdx.x; i < a.H * none * (D / 8); i += blockDim.x) {
      const int c = i % (D / 8), row = i / (D / 8), h = row / none;
      const size_t at = ((size_t)b * a.H + h) * a.N_q + from + row - h * none;
      reinterpret_cast<uint4*>(a.o)[at * (D / 8) + c] = make_uint4(0, 0, 0, 0);
      if (c == 0) a.lse[at] = -INFINITY;
    }
  }
}
// The CTA whose stretch [c T / G, (c + 1) T / G) holds tile x.
__device__ __forceinline__ int wide_cta_of(int x, int T, int G) { return (int)((((long long)x + 1) * G - 1) / T); }

// A tile item e of a unit with n tiles, in the order in which products take them:
// K(0) K(1) V(0) K(2) V(1) ... K(n-1) V(n-2) V(n-1).
__device__ __forceinline__ int wide_item(int e, int n, bool& is_v) {
  if (e == 0) {
    is_v = false;
    return 0;
  }
  if (e == 2 * n - 1) {
    is_v = true;
    return n - 1;
  }
  is_v = !(e & 1);
  return (e & 1) ? (e + 1) >> 1 : (e >> 1) - 1;
}

template <bool BF16>
__device__ __forceinline__ void unpack8(uint32_t codes, uint32_t s2, uint32_t l2, uint32_t (&v)[4]) {
  if constexpr (BF16)
    values4_scaled(codes, Scaled(s2, l2), v);
  else
    values4<false>(codes, s2, l2, v);
}

template <int D, bool BF16>
__global__ void __launch_bounds__(Wide<D>::kThreads, 1) kv4_wide_kernel(const Kv4TreeArgs a, WideCut* cuts) {
  using W = Wide<D>;
  constexpr int kTok = W::kTok;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  auto bar = [&](int i) -> uint32_t { return sbase + W::kBar + 8u * i; };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Kv4Pool& pool = a.pool;
  uint32_t* const err = pool.err;

  if (threadIdx.x == 0) {
    for (int s = 0; s < W::kRaws; ++s) mbar_init(bar(W::kRawFull + s), 1), mbar_init(bar(W::kRawEmpty + s), W::kUnpack);
    for (int s = 0; s < W::kItems; ++s) mbar_init(bar(W::kFull + s), W::kUnpack), mbar_init(bar(W::kEmpty + s), 1);
    for (int s = 0; s < 2; ++s)
      mbar_init(bar(W::kSFull + s), 1), mbar_init(bar(W::kPFull + s), 4), mbar_init(bar(W::kODone + s), 1);
    mbar_init(bar(W::kQFull), W::kUnpack);
    mbar_init(bar(W::kQEmpty), 1);
    mbar_init(bar(W::kUnitDone), 2);
    mbar_init(bar(W::kMlFull), W::kSoftmax);
    mbar_init(bar(W::kOFree), W::kSoftmax);
    mbar_init(bar(W::kDrain), 1);
    fence_mbar_init();
  }
  if (threadIdx.x < W::kGroups * 4) reinterpret_cast<uint32_t*>(smem + W::kBad)[threadIdx.x] = 0;
  grid_dep_wait();
  // ---- this CTA's stretch of all tiles
  WideWalk<kTok> walk;
  {
    wide_no_rows<D, kTok>(a);
    const int total = wide_begin<kTok>(a, walk);
    if (threadIdx.x == 0) {
      WideWalk<kTok> first = walk;
      const bool some = first.next(a);  // (without a stretch: nothing)
      cuts[blockIdx.x] = some ? WideCut{first.b, first.unit, first.p0, total} : WideCut{0, 0, 0, total};
    }
    if (walk.x == walk.x_end) return;
  }
  if (warp == W::kWarpIssue) {
    tmem_alloc(sbase + W::kTmemSlot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + W::kTmemSlot);
  debug_context(tmem, err);

  const int run = min(kTok, 1 << pool.page_shift), runs = kTok / run;  // tokens of a run
  bool ok = true;

  if (warp == W::kWarpLoad) {
    // ------------------------------------------------------------ loader
    uint32_t item = 0;
    while (ok && walk.next(a)) {
      const int32_t* table = pool.table + (size_t)walk.b * pool.max_pages;
      const int n = walk.p1 - walk.p0, h_kv = walk.h_kv(), len = walk.seq.len;
      // a run's lane looks its page up: -1 none
      auto page_of = [&](int p) -> int {
        const int tok = p * kTok + lane * run;
        return p < walk.p1 && lane < runs && tok < len ? kv4_page(table, pool.num_pages, tok >> pool.page_shift) : -1;
      };
      int k_page = page_of(walk.p0), v_page = k_page, next_page = page_of(walk.p0 + 1);
      for (int e = 0; e < 2 * n; ++e, ++item) {
        const int s = item % W::kRaws;
        const uint32_t use = item / W::kRaws;
        if (use > 0 && !(ok = warp_wait(bar(W::kRawEmpty + s), (use - 1) & 1, err, kErrTimeoutRing))) break;
        bool is_v;
        const int j = wide_item(e, n, is_v), p = walk.p0 + j, tok = p * kTok + lane * run;
        // keys run a tile ahead of values
        if (!is_v && j > 0) {
          v_page = k_page;
          k_page = next_page;
          next_page = page_of(p + 1);
        }
        const int page = !is_v ? k_page : j == n - 1 ? k_page : v_page;
        const bool there = lane < runs && tok < len;
        if (!is_v && there && page < 0) record_check(err, kDbgPage, (uint32_t)tok);
        const uint32_t have = __ballot_sync(0xffffffffu, page >= 0);
        if (lane == 0) {
          *reinterpret_cast<volatile uint32_t*>(smem + W::kHave + 4 * s) = have;
          mbar_expect_tx(bar(W::kRawFull + s), __popc(have) * run * (W::kRow + W::kPar));
        }
        __syncwarp();
        if (page >= 0) {
          const size_t row = (((size_t)page * pool.H_kv + h_kv) << pool.page_shift) + (tok & ((1 << pool.page_shift) - 1));
          const uint32_t to = sbase + W::kRawRing + s * W::kRaw;
          bulk_load(to + lane * run * W::kRow, pool.codes[is_v] + row * W::kRow, run * W::kRow, bar(W::kRawFull + s));
          bulk_load(to + kTok * W::kRow + lane * run * W::kPar, reinterpret_cast<const uint8_t*>(pool.params[is_v]) + row * W::kPar,
                    run * W::kPar, bar(W::kRawFull + s));
        }
      }
    }
    // every copy that was asked for lands before the CTA ends
    for (int s = 0; s < W::kRaws; ++s)
      if ((int)item > s) warp_wait_all(bar(W::kRawFull + s), ((item - 1 - s) / W::kRaws) & 1, err);
  } else if (warp == W::kWarpIssue) {
    // ------------------------------------------------------------ products
    if (lane == 0) {
      constexpr uint32_t kIdS = make_idesc_f16(BF16, kWideRows, kTok, false, false);
      constexpr uint32_t kIdPV = make_idesc_f16(BF16, kWideRows, D, false, true);
      constexpr uint32_t kHi = sdesc_hi_sw128(1024);
      uint32_t item = 0, units = 0, uses[2] = {0, 0};  // uses of the score buffers
      auto values = [&](uint32_t i) -> uint32_t { return sbase + W::kValues + (i % W::kItems) * W::kItem; };
      auto wait_item = [&](uint32_t i) -> bool {
        return mbar_wait(bar(W::kFull + i % W::kItems), (i / W::kItems) & 1, err, kErrTimeoutRing);
      };
      auto issue_s = [&](int buf, uint32_t i) {
        const uint32_t a0 = sdesc_lo(sbase + W::kQ, 16), b0 = sdesc_lo(values(i), 16);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          mma_ss_lohi(tmem + W::s_col(buf), a0 + (((kk >> 2) * W::kQPanel + (kk & 3) * 32) >> 4), kHi,
                      b0 + (((kk >> 2) * W::kPanel + (kk & 3) * 32) >> 4), kHi, kIdS, kk > 0);
        mma_commit(bar(W::kSFull + buf));
        mma_commit(bar(W::kEmpty + i % W::kItems));
      };
      while (ok && walk.next(a)) {
        const int n = walk.p1 - walk.p0;
        if (!(ok = mbar_wait(bar(W::kQFull), units & 1, err, kErrTimeoutRing))) break;
        // items of S(j): 0, 2 j - 1; of P(j) V(j): 2 j + 2, the last 2 n - 1
        for (int j = 0; ok && j < min(n, 2); ++j) {
          if (!(ok = wait_item(item + j))) break;
          tc_fence_after();
          issue_s(j, item + j);
          if (j == n - 1) mma_commit(bar(W::kQEmpty));
        }
        for (int j = 0; ok && j < n; ++j) {
          const int buf = j & 1, chain = W::kChains == 2 ? buf : 0;
          const uint32_t ev = item + (j == n - 1 ? 2 * n - 1 : 2 * j + 2);
          if (!(ok = wait_item(ev) && mbar_wait(bar(W::kPFull + buf), uses[buf] & 1, err, kErrTimeoutSoftmax))) break;
          ++uses[buf];
          tc_fence_after();
          const uint32_t b0 = sdesc_lo(values(ev), W::kPanel);
          const bool first = j < W::kChains;
#pragma unroll
          for (int kk = 0; kk < kTok / 16; ++kk)
            mma_ts_lohi(tmem + W::o_col(chain), tmem + W::s_col(buf) + 8 * kk, b0 + ((kk * 2048) >> 4), kHi, kIdPV,
                        first && kk == 0 ? 0u : 1u);
          mma_commit(bar(W::kODone + chain));
          mma_commit(bar(W::kEmpty + ev % W::kItems));
          if (j + 2 < n) {
            const uint32_t ek = item + 2 * j + 3;
            if (!(ok = wait_item(ek))) break;
            tc_fence_after();
            issue_s(buf, ek);
            if (j + 2 == n - 1) mma_commit(bar(W::kQEmpty));
          }
        }
        if (!ok) break;
        // the unit's products are done, and (an arrival of this thread, which has waited for every
        // item) what the unpacking warps noted of it can be read
        mma_commit(bar(W::kUnitDone));
        mbar_arrive(bar(W::kUnitDone));
        item += 2 * n;
        ++units;
      }
      mma_commit(bar(W::kDrain));
      mbar_wait(bar(W::kDrain), 0, err, kErrTimeoutMma, false);
    }
  } else if (warp >= W::kSoftmax) {
    // ------------------------------------------------------------ codes to values
    const int t = threadIdx.x - 32 * W::kSoftmax;
    uint32_t item = 0, units = 0;
    while (ok && walk.next(a)) {
      const int n = walk.p1 - walk.p0, len = walk.seq.len, count = walk.seq.count, prefix = len - count;
      uint32_t* bad = reinterpret_cast<uint32_t*>(smem + W::kBad) + (units & 3) * W::kGroups * 4;
      if (units > 0 && !(ok = warp_wait(bar(W::kQEmpty), (units - 1) & 1, err, kErrTimeoutMma))) break;
      // The next unit's notes are cleared here: every warp comes by here before any takes the
      // next unit, and those of three units ago have been read (the score products of the last
      // unit are done, so the products of the one before it were asked for, which the softmax
      // allows when it has written the one before that).
      if (t < W::kGroups * 4) (reinterpret_cast<uint32_t*>(smem + W::kBad) + ((units + 1) & 3) * W::kGroups * 4)[t] = 0;
      {
        const int h_kv = walk.h_kv(), rows = a.group * count - walk.row0();
#pragma unroll 2
        for (int i = t; i < kWideRows * (D / 8); i += 32 * W::kUnpack) {
          const int r = i / (D / 8), c = i % (D / 8);  // row, 16-byte chunk
          uint4 w = make_uint4(0, 0, 0, 0);
          if (r < rows) {
            const int col = walk.row0() + r, hh = col / count, qi = col - hh * count;
            const size_t at = ((size_t)walk.b * a.H + (size_t)h_kv * a.group + hh) * a.N_q + qi;
            w = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) + at * D + 8 * c);
          }
          st_shared_v4(sbase + W::kQ + (c >> 3) * W::kQPanel + sw128_offset(r, c & 7), __byte_perm(w.x, w.z, 0x5410),
                       __byte_perm(w.x, w.z, 0x7632), __byte_perm(w.y, w.w, 0x5410), __byte_perm(w.y, w.w, 0x7632));
        }
        fence_proxy_async_smem();
        warp_arrive(bar(W::kQFull));
      }
      for (int e = 0; e < 2 * n; ++e, ++item) {
        bool is_v;
        const int j = wide_item(e, n, is_v), tok0 = (walk.p0 + j) * kTok;
        const int rs = item % W::kRaws, s = item % W::kItems;
        if (!(ok = warp_wait(bar(W::kRawFull + rs), (item / W::kRaws) & 1, err, kErrTimeoutTma))) break;
        const uint32_t raw = sbase + W::kRawRing + rs * W::kRaw;
        const uint32_t have = *reinterpret_cast<volatile uint32_t*>(smem + W::kHave + 4 * rs);
        constexpr int kPer = kTok * W::kGroups / (32 * W::kUnpack);  // groups of 32 channels a thread
        uint32_t w[kPer][4], par[kPer];
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
          const int i = t + k * 32 * W::kUnpack;
          ld_shared_v4(raw + 16 * i, w[k][0], w[k][1], w[k][2], w[k][3]);
          asm volatile("ld.shared.b32 %0, [%1];" : "=r"(par[k]) : "r"(raw + kTok * W::kRow + 4 * i));
        }
        warp_arrive(bar(W::kRawEmpty + rs));
        // tokens that are not there stand for zeros, whatever the slot holds; so do drafted values
        // that are not finite, which are noted
        if (tok0 + kTok > prefix || have != (1u << runs) - 1u) {
#pragma unroll
          for (int k = 0; k < kPer; ++k) {
            const int i = t + k * 32 * W::kUnpack, in = i / W::kGroups, tok = tok0 + in;
            if (tok >= len || !((have >> (in / run)) & 1u)) {
              par[k] = 0;
            } else if (is_v && tok >= prefix && not_finite<BF16>(par[k])) {
              par[k] = 0;
              atomicOr(bad + i % W::kGroups * 4 + ((tok - prefix) >> 5), 1u << ((tok - prefix) & 31));
            }
          }
        }
        if (item >= W::kItems && !(ok = warp_wait(bar(W::kEmpty + s), (item / W::kItems - 1) & 1, err, kErrTimeoutMma))) break;
        const uint32_t to = sbase + W::kValues + s * W::kItem;
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
          const int i = t + k * 32 * W::kUnpack, r = i / W::kGroups, g = i % W::kGroups;
          // Threads next to each other write different 16-byte columns of the swizzle: those of the
          // other panels begin with another word of the group.
          const int turn = D == 64 ? 0 : D == 128 ? 2 * (g >> 1) : g >> 1;
          if (D > 64 && (turn & 2)) {
            uint32_t x = w[k][0];
            w[k][0] = w[k][2], w[k][2] = x;
            x = w[k][1], w[k][1] = w[k][3], w[k][3] = x;
          }
          if (D > 128 && (turn & 1)) {
            uint32_t x = w[k][0];
            w[k][0] = w[k][1], w[k][1] = x;
            x = w[k][2], w[k][2] = w[k][3], w[k][3] = x;
          }
          const uint32_t s2 = __byte_perm(par[k], par[k], 0x1010), l2 = __byte_perm(par[k], par[k], 0x3232);
          const uint32_t row = to + (g >> 1) * W::kPanel + r * 128;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t v[4];
            unpack8<BF16>(w[k][c], s2, l2, v);
            st_shared_v4(row + ((((g & 1) * 4 + (c ^ turn)) ^ (r & 7)) << 4), v[0], v[1], v[2], v[3]);
          }
        }
        fence_proxy_async_smem();
        warp_arrive(bar(W::kFull + s));
      }
      ++units;
    }
  } else {
    // ------------------------------------------------------------ softmax
    const int chain = warp >> 2;
    const int r = ((warp & 3) << 5) + lane;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const bool bias = a.rule.slopes != nullptr;
    const float scale2 = a.scale_log2 * (BF16 ? kScaledBack : 1.f);
    const float c = bias ? 1.f : a.cap ? a.rule.cap2 : scale2;  // from what the maximum works on to base 2
    float2* const ml = reinterpret_cast<float2*>(smem + W::kMl);
    uint32_t uses[2] = {0, 0}, o_uses = 0, units = 0;
    while (ok && walk.next(a)) {
      const int n = walk.p1 - walk.p0, len = walk.seq.len, count = walk.seq.count, prefix = len - count;
      const int h_kv = walk.h_kv(), col = walk.row0() + r, rows = a.group * count;
      const int hh = col < rows ? col / count : 0, qi = col < rows ? col - hh * count : 0;
      const bool warp_rows = walk.row0() + ((warp & 3) << 5) < rows;
      uint64_t see[2] = {0, 0};
      const int depth = col < rows ? tree_row(a, walk.b, count, prefix, qi, see) : -1;
      const float slope2 = bias && col < rows ? rule_slope2(a.rule, h_kv * a.group + hh) : 0.f;
      const int32_t* table = pool.table + (size_t)walk.b * pool.max_pages;
      // runs of a tile without a page, by a look at the table a tile ahead
      auto run_gone = [&](int p) -> bool {
        const int tok = p * kTok + lane * run;
        return p < walk.p1 && lane < runs && tok < len && kv4_page(table, pool.num_pages, tok >> pool.page_shift) < 0;
      };
      float m = -INFINITY, l = 0.f;
      bool gone = run_gone(walk.p0 + (W::kChains == 2 ? chain : 0));
      for (int j = W::kChains == 2 ? chain : 0; j < n; j += W::kChains) {
        const int buf = j & 1, tok0 = (walk.p0 + j) * kTok;
        const uint32_t tS = tmem + lanes + W::s_col(buf), tO = tmem + lanes + W::o_col(W::kChains == 2 ? chain : 0);
        const uint32_t missing = __ballot_sync(0xffffffffu, gone);
        gone = run_gone(walk.p0 + j + W::kChains);
        if (!(ok = warp_wait(bar(W::kSFull + buf), uses[buf] & 1, err, kErrTimeoutMma))) break;
        ++uses[buf];
        if (!warp_rows) {  // no row of the warp's: nobody looks at its P
          ++o_uses;
          warp_arrive(bar(W::kPFull + buf));
          continue;
        }
        tc_fence_after();
        const bool edge = tok0 + kTok > prefix || missing;
        uint64_t win[kTok / 64];
#pragma unroll
        for (int h = 0; h < kTok / 64; ++h) {
          win[h] = tree_window(see, tok0 + 64 * h - prefix);
          if (missing)
            for (int i = 0; i < runs; ++i)
              if ((missing >> i) & 1u)
                for (int k = max(i * run - 64 * h, 0); k < min((i + 1) * run - 64 * h, 64); ++k) win[h] &= ~(1ull << k);
        }
        // 32 scores: raw, or with a bias in base 2; hidden ones -inf
        auto scores = [&](int h, float (&s)[32], bool for_max) {
          uint32_t x[32];
          tmem_ld_32x32b_x32(tS + 32 * h, x);
          tmem_wait_ld();
          reg_fence32(x);
#pragma unroll
          for (int i = 0; i < 32; ++i) s[i] = __uint_as_float(x[i]);
          if (a.cap && (bias || !for_max)) {
            if constexpr (BF16) {
#pragma unroll
              for (int i = 0; i < 32; ++i) s[i] *= kScaledBack;
            }
            rule_tanh<32, true>(s, a.rule);
          }
          if (bias) {
            const float mul2 = a.cap ? a.rule.cap2 : scale2;
            const int d0 = prefix + depth - tok0 - 32 * h;  // distance to the chunk's first token
            if (!edge || tok0 + 32 * h + 32 <= prefix) {
              const float f0 = (float)d0;  // integers first: positions past 2^24 are not exact in fp32
#pragma unroll
              for (int i = 0; i < 32; ++i) s[i] = fmaf(-slope2, fabsf(f0 - (float)i), s[i] * mul2);
            } else {
              // a drafted token that this row sees is as deep as it has ancestors, which the row sees too
              const int dj = tok0 + 32 * h - prefix;
              int deep = dj <= 0 ? 0 : __popcll(dj < 64 ? see[0] & ((1ull << dj) - 1) : see[0]) +
                                           (dj <= 64 ? 0 : __popcll(see[1] & (dj < 128 ? (1ull << (dj - 64)) - 1 : ~0ull)));
              const uint32_t up = (uint32_t)tree_window(see, dj);
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                const bool drafted = dj + i >= 0;
                const int away = drafted ? depth - deep : d0 - i;
                if (drafted && ((up >> i) & 1u)) ++deep;
                s[i] = fmaf(-slope2, fabsf((float)away), s[i] * mul2);
              }
            }
          }
          if (edge) {
            const uint32_t part = (uint32_t)(win[h >> 1] >> (32 * (h & 1)));
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (!((part >> i) & 1u)) s[i] = -INFINITY;
          }
        };
        float top = -INFINITY;
#pragma unroll 1
        for (int h = 0; h < kTok / 32; ++h) {
          float s[32];
          scores(h, s, true);
          float x0 = max3f(s[0], s[1], s[2]), x1 = max3f(s[3], s[4], s[5]);
#pragma unroll
          for (int i = 6; i < 30; i += 4) x0 = max3f(x0, s[i], s[i + 1]), x1 = max3f(x1, s[i + 2], s[i + 3]);
          top = max3f(top, max3f(x0, s[30], s[31]), x1);
        }
        if (a.cap && !bias && top != -INFINITY) top = rule_tanh1(top * (BF16 ? kScaledBack : 1.f), a.rule);
        const float m_new = fmaxf(m, top);
        // the reference follows when the maximum is over 8 above it (base 2)
        const float m_use = m == -INFINITY || (m_new - m) * c > 8.f ? m_new : m;
        const float mc = m_use == -INFINITY ? 0.f : m_use * c;
        const float alpha = ex2_approx(fmaf(m, c, -mc));
        float l0 = 0.f, l1 = 0.f;
#pragma unroll 1
        for (int h = 0; h < kTok / 32; ++h) {
          float s[32];
          scores(h, s, false);
          uint32_t pw[16];
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            float x0, x1;
            fma2(s[i], s[i + 1], c, -mc, x0, x1);
            const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
            add2(l0, l1, p0, p1);
            pw[i >> 1] = pack2<BF16>(p0, p1);
          }
          tmem_st_32x32b_x16(tS + 16 * h, pw);
        }
        l = l * alpha + (l0 + l1);
        tmem_wait_st();
        if (j >= W::kChains && __any_sync(0xffffffffu, alpha != 1.f)) {
          // (the product before: the score product that this tile waited for came behind the one
          // before that, so the parity is not two phases old)
          if (!(ok = warp_wait(bar(W::kODone + (W::kChains == 2 ? chain : 0)), (o_uses - 1) & 1, err, kErrTimeoutMma))) break;
          tc_fence_after();
#pragma unroll 1
          for (int ch = 0; ch < D / 32; ++ch) {
            uint32_t o[32];
            tmem_ld_32x32b_x32(tO + 32 * ch, o);
            tmem_wait_ld();
            reg_fence32(o);
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
            tmem_st_32x32b_x32(tO + 32 * ch, o);
          }
          tmem_wait_st();
        }
        ++o_uses;
        tc_fence_before();
        warp_arrive(bar(W::kPFull + buf));
        m = m_use;
      }
      if (!ok) break;
      // ---- the unit's end: chains joined, rows or parts written
      if (!(ok = warp_wait(bar(W::kUnitDone), units & 1, err, kErrTimeoutMma))) break;
      tc_fence_after();
      if (depth < 0) m = -INFINITY, l = 0.f;
      float f[2] = {1.f, 0.f}, mm = m, ll = l;
      if constexpr (W::kChains == 2) {
        ml[chain * kWideRows + r] = make_float2(m, l);
        warp_arrive(bar(W::kMlFull));
        if (!(ok = warp_wait(bar(W::kMlFull), units & 1, err, kErrTimeoutSync))) break;
        const float2 x = ml[r], y = ml[kWideRows + r];
        mm = fmaxf(x.x, y.x);
        f[0] = mm == -INFINITY ? 0.f : ex2_approx((x.x - mm) * c);
        f[1] = mm == -INFINITY ? 0.f : ex2_approx((y.x - mm) * c);
        ll = f[0] * x.y + f[1] * y.y;
      }
      const float m2 = mm == -INFINITY ? mm : mm * c;  // base 2
      const bool whole = walk.whole(), live = depth >= 0;
      const size_t slot = blockIdx.x + (walk.p0 == 0 ? kWideMaxCtas : 0);
      const size_t out = ((size_t)walk.b * a.H + (size_t)h_kv * a.group + hh) * a.N_q + qi;
      const float inv = (whole ? (ll > 0.f ? 1.f / ll : 0.f) : 1.f) * (BF16 ? kScaledBack : 1.f);
      const uint32_t* bad = reinterpret_cast<const uint32_t*>(smem + W::kBad) + (units & 3) * W::kGroups * 4;
      if (warp_rows) {
        constexpr int kChunks = D / 32 / W::kChains;  // of 32 channels, a warpgroup
#pragma unroll 1
        for (int ch = chain * kChunks; ch < (chain + 1) * kChunks; ++ch) {
          float o[32];
          uint32_t x[32];
          tmem_ld_32x32b_x32(tmem + lanes + W::o_col(0) + 32 * ch, x);
          tmem_wait_ld();
          reg_fence32(x);
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = W::kChains == 2 ? __uint_as_float(x[i]) * f[0] : __uint_as_float(x[i]);
          if (W::kChains == 2 && n > 1) {
            tmem_ld_32x32b_x32(tmem + lanes + W::o_col(1) + 32 * ch, x);
            tmem_wait_ld();
            reg_fence32(x);
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = fmaf(__uint_as_float(x[i]), f[1], o[i]);
          }
          // a drafted value that is not finite, in this group of channels, of a token that the row sees
          const uint32_t* bg = bad + 4 * ch;
          const bool nan = ((uint32_t)see[0] & bg[0]) | ((uint32_t)(see[0] >> 32) & bg[1]) | ((uint32_t)see[1] & bg[2]) |
                           ((uint32_t)(see[1] >> 32) & bg[3]);
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = !live ? 0.f : nan ? NAN : o[i] * inv;
          if (whole) {
            if (col < rows)
#pragma unroll
              for (int q = 0; q < 32; q += 8)  // channels 0 4 1 5 2 6 3 7
                *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.o) + out * D + 32 * ch + q) =
                    make_uint4(pack2<BF16>(o[q], o[q + 2]), pack2<BF16>(o[q + 4], o[q + 6]), pack2<BF16>(o[q + 1], o[q + 3]),
                               pack2<BF16>(o[q + 5], o[q + 7]));
          } else {
            float* part = a.part_o + slot * (kWideRows * D) + (size_t)32 * ch * kWideRows + r;
#pragma unroll
            for (int i = 0; i < 32; ++i) part[i * kWideRows] = o[i];
          }
        }
        if (chain == 0) {
          if (!whole)
            *reinterpret_cast<float2*>(a.part_ml + (slot * kWideRows + r) * 2) = make_float2(m2, ll);
          else if (col < rows)
            a.lse[out] = ll == 0.f ? -INFINITY : m2 * kLn2 + logf(ll);
        }
      }
      tc_fence_before();
      if constexpr (W::kChains == 2) {  // both have read both O and their (m, l)
        warp_arrive(bar(W::kOFree));
        if (!(ok = warp_wait(bar(W::kOFree), units & 1, err, kErrTimeoutSync))) break;
      }
      ++units;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == W::kWarpIssue) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the parts of the units that several CTAs did, in CTA order.  Every such unit is cut where a
// CTA's stretch begins; the first of its cuts does it.  A block: kWideJoin channels of 128 rows,
// whose parts are shared by kWideShare threads a row.
constexpr int kWideJoin = 8, kWideShare = 4;
template <int D, bool BF16>
__global__ void __launch_bounds__(kWideRows* kWideShare) kv4_wide_join_kernel(const Kv4TreeArgs a, const WideCut* cuts) {
  constexpr int kSplit = D / kWideJoin;
  __shared__ float acc_of[kWideShare][kWideJoin][kWideRows];
  __shared__ float2 ml_of[kWideShare][kWideRows];
  grid_dep_launch();
  grid_dep_wait();
  const int cta = blockIdx.x / kSplit + 1, part = blockIdx.x % kSplit;
  const WideCut cut = cuts[cta];
  if (cut.p0 == 0) return;
  const int G = min(a.ctas, cut.total), first = (int)((long long)cta * cut.total / G) - cut.p0;  // the unit's first tile
  const int c0 = wide_cta_of(first, cut.total, G);
  if (c0 != cta - 1) return;
  const WideSeq s = wide_seq<Wide<D>::kTok>(a, cut.b);
  const int c1 = wide_cta_of(first + s.tiles - 1, cut.total, G);
  const int r = threadIdx.x % kWideRows, share = threadIdx.x / kWideRows;
  float mm = -INFINITY, ll = 0.f, acc[kWideJoin];
#pragma unroll
  for (int i = 0; i < kWideJoin; ++i) acc[i] = 0.f;
  auto slot_of = [&](int c) { return (size_t)c + (c == c0 ? kWideMaxCtas : 0); };
#pragma unroll 4
  for (int c = c0 + share; c <= c1; c += kWideShare) mm = fmaxf(mm, a.part_ml[(slot_of(c) * kWideRows + r) * 2]);
  const float ref = mm == -INFINITY ? 0.f : mm;
#pragma unroll 4
  for (int c = c0 + share; c <= c1; c += kWideShare) {
    const float2 ml = *reinterpret_cast<const float2*>(a.part_ml + (slot_of(c) * kWideRows + r) * 2);
    const float f = ex2_approx(ml.x - ref);
    ll = fmaf(f, ml.y, ll);
    const float* p = a.part_o + slot_of(c) * (kWideRows * D) + (size_t)part * kWideJoin * kWideRows + r;
#pragma unroll
    for (int i = 0; i < kWideJoin; ++i) acc[i] = fmaf(f, p[i * kWideRows], acc[i]);
  }
#pragma unroll
  for (int i = 0; i < kWideJoin; ++i) acc_of[share][i][r] = acc[i];
  ml_of[share][r] = make_float2(mm, ll);
  __syncthreads();
  const int h_kv = cut.unit / s.row_tiles, col = cut.unit % s.row_tiles * kWideRows + r;
  if (share > 0 || col >= a.group * s.count) return;
#pragma unroll
  for (int k = 1; k < kWideShare; ++k) mm = fmaxf(mm, ml_of[k][r].x);
  ll = 0.f;
#pragma unroll
  for (int i = 0; i < kWideJoin; ++i) acc[i] = 0.f;
#pragma unroll
  for (int k = 0; k < kWideShare; ++k) {
    const float2 ml = ml_of[k][r];
    const float f = mm == -INFINITY ? 0.f : ex2_approx(ml.x - mm);
    ll = fmaf(f, ml.y, ll);
#pragma unroll
    for (int i = 0; i < kWideJoin; ++i) acc[i] = fmaf(f, acc_of[k][i][r], acc[i]);
  }
  const int hh = col / s.count, qi = col - hh * s.count;
  const size_t out = ((size_t)cut.b * a.H + (size_t)h_kv * a.group + hh) * a.N_q + qi;
#pragma unroll
  for (int i = 0; i < kWideJoin; ++i) acc[i] = ll == 0.f ? 0.f : acc[i] / ll;
  static_assert(kWideJoin == 8, "channels 0 4 1 5 2 6 3 7");
  *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.o) + out * D + part * kWideJoin) =
      make_uint4(pack2<BF16>(acc[0], acc[2]), pack2<BF16>(acc[4], acc[6]), pack2<BF16>(acc[1], acc[3]), pack2<BF16>(acc[5], acc[7]));
  if (part == 0) a.lse[out] = ll == 0.f ? -INFINITY : mm * kLn2 + logf(ll);
}

template <int D, bool BF16>
cudaError_t launch_wide_t(Kv4TreeArgs a, long long room, int num_sms, cudaStream_t stream) {
  using W = Wide<D>;
  const long long tiles = (a.cols + kWideRows - 1) / kWideRows;
  const long long work = (long long)a.B * a.pool.H_kv * tiles * ((room + W::kTok - 1) / W::kTok);
  a.ctas = (int)std::max<long long>(1, std::min<long long>({work, (long long)num_sms, (long long)kWideMaxCtas}));
  auto kern = kv4_wide_kernel<D, BF16>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)W::kAlloc);
  if (e != cudaSuccess) return e;
  WideCut* cuts = reinterpret_cast<WideCut*>(a.part_ml + 2 * kWideMaxCtas * kWideRows * 2);
  e = launch_dependent(kern, (unsigned)a.ctas, W::kThreads, W::kAlloc, stream, a, cuts);
  if (e != cudaSuccess || a.ctas == 1) return e;
  return launch_dependent(kv4_wide_join_kernel<D, BF16>, (unsigned)((a.ctas - 1) * (D / kWideJoin)), kWideRows * kWideShare, 0,
                          stream, a, cuts);
}
}  // namespace
}  // namespace fa
