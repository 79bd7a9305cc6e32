// A tree of drafted tokens over the paged 4-bit cache when it has many rows (query heads of a
// group times drafted tokens): each cached token is read and turned into values once for 128 rows.
//
// The kernels of fa_kv4_attend.cuh turn codes into the register operands of narrow products, 16
// rows at a time, and read the cache again for every 16.  Here the values of a tile of T tokens
// are written to shared memory once and the fifth-generation tensor cores take them from there:
//   S = Q K^T  [128 rows x T tokens],  O += P V  [128 rows x d],  P from tensor memory, Q too where
// there is room for it (two operands in shared memory are all that it can read).
// One CTA an SM, whose warps hand items (a tile's keys, a tile's values) along rings:
//   loaders   (of keys, of values) bulk copies of codes and parameters of whole runs of pages into
//             the raw ring;
//   unpack    4 warps for keys and 4 for values (at d = 64 and 128 teams of two, tile by tile in turn):
//             codes to 16-bit values, into the value ring as the products want them (128-byte swizzle);
//             those for values also lay Q out where it is in shared memory;
//   issuer    S(0) S(1) | P(j) V(j), S(j + 2) | ...: S(j + 2) takes the columns of P(j);
//   softmax   a thread a row.  At d = 64 and 128 two warpgroups take turns at the tiles, each with an
//             O, a maximum and a sum of its own (a chain), so that one works while the other waits; at
//             d = 256, where tensor memory holds one O, they take halves of a tile's scores.
// Units of at most 64 (32) rows have them two (four) times over in the 128 rows of the product,
// whose other rows are for nothing: each copy takes its part of a tile's tokens (and 0 for the
// others), so that the exponentials are spread over all lanes.  Chains and copies are softmaxes of
// their own until the unit's end, where they are joined.
// Scores, maxima, sums and O are fp32.  P is rounded to the cache's type, the only one that a product with
// its values takes (half a step of each, against O's own rounding of half a step), its sum is taken before.
// Eight channels lie in the order 0 4 1 5 2 6 3 7, as the codes' bits come out, in K and Q (the
// order of a contraction does not matter) and in V, whose columns are put right when O is stored.
//
// Rows are those of the sequence's drafted tokens (count, not N_q).  Tiles of all units, and for each
// unit as many more as its beginning and end cost, are dealt to the CTAs in equal stretches; parts of
// units that a stretch cuts are joined by a second kernel in CTA order.
//
// Measured (one GB300, bf16): 32 sequences of 2048 to 16384 tokens, 16 drafted, 8 heads of 4, d 128, 150 us
// (389 MB, 57 us at the copy's rate; the products of 128 rows, half of them or more for nothing here, 70);
// 2 of 100003 tokens, 37 drafted, 4 heads of 4, d 256, 176 us.  A tile of 128 tokens takes 0.87 us with 64
// rows and 1.17 with 128 at d 128, where its products are 0.58: a place of the value ring is unpacked (1.2 us
// for two warps), taken by a product and only then unpacked again, and shared memory holds two places for
// each of keys and values.  The ALU is 40 % busy, 0.5 instructions a clock of each scheduler.  Teams of four
// warps instead of two at d 128: 156 us; of two at d 256: 187; a tile's codes loaded in front of the wait
// for its place: no change.
#pragma once
#include <algorithm>
#include <climits>
#include <type_traits>

#include "fa_kv4.cuh"
#include "fa_kv4_tree.cuh"
#include "fa_rule.cuh"
#include "fa_kv4_ptx.cuh"

namespace fa {
namespace {

template <int D>
struct Wide {
  static constexpr int kTok = D == 256 ? 64 : 128;       // tokens of a tile
  // The two softmax warpgroups: chains, or, where tensor memory holds one O, halves of a tile's scores.
  static constexpr int kChains = D == 256 ? 1 : 2, kSides = 3 - kChains;
  static constexpr bool kQTmem = D != 128;               // where Q is
  static constexpr int kPanels = D / 64;
  static constexpr uint32_t kPanel = kTok * 128;         // a panel of 64 channels of a tile
  static constexpr uint32_t kQPanel = kWideRows * 128;
  static constexpr uint32_t kItem = kPanels * kPanel;    // a tile's keys or values
  static constexpr int kItems = 4;
  static constexpr int kRow = D / 2, kPar = D / 8;       // bytes of a row's codes, parameters
  static constexpr uint32_t kRaw = kTok * (kRow + kPar);
  static constexpr int kRaws = D == 128 ? 2 : 4;         // raw slots of keys, and of values (even: each is one team's)
  static constexpr int kGroups = D / kKv4Group;
  static constexpr int kCopies = D == 256 ? 2 : 4;       // of a unit's rows, at most
  // warps: whole warpgroups, which share the registers out
  static constexpr int kSoftmax = 8, kUnpack = 8, kTeam = D == 256 ? 4 : 2, kTeams = 4 / kTeam;
  static constexpr int kWarpIssue = kSoftmax + kUnpack, kWarpLoad = kWarpIssue + 1, kWarpSpare = kWarpIssue + 3;
  static constexpr int kThreads = 32 * (kWarpIssue + 4);
  static constexpr int kRegsLaunch = 96, kRegsSoftmax = 144, kRegsUnpack = 72, kRegsRest = 48;
  static_assert(2 * kRegsSoftmax + 2 * kRegsUnpack + kRegsRest <= 5 * kRegsLaunch, "the split stays inside the launch's registers");
  // shared memory
  static constexpr uint32_t kQ = 0;
  static constexpr uint32_t kValues = kQ + (kQTmem ? 0 : kPanels * kQPanel);
  static constexpr uint32_t kRawRing = kValues + kItems * kItem;
  static constexpr int kAddCh = 16;                                // channels of the copies' O that are added at a time
  static constexpr uint32_t kAdd = kRawRing + 2 * kRaws * kRaw;        // [warpgroups][kAddCh][96]
  static constexpr uint32_t kMl = kAdd + 2 * kAddCh * 96 * 4;       // (m, l) of a row's parts
  static constexpr uint32_t kMax = kMl + 2 * kWideRows * 8;         // [2][sides][rows]: maxima of halves
  static constexpr uint32_t kBar = kMax + (kSides == 2 ? 4 * kWideRows * 4 : 0);
  static constexpr int kRawFull = 0, kRawEmpty = kRawFull + 2 * kRaws, kFull = kRawEmpty + 2 * kRaws, kEmpty = kFull + kItems,
                       kSFull = kEmpty + kItems, kPFull = kSFull + 2, kODone = kPFull + 2, kQFull = kODone + 1,
                       kQEmpty = kQFull + 1, kUnitDone = kQEmpty + 1, kDrain = kUnitDone + 1, kBars = kDrain + 1;
  static constexpr uint32_t kHave = kBar + 8 * kBars;              // runs of each raw slot that have a page
  static constexpr uint32_t kAsked = kHave + 8 * kRaws;            // how often each raw slot was asked for
  static constexpr uint32_t kGone = kAsked + 8 * kRaws;            // [4 tiles]: runs without a page
  static constexpr uint32_t kBad = kGone + 16;             // [4 units][groups][4]: drafted values that are not finite
  static constexpr uint32_t kTmemSlot = (kBad + 64 * kGroups + 15) / 16 * 16;
  static constexpr uint32_t kBytes = kTmemSlot + 16;
  static constexpr uint32_t kAlloc = kBytes + 1024;
  static_assert(kAlloc + 512 <= 232448, "shared memory budget");
  // tensor memory columns
  static constexpr __host__ __device__ uint32_t s_col(int b) { return (uint32_t)kTok * b; }
  static constexpr __host__ __device__ uint32_t o_col(int c) { return 2u * kTok + (uint32_t)D * c; }
  static constexpr uint32_t kQCol = 2u * kTok + (uint32_t)D * kChains;
  static_assert(kQCol + (kQTmem ? D / 2 : 0) <= 512, "tensor memory budget");
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
// What a unit costs beside its tiles, in tiles: its rows, the first tiles' latency, the join of its
// chains and copies.  6 us, where a tile of 128 tokens takes 0.9 (a fit of the blocks' times for 32
// sequences of 2048 to 16384 tokens at d 128).  With 3, 7 and 12 tiles, us: those sequences 160.4, 150.6 and
// 153; at d 64 121, 117.5 and 119.7, 32 of up to 2000 tokens 42.3, 39.8 and 41.5.
template <int TOK>
constexpr int kWideUnit = TOK == 64 ? 5 : 7;
template <int TOK>
__device__ __forceinline__ int wide_unit(const WideSeq& s) { return s.tiles > 0 ? s.tiles + kWideUnit<TOK> : 0; }
template <int TOK>
__device__ __forceinline__ int wide_work(const Kv4TreeArgs& a, int b) {
  const WideSeq s = wide_seq<TOK>(a, b);
  return wide_unit<TOK>(s) * s.row_tiles * a.pool.H_kv;
}

// A unit (a sequence's key/value head and 128 of its rows) and the tiles of it in a stretch.
struct WideUnit {
  int b, h_kv, row0;
  int p0, n;          // first tile, tiles
  int len, count;     // of the sequence: cached tokens, drafted ones
  uint32_t by_count;  // ceil(2^32 / count), 0 for 1
  bool whole;         // no other CTA has tiles of it
  // Row `col` of the group as query head of it and drafted token (col count < 2^32).
  __device__ __forceinline__ void split(int col, int& hh, int& qi) const {
    hh = by_count ? (int)__umulhi((uint32_t)col, by_count) : col;
    qi = col - hh * count;
  }
};
// The tiles of a stretch, unit by unit: all roles of a CTA walk through it alike.
template <int TOK>
struct WideWalk {
  int x, x_end;       // places of tiles, counted over all units
  int b, before;      // the sequence of tile x, tiles of the sequences in front of it
  __device__ __forceinline__ bool next(const Kv4TreeArgs& a, WideUnit& u) {
    WideSeq seq;
    int cost, unit;
    for (;;) {
      if (x >= x_end) return false;
      seq = wide_seq<TOK>(a, b);
      cost = wide_unit<TOK>(seq);
      const int work = cost * seq.row_tiles * a.pool.H_kv;
      if (x >= before + work) {
        before += work;
        ++b;
        continue;
      }
      unit = (x - before) / cost;
      u.p0 = x - before - unit * cost;
      if (u.p0 < seq.tiles) break;
      x += cost - u.p0;  // the end of a unit that another CTA has
    }
    u.b = b;
    u.h_kv = unit / seq.row_tiles;
    u.row0 = unit % seq.row_tiles * kWideRows;
    u.n = min(seq.tiles - u.p0, x_end - x);
    x += u.p0 + u.n == seq.tiles ? cost - u.p0 : u.n;
    u.len = seq.len, u.count = seq.count;
    u.by_count = 0xFFFFFFFFu / (uint32_t)seq.count + 1u;
    u.whole = u.n == seq.tiles;
    return true;
  }
};

// The stretch of this CTA: of all places, [c T / G, (c + 1) T / G) for CTA c of G; and the
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
  return total;
}
// Where a CTA's stretch begins, for the join: the unit, the tile of it (0: it begins there, or the
// CTA has none), all tiles.
struct WideCut {
  int b, h_kv, row0, p0, total, len, count, none;
};
// O = 0 and L = -inf for rows that no tile has: those behind a sequence's count, all of one
// without a token.  Query heads are dealt to the CTAs and in a CTA to `warps` warps, whatever the
// CTAs have of the tiles, and a warp looks 32 of them up at once: there may be more of these rows than
// of the others (one sequence of 1024 tokens with 1 of 128 rows real, H 64/8, d 256: 547 us with a
// sequence a warp, 26 so, where 128 real rows take 38).
template <int D, int TOK>
__device__ __forceinline__ void wide_no_rows(const Kv4TreeArgs& a, int warp, int warps) {
  const int lane = threadIdx.x & 31, heads = a.B * a.H, ctas = gridDim.x;
#pragma unroll 1
  for (int k = warp; (int)blockIdx.x + k * ctas < heads; k += 32 * warps) {
    const int mine = blockIdx.x + (k + lane * warps) * ctas;
    int none = 0;
    if (mine < heads) {
      const WideSeq s = wide_seq<TOK>(a, mine / a.H);
      none = a.N_q - (s.tiles > 0 ? s.count : 0);
    }
    for (uint32_t some = __ballot_sync(0xffffffffu, none > 0); some; some &= some - 1) {
      const int from = __ffs(some) - 1, rows = __shfl_sync(0xffffffffu, none, from);
      const size_t at = ((size_t)__shfl_sync(0xffffffffu, mine, from) + 1) * a.N_q - rows;
      uint4* o = reinterpret_cast<uint4*>(a.o) + at * (D / 8);
#pragma unroll 1
      for (int i = lane; i < rows * (D / 8); i += 32) o[i] = make_uint4(0, 0, 0, 0);
#pragma unroll 1
      for (int i = lane; i < rows; i += 32) a.lse[at + i] = -INFINITY;
    }
  }
}
// The CTA whose stretch [c T / G, (c + 1) T / G) holds tile x.
__device__ __forceinline__ int wide_cta_of(int x, int T, int G) { return (int)((((long long)x + 1) * G - 1) / T); }

// The place of tile j's keys or values among the items of a unit with n tiles, in the order in which
// products take them: K(0) K(1) V(0) K(2) V(1) ... K(n-1) V(n-2) V(n-1).  Tiles are counted from the
// stretch's last: with a distance bias the maximum is among the first then, and O need not be rescaled
// tile after tile.
__device__ __forceinline__ int wide_item(bool values, int j, int n) {
  if (values) return j == n - 1 ? 2 * n - 1 : 2 * j + 2;
  return j == 0 ? 0 : 2 * j - 1;
}

// The values of 8 codes of a group; bf16 ones times 2^-32.
struct ScaleLow {
  uint32_t s, low;
  __device__ __forceinline__ ScaleLow(uint32_t s2, uint32_t l2) : s(s2), low(l2) {}
};
template <bool BF16>
struct Unpack {
  std::conditional_t<BF16, Scaled, ScaleLow> par;
  __device__ __forceinline__ Unpack(uint32_t s2, uint32_t l2) : par(s2, l2) {}
  __device__ __forceinline__ void operator()(uint32_t codes, uint32_t (&v)[4]) const {
    if constexpr (BF16) values4_scaled(codes, par, v);
    else values4<false>(codes, par.s, par.low, v);
  }
};

// The rows of a unit as a softmax thread sees them.
struct WideRow {
  int copies, rows, row;  // of the unit's rows; rows of the tile; this thread's among them
  int copy;               // which copy the thread is in
  bool warp_live;         // whether the warp has any
};
template <int COPIES>
__device__ __forceinline__ WideRow wide_row(int rows, int r) {
  WideRow w;
  w.copies = COPIES == 4 && rows <= 32 ? 4 : rows <= 64 ? 2 : 1;
  const int each = kWideRows / w.copies;
  w.rows = rows;
  w.row = r % each;
  w.copy = r / each;
  w.warp_live = (r & ~31) % each < rows;
  return w;
}

// RULE: whether scores may have a cap or a bias.
template <int D, bool BF16, bool RULE>
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
    for (int s = 0; s < 2 * W::kRaws; ++s) mbar_init(bar(W::kRawFull + s), 1), mbar_init(bar(W::kRawEmpty + s), W::kTeam);
    for (int s = 0; s < W::kItems; ++s) mbar_init(bar(W::kFull + s), W::kTeam), mbar_init(bar(W::kEmpty + s), 1);
    for (int s = 0; s < 2; ++s) mbar_init(bar(W::kSFull + s), 2), mbar_init(bar(W::kPFull + s), 4 * W::kSides);
    mbar_init(bar(W::kODone), 1);
    mbar_init(bar(W::kQFull), W::kQTmem ? W::kSoftmax : W::kUnpack / 2);
    mbar_init(bar(W::kQEmpty), 1);
    mbar_init(bar(W::kUnitDone), 2);
    mbar_init(bar(W::kDrain), 1);
    fence_mbar_init();
  }
  for (int i = threadIdx.x; i < 16 * W::kGroups; i += W::kThreads) reinterpret_cast<uint32_t*>(smem + W::kBad)[i] = 0;
  if (threadIdx.x < 2 * W::kRaws) reinterpret_cast<uint32_t*>(smem + W::kAsked)[threadIdx.x] = 0;
  grid_dep_wait();
  // ---- this CTA's stretch of all tiles
  WideWalk<kTok> walk;
  {
    const int total = wide_begin<kTok>(a, walk);
    // A warp that has no part in the tiles does what the join wants to know and the rows without any.
    if (warp == W::kWarpSpare) {
      WideWalk<kTok> first = walk;
      WideUnit u{};
      first.next(a, u);  // (without a stretch: nothing)
      if (lane == 0) cuts[blockIdx.x] = WideCut{u.b, u.h_kv, u.row0, u.p0, total, u.len, u.count, 0};
    }
    if (walk.x == walk.x_end) {
      wide_no_rows<D, kTok>(a, warp, W::kThreads / 32);
      return;
    }
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

  if (warp >= W::kWarpIssue) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(W::kRegsRest));
    if (warp == W::kWarpLoad || warp == W::kWarpLoad + 1) {
      // ---------------------------------------------------------- loaders: of keys, of values
      const int which = warp - W::kWarpLoad;
      const uint8_t* const codes = pool.codes[which];
      const uint8_t* const params = reinterpret_cast<const uint8_t*>(pool.params[which]);
      const uint32_t at_codes = lane * run * W::kRow, at_params = kTok * W::kRow + lane * run * W::kPar;
      uint32_t slot = which * W::kRaws, uses = 0;  // the next one to fill, and how often it was
      WideUnit u;
      while (ok && walk.next(a, u)) {
        const int32_t* table = pool.table + (size_t)u.b * pool.max_pages;
        const int n = u.n, len = u.len;
        const size_t head = (size_t)u.h_kv << pool.page_shift;
        // a run's lane looks its page up, a tile ahead (and looks at what it got a tile later)
        auto look_up = [&](int p) -> int {
          const int tok = p * kTok + lane * run;
          return p >= u.p0 && lane < runs && tok < len ? table[tok >> pool.page_shift] : -1;
        };
        // pages of the next tiles, the nearest first
        int ahead[3] = {look_up(u.p0 + n - 1), look_up(u.p0 + n - 2), look_up(u.p0 + n - 3)};
        for (int j = 0; j < n; ++j) {
          const int p = u.p0 + n - 1 - j, tok = p * kTok + lane * run;
          const int page = ahead[0] < 0 || ahead[0] >= pool.num_pages ? -1 : ahead[0];
          ahead[0] = ahead[1], ahead[1] = ahead[2];
          ahead[2] = look_up(p - 3);
          if (uses > 0 && !(ok = warp_nap(bar(W::kRawEmpty + slot), (uses - 1) & 1, err, kErrTimeoutRing))) break;
          if (!which && lane < runs && tok < len && page < 0) record_check(err, kDbgPage, (uint32_t)tok);
          const uint32_t have = __ballot_sync(0xffffffffu, page >= 0);
          if (lane == 0) {
            *reinterpret_cast<volatile uint32_t*>(smem + W::kHave + 4 * slot) = have;
            *reinterpret_cast<volatile uint32_t*>(smem + W::kAsked + 4 * slot) = uses + 1;
            mbar_expect_tx(bar(W::kRawFull + slot), __popc(have) * run * (W::kRow + W::kPar));
          }
          __syncwarp();
          if (page >= 0) {
            const size_t row = (((size_t)page * pool.H_kv) << pool.page_shift) + head + (tok & ((1 << pool.page_shift) - 1));
            const uint32_t to = sbase + W::kRawRing + slot * W::kRaw;
            bulk_load(to + at_codes, codes + row * W::kRow, run * W::kRow, bar(W::kRawFull + slot));
            bulk_load(to + at_params, params + row * W::kPar, run * W::kPar, bar(W::kRawFull + slot));
          }
          if (++slot == (which + 1) * W::kRaws) slot = which * W::kRaws, ++uses;
          // the tile behind the next is asked for in L2: memory's latency would be most of a load's
          const int later = ahead[1];
          if (p - 2 >= u.p0 && (uint32_t)later < (uint32_t)pool.num_pages) {
            const size_t row = (((size_t)later * pool.H_kv) << pool.page_shift) + head + ((tok - 2 * kTok) & ((1 << pool.page_shift) - 1));
            bulk_prefetch(codes + row * W::kRow, run * W::kRow);
            bulk_prefetch(params + row * W::kPar, run * W::kPar);
          }
        }
      }
    } else if (warp == W::kWarpSpare) {
      wide_no_rows<D, kTok>(a, 0, 1);
    } else if (warp == W::kWarpIssue) {
      // ---------------------------------------------------------- products
      constexpr uint32_t kIdS = make_idesc_f16(BF16, kWideRows, kTok, false, false);
      constexpr uint32_t kIdPV = make_idesc_f16(BF16, kWideRows, D, false, true);
      constexpr uint32_t kHi = sdesc_hi_sw128(1024);
      uint32_t item = 0, units = 0, parity = 0;  // bit b: of score buffer b's next P
      auto values = [&](uint32_t i) -> uint32_t { return sbase + W::kValues + (i % W::kItems) * W::kItem; };
      auto wait_item = [&](uint32_t i) -> bool {
        return warp_nap(bar(W::kFull + i % W::kItems), (i / W::kItems) & 1, err, kErrTimeoutRing);
      };
      // (the whole warp goes through the loop and one lane issues: descriptors stay in uniform registers)
      auto issue_s = [&](int buf, uint32_t i, bool last) {
        const uint32_t a0 = sdesc_lo(sbase + W::kQ, 16), b0 = sdesc_lo(values(i), 16);
        if (elect_one()) {
#pragma unroll 2
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t b = b0 + (((kk >> 2) * W::kPanel + (kk & 3) * 32) >> 4);
            if constexpr (W::kQTmem)
              mma_ts_lohi(tmem + W::s_col(buf), tmem + W::kQCol + 8 * kk, b, kHi, kIdS, kk > 0);
            else
              mma_ss_lohi(tmem + W::s_col(buf), a0 + (((kk >> 2) * W::kQPanel + (kk & 3) * 32) >> 4), kHi, b, kHi, kIdS, kk > 0);
          }
          mma_commit(bar(W::kSFull + buf));
          mbar_arrive(bar(W::kSFull + buf));  // what the unpacking warps noted of the tile can be read
          mma_commit(bar(W::kEmpty + i % W::kItems));
          if (last) mma_commit(bar(W::kQEmpty));
        }
      };
      WideUnit u;
      while (ok && walk.next(a, u)) {
        const int n = u.n;
        if (!(ok = warp_nap(bar(W::kQFull), units & 1, err, kErrTimeoutSoftmax))) break;
        // items of S(j): 0, 2 j - 1; of P(j) V(j): 2 j + 2, the last 2 n - 1
        for (int j = 0; ok && j < min(n, 2); ++j) {
          if (!(ok = wait_item(item + j))) break;
          tc_fence_after();
          issue_s(j, item + j, j == n - 1);
        }
        for (int j = 0; ok && j < n; ++j) {
          const int buf = j & 1;
          const uint32_t ev = item + wide_item(true, j, n), ek = item + 2 * j + 3;
          // What has mostly come by now is asked for at once: a wait after the other, each a vote of the warp,
          // would be most of the time between two products.  (Tests: a wait for the keys of two tiles on
          // would hold back the product whose operands are there.)
          const bool p_v = mbar_test_wait(bar(W::kFull + ev % W::kItems), (ev / W::kItems) & 1) &
                           mbar_test_wait(bar(W::kPFull + buf), (parity >> buf) & 1);
          const bool k = j + 2 >= n || mbar_test_wait(bar(W::kFull + ek % W::kItems), (ek / W::kItems) & 1);
          const bool have_k = __all_sync(0xffffffffu, k);
          if (!__all_sync(0xffffffffu, p_v) &&
              !(ok = wait_item(ev) && warp_nap(bar(W::kPFull + buf), (parity >> buf) & 1, err, kErrTimeoutSoftmax)))
            break;
          parity ^= 1u << buf;
          tc_fence_after();
          const uint32_t b0 = sdesc_lo(values(ev), W::kPanel);
          if (elect_one()) {
#pragma unroll 2
            for (int kk = 0; kk < kTok / 16; ++kk)
              mma_ts_lohi(tmem + W::o_col(W::kChains == 2 ? buf : 0), tmem + W::s_col(buf) + 8 * kk, b0 + ((kk * 2048) >> 4), kHi, kIdPV,
                          j >= W::kChains || kk > 0);
            if constexpr (W::kChains == 1) mma_commit(bar(W::kODone));
            mma_commit(bar(W::kEmpty + ev % W::kItems));
          }
          if (j + 2 < n) {
            if (!have_k && !(ok = wait_item(ek))) break;
            tc_fence_after();
            issue_s(buf, ek, j + 2 == n - 1);
          }
        }
        if (!ok) break;
        // the unit's products are done, and (an arrival of this thread, which has waited for every
        // item) what the unpacking warps noted of it can be read
        if (elect_one()) {
          mma_commit(bar(W::kUnitDone));
          mbar_arrive(bar(W::kUnitDone));
        }
        item += 2 * n;
        ++units;
      }
      if (elect_one()) mma_commit(bar(W::kDrain));
      warp_wait_all(bar(W::kDrain), 0, err);
    }
  } else if (warp >= W::kSoftmax) {
    // ------------------------------------------------------------ codes to values
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(W::kRegsUnpack));
    // Teams of two warps take the keys, or the values, of every other tile: one is at its barriers while
    // the other computes.  At d = 256, where a chain of
    // softmaxes waits for each item, four warps take every one.
    const int is_v = (warp - W::kSoftmax) / 4, team = W::kTeams == 2 ? (warp >> 1) & 1 : 0, t = threadIdx.x % (32 * W::kTeam);
    // A thread takes group g (of 32 channels) of rows r, r + kRows, ...: its places in an item are
    // those of row r and a constant.
    constexpr int kRows = 32 * W::kTeam / W::kGroups, kPer = 4, kTimes = kTok / (kRows * kPer);
    static_assert(kRows % 8 == 0 && kRows * kPer * kTimes == kTok, "the swizzle of a thread's rows");
    const int r = t / W::kGroups, g = t % W::kGroups;
    // Threads next to each other write different 16-byte columns of the swizzle: those of the other
    // panels begin with another word of the group.
    const int turn = D == 64 ? 0 : D == 128 ? 2 * (g >> 1) : g >> 1;
    uint32_t column[4];  // where word c ^ turn of row r goes, in an item
#pragma unroll
    for (int c = 0; c < 4; ++c) column[c] = (g >> 1) * W::kPanel + r * 128 + ((((g & 1) * 4 + (c ^ turn)) ^ (r & 7)) << 4);
    uint32_t item0 = 0, units = 0, tile0 = 0, slot = team, raw_uses = 0;  // slot: of this class
    // Q of a unit, as the score products want it: the warps that unpack values, whose first item of a
    // unit is wanted last.  The rows are on their way while the unit before is worked on.
    auto put_q = [&](const WideUnit& w) -> bool {
      constexpr int kStep = 128 / (D / 8), kAhead = 8;
      const int t4 = threadIdx.x % 128, c = t4 % (D / 8), rows = min(a.group * w.count - w.row0, kWideRows);
      const int copies = wide_row<W::kCopies>(rows, 0).copies, each = kWideRows / copies;
      const uint4* q = static_cast<const uint4*>(a.q) + ((size_t)w.b * a.H + (size_t)w.h_kv * a.group) * a.N_q * (D / 8) + c;
#pragma unroll 1
      for (int r0 = t4 / (D / 8); r0 < each; r0 += kStep * kAhead) {
        uint4 v[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          const int r = r0 + k * kStep;
          int hh, qi;
          w.split(w.row0 + r, hh, qi);
          v[k] = r < rows ? q[(hh * a.N_q + qi) * (D / 8)] : make_uint4(0, 0, 0, 0);
        }
        if (r0 < kStep && units > 0 && !warp_nap(bar(W::kQEmpty), (units - 1) & 1, err, kErrTimeoutMma)) return false;
#pragma unroll 1
        for (int copy = 0; copy < kWideRows; copy += each)
#pragma unroll
          for (int k = 0; k < kAhead; ++k)
            if (r0 + k * kStep < each)
              st_shared_v4(sbase + W::kQ + (c >> 3) * W::kQPanel + sw128_offset(r0 + k * kStep + copy, c & 7),
                           __byte_perm(v[k].x, v[k].z, 0x5410), __byte_perm(v[k].x, v[k].z, 0x7632),
                           __byte_perm(v[k].y, v[k].w, 0x5410), __byte_perm(v[k].y, v[k].w, 0x7632));
      }
      fence_proxy_async_smem();
      warp_arrive(bar(W::kQFull));
      return true;
    };
    WideUnit u;
    while (ok && walk.next(a, u)) {
      if (!W::kQTmem && is_v && !(ok = put_q(u))) break;
      const int n = u.n, len = u.len, prefix = len - u.count;
      uint32_t* bad = reinterpret_cast<uint32_t*>(smem + W::kBad) + (units & 3) * W::kGroups * 4;
      for (int j = W::kTeams == 2 ? (tile0 ^ team) & 1 : 0; j < n; j += W::kTeams) {
        const uint32_t item = item0 + wide_item(is_v, j, n), s = item % W::kItems;
        const int tok0 = (u.p0 + n - 1 - j) * kTok;
        const uint32_t rs = is_v * W::kRaws + slot, raw = sbase + W::kRawRing + rs * W::kRaw, to = sbase + W::kValues + s * W::kItem;
        if (!(ok = warp_nap(bar(W::kRawFull + rs), raw_uses & 1, err, kErrTimeoutTma))) break;
        // the item four in front has been taken
        if (item >= W::kItems && !(ok = warp_nap(bar(W::kEmpty + s), (item / W::kItems - 1) & 1, err, kErrTimeoutMma))) break;
        const uint32_t have = *reinterpret_cast<volatile uint32_t*>(smem + W::kHave + 4 * rs);
        if (!is_v && t == 0) {
          // runs in front of the sequence's end without a page
          const int some = min(runs, (len - tok0 + run - 1) / run);
          *reinterpret_cast<volatile uint32_t*>(smem + W::kGone + 4 * ((tile0 + j) & 3)) = ~have & ((1u << some) - 1u);
        }
        const bool edge = tok0 + kTok > prefix || have != (1u << runs) - 1u;
#pragma unroll 1
        for (int half = 0; half < kTimes; ++half) {
          uint32_t w[kPer][4], par[kPer];
#pragma unroll
          for (int k = 0; k < kPer; ++k) {
            const uint32_t i = t + (half * kPer + k) * 32 * W::kTeam;
            ld_shared_v4(raw + 16 * i, w[k][0], w[k][1], w[k][2], w[k][3]);
            asm volatile("ld.shared.b32 %0, [%1];" : "=r"(par[k]) : "r"(raw + kTok * W::kRow + 4 * i));
          }
          if (half == kTimes - 1) warp_arrive(bar(W::kRawEmpty + rs));
          // tokens that are not there stand for zeros, whatever the slot holds; so do drafted values
          // that are not finite, which are noted
          if (edge) {
#pragma unroll
            for (int k = 0; k < kPer; ++k) {
              const int in = r + (half * kPer + k) * kRows, tok = tok0 + in;
              if (tok >= len || !((have >> (in / run)) & 1u)) {
                par[k] = 0;
              } else if (is_v && tok >= prefix && not_finite<BF16>(par[k])) {
                par[k] = 0;
                atomicOr(bad + g * 4 + ((tok - prefix) >> 5), 1u << ((tok - prefix) & 31));
              }
            }
          }
          const uint32_t at = to + half * kPer * kRows * 128;
#pragma unroll
          for (int k = 0; k < kPer; ++k) {
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
            const Unpack<BF16> unpack(__byte_perm(par[k], par[k], 0x1010), __byte_perm(par[k], par[k], 0x3232));
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              uint32_t v[4];
              unpack(w[k][c], v);
              st_shared_v4(at + column[c] + k * kRows * 128, v[0], v[1], v[2], v[3]);
            }
          }
        }
        fence_proxy_async_smem();
        // A team's next item is three to five behind this one, and the place of one five behind has one
        // three in front of this.  That has to have been taken when the next asks for the place, or the
        // parity that it asks for could be two phases old; here, in front of this item's arrival, the one
        // five behind this cannot have been there, so that this parity cannot be either.
        if (W::kTeams == 2 && j + 2 >= n && item >= 3 &&
            !(ok = warp_nap(bar(W::kEmpty + (item + 1) % W::kItems), ((item - 3) / W::kItems) & 1, err, kErrTimeoutMma)))
          break;
        warp_arrive(bar(W::kFull + s));
        if ((slot += W::kTeams) >= (uint32_t)W::kRaws) slot -= W::kRaws, ++raw_uses;
      }
      if (!ok) break;
      tile0 += n;
      item0 += 2 * n;
      ++units;
    }
  } else {
    // ------------------------------------------------------------ softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(W::kRegsSoftmax));
    const int wg = warp >> 2, chain = W::kChains == 2 ? wg : 0, side = W::kSides == 2 ? wg : 0;
    const int r = ((warp & 3) << 5) + lane;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const bool cap = RULE && a.cap, bias = RULE && a.rule.slopes != nullptr;
    const float scale2 = a.scale_log2 * (BF16 ? kScaledBack : 1.f);
    const float c = bias ? 1.f : cap ? a.rule.cap2 : scale2;  // from what the maximum works on to base 2
    float2* const ml = reinterpret_cast<float2*>(smem + W::kMl);
    float* const add = reinterpret_cast<float*>(smem + W::kAdd) + wg * W::kAddCh * 96;
    float* const maxima = reinterpret_cast<float*>(smem + W::kMax);
    constexpr int kSide = D / 2;  // channels that a warpgroup writes
    uint32_t o_uses = 0, units = 0, tile0 = 0;   // tiles of the chain, units, all tiles of those
    uint32_t parity = 0;                         // bit b: of score buffer b's next tile

    // Q of unit w into tensor memory: this warpgroup's channels of each row
    auto put_q = [&](const WideUnit& w) {
      if constexpr (W::kQTmem) {
        const WideRow x = wide_row<W::kCopies>(min(a.group * w.count - w.row0, kWideRows), r);
        const uint4* q = nullptr;
        if (x.row < x.rows) {
          int hh, qi;
          w.split(w.row0 + x.row, hh, qi);
          q = reinterpret_cast<const uint4*>(a.q) +
              ((((size_t)w.b * a.H + (size_t)w.h_kv * a.group + hh) * a.N_q + qi) * D + wg * kSide) / 8;
        }
#pragma unroll
        for (int h = 0; h < kSide; h += 32) {
          uint32_t y[16];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint4 v = q ? q[h / 8 + i] : make_uint4(0, 0, 0, 0);
            y[4 * i] = __byte_perm(v.x, v.z, 0x5410), y[4 * i + 1] = __byte_perm(v.x, v.z, 0x7632);
            y[4 * i + 2] = __byte_perm(v.y, v.w, 0x5410), y[4 * i + 3] = __byte_perm(v.y, v.w, 0x7632);
          }
          tmem_st_32x32b_x16(tmem + lanes + W::kQCol + (wg * kSide + h) / 2, y);
        }
        tmem_wait_st();
        tc_fence_before();
        warp_arrive(bar(W::kQFull));
      }
    };

    WideUnit next;
    bool more = walk.next(a, next);
    if (more) put_q(next);
    // (a warp whose wait gave up goes on to the end without waiting, for the others' named barriers)
    while (more) {
      const WideUnit u = next;
      const int n = u.n, len = u.len, count = u.count, prefix = len - count, h_kv = u.h_kv;
      const WideRow w = wide_row<W::kCopies>(min(a.group * count - u.row0, kWideRows), r);
      const int each = kWideRows / w.copies;
      const bool has = w.row < w.rows;
      int hh, qi;
      u.split(has ? u.row0 + w.row : 0, hh, qi);
      uint64_t see[2] = {0, 0};
      const int depth = has ? tree_row(a, u.b, count, prefix, qi, see) : -1;
      const float slope2 = bias && has ? rule_slope2(a.rule, h_kv * a.group + hh) : 0.f;
      float m = -INFINITY, l = 0.f;

      // A tile: this copy's scores, `part` from column c0 on, in chunks of C.  Two chunks are read a
      // second time for the exponentials, as a thread has no room for them; P lies under scores that have
      // been read by then.
      auto tile = [&](auto size, auto chunks, int j, uint32_t missing) {
        constexpr int C = decltype(size)::value, part = C * decltype(chunks)::value;
        constexpr bool kAgain = part > C;
        const int buf = j & 1, tok0 = (u.p0 + n - 1 - j) * kTok, c0 = (w.copy * W::kSides + side) * part;
        const uint32_t tS = tmem + lanes + W::s_col(buf);
        const bool edge = tok0 + kTok > prefix || missing, changed = cap || bias || edge;
        float s[C];
        auto load = [&](int h) {
          constexpr int kLoad = C < 32 ? C : 32;
          uint32_t x[C / kLoad][kLoad];
#pragma unroll
          for (int k = 0; k < C / kLoad; ++k) {
            if constexpr (kLoad == 32) tmem_ld_32x32b_x32(tS + c0 + h + 32 * k, x[k]);
            else tmem_ld_32x32b_x16(tS + c0 + h, x[k]);
          }
          tmem_wait_ld();
#pragma unroll
          for (int k = 0; k < C / kLoad; ++k) reg_fence(x[k]);
#pragma unroll
          for (int i = 0; i < C; ++i) s[i] = __uint_as_float(x[i / kLoad][i % kLoad]);
        };
        // what the softmax works on: the cap's tanh, base 2 with a bias, -inf where hidden
        auto rules = [&](int h) {
          if (cap) {
            if constexpr (BF16) {
#pragma unroll
              for (int i = 0; i < C; ++i) s[i] *= kScaledBack;
            }
            rule_tanh<C, true>(s, a.rule);
          }
          const int dj = tok0 + c0 + h - prefix;  // the first score's token, counted from the prefix's end
          if (bias) {
            const float mul2 = cap ? a.rule.cap2 : scale2;
            if (dj + C <= 0) {
              // Tokens of the prefix lie in front of every row.  Integers first: positions past 2^24 are not
              // exact in fp32.  What is lost of a far token's bias, 2^-24 of it, is lost of a score far
              // below the others.
              const float base = -slope2 * (float)(depth - dj);
#pragma unroll
              for (int i = 0; i < C; i += 2) {
                float b0, b1;
                fma2((float)i, (float)(i + 1), slope2, base, b0, b1);
                fma2v(s[i], s[i + 1], mul2, b0, b1, s[i], s[i + 1]);
              }
            } else {
              // a drafted token that this row sees is as deep as it has ancestors, which the row sees too
              int deep = dj <= 0 ? 0 : __popcll(dj < 64 ? see[0] & ((1ull << dj) - 1) : see[0]) +
                                           (dj <= 64 ? 0 : __popcll(see[1] & (dj < 128 ? (1ull << (dj - 64)) - 1 : ~0ull)));
              const uint64_t up = tree_window(see, dj);
#pragma unroll
              for (int i = 0; i < C; ++i) {
                const bool drafted = dj + i >= 0;
                const int away = depth - (drafted ? deep : dj + i);
                if (drafted && ((up >> i) & 1u)) ++deep;
                s[i] = fmaf(-slope2, fabsf((float)away), s[i] * mul2);
              }
            }
          }
          if (edge) {
            uint64_t win = tree_window(see, dj);
            if (missing)
#pragma unroll 1
              for (int i = 0; i < C; ++i)
                if ((missing >> ((c0 + h + i) / run)) & 1u) win &= ~(1ull << i);
#pragma unroll
            for (int i = 0; i < C; ++i)
              if (!((win >> i) & 1u)) s[i] = -INFINITY;
          }
        };
        auto put = [](uint32_t at, const uint32_t (&x)[C / 2]) {
          if constexpr (C == 64) tmem_st_32x32b_x32(at, x);
          else if constexpr (C == 32) tmem_st_32x32b_x16(at, x);
          else tmem_st_32x32b_x8(at, x);
        };
        float top = m;
#pragma unroll 1
        for (int h = 0; h < part; h += C) {
          load(h);
          if (changed) {
            rules(h);
            if constexpr (kAgain) {
#pragma unroll
              for (int k = 0; k < C; k += 32) {
                uint32_t y[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) y[i] = __float_as_uint(s[k + i]);
                tmem_st_32x32b_x32(tS + c0 + h + k, y);
              }
            }
          }
          float x0 = fmaxf(s[0], s[1]), x1 = fmaxf(s[2], s[3]);
#pragma unroll
          for (int i = 4; i < C; i += 4) x0 = max3f(x0, s[i], s[i + 1]), x1 = max3f(x1, s[i + 2], s[i + 3]);
          top = max3f(top, x0, x1);
        }
        if (kAgain && changed) tmem_wait_st();
        if constexpr (W::kSides == 2) {
          // the row's other half; behind the barrier of the two warps both have their scores
          float* mx = maxima + (o_uses & 1) * 2 * kWideRows;
          mx[side * kWideRows + r] = top;
          tc_fence_before();
          named_bar_sync(4 + (warp & 3), 64);
          tc_fence_after();
          top = fmaxf(top, mx[(side ^ 1) * kWideRows + r]);
        }
        // the reference follows when the maximum is over 8 above it (base 2)
        const bool moved = m == -INFINITY ? top != m : (top - m) * c > 8.f;
        const float m_use = moved ? top : m;
        const float mc = m_use == -INFINITY ? 0.f : m_use * c;
        // (2^(m c - m c) by a fused multiply-add would not be 1)
        const float alpha = moved ? ex2_approx(fmaf(m, c, -mc)) : 1.f;
        m = m_use;
        float l0 = 0.f, l1 = 0.f;
#pragma unroll 1
        for (int h = 0; h < part; h += C) {
          if constexpr (kAgain) load(h);
          uint32_t pw[C / 2];
#pragma unroll
          for (int i = 0; i < C; i += 2) {
            float x0, x1;
            fma2(s[i], s[i + 1], c, -mc, x0, x1);
            const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
            add2(l0, l1, p0, p1);
            pw[i >> 1] = pack2<BF16>(p0, p1);
          }
          put(tS + (c0 + h) / 2, pw);
        }
        l = l * alpha + (l0 + l1);
        // the other copies' tokens are not this row's
        if constexpr (part * W::kSides < kTok) {
          const uint32_t zero[C / 2] = {};
#pragma unroll
          for (int k = 0; k < kTok / (part * W::kSides); ++k)
            if (k != w.copy) put(tS + (k * W::kSides + side) * part / 2, zero);
        }
        tmem_wait_st();
        if (j >= W::kChains && __any_sync(0xffffffffu, moved)) {
          // With two chains the chain's last product is done: this tile's scores came behind it.  With
          // one, the product before that one is, so the parity is not two phases old.
          if constexpr (W::kChains == 1) ok = ok && warp_nap(bar(W::kODone), (o_uses - 1) & 1, err, kErrTimeoutMma);
          tc_fence_after();
#pragma unroll 1
          for (int ch = 0; ch < D / 32 / W::kSides; ++ch) {
            uint32_t o[32];
            const uint32_t at = tmem + lanes + W::o_col(chain) + side * (D / 2) + 32 * ch;
            tmem_ld_32x32b_x32(at, o);
            tmem_wait_ld();
            reg_fence32(o);
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
            tmem_st_32x32b_x32(at, o);
          }
          tmem_wait_st();
        }
      };
      auto tiles = [&](auto size, auto chunks) {
        for (int j = chain; j < n; j += W::kChains, ++o_uses) {
          const int buf = j & 1;
          ok = ok && warp_nap(bar(W::kSFull + buf), (parity >> buf) & 1, err, kErrTimeoutMma);
          parity ^= 1u << buf;
          tc_fence_after();
          if (w.warp_live) tile(size, chunks, j, *reinterpret_cast<volatile uint32_t*>(smem + W::kGone + 4 * ((tile0 + j) & 3)));
          tc_fence_before();
          warp_arrive(bar(W::kPFull + buf));
        }
      };
      constexpr std::integral_constant<int, 1> kOne{};
      if constexpr (W::kSides == 2) {
        if (w.copies == 2) tiles(std::integral_constant<int, kTok / 4>{}, kOne);
        else tiles(std::integral_constant<int, kTok / 2>{}, kOne);
      } else {
        if (w.copies == 4) tiles(std::integral_constant<int, kTok / 4>{}, kOne);
        else if (w.copies == 2) tiles(std::integral_constant<int, kTok / 2>{}, kOne);
        else tiles(std::integral_constant<int, kTok / 2>{}, std::integral_constant<int, 2>{});
      }
      tile0 += n;
      more = walk.next(a, next);
      if constexpr (W::kQTmem) {
        // the next unit's Q, when the score products of this one are done
        if (more) {
          ok = ok && warp_nap(bar(W::kQEmpty), units & 1, err, kErrTimeoutMma);
          put_q(next);
        }
      }

      // ---- the unit's end: chains and copies joined, rows or parts written
      ok = ok && warp_nap(bar(W::kUnitDone), units & 1, err, kErrTimeoutMma);
      tc_fence_after();
      ml[(w.copy * 2 + wg) * each + w.row] = make_float2(m, l);
      named_bar_sync(1, 256);
      // a whole unit's copies are joined here; a part's go as they are
      const int k0 = u.whole ? 0 : 2 * w.copy, k1 = u.whole ? 2 * w.copies : k0 + 2;
      float mm = -INFINITY, ll = 0.f, f[2] = {0.f, 0.f};
      for (int k = k0; k < k1; ++k) mm = fmaxf(mm, ml[k * each + w.row].x);
      for (int k = k0; k < k1; ++k) {
        const float2 x = ml[k * each + w.row];
        const float y = mm == -INFINITY ? 0.f : ex2_approx((x.x - mm) * c);
        ll = fmaf(y, x.y, ll);
        if (k == w.copy * 2) f[0] = y;  // (halves of a row's scores have one maximum)
        if (k == w.copy * 2 + 1) f[1] = y;
      }
      if (depth < 0) mm = -INFINITY, ll = 0.f;
      const float m2 = mm == -INFINITY ? mm : mm * c;  // base 2
      const bool live = depth >= 0, writes = has && ok && (w.copy == 0 || !u.whole);
      const size_t slot = blockIdx.x + (u.p0 == 0 ? kWideMaxCtas : 0);
      const size_t out = ((size_t)u.b * a.H + (size_t)h_kv * a.group + hh) * a.N_q + qi;
      const float inv = (u.whole ? (ll > 0.f ? 1.f / ll : 0.f) : 1.f) * (BF16 ? kScaledBack : 1.f);
      uint32_t* bad = reinterpret_cast<uint32_t*>(smem + W::kBad) + (units & 3) * W::kGroups * 4;
      // (pieces of 16 channels: a short loop, as code that runs once a unit comes from far)
#pragma unroll 1
      for (int ch = wg * kSide; ch < (wg + 1) * kSide; ch += 16) {
        uint32_t x[16];
        float o[16];
        tmem_ld_32x32b_x16(tmem + lanes + W::o_col(0) + ch, x);
        tmem_wait_ld();
        reg_fence(x);
#pragma unroll
        for (int i = 0; i < 16; ++i) o[i] = __uint_as_float(x[i]) * f[0];
        if (W::kChains == 2 && n > 1) {
          tmem_ld_32x32b_x16(tmem + lanes + W::o_col(1) + ch, x);
          tmem_wait_ld();
          reg_fence(x);
#pragma unroll
          for (int i = 0; i < 16; ++i) o[i] = fmaf(__uint_as_float(x[i]), f[1], o[i]);
        }
        if (u.whole && w.copies > 1) {
          if (w.copy > 0)
#pragma unroll
            for (int i = 0; i < 16; ++i) add[i * 96 + r - each] = o[i];
          named_bar_sync(2 + wg, 128);
          if (w.copy == 0)
#pragma unroll 1
            for (int k = 0; k < kWideRows - each; k += each)
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] += add[i * 96 + r + k];
          named_bar_sync(2 + wg, 128);
        }
        if (!writes) continue;
        // a drafted value that is not finite, in this group of channels, of a token that the row sees
        const uint32_t* bg = bad + 4 * (ch / kKv4Group);
        const bool nan = ((uint32_t)see[0] & bg[0]) | ((uint32_t)(see[0] >> 32) & bg[1]) | ((uint32_t)see[1] & bg[2]) |
                         ((uint32_t)(see[1] >> 32) & bg[3]);
        const float times = live ? inv : 0.f, plus = nan ? NAN : 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) o[i] = live ? fmaf(o[i], times, plus) : 0.f;
        if (u.whole) {
#pragma unroll
          for (int q = 0; q < 16; q += 8)  // channels 0 4 1 5 2 6 3 7
            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.o) + out * D + ch + q) =
                make_uint4(pack2<BF16>(o[q], o[q + 2]), pack2<BF16>(o[q + 4], o[q + 6]), pack2<BF16>(o[q + 1], o[q + 3]),
                           pack2<BF16>(o[q + 5], o[q + 7]));
        } else {
          float* part = a.part_o + slot * (kWideRows * D) + (size_t)ch * kWideRows + r;
#pragma unroll
          for (int i = 0; i < 16; ++i) part[i * kWideRows] = o[i];
        }
      }
      if (writes && wg == 0) {
        if (!u.whole)
          *reinterpret_cast<float2*>(a.part_ml + (slot * kWideRows + r) * 2) = make_float2(m2, ll);
        else
          a.lse[out] = ll == 0.f ? -INFINITY : m2 * kLn2 + logf(ll);
      }
      tc_fence_before();
      // Both chains' O, (m, l) and notes have been read: products may write them again, and the notes
      // are cleared for the unit four on.
      named_bar_sync(1, 256);
      if (threadIdx.x < W::kGroups * 4) bad[threadIdx.x] = 0;
      ++units;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == W::kWarpIssue) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  } else if (warp == W::kWarpLoad) {
    // after a wait that gave up: every copy that was asked for lands before the CTA ends
    for (int s = 0; s < 2 * W::kRaws; ++s) {
      const uint32_t uses = *reinterpret_cast<volatile uint32_t*>(smem + W::kAsked + 4 * s);
      if (uses > 0) warp_wait_all(bar(W::kRawFull + s), (uses - 1) & 1, err);
    }
  }
}

// Joins the parts of the units that several CTAs did, in CTA order.  Every such unit is cut where a
// CTA's stretch begins; the first of its cuts does it.  A block: kWideJoin channels of 128 rows,
// whose parts are shared by kWideShare threads a row: two, as most units have two or three CTAs and the
// blocks of four threads a row come in four waves (8 sequences of up to 2000 tokens, d 256, 128 rows: 64 us
// with four, 59 with two, 57 with one; but one of 16000 42, 43 and 50).  Maximum and sums run along in one
// pass, so that a part's loads wait for nothing (the last 43 then 40).
constexpr int kWideJoin = 8, kWideShare = 2;
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
  const int c1 = wide_cta_of(first + (cut.len - 1) / Wide<D>::kTok, cut.total, G);
  const int r = threadIdx.x % kWideRows, share = threadIdx.x / kWideRows, left = a.group * cut.count - cut.row0;
  const int copies = wide_row<Wide<D>::kCopies>(min(left, kWideRows), r).copies, each = kWideRows / copies;
  float mm = -INFINITY, ll = 0.f, acc[kWideJoin];
#pragma unroll
  for (int i = 0; i < kWideJoin; ++i) acc[i] = 0.f;
  // the row's parts: CTA after CTA, in each copy after copy
  auto at = [&](int k) { return (size_t)(c0 + k / copies + (k < copies ? kWideMaxCtas : 0)) * kWideRows; };
  auto lane_of = [&](int k) { return k % copies * each + r; };
  const int parts = r < each && r < left ? (c1 - c0 + 1) * copies : 0;
#pragma unroll 4
  for (int k = share; k < parts; k += kWideShare) {
    const float2 ml = *reinterpret_cast<const float2*>(a.part_ml + (at(k) + lane_of(k)) * 2);
    const float* p = a.part_o + at(k) * D + (size_t)part * kWideJoin * kWideRows + lane_of(k);
    float x[kWideJoin];
#pragma unroll
    for (int i = 0; i < kWideJoin; ++i) x[i] = p[i * kWideRows];
    const float top = fmaxf(mm, ml.x), ref = top == -INFINITY ? 0.f : top;
    const float f = ex2_approx(ml.x - ref), g = ex2_approx(mm - ref);
    mm = top;
    ll = fmaf(f, ml.y, ll * g);
#pragma unroll
    for (int i = 0; i < kWideJoin; ++i) acc[i] = fmaf(f, x[i], acc[i] * g);
  }
#pragma unroll
  for (int i = 0; i < kWideJoin; ++i) acc_of[share][i][r] = acc[i];
  ml_of[share][r] = make_float2(mm, ll);
  __syncthreads();
  const int col = cut.row0 + r;
  if (share > 0 || parts == 0) return;
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
  const int hh = col / cut.count, qi = col - hh * cut.count;
  const size_t out = ((size_t)cut.b * a.H + (size_t)cut.h_kv * a.group + hh) * a.N_q + qi;
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
  auto kern = a.cap || a.rule.slopes ? kv4_wide_kernel<D, BF16, true> : kv4_wide_kernel<D, BF16, false>;
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
