// A few new query rows of each sequence attending over its paged 4-bit cache.
//
// What bounds it is the cache: d / 2 + d / 8 bytes per token, for keys and values, read
// once per key/value head and tile of columns: the query heads of a group and the query rows
// share that read as the columns of one product, up to 16 of them (32 at d 64); more columns
// are further tiles, each of which reads the codes again (32 sequences of 8192 tokens, 8 heads
// of 8, d 128: 104 us with 16 columns, 190 with 32).  With so few columns the products are
// narrow: the tokens (for S^T = K Q^T) and the channels (for O^T = V^T P^T) are the rows of
// mma.sync m16n8k16, which takes its 16-row operand from registers, where the codes are turned
// into values anyway.  (tcgen05 would want the values written to shared or tensor memory
// first, 128 rows at a time.)
//
// The contraction index of a product may be permuted as long as both operands agree, so no
// code is moved between threads.  With g = lane / 4 and t = lane % 4:
//   S^T: row g of 8 tokens is token g / 2 + 4 (g % 2), and the thread takes the t-th quarter
//        of its channels (one 16-byte load at d = 128), which lies in one group of 32: one
//        (scale, low) pair.  Q is laid out in shared memory in the same order.
//   O^T: the thread takes d / 8 channels (a row's g-th eighth) of tokens t, t + 4, t + 8, t + 12;
//        one byte permutation puts two tokens' codes side by side, as the operand wants them.
// Codes become 16-bit values (fa_kv4.cuh) by one fused multiply-add with (scale, low): the
// value that the cache's definition gives, rounded once.  P is rounded to 16 bits as in the
// other kernels; scores, maxima, sums and O stay in fp32.
//
// Work: units of (sequence, key/value head, tile of columns), cut into pieces of 256 (or 128)
// tokens, 64 (or 32) a warp; which of the two, and whether clusters do the units, goes by the
// tokens that the page table has room for (launch_n).
// The pieces of all units in one row are dealt to the CTAs in equal stretches, whatever
// the lengths (which only the device knows), so a long sequence is spread over many CTAs
// and short ones share one.  A unit that one CTA does alone is written by it; the others
// leave (m, l, O) per CTA, and a second kernel joins them in CTA order, so results do not
// depend on timing.  Each of the 4 warps runs its own softmax over its tokens of every
// piece; they meet at the end of a unit only.  A tile's keys and values come by bulk copies
// into one slot each (two copies for each run of a page, by one lane a run): the next
// tile's keys are asked for when this tile's have been read, while its values are being
// worked on, and the other way round.  Short sequences take one launch: a cluster of CTAs
// does a unit and joins it through its shared memories.
//
// Measured: 32 sequences of up to 16384 tokens, 32 query heads on 8, d 128, bf16: 82 us for 382
// MB (4.6 TB/s, 69 % of a copy's rate; fp16, whose values take 13 instructions for 8 and not 9,
// 92 us), 64 sequences 157 us (75 %), at d 64 with 64 heads on 8 58 us (49 %); three rows of two
// sequences of up to 100003 tokens, 16 heads on 4, d 256: 80 us (39 %), where 16 columns of O
// take 128 registers a thread and leave 8 warps an SM.  Without its products the first case
// takes 71 us: about 9 us of start, ends of units and join, and 62 at 90 % of a copy's rate.
// What is between is the unpacking, 9 instructions for 8 values on half-rate pipes (ALU 48 %
// busy, 2.3 instructions a clock).
#pragma once
#include <algorithm>
#include <climits>
#include <type_traits>

#include "fa_kv4.cuh"
#include "fa_kv4.h"
#include "fa_kv4_tree.cuh"
#include "fa_rule.cuh"
#include "ptx.cuh"

namespace fa {
namespace {

constexpr int kWarps = 4;

// TOK: tokens of a warp's tile.  64 amortise a tile's waits, votes and lookups best, but
// with few tokens in all, 32 give work to more CTAs, and at d 256 O leaves registers for 32
// only (launch_n).
template <int D, int TOK>
struct Cfg {
  static constexpr int kTok = TOK;
  static constexpr int kMt = kTok / 16;            // row tiles of a product
  static constexpr int kPiece = kWarps * kTok;     // tokens of a piece
  static constexpr int kRow = D / 2;                 // bytes of a row's codes
  static constexpr int kGroups = D / kKv4Group;
  static constexpr int kPar = 4 * kGroups;           // bytes of a row's parameters
  static constexpr int kKWords = D / 32;             // words of codes a thread takes of a key row
  static constexpr int kVWords = D / 64;             // words a thread takes of a value row
  static constexpr int kSlotBytes = kTok * (kRow + kPar);  // a tile's keys, or its values
};
// As many as the registers of a thread's O and scores allow (measured with one less: d 64,
// 8 columns 57.8 against 59.4 us, d 256, 8 columns 54.3 against 57.2).
constexpr int ctas_per_sm(int d, int nt) { return nt * d <= 64 ? 4 : nt * d <= 128 || nt == 1 ? 3 : 2; }

template <int D, int NT, int TOK, bool TREE>
struct Smem {
  static constexpr int kCols = 8 * NT;
  static constexpr int kQ = 0;                                   // Q as operand fragments
  static constexpr int kQBytes = D * kCols * 2;
  static constexpr int kRing = kQ + kQBytes;
  static constexpr int kRingBytes = kWarps * 2 * Cfg<D, TOK>::kSlotBytes;
  // the join of the warps reuses the slots: O [warps][D][cols] (order below) and (m, l)
  static constexpr int kJoin = kWarps * kCols * (D + 2) * 4;
  static constexpr int kBar = kRing + (kRingBytes > kJoin ? kRingBytes : kJoin);
  static constexpr int kTree = kBar + 8 * kWarps * 2;            // a unit's tree
  static constexpr int kCum = kTree + (TREE ? (int)sizeof(TreeRows) : 0);
  static int bytes(int B) { return kCum + 4 * (B + 1); }
};

__device__ __forceinline__ void mma16816(bool bf16, float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  if (bf16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(a));
  return r;
}
template <int W>
__device__ __forceinline__ void lds_words(uint32_t addr, uint32_t (&w)[W]) {
  if constexpr (W == 1)
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w[0]) : "r"(addr));
  else if constexpr (W == 2)
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr));
  else {
#pragma unroll
    for (int i = 0; i < W; i += 4)
      asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(w[i]), "=r"(w[i + 1]), "=r"(w[i + 2]), "=r"(w[i + 3])
                   : "r"(addr + 64 * (i / 4)));  // d = 256: the second 16 bytes lie 64 further
  }
}

// The values a product takes, and what it is multiplied with afterwards: bf16 values come
// times 2^-32.
template <bool BF16>
__device__ __forceinline__ void tile_values(uint32_t x, uint32_t s2, uint32_t l2, uint32_t (&v)[4]) {
  if constexpr (BF16)
    values4_scaled(x, Scaled(s2, l2), v);
  else
    values4<false>(x, s2, l2, v);
}
template <bool BF16>
constexpr float kTileBack = BF16 ? kScaledBack : 1.f;

// Pieces of a sequence, per unit of it.
template <int PIECE>
__device__ __forceinline__ int pieces_of(const Kv4AttendArgs& a, int b) {
  const long long room = (long long)a.pool.max_pages << a.pool.page_shift;
  const long long n = min((long long)max(a.lengths[b], 0), room);
  return (int)((n + PIECE - 1) / PIECE);
}
// cum[b] = pieces of all units of the sequences before b, for b = 0..B; every thread of the
// block calls it (64 * 32 threads at most).
template <int PIECE>
__device__ void scan_pieces(const Kv4AttendArgs& a, int* cum) {
  __shared__ int warp_sum[32];
  const int per = (a.B + blockDim.x - 1) / blockDim.x, b0 = threadIdx.x * per;
  const int units = a.pool.H_kv * a.col_tiles;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int mine = 0;
  for (int i = 0; i < per; ++i)
    if (b0 + i < a.B) mine += pieces_of<PIECE>(a, b0 + i) * units;
  int x = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, off);
    if (lane >= off) x += y;
  }
  if (lane == 31) warp_sum[warp] = x;
  __syncthreads();
  int at = x - mine;
  for (int w = 0; w < warp; ++w) at += warp_sum[w];
  for (int i = 0; i < per; ++i)
    if (b0 + i < a.B) {
      cum[b0 + i] = at;
      at += pieces_of<PIECE>(a, b0 + i) * units;
    }
  if (b0 < a.B && b0 + per >= a.B) cum[a.B] = at;
  __syncthreads();
}
// The CTA whose stretch [c T / G, (c + 1) T / G) holds piece x.
__device__ __forceinline__ int cta_of(int x, int T, int G) { return (int)((((long long)x + 1) * G - 1) / T); }

// Order of a unit's O, in shared memory and in the parts: element (r 8 + g) cols + col is
// channel g (D / 8) + r of column col.  A warp's accumulators are written and read in it
// without bank conflicts, and the parts without gaps.
template <int D>
__device__ __forceinline__ int channel_of(int e, int cols) {
  const int rg = e / cols;
  return (rg & 7) * (D / 8) + (rg >> 3);
}

// Where a unit's column lies in o and lse.
__device__ __forceinline__ size_t out_row(const Kv4AttendArgs& a, int b, int h_kv, int col) {
  const int hh = col / a.N_q, qi = col - hh * a.N_q;
  return ((size_t)b * a.H + (size_t)h_kv * a.group + hh) * a.N_q + qi;
}
template <bool BF16>
__device__ __forceinline__ void store16(void* o, size_t at, float x) {
  static_cast<uint16_t*>(o)[at] = (uint16_t)(pack2<BF16>(x, 0.f) & 0xFFFFu);
}

// L of a row from its reference and sum; -inf for one that sees nothing.  A NaN is a sum of
// NaN, whatever the reference is (a maximum passes NaN over).
__device__ __forceinline__ float lse_of(float m, float l) { return l == 0.f ? -INFINITY : m * kLn2 + logf(l); }

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\nbarrier.cluster.wait.acquire;" ::: "memory");
}
// A float of the CTA `rank` of the cluster, at the address `p` has in this CTA.
__device__ __forceinline__ float ld_cluster(const float* p, int rank) {
  uint32_t at;
  float v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
  return v;
}

// Joins the warps' O (jo) and (m, l) (jm) of the CTAs of a cluster, in the order of their
// ranks, and writes the unit.  Each CTA first leaves its own sums in warp 0's places.
template <int D, int NT, bool BF16>
__device__ __forceinline__ void join_cluster(const Kv4AttendArgs& a, float* jo, float* jm, int b, int h_kv, int col0) {
  constexpr int kCols = 8 * NT, kElems = kCols * D;
  const int col = threadIdx.x % kCols;  // the same for every element of the thread
  float mm = -INFINITY, ll = 0.f, f[kWarps];
#pragma unroll
  for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, jm[(w * kCols + col) * 2]);
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    f[w] = mm == -INFINITY ? 0.f : ex2_approx(jm[(w * kCols + col) * 2] - mm);
    ll += f[w] * jm[(w * kCols + col) * 2 + 1];
  }
#pragma unroll 4
  for (int e = threadIdx.x; e < kElems; e += 32 * kWarps) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) v += f[w] * jo[w * kElems + e];
    jo[e] = v;
  }
  __syncthreads();  // every thread has read the warps' (m, l)
  if (threadIdx.x < kCols) jm[2 * col] = mm, jm[2 * col + 1] = ll;
  cluster_sync();
  const int ctas = a.ctas, rank = blockIdx.x % ctas;
  float top = -INFINITY, sum = 0.f, g[kKv4MaxCluster];
#pragma unroll
  for (int k = 0; k < kKv4MaxCluster; ++k) {
    g[k] = k < ctas ? ld_cluster(jm + 2 * col, k) : -INFINITY;
    top = fmaxf(top, g[k]);
  }
#pragma unroll
  for (int k = 0; k < kKv4MaxCluster; ++k) {
    g[k] = g[k] == -INFINITY ? 0.f : ex2_approx(g[k] - top);
    if (k < ctas) sum = fmaf(g[k], ld_cluster(jm + 2 * col + 1, k), sum);
  }
  const bool live = col0 + col < a.cols;
  const size_t r = live ? out_row(a, b, h_kv, col0 + col) : 0;
  const float inv = sum > 0.f ? 1.f / sum : 0.f;
  // (1, 2, 4 or 8 CTAs: each takes a multiple of kCols elements, so a thread keeps its column)
  const int part = kElems / ctas;
  for (int e = rank * part + threadIdx.x; e < (rank + 1) * part; e += 32 * kWarps) {
    float v = 0.f;
#pragma unroll
    for (int k = 0; k < kKv4MaxCluster; ++k)
      if (k < ctas) v = fmaf(g[k], ld_cluster(jo + e, k), v);
    if (live) store16<BF16>(a.o, r * D + channel_of<D>(e, kCols), v * inv);
  }
  if (rank == 0 && threadIdx.x < kCols && live) a.lse[r] = lse_of(top, sum);
  cluster_sync();  // no CTA ends while another reads its shared memory
}

// CL: a cluster of a.ctas CTAs does one unit and joins it in shared memory.  Args: with a tree
// (Kv4TreeArgs) or without.
template <int D, int NT, int TOK, bool BF16, bool CL, class Args>
__global__ void __launch_bounds__(32 * kWarps, ctas_per_sm(D, NT)) kv4_attend_kernel(const Args a) {
  constexpr bool TREE = std::is_same_v<Args, Kv4TreeArgs>;
  using C = Cfg<D, TOK>;
  using S = Smem<D, NT, TOK, TREE>;
  constexpr int kTok = C::kTok, kMt = C::kMt, kPiece = C::kPiece, PIECE = kPiece;
  extern __shared__ __align__(128) uint8_t smem[];
  int* cum = reinterpret_cast<int*>(smem + S::kCum);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  // Token of a 16-token tile that a thread takes as row g: rows 2t and 2t + 1 are tokens t
  // and t + 4, so that the value rows which the threads t read together are neighbours
  // (84.7 to 82.5 us, a third of the bank conflicts gone).
  const int gk = (g >> 1) | ((g & 1) << 2);
  const uint32_t sbase = smem_u32(smem);
  const uint32_t slots = sbase + S::kRing + warp * 2 * C::kSlotBytes;  // keys, then values
  const uint32_t bars = sbase + S::kBar + 16 * warp;
  const Kv4Pool& pool = a.pool;

  if (lane < 2) mbar_init(bars + 8 * lane, 1);
  fence_mbar_init();
  grid_dep_wait();
  if (a.early) grid_dep_launch();
  int x = 0, x_end = 1, T = 0, G = 0;
  if constexpr (!CL) {
    scan_pieces<PIECE>(a, cum);  // (ends with a barrier of the CTA)
    T = cum[a.B];
    if (T == 0) return;
    G = min(a.ctas, T);
    if ((int)blockIdx.x >= G) return;
    x = (int)((long long)blockIdx.x * T / G);
    x_end = (int)(((long long)blockIdx.x + 1) * T / G);
  } else {
    __syncthreads();
  }
  const int run = min(kTok, 1 << pool.page_shift);  // tokens of a run: 16, 32 or 64
  int reads = 0;                                    // tiles this warp has taken
  int asked[2] = {0, 0};                            // tiles whose keys, values it has asked for
  bool ok = true;
  const float scale2 = a.scale_log2 * kTileBack<BF16>;  // from the products to base-2 scores

  while (x < x_end) {
    // ---- the unit that piece x belongs to, and this CTA's pieces of it
    int b, u_in, np, p0, p1;  // sequence, unit of it, the unit's pieces, this CTA's
    [[maybe_unused]] int u_begin = 0;
    if constexpr (CL) {
      const int unit = blockIdx.x / a.ctas, units_b = pool.H_kv * a.col_tiles, rank = blockIdx.x % a.ctas;
      b = unit / units_b;
      u_in = unit % units_b;
      np = pieces_of<PIECE>(a, b);
      p0 = rank * np / a.ctas;
      p1 = (rank + 1) * np / a.ctas;
    } else {
      int lo = 0, hi = a.B;  // the last b with cum[b] <= x
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cum[mid] <= x) lo = mid; else hi = mid;
      }
      b = lo;
      np = pieces_of<PIECE>(a, b);
      u_in = (x - cum[b]) / np;
      u_begin = cum[b] + u_in * np;
      p0 = x - u_begin;
      p1 = min(np, x_end - u_begin);
    }
    const int h_kv = u_in / a.col_tiles, ct = u_in % a.col_tiles;
    const int len = (int)min((long long)max(a.lengths[b], 0), (long long)pool.max_pages << pool.page_shift);
    const int col0 = ct * S::kCols;
    __syncthreads();  // the previous unit is done with Q and the rings

    // ---- copies: this warp's tokens of a piece.  A run's lane looks its page up (a tile
    // ahead, so that the table's latency is hidden) and asks for whole runs, which lie
    // inside the page whatever the length.
    const int32_t* table = pool.table + (size_t)b * pool.max_pages;
    auto page_of = [&](int p) -> int {  // -1: not asked for, -2: none
      const int tok = p * kPiece + warp * kTok + lane * run;
      if (p >= p1 || lane * run >= kTok || tok >= len) return -1;
      const int page = kv4_page(table, pool.num_pages, tok >> pool.page_shift);  // inside the table: len is
      return page < 0 ? -2 : page;
    };
    int page = page_of(p0), next_page = -1;  // of the tile whose copies are asked for now, and of the one behind
    auto load = [&](int p, int which) {      // keys (0), then values (1) of piece p
      if (p >= p1 || !ok) return;
      const uint32_t slot = slots + which * C::kSlotBytes, bar = bars + 8 * which;
      const int tok = p * kPiece + warp * kTok + lane * run;
      if (which == 0) {
        next_page = page_of(p + 1);
        if (page == -2) record_check(pool.err, kDbgPage, (uint32_t)tok);
      }
      const uint32_t have = __ballot_sync(0xffffffffu, page >= 0);
      if (lane == 0) mbar_expect_tx(bar, __popc(have) * run * (C::kRow + C::kPar));
      __syncwarp();
      if (page >= 0) {
        const size_t row = (((size_t)page * pool.H_kv + h_kv) << pool.page_shift) + (tok & ((1 << pool.page_shift) - 1));
        const uint32_t at = lane * run;
        bulk_load(slot + at * C::kRow, pool.codes[which] + row * C::kRow, run * C::kRow, bar);
        bulk_load(slot + kTok * C::kRow + at * C::kPar,
                  reinterpret_cast<const uint8_t*>(pool.params[which]) + row * C::kPar, run * C::kPar, bar);
      }
      if (which == 1) page = next_page;
      ++asked[which];
    };
    // zeroes the scale and low of tokens that are not there in a slot: the values are then
    // 0, whatever the slot holds
    auto blank = [&](int which, uint64_t gone) {
#pragma unroll
      for (int h = 0; h < kTok; h += 32)
        if ((gone >> (h + lane)) & 1u)
#pragma unroll
          for (int i = 0; i < C::kPar; i += 8)
            asm volatile("st.shared.v2.b32 [%0], {%1, %1};" ::"r"(slots + which * C::kSlotBytes + kTok * C::kRow +
                                                                   (h + lane) * C::kPar + i), "r"(0) : "memory");
      fence_proxy_async_smem();  // before the slot is copied to again
      __syncwarp();
    };
    uint32_t bad = 0;  // runs of the tile without a page
    auto note_bad = [&] { bad = ~__ballot_sync(0xffffffffu, page >= 0); };
    note_bad();
    load(p0, 0);
    load(p0, 1);
    [[maybe_unused]] int prefix = 0;
    [[maybe_unused]] TreeRows* const tree = reinterpret_cast<TreeRows*>(smem + S::kTree);
    if constexpr (TREE) {
      const int count = draft_count(a, b);
      prefix = len - count;
      tree_rows(a, b, count, prefix, *tree, threadIdx.x);
      static_assert(kKv4MaxDraft <= 32 * kWarps, "a thread a row");
    }

    // ---- Q as fragments: word j, pair m of channels, column n (kept in the order the
    // products read it: [j][nt][lane][4 x 16-bit pairs])
    for (int i = threadIdx.x; i < C::kKWords * NT * 32 * 4; i += 32 * kWarps) {
      const int m = i & 3, l = (i >> 2) & 31, nt = (i >> 7) % NT, j = (i >> 7) / NT;
      const int col = col0 + 8 * nt + (l >> 2);
      // channels of word j of quarter l % 4 of a key row (d = 256 takes two 16-byte parts)
      const int ch = D == 256 ? ((j >> 2) * 128 + (l & 3) * 32 + (j & 3) * 8) : ((l & 3) * (D / 4) + j * 8);
      uint32_t w = 0;
      if (col < a.cols) {
        const uint16_t* q = static_cast<const uint16_t*>(a.q) + out_row(a, b, h_kv, col) * D + ch;
        w = (uint32_t)q[m] | ((uint32_t)q[m + 4] << 16);
      }
      *reinterpret_cast<uint32_t*>(smem + S::kQ + 4 * i) = w;
    }
    if constexpr (TREE) __syncthreads();
    // this thread's columns: 8 nt + 2t and + 1 (those past the end are computed, not written)
    int last[NT][2];        // last key each column sees (with a tree: the column's row of it)
    int pos[NT][2];         // the column's position
    float slope2[NT][2], m[NT][2], mref[NT][2], l[NT][2];
    float o[C::kVWords][4][NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int col = col0 + 8 * nt + 2 * t + e;
        const int hh = col / a.N_q, qi = col - hh * a.N_q;
        if constexpr (TREE) {
          pos[nt][e] = prefix + tree->depth[qi];
          last[nt][e] = qi;  // the row of the tree
        } else {
          pos[nt][e] = len - a.N_q + qi;
          last[nt][e] = a.causal && col < a.cols ? pos[nt][e] : len - 1;
        }
        slope2[nt][e] = col < a.cols ? rule_slope2(a.rule, h_kv * a.group + hh) : 0.f;
        m[nt][e] = -INFINITY;
        mref[nt][e] = 0.f;
        l[nt][e] = 0.f;
#pragma unroll
        for (int w = 0; w < C::kVWords; ++w)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[w][i][nt][e] = o[w][i][nt][2 + e] = 0.f;
      }
    // last key that every column sees
    const int all_see = TREE ? prefix - 1 : a.causal ? len - a.N_q : len - 1;
    __syncthreads();

    for (int p = p0; p < p1; ++p) {
      // (a warp whose wait gave up takes part in the CTA's barriers to the end)
      if (!ok || !(ok = warp_wait(bars, reads & 1, pool.err, kErrTimeoutTma))) break;
      const uint32_t sKc = slots, sKp = sKc + kTok * C::kRow;
      const uint32_t sVc = slots + C::kSlotBytes, sVp = sVc + kTok * C::kRow;
      const int tok0 = p * kPiece + warp * kTok;
      if (tok0 >= len) {  // nothing of the piece, its unit's last, is this warp's
        if (!(ok = warp_wait(bars + 8, reads & 1, pool.err, kErrTimeoutTma))) break;
        ++reads;
        continue;
      }
      // tokens that are not there: behind the end, or of a run without a page
      uint64_t gone = 0;
      if (tok0 + kTok > len || (bad & ((1u << (kTok / run)) - 1u))) {
#pragma unroll
        for (int h = 0; h < kTok; h += 32) {
          const int in = h + lane;
          gone |= (uint64_t)__ballot_sync(0xffffffffu, tok0 + in >= len || ((bad >> (in / run)) & 1u)) << h;
        }
        blank(0, gone);
      }

      // ---- S^T = K Q^T
      float s[kMt][NT][4];
#pragma unroll
      for (int mt = 0; mt < kMt; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[mt][nt][e] = 0.f;
      // Two row tiles at a time: their products do not wait for each other.
#pragma unroll
      for (int mp = 0; mp < kMt; mp += 2) {
        constexpr int kPar = C::kKWords > 4 ? 2 : 1;
        uint32_t w[4][C::kKWords];
        uint32_t par[4][kPar];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int tok = 16 * mp + 8 * r + gk;
          lds_words(sKc + tok * C::kRow + t * (D == 256 ? 16 : C::kRow / 4), w[r]);
#pragma unroll
          for (int i = 0; i < kPar; ++i) {
            uint32_t pw[1];
            lds_words(sKp + tok * C::kPar + 4 * (D == 64 ? t / 2 : t + 4 * i), pw);
            par[r][i] = pw[0];
          }
        }
#pragma unroll
        for (int j = 0; j < C::kKWords; ++j) {
          uint32_t v[4][4];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const uint32_t pp = par[r][j >> 2];
            tile_values<BF16>(w[r][j], __byte_perm(pp, pp, 0x1010), __byte_perm(pp, pp, 0x3232), v[r]);
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            uint32_t q0, q1, q2, q3;
            ld_shared_v4(sbase + S::kQ + ((j * NT + nt) * 32 + lane) * 16, q0, q1, q2, q3);
            mma16816(BF16, s[mp][nt], v[0][0], v[1][0], v[0][1], v[1][1], q0, q1);
            mma16816(BF16, s[mp + 1][nt], v[2][0], v[3][0], v[2][1], v[3][1], q0, q1);
            mma16816(BF16, s[mp][nt], v[0][2], v[1][2], v[0][3], v[1][3], q2, q3);
            mma16816(BF16, s[mp + 1][nt], v[2][2], v[3][2], v[2][3], v[3][3], q2, q3);
          }
        }
      }

      // the keys have been read: the next tile's are asked for
      __syncwarp();
      load(p + 1, 0);

      // ---- scores to base 2, masks, the running maximum
      const bool edge = gone != 0 || tok0 + kTok - 1 > all_see;
      bool moved = false;
      float mx[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int mt = 0; mt < kMt; ++mt)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              float& y = s[mt][nt][2 * r + e];
              y = a.cap ? rule_tanh1(y * kTileBack<BF16>, a.rule) * a.rule.cap2 : y * scale2;
            }
          if (a.rule.slopes) {
            // integers first: positions past 2^24 are not exact in fp32, near distances are
            const float dist = (float)(pos[nt][e] - tok0 - gk);
            if (TREE && edge) {
              // a drafted token's position is its depth behind the prefix
#pragma unroll
              for (int mt = 0; mt < kMt; ++mt)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                  const int tok = tok0 + 16 * mt + 8 * r + gk;
                  const int at = tok < prefix ? tok : prefix + tree->depth[min(tok - prefix, a.N_q - 1)];
                  s[mt][nt][2 * r + e] = fmaf(-slope2[nt][e], fabsf((float)(pos[nt][e] - at)), s[mt][nt][2 * r + e]);
                }
            } else {
#pragma unroll
            for (int mt = 0; mt < kMt; ++mt)
#pragma unroll
              for (int r = 0; r < 2; ++r)
                s[mt][nt][2 * r + e] = fmaf(-slope2[nt][e], fabsf(dist - (float)(16 * mt + 8 * r)),
                                            s[mt][nt][2 * r + e]);
            }
          }
          if (TREE && edge) {
            const uint64_t win = tree_window(tree->see[last[nt][e]], tok0 - prefix) & ~gone;
#pragma unroll
            for (int mt = 0; mt < kMt; ++mt)
#pragma unroll
              for (int r = 0; r < 2; ++r)
                if (!((win >> (16 * mt + 8 * r + gk)) & 1)) s[mt][nt][2 * r + e] = -INFINITY;
          } else if (edge) {
#pragma unroll
            for (int mt = 0; mt < kMt; ++mt)
#pragma unroll
              for (int r = 0; r < 2; ++r) {
                const int in = 16 * mt + 8 * r + gk;
                if (tok0 + in > last[nt][e] || ((gone >> in) & 1)) s[mt][nt][2 * r + e] = -INFINITY;
              }
          }
          mx[nt][e] = fmaxf(s[0][nt][e], s[0][nt][2 + e]);
#pragma unroll
          for (int mt = 1; mt < kMt; ++mt) mx[nt][e] = max3f(mx[nt][e], s[mt][nt][e], s[mt][nt][2 + e]);
          moved |= mx[nt][e] > m[nt][e];
        }
      // the reference follows the maximum; O and the sums are rescaled only when it moves
      if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) mx[nt][e] = fmaxf(mx[nt][e], __shfl_xor_sync(0xffffffffu, mx[nt][e], off));
            const float mn = fmaxf(m[nt][e], mx[nt][e]);
            const float alpha = mn == -INFINITY ? 1.f : ex2_approx(m[nt][e] - mn);
            m[nt][e] = mn;
            mref[nt][e] = mn == -INFINITY ? 0.f : mn;
            l[nt][e] *= alpha;
#pragma unroll
            for (int w = 0; w < C::kVWords; ++w)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                o[w][i][nt][e] *= alpha;
                o[w][i][nt][2 + e] *= alpha;
              }
          }
      }
      uint32_t pb[kMt][NT][2];  // P^T as the 8-column operand: tokens 2t, 2t+1 (+8, +9) of column g
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int mt = 0; mt < kMt; ++mt)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float p0v = ex2_approx(s[mt][nt][2 * r] - mref[nt][0]);
            const float p1v = ex2_approx(s[mt][nt][2 * r + 1] - mref[nt][1]);
            l[nt][0] += p0v;
            l[nt][1] += p1v;
            pb[mt][nt][r] = transpose8x8(pack2<BF16>(p0v, p1v));
          }

      if (!(ok = warp_wait(bars + 8, reads & 1, pool.err, kErrTimeoutTma))) break;
      if (gone != 0) blank(1, gone);

      // ---- O^T += V^T P^T
      [[maybe_unused]] uint64_t bad_v = 0;  // drafted tokens with a value in this thread's channels that is not finite
#pragma unroll
      for (int mt = 0; mt < kMt; ++mt) {
        uint32_t w[4][C::kVWords], par[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int tok = 16 * mt + t + 4 * (r & 1) + 8 * (r >> 1);
          lds_words(sVc + tok * C::kRow + g * (C::kRow / 8), w[r]);
          uint32_t pw[1];
          lds_words(sVp + tok * C::kPar + 4 * (g * (D / 8) / kKv4Group), pw);
          par[r] = pw[0];
          if constexpr (TREE)
            if (edge && tok0 + tok >= prefix && not_finite<BF16>(pw[0])) {
              // 0 times it is not 0: left out here, and put in below where it is seen
              par[r] = 0;
              bad_v |= 1ull << tok;
            }
        }
        const uint32_t sA = __byte_perm(par[0], par[1], 0x5410), lA = __byte_perm(par[0], par[1], 0x7632);
        const uint32_t sB = __byte_perm(par[2], par[3], 0x5410), lB = __byte_perm(par[2], par[3], 0x7632);
#pragma unroll
        for (int j = 0; j < C::kVWords; ++j) {
#pragma unroll
          for (int half = 0; half < 2; ++half) {  // nibbles 0-3, then 4-7
            const uint32_t sel = half ? 0x7632 : 0x5410;
            uint32_t va[4], vb[4];
            tile_values<BF16>(__byte_perm(w[0][j], w[1][j], sel), sA, lA, va);
            tile_values<BF16>(__byte_perm(w[2][j], w[3][j], sel), sB, lB, vb);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              mma16816(BF16, o[j][2 * half][nt], va[0], va[1], vb[0], vb[1], pb[mt][nt][0], pb[mt][nt][1]);
              mma16816(BF16, o[j][2 * half + 1][nt], va[2], va[3], vb[2], vb[3], pb[mt][nt][0], pb[mt][nt][1]);
            }
          }
        }
      }
      if constexpr (TREE)
        if (edge) {
          bad_v |= __shfl_xor_sync(0xffffffffu, bad_v, 1);
          bad_v |= __shfl_xor_sync(0xffffffffu, bad_v, 2);
          if (bad_v)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 2; ++e)
                if (tree_window(tree->see[last[nt][e]], tok0 - prefix) & ~gone & bad_v)
#pragma unroll
                  for (int w = 0; w < C::kVWords; ++w)
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[w][i][nt][e] = o[w][i][nt][2 + e] = NAN;
        }
      ++reads;
      __syncwarp();  // the values have been read
      note_bad();
      load(p + 1, 1);
    }
    if constexpr (TREE) {
      // rows that are no token of the tree see nothing, whatever their queries hold
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          if (tree->depth[last[nt][e]] < 0) {
            m[nt][e] = -INFINITY;
            l[nt][e] = 0.f;
#pragma unroll
            for (int w = 0; w < C::kVWords; ++w)
#pragma unroll
              for (int i = 0; i < 4; ++i) o[w][i][nt][e] = o[w][i][nt][2 + e] = 0.f;
          }
    }
    // ---- join the warps: (m, l) and O through shared memory (the rings are free: every
    // tile asked for has been waited for)
    __syncthreads();
    float* jo = reinterpret_cast<float*>(smem + S::kRing);
    float* jm = jo + kWarps * S::kCols * D;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float sum = l[nt][e];
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        if (g == 0)
          *reinterpret_cast<float2*>(jm + (warp * S::kCols + 8 * nt + 2 * t + e) * 2) = make_float2(m[nt][e], sum);
      }
      float* dst = jo + warp * S::kCols * D + g * S::kCols + 8 * nt + 2 * t;
#pragma unroll
      for (int w = 0; w < C::kVWords; ++w)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          *reinterpret_cast<float2*>(dst + (8 * w + 2 * i) * 8 * S::kCols) =
              make_float2(o[w][i][nt][0] * kTileBack<BF16>, o[w][i][nt][1] * kTileBack<BF16>);
          *reinterpret_cast<float2*>(dst + (8 * w + 2 * i + 1) * 8 * S::kCols) =
              make_float2(o[w][i][nt][2] * kTileBack<BF16>, o[w][i][nt][3] * kTileBack<BF16>);
        }
    }
    __syncthreads();
    if constexpr (CL) {
      join_cluster<D, NT, BF16>(a, jo, jm, b, h_kv, col0);
      x = x_end;
      continue;
    }
    const bool whole = p0 == 0 && p1 == np;
    // a stretch cuts its first unit, whose first piece it does not have, and its last
    const size_t slot = blockIdx.x + (x == u_begin ? kKv4MaxCtas : 0);
    {
      const int col = threadIdx.x % S::kCols;  // the same for every element of the thread
      float mm = -INFINITY, ll = 0.f, f[kWarps];
#pragma unroll
      for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, jm[(w * S::kCols + col) * 2]);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        f[w] = mm == -INFINITY ? 0.f : ex2_approx(jm[(w * S::kCols + col) * 2] - mm);
        ll += f[w] * jm[(w * S::kCols + col) * 2 + 1];
      }
      const bool live = col0 + col < a.cols;
      const float inv = ll > 0.f ? 1.f / ll : 0.f;
      const size_t r = live ? out_row(a, b, h_kv, col0 + col) : 0;
#pragma unroll 4
      for (int e = threadIdx.x; e < S::kCols * D; e += 32 * kWarps) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) v += f[w] * jo[w * S::kCols * D + e];
        if (!whole)
          a.part_o[slot * (S::kCols * D) + e] = v;
        else if (live)
          store16<BF16>(a.o, r * D + channel_of<D>(e, S::kCols), v * inv);
      }
      if (threadIdx.x < S::kCols) {
        if (!whole)
          *reinterpret_cast<float2*>(a.part_ml + (slot * S::kCols + col) * 2) = make_float2(mm, ll);
        else if (live)
          a.lse[r] = lse_of(mm, ll);
      }
    }
    fence_proxy_async_smem();  // the join's writes, before the rings are copied to again
    x = u_begin + p1;
  }
  // after a wait that gave up: the copies still in flight land before the CTA ends
  if (!ok)
    for (int which = 0; which < 2; ++which)
      if (asked[which] > reads) warp_wait_all(bars + 8 * which, (asked[which] - 1) & 1, pool.err);
}

// Joins the parts of the units that several CTAs did, in CTA order, and writes the rows of
// sequences without a token.  A block takes kJoinElems elements of a unit; CG groups of
// threads share its parts (many when a unit has many parts) and meet in shared memory.
constexpr int kJoinElems = 128;
template <int D, int NT, int TOK, bool BF16, int CG>
__global__ void __launch_bounds__(kJoinElems * CG) kv4_join_kernel(const Kv4AttendArgs a) {
  constexpr int PIECE = Cfg<D, TOK>::kPiece;
  constexpr int kCols = 8 * NT, kSplit = kCols * D / kJoinElems;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float sum_o[CG][kJoinElems], sum_l[CG][kJoinElems], top[CG][kJoinElems];
  int* cum = reinterpret_cast<int*>(smem);
  if (a.early) grid_dep_launch();
  grid_dep_wait();  // in front of every read, the lengths' too
  scan_pieces<PIECE>(a, cum);
  const int T = cum[a.B], G = min(a.ctas, max(T, 1));
  const int unit = blockIdx.x / kSplit, part = blockIdx.x % kSplit;
  const int units_b = a.pool.H_kv * a.col_tiles;
  const int b = unit / units_b, u_in = unit % units_b, h_kv = u_in / a.col_tiles, ct = u_in % a.col_tiles;
  const int np = pieces_of<PIECE>(a, b);
  int c0 = 0, c1 = -1;
  if (np > 0) {
    const int u_begin = cum[b] + u_in * np;
    c0 = cta_of(u_begin, T, G);
    c1 = cta_of(u_begin + np - 1, T, G);
  }
  if (c0 == c1) return;    // written by that CTA
  const int i = threadIdx.x % kJoinElems, cg = threadIdx.x / kJoinElems;
  const int e = part * kJoinElems + i, col = e % kCols;
  float mm = -INFINITY, ll = 0.f, acc = 0.f;
  auto slot_of = [&](int c) { return (size_t)c + (c == c0 ? kKv4MaxCtas : 0); };
  for (int c = c0 + cg; c <= c1; c += CG) mm = fmaxf(mm, a.part_ml[(slot_of(c) * kCols + col) * 2]);
  if constexpr (CG > 1) {
    top[cg][i] = mm;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < CG; ++k) mm = fmaxf(mm, top[k][i]);
  }
  const float ref = mm == -INFINITY ? 0.f : mm;
#pragma unroll 8
  for (int c = c0 + cg; c <= c1; c += CG) {
    const float2 ml = *reinterpret_cast<const float2*>(a.part_ml + (slot_of(c) * kCols + col) * 2);
    const float f = ex2_approx(ml.x - ref);
    ll = fmaf(f, ml.y, ll);
    acc = fmaf(f, a.part_o[slot_of(c) * (kCols * D) + e], acc);
  }
  if constexpr (CG > 1) {
    sum_o[cg][i] = acc;
    sum_l[cg][i] = ll;
    __syncthreads();
    if (cg > 0) return;
    acc = ll = 0.f;
#pragma unroll
    for (int k = 0; k < CG; ++k) acc += sum_o[k][i], ll += sum_l[k][i];
  }
  const int col_all = ct * kCols + col;
  if (col_all >= a.cols) return;
  const size_t r = out_row(a, b, h_kv, col_all);
  store16<BF16>(a.o, r * D + channel_of<D>(e, kCols), ll == 0.f ? 0.f : acc / ll);
  if (part == 0 && i < kCols) a.lse[r] = lse_of(mm, ll);
}

template <int D, int NT, int TOK, bool BF16, int CG>
cudaError_t launch_join(const Kv4AttendArgs& a, cudaStream_t stream) {
  const long long units = (long long)a.B * a.pool.H_kv * a.col_tiles;
  return launch_dependent(kv4_join_kernel<D, NT, TOK, BF16, CG>, (unsigned)(units * (8 * NT * D / kJoinElems)), kJoinElems * CG,
                          4 * (a.B + 1), stream, static_cast<const Kv4AttendArgs&>(a));
}

template <int D, int NT, int TOK, bool BF16, class Args>
cudaError_t launch_t(Args a, long long tokens_bound, int num_sms, cudaStream_t stream) {
  using S = Smem<D, NT, TOK, std::is_same_v<Args, Kv4TreeArgs>>;
  a.ctas = (int)std::max<long long>(1, std::min<long long>({tokens_bound / Cfg<D, TOK>::kPiece + 1, (long long)ctas_per_sm(D, NT) * num_sms,
                                                            (long long)kKv4MaxCtas}));
  auto kern = kv4_attend_kernel<D, NT, TOK, BF16, false, Args>;
  const int bytes = S::bytes(a.B);
  // The limit belongs to the kernel, not to the call: one value for every batch, so that calls
  // of several threads do not lower each other's.
  static_assert(S::kCum + 4 * (kKv4MaxBatch + 1) <= 232448, "shared memory budget");
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::bytes(kKv4MaxBatch));
  if (e != cudaSuccess) return e;
  // A small grid starts while the kernel ahead ends, and lets the one behind do so (one
  // key/value head over 8000 tokens 12.6 to 11.9 us).  A full one does not: CTAs that come
  // while an SM's shared memory is divided for a kernel that needs little of it find room for
  // fewer than the others, and the stretches of all CTAs are equal (32 sequences 82 to 107 us).
  a.early = a.ctas <= num_sms ? 1 : 0;
  if (a.early) {
    e = launch_dependent(kern, (unsigned)a.ctas, 32 * kWarps, bytes, stream, a);
  } else {
    kern<<<a.ctas, 32 * kWarps, bytes, stream>>>(a);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess) return e;
  // parts of a unit, at most about
  const long long parts = a.ctas / std::max<long long>(1, (long long)a.B * a.pool.H_kv * a.col_tiles) + 1;
  return parts > 8 ? launch_join<D, NT, TOK, BF16, 8>(a, stream) : launch_join<D, NT, TOK, BF16, 1>(a, stream);
}

// One launch for short sequences: a cluster for each unit.
template <int D, int NT, bool BF16, class Args>
cudaError_t launch_cluster(Args a, int ctas, cudaStream_t stream) {
  auto kern = kv4_attend_kernel<D, NT, 32, BF16, true, Args>;
  const int bytes = Smem<D, NT, 32, std::is_same_v<Args, Kv4TreeArgs>>::bytes(0);
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  a.ctas = ctas;
  a.early = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(a.B * a.pool.H_kv * a.col_tiles * ctas));
  cfg.blockDim = dim3(32 * kWarps);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = stream;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = (unsigned)ctas;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, a);
}

// A cluster a unit, and no second launch, where no CTA then has more than four pieces of 128
// tokens (two of the wider ones) and all CTAs are on the GPU at once: the CTAs of such a cluster, 0 where
// there is none.  Against stretches and a join, us, with tables cut to the sequences: one sequence of 517
// tokens 6.7 (10.2), of 4000 10.6 (12.4; at d 256, with four pieces, 14.6 and 15.1), 8 of 300 8.0 (11.5),
// 40 of 120 8.7 (18.1); beyond what is there at once, 8 of 1000, 15.2 (12.4).
inline int cluster_ctas(int d, int nt, long long units, long long tokens_bound, int num_sms) {
  constexpr int kPiece = 32 * kWarps;
  const long long pieces = (tokens_bound / units + kPiece - 1) / kPiece;
  int ctas = 1;
  while (ctas < pieces && ctas < kKv4MaxCluster) ctas *= 2;
  return pieces <= (d * nt <= 128 ? 4 : 2) * kKv4MaxCluster && units * ctas <= ctas_per_sm(d, nt) * num_sms ? ctas : 0;
}

template <int D, int NT, class Args>
cudaError_t launch_n(const Args& a, bool bf16, long long tokens_bound, int num_sms, cudaStream_t stream) {
  // The host does not know the lengths, so every choice here goes by the room of the page
  // table: with one for 131072 tokens, 517 tokens take the form of many (11.8 us against 6.7),
  // 40 sequences of 120 13.1 against 8.7, 8 of 300 11.8 against 8.0.
  const int ctas = cluster_ctas(D, NT, (long long)a.B * a.pool.H_kv * a.col_tiles, tokens_bound, num_sms);
  if (ctas > 0)
    return bf16 ? launch_cluster<D, NT, true>(a, ctas, stream) : launch_cluster<D, NT, false>(a, ctas, stream);
  // 64-token tiles when they would fill the GPU once: measured at d 128, 8 key/value heads,
  // 32 sequences up to 16384 tokens 82 us (32-token tiles 97), one sequence of 517 tokens
  // 12.7 us (11.0); with 16 columns 73 us (85).  At d 256 they leave one CTA less an SM
  // and gain nothing.
  if constexpr (D < 256)
    if (tokens_bound >= (long long)num_sms * Cfg<D, 64>::kPiece)
      return bf16 ? launch_t<D, NT, 64, true>(a, tokens_bound, num_sms, stream)
                  : launch_t<D, NT, 64, false>(a, tokens_bound, num_sms, stream);
  return bf16 ? launch_t<D, NT, 32, true>(a, tokens_bound, num_sms, stream)
              : launch_t<D, NT, 32, false>(a, tokens_bound, num_sms, stream);
}

template <class Args>
cudaError_t launch_units(const Args& a, int d, bool bf16, long long tokens_bound, int num_sms, cudaStream_t stream) {
  const int nt = kv4_unit_cols(d, a.cols) / 8;
  switch (d) {
    case 64:
      return nt == 1 ? launch_n<64, 1>(a, bf16, tokens_bound, num_sms, stream)
             : nt == 2 ? launch_n<64, 2>(a, bf16, tokens_bound, num_sms, stream)
                       : launch_n<64, 4>(a, bf16, tokens_bound, num_sms, stream);
    case 128:
      return nt == 1 ? launch_n<128, 1>(a, bf16, tokens_bound, num_sms, stream)
                     : launch_n<128, 2>(a, bf16, tokens_bound, num_sms, stream);
    case 256:
      return nt == 1 ? launch_n<256, 1>(a, bf16, tokens_bound, num_sms, stream)
                     : launch_n<256, 2>(a, bf16, tokens_bound, num_sms, stream);
    default:
      return cudaErrorInvalidValue;
  }
}

}  // namespace
}  // namespace fa
