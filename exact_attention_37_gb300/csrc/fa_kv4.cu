// Rows into the paged 4-bit cache and back out (layout in fa_kv4.h).
//
// A group of 32 channels x of a key or value row, all steps in fp32 so that every reader
// of the format gets the same codes:
//   low = min x,  scale = T((max x - low) / 15) (0 below 2^-126),  inv = 1 / scale (0 for 0),
//   code = min(15, rint((x - low) * inv)),  and the code stands for T(low + scale * code).
//
// Both kernels move 32 bytes of the 16-bit side per thread and row: 16 channels, two words
// of codes; two lanes share a group, whose extremes one shuffle finds.  They are bound by
// memory (per row 2 d bytes on one side, d / 2 codes and d / 8 parameters on the other)
// only if the arithmetic is short, so extremes and codes are found two channels at a time,
// values come from the codes' bits (fa_kv4.cuh), and each thread has several rows in
// flight.  Rows are numbered as they lie in k, v [B, H_kv, N, d] (all of k, then all of
// v); only the cache's side needs the sequence, head and token of a number, two divisions
// by multiplication.
//
// Measured, 4 sequences of up to 4096 tokens (12010 in all), 8 heads, d 128: append 18 us (63 MB
// of it needed: 3.5 TB/s), read 15.5 us (81 MB: 5.2 TB/s); with 16-byte accesses and one
// channel at a time 20 us each.  One token of 64 sequences: 2.4 us each, most of it a launch.
#include <algorithm>
#include <climits>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fa_kv4.cuh"
#include "fa_kv4.h"
#include "fa_rule.cuh"
#include "ptx.cuh"

namespace fa {
namespace {

template <bool BF16>
__device__ __forceinline__ uint16_t round16(float x) {
  return (uint16_t)(pack2<BF16>(x, 0.f) & 0xFFFFu);
}

// n / d and n % d for 0 <= n < 2^31 by a multiplication: T. Granlund and P. Montgomery,
// "Division by invariant integers using multiplication", 1994.
struct FastDiv {
  uint32_t d, mul, shift;
  explicit FastDiv(uint32_t div) : d(div), mul(0), shift(0) {
    while ((1ull << shift) < d) ++shift;
    mul = (uint32_t)((((1ull << shift) - d) << 32) / d + 1);
  }
  __device__ __forceinline__ uint32_t div(uint32_t n) const {
    return (uint32_t)(((uint64_t)__umulhi(n, mul) + n) >> shift);
  }
};

constexpr int kThreads = 256;

struct RowArgs {
  uint32_t rows;       // B H_kv N
  FastDiv by_n, by_h;
  RowArgs(int B, int H, int N) : rows((uint32_t)B * H * N), by_n(N), by_h(H) {}
};
// Sequence, head and token of row r (r < rows).
struct RowAt {
  int b, h, i;
  __device__ __forceinline__ RowAt(const RowArgs& a, uint32_t r) {
    const uint32_t bh = a.by_n.div(r);
    i = (int)(r - bh * a.by_n.d);
    b = (int)a.by_h.div(bh);
    h = (int)(bh - (uint32_t)b * a.by_h.d);
  }
};

// The pool's row (page, head, token) of a token, -1 where there is none.
__device__ __forceinline__ long long pool_row(const Kv4Pool& c, int b, int h, long long pos) {
  const long long row = kv4_row(c.table + (size_t)b * c.max_pages, c.max_pages, c.page_shift, c.num_pages, pos);
  return row < 0 ? -1 : kv4_head_row(row, c.page_shift, c.H_kv, h);
}

// 32 bytes at once where the addresses allow it (WIDE): two 16-byte accesses would touch
// every 32-byte sector twice.
template <bool WIDE>
__device__ __forceinline__ void load32(const uint16_t* p, uint32_t (&w)[8]) {
  if constexpr (WIDE) {
    asm volatile("ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                 : "l"(p));
  } else {
    const uint4 a = reinterpret_cast<const uint4*>(p)[0], b = reinterpret_cast<const uint4*>(p)[1];
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
  }
}
template <bool WIDE>
__device__ __forceinline__ void store32(uint16_t* p, const uint32_t (&w)[8]) {
  if constexpr (WIDE) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    reinterpret_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    reinterpret_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}
// Extremes of two pairs, NaN where an operand is: a NaN in a group becomes its low value, and
// so every value of it.
template <bool BF16>
__device__ __forceinline__ uint32_t min16(uint32_t a, uint32_t b) {
  uint32_t r;
  if constexpr (BF16)
    asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else
    asm("min.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
template <bool BF16>
__device__ __forceinline__ uint32_t max16(uint32_t a, uint32_t b) {
  uint32_t r;
  if constexpr (BF16)
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else
    asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Codes of 8 channels x as a word: channel e in bits 4 e to 4 e + 3.  Channels e and e + 4 go
// through the packed instructions together; adding 1.5 2^23 rounds to an integer, four
// of which are joined in floating point (below 2^16, exact) and read off the bits.
template <bool BF16>
__device__ __forceinline__ uint32_t codes8(const float* x, float lo, float inv) {
  constexpr float kRound = 12582912.f;
  const F2 nlo(-lo, -lo), up(kRound, kRound), down(-kRound, -kRound), sixteen(16.f, 16.f);
  F2 sum;
#pragma unroll
  for (int e = 3; e >= 0; --e) {
    // (a packed product would be joined with the packed sum behind it into one multiply-add,
    // whose single rounding gives other codes at ties, 1 in 1000: the product is scalar)
    float a, b;
    add(F2(x[e], x[e + 4]), nlo).get(a, b);
    a = __fmul_rn(a, inv), b = __fmul_rn(b, inv);
    if constexpr (!BF16)  // a subnormal fp16 scale may be far below (max - min) / 15; a bf16 one is within 2^-9 of it
      a = fminf(a, 15.f), b = fminf(b, 15.f);
    const F2 c = add(add(F2(a, b), up), down);
    sum = e == 3 ? c : fma(sum, sixteen, c);
  }
  float a, b;
  add(sum, F2(8388608.f, 8388608.f)).get(a, b);
  return __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x5410);
}

template <int D, bool BF16, int ROWS, bool WIDE>
__global__ void __launch_bounds__(kThreads) kv4_append_kernel(const Kv4Pool c, const RowArgs a, const uint16_t* k,
                                                              const uint16_t* v, const int32_t* start,
                                                              const int32_t* count) {
  grid_dep_launch();
  grid_dep_wait();
  constexpr int kParts = D / 16, kStep = kThreads / kParts;
  const int part = threadIdx.x % kParts;
  const uint32_t first = blockIdx.x * (uint32_t)(kStep * ROWS) + threadIdx.x / kParts;
  // rows that count asks for are found first (count and table come from the caches), so
  // that nothing of a ragged batch's padding is read
  uint32_t ws[ROWS][8];
  long long hrs[ROWS];
#pragma unroll
  for (int n = 0; n < ROWS; ++n) {
    const uint32_t r = first + n * kStep;
    const bool is_v = r >= a.rows;
#pragma unroll
    for (int e = 0; e < 8; ++e) ws[n][e] = 0;
    hrs[n] = -1;
    if (r < 2 * a.rows) {
      const RowAt at(a, is_v ? r - a.rows : r);
      if (!count || at.i < count[at.b]) {
        load32<WIDE>((is_v ? v : k) + (size_t)(is_v ? r - a.rows : r) * D + part * 16, ws[n]);
        const long long pos = (long long)start[at.b] + at.i;
        hrs[n] = pool_row(c, at.b, at.h, pos);
        if (hrs[n] < 0 && part == 0) record_check(c.err, kDbgPage, (uint32_t)pos);
      }
    }
  }
#pragma unroll
  for (int n = 0; n < ROWS; ++n) {
    const bool is_v = first + n * kStep >= a.rows;
    const long long hr = hrs[n];
    const uint32_t(&w)[8] = ws[n];
    // extremes of the thread's 16 channels in pairs, then of the group: whole groups of two
    // lanes, each of one row, take part in the shuffle
    uint32_t mn = w[0], mx = w[0];
#pragma unroll
    for (int e = 1; e < 8; ++e) mn = min16<BF16>(mn, w[e]), mx = max16<BF16>(mx, w[e]);
    mn = min16<BF16>(mn, __byte_perm(mn, mn, 0x1032));
    mx = max16<BF16>(mx, __byte_perm(mx, mx, 0x1032));
    const uint32_t mine = __byte_perm(mn, mx, 0x5410), other = __shfl_xor_sync(0xffffffffu, mine, 1);
    const uint16_t lo16 = (uint16_t)(min16<BF16>(mine, other) & 0xFFFFu);
    const float lo = widen16<BF16>(lo16), hi = widen16<BF16>((uint16_t)(max16<BF16>(mine, other) >> 16));
    const uint16_t s16 = round16<BF16>(__fdiv_rn(hi - lo, 15.f));
    float s = widen16<BF16>(s16);
    if (s < 1.17549435e-38f) s = 0.f;
    const float inv = s > 0.f ? __fdiv_rn(1.f, s) : 0.f;
    uint32_t codes[2];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      float x[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[2 * e] = widen16<BF16>((uint16_t)(w[4 * half + e] & 0xFFFFu));
        x[2 * e + 1] = widen16<BF16>((uint16_t)(w[4 * half + e] >> 16));
      }
      codes[half] = codes8<BF16>(x, lo, inv);
    }
    if (hr >= 0) {
      reinterpret_cast<uint2*>(c.codes[is_v])[(size_t)hr * (D / 16) + part] = make_uint2(codes[0], codes[1]);
      if ((part & 1) == 0)
        c.params[is_v][(size_t)hr * (D / kKv4Group) + (part >> 1)] = (uint32_t)(s > 0.f ? s16 : 0) | ((uint32_t)lo16 << 16);
    }
  }
}

template <int D, bool BF16, int ROWS, bool WIDE>
__global__ void __launch_bounds__(kThreads) kv4_read_kernel(const Kv4Pool c, const RowArgs a, const int32_t* start,
                                                            const int32_t* lengths, uint16_t* k, uint16_t* v) {
  grid_dep_launch();
  grid_dep_wait();
  constexpr int kParts = D / 16, kStep = kThreads / kParts;
  const int part = threadIdx.x % kParts;
  const uint32_t first = blockIdx.x * (uint32_t)(kStep * ROWS) + threadIdx.x / kParts;
  uint2 codes[ROWS];
  uint32_t par[ROWS];
#pragma unroll
  for (int n = 0; n < ROWS; ++n) {
    const uint32_t r = first + n * kStep;
    codes[n] = make_uint2(0, 0);
    par[n] = 0;  // stands for zeros
    if (r < 2 * a.rows) {
      const bool is_v = r >= a.rows;
      const RowAt at(a, is_v ? r - a.rows : r);
      const long long pos = (long long)start[at.b] + at.i;
      if (pos < lengths[at.b]) {
        const long long hr = pool_row(c, at.b, at.h, pos);
        if (hr >= 0) {
          codes[n] = reinterpret_cast<const uint2*>(c.codes[is_v])[(size_t)hr * (D / 16) + part];
          par[n] = c.params[is_v][(size_t)hr * (D / kKv4Group) + (part >> 1)];
        } else if (part == 0) {
          record_check(c.err, kDbgPage, (uint32_t)pos);
        }
      }
    }
  }
#pragma unroll
  for (int n = 0; n < ROWS; ++n) {
    const uint32_t r = first + n * kStep;
    if (r >= 2 * a.rows) break;
    const bool is_v = r >= a.rows;
    const uint32_t s2 = __byte_perm(par[n], par[n], 0x1010), l2 = __byte_perm(par[n], par[n], 0x3232);
    uint32_t out[8];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      uint32_t p[4];  // channels (e, e + 4)
      values4<BF16>(half ? codes[n].y : codes[n].x, s2, l2, p);
      out[4 * half] = __byte_perm(p[0], p[1], 0x5410);
      out[4 * half + 1] = __byte_perm(p[2], p[3], 0x5410);
      out[4 * half + 2] = __byte_perm(p[0], p[1], 0x7632);
      out[4 * half + 3] = __byte_perm(p[2], p[3], 0x7632);
    }
    store32<WIDE>((is_v ? v : k) + (size_t)(is_v ? r - a.rows : r) * D + part * 16, out);
  }
}

// Rows a thread has in flight, to hide the chain of count, table and row: 2 and 4 for
// prompts (append 18.1 us with one row, 18.2 with two, 19.6 with four, ragged batches gain
// with two; read 19.5, 16.1, 15.5), 1 when the grid would not fill the GPU otherwise (a
// step's rows: 5.3 us for both kernels against 8.2 with four).
constexpr int kRowsAppend = 2, kRowsRead = 4;
template <int D>
bool few_rows(long long rows, int sms, int many) { return 2 * rows * (D / 16) < (long long)sms * 4 * kThreads * many; }
template <int D>
unsigned grid_of(long long rows, int per_thread) {
  const long long step = (long long)(kThreads / (D / 16)) * per_thread;
  return (unsigned)((2 * rows + step - 1) / step);
}

template <int D, bool BF16>
cudaError_t append_t(const Kv4Pool& c, const void* k, const void* v, const int32_t* start, const int32_t* count, int B,
                     int N, int sms, cudaStream_t s) {
  const long long rows = (long long)B * c.H_kv * N;
  const bool few = few_rows<D>(rows, sms, kRowsAppend);
  const bool wide = ((reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v)) & 31u) == 0;
  auto kern = wide ? (few ? kv4_append_kernel<D, BF16, 1, true> : kv4_append_kernel<D, BF16, kRowsAppend, true>)
                   : (few ? kv4_append_kernel<D, BF16, 1, false> : kv4_append_kernel<D, BF16, kRowsAppend, false>);
  return launch_dependent(kern, grid_of<D>(rows, few ? 1 : kRowsAppend), kThreads, 0, s, c, RowArgs(B, c.H_kv, N),
                          static_cast<const uint16_t*>(k), static_cast<const uint16_t*>(v), start, count);
}
template <int D, bool BF16>
cudaError_t read_t(const Kv4Pool& c, const int32_t* start, const int32_t* lengths, void* k, void* v, int B, int N,
                   int sms, cudaStream_t s) {
  const long long rows = (long long)B * c.H_kv * N;
  const bool few = few_rows<D>(rows, sms, kRowsRead);
  const bool wide = ((reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v)) & 31u) == 0;
  auto kern = wide ? (few ? kv4_read_kernel<D, BF16, 1, true> : kv4_read_kernel<D, BF16, kRowsRead, true>)
                   : (few ? kv4_read_kernel<D, BF16, 1, false> : kv4_read_kernel<D, BF16, kRowsRead, false>);
  return launch_dependent(kern, grid_of<D>(rows, few ? 1 : kRowsRead), kThreads, 0, s, c, RowArgs(B, c.H_kv, N), start,
                          lengths, static_cast<uint16_t*>(k), static_cast<uint16_t*>(v));
}

}  // namespace

cudaError_t launch_kv4_append(const Kv4Pool& c, int d, bool bf16, const void* k, const void* v, const int32_t* start,
                              const int32_t* count, int B, int N, int sms, cudaStream_t s) {
  switch (d) {
    case 64:
      return bf16 ? append_t<64, true>(c, k, v, start, count, B, N, sms, s)
                  : append_t<64, false>(c, k, v, start, count, B, N, sms, s);
    case 128:
      return bf16 ? append_t<128, true>(c, k, v, start, count, B, N, sms, s)
                  : append_t<128, false>(c, k, v, start, count, B, N, sms, s);
    case 256:
      return bf16 ? append_t<256, true>(c, k, v, start, count, B, N, sms, s)
                  : append_t<256, false>(c, k, v, start, count, B, N, sms, s);
    default:
      return cudaErrorInvalidValue;
  }
}

cudaError_t launch_kv4_read(const Kv4Pool& c, int d, bool bf16, const int32_t* start, const int32_t* lengths, void* k,
                            void* v, int B, int N, int sms, cudaStream_t s) {
  switch (d) {
    case 64:
      return bf16 ? read_t<64, true>(c, start, lengths, k, v, B, N, sms, s)
                  : read_t<64, false>(c, start, lengths, k, v, B, N, sms, s);
    case 128:
      return bf16 ? read_t<128, true>(c, start, lengths, k, v, B, N, sms, s)
                  : read_t<128, false>(c, start, lengths, k, v, B, N, sms, s);
    case 256:
      return bf16 ? read_t<256, true>(c, start, lengths, k, v, B, N, sms, s)
                  : read_t<256, false>(c, start, lengths, k, v, B, N, sms, s);
    default:
      return cudaErrorInvalidValue;
  }
}

}  // namespace fa
