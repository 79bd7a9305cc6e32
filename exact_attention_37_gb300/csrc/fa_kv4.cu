// Rows into the paged 4-bit cache and back out (layout in fa_kv4.h).
//
// A group of 32 channels x of a key or value row, all steps in fp32 so that every reader
// of the format gets the same codes:
//   low = min x,  scale = T((max x - low) / 15) (0 below 2^-126),  inv = 1 / scale (0 for 0),
//   code = min(15, rint((x - low) * inv)),  and the code stands for T(low + scale * code).
//
// Both kernels move 16 bytes of the 16-bit side per thread and row: 8 channels, a 32-bit
// word of codes; four lanes share a group, whose extremes two shuffles find.  They are
// bound by memory: per row 2 d bytes on one side, d / 2 codes and d / 8 parameters on the
// other, so each thread has kRows rows in flight.  Rows are numbered as they lie in k, v
// [B, H_kv, N, d] (all of k, then all of v); only the cache's side needs the sequence,
// head and token of a number, two divisions by multiplication.
#include <algorithm>
#include <climits>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fa_kv4.h"
#include "ptx.cuh"

namespace fa {
namespace {

template <bool BF16>
__device__ __forceinline__ uint16_t round16(float x) {
  return (uint16_t)(pack2<BF16>(x, 0.f) & 0xFFFFu);
}

// T(low + scale * code) of two values packed: the fused product has one rounding.
template <bool BF16>
__device__ __forceinline__ uint32_t value2(uint32_t code2, uint32_t scale2, uint32_t low2) {
  uint32_t r;
  if constexpr (BF16)
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(code2), "r"(scale2), "r"(low2));
  else
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(code2), "r"(scale2), "r"(low2));
  return r;
}

// n / d and n % d for 0 <= n < 2^31 by a multiplication.
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
constexpr int kRows = 4;  // rows a thread has in flight

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

template <int D, bool BF16>
__global__ void __launch_bounds__(kThreads) kv4_append_kernel(const Kv4Pool c, const RowArgs a, const uint16_t* k,
                                                              const uint16_t* v, const int32_t* start,
                                                              const int32_t* count) {
  constexpr int kParts = D / 8, kStep = kThreads / kParts;
  const int part = threadIdx.x % kParts;
  const uint32_t first = blockIdx.x * (uint32_t)(kStep * kRows) + threadIdx.x / kParts;
  uint4 x4[kRows];
#pragma unroll
  for (int n = 0; n < kRows; ++n) {
    const uint32_t r = first + n * kStep;
    x4[n] = make_uint4(0, 0, 0, 0);
    if (r < 2 * a.rows) {
      const bool is_v = r >= a.rows;
      x4[n] = *reinterpret_cast<const uint4*>((is_v ? v : k) + (size_t)(is_v ? r - a.rows : r) * D + part * 8);
    }
  }
#pragma unroll
  for (int n = 0; n < kRows; ++n) {
    const uint32_t r = first + n * kStep;
    const bool is_v = r >= a.rows;
    long long hr = -1;
    if (r < 2 * a.rows) {
      const RowAt at(a, is_v ? r - a.rows : r);
      if (!count || at.i < count[at.b]) {
        const long long pos = (long long)start[at.b] + at.i;
        hr = pool_row(c, at.b, at.h, pos);
        if (hr < 0 && part == 0) record_check(c.err, kDbgPage, (uint32_t)pos);
      }
    }
    // whole groups of four lanes, each of one row, take part in the shuffles
    const uint32_t w[4] = {x4[n].x, x4[n].y, x4[n].z, x4[n].w};
    float x[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[2 * e] = widen16<BF16>((uint16_t)(w[e] & 0xFFFFu));
      x[2 * e + 1] = widen16<BF16>((uint16_t)(w[e] >> 16));
    }
    float lo = x[0], hi = x[0];
#pragma unroll
    for (int e = 1; e < 8; ++e) lo = fminf(lo, x[e]), hi = fmaxf(hi, x[e]);
#pragma unroll
    for (int off = 1; off < 4; off <<= 1) {
      lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, off));
      hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, off));
    }
    const uint16_t s16 = round16<BF16>(__fdiv_rn(hi - lo, 15.f));
    float s = widen16<BF16>(s16);
    if (s < 1.17549435e-38f) s = 0.f;
    const float inv = s > 0.f ? __fdiv_rn(1.f, s) : 0.f;
    uint32_t codes = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int q = min(15, max(0, __float2int_rn(__fmul_rn(x[e] - lo, inv))));
      codes |= (uint32_t)q << (4 * e);
    }
    if (hr >= 0) {
      reinterpret_cast<uint32_t*>(c.codes[is_v])[(size_t)hr * (D / 8) + part] = codes;
      if ((part & 3) == 0)
        c.params[is_v][(size_t)hr * (D / kKv4Group) + (part >> 2)] =
            (uint32_t)(s > 0.f ? s16 : 0) | ((uint32_t)round16<BF16>(lo) << 16);
    }
  }
}

template <int D, bool BF16>
__global__ void __launch_bounds__(kThreads) kv4_read_kernel(const Kv4Pool c, const RowArgs a, const int32_t* start,
                                                            const int32_t* lengths, uint16_t* k, uint16_t* v) {
  constexpr int kParts = D / 8, kStep = kThreads / kParts;
  const int part = threadIdx.x % kParts;
  const uint32_t first = blockIdx.x * (uint32_t)(kStep * kRows) + threadIdx.x / kParts;
  uint32_t codes[kRows], par[kRows];
#pragma unroll
  for (int n = 0; n < kRows; ++n) {
    const uint32_t r = first + n * kStep;
    codes[n] = par[n] = 0;  // stands for zeros
    if (r < 2 * a.rows) {
      const bool is_v = r >= a.rows;
      const RowAt at(a, is_v ? r - a.rows : r);
      const long long pos = (long long)start[at.b] + at.i;
      if (pos < lengths[at.b]) {
        const long long hr = pool_row(c, at.b, at.h, pos);
        if (hr >= 0) {
          codes[n] = reinterpret_cast<const uint32_t*>(c.codes[is_v])[(size_t)hr * (D / 8) + part];
          par[n] = c.params[is_v][(size_t)hr * (D / kKv4Group) + (part >> 2)];
        } else if (part == 0) {
          record_check(c.err, kDbgPage, (uint32_t)pos);
        }
      }
    }
  }
#pragma unroll
  for (int n = 0; n < kRows; ++n) {
    const uint32_t r = first + n * kStep;
    if (r >= 2 * a.rows) break;
    const bool is_v = r >= a.rows;
    const uint32_t s2 = __byte_perm(par[n], par[n], 0x1010), l2 = __byte_perm(par[n], par[n], 0x3232);
    uint32_t out[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      out[e] = value2<BF16>(pack2<BF16>((float)((codes[n] >> (8 * e)) & 15u), (float)((codes[n] >> (8 * e + 4)) & 15u)),
                            s2, l2);
    *reinterpret_cast<uint4*>((is_v ? v : k) + (size_t)(is_v ? r - a.rows : r) * D + part * 8) =
        make_uint4(out[0], out[1], out[2], out[3]);
  }
}

template <int D>
unsigned grid_of(int B, int H, int N) {
  const long long step = (long long)(kThreads / (D / 8)) * kRows;
  return (unsigned)((2LL * B * H * N + step - 1) / step);
}

template <int D, bool BF16>
cudaError_t append_t(const Kv4Pool& c, const void* k, const void* v, const int32_t* start, const int32_t* count, int B,
                     int N, cudaStream_t s) {
  kv4_append_kernel<D, BF16><<<grid_of<D>(B, c.H_kv, N), kThreads, 0, s>>>(
      c, RowArgs(B, c.H_kv, N), static_cast<const uint16_t*>(k), static_cast<const uint16_t*>(v), start, count);
  return cudaGetLastError();
}
template <int D, bool BF16>
cudaError_t read_t(const Kv4Pool& c, const int32_t* start, const int32_t* lengths, void* k, void* v, int B, int N,
                   cudaStream_t s) {
  kv4_read_kernel<D, BF16><<<grid_of<D>(B, c.H_kv, N), kThreads, 0, s>>>(
      c, RowArgs(B, c.H_kv, N), start, lengths, static_cast<uint16_t*>(k), static_cast<uint16_t*>(v));
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv4_append(const Kv4Pool& c, int d, bool bf16, const void* k, const void* v, const int32_t* start,
                              const int32_t* count, int B, int N, cudaStream_t s) {
  switch (d) {
    case 64: return bf16 ? append_t<64, true>(c, k, v, start, count, B, N, s) : append_t<64, false>(c, k, v, start, count, B, N, s);
    case 128: return bf16 ? append_t<128, true>(c, k, v, start, count, B, N, s) : append_t<128, false>(c, k, v, start, count, B, N, s);
    case 256: return bf16 ? append_t<256, true>(c, k, v, start, count, B, N, s) : append_t<256, false>(c, k, v, start, count, B, N, s);
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t launch_kv4_read(const Kv4Pool& c, int d, bool bf16, const int32_t* start, const int32_t* lengths, void* k,
                            void* v, int B, int N, cudaStream_t s) {
  switch (d) {
    case 64: return bf16 ? read_t<64, true>(c, start, lengths, k, v, B, N, s) : read_t<64, false>(c, start, lengths, k, v, B, N, s);
    case 128: return bf16 ? read_t<128, true>(c, start, lengths, k, v, B, N, s) : read_t<128, false>(c, start, lengths, k, v, B, N, s);
    case 256: return bf16 ? read_t<256, true>(c, start, lengths, k, v, B, N, s) : read_t<256, false>(c, start, lengths, k, v, B, N, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace fa
