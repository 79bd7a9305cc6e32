// Rows into the paged 4-bit cache and back out (layout in fa_kv4.h).
//
// A group of 32 channels x of a key or value row, all steps in fp32 so that every reader
// of the format gets the same codes:
//   low = min x,  scale = T((max x - low) / 15) (0 below 2^-126),  inv = 1 / scale (0 for 0),
//   code = min(15, rint((x - low) * inv)),  and the code stands for T(low + scale * code).
//
// Both kernels move 16 bytes of the 16-bit side per thread: 8 channels, a 32-bit word of
// codes; four lanes share a group, whose extremes two shuffles find.  They are bound by
// memory: per row 2 d bytes on one side, d / 2 codes and d / 8 parameters on the other.
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

// Thread -> (tensor, sequence, head, row, 16-byte part), parts of a row fastest.
template <int D>
struct Place {
  static constexpr int kParts = D / 8;
  int part, i, h, b, which;
  bool in;
  __device__ Place(long long idx, int N, int H, int B) {
    part = (int)(idx % kParts);
    idx /= kParts;
    i = (int)(idx % N);
    idx /= N;
    h = (int)(idx % H);
    idx /= H;
    b = (int)(idx % B);
    idx /= B;
    which = (int)idx;
    in = idx < 2;
  }
};

template <int D, bool BF16>
__global__ void __launch_bounds__(256) kv4_append_kernel(const Kv4Pool c, const uint16_t* k, const uint16_t* v,
                                                         const int32_t* start, const int32_t* count, int B, int N) {
  const Place<D> p((long long)blockIdx.x * 256 + threadIdx.x, N, c.H_kv, B);
  // whole groups of four lanes take part in the shuffles: a group is one row's, and the
  // grid's tail ends between rows
  bool live = p.in;
  if (live && count) live = p.i < count[p.b];
  long long row = -1;
  if (live) {
    row = kv4_row(c.table + (size_t)p.b * c.max_pages, c.max_pages, c.page_shift, c.num_pages,
                  (long long)start[p.b] + p.i);
    if (row < 0 && p.part == 0) record_check(c.err, kDbgPage, (uint32_t)(start[p.b] + p.i));
  }
  uint4 x4 = make_uint4(0, 0, 0, 0);
  if (row >= 0)
    x4 = *reinterpret_cast<const uint4*>((p.which ? v : k) + (((size_t)p.b * c.H_kv + p.h) * N + p.i) * D + p.part * 8);
  const uint32_t w[4] = {x4.x, x4.y, x4.z, x4.w};
  float x[8];
#pragma unroll
  for (int n = 0; n < 4; ++n) {
    x[2 * n] = widen16<BF16>((uint16_t)(w[n] & 0xFFFFu));
    x[2 * n + 1] = widen16<BF16>((uint16_t)(w[n] >> 16));
  }
  float lo = x[0], hi = x[0];
#pragma unroll
  for (int n = 1; n < 8; ++n) lo = fminf(lo, x[n]), hi = fmaxf(hi, x[n]);
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
  for (int n = 0; n < 8; ++n) {
    const int q = min(15, max(0, __float2int_rn(__fmul_rn(x[n] - lo, inv))));
    codes |= (uint32_t)q << (4 * n);
  }
  if (row < 0) return;
  const long long hr = kv4_head_row(row, c.page_shift, c.H_kv, p.h);
  reinterpret_cast<uint32_t*>(c.codes[p.which])[(size_t)hr * (D / 8) + p.part] = codes;
  if ((p.part & 3) == 0)
    c.params[p.which][(size_t)hr * (D / kKv4Group) + (p.part >> 2)] =
        (uint32_t)(s > 0.f ? s16 : 0) | ((uint32_t)round16<BF16>(lo) << 16);
}

template <int D, bool BF16>
__global__ void __launch_bounds__(256) kv4_read_kernel(const Kv4Pool c, const int32_t* start, const int32_t* lengths,
                                                       uint16_t* k, uint16_t* v, int B, int N) {
  const Place<D> p((long long)blockIdx.x * 256 + threadIdx.x, N, c.H_kv, B);
  if (!p.in) return;
  const long long pos = (long long)start[p.b] + p.i;
  uint32_t out[4] = {0, 0, 0, 0};
  if (pos < lengths[p.b]) {
    const long long row = kv4_row(c.table + (size_t)p.b * c.max_pages, c.max_pages, c.page_shift, c.num_pages, pos);
    if (row >= 0) {
      const long long hr = kv4_head_row(row, c.page_shift, c.H_kv, p.h);
      const uint32_t codes = reinterpret_cast<const uint32_t*>(c.codes[p.which])[(size_t)hr * (D / 8) + p.part];
      const uint32_t par = c.params[p.which][(size_t)hr * (D / kKv4Group) + (p.part >> 2)];
      const uint32_t s2 = __byte_perm(par, par, 0x1010), l2 = __byte_perm(par, par, 0x3232);
#pragma unroll
      for (int n = 0; n < 4; ++n)
        out[n] = value2<BF16>(pack2<BF16>((float)((codes >> (8 * n)) & 15u), (float)((codes >> (8 * n + 4)) & 15u)), s2, l2);
    } else if (p.part == 0) {
      record_check(c.err, kDbgPage, (uint32_t)pos);
    }
  }
  *reinterpret_cast<uint4*>((p.which ? v : k) + (((size_t)p.b * c.H_kv + p.h) * N + p.i) * D + p.part * 8) =
      make_uint4(out[0], out[1], out[2], out[3]);
}

template <int D>
unsigned grid_of(int B, int H, int N) {
  return (unsigned)((2LL * B * H * N * (D / 8) + 255) / 256);
}

template <int D, bool BF16>
cudaError_t append_t(const Kv4Pool& c, const void* k, const void* v, const int32_t* start, const int32_t* count, int B,
                     int N, cudaStream_t s) {
  kv4_append_kernel<D, BF16><<<grid_of<D>(B, c.H_kv, N), 256, 0, s>>>(
      c, static_cast<const uint16_t*>(k), static_cast<const uint16_t*>(v), start, count, B, N);
  return cudaGetLastError();
}
template <int D, bool BF16>
cudaError_t read_t(const Kv4Pool& c, const int32_t* start, const int32_t* lengths, void* k, void* v, int B, int N,
                   cudaStream_t s) {
  kv4_read_kernel<D, BF16><<<grid_of<D>(B, c.H_kv, N), 256, 0, s>>>(c, start, lengths, static_cast<uint16_t*>(k),
                                                                     static_cast<uint16_t*>(v), B, N);
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
