// Rotary positions: arguments of the kernel, and the angle arithmetic that the host's query
// and the kernel share.
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

namespace fa {

// High and low 64 bits of 2^128 / (2 pi).
constexpr uint64_t kTurnHi = 0x28BE60DB9391054Aull, kTurnLo = 0x7F09D5F47D4D3770ull;

// f / (2 pi) turns as a fraction of 2^64, for a finite f (whole turns drop out).  A product
// with an integer position, modulo 2^64, is then the angle of that position as a fraction of a
// turn, off by at most |position| 2^-64 turns: exact at any distance, where radians in fp32
// lose 0.01 at 10^5 and a product in fp64 would be on units that this GPU has few of.
__host__ __device__ inline uint64_t turns_of(double f) {
  uint64_t bits;
#ifdef __CUDA_ARCH__
  bits = (uint64_t)__double_as_longlong(f);
#else
  __builtin_memcpy(&bits, &f, 8);
#endif
  const int e = (int)((bits >> 52) & 0x7FF);
  const uint64_t m = (bits & ((1ull << 52) - 1)) | (e ? 1ull << 52 : 0);
  // f = m 2^(max(e, 1) - 1075), so f / (2 pi) 2^64 = m (kTurnHi 2^64 + kTurnLo) 2^(max(e, 1) - 1139)
  uint64_t hi, lo, low_hi;
#ifdef __CUDA_ARCH__
  hi = __umul64hi(m, kTurnHi), lo = m * kTurnHi, low_hi = __umul64hi(m, kTurnLo);
#else
  const unsigned __int128 a = (unsigned __int128)m * kTurnHi, b = (unsigned __int128)m * kTurnLo;
  hi = (uint64_t)(a >> 64), lo = (uint64_t)a, low_hi = (uint64_t)(b >> 64);
#endif
  lo += low_hi;
  hi += lo < low_hi;
  const int right = 1075 - (e ? e : 1);  // of the 128 bits hi, lo
  uint64_t t;
  if (right >= 128) t = 0;
  else if (right >= 64) t = hi >> (right - 64);
  else if (right > 0) t = (hi << (64 - right)) | (lo >> right);
  else t = right > -64 ? lo << -right : 0;  // 2^52 and above: bits of 1 / (2 pi) that are not held
  return bits >> 63 ? 0 - t : t;
}

struct RotaryRows {
  const void* in;
  void* out;
  long long in_b, in_h, in_n, out_b, out_h, out_n;  // strides in elements
};
struct RotaryArgs {
  RotaryRows part[2];      // queries, keys
  const int32_t* positions;
  const double* freqs;
  int B, H, H_kv, N, dims;
  int backward, tail;      // tail: channels behind dims are copied
  float amplitude;
  int heads_per_block;
};
cudaError_t launch_rotary(RotaryArgs a, int d, bool bf16, bool interleaved, int num_sms, cudaStream_t stream);

}  // namespace fa
