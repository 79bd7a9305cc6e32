// Rotary positions: pairs of channels of queries and keys turned by the angle of their
// position, forward and backward.
//
//   theta_i = position * freqs_i,  i < dims / 2
//   y1 = amplitude (x1 cos theta - x2 sin theta),  y2 = amplitude (x2 cos theta + x1 sin theta)
//
// for the pairs (x_i, x_(i + dims/2)), or (x_2i, x_(2i+1)) when interleaved; channels from dims
// on are copied.  The gradient of y is turned back: the same with -theta.
//
// It is bound by memory: every element is read and written once.  A thread takes 8 pairs (16
// channels, 32 bytes) of one row (sequence and token) and of several heads: the angles are the
// same in all of them, so cosines and sines cost little.  An angle is a fraction of a turn in 64
// bits of fixed point (fa_rotary.h); its upper 32 bits go to fp32 as half turns in [-1, 1) and
// through the fast cosine and sine, whose error there is under 2^-21, far below a rounding to
// 16 bits.
//
// Measured (one GB300, the kernel alone in a captured graph; in brackets a Python call among others): 2 x 8192
// rows of 16 + 4 heads out of and into a joint projection, d 128 bf16, 27.7 us (29.0; 168 MB, 6.1 TB/s, 89 % of
// the copy's rate); 4 x 2048 rows of 16 + 16 heads, d 64 fp16, neighbours as pairs, backward, 12.4 (13.7); 2 x
// 2001 rows of 8 + 4 heads, d 256, 64 channels turned, 8.8 (9.2).  The small ones are a start, a frequency's
// division and one wave of loads and stores; 64 single rows of 32 + 8 heads take 2.2 (5.7).
#include <algorithm>
#include <climits>

#include "fa_internal.h"
#include "fa_rotary.h"
#include "fa_rule.cuh"
#include "ptx.cuh"

namespace fa {
namespace {

constexpr int kThreads = 256;
constexpr int kHeads = 2;  // heads whose loads are in flight together

__device__ __forceinline__ uint4 load16(const uint16_t* p) {
  uint4 w;
  asm volatile("ld.global.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w) : "l"(p));
  return w;
}

// 8 pairs of channels turned: two groups of 8 whose channels i make pairs, or 16 neighbours.
template <bool BF16, bool INTERLEAVED>
__device__ __forceinline__ void turn_pairs(uint4 (&x)[2], const float (&c)[8], const float (&s)[8]) {
  uint32_t w[8] = {x[0].x, x[0].y, x[0].z, x[0].w, x[1].x, x[1].y, x[1].z, x[1].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (INTERLEAVED) {
#pragma unroll
      for (int g = 0; g < 8; g += 4) {
        const float u = widen16<BF16>((uint16_t)(w[g + i] & 0xFFFFu)), v = widen16<BF16>((uint16_t)(w[g + i] >> 16));
        w[g + i] = pack2<BF16>(u * c[g + i] - v * s[g + i], v * c[g + i] + u * s[g + i]);
      }
    } else {
      const float u0 = widen16<BF16>((uint16_t)(w[i] & 0xFFFFu)), u1 = widen16<BF16>((uint16_t)(w[i] >> 16));
      const float v0 = widen16<BF16>((uint16_t)(w[4 + i] & 0xFFFFu)), v1 = widen16<BF16>((uint16_t)(w[4 + i] >> 16));
      w[i] = pack2<BF16>(u0 * c[2 * i] - v0 * s[2 * i], u1 * c[2 * i + 1] - v1 * s[2 * i + 1]);
      w[4 + i] = pack2<BF16>(v0 * c[2 * i] + u0 * s[2 * i], v1 * c[2 * i + 1] + u1 * s[2 * i + 1]);
    }
  }
  x[0] = make_uint4(w[0], w[1], w[2], w[3]);
  x[1] = make_uint4(w[4], w[5], w[6], w[7]);
}

template <int D, bool BF16, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const RotaryArgs a) {
  __shared__ uint64_t turn[D / 2];
  constexpr int kUnits = D / 16, kRows = kThreads / kUnits;  // 16 channels a thread
  grid_dep_launch();
  grid_dep_wait();
  if ((int)threadIdx.x < a.dims / 2) {
    const uint64_t t = turns_of(a.freqs[threadIdx.x]);
    turn[threadIdx.x] = a.backward ? 0 - t : t;
  }
  __syncthreads();
  const int unit = threadIdx.x % kUnits;
  const long long row = (long long)blockIdx.x * kRows + threadIdx.x / kUnits;
  if (row >= (long long)a.B * a.N) return;
  const int b = (int)(row / a.N), n = (int)(row - (long long)b * a.N);
  const bool turned = unit < a.dims / 16;
  if (!turned && !a.tail) return;
  // the thread's two groups of 8 channels
  const int ch0 = INTERLEAVED || !turned ? 16 * unit : 8 * unit;
  const int ch1 = INTERLEAVED || !turned ? ch0 + 8 : ch0 + a.dims / 2;
  float c[8], s[8];
  if (turned) {
    const uint32_t pos = (uint32_t)(a.positions ? a.positions[row] : n);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      // (a negative position is 2^32 more here: 2^32 times the fraction is taken off again)
      uint64_t t = turn[8 * unit + i] * pos;
      if ((int32_t)pos < 0) t -= turn[8 * unit + i] << 32;
      const float x = (float)(int32_t)(t >> 32) * (3.14159265358979f * 4.656612873077393e-10f);  // pi 2^-31
      c[i] = __cosf(x) * a.amplitude;
      s[i] = __sinf(x) * a.amplitude;
    }
  }
  const int h0 = blockIdx.y * a.heads_per_block, h1 = min(h0 + a.heads_per_block, a.H + a.H_kv);
  auto part_of = [&](int h) -> const RotaryRows& { return a.part[h >= a.H]; };
  for (int h = h0; h < h1; h += kHeads) {
    uint4 x[kHeads][2];
#pragma unroll
    for (int j = 0; j < kHeads; ++j)
      if (h + j < h1) {
        const RotaryRows& p = part_of(h + j);
        const uint16_t* in = static_cast<const uint16_t*>(p.in) + b * p.in_b + (h + j >= a.H ? h + j - a.H : h + j) * p.in_h + n * p.in_n;
        x[j][0] = load16(in + ch0), x[j][1] = load16(in + ch1);
      }
#pragma unroll
    for (int j = 0; j < kHeads; ++j)
      if (h + j < h1) {
        if (turned) turn_pairs<BF16, INTERLEAVED>(x[j], c, s);
        const RotaryRows& p = part_of(h + j);
        uint16_t* out = static_cast<uint16_t*>(p.out) + b * p.out_b + (h + j >= a.H ? h + j - a.H : h + j) * p.out_h + n * p.out_n;
        *reinterpret_cast<uint4*>(out + ch0) = x[j][0];
        *reinterpret_cast<uint4*>(out + ch1) = x[j][1];
      }
  }
}

template <int D>
cudaError_t launch_d(RotaryArgs a, bool bf16, bool interleaved, int num_sms, cudaStream_t stream) {
  constexpr int kRows = kThreads / (D / 16);
  const long long blocks = ((long long)a.B * a.N + kRows - 1) / kRows;
  const int heads = a.H + a.H_kv;
  // As many heads a block as leave 16 blocks an SM, two or three waves of those that fit there: one wave of
  // 8 leaves the loads of a block's later heads without others beside them, and with more than 16 the angles
  // weigh (us in a graph with 4, 8, 16 and 32: the training rows above 29.2, 29.0, 27.7 and 29.5, the backward ones 14.4,
  // 13.0, 12.4 and 14.8; four heads in flight instead of two 27.2 and 12.9 with 16, 31.5 and 16.4 with 32).
  const long long groups = std::min<long long>(heads, std::max<long long>(1, (16LL * num_sms + blocks - 1) / blocks));
  a.heads_per_block = (int)((heads + groups - 1) / groups);
  auto kern = bf16 ? (interleaved ? rotary_kernel<D, true, true> : rotary_kernel<D, true, false>)
                   : (interleaved ? rotary_kernel<D, false, true> : rotary_kernel<D, false, false>);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)blocks, (unsigned)((heads + a.heads_per_block - 1) / a.heads_per_block));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, a);
}

}  // namespace

cudaError_t launch_rotary(RotaryArgs a, int d, bool bf16, bool interleaved, int num_sms, cudaStream_t stream) {
  switch (d) {
    case 64:
      return launch_d<64>(a, bf16, interleaved, num_sms, stream);
    case 128:
      return launch_d<128>(a, bf16, interleaved, num_sms, stream);
    case 256:
      return launch_d<256>(a, bf16, interleaved, num_sms, stream);
    default:
      return cudaErrorInvalidValue;
  }
}

}  // namespace fa
