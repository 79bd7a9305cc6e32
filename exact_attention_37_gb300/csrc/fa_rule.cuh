// Score rules: what may happen to a score between Q K^T and the softmax, shared by the
// forward and backward kernels.  For query row i of a head and key j, with the query's
// position p = i + N_k - N_q:
//
//   u = scale q_i.k_j
//   z = cap tanh(u / cap)  (cap > 0; z = u otherwise)
//   y = z - slope_h |p - j|
//   visible when  (no ids, or q_doc_i == k_doc_j >= 0)  and  (not causal, or j <= p, or j < prefix_b)
//
// The kernels work in base 2, y2 = y log2 e.  tanh.approx has a relative error of 2^-11,
// which would show in L, so tanh(x) is
//   |x| <= 0.35:  x + x w (c1 + w (c2 + w (c3 + w c4))), w = x^2, the Taylor series of
//                 tanh to x^9 (the next term is 0.0089 x^11: 2.4e-7 of the value), and
//   otherwise  :  1 - 2 / (1 + 2^(2 x log2 e)), the exponent limited to 30 (there the
//                 result is 1 to the last bit); one rcp serves four scores,
//                 1/a = (1/abcd) b cd, as MUFU is what bounds this form.
// A warp takes the series when every score of its chunk allows it.
#pragma once
#include "fa_internal.h"
#include "ptx.cuh"

namespace fa {

// What a kernel instance applies: nothing (plain attention), masks only, masks and a
// distance bias, or masks, a cap and a bias (slope 0 without one).
enum : int { kRuleOff = -1, kRuleMask = 0, kRuleBias = 1, kRuleCap = 2 };

// Entries of the block lists: the block index above the flag bits.
constexpr int kListShift = 2;
constexpr int kListPartial = 1;  // some pair of the block is hidden
constexpr int kListClean = 2;    // the streamed block holds rows with a negative id

constexpr float kLog2eF = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ int rule_prefix(const RuleArgs& r, int b, int Nk) {
  return r.prefix ? max(0, min(r.prefix[b], Nk)) : 0;
}
__device__ __forceinline__ float rule_slope2(const RuleArgs& r, int h) { return r.slopes ? r.slopes[h] * kLog2eF : 0.f; }

__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two floats in a register pair, for the packed f32x2 instructions.
struct F2 {
  uint64_t v;
  __device__ __forceinline__ F2() {}
  __device__ __forceinline__ F2(float a, float b) { asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b)); }
  __device__ __forceinline__ void get(float& a, float& b) const {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
  }
};
__device__ __forceinline__ F2 fma(F2 a, F2 b, F2 c) {
  F2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return d;
}
__device__ __forceinline__ F2 mul(F2 a, F2 b) {
  F2 d;
  asm("mul.f32x2 %0, %1, %2;" : "=l"(d.v) : "l"(a.v), "l"(b.v));
  return d;
}

// tanh(s cap_x) of a row's 32 raw scores in place (the bits of fp32 values); every lane
// of the warp calls it.
__device__ __forceinline__ void rule_tanh(uint32_t (&s)[32], float cap_x) {
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < 32; i += 2) top = max3f(top, fabsf(__uint_as_float(s[i])), fabsf(__uint_as_float(s[i + 1])));
  if (__all_sync(0xffffffffu, top * cap_x <= 0.35f)) {
    const F2 k(cap_x, cap_x), c1(-1.f / 3.f, -1.f / 3.f), c2(2.f / 15.f, 2.f / 15.f), c3(-17.f / 315.f, -17.f / 315.f),
        c4(62.f / 2835.f, 62.f / 2835.f);
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
      const F2 x = mul(F2(__uint_as_float(s[i]), __uint_as_float(s[i + 1])), k);
      const F2 w = mul(x, x);
      const F2 p = fma(fma(fma(c4, w, c3), w, c2), w, c1);
      float t0, t1;
      fma(mul(x, w), p, x).get(t0, t1);
      s[i] = __float_as_uint(t0);
      s[i + 1] = __float_as_uint(t1);
    }
  } else {
    const float k = 2.f * kLog2eF * cap_x;
#pragma unroll
    for (int i = 0; i < 32; i += 4) {
      float e[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) e[j] = ex2_approx(fminf(__uint_as_float(s[i + j]) * k, 30.f)) + 1.f;
      const float ab = e[0] * e[1], cd = e[2] * e[3], q = -2.f * rcp_approx(ab * cd);
      const float qab = q * cd, qcd = q * ab;  // -2 / ab, -2 / cd
      s[i] = __float_as_uint(fmaf(qab, e[1], 1.f));
      s[i + 1] = __float_as_uint(fmaf(qab, e[0], 1.f));
      s[i + 2] = __float_as_uint(fmaf(qcd, e[3], 1.f));
      s[i + 3] = __float_as_uint(fmaf(qcd, e[2], 1.f));
    }
  }
}

// tanh(s cap_x) of one score.
__device__ __forceinline__ float rule_tanh1(float s, float cap_x) {
  const float x = s * cap_x;
  if (fabsf(x) <= 0.35f) {
    const float w = x * x;
    return fmaf(x * w, fmaf(fmaf(fmaf(62.f / 2835.f, w, -17.f / 315.f), w, 2.f / 15.f), w, -1.f / 3.f), x);
  }
  return fmaf(-2.f, rcp_approx(ex2_approx(x * (2.f * kLog2eF)) + 1.f), 1.f);
}

// One row's 128 raw scores to base-2 scores y2; d0 = first key - the row's position.
template <bool CAP>
__device__ __forceinline__ void rule_scores(float (&s)[128], const RuleArgs& rule, float scale_log2, float slope2,
                                            int d0) {
  const float f0 = (float)d0;
  const float mul = CAP ? rule.cap2 : scale_log2;
  if constexpr (CAP) {
#pragma unroll
    for (int ch = 0; ch < 4; ++ch) {
      uint32_t t[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) t[i] = __float_as_uint(s[32 * ch + i]);
      rule_tanh(t, rule.cap_x);
#pragma unroll
      for (int i = 0; i < 32; ++i) s[32 * ch + i] = __uint_as_float(t[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < 128; ++i) s[i] = fmaf(-slope2, fabsf(f0 + (float)i), s[i] * mul);
}

// Hides the N columns whose id differs from the row's (row_id < 0 hides all of them).
// ids points at N padded ids, 16-byte aligned; the column count is a multiple of 4.
template <int N>
__device__ __forceinline__ void rule_hide_ids(float (&s)[N], const int* ids, int row_id, float hidden) {
  const int4* p = reinterpret_cast<const int4*>(ids);
  const int id = row_id < 0 ? (int)0x80000000 : row_id;  // padded ids are >= -1
#pragma unroll
  for (int i = 0; i < N; i += 4) {
    const int4 k = __ldg(p + (i >> 2));
    if (k.x != id) s[i] = hidden;
    if (k.y != id) s[i + 1] = hidden;
    if (k.z != id) s[i + 2] = hidden;
    if (k.w != id) s[i + 3] = hidden;
  }
}

// The same for probabilities: hidden ones become 0.
template <int N>
__device__ __forceinline__ void rule_hide_ids_at(float* p, const int* ids, int row_id) {
  const int4* v = reinterpret_cast<const int4*>(ids);
  const int id = row_id < 0 ? (int)0x80000000 : row_id;
#pragma unroll
  for (int i = 0; i < N; i += 4) {
    const int4 k = __ldg(v + (i >> 2));
    if (k.x != id) p[i] = 0.f;
    if (k.y != id) p[i + 1] = 0.f;
    if (k.z != id) p[i + 2] = 0.f;
    if (k.w != id) p[i + 3] = 0.f;
  }
}

// Backward: the exponent y2 - L log2 e of a raw score (with a cap, of its tanh), f0 the
// signed distance.
template <bool CAP>
__device__ __forceinline__ void rule_exponent(uint32_t s, const RuleArgs& rule, float scale_log2, float slope2,
                                              float f0, float l2, float& x) {
  x = fmaf(-slope2, fabsf(f0), fmaf(__uint_as_float(s), CAP ? rule.cap2 : scale_log2, -l2));
}
// 1 - tanh^2
__device__ __forceinline__ float rule_dtanh(uint32_t t) {
  const float f = __uint_as_float(t);
  return fmaf(-f, f, 1.f);
}

// Zeroes row r of a tile of PANELS panels of 128-byte rows.
template <int PANELS, uint32_t PANEL_BYTES>
__device__ __forceinline__ void clear_row(uint32_t tile, int r) {
#pragma unroll
  for (int p = 0; p < PANELS; ++p)
#pragma unroll
    for (int c = 0; c < 8; ++c) st_shared_v4(tile + p * PANEL_BYTES + r * 128u + 16u * c, 0u, 0u, 0u, 0u);
}

}  // namespace fa
