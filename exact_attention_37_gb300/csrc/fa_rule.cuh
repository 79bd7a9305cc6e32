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
// which would show in L, so tanh(x), x = u / cap = s k with s = q.k and k = scale / cap, is
//   |x| <= 0.35:  s (k + W (a1 + W (a2 + W a3))), W = s^2, a_n = c_n k^(2n+1): the
//                 polynomial x (1 + w (c1 + w (c2 + w c3))), w = x^2, whose c_n were fitted
//                 here to tanh(x) / x with the smallest largest relative error, 4.2e-8
//                 (the series would need two more terms); five multiply-adds a score; and
//   otherwise  :  1 - 2 / (1 + 2^(2 x log2 e)), the exponent limited to 30 (there the
//                 result is 1 to the last bit); one rcp serves four scores,
//                 1/a = (1/abcd) b cd, as MUFU is what bounds this form.
// A warp takes the polynomial when every score of its rows' part allows it: one vote for as
// many columns as are at hand, so that their multiply-adds overlap (forward, 128 columns
// against 32: B4 H16 N2048 d64 156 to 141 us with cap 50, B2 H16 N8192 d128 packed 197 to
// 189).  The rules lengthen a row's chain of instructions, and two softmax or elementwise
// warps a scheduler do not hide it (1.2 to 2.1 instructions a clock of 4): at B4 H16 N2048 d64
// without a mask, plain, capped by 50 (polynomial) and by 15 (exponentials), the forward
// takes 88, 141 and 174 us, the backward 279, 393 and 440.  (A longer polynomial, five terms
// up to 0.75, between the two forms: forward 176 to 167 with cap 30, but 174 to 207 with
// 15, and nothing in the backward.)
//
// What a row sees is a range [lo, hi) of the other side: the causal mask, a prefix and the
// length give one, and so do document ids that do not decrease (padding in front or
// behind).  Other ids are compared one by one, in the blocks marked for it.
#pragma once
#include "fa_internal.h"
#include "ptx.cuh"

namespace fa {

// What a kernel instance applies: nothing (plain attention), or a rule with a distance
// bias, a cap, document ids, each or not.  A mask and a prefix are always there.
enum : int { kRuleOff = -1, kRuleBias = 1, kRuleCap = 2, kRuleDocs = 4, kRuleKinds = 8 };
constexpr bool rule_has(int rule, int what) { return rule >= 0 && (rule & what) != 0; }

// Entries of the block lists: the block index above the flag bits.
constexpr int kListShift = 2;
constexpr int kListIds = 1;    // ids are compared one by one (they are in no order)
constexpr int kListClean = 2;  // the streamed block holds rows with a negative id

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
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d.v) : "l"(a.v), "l"(b.v));
  return d;
}

__device__ __forceinline__ F2 add(F2 a, F2 b) {
  F2 d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d.v) : "l"(a.v), "l"(b.v));
  return d;
}

// max(a, |b|, |c|) and min(a, b) that are NaN when an operand is.
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(fabsf(b)), "f"(fabsf(c)));
  return d;
}
__device__ __forceinline__ float min_nan(float a, float b) {
  float d;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// 1 - 2 / (1 + 2^x), x = s k with k = 2 log2(e) scale / cap
__device__ __forceinline__ float rule_tanh_exp(float s, float k) {
  return fmaf(-2.f, rcp_approx(ex2_approx(min_nan(s * k, 30.f)) + 1.f), 1.f);
}
// tanh(s k) of a row's N raw scores in place; every lane of the warp calls it.  A NaN stays
// one.  Four scores that share a reciprocal hand it to each other; with document ids (IDS),
// where padding may hold NaN next to keys that are seen, a warp that has one takes its scores
// one by one.  (That third form in every kind: exponentials at B4 H16 N2048 d64 174 to 183 us
// forward, 440 to 447 backward.)
template <int N, bool IDS>
__device__ __forceinline__ void rule_tanh(float* s, const RuleArgs& r) {
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    if constexpr (IDS) top = max3_nan(top, s[i], s[i + 1]);
    else top = max3f(top, fabsf(s[i]), fabsf(s[i + 1]));
  }
  const float k2 = 2.f * kLog2eF * r.cap_x;
  if (__all_sync(0xffffffffu, top <= r.tanh_top)) {
    const F2 k(r.cap_x, r.cap_x), a1(r.tanh_a1, r.tanh_a1), a2(r.tanh_a2, r.tanh_a2), a3(r.tanh_a3, r.tanh_a3);
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const F2 x(s[i], s[i + 1]);
      const F2 w = mul(x, x);
      mul(x, fma(fma(fma(a3, w, a2), w, a1), w, k)).get(s[i], s[i + 1]);
    }
  } else if (IDS && __any_sync(0xffffffffu, top != top)) {
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] = rule_tanh_exp(s[i], k2);
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      float e[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) e[j] = ex2_approx(min_nan(s[i + j] * k2, 30.f)) + 1.f;
      const float ab = e[0] * e[1], cd = e[2] * e[3], q = -2.f * rcp_approx(ab * cd);
      const float qab = q * cd, qcd = q * ab;  // -2 / ab, -2 / cd
      s[i] = fmaf(qab, e[1], 1.f);
      s[i + 1] = fmaf(qab, e[0], 1.f);
      s[i + 2] = fmaf(qcd, e[3], 1.f);
      s[i + 3] = fmaf(qcd, e[2], 1.f);
    }
  }
}
// The same of one score (branching per lane).
__device__ __forceinline__ float rule_tanh1(float s, const RuleArgs& r) {
  if (fabsf(s) <= r.tanh_top) {
    const float w = s * s;
    return s * fmaf(fmaf(fmaf(r.tanh_a3, w, r.tanh_a2), w, r.tanh_a1), w, r.cap_x);
  }
  return rule_tanh_exp(s, 2.f * kLog2eF * r.cap_x);
}
// 1 - tanh^2
__device__ __forceinline__ float rule_dtanh(float t) { return fmaf(-t, t, 1.f); }

// The bias -slope2 |d0 + i| over columns i = 0 .. n-1, as base + sl i where the sign of
// d0 + i does not change for any lane of the warp (every block off the diagonal); mixed
// otherwise.
struct RuleBias {
  float base = 0.f, sl = 0.f;
  bool mixed = false;
  __device__ __forceinline__ RuleBias() {}
  __device__ __forceinline__ RuleBias(float slope2, int d0, int n) {
    const bool before = __all_sync(0xffffffffu, d0 + n - 1 <= 0), behind = __all_sync(0xffffffffu, d0 >= 0);
    mixed = !before && !behind;
    sl = mixed ? 0.f : before ? slope2 : -slope2;
    base = sl * (float)d0;
  }
};

// z - slope2 |idx| of two columns: the bias in a mixed block.
__device__ __forceinline__ F2 bias_mixed(F2 idx, float slope2, F2 z) {
  float i0, i1, z0, z1;
  idx.get(i0, i1);
  z.get(z0, z1);
  return F2(fmaf(-slope2, fabsf(i0), z0), fmaf(-slope2, fabsf(i1), z1));
}

// Columns i outside [lo, hi) of N become `hidden`.  One bit test and one select a column.
template <int N>
__device__ __forceinline__ void rule_hide_range(float* s, int lo, int hi, float hidden) {
#pragma unroll
  for (int c = 0; c < N; c += 32) {
    const int l = max(0, min(lo - c, 32)), h = max(0, min(hi - c, 32));
    const uint32_t above = l >= 32 ? 0u : 0xffffffffu << l, below = h >= 32 ? 0xffffffffu : ~(0xffffffffu << h);
    const uint32_t m = above & below;
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (!((m >> i) & 1u)) s[c + i] = hidden;
  }
}

// Columns whose id differs from the row's become `hidden` (row_id < 0 hides all of them).
// ids points at N padded ids, 16-byte aligned.
template <int N>
__device__ __forceinline__ void rule_hide_ids(float* s, const int* ids, int row_id, float hidden) {
  const int4* p = reinterpret_cast<const int4*>(ids);
  const int id = row_id < 0 ? (int)0x80000000 : row_id;  // padded ids are >= -1
#pragma unroll
  for (int i = 0; i < N; i += 4) {
    const int4 k = p[i >> 2];
    if (k.x != id) s[i] = hidden;
    if (k.y != id) s[i + 1] = hidden;
    if (k.z != id) s[i + 2] = hidden;
    if (k.w != id) s[i + 3] = hidden;
  }
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
