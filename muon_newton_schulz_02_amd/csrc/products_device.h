// Scalar device code shared by the kernels of the expert products and of the
// head's loss.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "numeric.h"
#include "products_internal.h"

namespace muon {

// Rows of group g: [lo, hi), clamped to [0, rows], hi >= lo.  Without offsets: all.
__device__ __forceinline__ void group_range(const ProductArgs& a, int g, int& lo, int& hi) {
  if (!a.offsets) {
    lo = 0;
    hi = a.rows;
    return;
  }
  lo = min(max(a.offsets[g], 0), a.rows);
  hi = max(lo, min(a.offsets[g + 1], a.rows));
}

// Pieces that a group's k of `rows` is cut into (TN).
__device__ __forceinline__ int pieces_of(int rows, int chunk) { return max(1, (rows + chunk - 1) / chunk); }

// Sums over the groups before each of them: pre[0] = 0, pre[g + 1] = pre[g] + value(g),
// 2^30 where they pass it (2048 groups that overlap may have 2^35 rows).
// All NT threads of the workgroup take part; wave_sum holds NT / 64 values.
template <int NT, class Value>
__device__ __forceinline__ void group_sums(int groups, int* pre, int* wave_sum, int tid, Value value) {
  const int lane = tid & 63, wave = tid >> 6;
  int carry = 0;
  if (tid == 0) pre[0] = 0;
  if (groups == 1) {
    if (tid == 0) pre[1] = value(0);
    __syncthreads();
    return;
  }
  for (int b = 0; b < groups; b += NT) {
    const int g = b + tid;
    int v = g < groups ? value(g) : 0;
#pragma unroll
    for (int s = 1; s < 64; s *= 2) {
      const int o = __shfl_up(v, s);
      if (lane >= s) v = min(v + o, 1 << 30);
    }
    if (lane == 63) wave_sum[wave] = v;
    __syncthreads();
    int before = carry;
#pragma unroll
    for (int w = 0; w < NT / 64; ++w) {
      if (w < wave) before = min(before + wave_sum[w], 1 << 30);
      carry = min(carry + wave_sum[w], 1 << 30);
    }
    if (g < groups) pre[g + 1] = min(before + v, 1 << 30);
    __syncthreads();
  }
  __syncthreads();
}

// The chunk that TN's groups are cut into: a.chunk, or everything where the groups'
// rows are more than there are (they overlap).  Uses pre[0 .. groups].
template <int NT>
__device__ __forceinline__ int safe_chunk(const ProductArgs& a, int* pre, int* wave_sum, int tid) {
  if (a.chunk >= a.rows || !a.offsets) return a.chunk;
  group_sums<NT>(a.groups, pre, wave_sum, tid, [&](int g) {
    int lo, hi;
    group_range(a, g, lo, hi);
    return hi - lo;
  });
  const bool apart = pre[a.groups] <= a.rows;
  __syncthreads();
  return apart ? a.chunk : 1 << 30;
}

// Column of this launch that is row i's target (any value outside: none here).
__device__ __forceinline__ int target_of(const ProductArgs& a, int i) {
  if (a.target) return a.target[i] - a.col0;
  const int64_t t = a.targets[i] - a.col0;
  return t >= 0 && t < a.n ? int(t) : -1;
}

// What rounding to bfloat16 leaves of a number; 0 where that is infinite or NaN.
__device__ __forceinline__ float rest_of(float v) {
  const float r = v - bf16_bits_to_float(float_to_bf16_bits(v));
  return fabsf(r) < INFINITY ? r : 0.f;
}

// Softmax in base 2: exponents are y = z log2 e, so that an exponential is one fma and
// one v_exp_f32.  With a soft cap z = cap tanh(l / cap), |z| = cap (1 - 2 r), r = 1 / (1 +
// e^(2 |l| / cap)), whose slope in l is 4 r (1 - r).  (r of l itself would be next to 1 for
// logits far below, and 1 - r the rounding of it.)
constexpr float LOG2E = 1.44269504088896340736f, LN2 = 0.69314718055994530942f;
struct SoftCap {
  float inv;        // 1 / cap
  float k;          // 2 log2 e / cap
  float c2;         // cap log2 e
};
__device__ __forceinline__ SoftCap soft_cap(const ProductArgs& a) { return {a.inv_cap, 2.f * LOG2E * a.inv_cap, a.cap * LOG2E}; }

__device__ __forceinline__ float cap_r(float l, const SoftCap& c) {
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(fabsf(l) * c.k));     // e^.. = inf: 0
}
__device__ __forceinline__ float cap_slope(float r) { return 4.f * __builtin_fmaf(-r, r, r); }
// z log2 e, off by some 5 2^-24 cap whatever l is.  EXACT: below |l / cap| = 0.3
// l times tanh's own series (its next term is 5e-8 there), so that the error is 18 2^-24 of
// the value at most, and a large cap leaves the logits as they are.
template <bool EXACT>
__device__ __forceinline__ float capped_y(float l, float r, const SoftCap& c) {
  if constexpr (!EXACT) return copysignf(__builtin_fmaf(-2.f * c.c2, r, c.c2), l);
  const float y = copysignf(c.c2 * __builtin_fmaf(-2.f, r, 1.f), l);
  const float u = l * c.inv, s = u * u;
  float p = __builtin_fmaf(s, 0.0218694881f, -0.0539682545f);
  p = __builtin_fmaf(s, p, 0.133333340f);
  p = __builtin_fmaf(s, p, -0.333333343f);
  p = __builtin_fmaf(s, p, 1.f);
  return fabsf(u) < 0.3f ? l * LOG2E * p : y;
}
// The same where no slope is needed: the short form with r of l itself saves the sign (8192 x
// 1536 by 32768 780 us, 788 with it).
template <bool EXACT>
__device__ __forceinline__ float capped_y(float l, const SoftCap& c) {
  if constexpr (EXACT) return capped_y<true>(l, cap_r(l, c), c);
  return __builtin_fmaf(-2.f * c.c2, __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(l * c.k)), c.c2);
}

}  // namespace muon
