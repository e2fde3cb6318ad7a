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

// z of a logit: cap tanh(l / cap), or l.  tanh u = 1 - 2 / (1 + e^2u) is off by
// 2^-24 or two, absolute, and e^2u = inf gives 1.
__device__ __forceinline__ float soft_capped(float l, float cap, float inv_cap) {
  if (cap == 0.f) return l;
  return cap * (1.f - 2.f / (1.f + __expf(2.f * (l * inv_cap))));
}

// Gradient with respect to the logit of column `col`: g_a p - g_b [col = target],
// times the soft cap's slope 1 - (z / cap)^2.
__device__ __forceinline__ float logit_gradient(const ProductArgs& a, float z, int col, int target, float lse,
                                                float ga, float gb) {
  float d = ga * __expf(z - lse);
  if (col == target) d -= gb;
  if (a.cap != 0.f) {
    const float t = z * a.inv_cap;
    d *= 1.f - t * t;
  }
  return d;
}

}  // namespace muon
