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
