// Device helpers of the block kernels: stack lookup, element access in either
// type, splitting into bfloat16 parts.
#pragma once

#include "blocks_internal.h"
#include "numeric.h"

#pragma clang fp contract(off)

namespace muon {

typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));

// The stack whose range of workgroups (by `key`) holds workgroup b.
template <class Key>
__device__ __forceinline__ BlockStack find_stack(const BlockTable& tab, int b, Key key) {
  const BlockStack* t = tab.ext ? tab.ext : tab.inl;
  int lo = 0, hi = tab.count;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (key(t[mid]) <= b) lo = mid; else hi = mid;
  }
  return t[lo];
}

__device__ __forceinline__ float load1f(const void* p, bool bf, int64_t e) {
  return bf ? bf16_bits_to_float(gmem(reinterpret_cast<const uint16_t*>(p))[e])
            : gmem(reinterpret_cast<const float*>(p))[e];
}

__device__ __forceinline__ void load8f(const void* p, bool bf, int64_t e, float v[8]) {
  if (bf) {
    const u32x4_t r = *gmem(reinterpret_cast<const u32x4_t*>(reinterpret_cast<const uint16_t*>(p) + e));
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      v[2 * q] = __uint_as_float(r[q] << 16);
      v[2 * q + 1] = __uint_as_float(r[q] & 0xFFFF0000u);
    }
  } else {
    const f32x4_t a = *gmem(reinterpret_cast<const f32x4_t*>(reinterpret_cast<const float*>(p) + e));
    const f32x4_t b = *gmem(reinterpret_cast<const f32x4_t*>(reinterpret_cast<const float*>(p) + e + 4));
#pragma unroll
    for (int q = 0; q < 4; ++q) { v[q] = a[q]; v[4 + q] = b[q]; }
  }
}

__device__ __forceinline__ void load4f(const void* p, bool bf, int64_t e, float v[4]) {
  if (bf) {
    const u32x2_t r = *gmem(reinterpret_cast<const u32x2_t*>(reinterpret_cast<const uint16_t*>(p) + e));
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      v[2 * q] = __uint_as_float(r[q] << 16);
      v[2 * q + 1] = __uint_as_float(r[q] & 0xFFFF0000u);
    }
  } else {
    const f32x4_t a = *gmem(reinterpret_cast<const f32x4_t*>(reinterpret_cast<const float*>(p) + e));
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] = a[q];
  }
}

// N (4 or 8) consecutive elements from e, `vec`: as 16- or 8-byte loads.
// Otherwise one by one, without branches: elements at or past `valid` are not
// read (the load goes to element `safe`, which exists) and come out as zero.
template <int N>
__device__ __forceinline__ void load_vec(const void* p, bool bf, int64_t e, float v[N]) {
  if constexpr (N == 8) load8f(p, bf, e, v); else load4f(p, bf, e, v);
}
template <int N>
__device__ __forceinline__ void load_masked(const void* p, bool bf, int64_t e, int valid, int64_t safe, float v[N]) {
  if (bf) {
#pragma unroll
    for (int q = 0; q < N; ++q) {
      const float f = load1f(p, true, q < valid ? e + q : safe);
      v[q] = q < valid ? f : 0.f;
    }
  } else {
#pragma unroll
    for (int q = 0; q < N; ++q) {
      const float f = load1f(p, false, q < valid ? e + q : safe);
      v[q] = q < valid ? f : 0.f;
    }
  }
}

// N (2, 4 or 8) consecutive elements to e.
template <int N>
__device__ __forceinline__ void store_vec(void* p, bool bf, int64_t e, const float v[N]) {
  if (bf) {
    uint32_t h[N / 2];
#pragma unroll
    for (int q = 0; q < N / 2; ++q) h[q] = float2_to_bf16x2_bits(v[2 * q], v[2 * q + 1]);
    uint16_t* o = reinterpret_cast<uint16_t*>(p) + e;
    if constexpr (N == 8) *gmem(reinterpret_cast<u32x4_t*>(o)) = u32x4_t{h[0], h[1], h[2], h[3]};
    else if constexpr (N == 4) *gmem(reinterpret_cast<u32x2_t*>(o)) = u32x2_t{h[0], h[1]};
    else *gmem(reinterpret_cast<uint32_t*>(o)) = h[0];
  } else {
    float* o = reinterpret_cast<float*>(p) + e;
    if constexpr (N == 2) {
      *gmem(reinterpret_cast<f32x2_t*>(o)) = f32x2_t{v[0], v[1]};
    } else {
#pragma unroll
      for (int q = 0; q < N; q += 4)
        *gmem(reinterpret_cast<f32x4_t*>(o + q)) = f32x4_t{v[q], v[q + 1], v[q + 2], v[q + 3]};
    }
  }
}
__device__ __forceinline__ void store1f(void* p, bool bf, int64_t e, float v) {
  if (bf) gmem(reinterpret_cast<uint16_t*>(p))[e] = float_to_bf16_bits(v);
  else gmem(reinterpret_cast<float*>(p))[e] = v;
}

// Two values as PL bfloat16 parts each (part p of v0 | part p of v1 << 16):
// every part is the nearest bfloat16 of what the parts before it leave, so
// PL parts carry 8 PL bits.
template <int PL>
__device__ __forceinline__ void split2(float v0, float v1, uint32_t part[PL]) {
#pragma unroll
  for (int p = 0; p < PL; ++p) {
    part[p] = float2_to_bf16x2_bits(v0, v1);
    if (p + 1 < PL) {
      v0 = v0 - __uint_as_float(part[p] << 16);
      v1 = v1 - __uint_as_float(part[p] & 0xFFFF0000u);
    }
  }
}

// Four runs of two values as PL operands of eight bfloat16.
template <int PL>
__device__ __forceinline__ void split8(const float v[8], bf16x8_t out[PL]) {
  u32x4_t o[PL];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    uint32_t part[PL];
    split2<PL>(v[2 * q], v[2 * q + 1], part);
#pragma unroll
    for (int l = 0; l < PL; ++l) o[l][q] = part[l];
  }
#pragma unroll
  for (int l = 0; l < PL; ++l) out[l] = __builtin_bit_cast(bf16x8_t, o[l]);
}

// acc += sum of the products of a's and b's parts that are not below the
// last part's place (hi*hi, hi*lo, lo*hi; with three parts also mid*mid,
// hi*lo2, lo2*hi), smallest first.
template <int PA, int PB>
__device__ __forceinline__ f32x4_t mfma_parts(const bf16x8_t a[PA], const bf16x8_t b[PB], f32x4_t acc) {
  constexpr int S = (PA > PB ? PA : PB) - 1;
#pragma unroll
  for (int s = S; s >= 0; --s)
#pragma unroll
    for (int p = 0; p <= s; ++p) {
      const int q = s - p;
      if (p < PA && q < PB) acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[p], b[q], acc, 0, 0, 0);
    }
  return acc;
}

// Momentum of one element (one rounding per operation): updates m, returns U.
__device__ __forceinline__ float momentum_elem(float g, float& m, const BlockMom& k) {
  const float gg = k.ema ? k.g1 * g : g;
  m = k.beta * m + gg;
  return k.nesterov ? gg + k.beta * m : m;
}
// U from the gradient and the momentum already updated.
__device__ __forceinline__ float momentum_dir(float g, float m, const BlockMom& k) {
  const float gg = k.ema ? k.g1 * g : g;
  return k.nesterov ? gg + k.beta * m : m;
}

}  // namespace muon
