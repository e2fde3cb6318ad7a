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

// The workgroup's number among those of all launches over the table.
__device__ __forceinline__ int block_number() {
  typedef __attribute__((address_space(4))) const BlockTable ConstTable;
  return int(blockIdx.x) + ((ConstTable*)__builtin_amdgcn_kernarg_segment_ptr())->first;
}

// The stack whose range of workgroups (or blocks) holds number b, the same in
// all lanes.  The table is the kernel's first argument.  The lanes compare 64
// keys at a time, every 64^k-th first, so that a workgroup waits for two loads
// (up to 64 stacks; four for 2^18), not for a search; the descriptor is read
// through the constant address space and stays in scalar registers.
template <int KEY>
__device__ __forceinline__ BlockStack find_stack(int b) {
  typedef __attribute__((address_space(4))) const BlockStack ConstStack;
  typedef __attribute__((address_space(4))) const BlockTable ConstTable;
  typedef __attribute__((address_space(4))) const int32_t ConstInt;
  ConstTable* tab = (ConstTable*)__builtin_amdgcn_kernarg_segment_ptr();
  const int count = tab->count;
  ConstInt* keys = tab->ext ? (ConstInt*)tab->ext_keys + KEY * count : &tab->keys[KEY][0];
  ConstStack* t = tab->ext ? (ConstStack*)tab->ext : &tab->inl[0];
  const int lane = threadIdx.x & 63;
  int step = 1, at = 0;  // keys ascend, and keys[at] <= b (the first is 0)
  while (step * 64 < count) step *= 64;
  for (;; step /= 64) {
    const int i = at + lane * step;
    const int below = __popcll(__ballot(i < count && keys[min(i, count - 1)] <= b));
    at += (__builtin_amdgcn_readfirstlane(below) - 1) * step;
    if (step == 1) break;
  }
  BlockStack s;
  __builtin_memcpy(&s, (const BlockStack*)(t + at), sizeof(s));
  return s;
}

// Eight consecutive elements as loaded: bfloat16 in a, binary32 in a and b.
struct Raw8 {
  u32x4_t a, b;
};
// 16 bytes at any element's address (global accesses need no alignment on
// this GPU; the compiler knows).
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(2)));
typedef uint32_t u32_any __attribute__((aligned(2)));

// The eight elements at byte `off` of `base` (the same in all lanes), of
// which the first `valid` exist (the others are not read and come out as
// zero).
__device__ __forceinline__ void load_raw(Raw8& o, const char* base, uint32_t off, bool bf, int valid) {
  const auto s = gmem(base) + off;
  o.a = u32x4_t{0, 0, 0, 0};
  o.b = u32x4_t{0, 0, 0, 0};
  typedef __attribute__((address_space(1))) const u32x4_any GV;
  if (valid >= 8) {
    o.a = *(GV*)s;
    if (!bf) o.b = *(GV*)(s + 16);
  } else if (valid > 0) {
    // runs of 4, 2 and 1 as the bits of valid say, put in their places: an
    // element at a time, a step of 297 blocks of 1111 x 90 took 120 us a pass, so 111
    // and 104
    typedef __attribute__((address_space(1))) const u32x2_any GV2;
    typedef __attribute__((address_space(1))) const u32_any GV1;
    typedef __attribute__((address_space(1))) const uint16_t GH;
    const bool four = valid & 4, two = valid & 2;
    if (bf) {
      u32x2_t q = {0, 0};
      uint32_t p2 = 0, p1 = 0;
      if (four) q = *(GV2*)s;
      if (two) p2 = *(GV1*)(s + 2 * (valid & 4));
      if (valid & 1) p1 = *(GH*)(s + 2 * (valid & 6));
      const uint32_t t0 = two ? p2 : p1, t1 = two ? p1 : 0;
      o.a = four ? u32x4_t{q[0], q[1], t0, t1} : u32x4_t{t0, t1, 0, 0};
    } else {
      u32x4_t q = {0, 0, 0, 0};
      u32x2_t p2 = {0, 0};
      uint32_t p1 = 0;
      if (four) q = *(GV*)s;
      if (two) p2 = *(GV2*)(s + 4 * (valid & 4));
      if (valid & 1) p1 = *(GV1*)(s + 4 * (valid & 6));
      const u32x4_t t = {two ? p2[0] : p1, p2[1], two ? p1 : 0, 0};
      o.a = four ? q : t;
      if (four) o.b = t;
    }
  }
}

__device__ __forceinline__ void unpack(const Raw8& o, bool bf, float v[8]) {
  if (bf) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      v[2 * q] = __uint_as_float(o.a[q] << 16);
      v[2 * q + 1] = __uint_as_float(o.a[q] & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      v[q] = __uint_as_float(o.a[q]);
      v[4 + q] = __uint_as_float(o.b[q]);
    }
  }
}

__device__ __forceinline__ void store8(char* base, uint32_t off, bool bf, int valid, const float v[8]) {
  const auto d = gmem(base) + off;
  typedef __attribute__((address_space(1))) u32x4_any GV;
  typedef __attribute__((address_space(1))) u32x2_any GV2;
  typedef __attribute__((address_space(1))) u32_any GV1;
  if (bf) {
    typedef __attribute__((address_space(1))) uint16_t GH;
    if (valid >= 8) {
      *(GV*)d = u32x4_t{float2_to_bf16x2_bits(v[0], v[1]), float2_to_bf16x2_bits(v[2], v[3]),
                        float2_to_bf16x2_bits(v[4], v[5]), float2_to_bf16x2_bits(v[6], v[7])};
    } else {
      const uint32_t w[4] = {float2_to_bf16x2_bits(v[0], v[1]), float2_to_bf16x2_bits(v[2], v[3]),
                             float2_to_bf16x2_bits(v[4], v[5]), float2_to_bf16x2_bits(v[6], v[7])};
      const uint32_t t0 = valid & 4 ? w[2] : w[0], t1 = valid & 4 ? w[3] : w[1];
      if (valid & 4) *(GV2*)d = u32x2_t{w[0], w[1]};
      if (valid & 2) *(GV1*)(d + 2 * (valid & 4)) = t0;
      if (valid & 1) *(GH*)(d + 2 * (valid & 6)) = uint16_t(valid & 2 ? t1 : t0);
    }
  } else {
    if (valid >= 8) {
      u32x4_t x, y;
#pragma unroll
      for (int q = 0; q < 4; ++q) { x[q] = __float_as_uint(v[q]); y[q] = __float_as_uint(v[4 + q]); }
      *(GV*)d = x;
      *(GV*)(d + 16) = y;
    } else {
      const bool four = valid & 4, two = valid & 2;
      uint32_t t[3];
#pragma unroll
      for (int q = 0; q < 3; ++q) t[q] = __float_as_uint(four ? v[4 + q] : v[q]);
      if (four)
        *(GV*)d = u32x4_t{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])};
      if (two) *(GV2*)(d + 4 * (valid & 4)) = u32x2_t{t[0], t[1]};
      if (valid & 1) *(GV1*)(d + 4 * (valid & 6)) = two ? t[2] : t[0];
    }
  }
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

// The i-th elements of two runs of eight bfloat16, side by side.
__device__ __forceinline__ uint32_t pair_bf16(const Raw8& r0, const Raw8& r1, int i) {
  return __builtin_amdgcn_perm(r1.a[i / 2], r0.a[i / 2], i & 1 ? 0x07060302u : 0x05040100u);
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
template <int PA, int PB, int S = (PA > PB ? PA : PB) - 1>
__device__ __forceinline__ f32x4_t mfma_parts(const bf16x8_t a[PA], const bf16x8_t b[PB], f32x4_t acc) {
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
