// The m x m recursion of the block operators, one workgroup per block:
//   A_0 = s^2 G ; Q = a I + b A + c A A ; P <- Q P ; A <- Q A Q
// with s = 1 / (||x|| + 1e-7), ||x||^2 the trace of G.  For the gradient also
// its tangent from D_0 = s sym(Z), Z = y x^T:
//   dQ = b D + c (D A + A D) ; dP <- dQ P + Q dP ; D <- dQ A Q + Q D Q + Q A dQ
// P and dP end as the polynomial at A_0 and its derivative in direction D_0;
// every matrix is a function of A_0, so the order of factors is free and the
// derivative is its own adjoint.
//
// Products run on v_mfma_f32_16x16x32_f16 with every operand split into two
// binary16 parts (22 bits) and three products, hi*hi + hi*lo + lo*hi, summed
// in binary32.  A panel of 16 columns is scaled by a power of two first, so
// that its largest element lies in [2^14, 2^15): parts of smaller elements
// then stay exact down to 2^-39 of it, and no matrix overflows the format.
// Against binary32 products (v_mfma_f32_16x16x4f32) the results' errors are
// the same to a factor of 1.3 (they come from the Gram matrix), at 3/16 of
// the matrix-core time: 48 blocks of 128 x 1536, 161 us before.
//
// Wave w of MT holds column panel w of every matrix in its registers, as the
// accumulator tiles of the products.  Two such tiles, one above the other,
// are at the same time the B operand of a later product's k-step of 32, with
// k taken in the order 32 kk + {4 g + v, 16 + 4 g + v} (g = lane / 16).  A
// product L R therefore needs only L in LDS, and as every matrix is symmetric
// but for rounding, row i of L is column i: the operand registers are stored
// as they are, 16 bytes a lane, and read back the same way by every wave.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "blocks_device.h"

#pragma clang fp contract(off)

namespace muon {
namespace {

constexpr float NORM_EPS = 1e-7f;

typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));

// A column panel as product operand: hi and lo parts per k-step of 32, and
// the power of two the values were multiplied with (the same in all lanes).
template <int MT>
struct Operand {
  f16x8_t f[MT / 2][2];
  int ex;
};

// The largest bits of a non-negative float over the wave, in a scalar register.
__device__ __forceinline__ uint32_t wave_max_bits(float v) {
  // rows of 16 lanes by rotation, then the four rows
#define MUON_ROW_MAX(ctl) \
  v = fmaxf(v, __uint_as_float(__builtin_amdgcn_update_dpp(0, int(__float_as_uint(v)), ctl, 0xF, 0xF, false)))
  MUON_ROW_MAX(0x128);  // row_ror:8
  MUON_ROW_MAX(0x124);
  MUON_ROW_MAX(0x122);
  MUON_ROW_MAX(0x121);
#undef MUON_ROW_MAX
  const uint32_t b = __float_as_uint(v);
  uint32_t m = __builtin_amdgcn_readlane(b, 0);
  m = max(m, uint32_t(__builtin_amdgcn_readlane(b, 16)));
  m = max(m, uint32_t(__builtin_amdgcn_readlane(b, 32)));
  return max(m, uint32_t(__builtin_amdgcn_readlane(b, 48)));
}

template <int MT>
__device__ __forceinline__ void split_panel(const f32x4_t (&X)[MT], Operand<MT>& o) {
  float mx = 0.f;
#pragma unroll
  for (int kt = 0; kt < MT; ++kt)
#pragma unroll
    for (int v = 0; v < 4; ++v) mx = fmaxf(mx, __builtin_fabsf(X[kt][v]));
  // mx in [2^e, 2^(e + 1)) goes to [2^14, 2^15) (subnormals and zero below it)
  o.ex = 14 + 127 - int(wave_max_bits(mx) >> 23);
#pragma unroll
  for (int kk = 0; kk < MT / 2; ++kk) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int v = 0; v < 4; v += 2) {
        const f32x2_t x = {__builtin_amdgcn_ldexpf(X[2 * kk + h][v], o.ex),
                           __builtin_amdgcn_ldexpf(X[2 * kk + h][v + 1], o.ex)};
        const f16x2_t hi = __builtin_convertvector(x, f16x2_t);
        const f32x2_t rest = {x[0] - float(hi[0]), x[1] - float(hi[1])};
        const f16x2_t lo = __builtin_convertvector(rest, f16x2_t);
        o.f[kk][0][4 * h + v] = hi[0];
        o.f[kk][0][4 * h + v + 1] = hi[1];
        o.f[kk][1][4 * h + v] = lo[0];
        o.f[kk][1][4 * h + v + 1] = lo[1];
      }
  }
}

// A matrix in LDS: row i holds column i of the matrix, two parts.
template <int MT>
struct Left {
  uint16_t v[2][16 * MT][16 * MT + 8];
  int32_t ex[MT];
};

template <int MT>
__device__ __forceinline__ void put_panel(Left<MT>& L, const Operand<MT>& o, int panel, int r, int g, int lane) {
#pragma unroll
  for (int kk = 0; kk < MT / 2; ++kk)
#pragma unroll
    for (int l = 0; l < 2; ++l)
      *reinterpret_cast<f16x8_t*>(&L.v[l][16 * panel + r][32 * kk + 8 * g]) = o.f[kk][l];
  if (lane == 0) L.ex[panel] = o.ex;
}

// acc = L X for the wave's panel X: MT independent sums.
template <int MT>
__device__ __forceinline__ void multiply(f32x4_t (&acc)[MT], const Left<MT>& L, const Operand<MT>& X, int r, int g) {
#pragma unroll
  for (int jt = 0; jt < MT; ++jt) acc[jt] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int kk = 0; kk < MT / 2; ++kk) {
#pragma unroll
    for (int jt = 0; jt < MT; ++jt) {
      const f16x8_t hi = *reinterpret_cast<const f16x8_t*>(&L.v[0][16 * jt + r][32 * kk + 8 * g]);
      const f16x8_t lo = *reinterpret_cast<const f16x8_t*>(&L.v[1][16 * jt + r][32 * kk + 8 * g]);
      acc[jt] = __builtin_amdgcn_mfma_f32_16x16x32_f16(lo, X.f[kk][0], acc[jt], 0, 0, 0);
      acc[jt] = __builtin_amdgcn_mfma_f32_16x16x32_f16(hi, X.f[kk][1], acc[jt], 0, 0, 0);
      acc[jt] = __builtin_amdgcn_mfma_f32_16x16x32_f16(hi, X.f[kk][0], acc[jt], 0, 0, 0);
    }
    if (MT >= 4) __builtin_amdgcn_sched_barrier(0);  // bounds how far the reads of L are hoisted
  }
#pragma unroll
  for (int jt = 0; jt < MT; ++jt) {
    const int e = -(L.ex[jt] + X.ex);
#pragma unroll
    for (int v = 0; v < 4; ++v) acc[jt][v] = __builtin_amdgcn_ldexpf(acc[jt][v], e);
  }
}

template <int MT, int KIND>
__global__ __launch_bounds__(64 * MT, 2) void block_iterate_kernel(
    BlockTable tab, const float* __restrict__ partials, uint16_t* __restrict__ p_out, uint16_t* __restrict__ t_out,
    float* __restrict__ scratch, BlockSteps steps, int32_t pp) {
  constexpr int MP = 16 * MT, NT = 64 * MT;
  constexpr bool VJP = KIND == BK_VJP;
  constexpr int LDM = MP + 4;
  // the Gram matrix (and Z) in binary32 first, then the left factors
  union Lds {
    float gram[VJP ? 2 : 1][MP][LDM];
    Left<MT> left[VJP ? 2 : 1];
  };
  __shared__ __attribute__((aligned(16))) Lds lds;
  __shared__ float red[8];

  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const int r = lane & 15, g = lane >> 4;
  const int blk = blockIdx.x;
  const BlockStack st = find_stack(&BlockStack::block0, blk);
  const int b = blk - st.block0;

  // sum the partials, in order, into LDS (both triangles)
  constexpr int PF = block_part_floats(MT, KIND);
  const int parts = st.gsplit;
  const float* src = partials + st.part0 + int64_t(b) * parts * PF;
  auto& L0 = lds.gram[0];
  auto& L1 = lds.gram[VJP ? 1 : 0];
  for (int e = tid; e < PF / 4; e += NT) {
    f32x4_t s = *gmem(reinterpret_cast<const f32x4_t*>(src + 4 * e));
#pragma unroll 4
    for (int q = 1; q < parts; ++q) s += *gmem(reinterpret_cast<const f32x4_t*>(src + int64_t(q) * PF + 4 * e));
    const int tile = e >> 6, rr = e & 15, gg = (e >> 4) & 3;
    constexpr int TRI = (MT / 2) * (MT + 1);
    if (!VJP || tile < TRI) {
      const int p = tile / (MT + 1), q = tile % (MT + 1);
      const int ti = q < MT - p ? p : MT - 1 - p, tj = q < MT - p ? p + q : MT - 1 - p + (q - (MT - p));
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int i = 16 * ti + 4 * gg + v, j = 16 * tj + rr;
        if (ti != tj || i <= j) {
          L0[i][j] = s[v];
          L0[j][i] = s[v];
        }
      }
    } else {
      const int z = tile - TRI, p = z / (2 * MT), q = z % (2 * MT);
      const int ti = q < MT ? p : MT - 1 - p, tj = q % MT;
#pragma unroll
      for (int v = 0; v < 4; ++v) L1[16 * ti + 4 * gg + v][16 * tj + rr] = s[v];
    }
  }
  __syncthreads();

  // ||x||^2
  float tr = 0.f;
  for (int i = lane; i < MP; i += 64) tr += L0[i][i];
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) tr += __shfl_xor(tr, d);
  const float norm = __builtin_sqrtf(tr);
  const float inv = steps.first ? 1.f / (norm + NORM_EPS) : 1.f;

  // A_j (and its tangent) in binary32; P lives as an operand only, and its
  // new value passes through A while A_j is one
  f32x4_t A[MT], D[VJP ? MT : 1];
#pragma unroll
  for (int kt = 0; kt < MT; ++kt)
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int i = 16 * kt + 4 * g + v, j = 16 * w + r;
      A[kt][v] = (L0[i][j] * inv) * inv;
      if constexpr (VJP) D[kt][v] = (0.5f * inv) * (L1[i][j] + L1[j][i]);
    }
  float* sc = nullptr;
  if constexpr (VJP) {
    // A_0 and D_0 are needed again for <dX_0, X_0>
    sc = scratch + int64_t(blk) * (2 * MP * MP) + 4 * tid;
#pragma unroll
    for (int kt = 0; kt < MT; ++kt) {
      *gmem(reinterpret_cast<f32x4_t*>(sc + kt * NT * 4)) = A[kt];
      *gmem(reinterpret_cast<f32x4_t*>(sc + (MT + kt) * NT * 4)) = D[kt];
    }
  }

  Left<MT>& LA = lds.left[0];
  Left<MT>& LD = lds.left[VJP ? 1 : 0];
  Operand<MT> oA, oP, oD, odP;  // oD, odP: the gradient's

  // A -> Q = a I + b A + c A A in its place (D -> dQ), A_t left in oA (oD)
  auto form_q = [&](int t) {
    const float ca = steps.a[t], cb = steps.b[t], cc = steps.c[t];
    split_panel<MT>(A, oA);
    if constexpr (VJP) split_panel<MT>(D, oD);
#pragma unroll
    for (int kt = 0; kt < MT; ++kt) {
      A[kt] *= cb;
      if constexpr (VJP) D[kt] *= cb;
    }
    if (cc != 0.f) {
      __syncthreads();  // the reads of LDS before are done
      put_panel<MT>(LA, oA, w, r, g, lane);
      if constexpr (VJP) put_panel<MT>(LD, oD, w, r, g, lane);
      __syncthreads();
      f32x4_t x[MT];
      multiply<MT>(x, LA, oA, r, g);
#pragma unroll
      for (int kt = 0; kt < MT; ++kt) A[kt] += cc * x[kt];
      if constexpr (VJP) {
        multiply<MT>(x, LA, oD, r, g);
#pragma unroll
        for (int kt = 0; kt < MT; ++kt) D[kt] += cc * x[kt];
        multiply<MT>(x, LD, oA, r, g);
#pragma unroll
        for (int kt = 0; kt < MT; ++kt) D[kt] += cc * x[kt];
      }
    }
#pragma unroll
    for (int kt = 0; kt < MT; ++kt)
#pragma unroll
      for (int v = 0; v < 4; ++v)
        if (16 * kt + 4 * g + v == 16 * w + r) A[kt][v] += ca;
  };
  // (A, D) <- L (o, od) and its tangent
  auto left_times = [&](const Operand<MT>& o, const Operand<MT>& od) {
    multiply<MT>(A, LA, o, r, g);
    if constexpr (VJP) {
      f32x4_t x[MT];
      multiply<MT>(D, LA, od, r, g);
      multiply<MT>(x, LD, o, r, g);
#pragma unroll
      for (int kt = 0; kt < MT; ++kt) D[kt] += x[kt];
    }
  };
  auto split_into = [&](Operand<MT>& o, Operand<MT>& od) {
    split_panel<MT>(A, o);
    if constexpr (VJP) split_panel<MT>(D, od);
  };
  if (steps.steps > 0) form_q(0);  // P = Q
  if (steps.steps > 1) {
    split_into(oP, odP);
    __syncthreads();
    put_panel<MT>(LA, oP, w, r, g, lane);
    if constexpr (VJP) put_panel<MT>(LD, odP, w, r, g, lane);
    __syncthreads();
#pragma unroll 1
    for (int t = 1; t < steps.steps; ++t) {
      left_times(oA, oD);  // R = Q A
      split_into(oA, oD);
      left_times(oA, oD);  // A <- Q R
      form_q(t);
      __syncthreads();
      {
        Operand<MT> o;
        split_panel<MT>(A, o);
        put_panel<MT>(LA, o, w, r, g, lane);
        if constexpr (VJP) {
          split_panel<MT>(D, o);
          put_panel<MT>(LD, o, w, r, g, lane);
        }
      }
      __syncthreads();
      left_times(oP, odP);  // P <- Q P
      split_into(oP, odP);
    }
  }
  // P is in A, dP in D
  if (steps.steps == 0) {
#pragma unroll
    for (int kt = 0; kt < MT; ++kt)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        A[kt][v] = 16 * kt + 4 * g + v == 16 * w + r ? 1.f : 0.f;
        if constexpr (VJP) D[kt][v] = 0.f;
      }
  }

  if constexpr (VJP) {
    float shift = 0.f;
    if (steps.first) {
      // <dX_0, X_0> = <P, D_0> + <2 dP, A_0>
      float k = 0.f;
#pragma unroll
      for (int kt = 0; kt < MT; ++kt) {
        const f32x4_t a0 = *gmem(reinterpret_cast<const f32x4_t*>(sc + kt * NT * 4));
        const f32x4_t d0 = *gmem(reinterpret_cast<const f32x4_t*>(sc + (MT + kt) * NT * 4));
#pragma unroll
        for (int v = 0; v < 4; ++v) k += A[kt][v] * d0[v] + 2.f * D[kt][v] * a0[v];
      }
#pragma unroll
      for (int d = 32; d > 0; d >>= 1) k += __shfl_xor(k, d);
      if (lane == 0) red[w] = k;
      __syncthreads();
      k = 0.f;
#pragma unroll
      for (int q = 0; q < MT; ++q) k += red[q];
      // a zero block has no direction: the norm's gradient is taken as zero
      shift = norm > 0.f ? inv * (k / norm) : 0.f;
    }
#pragma unroll
    for (int kt = 0; kt < MT; ++kt)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const float tt = (2.f * D[kt][v]) * inv * inv;
        D[kt][v] = 16 * kt + 4 * g + v == 16 * w + r ? tt - shift : tt;
      }
  }
#pragma unroll
  for (int kt = 0; kt < MT; ++kt) A[kt] *= inv;

  // out in bfloat16 parts, by rows, through LDS.  P X is not P^T X here: P is
  // the product Q_k ... Q_0, whose last factors carry the largest errors, and
  // they act on what the first ones have left of X's large singular values
  __syncthreads();
#pragma unroll
  for (int kt = 0; kt < MT; ++kt)
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      L0[16 * kt + 4 * g + v][16 * w + r] = A[kt][v];
      if constexpr (VJP) L1[16 * kt + 4 * g + v][16 * w + r] = D[kt][v];
    }
  __syncthreads();
#pragma unroll
  for (int mat = 0; mat < (VJP ? 2 : 1); ++mat) {
    uint16_t* out = (mat ? t_out : p_out) + int64_t(blk) * pp * (MP * MP);
#pragma unroll 2
    for (int u = tid; u < MP * (MP / 8); u += NT) {
      const int row = u / (MP / 8), col = (u % (MP / 8)) * 8;
      const f32x4_t x0 = *reinterpret_cast<const f32x4_t*>(&lds.gram[mat][row][col]);
      const f32x4_t x1 = *reinterpret_cast<const f32x4_t*>(&lds.gram[mat][row][col + 4]);
      const float v[8] = {x0[0], x0[1], x0[2], x0[3], x1[0], x1[1], x1[2], x1[3]};
      bf16x8_t o[3];
      split8<3>(v, o);
#pragma unroll
      for (int l = 0; l < 3; ++l)
        if (l < pp) *gmem(reinterpret_cast<bf16x8_t*>(out + l * (MP * MP) + row * MP + col)) = o[l];
    }
  }
}

}  // namespace

hipError_t launch_block_iterate(int mt, int pp, int kind, const BlockTable& tab, int32_t blocks,
                                const float* partials, uint16_t* p_out, uint16_t* t_out, float* scratch,
                                const BlockSteps& steps, hipStream_t stream) {
  if (blocks <= 0) return hipSuccess;
#define MUON_ITER(MT, KIND)                                                                                      \
  if (mt == MT && kind == KIND) {                                                                                \
    hipLaunchKernelGGL((block_iterate_kernel<MT, KIND>), dim3(blocks), dim3(64 * MT), 0, stream, tab, partials,  \
                       p_out, t_out, scratch, steps, pp);                                                        \
    return hipGetLastError();                                                                                    \
  }
  MUON_ITER(2, BK_X)
  MUON_ITER(4, BK_X)
  MUON_ITER(8, BK_X)
  MUON_ITER(2, BK_VJP)
  MUON_ITER(4, BK_VJP)
  MUON_ITER(8, BK_VJP)
#undef MUON_ITER
  return hipErrorInvalidValue;
}

}  // namespace muon
