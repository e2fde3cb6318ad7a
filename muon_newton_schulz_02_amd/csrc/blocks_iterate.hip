// The m x m recursion of the block operators, one workgroup per block:
//   A_0 = s^2 G ; Q = a I + b A + c A A ; P <- Q P ; A <- Q A Q
// with s = 1 / (||x|| + 1e-7), ||x||^2 the trace of G.  For the gradient also
// its tangent from D_0 = s sym(Z), Z = y x^T:
//   dQ = b D + c (D A + A D) ; dP <- dQ P + Q dP ; D <- dQ A Q + Q D Q + Q A dQ
// P and dP end as the polynomial at A_0 and its derivative in direction D_0;
// every matrix is a function of A_0, so the order of factors is free and the
// derivative is its own adjoint.
//
// Wave w of MT holds column panel w (16 columns) of every matrix in its
// registers, as the MT accumulator tiles of v_mfma_f32_16x16x4f32: such a
// tile is at the same time the B operand of the next product with k taken in
// the order 16 kt + 4 (lane / 16) + v, so a product L R only needs L in LDS,
// read along its rows 16 bytes a lane.  Within a step the left factors are A
// (and D), then Q (and dQ).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "blocks_device.h"

#pragma clang fp contract(off)

namespace muon {
namespace {

constexpr float NORM_EPS = 1e-7f;

template <int MT, int KIND>
__global__ __launch_bounds__(64 * MT) void block_iterate_kernel(BlockTable tab, const float* __restrict__ partials,
                                                                uint16_t* __restrict__ p_out,
                                                                uint16_t* __restrict__ t_out,
                                                                float* __restrict__ scratch, BlockSteps steps,
                                                                int32_t pp) {
  constexpr int MP = 16 * MT, LDM = MP + 4, NT = 64 * MT, KW = block_kw(MT);
  constexpr bool VJP = KIND == BK_VJP;
  __shared__ __attribute__((aligned(16))) float L0[MP][LDM];
  __shared__ __attribute__((aligned(16))) float L1[VJP ? MP : 1][LDM];
  __shared__ float red[8];

  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const int r = lane & 15, g = lane >> 4;
  const int blk = blockIdx.x;
  const BlockStack st = find_stack(tab, blk, [](const BlockStack& s) { return s.block0; });
  const int b = blk - st.block0;

  // sum the partials, in order, into LDS (both triangles)
  constexpr int PF = block_part_floats(MT, KIND);
  const int parts = st.gsplit * KW;
  const float* src = partials + st.part0 + int64_t(b) * parts * PF;
  for (int e = tid; e < PF / 4; e += NT) {
    f32x4_t s = *gmem(reinterpret_cast<const f32x4_t*>(src + 4 * e));
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

  f32x4_t A[MT], P[MT], D[VJP ? MT : 1], dP[VJP ? MT : 1];
#pragma unroll
  for (int kt = 0; kt < MT; ++kt)
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int i = 16 * kt + 4 * g + v, j = 16 * w + r;
      A[kt][v] = (L0[i][j] * inv) * inv;
      P[kt][v] = i == j ? 1.f : 0.f;
      if (VJP) {
        D[kt][v] = (0.5f * inv) * (L1[i][j] + L1[j][i]);
        dP[kt][v] = 0.f;
      }
    }
  float* sc = nullptr;
  if (VJP) {
    // A_0 and D_0 are needed again for <dX_0, X_0>
    sc = scratch + int64_t(blk) * (2 * MP * MP);
#pragma unroll
    for (int kt = 0; kt < MT; ++kt) {
      *gmem(reinterpret_cast<f32x4_t*>(sc + (kt * NT + tid) * 4)) = A[kt];
      *gmem(reinterpret_cast<f32x4_t*>(sc + ((MT + kt) * NT + tid) * 4)) = D[kt];
    }
  }

  auto put = [&](float (*L)[LDM], const f32x4_t* X) {
#pragma unroll
    for (int kt = 0; kt < MT; ++kt)
#pragma unroll
      for (int v = 0; v < 4; ++v) L[16 * kt + 4 * g + v][16 * w + r] = X[kt][v];
  };
  // C += L X
  auto mul = [&](f32x4_t* C, const float (*L)[LDM], const f32x4_t* X) {
#pragma unroll
    for (int jt = 0; jt < MT; ++jt)
#pragma unroll
      for (int kt = 0; kt < MT; ++kt) {
        const f32x4_t l = *reinterpret_cast<const f32x4_t*>(&L[16 * jt + r][16 * kt + 4 * g]);
#pragma unroll
        for (int v = 0; v < 4; ++v) C[jt] = __builtin_amdgcn_mfma_f32_16x16x4f32(l[v], X[kt][v], C[jt], 0, 0, 0);
        // without a bound on how far the reads of L are hoisted they spill
        if (MT == 8 && kt % 4 == 3) __builtin_amdgcn_sched_barrier(0);
      }
  };
  auto zero = [&](f32x4_t* C) {
#pragma unroll
    for (int kt = 0; kt < MT; ++kt) C[kt] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  };

  for (int t = 0; t < steps.steps; ++t) {
    const float ca = steps.a[t], cb = steps.b[t], cc = steps.c[t];
    const bool last = t + 1 == steps.steps;
    f32x4_t Q[MT], dQ[VJP ? MT : 1];
    zero(Q);
    if (VJP) zero(dQ);
    if (cc != 0.f) {
      __syncthreads();  // the reads of the step before are done
      put(L0, A);
      if (VJP) put(L1, D);
      __syncthreads();
      mul(Q, L0, A);
      if (VJP) {
        mul(dQ, L0, D);
        mul(dQ, L1, A);
      }
    }
#pragma unroll
    for (int kt = 0; kt < MT; ++kt)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const float q = cb * A[kt][v] + cc * Q[kt][v];
        Q[kt][v] = 16 * kt + 4 * g + v == 16 * w + r ? ca + q : q;
        if (VJP) dQ[kt][v] = cb * D[kt][v] + cc * dQ[kt][v];
      }
    __syncthreads();
    put(L0, Q);
    if (VJP) put(L1, dQ);
    __syncthreads();
    {
      f32x4_t N[MT], dN[VJP ? MT : 1];
      zero(N);
      mul(N, L0, P);
      if (VJP) {
        zero(dN);
        mul(dN, L0, dP);
        mul(dN, L1, P);
#pragma unroll
        for (int kt = 0; kt < MT; ++kt) dP[kt] = dN[kt];
      }
#pragma unroll
      for (int kt = 0; kt < MT; ++kt) P[kt] = N[kt];
    }
    if (!last) {
      f32x4_t R[MT], dR[VJP ? MT : 1];
      zero(R);
      mul(R, L0, A);
      if (VJP) {
        zero(dR);
        mul(dR, L0, D);
        mul(dR, L1, A);
      }
      zero(A);
      mul(A, L0, R);
      if (VJP) {
        zero(D);
        mul(D, L0, dR);
        mul(D, L1, R);
      }
    }
  }

  // P in bfloat16 parts (the panel's transpose: four consecutive columns of
  // row 16 w + r; P is symmetric)
  auto emit = [&](uint16_t* out, const f32x4_t* X) {
    out += int64_t(blk) * pp * (MP * MP);
#pragma unroll
    for (int kt = 0; kt < MT; ++kt) {
      uint32_t p01[3], p23[3];
      split2<3>(X[kt][0], X[kt][1], p01);
      split2<3>(X[kt][2], X[kt][3], p23);
#pragma unroll
      for (int l = 0; l < 3; ++l)
        if (l < pp)
          *gmem(reinterpret_cast<u32x2_t*>(out + (l * MP + 16 * w + r) * MP + 16 * kt + 4 * g)) =
              u32x2_t{p01[l], p23[l]};
    }
  };
  if (VJP) {
    float shift = 0.f;
    if (steps.first) {
      // <dX_0, X_0> = <P, D_0> + <2 dP, A_0>
      float k = 0.f;
#pragma unroll
      for (int kt = 0; kt < MT; ++kt) {
        const f32x4_t a0 = *gmem(reinterpret_cast<const f32x4_t*>(sc + (kt * NT + tid) * 4));
        const f32x4_t d0 = *gmem(reinterpret_cast<const f32x4_t*>(sc + ((MT + kt) * NT + tid) * 4));
#pragma unroll
        for (int v = 0; v < 4; ++v) k += P[kt][v] * d0[v] + 2.f * dP[kt][v] * a0[v];
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
        const float tt = (2.f * dP[kt][v]) * inv * inv;
        dP[kt][v] = 16 * kt + 4 * g + v == 16 * w + r ? tt - shift : tt;
      }
    emit(t_out, dP);
  }
#pragma unroll
  for (int kt = 0; kt < MT; ++kt)
#pragma unroll
    for (int v = 0; v < 4; ++v) P[kt][v] = P[kt][v] * inv;
  emit(p_out, P);
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
