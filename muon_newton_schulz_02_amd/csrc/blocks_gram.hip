// Gram pass of the block operators: per block, G = x x^T over a range of the
// n columns (x unnormalised, wide orientation m x n), for the gradient also
// Z = y x^T, for the step after the momentum update of the elements it reads.
//
// One workgroup takes `gchunk` columns of one block, KC at a time: its four
// waves load a tile of x (each element once), split the elements into PL
// bfloat16 parts and put them into LDS with k (the column) contiguous, then
// each wave multiplies its 16 x 16 tiles with 16x16x32 MFMAs.  G is
// symmetric: only tiles on or above the diagonal are formed, dealt out as
// tile rows {p, MT-1-p}, MT + 1 tiles for each of the MT/2 pairs.  With fewer
// than 8 tile rows the waves also share out the columns of a tile (KW = 8/MT
// ways), each way a partial of its own.  Partials are summed in a fixed order
// by the recursion kernel.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "blocks_device.h"

#pragma clang fp contract(off)

namespace muon {
namespace {

constexpr int GT = 256;  // threads

// Eight consecutive elements of x (mat 0) or y (mat 1), `valid` of which
// exist; for the step U, after the momentum is updated in place.
template <int KIND>
__device__ __forceinline__ void load_tile(const BlockStack& st, int mat, int64_t xe, int64_t ye, int valid,
                                          int64_t xs, int64_t ys, const BlockMom& mom, float v[8]) {
  const bool xbf = st.flags & BF_X_BF16, ybf = st.flags & BF_Y_BF16;
  const bool vec = valid >= 8 && (st.flags & (mat ? BF_Y_VEC : BF_X_VEC));
  if (mat == 0) {
    if (vec) load_vec<8>(st.x, xbf, xe, v);
    else load_masked<8>(st.x, xbf, xe, valid, xs, v);
    if (KIND == BK_STEP) {
      float* mo = reinterpret_cast<float*>(const_cast<void*>(st.y));
      float m[8];
      if (valid >= 8 && (st.flags & BF_Y_VEC)) {
        load_vec<8>(mo, false, ye, m);
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] = momentum_elem(v[q], m[q], mom);
        store_vec<8>(mo, false, ye, m);
      } else {
        load_masked<8>(mo, false, ye, valid, ys, m);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          v[q] = momentum_elem(v[q], m[q], mom);
          if (q < valid) gmem(mo)[ye + q] = m[q];
        }
      }
    }
  } else {
    if (vec) load_vec<8>(st.y, ybf, ye, v);
    else load_masked<8>(st.y, ybf, ye, valid, ys, v);
  }
}

template <int MT, int PL, int KIND>
__global__ __launch_bounds__(GT, 2) void block_gram_kernel(BlockTable tab, float* __restrict__ partials,
                                                           BlockMom mom) {
  constexpr int MP = 16 * MT, KC = block_kc(MT), KW = block_kw(MT), LDK = KC + 8;
  constexpr int NM = KIND == BK_VJP ? 2 : 1;       // matrices staged: x (and y)
  constexpr int KS = KC / 32 / KW;                 // k-steps of 32 per wave and tile
  __shared__ __attribute__((aligned(16))) uint16_t lds[NM][PL][MP][LDK];

  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int r = lane & 15, g = lane >> 4;
  const BlockStack st = find_stack(tab, blockIdx.x, [](const BlockStack& s) { return s.goff; });
  const int local = int(blockIdx.x) - st.goff;
  const int b = local / st.gsplit, sp = local - b * st.gsplit;
  const int k0 = sp * st.gchunk, k1 = min(st.n, k0 + st.gchunk);
  const int64_t xo = int64_t(b) * st.x_bs, yo = int64_t(b) * st.y_bs;

  const int p = wave % (MT / 2), kw = wave / (MT / 2);
  f32x4_t acc[MT + 1];
#pragma unroll
  for (int q = 0; q <= MT; ++q) acc[q] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  f32x4_t zacc[KIND == BK_VJP ? 2 * MT : 1];
#pragma unroll
  for (int q = 0; q < (KIND == BK_VJP ? 2 * MT : 1); ++q) zacc[q] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  for (int kb = k0; kb < k1; kb += KC) {
    const int kn = min(KC, k1 - kb);  // columns of this tile
    if (kb > k0) __syncthreads();     // the last tile's reads are done
    if (!(st.flags & BF_TR)) {
      // rows contiguous along k: a thread takes 8 columns of one row
      constexpr int UNITS = MP * (KC / 8);
#pragma unroll
      for (int u0 = 0; u0 < UNITS; u0 += GT) {
        const int u = u0 + tid, row = u / (KC / 8), kk = (u % (KC / 8)) * 8;
        const int valid = row < st.m ? kn - kk : 0;
        bf16x8_t o[PL];
#pragma unroll
        for (int mat = 0; mat < NM; ++mat) {
          float v[8];
          load_tile<KIND>(st, mat, xo + int64_t(row) * st.x_ld + kb + kk, yo + int64_t(row) * st.y_ld + kb + kk, valid,
                          xo, yo, mom, v);
          split8<PL>(v, o);
#pragma unroll
          for (int l = 0; l < PL; ++l) *reinterpret_cast<bf16x8_t*>(&lds[mat][l][row][kk]) = o[l];
        }
      }
    } else {
      // contiguous along i: a thread takes 8 rows (i) of 4 columns (k)
      constexpr int UNITS = (MP / 8) * (KC / 4);
      if (UNITS >= GT || tid < UNITS) {
        const int i0 = (tid % (MP / 8)) * 8, kk = (tid / (MP / 8)) * 4;
#pragma unroll
        for (int mat = 0; mat < NM; ++mat) {
          float v[4][8];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            load_tile<KIND>(st, mat, xo + int64_t(kb + kk + k) * st.x_ld + i0, yo + int64_t(kb + kk + k) * st.y_ld + i0,
                            kk + k < kn ? st.m - i0 : 0, xo, yo, mom, v[k]);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            uint32_t p01[PL], p23[PL];
            split2<PL>(v[0][i], v[1][i], p01);
            split2<PL>(v[2][i], v[3][i], p23);
#pragma unroll
            for (int l = 0; l < PL; ++l)
              *reinterpret_cast<u32x2_t*>(&lds[mat][l][i0 + i][kk]) = u32x2_t{p01[l], p23[l]};
          }
        }
      }
      static_assert(UNITS <= GT, "one unit per thread");
    }
    __syncthreads();
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      const int ko = (kw * KS + ks) * 32 + 8 * g;
      bf16x8_t a0[PL], a1[PL];
#pragma unroll
      for (int l = 0; l < PL; ++l) {
        a0[l] = *reinterpret_cast<const bf16x8_t*>(&lds[0][l][16 * p + r][ko]);
        a1[l] = *reinterpret_cast<const bf16x8_t*>(&lds[0][l][16 * (MT - 1 - p) + r][ko]);
      }
#pragma unroll
      for (int q = 0; q <= MT; ++q) {
        const bool row0 = q < MT - p;
        const int tj = row0 ? p + q : MT - 1 - p + (q - (MT - p));
        bf16x8_t bb[PL];
#pragma unroll
        for (int l = 0; l < PL; ++l) bb[l] = *reinterpret_cast<const bf16x8_t*>(&lds[0][l][16 * tj + r][ko]);
        if (row0) acc[q] = mfma_parts<PL, PL>(a0, bb, acc[q]);
        else acc[q] = mfma_parts<PL, PL>(a1, bb, acc[q]);
      }
      if (KIND == BK_VJP) {
#pragma unroll
        for (int l = 0; l < PL; ++l) {
          a0[l] = *reinterpret_cast<const bf16x8_t*>(&lds[NM - 1][l][16 * p + r][ko]);
          a1[l] = *reinterpret_cast<const bf16x8_t*>(&lds[NM - 1][l][16 * (MT - 1 - p) + r][ko]);
        }
#pragma unroll
        for (int tj = 0; tj < MT; ++tj) {
          bf16x8_t bb[PL];
#pragma unroll
          for (int l = 0; l < PL; ++l) bb[l] = *reinterpret_cast<const bf16x8_t*>(&lds[0][l][16 * tj + r][ko]);
          zacc[tj] = mfma_parts<PL, PL>(a0, bb, zacc[tj]);
          zacc[MT + tj] = mfma_parts<PL, PL>(a1, bb, zacc[MT + tj]);
        }
      }
    }
  }

  constexpr int PF = block_part_floats(MT, KIND);
  float* out = partials + st.part0 + (int64_t(b) * (st.gsplit * KW) + sp * KW + kw) * PF;
#pragma unroll
  for (int q = 0; q <= MT; ++q)
    *gmem(reinterpret_cast<f32x4_t*>(out + ((p * (MT + 1) + q) * 64 + lane) * 4)) = acc[q];
  if (KIND == BK_VJP) {
    out += (MT / 2) * (MT + 1) * 256;
#pragma unroll
    for (int q = 0; q < 2 * MT; ++q)
      *gmem(reinterpret_cast<f32x4_t*>(out + ((p * 2 * MT + q) * 64 + lane) * 4)) = zacc[q];
  }
}

struct BlockStackBatch {
  BlockStack s[BLOCK_INLINE];
};

__global__ void block_table_kernel(BlockStackBatch in, int32_t n, BlockStack* __restrict__ out) {
  const int i = threadIdx.x;
  if (i < n) out[i] = in.s[i];
}

template <int MT>
hipError_t gram_mt(int pl, int kind, const BlockTable& tab, int32_t wgs, float* partials, const BlockMom& mom,
                   hipStream_t stream) {
#define MUON_GRAM(PL, KIND)                                                                                   \
  if (pl == PL && kind == KIND) {                                                                             \
    hipLaunchKernelGGL((block_gram_kernel<MT, PL, KIND>), dim3(wgs), dim3(GT), 0, stream, tab, partials, mom); \
    return hipGetLastError();                                                                                 \
  }
  MUON_GRAM(1, BK_X)
  MUON_GRAM(2, BK_X)
  MUON_GRAM(3, BK_X)
  MUON_GRAM(2, BK_STEP)
  MUON_GRAM(3, BK_STEP)
  MUON_GRAM(1, BK_VJP)
  MUON_GRAM(2, BK_VJP)
  MUON_GRAM(3, BK_VJP)
#undef MUON_GRAM
  return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_block_table(const BlockStack* host, int32_t count, BlockStack* dev, hipStream_t stream) {
  for (int32_t i = 0; i < count; i += BLOCK_INLINE) {
    BlockStackBatch batch = {};
    const int32_t n = count - i < BLOCK_INLINE ? count - i : BLOCK_INLINE;
    for (int32_t k = 0; k < n; ++k) batch.s[k] = host[i + k];
    hipLaunchKernelGGL(block_table_kernel, dim3(1), dim3(64), 0, stream, batch, n, dev + i);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_block_gram(int mt, int pl, int kind, const BlockTable& tab, int32_t wgs, float* partials,
                             const BlockMom& mom, hipStream_t stream) {
  if (wgs <= 0) return hipSuccess;
  return mt == 2   ? gram_mt<2>(pl, kind, tab, wgs, partials, mom, stream)
         : mt == 4 ? gram_mt<4>(pl, kind, tab, wgs, partials, mom, stream)
                   : gram_mt<8>(pl, kind, tab, wgs, partials, mom, stream);
}

}  // namespace muon
