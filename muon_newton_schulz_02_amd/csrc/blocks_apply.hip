// Apply pass of the block operators: per block, O = P x (m x m by m x n), for
// the gradient O = P y + T x, for the step with x formed again from the
// gradient and the updated momentum; then the store, or the write-back
//   W <- rnd(fl32(W d) - fl32(t O)).
//
// A workgroup keeps P in LDS (PP bfloat16 parts, rows along k) and walks its
// columns in strips of 256, 64 for each of its four waves.  x needs no LDS:
// a lane loads runs of 4 columns from 8 rows (or, where columns are
// contiguous, 8 rows of one column) and so holds, after the split into parts,
// whole operands of v_mfma_f32_16x16x32_bf16 with the tile's columns
// interleaved: column 4 r + t of the strip is column r of tile t, so that a
// lane's results for the four tiles are four consecutive columns again.
// Where the block is stored transposed (rows > cols) the roles of the
// operands change, and rows of P are interleaved the same way in LDS.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "blocks_device.h"

#pragma clang fp contract(off)

namespace muon {
namespace {

constexpr int AT = 256;  // threads

// One run of results: N consecutive elements of a row of the output, element
// e of it and element ue of the exported update.
template <int N, bool VEC>
__device__ __forceinline__ void finish_run(const BlockStack& st, int64_t e, int64_t ue, int valid, float o[N]) {
  const bool bf = st.flags & BF_OUT_BF16;
  if (st.flags & BF_WRITEBACK) {
    float wv[N];
    if (st.upd) {
#pragma unroll
      for (int q = 0; q < N; ++q)
        if (VEC || q < valid) gmem(st.upd)[ue + q] = o[q];
    }
    if constexpr (VEC && N >= 4) load_vec<N>(st.out, bf, e, wv);
    else {
#pragma unroll
      for (int q = 0; q < N; ++q) wv[q] = load1f(st.out, bf, e + (VEC || q < valid ? q : 0));
    }
#pragma unroll
    for (int q = 0; q < N; ++q) {
      const float wd = wv[q] * st.d;
      const float to = st.t * o[q];
      o[q] = wd - to;
    }
  }
  if constexpr (VEC) store_vec<N>(st.out, bf, e, o);
  else {
#pragma unroll
    for (int q = 0; q < N; ++q)
      if (q < valid) store1f(st.out, bf, e + q, o[q]);
  }
}

// A strided matrix of the caller's: rows of ld elements from `base`.
struct View {
  const void* p;
  int64_t base, ld;
  bool bf, vec;
};

// N consecutive elements from (row, col); `valid` of them exist.
template <int N, bool FAST, int SRC>
__device__ __forceinline__ void load_x(const View& x, const View& mo, int row, int col, int valid,
                                       const BlockMom& mom, float v[N]) {
  const int64_t e = x.base + int64_t(row) * x.ld + col;
  if constexpr (FAST) load_vec<N>(x.p, x.bf, e, v);
  else load_masked<N>(x.p, x.bf, e, valid, x.base, v);
  if constexpr (SRC == BK_STEP) {
    float m[N];
    const int64_t me = mo.base + int64_t(row) * mo.ld + col;
    if constexpr (FAST) load_vec<N>(mo.p, false, me, m);
    else load_masked<N>(mo.p, false, me, valid, mo.base, m);
#pragma unroll
    for (int q = 0; q < N; ++q) v[q] = momentum_dir(v[q], m[q], mom);
  }
}

// The operands of one k-step of 32 for the 64 columns from j0.
template <int PL, bool TR, bool FAST, int SRC>
__device__ __forceinline__ void load_operands(bf16x8_t (&x)[4][PL], const View& xs, const View& mo, int m, int n,
                                              int kk, int j0, const BlockMom& mom, int r, int g) {
  if constexpr (!TR) {
    float v[8][4];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int row = 32 * kk + 8 * g + e, col = j0 + 4 * r;
      load_x<4, FAST, SRC>(xs, mo, row, col, row < m ? n - col : 0, mom, v[e]);
    }
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const float c[8] = {v[0][t], v[1][t], v[2][t], v[3][t], v[4][t], v[5][t], v[6][t], v[7][t]};
      split8<PL>(c, x[t]);
    }
  } else {
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      float v[8];
      const int j = j0 + 16 * t + r, i0 = 32 * kk + 8 * g;
      load_x<8, FAST, SRC>(xs, mo, j, i0, j < n ? m - i0 : 0, mom, v);
      split8<PL>(v, x[t]);
    }
  }
}

// acc += F x over the 64 columns from j0; F in LDS.  SRC: BK_X reads xs,
// BK_STEP forms U from xs (gradient) and mo (updated momentum).
template <int MT, int PL, int PP, bool TR, int SRC>
__device__ __forceinline__ void strip_product(f32x4_t (&acc)[MT][4], const uint16_t* F, const View& xs,
                                              const View& mo, int m, int n, int j0, const BlockMom& mom, int r,
                                              int g) {
  constexpr int MP = 16 * MT, LDP = MP + 8;
  asm volatile("" : "+v"(r), "+v"(g));  // as in finish_strip
  const bool vec = xs.vec && (SRC != BK_STEP || mo.vec) && j0 + 64 <= n;
#pragma unroll 1
  for (int kk = 0; kk < MP / 32; ++kk) {
    bf16x8_t x[4][PL];
    if (vec && 32 * kk + 32 <= m) load_operands<PL, TR, true, SRC>(x, xs, mo, m, n, kk, j0, mom, r, g);
    else load_operands<PL, TR, false, SRC>(x, xs, mo, m, n, kk, j0, mom, r, g);
#pragma unroll
    for (int it = 0; it < MT; ++it) {
      bf16x8_t f[PP];
#pragma unroll
      for (int l = 0; l < PP; ++l)
        f[l] = *reinterpret_cast<const bf16x8_t*>(F + (l * MP + 16 * it + r) * LDP + 32 * kk + 8 * g);
#pragma unroll
      for (int t = 0; t < 4; ++t)
        acc[it][t] = TR ? mfma_parts<PL, PP>(x[t], f, acc[it][t]) : mfma_parts<PP, PL>(f, x[t], acc[it][t]);
      if (it % 2) __builtin_amdgcn_sched_barrier(0);  // bounds how far the reads of F are hoisted
    }
  }
}

// Stores (or writes back) the results of the 64 columns from j0.
template <int MT, bool TR, bool FAST>
__device__ __forceinline__ void finish_strip(f32x4_t (&acc)[MT][4], const BlockStack& st, int64_t b, int j0, int r,
                                             int g) {
  // opaque here, so that the addresses of a lane's 32 rows are formed one after
  // the other and not all before the strips' loop (they spilled)
  asm volatile("" : "+v"(r), "+v"(g));
  const int64_t ob = b * st.out_bs, ub = b * (int64_t(TR ? st.n : st.m) * st.cols);
  if constexpr (!TR) {
#pragma unroll
    for (int it = 0; it < MT; ++it)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int row = 16 * it + 4 * g + v, col = j0 + 4 * r;
        const int valid = row < st.m ? st.n - col : 0;
        float o[4] = {acc[it][0][v], acc[it][1][v], acc[it][2][v], acc[it][3][v]};
        if (valid > 0)
          finish_run<4, FAST>(st, ob + int64_t(row) * st.out_ld + col, ub + int64_t(row) * st.cols + col, valid, o);
        if (v == 3) __builtin_amdgcn_sched_barrier(0);
      }
  } else {
#pragma unroll
    for (int jt = 0; jt < 4; ++jt)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int j = j0 + 16 * jt + 4 * g + v, i0 = MT * r;
        const int valid = j < st.n ? st.m - i0 : 0;
        float o[MT];
#pragma unroll
        for (int q = 0; q < MT; ++q) o[q] = acc[q][jt][v];
        if (valid > 0)
          finish_run<MT, FAST>(st, ob + int64_t(j) * st.out_ld + i0, ub + int64_t(j) * st.cols + i0, valid, o);
        if (v == 3) __builtin_amdgcn_sched_barrier(0);
      }
  }
}

template <int MT, int PP>
__device__ __forceinline__ void load_factor(uint16_t* F, const uint16_t* src, bool tr, int tid) {
  constexpr int MP = 16 * MT, LDP = MP + 8;
  for (int u = tid; u < PP * MP * (MP / 8); u += AT) {
    const int k8 = u % (MP / 8), row = u / (MP / 8), l = row / MP, i = row % MP;
    // transposed blocks: row MT r + t of P is row r of tile t
    const int ii = tr ? (i % MT) * 16 + i / MT : i;
    *reinterpret_cast<u32x4_t*>(F + (l * MP + ii) * LDP + 8 * k8) =
        *gmem(reinterpret_cast<const u32x4_t*>(src + int64_t(row) * MP + 8 * k8));
  }
}

template <int MT, int PL, int PP, int KIND, bool TR>
__device__ __forceinline__ void apply_block(const BlockStack& st, uint16_t* F, int b, int c0, int c1,
                                            const uint16_t* p, const uint16_t* t, const BlockMom& mom) {
  constexpr int MP = 16 * MT;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int r = lane & 15, g = lane >> 4;
  const View xs{st.x, int64_t(b) * st.x_bs, st.x_ld, (st.flags & BF_X_BF16) != 0, (st.flags & BF_X_VEC) != 0};
  const View ys{st.y, int64_t(b) * st.y_bs, st.y_ld, (st.flags & BF_Y_BF16) != 0, (st.flags & BF_Y_VEC) != 0};
  const uint16_t* pb = p + int64_t(st.block0 + b) * PP * (MP * MP);
  if (KIND != BK_VJP) {
    load_factor<MT, PP>(F, pb, TR, tid);
    __syncthreads();
  }
  for (int s0 = c0; s0 < c1; s0 += BLOCK_STRIP) {
    const int j0 = s0 + 64 * wave;
    f32x4_t acc[MT][4];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) acc[i][q] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    if (KIND == BK_VJP) {
      const uint16_t* tb = t + int64_t(st.block0 + b) * PP * (MP * MP);
      if (s0 > c0) __syncthreads();
      load_factor<MT, PP>(F, pb, TR, tid);
      __syncthreads();
      if (j0 < c1) strip_product<MT, PL, PP, TR, BK_X>(acc, F, ys, ys, st.m, st.n, j0, mom, r, g);
      __syncthreads();
      load_factor<MT, PP>(F, tb, TR, tid);
      __syncthreads();
    }
    if (j0 < c1) {
      strip_product<MT, PL, PP, TR, KIND == BK_STEP ? BK_STEP : BK_X>(acc, F, xs, ys, st.m, st.n, j0, mom, r, g);
      const bool fast = (st.flags & BF_OUT_VEC) && j0 + 64 <= st.n && (!TR || st.m == MP);
      if (fast) finish_strip<MT, TR, true>(acc, st, b, j0, r, g);
      else finish_strip<MT, TR, false>(acc, st, b, j0, r, g);
    }
  }
}

template <int MT, int PL, int PP, int KIND>
__global__ __launch_bounds__(AT, 2) void block_apply_kernel(BlockTable tab, const uint16_t* __restrict__ p,
                                                            const uint16_t* __restrict__ t, BlockMom mom) {
  constexpr int MP = 16 * MT, LDP = MP + 8;
  __shared__ __attribute__((aligned(16))) uint16_t F[PP * MP * LDP];
  const BlockStack st = find_stack(tab, blockIdx.x, [](const BlockStack& s) { return s.aoff; });
  const int local = int(blockIdx.x) - st.aoff;
  const int b = local / st.asplit, sp = local - b * st.asplit;
  const int c0 = sp * st.achunk, c1 = min(st.n, c0 + st.achunk);
  if (st.flags & BF_TR) apply_block<MT, PL, PP, KIND, true>(st, F, b, c0, c1, p, t, mom);
  else apply_block<MT, PL, PP, KIND, false>(st, F, b, c0, c1, p, t, mom);
}

template <int MT>
hipError_t apply_mt(int pl, int pp, int kind, const BlockTable& tab, int32_t wgs, const uint16_t* p,
                    const uint16_t* t, const BlockMom& mom, hipStream_t stream) {
#define MUON_APPLY(PL, PP, KIND)                                                                             \
  if (pl == PL && pp == PP && kind == KIND) {                                                                \
    hipLaunchKernelGGL((block_apply_kernel<MT, PL, PP, KIND>), dim3(wgs), dim3(AT), 0, stream, tab, p, t, mom); \
    return hipGetLastError();                                                                                \
  }
  MUON_APPLY(1, 2, BK_X)
  MUON_APPLY(2, 2, BK_X)
  MUON_APPLY(3, 3, BK_X)
  MUON_APPLY(2, 2, BK_STEP)
  MUON_APPLY(3, 3, BK_STEP)
  MUON_APPLY(1, 2, BK_VJP)
  MUON_APPLY(2, 2, BK_VJP)
  MUON_APPLY(3, 3, BK_VJP)
#undef MUON_APPLY
  return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_block_apply(int mt, int pl, int pp, int kind, const BlockTable& tab, int32_t wgs,
                              const uint16_t* p, const uint16_t* t, const BlockMom& mom, hipStream_t stream) {
  if (wgs <= 0) return hipSuccess;
  return mt == 2   ? apply_mt<2>(pl, pp, kind, tab, wgs, p, t, mom, stream)
         : mt == 4 ? apply_mt<4>(pl, pp, kind, tab, wgs, p, t, mom, stream)
                   : apply_mt<8>(pl, pp, kind, tab, wgs, p, t, mom, stream);
}

}  // namespace muon
