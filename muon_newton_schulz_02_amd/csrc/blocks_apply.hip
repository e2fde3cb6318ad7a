// Apply pass of the block operators: per block, O = P x (m x m by m x n), for
// the gradient O = P y + T x, for the step with x formed again from the
// gradient and the updated momentum; then the store, or the write-back
//   W <- rnd(fl32(W d) - fl32(t O)).
//
// One workgroup of eight waves walks its columns of one block in tiles of KC.
// Every thread holds 16 elements of the next tile in flight (and the weights
// that the current one updates) while the current one, split into PL bfloat16
// parts, lies in LDS with the block's rows, the product's k, contiguous.  A
// wave keeps its 16 rows of P (PP parts) in registers for the whole walk and
// multiplies them with 64 columns by v_mfma_f32_16x16x32_bf16.  The tile of
// results goes through LDS once, so that loads and stores of the output are
// runs of 8 elements of its rows, whichever way the block is stored.
//
// Bound by memory: the step's pass over 1152 bfloat16 blocks of 128 x 1536
// (gradient, momentum and weight read, weight written, 2.27 GB) 487 us, 4.7
// TB/s; 576 blocks read and written (0.45 GB) 114 us, 4.0 TB/s; 576 binary32
// blocks of 64 x 768 (0.23 GB) 55 us, 4.1 TB/s; the gradient of 288 blocks of
// 128 x 1536 (0.34 GB) 99 to 103 us, 3.4 TB/s.  Loads and stores past the caches
// (nontemporal) gave the largest call 4% and took 5% to 10% from calls whose
// tensors stay in the last-level cache.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "blocks_device.h"

#pragma clang fp contract(off)

namespace muon {
namespace {

constexpr int AT = BLOCK_THREADS;

// Row of the x tile in LDS that holds column j: the four 16-column tiles of a
// group of 64 take every fourth column, so that the accumulators of a lane
// are four consecutive columns.
__device__ __forceinline__ int tile_row(int j) { return (j & ~63) + (j & 3) * 16 + ((j & 63) >> 2); }

// Whether a compute unit holds two workgroups (four waves a SIMD, 128
// registers each): not where those do not reach, which are the gradient on
// more parts or rows (146 to 256 registers) and the binary32 step at 128 rows
// (198; it moves 4.9 TB/s with one workgroup or two).
constexpr bool two_resident(int mt, int pl, int kind) {
  return kind == BK_VJP ? pl == 1 || (pl == 2 && mt < 8) : kind == BK_X || pl < 3 || mt < 8;
}

template <int MT, int PL, int PP, int KIND, int XT>
__global__ __launch_bounds__(AT, two_resident(MT, PL, KIND) ? 4 : 2) void block_apply_kernel(
    BlockTable tab, const uint16_t* __restrict__ pf, const uint16_t* __restrict__ tf, BlockMom mom) {
  constexpr int MP = 16 * MT, KC = block_kc(MT), LDX = MP + 8;
  constexpr int NM = KIND == BK_VJP ? 2 : 1;
  constexpr int LDO = KC + 4, LDT = MP + 4;  // results by rows of x, or by columns
  constexpr int OB = (MP * LDO > KC * LDT ? MP * LDO : KC * LDT);
  // the results' tile takes the place of x's (two more barriers a tile) where
  // both would leave no room for the second workgroup.  Binary32, 576 blocks
  // of 64 x 768: 63 us apart, 53 us together, with the write-back 92 and 79;
  // 600 of 128 x 1536: 309 and 251; bfloat16 gradients of binary32 blocks,
  // 576 of 64 x 768: 86 and 63, 1000 of 32 x 1536: 126 and 101
  constexpr int XB = NM * PL * KC * LDX * 2;
  constexpr bool SHARE = two_resident(MT, PL, KIND) && XB + OB * 4 > 80 * 1024 && XB >= OB * 4;
  __shared__ __attribute__((aligned(16))) unsigned char lds_raw[SHARE ? XB : XB + OB * 4];
  typedef uint16_t XTile[PL][KC][LDX];
  XTile* const xs = reinterpret_cast<XTile*>(lds_raw);
  float* const os = reinterpret_cast<float*>(SHARE ? lds_raw : lds_raw + XB);

  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int r = lane & 15, g = lane >> 4;
  const int wr = wave % MT, wc = wave / MT;  // the wave's row tile and group of 64 columns
  const int wg = block_number();
  const BlockStack st = find_stack<KEY_APPLY>(wg);
  const int local = wg - st.aoff;
  const int b = local / st.asplit, sp = local - b * st.asplit;
  const int c0 = sp * st.achunk, c1 = min(st.n, c0 + st.achunk);
  const bool tr = st.flags & BF_TR;
  const bool xbf = XT == BX_ANY ? (st.flags & BF_X_BF16) != 0 : XT == BX_BF16;
  const bool ybf = KIND == BK_VJP && (PL == 1 || (st.flags & BF_Y_BF16));
  const bool obf = PP == 2 && (st.flags & BF_OUT_BF16);
  const bool wback = KIND != BK_VJP && (st.flags & BF_WRITEBACK);
  const int xsz = xbf ? 2 : 4, ysz = ybf ? 2 : 4, osz = obf ? 2 : 4;

  // the thread's two runs of 8 elements of x: 8 columns of two rows, or
  // transposed 8 rows of two columns (512 threads apart)
  const int row0 = tr ? (tid % (MP / 8)) * 8 : (tid / (KC / 8)) * 2;
  const int col0 = tr ? tid / (MP / 8) : (tid % (KC / 8)) * 8;
  constexpr int DC = AT / (MP / 8), DR = AT / (KC / 8);
  const int dcol = tr ? DC : 0;
  // first byte of the first tile, bytes from tile to tile, and the first
  // run's byte offset in a tile
  const char* xp = reinterpret_cast<const char*>(st.x) + (int64_t(b) * st.x_bs + (tr ? c0 * st.x_ld : c0)) * xsz;
  const char* yp = reinterpret_cast<const char*>(st.y) + (int64_t(b) * st.y_bs + (tr ? c0 * st.y_ld : c0)) * ysz;
  char* op = reinterpret_cast<char*>(st.out) + (int64_t(b) * st.out_bs + (tr ? c0 * st.out_ld : c0)) * osz;
  const int64_t xt = (tr ? KC * st.x_ld : KC) * xsz, yt = (tr ? KC * st.y_ld : KC) * ysz;
  const int64_t ot = (tr ? KC * st.out_ld : KC) * osz;
  const uint32_t xl = uint32_t(st.x_ld) * xsz, yl = uint32_t(st.y_ld) * ysz, ol = uint32_t(st.out_ld) * osz;
  const uint32_t xo = tr ? col0 * xl + row0 * xsz : row0 * xl + col0 * xsz;
  const uint32_t yo = tr ? col0 * yl + row0 * ysz : row0 * yl + col0 * ysz;
  const uint32_t xd = tr ? DC * xl : xl, yd = tr ? DC * yl : yl;
  // and of the output: the same, or 8 columns of two rows (512 threads apart)
  const int orow = tr ? row0 : tid / (KC / 8);
  const uint32_t oo = tr ? col0 * ol + orow * osz : orow * ol + col0 * osz;
  const uint32_t od = tr ? DC * ol : DR * ol;

  Raw8 rx[2], ry[2], rw[2];
  auto fetch = [&](int cn) {  // cn: columns from the tile's first one on
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int valid = tr ? (col0 + q * DC < cn ? st.m - row0 : 0) : (row0 + q < st.m ? cn - col0 : 0);
      load_raw(rx[q], xp, xo + q * xd, xbf, valid);
      if (KIND == BK_STEP) load_raw(ry[q], yp, yo + q * yd, false, valid);
      if (KIND == BK_VJP) load_raw(ry[q], yp, yo + q * yd, ybf, valid);
    }
  };
  auto ovalid = [&](int q, int cn) {
    return tr ? (col0 + q * DC < cn ? st.m - orow : 0) : (orow + q * DR < st.m ? cn - col0 : 0);
  };
  fetch(c1 - c0);

  // the wave's rows of P (and T)
  constexpr int NK = MP / 32;
  bf16x8_t f[NM][PP][NK];
#pragma unroll
  for (int mat = 0; mat < NM; ++mat) {
    // x is multiplied with P, for the gradient with T, and y with P
    const uint16_t* src = (KIND == BK_VJP && mat == 0 ? tf : pf) + int64_t(st.block0 + b) * PP * (MP * MP);
#pragma unroll
    for (int l = 0; l < PP; ++l)
#pragma unroll
      for (int kk = 0; kk < NK; ++kk)
        f[mat][l][kk] = *gmem(reinterpret_cast<const bf16x8_t*>(src + (l * MP + 16 * wr + r) * MP + 32 * kk + 8 * g));
  }

#pragma unroll 1
  for (int kb = c0; kb < c1; kb += KC) {
#pragma unroll
    for (int mat = 0; mat < NM; ++mat) {
      // bfloat16 as it is (the gradient at 128 rows would spill: 98 us, 110 so)
      if constexpr (PL == 1 && (KIND != BK_VJP || MT < 8)) {
        const Raw8(&raw)[2] = mat ? ry : rx;
        if (!tr) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            *reinterpret_cast<uint32_t*>(&xs[mat][0][tile_row(col0 + i)][row0]) = pair_bf16(raw[0], raw[1], i);
        } else {
#pragma unroll
          for (int q = 0; q < 2; ++q)
            *reinterpret_cast<u32x4_t*>(&xs[mat][0][tile_row(col0 + q * dcol)][row0]) = raw[q].a;
        }
        continue;
      }
      float v[2][8];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        unpack(mat ? ry[q] : rx[q], mat ? ybf : xbf, v[q]);
        if (KIND == BK_STEP) {
          float m[8];
          unpack(ry[q], false, m);
#pragma unroll
          for (int i = 0; i < 8; ++i) v[q][i] = momentum_dir(v[q][i], m[i], mom);
        }
      }
      if (!tr) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          uint32_t o[PL];
          split2<PL>(v[0][i], v[1][i], o);
#pragma unroll
          for (int l = 0; l < PL; ++l) *reinterpret_cast<uint32_t*>(&xs[mat][l][tile_row(col0 + i)][row0]) = o[l];
        }
      } else {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          bf16x8_t o[PL];
          split8<PL>(v[q], o);
#pragma unroll
          for (int l = 0; l < PL; ++l)
            *reinterpret_cast<bf16x8_t*>(&xs[mat][l][tile_row(col0 + q * dcol)][row0]) = o[l];
        }
      }
    }
    if (wback)
#pragma unroll
      for (int q = 0; q < 2; ++q) load_raw(rw[q], op, oo + q * od, obf, ovalid(q, c1 - kb));
    if (kb + KC < c1) {
      xp += xt;
      yp += yt;
      fetch(c1 - kb - KC);
    }
    __syncthreads();
    f32x4_t acc[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) acc[t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int mat = 0; mat < NM; ++mat)
#pragma unroll
      for (int kk = 0; kk < NK; ++kk) {
        bf16x8_t a[PP];
#pragma unroll
        for (int l = 0; l < PP; ++l) a[l] = f[mat][l][kk];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          bf16x8_t x[PL];
#pragma unroll
          for (int l = 0; l < PL; ++l)
            x[l] = *reinterpret_cast<const bf16x8_t*>(&xs[mat][l][64 * wc + 16 * t + r][32 * kk + 8 * g]);
          acc[t] = mfma_parts<PP, PL>(a, x, acc[t]);
        }
      }
    if (SHARE) __syncthreads();
    // row 16 wr + 4 g + v, columns 64 wc + 4 r + {0 .. 3}
    if (!tr) {
#pragma unroll
      for (int v = 0; v < 4; ++v)
        *reinterpret_cast<f32x4_t*>(&os[(16 * wr + 4 * g + v) * LDO + 64 * wc + 4 * r]) =
            f32x4_t{acc[0][v], acc[1][v], acc[2][v], acc[3][v]};
    } else {
#pragma unroll
      for (int t = 0; t < 4; ++t)
        *reinterpret_cast<f32x4_t*>(&os[(64 * wc + 4 * r + t) * LDT + 16 * wr + 4 * g]) = acc[t];
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int valid = ovalid(q, c1 - kb);
      if (valid <= 0) continue;
      const float* s = tr ? &os[(col0 + q * DC) * LDT + orow] : &os[(orow + q * DR) * LDO + col0];
      const f32x4_t o0 = *reinterpret_cast<const f32x4_t*>(s), o1 = *reinterpret_cast<const f32x4_t*>(s + 4);
      float o[8] = {o0[0], o0[1], o0[2], o0[3], o1[0], o1[1], o1[2], o1[3]};
      if (wback) {
        if (st.upd) {
          const int64_t rows = tr ? st.n : st.m;
          const int64_t row = tr ? kb + col0 + q * DC : orow + q * DR, col = tr ? orow : kb + col0;
          store8(reinterpret_cast<char*>(st.upd + (b * rows + row) * st.cols + col), 0, false, valid, o);
        }
        float wv[8];
        unpack(rw[q], obf, wv);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float wd = wv[i] * st.d;
          const float to = st.t * o[i];
          o[i] = wd - to;
        }
      }
      store8(op, oo + q * od, obf, valid, o);
    }
    op += ot;
    if (SHARE && kb + KC < c1) __syncthreads();
  }
}

template <int MT>
hipError_t apply_mt(int pl, int pp, int kind, bool xbf, const BlockTable& tab, int32_t wgs, const uint16_t* p,
                    const uint16_t* t, const BlockMom& mom, hipStream_t stream) {
#define MUON_APPLY(PL, PP, KIND, XT)                                                                             \
  if (pl == PL && pp == PP && kind == KIND && (XT == BX_ANY || xbf == (XT == BX_BF16))) {                        \
    hipLaunchKernelGGL((block_apply_kernel<MT, PL, PP, KIND, XT>), dim3(wgs), dim3(AT), 0, stream, tab, p, t, mom); \
    return hipGetLastError();                                                                                    \
  }
  MUON_APPLY(1, 2, BK_X, BX_BF16)
  MUON_APPLY(2, 2, BK_X, BX_F32)
  MUON_APPLY(3, 3, BK_X, BX_ANY)
  MUON_APPLY(2, 2, BK_STEP, BX_BF16)
  MUON_APPLY(2, 2, BK_STEP, BX_F32)
  MUON_APPLY(3, 3, BK_STEP, BX_ANY)
  MUON_APPLY(1, 2, BK_VJP, BX_BF16)
  MUON_APPLY(2, 2, BK_VJP, BX_ANY)
  MUON_APPLY(3, 3, BK_VJP, BX_ANY)
#undef MUON_APPLY
  return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_block_apply(int mt, int pl, int pp, int kind, bool xbf, const BlockTable& tab, int32_t wgs,
                              const uint16_t* p, const uint16_t* t, const BlockMom& mom, hipStream_t stream) {
  if (wgs <= 0) return hipSuccess;
  return mt == 2   ? apply_mt<2>(pl, pp, kind, xbf, tab, wgs, p, t, mom, stream)
         : mt == 4 ? apply_mt<4>(pl, pp, kind, xbf, tab, wgs, p, t, mom, stream)
                   : apply_mt<8>(pl, pp, kind, xbf, tab, wgs, p, t, mom, stream);
}

}  // namespace muon
