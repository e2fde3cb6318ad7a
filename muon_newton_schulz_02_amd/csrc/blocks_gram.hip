// Gram pass of the block operators: per block, G = x x^T over a range of the
// n columns (x unnormalised, wide orientation m x n), for the gradient also
// Z = y x^T, for the step after the momentum update of the elements it reads.
//
// One workgroup of eight waves takes `gchunk` columns of one block, a tile of
// KC at a time: every thread holds 16 elements of the next tile in flight
// while the current one, split into PL bfloat16 parts, lies in LDS with k
// (the column) contiguous, and the waves multiply its 16 x 16 tiles with
// 16x16x32 MFMAs.  G is symmetric: only tiles on or above the diagonal are
// formed, dealt out as tile rows {p, MT-1-p}, MT + 1 tiles for each of the
// MT/2 pairs; the waves of a pair share out the tile's k-steps of 32, one
// each, and add their sums up at the end, in order.  The partials of the
// workgroups of a block are summed in order by the recursion kernel.
//
// Bound by memory from some hundred blocks on, by the latency of a few
// dependent loads below: the step's pass over 1152 bfloat16 blocks of
// 128 x 1536 (gradient and momentum read, momentum written, 2.27 GB) 451 us,
// 5.0 TB/s, as fast as a copy; 576 blocks read only (0.23 GB) 70 us, 3.2 TB/s;
// 576 binary32 blocks of 64 x 768 32 us, 3.5 TB/s; 12 bfloat16 ones 4.8 us.
// Two tiles in flight instead of one took the same time.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <cstring>

#include "blocks_device.h"

#pragma clang fp contract(off)

namespace muon {
namespace {

constexpr int GT = BLOCK_THREADS;

// LDS bytes of the gram kernel's tiles with NBUF buffers.
template <int MT, int PL, int KIND>
constexpr int gram_tile_bytes() {
  return (KIND == BK_VJP ? 2 : 1) * PL * 16 * MT * (block_kc(MT) + 8) * 2;
}

template <int MT, int PL, int KIND, int XT>
__global__ __launch_bounds__(GT, KIND == BK_VJP ? 2 : 4) void block_gram_kernel(BlockTable tab,
                                                                               float* __restrict__ partials,
                                                                               BlockMom mom) {
  constexpr int MP = 16 * MT, KC = block_kc(MT), LDK = KC + 8;
  constexpr int NM = KIND == BK_VJP ? 2 : 1;       // matrices staged: x (and y)
  // two parts: lo*lo too, so that G is the Gram matrix of the values as split.
  // Its sum of squares, 2^-19 of the trace, would else be missing on the
  // diagonal, where small singular values show it (one and three at 1/200 of
  // it: error 1.8e-2 without, 2.1e-3 with; no change in time)
  constexpr int GS = PL == 2 ? 2 : PL - 1;
  constexpr int KW = 16 / MT;                      // waves of a pair of tile rows = k-steps of a tile
  // two buffers where two workgroups still fit a compute unit
  constexpr int TB = gram_tile_bytes<MT, PL, KIND>(), NBUF = 2 * TB <= 80 * 1024 ? 2 : 1;
  constexpr int NG = MT + 1, NZ = KIND == BK_VJP ? 2 * MT : 0;  // tiles of a wave
  constexpr int RED = (MT / 2) * (NZ > NG ? NZ : NG) * 1024;    // the final sum's LDS
  constexpr int LB = NBUF * TB > RED ? NBUF * TB : RED;
  __shared__ __attribute__((aligned(16))) unsigned char lds_raw[LB];
  typedef uint16_t Tile[NM][PL][MP][LDK];
  Tile* const lds = reinterpret_cast<Tile*>(lds_raw);

  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int r = lane & 15, g = lane >> 4;
  const int wg = block_number();
  const BlockStack st = find_stack<KEY_GRAM>(wg);
  const int local = wg - st.goff;
  const int b = local / st.gsplit, sp = local - b * st.gsplit;
  const int k0 = sp * st.gchunk, k1 = min(st.n, k0 + st.gchunk);
  const bool tr = st.flags & BF_TR;
  const bool xbf = XT == BX_ANY ? (st.flags & BF_X_BF16) != 0 : XT == BX_BF16;
  const bool ybf = KIND == BK_VJP && (PL == 1 || (st.flags & BF_Y_BF16));
  const int xs = xbf ? 2 : 4, ys = ybf ? 2 : 4;

  // the thread's two runs of 8 elements: rows contiguous along k, two runs of
  // 8 columns (512 threads apart); transposed, 8 rows of two columns
  // (transposed, a wave takes 32 rows of 32 columns: its stores to LDS, a row
  // of x each, then meet two to a bank, eight with all rows of 8 columns)
  constexpr int RB = MP / 32;
  const int row0 = tr ? (tid & 3) * 8 + wave % RB * 32 : tid / (KC / 8);
  const int col0 = tr ? (lane >> 2) * 2 + wave / RB * 32 : (tid % (KC / 8)) * 8;
  constexpr int DR = GT / (KC / 8);
  // first byte of the first tile, bytes from tile to tile, and the first
  // run's byte offset in a tile
  const char* xp = reinterpret_cast<const char*>(st.x) + (int64_t(b) * st.x_bs + (tr ? k0 * st.x_ld : k0)) * xs;
  char* yp = reinterpret_cast<char*>(const_cast<void*>(st.y)) + (int64_t(b) * st.y_bs + (tr ? k0 * st.y_ld : k0)) * ys;
  const int64_t xt = (tr ? KC * st.x_ld : KC) * xs, yt = (tr ? KC * st.y_ld : KC) * ys;
  const uint32_t xl = uint32_t(st.x_ld) * xs, yl = uint32_t(st.y_ld) * ys;
  const uint32_t xo = tr ? col0 * xl + row0 * xs : row0 * xl + col0 * xs;
  const uint32_t yo = tr ? col0 * yl + row0 * ys : row0 * yl + col0 * ys;
  const uint32_t xd = tr ? xl : DR * xl, yd = tr ? yl : DR * yl;
  auto valid_of = [&](int q, int kn) {  // kn: columns from the tile's first one on
    return tr ? (col0 + q < kn ? st.m - row0 : 0) : (row0 + q * DR < st.m ? kn - col0 : 0);
  };

  Raw8 rx[2], ry[2];
  auto fetch = [&](int kn) {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int valid = valid_of(q, kn);
      load_raw(rx[q], xp, xo + q * xd, xbf, valid);
      if (KIND == BK_STEP) load_raw(ry[q], yp, yo + q * yd, false, valid);
      if (KIND == BK_VJP) load_raw(ry[q], yp, yo + q * yd, ybf, valid);
    }
  };

  const int p = wave % (MT / 2), kw = wave / (MT / 2);
  f32x4_t acc[NG], zacc[NZ ? NZ : 1];
#pragma unroll
  for (int q = 0; q < NG; ++q) acc[q] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int q = 0; q < NZ; ++q) zacc[q] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  fetch(k1 - k0);
  int buf = 0;
#pragma unroll 1
  for (int kb = k0; kb < k1; kb += KC) {
    if (NBUF == 1 && kb > k0) __syncthreads();  // the last tile's reads are done
    Tile& tile = lds[buf];
#pragma unroll
    for (int mat = 0; mat < NM; ++mat) {
      if constexpr (PL == 1) {  // bfloat16 as it is
        const Raw8(&raw)[2] = mat ? ry : rx;
        if (!tr) {
#pragma unroll
          for (int q = 0; q < 2; ++q)
            *reinterpret_cast<u32x4_t*>(&tile[mat][0][row0 + q * DR][col0]) = raw[q].a;
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            *reinterpret_cast<uint32_t*>(&tile[mat][0][row0 + i][col0]) = pair_bf16(raw[0], raw[1], i);
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
          for (int i = 0; i < 8; ++i) v[q][i] = momentum_elem(v[q][i], m[i], mom);
          const int valid = valid_of(q, k1 - kb);
          if (valid > 0) store8(yp, yo + q * yd, false, valid, m);
        }
      }
      if (!tr) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          bf16x8_t o[PL];
          split8<PL>(v[q], o);
#pragma unroll
          for (int l = 0; l < PL; ++l) *reinterpret_cast<bf16x8_t*>(&tile[mat][l][row0 + q * DR][col0]) = o[l];
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          uint32_t o[PL];
          split2<PL>(v[0][i], v[1][i], o);
#pragma unroll
          for (int l = 0; l < PL; ++l) *reinterpret_cast<uint32_t*>(&tile[mat][l][row0 + i][col0]) = o[l];
        }
      }
    }
    if (kb + KC < k1) {
      xp += xt;
      yp += yt;
      fetch(k1 - kb - KC);
    }
    __syncthreads();
    const int ko = kw * 32 + 8 * g;
    bf16x8_t a0[PL], a1[PL];
#pragma unroll
    for (int l = 0; l < PL; ++l) {
      a0[l] = *reinterpret_cast<const bf16x8_t*>(&tile[0][l][16 * p + r][ko]);
      a1[l] = *reinterpret_cast<const bf16x8_t*>(&tile[0][l][16 * (MT - 1 - p) + r][ko]);
    }
#pragma unroll
    for (int q = 0; q < NG; ++q) {
      const bool first = q < MT - p;
      const int tj = first ? p + q : MT - 1 - p + (q - (MT - p));
      bf16x8_t bb[PL];
#pragma unroll
      for (int l = 0; l < PL; ++l) bb[l] = *reinterpret_cast<const bf16x8_t*>(&tile[0][l][16 * tj + r][ko]);
      if (first) acc[q] = mfma_parts<PL, PL, GS>(a0, bb, acc[q]);
      else acc[q] = mfma_parts<PL, PL, GS>(a1, bb, acc[q]);
    }
    if (KIND == BK_VJP) {
#pragma unroll
      for (int l = 0; l < PL; ++l) {
        a0[l] = *reinterpret_cast<const bf16x8_t*>(&tile[NM - 1][l][16 * p + r][ko]);
        a1[l] = *reinterpret_cast<const bf16x8_t*>(&tile[NM - 1][l][16 * (MT - 1 - p) + r][ko]);
      }
#pragma unroll
      for (int tj = 0; tj < MT; ++tj) {
        bf16x8_t bb[PL];
#pragma unroll
        for (int l = 0; l < PL; ++l) bb[l] = *reinterpret_cast<const bf16x8_t*>(&tile[0][l][16 * tj + r][ko]);
        zacc[tj] = mfma_parts<PL, PL, GS>(a0, bb, zacc[tj]);
        zacc[MT + tj] = mfma_parts<PL, PL, GS>(a1, bb, zacc[MT + tj]);
      }
    }
    if (NBUF == 2) buf ^= 1;
  }

  // add up the KW sums of every tile, in order, and store them
  f32x4_t* const red = reinterpret_cast<f32x4_t*>(lds_raw);
  auto gather = [&](f32x4_t* t, int n) {
    for (int s = 1; s < KW; ++s) {
      __syncthreads();
      if (kw == s)
#pragma unroll
        for (int q = 0; q < n; ++q) red[(p * n + q) * 64 + lane] = t[q];
      __syncthreads();
      if (kw == 0)
#pragma unroll
        for (int q = 0; q < n; ++q) t[q] += red[(p * n + q) * 64 + lane];
    }
  };
  gather(acc, NG);
  if (KIND == BK_VJP) gather(zacc, NZ);
  if (kw == 0) {
    float* out = partials + st.part0 + (int64_t(b) * st.gsplit + sp) * st.part;
#pragma unroll
    for (int q = 0; q < NG; ++q) *gmem(reinterpret_cast<f32x4_t*>(out + ((p * NG + q) * 64 + lane) * 4)) = acc[q];
    if (KIND == BK_VJP) {
      out += (MT / 2) * NG * 256;
#pragma unroll
      for (int q = 0; q < NZ; ++q) *gmem(reinterpret_cast<f32x4_t*>(out + ((p * NZ + q) * 64 + lane) * 4)) = zacc[q];
    }
  }
}

__global__ void block_table_kernel(BlockTableBatch in, BlockStack* __restrict__ out, int32_t* __restrict__ keys,
                                   int32_t stride) {
  const int i = threadIdx.x;
  if (i >= in.n) return;
  int c = 0;
#pragma unroll
  for (int q = 1; q < BLOCK_CLASSES; ++q)
    if (i >= in.first[q]) c = q;
  BlockStack s = in.cls[c];
  const int k = i - in.first[c];
  s.x = in.x[i];
  s.y = in.y[i];
  s.out = in.out[i];
  s.upd = in.upd[i];
  s.block0 += k * s.blocks;
  s.goff += k * s.blocks * s.gsplit;
  s.aoff += k * s.blocks * s.asplit;
  s.part0 += int64_t(k) * s.blocks * s.gsplit * s.part;
  out[i] = s;
  keys[KEY_GRAM * stride + i] = s.goff;
  keys[KEY_BLOCK * stride + i] = s.block0;
  keys[KEY_APPLY * stride + i] = s.aoff;
}

template <int MT>
hipError_t gram_mt(int pl, int kind, bool xbf, const BlockTable& tab, int32_t wgs, float* partials,
                   const BlockMom& mom, hipStream_t stream) {
#define MUON_GRAM(PL, KIND, XT)                                                                             \
  if (pl == PL && kind == KIND && (XT == BX_ANY || xbf == (XT == BX_BF16))) {                               \
    hipLaunchKernelGGL((block_gram_kernel<MT, PL, KIND, XT>), dim3(wgs), dim3(GT), 0, stream, tab, partials, \
                       mom);                                                                                \
    return hipGetLastError();                                                                               \
  }
  MUON_GRAM(1, BK_X, BX_BF16)
  MUON_GRAM(2, BK_X, BX_F32)
  MUON_GRAM(3, BK_X, BX_ANY)
  MUON_GRAM(2, BK_STEP, BX_BF16)
  MUON_GRAM(2, BK_STEP, BX_F32)
  MUON_GRAM(3, BK_STEP, BX_ANY)
  MUON_GRAM(1, BK_VJP, BX_BF16)
  MUON_GRAM(2, BK_VJP, BX_ANY)
  MUON_GRAM(3, BK_VJP, BX_ANY)
#undef MUON_GRAM
  return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_block_table(const BlockStack* host, int32_t count, BlockStack* dev, int32_t* keys,
                              hipStream_t stream) {
  // what two stacks of a run share
  auto key = [](BlockStack s) {
    s.x = s.y = nullptr;
    s.out = nullptr;
    s.upd = nullptr;
    s.part0 = 0;
    s.block0 = s.goff = s.aoff = 0;
    return s;
  };
  for (int32_t i = 0; i < count;) {
    BlockTableBatch b;
    memset(&b, 0, sizeof(b));
    int32_t classes = 0;
    BlockStack last;
    while (i + b.n < count && b.n < BLOCK_BATCH) {
      const BlockStack& s = host[i + b.n];
      const BlockStack k = key(s);
      if (classes == 0 || memcmp(&k, &last, sizeof(k)) != 0) {
        if (classes == BLOCK_CLASSES) break;
        b.first[classes] = b.n;
        b.cls[classes++] = s;
        last = k;
      }
      b.x[b.n] = s.x;
      b.y[b.n] = s.y;
      b.out[b.n] = s.out;
      b.upd[b.n] = s.upd;
      ++b.n;
    }
    for (int32_t c = classes; c < BLOCK_CLASSES; ++c) b.first[c] = b.n;
    hipLaunchKernelGGL(block_table_kernel, dim3(1), dim3(128), 0, stream, b, dev + i, keys + i, count);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    i += b.n;
  }
  return hipSuccess;
}

hipError_t launch_block_gram(int mt, int pl, int kind, bool xbf, const BlockTable& tab, int32_t wgs,
                             float* partials, const BlockMom& mom, hipStream_t stream) {
  if (wgs <= 0) return hipSuccess;
  return mt == 2   ? gram_mt<2>(pl, kind, xbf, tab, wgs, partials, mom, stream)
         : mt == 4 ? gram_mt<4>(pl, kind, xbf, tab, wgs, partials, mom, stream)
                   : gram_mt<8>(pl, kind, xbf, tab, wgs, partials, mom, stream);
}

}  // namespace muon
