// The m x m recursion of the block operators, one workgroup per block:
//   A_0 = s^2 G ; Q = a I + b A + c A A ; P <- Q P ; A <- Q A Q
// with s = 1 / (||x|| + 1e-7), ||x||^2 the trace of G.  For the gradient also
// its tangent from D_0 = s sym(Z), Z = y x^T:
//   dQ = b D + c (D A + A D) ; dP <- dQ P + Q dP ; D <- dQ A Q + Q D Q + Q A dQ
// P and dP end as the polynomial at A_0 and its derivative in direction D_0;
// every matrix is a function of A_0, so the order of factors is free and the
// derivative is its own adjoint.
//
// Products run on binary16 MFMAs with every operand split into two parts (24
// bits with their signs) and three products, hi*hi + hi*lo + lo*hi, summed in binary32.  A
// matrix is scaled by a power of two first, so that its largest element lies
// in [2^14, 2^15): parts of smaller elements then stay exact down to 2^-39 of
// it, and no matrix overflows the format.  Against binary32 products
// (v_mfma_f32_16x16x4f32) the results' errors are the same to a factor of 1.3
// (they come from the Gram matrix), at 3/16 of the matrix-core time.
//
// A wave holds TS columns of every matrix in its registers (TS = 16 or 32), as
// the accumulator tiles of v_mfma_f32_16x16x32_f16 or _32x32x16_f16.  A lane's
// values 8 q, ..., 8 q + 7, counted through the tiles, are at the same time
// the B operand of a later product's k-step q, with k taken in the order of
// their rows.  A product L R therefore needs only L in LDS, and as every
// matrix is symmetric but for rounding, row i of L is column i: the operand
// registers are stored as they are, 16 bytes a lane, and read back the same
// way by every wave.
//
// Bound by the chain of products (each waits for the one before, and for one
// exchange of its largest element) with few blocks, by the matrix cores and
// LDS with many.  Five quintic steps: 12 blocks of 64 rows 17 us; 48 of 128
// rows 56 us; 1152 of them 250 to 269 us (17 products of three parts each,
// 0.25 PFLOP, 0.95 PFLOP/s of about 1.8 that MFMAs alone reach); the gradient
// of 288 of 128 rows, one to a compute unit (256 registers a lane, 38 spilled),
// 295 to 315 us, of 216 of 64 rows 23 us a stage.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "blocks_device.h"

#pragma clang fp contract(off)

#define MUON_INLINE __attribute__((always_inline))

namespace muon {
namespace {

constexpr float NORM_EPS = 1e-7f;

typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));

typedef float f32x16_t __attribute__((ext_vector_type(16)));

// Accumulator tiles of TS x TS: V values a lane, of column lane % TS.
template <int TS>
struct Tile;
template <>
struct Tile<16> {
  static constexpr int V = 4;
  typedef f32x4_t Acc;
  static __device__ __forceinline__ Acc mfma(f16x8_t a, f16x8_t b, Acc c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
  }
  static __device__ __forceinline__ int row(int v, int h) { return 4 * h + v; }
};
template <>
struct Tile<32> {
  static constexpr int V = 16;
  typedef f32x16_t Acc;
  static __device__ __forceinline__ Acc mfma(f16x8_t a, f16x8_t b, Acc c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
  }
  static __device__ __forceinline__ int row(int v, int h) { return 8 * (v >> 2) + 4 * h + (v & 3); }
};

// Shapes of an MP x MP matrix on waves of TS columns each.
template <int MP, int TS>
struct Shape {
  static constexpr int NR = MP / TS, V = Tile<TS>::V, NV = NR * V, NQ = NV / 8;  // row tiles, values, k-steps
  static constexpr int KS = MP / NQ;                                             // columns of a k-step
  typedef typename Tile<TS>::Acc Acc;
};

// A wave's columns as product operand: 2^ex times the values, as hi and lo
// parts.  ex is the same for all waves where the matrix goes to LDS too.
template <int NQ>
struct Operand {
  f16x8_t f[NQ][2];
  int ex;
};

// The bits of the largest |X| over the wave, in a scalar register.
template <class Acc, int NR, int V>
__device__ __forceinline__ uint32_t max_bits(const Acc (&X)[NR]) {
  float v = 0.f;
#pragma unroll
  for (int kt = 0; kt < NR; ++kt)
#pragma unroll
    for (int i = 0; i < V; ++i) v = fmaxf(v, __builtin_fabsf(X[kt][i]));
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

// 2^x takes a largest element in [2^e, 2^(e + 1)) to [2^14, 2^15); bounded so
// that 2^x is a binary32 number (elements below 2^-106 come out smaller).
__device__ __forceinline__ int scale_for(uint32_t bits) { return min(14 + 127 - int(bits >> 23), 120); }

// The parts of s X for k-step q.  hi is the binary32 product rounded to 11
// bits (its conversion is then exact), lo what is left of it, rounded to 11
// more.  Cutting hi off instead saves an addition, 1% of the call, and costs
// two bits: one singular value and three at 1/100 of it, 8e-3 for 4e-3.
template <class Acc, int NR, int V>
__device__ __forceinline__ void split_step(const Acc (&X)[NR], int q, float s, f16x8_t& hi, f16x8_t& lo) {
#pragma unroll
  for (int e = 0; e < 8; e += 2) {
    const int i = 8 * q + e;
    const f32x2_t x = {X[i / V][i % V] * s, X[(i + 1) / V][(i + 1) % V] * s};
    const f32x2_t top = {__uint_as_float((__float_as_uint(x[0]) + 0x1000u) & 0xFFFFE000u),
                         __uint_as_float((__float_as_uint(x[1]) + 0x1000u) & 0xFFFFE000u)};
    const f32x2_t rest = {x[0] - top[0], x[1] - top[1]};
    const f16x2_t a = __builtin_convertvector(top, f16x2_t), b = __builtin_convertvector(rest, f16x2_t);
    hi[e] = a[0];
    hi[e + 1] = a[1];
    lo[e] = b[0];
    lo[e + 1] = b[1];
  }
  // opaque from here on: binary32 copies of the parts, kept for combine(),
  // would spill
  asm volatile("" : "+v"(hi), "+v"(lo));
}

// A matrix in LDS: row i holds column i of the matrix, two parts.
template <int MP>
struct Left {
  uint16_t v[2][MP][MP + 8];
};

template <class Acc, int NR, int V>
__device__ __forceinline__ void zero_sums(Acc (&acc)[NR]) {
#pragma unroll
  for (int jt = 0; jt < NR; ++jt)
#pragma unroll
    for (int v = 0; v < V; ++v) acc[jt][v] = 0.f;
}

// acc[k] += L X[k], k < N, for the wave's columns X, all as scaled: every read
// of L serves N products.
template <int MP, int TS, int N>
__device__ __forceinline__ void multiply(typename Tile<TS>::Acc (*const (&acc)[N])[MP / TS], const Left<MP>& L,
                                         const Operand<Shape<MP, TS>::NQ>* const (&X)[N], int c, int h) {
  using S = Shape<MP, TS>;
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int q = 0; q < S::NQ; ++q)
#pragma unroll
    for (int jt = 0; jt < S::NR; ++jt) {
      const f16x8_t hi = *reinterpret_cast<const f16x8_t*>(&L.v[0][TS * jt + c][S::KS * q + 8 * h]);
      const f16x8_t lo = *reinterpret_cast<const f16x8_t*>(&L.v[1][TS * jt + c][S::KS * q + 8 * h]);
#pragma unroll
      for (int k = 0; k < N; ++k) (*acc[k])[jt] = Tile<TS>::mfma(lo, X[k]->f[q][0], (*acc[k])[jt]);
#pragma unroll
      for (int k = 0; k < N; ++k) (*acc[k])[jt] = Tile<TS>::mfma(hi, X[k]->f[q][1], (*acc[k])[jt]);
#pragma unroll
      for (int k = 0; k < N; ++k) (*acc[k])[jt] = Tile<TS>::mfma(hi, X[k]->f[q][0], (*acc[k])[jt]);
    }
  // the reads of L run AHEAD pairs ahead of the products that take them (all
  // of them at once would spill, one at a time waits for LDS)
  constexpr int ITEMS = S::NQ * S::NR, AHEAD = ITEMS < 4 ? ITEMS : 4;
  __builtin_amdgcn_sched_group_barrier(0x100, 2 * AHEAD, 0);
#pragma unroll
  for (int i = 0; i < ITEMS - AHEAD; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x008, 3 * N, 0);
    __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
  }
  __builtin_amdgcn_sched_group_barrier(0x008, 3 * N * AHEAD, 0);
  __builtin_amdgcn_sched_barrier(0);
}

// acc = c 2^-e acc + b X
template <int MP, int TS>
__device__ __forceinline__ void combine(typename Tile<TS>::Acc (&acc)[MP / TS], float c, int e, float b,
                                        const Operand<Shape<MP, TS>::NQ>& X) {
  using S = Shape<MP, TS>;
  const float ce = __builtin_amdgcn_ldexpf(c, -e), be = __builtin_amdgcn_ldexpf(b, -X.ex);
#pragma unroll
  for (int i = 0; i < S::NV; ++i) {
    float t = ce * acc[i / S::V][i % S::V];
    t = __builtin_fmaf(float(X.f[i / 8][0][i % 8]), be, t);
    acc[i / S::V][i % S::V] = __builtin_fmaf(float(X.f[i / 8][1][i % 8]), be, t);
  }
}

// Columns of a wave.  With 32 a 128 x 128 product reads half as much of L,
// whose reads otherwise take longer than the MFMAs (1152 blocks: 302 us with
// 16, 238 with 32); the gradient's matrices would not fit the registers (993
// us against 762), and smaller blocks would have too few waves (64 rows, 12
// blocks: 27 us against 17).
constexpr int tile_size(int mt, int kind) { return mt == 8 && kind != BK_VJP ? 32 : 16; }
constexpr int iterate_threads(int mt, int kind) { return 64 * 16 * mt / tile_size(mt, kind); }

template <int MT, int KIND>
__global__ __launch_bounds__(iterate_threads(MT, KIND), 2) void block_iterate_kernel(
    BlockTable tab, const float* __restrict__ partials, uint16_t* __restrict__ p_out, uint16_t* __restrict__ t_out,
    float* __restrict__ scratch, BlockSteps steps, int32_t pp) {
  constexpr int MP = 16 * MT, TS = tile_size(MT, KIND), NW = MP / TS, NT = 64 * NW;
  using S = Shape<MP, TS>;
  using Acc = typename S::Acc;
  constexpr int NR = S::NR, V = S::V, NV = S::NV, NQ = S::NQ;
  constexpr bool VJP = KIND == BK_VJP;
  constexpr int LDM = MP + 4;
  // the Gram matrix (and Z) in binary32 first, then the left factors
  union Lds {
    float gram[VJP ? 2 : 1][MP][LDM];
    Left<MP> left[VJP ? 2 : 1];
  };
  __shared__ __attribute__((aligned(16))) Lds lds;
  __shared__ float red[8];
  __shared__ int32_t mx[2][8];

  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const int c = lane % TS, h = lane / TS;
  const int blk = block_number();
  const BlockStack st = find_stack<KEY_BLOCK>(blk);
  const int b = blk - st.block0;

  // sum the partials, in order, into LDS (both triangles)
  constexpr int PF = block_part_floats(MT, KIND);
  const int parts = st.gsplit;
  const float* src = partials + st.part0 + int64_t(b) * parts * st.part;
  auto& L0 = lds.gram[0];
  auto& L1 = lds.gram[VJP ? 1 : 0];
  constexpr int IT = (PF / 4 + NT - 1) / NT;
  f32x4_t sum[IT];
#pragma unroll
  for (int it = 0; it < IT; ++it) {
    const int e = min(it * NT + tid, PF / 4 - 1);
    sum[it] = *gmem(reinterpret_cast<const f32x4_t*>(src + 4 * e));
  }
  for (int q = 1; q < parts; ++q) {
    src += st.part;
#pragma unroll
    for (int it = 0; it < IT; ++it) {
      const int e = min(it * NT + tid, PF / 4 - 1);
      sum[it] += *gmem(reinterpret_cast<const f32x4_t*>(src + 4 * e));
    }
  }
#pragma unroll
  for (int it = 0; it < IT; ++it) {
    const int e = it * NT + tid;
    if (e >= PF / 4) break;
    const int tile = e >> 6, rr = e & 15, gg = (e >> 4) & 3;
    constexpr int TRI = (MT / 2) * (MT + 1);
    if (!VJP || tile < TRI) {
      const int p = tile / (MT + 1), q = tile % (MT + 1);
      const int ti = q < MT - p ? p : MT - 1 - p, tj = q < MT - p ? p + q : MT - 1 - p + (q - (MT - p));
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int i = 16 * ti + 4 * gg + v, j = 16 * tj + rr;
        if (ti != tj || i <= j) {
          L0[i][j] = sum[it][v];
          L0[j][i] = sum[it][v];
        }
      }
    } else {
      const int z = tile - TRI, p = z / (2 * MT), q = z % (2 * MT);
      const int ti = q < MT ? p : MT - 1 - p, tj = q % MT;
#pragma unroll
      for (int v = 0; v < 4; ++v) L1[16 * ti + 4 * gg + v][16 * tj + rr] = sum[it][v];
    }
  }
  __syncthreads();

  // ||x||^2
  float tr = 0.f;
  for (int i = lane; i < MP; i += 64) tr += L0[i][i];
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) tr += __shfl_xor(tr, d);
  const float norm = __builtin_sqrtf(tr);
  // an infinite ||x||^2 may be the sum of finite squares: A_0 = (G 0) 0 would
  // be zero and P finite, so that the results came out as zeros
  const float inv = !steps.first ? 1.f : tr < __builtin_inff() ? 1.f / (norm + NORM_EPS) : __builtin_nanf("");

  // A_j and P (and their tangents D and dP) live as operands; C (E) holds what
  // the last product gave, 2^ec (2^ee) times the matrix.  Value i of a lane is
  // row row_of(i) of column col.
  Acc C[NR], E[VJP ? NR : 1];
  int ec = 0, ee = 0;
  Operand<NQ> oA, oP, oD, odP;
  const int col = TS * w + c;
  auto row_of = [&](int i) { return TS * (i / V) + Tile<TS>::row(i % V, h); };
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    C[i / V][i % V] = (L0[row_of(i)][col] * inv) * inv;
    if constexpr (VJP) E[i / V][i % V] = (0.5f * inv) * (L1[row_of(i)][col] + L1[col][row_of(i)]);
  }
  float* sc = nullptr;
  if constexpr (VJP) {
    // A_0 and D_0 are needed again for <dX_0, X_0>
    sc = scratch + int64_t(blk) * (2 * MP * MP) + 4 * tid;
#pragma unroll
    for (int i = 0; i < NV; i += 4) {
      *gmem(reinterpret_cast<f32x4_t*>(sc + i * NT)) = f32x4_t{C[i / V][i % V], C[i / V][i % V + 1], C[i / V][i % V + 2],
                                                               C[i / V][i % V + 3]};
      *gmem(reinterpret_cast<f32x4_t*>(sc + (NV + i) * NT)) = f32x4_t{E[i / V][i % V], E[i / V][i % V + 1],
                                                                      E[i / V][i % V + 2], E[i / V][i % V + 3]};
    }
  }

  Left<MP>& LA = lds.left[0];
  Left<MP>& LD = lds.left[VJP ? 1 : 0];
  int la = 0, ld = 0;  // powers of two of LA and LD
  auto split_one = [&](const Acc (&X)[NR], int e, Operand<NQ>& o) MUON_INLINE {
    const int x = scale_for(max_bits<Acc, NR, V>(X));
    o.ex = e + x;
    const float s = __builtin_amdgcn_ldexpf(1.f, x);
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      split_step<Acc, NR, V>(X, q, s, o.f[q][0], o.f[q][1]);
      if (NV >= 32) __builtin_amdgcn_sched_barrier(0);
    }
  };
  // C (E) as the wave's operand o (od)
  auto split_into = [&](Operand<NQ>& o, Operand<NQ>& od) MUON_INLINE {
    split_one(C, ec, o);
    if constexpr (VJP) split_one(E, ee, od);
  };
  // X to LDS, and as operand o
  auto put_one = [&](auto keep, const Acc (&X)[NR], Left<MP>& L, int x, Operand<NQ>& o) MUON_INLINE {
    const float s = __builtin_amdgcn_ldexpf(1.f, x);
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      f16x8_t f[2];
      split_step<Acc, NR, V>(X, q, s, f[0], f[1]);
#pragma unroll
      for (int l = 0; l < 2; ++l) {
        *reinterpret_cast<f16x8_t*>(&L.v[l][col][S::KS * q + 8 * h]) = f[l];
        if constexpr (decltype(keep)::value) o.f[q][l] = f[l];
      }
      if (NV >= 32) __builtin_amdgcn_sched_barrier(0);
    }
  };
  // C (E) to LDS, with one power of two for all waves; and as operand o (od)
  auto put = [&](auto keep, Operand<NQ>& o, Operand<NQ>& od) MUON_INLINE {
    // the power of two that each wave would take, and the least of them
    const int xc = ec + scale_for(max_bits<Acc, NR, V>(C));
    int xe = 0;
    if constexpr (VJP) xe = ee + scale_for(max_bits<Acc, NR, V>(E));
    if (lane == 0) {
      mx[0][w] = xc;
      if constexpr (VJP) mx[1][w] = xe;
    }
    __syncthreads();  // also: the reads of LDS before are done
    la = mx[0][0];
    if constexpr (VJP) ld = mx[1][0];
#pragma unroll
    for (int i = 1; i < NW; ++i) {
      la = min(la, mx[0][i]);
      if constexpr (VJP) ld = min(ld, mx[1][i]);
    }
    la = __builtin_amdgcn_readfirstlane(la);
    put_one(keep, C, LA, la - ec, o);
    if constexpr (VJP) {
      ld = __builtin_amdgcn_readfirstlane(ld);
      put_one(keep, E, LD, ld - ee, od);
    }
    if constexpr (decltype(keep)::value) {
      o.ex = la;
      od.ex = ld;
    }
    __syncthreads();
  };
  // (C, E) <- L (o, od) and its tangent LA od + LD o
  auto left_times = [&](const Operand<NQ>& o, const Operand<NQ>& od) MUON_INLINE {
    zero_sums<Acc, NR, V>(C);
    ec = la + o.ex;
    if constexpr (VJP) {
      zero_sums<Acc, NR, V>(E);
      multiply<MP, TS, 2>({&C, &E}, LA, {&o, &od}, c, h);
      // with the larger power of two for the sum, unless it could overflow:
      // where o is zero or below 2^-48 of what LD o adds to (rows of x that
      // are zero, y's are not)
      const int d = (ld + o.ex) - (la + od.ex);
      ee = la + od.ex;
      if (d <= 48) {
        ee = ld + o.ex;
        if (d != 0) {
#pragma unroll
          for (int i = 0; i < NV; ++i) E[i / V][i % V] = __builtin_amdgcn_ldexpf(E[i / V][i % V], d);
        }
        multiply<MP, TS, 1>({&E}, LD, {&o}, c, h);
      }
    } else {
      multiply<MP, TS, 1>({&C}, LA, {&o}, c, h);
    }
  };
  // C <- Q = a I + b A + c A A (E <- dQ) from A in C (D in E), left in oA (oD)
  auto form_q = [&](int t) MUON_INLINE {
    const float ca = steps.a[t], cb = steps.b[t], cc = steps.c[t];
    put(std::true_type{}, oA, oD);
    if (cc != 0.f) {
      left_times(oA, oD);
    } else {
      zero_sums<Acc, NR, V>(C);
      if constexpr (VJP) zero_sums<Acc, NR, V>(E);
    }
    combine<MP, TS>(C, cc, ec, cb, oA);
    if constexpr (VJP) combine<MP, TS>(E, cc, ee, cb, oD);
    ec = ee = 0;
#pragma unroll
    for (int kt = 0; kt < NR; ++kt)
      if (kt == w) {
#pragma unroll
        for (int v = 0; v < V; ++v) C[kt][v] += Tile<TS>::row(v, h) == c ? ca : 0.f;
      }
  };
  if (steps.steps > 0) form_q(0);  // P = Q
  if (steps.steps > 1) {
    put(std::true_type{}, oP, odP);
#pragma unroll 1
    for (int t = 1; t < steps.steps; ++t) {
      left_times(oA, oD);  // R = Q A
      split_into(oA, oD);
      left_times(oA, oD);  // A <- Q R
      form_q(t);
      put(std::false_type{}, oA, oD);
      left_times(oP, odP);  // P <- Q P
      if (t + 1 < steps.steps) split_into(oP, odP);
    }
  }
  // P is in C, dP in E
  if (steps.steps == 0) {
    ec = ee = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      C[i / V][i % V] = row_of(i) == col ? 1.f : 0.f;
      if constexpr (VJP) E[i / V][i % V] = 0.f;
    }
  }

#pragma unroll
  for (int i = 0; i < NV; ++i) {
    C[i / V][i % V] = __builtin_amdgcn_ldexpf(C[i / V][i % V], -ec);
    if constexpr (VJP) E[i / V][i % V] = __builtin_amdgcn_ldexpf(E[i / V][i % V], -ee);
  }
  if constexpr (VJP) {
    float shift = 0.f;
    if (steps.first) {
      // <dX_0, X_0> = <P, D_0> + <2 dP, A_0>
      float k = 0.f;
#pragma unroll
      for (int i = 0; i < NV; i += 4) {
        const f32x4_t a0 = *gmem(reinterpret_cast<const f32x4_t*>(sc + i * NT));
        const f32x4_t d0 = *gmem(reinterpret_cast<const f32x4_t*>(sc + (NV + i) * NT));
#pragma unroll
        for (int j = 0; j < 4; ++j) k += C[i / V][i % V + j] * d0[j] + 2.f * E[i / V][i % V + j] * a0[j];
      }
#pragma unroll
      for (int d = 32; d > 0; d >>= 1) k += __shfl_xor(k, d);
      if (lane == 0) red[w] = k;
      __syncthreads();
      k = 0.f;
#pragma unroll
      for (int q = 0; q < NW; ++q) k += red[q];
      // a zero block has no direction: the norm's gradient is taken as zero
      shift = norm > 0.f ? inv * (k / norm) : 0.f;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const float tt = (2.f * E[i / V][i % V]) * inv * inv;
      E[i / V][i % V] = row_of(i) == col ? tt - shift : tt;
    }
  }

  // out in bfloat16 parts, by rows, through LDS.  P X is not P^T X here: P is
  // the product Q_k ... Q_0, whose last factors carry the largest errors, and
  // they act on what the first ones have left of X's large singular values
  __syncthreads();
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    L0[row_of(i)][col] = C[i / V][i % V] * inv;
    if constexpr (VJP) L1[row_of(i)][col] = E[i / V][i % V];
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
    hipLaunchKernelGGL((block_iterate_kernel<MT, KIND>), dim3(blocks), dim3(iterate_threads(MT, KIND)), 0, stream, tab, partials,  \
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
