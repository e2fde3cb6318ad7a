// Tile code of the products of the experts and of the head (products_internal.h):
// operand staging, the MFMA k-loop and the epilogues.  Each including file gets its
// own copy (anonymous namespace).
//
// A persistent grid walks the tiles of C, BM x BN each.  Operands go from memory
// through registers to LDS, one stage (128 bytes of k a row: 64 bfloat16 or 32
// binary32) at a time, double-buffered; the k-loop overlaps, inside each wave, a
// k-slab's MFMAs with the LDS reads of the next one, the LDS writes of the next
// stage and the loads of the one after it.  A tile's first stage is loaded during
// the tile before.
//
// Operands are the caller's tensors as they lie: any row stride, any alignment of
// their element.  A load is 16 bytes at an element boundary (the memory unit takes
// any), and which 16 bytes is clamped so that none lies outside the tensor: rows
// past the tile's end read its last row, which only changes results that are not
// stored; the last stage of a tile moves a chunk that would leave the tensor back to
// its last 16 bytes, and shifts and masks it on the way to LDS, so that everything
// past the end of k is zero whatever memory holds there.  (A chunk of an earlier
// stage can pass the end of its row in k-row form only; the row after it is there, and
// as long as rows are 16 bytes apart that is inside the tensor.  The launcher sends
// anything narrower, and operands below 16 bytes, to the small kernel.)
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "products_device.h"

#pragma clang fp contract(off)

namespace muon {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef u32x4 u32x4_any __attribute__((aligned(2)));   // 16 bytes at any element
typedef __attribute__((address_space(1))) const char gchar;
typedef __attribute__((address_space(3))) char lchar;
typedef __attribute__((address_space(3))) u32x4 lu32x4;
typedef __attribute__((address_space(3))) u32x2 lu32x2;
typedef __attribute__((address_space(1))) const u32x4_any gload16;
typedef __attribute__((address_space(1))) u32x4_any gstore16;

constexpr int NUM_XCD = 8;
constexpr int KB = 128;     // bytes of k per stage

// This wave's LDS accesses complete, then s_barrier: unlike __syncthreads it does
// not wait for global loads and stores in flight.
__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// Tile shapes: BM x BN over WM x WN waves.  Binary32 operands become three bfloat16
// parts on their way to LDS, x = hi + mid + lo, each rounded to nearest: of an x in [1, 2)
// mid is 2^-8 at most and lo 2^-17, and the sum is x (but for bits below 2^-133, bfloat16's
// least number: elements under 2^-110 lose some).  A product is six on the bfloat16 matrix
// cores: hi hi, hi mid, mid hi, mid mid, hi lo, lo hi; the three left out are 2^-24 of it
// at most, and of either sign.  The binary32 matrix instructions do 1 / 16 of the bfloat16
// ones' work a cycle, so six of these are 2.7 times as fast.
template <int BM_, int BN_, int WM_, int WN_, bool F32_>
struct Shape {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, NT = WM_ * WN_ * 64;
  static constexpr bool F32 = F32_;
  static constexpr int ESZ = F32 ? 4 : 2, KE = KB / ESZ, PARTS = F32 ? 3 : 1, SLABS = KE / 16;
  static constexpr int WTP = BM / WM, WTQ = BN / WN, FP = WTP / 32, FQ = WTQ / 32;
  static constexpr int CP = BM * 8 / NT, CQ = BN * 8 / NT;   // 16-byte chunks of a stage per thread
  // One LDS buffer where two would not fit: a stage's fragments are then all in registers
  // before the next stage is stored.
  static constexpr bool SINGLE = F32 && BM + BN > 256;
  static_assert(CP >= 1 && CQ >= 1 && BM * 8 % NT == 0 && BN * 8 % NT == 0, "whole chunks per thread");
};

// LDS of an operand of R rows, bfloat16, part after part.  Row form: row r at r pitch,
// 16 bytes more than its k, so that a fragment read of 32 rows meets every bank evenly
// (144 and 80 bytes).  k-row form: k-row k at k * pitch; fragments come from
// ds_read_b64_tr_b16, whose half-wave reads 4 k-rows x 64 bytes, on distinct banks
// where the pitch is 64 or 192 modulo 256.
template <class S, int R, bool KROW>
struct Lds {
  static constexpr int pitch = !KROW ? S::KE * 2 + 16 : (R * 2 % 256 == 0 || R * 2 % 256 == 128) ? R * 2 + 64 : R * 2;
  static_assert(!KROW || pitch % 256 == 64 || pitch % 256 == 192, "banks");
  static constexpr int part = KROW ? S::KE * pitch : R * pitch;
  static constexpr int bytes = S::PARTS * part;
};

template <class S, int FORM>
struct Layout {
  static constexpr bool PK = FORM == FORM_TN, QK = FORM != FORM_NT;   // k-row form
  using LP = Lds<S, S::BM, PK>;
  using LQ = Lds<S, S::BN, QK>;
  // buffer b: P at b BUF, Q behind it
  static constexpr int BUF = LP::bytes + LQ::bytes, BYTES = (S::SINGLE ? 1 : 2) * BUF;
};

// ------------------------------------------------------------------ tiles

// One tile of C.
struct Tile {
  int g;            // group
  int lo;           // the group's first row
  int i0, j0;       // first row of C in the group, first column
  int m, n;         // rows and columns from there on
  int k0, k;        // first k, and how many
  int part;         // partial matrix that it goes to, or -1: it is all of k
};

// Where an operand of a tile comes from.
struct Source {
  const char* base;     // element (row 0 of the tile, k = 0)
  const char* begin;    // first byte of the tensor
  const char* end;      // one past its last
  // row stride in bytes: 2^23 at most, the head's logits' gradients (few rows of a long
  // vocabulary) 2^26; the rows of a tile that there are span less than 2^32
  uint32_t ld;
  int valid;            // rows (row form) or columns (k-row form) of the tile that exist
};

template <class S, int FORM, int OPD>
__device__ __forceinline__ Source source_of(const ProductArgs& a, const Tile& t) {
  constexpr int E = S::ESZ;
  Source s;
  // formed where it is used, from values the compiler takes for new ones: kept
  // through the k-loop the sources of two tiles would not fit the scalar registers
  int lo = __builtin_amdgcn_readfirstlane(t.lo), i0 = __builtin_amdgcn_readfirstlane(t.i0),
      j0 = __builtin_amdgcn_readfirstlane(t.j0), grp = __builtin_amdgcn_readfirstlane(t.g),
      k0 = __builtin_amdgcn_readfirstlane(t.k0);
  asm volatile("" : "+s"(lo), "+s"(i0), "+s"(j0), "+s"(grp), "+s"(k0));
  if constexpr (OPD == 0) {
    s.begin = reinterpret_cast<const char*>(a.p);
    s.end = s.begin + a.p_elems * E;
    s.ld = uint32_t(a.ld_p * E);
    s.valid = t.m;
    s.base = FORM == FORM_TN ? s.begin + (int64_t(lo) + k0) * s.ld + i0 * E : s.begin + (int64_t(lo) + i0) * s.ld + k0 * E;
  } else {
    s.begin = reinterpret_cast<const char*>(a.q) + (FORM == FORM_TN ? 0 : grp * a.es_q * E);
    s.end = s.begin + a.q_elems * E;
    s.ld = uint32_t(a.ld_q * E);
    s.valid = t.n;
    s.base = FORM == FORM_NT   ? s.begin + int64_t(j0) * s.ld + k0 * E
             : FORM == FORM_NN ? s.begin + int64_t(k0) * s.ld + j0 * E
                               : s.begin + (int64_t(lo) + k0) * s.ld + j0 * E;
  }
  return s;
}

// The address in scalar registers.
__device__ __forceinline__ const char* uniform(const char* p) {
  const uint64_t v = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane(uint32_t(v)), hi = __builtin_amdgcn_readfirstlane(uint32_t(v >> 32));
  return reinterpret_cast<const char*>(lo | (uint64_t(hi) << 32));
}

// This thread's loads of an operand: `at` advances from stage to stage, the
// offsets stay, until the last stage has its own.
template <int C>
struct Loads {
  const char* at;
  uint32_t off[C];
};

// Chunk c of a stage: row form, row c / 8 and 16 bytes at 16 (c % 8); k-row form,
// k-row c / (R ESZ / 16) and 16 bytes of it.
template <class S, int R, bool KROW>
__device__ __forceinline__ void chunk_at(int c, int& row, int& byte) {
  constexpr int PER = KROW ? R * S::ESZ / 16 : 8;
  row = c / PER;
  byte = (c % PER) * 16;
}

// A copy of the thread's index that the compiler takes for a new value: what is
// computed from it stays where it is used, instead of being kept in registers (or in
// scratch memory) through the k-loop.
__device__ __forceinline__ int fresh(int tid) {
  int t;
  asm volatile("v_mov_b32 %0, %1" : "=v"(t) : "v"(tid));
  return t;
}

template <class S, int R, bool KROW, int C>
__device__ __forceinline__ void first_loads(Loads<C>& l, const Source& s, int tid) {
  l.at = uniform(s.base);
  tid = fresh(tid);
#pragma unroll
  for (int i = 0; i < C; ++i) {
    int row, byte;
    chunk_at<S, R, KROW>(tid + S::NT * i, row, byte);
    if constexpr (KROW) l.off[i] = row * s.ld + (byte < s.valid * S::ESZ ? byte : 0);
    else l.off[i] = min(row, s.valid - 1) * s.ld + byte;
  }
}

// The last stage, kt, of k values in all.  Its loads count from `at`, 16 bytes
// before its base, or the tensor's begin; `most` is the offset of the tensor's last
// 16 bytes from there, which is then never negative.
struct Last {
  const char* at;
  uint32_t back;        // base - at
  uint32_t most;
};
template <class S, bool KROW>
__device__ __forceinline__ Last last_of(const Source& s, int kt) {
  const char* base = s.base + (KROW ? int64_t(kt) * S::KE * s.ld : int64_t(0));
  Last l;
  l.back = uint32_t(min(int64_t(16), int64_t(base - s.begin)));
  l.at = base - l.back;
  l.most = uint32_t(min(int64_t(0xFFFFFFFF), int64_t(s.end - 16 - l.at)));
  return l;
}

// The offset wanted for chunk c of it; false: past the end of k.
template <class S, int R, bool KROW>
__device__ __forceinline__ bool last_chunk(const Source& s, const Last& l, int c, int kt, int k, uint32_t& off, int& row,
                                           int& byte) {
  chunk_at<S, R, KROW>(c, row, byte);
  if constexpr (KROW) {
    off = row * s.ld + (byte < s.valid * S::ESZ ? byte : 0) + l.back;
    return kt * S::KE + row < k;
  } else {
    off = min(row, s.valid - 1) * s.ld + uint32_t(kt * KB + byte) + l.back;
    return kt * KB + byte < k * S::ESZ;
  }
}

// The last stage's loads.  WHOLE: every chunk of the product's operands lies inside its
// row or behind the end of k; one behind it reads the first of its row (k-row) instead.
template <class S, int R, bool KROW, bool WHOLE, int C>
__device__ __forceinline__ void last_loads(Loads<C>& l, const Source& s, int kt, int k, int tid) {
  tid = fresh(tid);
  if constexpr (WHOLE) {
    l.at = uniform(s.base + int64_t(kt) * (KROW ? int64_t(S::KE) * s.ld : int64_t(KB)));
#pragma unroll
    for (int i = 0; i < C; ++i) {
      int row, byte;
      chunk_at<S, R, KROW>(tid + S::NT * i, row, byte);
      if constexpr (KROW) l.off[i] = (kt * S::KE + row < k ? row * s.ld : 0u) + (byte < s.valid * S::ESZ ? byte : 0);
      else l.off[i] = min(row, s.valid - 1) * s.ld + (kt * KB + byte < k * S::ESZ ? byte : 0);
    }
    return;
  }
  const Last z = last_of<S, KROW>(s, kt);
  l.at = uniform(z.at);
#pragma unroll
  for (int i = 0; i < C; ++i) {
    int row, byte;
    uint32_t off;
    const bool in = last_chunk<S, R, KROW>(s, z, tid + S::NT * i, kt, k, off, row, byte);
    l.off[i] = in ? min(off, z.most) : 0u;
  }
}

template <int C>
__device__ __forceinline__ void load_chunks(u32x4 (&r)[C], const Loads<C>& l) {
  gchar* at = (gchar*)l.at;
#pragma unroll
  for (int i = 0; i < C; ++i) {
    uint32_t off = l.off[i];
    asm volatile("" : "+v"(off));      // 32 bits up to here: the instruction adds them to a scalar base
    r[i] = *reinterpret_cast<gload16*>(at + off);
  }
}

// bytes [s, 16) of v, zeros behind; s in [0, 16]
__device__ __forceinline__ u32x4 shift_down(u32x4 v, int s) {
  const uint64_t lo = v[0] | (uint64_t(v[1]) << 32), hi = v[2] | (uint64_t(v[3]) << 32);
  const int b = (8 * s) & 63;
  const uint64_t high = hi >> b, mixed = (lo >> b) | ((hi << 1) << (63 - b));
  const uint64_t l = s >= 16 ? 0 : s >= 8 ? high : mixed, h = s >= 8 ? 0 : high;
  return u32x4{uint32_t(l), uint32_t(l >> 32), uint32_t(h), uint32_t(h >> 32)};
}

// v's first `bytes` bytes, zeros behind (a multiple of 2; 16 and more: all)
__device__ __forceinline__ u32x4 keep_first(u32x4 v, int bytes) {
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    const int b = bytes - 4 * d;
    v[d] = b >= 4 ? v[d] : b == 2 ? (v[d] & 0xFFFFu) : 0u;
  }
  return v;
}

// Where this thread's chunk 0 lies in an operand's LDS buffer; chunk i is
// i chunk_step further.
template <class S, int R, bool KROW>
__device__ __forceinline__ int chunk_lds(int tid) {
  int row, byte;
  chunk_at<S, R, KROW>(tid, row, byte);
  return row * Lds<S, R, KROW>::pitch + byte * 2 / S::ESZ;
}
template <class S, int R, bool KROW>
constexpr int chunk_step() {
  constexpr int PER = KROW ? R * S::ESZ / 16 : 8;
  static_assert(S::NT % PER == 0, "whole rows between a thread's chunks");
  return S::NT / PER * Lds<S, R, KROW>::pitch;
}

// Four binary32 values as three times four bfloat16: the value, what is left, and what is
// left then, each rounded to nearest.  Values that would round to infinity start from the
// largest bfloat16 instead.  Infinities and NaN have NaN parts.  (A first part that is cut
// off, not rounded, saves two of 6.5 instructions a value and 1.5 % of the time, and leaves out
// four times as much.)
__device__ __forceinline__ void split4(const u32x4& x, u32x2 (&out)[3]) {
  constexpr float MOST = 3.38953139e38f;      // 0x7F7F0000
  float v[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = __uint_as_float(x[e]);
  out[0] = u32x2{float2_to_bf16x2_bits(__builtin_amdgcn_fmed3f(v[0], -MOST, MOST), __builtin_amdgcn_fmed3f(v[1], -MOST, MOST)),
                 float2_to_bf16x2_bits(__builtin_amdgcn_fmed3f(v[2], -MOST, MOST), __builtin_amdgcn_fmed3f(v[3], -MOST, MOST))};
#pragma unroll
  for (int p = 1; p < 3; ++p) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      v[2 * h] -= __uint_as_float(out[p - 1][h] << 16);
      v[2 * h + 1] -= __uint_as_float(out[p - 1][h] & 0xFFFF0000u);
      out[p][h] = float2_to_bf16x2_bits(v[2 * h], v[2 * h + 1]);
    }
  }
}

template <class S, int R, bool KROW>
__device__ __forceinline__ void store_chunk(const u32x4& v, lchar* dst) {
  if constexpr (!S::F32) {
    *reinterpret_cast<lu32x4*>(dst) = v;
  } else {
    u32x2 p[3];
    split4(v, p);
#pragma unroll
    for (int i = 0; i < 3; ++i) *reinterpret_cast<lu32x2*>(dst + i * Lds<S, R, KROW>::part) = p[i];
  }
}

// Chunks I0 .. I1 - 1 of a stage to LDS; `dst`: this thread's chunk 0.
template <class S, int R, bool KROW, int C>
__device__ __forceinline__ void store_chunks(const u32x4 (&r)[C], lchar* dst, int i0, int i1) {
#pragma unroll
  for (int i = 0; i < C; ++i)
    if (i >= i0 && i < i1) store_chunk<S, R, KROW>(r[i], dst + i * chunk_step<S, R, KROW>());
}

// The same for the last stage: what last_loads moved back is moved forward again,
// and what lies past the end of k becomes zero.
template <class S, int R, bool KROW, bool WHOLE, int C>
__device__ __forceinline__ void store_last(const u32x4 (&r)[C], const Source& s, int kt, int k, lchar* dst, int tid,
                                           int i0, int i1) {
  tid = fresh(tid);
  if constexpr (WHOLE) {
#pragma unroll
    for (int i = 0; i < C; ++i) {
      if (i < i0 || i >= i1) continue;
      int row, byte;
      chunk_at<S, R, KROW>(tid + S::NT * i, row, byte);
      const bool in = KROW ? kt * S::KE + row < k : kt * KB + byte < k * S::ESZ;
      u32x4 v = r[i];
#pragma unroll
      for (int d = 0; d < 4; ++d) v[d] = in ? v[d] : 0u;
      store_chunk<S, R, KROW>(v, dst + i * chunk_step<S, R, KROW>());
    }
    return;
  }
  const Last z = last_of<S, KROW>(s, kt);
#pragma unroll
  for (int i = 0; i < C; ++i) {
    if (i < i0 || i >= i1) continue;
    int row, byte;
    uint32_t off;
    const bool in = last_chunk<S, R, KROW>(s, z, tid + S::NT * i, kt, k, off, row, byte);
    u32x4 v = shift_down(r[i], in ? (off > z.most ? int(off - z.most) : 0) : 16);
    if constexpr (!KROW) v = keep_first(v, k * S::ESZ - (kt * KB + byte));
    store_chunk<S, R, KROW>(v, dst + i * chunk_step<S, R, KROW>());
  }
}

// ------------------------------------------------------------------ fragments

// This lane's place in fragment 0, k-slab 0 of a wave whose first row of the operand
// (column of C for Q) is w0.
template <class S, int R, bool KROW>
__device__ __forceinline__ int frag_lds(int w0, int lane) {
  using L = Lds<S, R, KROW>;
  const int half = lane >> 5;
  if constexpr (!KROW) return (w0 + (lane & 31)) * L::pitch + half * 16;
  // lane 4 e + m of each 16-lane group points at k-row e, columns 4 m .. 4 m + 3 of
  // its 16; lane j of the group receives k-rows 0 .. 3 of column j
  else return (8 * half + ((lane & 15) >> 2)) * L::pitch + 2 * (w0 + 16 * ((lane >> 4) & 1) + 4 * (lane & 3));
}

// F fragments of 32 rows of every part, one k-slab ks; `p`: this lane's place.
template <class S, int R, bool KROW, int F>
__device__ __forceinline__ void read_frags(u32x4* f, lchar* p, int ks) {
  using L = Lds<S, R, KROW>;
#pragma unroll
  for (int part = 0; part < S::PARTS; ++part) {
    lchar* q = p + part * L::part + ks * (KROW ? 16 * L::pitch : 32);
#pragma unroll
    for (int x = 0; x < F; ++x) {
      if constexpr (!KROW) {
        f[part * F + x] = *reinterpret_cast<const lu32x4*>(q + x * 32 * L::pitch);
      } else {
        typedef short s16x4 __attribute__((ext_vector_type(4)));
        typedef __attribute__((address_space(3))) s16x4 ls16x4;
        const u32x2 lo = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((ls16x4*)(q + x * 64)));
        const u32x2 hi = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((ls16x4*)(q + x * 64 + 4 * L::pitch)));
        f[part * F + x] = u32x4{lo[0], lo[1], hi[0], hi[1]};
      }
    }
  }
}

__device__ __forceinline__ void mfma(f32x16& acc, const u32x4& q, const u32x4& p) {
  acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, q), __builtin_bit_cast(bf16x8, p), acc, 0, 0, 0);
}

// ------------------------------------------------------------------ epilogues

// Accumulators: acc[j][i][4 g + e] is row wp WTP + 32 i + (lane & 31) and column
// wq WTQ + 32 j + 8 g + 4 (lane / 32) + e of the tile.

// Where a tile goes: its element (0, 0).
struct Out {
  char* at;
  const char* add;          // addend's element (0, 0), or null
  const int32_t* map;       // row of `at` for a row of the tile (from the tile's first), or null
  int64_t ld, ld_add;
};

template <int FORM>
__device__ __forceinline__ Out out_of(const ProductArgs& a, const Tile& t) {
  Out o;
  const int64_t row = t.i0 + (FORM == FORM_TN ? 0 : t.lo), g0 = FORM == FORM_TN ? t.g * a.es_out : 0;
  if (t.part >= 0) {
    o.ld = part_ld(a.n);
    o.at = reinterpret_cast<char*>(a.part + (int64_t(t.part) * (FORM == FORM_TN ? a.m : a.rows) + row) * o.ld + t.j0);
    o.add = nullptr;
    o.map = nullptr;
    o.ld_add = 0;
    return o;
  }
  const int64_t first = g0 + (a.map ? 0 : row * a.ld_out) + t.j0, first_add = g0 + row * a.ld_add + t.j0;
  o.at = reinterpret_cast<char*>(a.out) + first * (a.out_f32 ? 4 : 2);
  o.add = a.add ? reinterpret_cast<const char*>(a.add) + first_add * (a.add_f32 ? 4 : 2) : nullptr;
  o.map = a.map ? a.map + row : nullptr;
  o.ld = a.ld_out;
  o.ld_add = a.ld_add;
  return o;
}

// v[0 .. 7] (OF32: 4), `cnt` of them, to element `at` of out, + addend's `add_at`.
template <bool OF32>
__device__ __forceinline__ void store_run(const Out& out, bool add_f32, float* v, int64_t at, int64_t add_at, int cnt) {
  constexpr int N = OF32 ? 4 : 8;
  if (out.add) {
    if (add_f32) {
      const float* ad = reinterpret_cast<const float*>(out.add) + add_at;
      if (cnt == N) {
#pragma unroll
        for (int h = 0; h < N / 4; ++h) {
          const u32x4 w = *reinterpret_cast<gload16*>((gchar*)(ad + 4 * h));
#pragma unroll
          for (int e = 0; e < 4; ++e) v[4 * h + e] += __uint_as_float(w[e]);
        }
      } else {
#pragma unroll
        for (int e = 0; e < N; ++e)
          if (e < cnt) v[e] += ad[e];
      }
    } else {
      const uint16_t* ad = reinterpret_cast<const uint16_t*>(out.add) + add_at;
#pragma unroll
      for (int e = 0; e < N; ++e)
        if (e < cnt) v[e] += bf16_bits_to_float(ad[e]);
    }
  }
  if constexpr (OF32) {
    float* o = reinterpret_cast<float*>(out.at) + at;
    if (cnt == N) {
      *reinterpret_cast<gstore16*>((__attribute__((address_space(1))) char*)o) =
          u32x4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])};
    } else {
#pragma unroll
      for (int e = 0; e < N; ++e)
        if (e < cnt) o[e] = v[e];
    }
  } else {
    uint16_t* o = reinterpret_cast<uint16_t*>(out.at) + at;
    if (cnt == N) {
      *reinterpret_cast<gstore16*>((__attribute__((address_space(1))) char*)o) =
          u32x4{float2_to_bf16x2_bits(v[0], v[1]), float2_to_bf16x2_bits(v[2], v[3]),
                float2_to_bf16x2_bits(v[4 % N], v[5 % N]), float2_to_bf16x2_bits(v[6 % N], v[7 % N])};
    } else {
#pragma unroll
      for (int e = 0; e < N; ++e)
        if (e < cnt) o[e] = float_to_bf16_bits(v[e]);
    }
  }
}

// What a lane writes over its row's element in the target's column, for its FP rows:
// the accumulators have the softmax's part alone (a change of theirs under a branch
// costs as many copies as there are).
template <class S>
struct Patch {
  int col[S::FP];           // column of the tile; -1: not this lane
  float value[S::FP];
};

// grad_x = dl W (NN): the rest of a row whose target is among the tile's k, and that target's
// row of W, from which it is added to C (8192 x 1536 by 32768 707 us, 690 without; under a trace).
struct RowTarget {
  const uint16_t* q;        // W's row of the target, at the tile's first column
  int most;                 // four elements from there on end with W
  bool in;
  float rest;
};
__device__ __forceinline__ RowTarget row_target(const ProductArgs& a, const Tile& t, int r) {
  const int row = t.lo + t.i0 + min(r, t.m - 1), k = a.target[row] - a.col0 - t.k0;
  RowTarget z;
  z.in = r < t.m && k >= 0 && k < t.k;
  z.rest = z.in ? a.rest[row] : 0.f;
  const int64_t at = int64_t(t.k0 + (z.in ? k : 0)) * a.ld_q + t.j0;
  z.most = int(min(a.q_elems - 4 - at, int64_t(1) << 30));
  z.q = reinterpret_cast<const uint16_t*>(a.q) + at;
  return z;
}
// Four elements of it from column c; what would lie behind W's end is read before it, and shifted.
__device__ __forceinline__ uint64_t target_run(const RowTarget& z, int c) {
  typedef uint64_t u64_any __attribute__((aligned(2)));
  const int o = min(c, z.most);
  const uint64_t v = *gmem(reinterpret_cast<const u64_any*>(z.q + o)) >> (16 * (c - o) & 63);
  return z.in ? v : 0;                // a row without a target has read one that may hold anything
}

// C to `out` through LDS, a part of the tile's rows at a time where all do not fit ROOM
// bytes.  OF32: out is binary32.  WIDE: staged as binary32 (for binary32 outputs and
// addends), else as bfloat16.  TARGET: with what row_target adds.
template <class S, bool OF32, bool WIDE, int ROOM, bool TARGET = false>
__device__ __forceinline__ void store_tile(const f32x16 (&acc)[S::FQ][S::FP], const Out& out, bool add_f32, const Tile& t, char* stg, int tid,
                                           const Patch<S>* patch = nullptr, const ProductArgs* args = nullptr) {
  constexpr int ES = WIDE ? 4 : 2, EP = S::BN * ES + 16;
  constexpr int PASSES = S::BM * EP <= ROOM ? 1 : S::BM / 2 * EP <= ROOM ? 2 : S::BM / 4 * EP <= ROOM ? 4 : 8;
  constexpr int ROWS = S::BM / PASSES;
  static_assert(ROWS * EP <= ROOM && ROWS % 32 == 0, "staging fits");
  const int tt = fresh(tid);
  const int lane = tt & 63, half = lane >> 5, w = __builtin_amdgcn_readfirstlane(tt >> 6), wq = w % S::WN, wp = w / S::WN;
  constexpr int N = OF32 ? 4 : 8, CPR = S::BN / N;        // elements of a run, runs of a row
  constexpr int ITER = ROWS * CPR / S::NT, STEP = S::NT / CPR;
  static_assert(ITER * STEP == ROWS, "whole rows a step");
  const int row0 = tt / CPR, col = tt % CPR * N;
  // whole rows of the tile that lie evenly spaced: 32-bit offsets, no questions
  const bool plain = t.n >= S::BN && !out.map && !(WIDE && (out.add || !OF32));
  const uint32_t ld = uint32_t(out.ld * (OF32 ? 4 : 2));
  // the targets of all of a lane's rows at once, where the registers hold them
  constexpr bool AHEAD = TARGET && S::FP * S::FQ <= 4;
  RowTarget target[S::FP];
  if constexpr (AHEAD) {
#pragma unroll
    for (int i = 0; i < S::FP; ++i) target[i] = row_target(*args, t, wp * S::WTP + 32 * i + (lane & 31));
    __builtin_amdgcn_sched_barrier(0);
  }
#pragma unroll 1
  for (int pass = 0; pass < PASSES; ++pass) {
    if (pass > 0) lds_barrier();
    char* const lane_at = stg + (lane & 31) * EP + (wq * S::WTQ + 4 * half) * ES;
#pragma unroll
    for (int i = 0; i < S::FP; ++i) {
      const int r0 = wp * S::WTP + 32 * i - pass * ROWS;
      if (PASSES == 1 || (r0 >= 0 && r0 < ROWS)) {
        char* const at = lane_at + r0 * EP;
        // (all of a row's loads before the first is used)
        float rest = 0.f;
        uint64_t run[TARGET ? S::FQ : 1][4];
        if constexpr (TARGET) {
          if constexpr (!AHEAD) target[i] = row_target(*args, t, wp * S::WTP + 32 * i + (lane & 31));
          rest = target[i].rest;
#pragma unroll
          for (int j = 0; j < S::FQ; ++j)
#pragma unroll
            for (int g = 0; g < 4; ++g) run[j][g] = target_run(target[i], wq * S::WTQ + 4 * half + 32 * j + 8 * g);
          __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int j = 0; j < S::FQ; ++j)
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            char* d = at + (32 * j + 8 * g) * ES;
            float c0 = acc[j][i][4 * g], c1 = acc[j][i][4 * g + 1], c2 = acc[j][i][4 * g + 2], c3 = acc[j][i][4 * g + 3];
            if constexpr (TARGET) {
              const uint64_t v = run[j][g];
              c0 = __builtin_fmaf(rest, bf16_bits_to_float(uint32_t(v)), c0);
              c1 = __builtin_fmaf(rest, bf16_bits_to_float(uint32_t(v >> 16)), c1);
              c2 = __builtin_fmaf(rest, bf16_bits_to_float(uint32_t(v >> 32)), c2);
              c3 = __builtin_fmaf(rest, bf16_bits_to_float(uint32_t(v >> 48)), c3);
            }
            if constexpr (WIDE) *reinterpret_cast<f32x4*>(d) = f32x4{c0, c1, c2, c3};
            else *reinterpret_cast<u32x2*>(d) = u32x2{float2_to_bf16x2_bits(c0, c1), float2_to_bf16x2_bits(c2, c3)};
            if (g == 3) __builtin_amdgcn_sched_barrier(0);   // else all are rounded before any is stored
          }
        // after this lane's own write of the column, in order
        if (patch && patch->col[i] >= 0) {
          char* d = stg + (r0 + (lane & 31)) * EP + patch->col[i] * ES;
          if constexpr (WIDE) *reinterpret_cast<float*>(d) = patch->value[i];
          else *reinterpret_cast<uint16_t*>(d) = float_to_bf16_bits(patch->value[i]);
        }
      }
    }
    lds_barrier();
    const int rows = min(ROWS, t.m - pass * ROWS);
    const char* src = stg + row0 * EP + col * ES;
    if (plain) {
      auto to = (__attribute__((address_space(1))) char*)(out.at + int64_t(pass) * ROWS * ld);
      uint32_t off = row0 * ld + col * (OF32 ? 4 : 2);
#pragma unroll 4
      for (int k = 0; k < ITER; ++k) {
        if (row0 + k * STEP < rows) {
          const u32x4 v = *reinterpret_cast<const u32x4*>(src + k * STEP * EP);
          *reinterpret_cast<gstore16*>(to + off) = v;
        }
        off += STEP * ld;
      }
      continue;
    }
    const int cnt = min(N, t.n - col);
    if (cnt <= 0) continue;
#pragma unroll 1
    for (int r = row0; r < rows; r += STEP, src += STEP * EP) {
      const int row = pass * ROWS + r;
      const int64_t at = int64_t(out.map ? out.map[row] : row) * out.ld + col;
      if constexpr (!WIDE) {
        const u32x4 v = *reinterpret_cast<const u32x4*>(src);
        uint16_t* o = reinterpret_cast<uint16_t*>(out.at) + at;
        if (cnt == N) {
          *reinterpret_cast<gstore16*>((__attribute__((address_space(1))) char*)o) = v;
        } else {
#pragma unroll
          for (int e = 0; e < N; ++e)
            if (e < cnt) o[e] = uint16_t(v[e / 2] >> (16 * (e & 1)));
        }
      } else {
        float v[N];
#pragma unroll
        for (int h = 0; h < N / 4; ++h) {
          const f32x4 x = *reinterpret_cast<const f32x4*>(src + 16 * h);
#pragma unroll
          for (int e = 0; e < 4; ++e) v[4 * h + e] = x[e];
        }
        store_run<OF32>(out, add_f32, v, at, row * out.ld_add + col, cnt);
      }
    }
  }
}

// Every row's maximum and sum of exponentials over the tile's columns, and the
// target's logit: 8 bytes a row and tile go to memory instead of its logits.  A lane has
// 64 of a row's 256 columns (FQ 16-column parts of its wave's, a half of each), so its
// reductions are registers, one exchange between half-waves and four values in LDS.  Some
// 12 instructions a logit with a soft cap (two exponentials, a reciprocal), 4 without:
// 8192 x 1536 by 32768 786 us and 755.
template <class S, bool CAP, bool EXACT>
__device__ __forceinline__ void lse_tile(f32x16 (&acc)[S::FQ][S::FP], const ProductArgs& a, const Tile& t, char* smem,
                                         int tid) {
  const int tt = fresh(tid);
  const int lane = tt & 63, half = lane >> 5, w = tt >> 6, wq = w % S::WN, wp = w / S::WN;
  const int c0 = wq * S::WTQ + 4 * half;
  const bool whole = t.n >= S::BN;
  float2* part = reinterpret_cast<float2*>(smem);           // [row of the tile][wave column]
  const SoftCap cap = soft_cap(a);
  constexpr float scale = CAP ? 1.f : LOG2E;                // y = acc scale from here on
#pragma unroll
  for (int i = 0; i < S::FP; ++i) {
    const int r = wp * S::WTP + 32 * i + (lane & 31);
    const int target = r < t.m ? target_of(a, t.i0 + r) - t.j0 : -1;
    if constexpr (CAP) {
#pragma unroll
      for (int j = 0; j < S::FQ; ++j)
#pragma unroll
        for (int v = 0; v < 16; ++v) {
          acc[j][i][v] = capped_y<EXACT>(acc[j][i][v], cap);
          if (v % 8 == 7) __builtin_amdgcn_sched_barrier(0);     // few values at a time, or the chains spill
        }
    }
    if (!whole) {
#pragma unroll
      for (int j = 0; j < S::FQ; ++j)
#pragma unroll
        for (int v = 0; v < 16; ++v)
          if (c0 + 32 * j + 8 * (v >> 2) + (v & 3) >= t.n) acc[j][i][v] = -INFINITY;
    }
    if (__any(target >= wq * S::WTQ && target < (wq + 1) * S::WTQ)) {
#pragma unroll
      for (int j = 0; j < S::FQ; ++j)
#pragma unroll
        for (int v = 0; v < 16; ++v)
          if (target == c0 + 32 * j + 8 * (v >> 2) + (v & 3)) a.logit[t.i0 + r] = acc[j][i][v] * (CAP ? LN2 : 1.f);
    }
    float mx = -INFINITY;
#pragma unroll
    for (int j = 0; j < S::FQ; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) mx = fmaxf(mx, acc[j][i][v]);
    mx = fmaxf(mx, __shfl_xor(mx, 32)) * scale;
    const float base = mx == -INFINITY ? 0.f : mx;
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < S::FQ; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) {
        sum += __builtin_amdgcn_exp2f(__builtin_fmaf(acc[j][i][v], scale, -base));
        if (v % 8 == 7) __builtin_amdgcn_sched_barrier(0);
      }
    sum += __shfl_xor(sum, 32);
    if (half == 0) part[r * S::WN + wq] = make_float2(mx, sum);
  }
  lds_barrier();
  for (int r = tt; r < min(S::BM, t.m); r += S::NT) {
    float m = -INFINITY;
#pragma unroll
    for (int q = 0; q < S::WN; ++q) m = fmaxf(m, part[r * S::WN + q].x);
    const float base = m == -INFINITY ? 0.f : m;
    float sum = 0.f;
#pragma unroll
    for (int q = 0; q < S::WN; ++q) sum += part[r * S::WN + q].y * __builtin_amdgcn_exp2f(part[r * S::WN + q].x - base);
    a.stats[int64_t(t.i0 + r) * a.stat_tiles + t.j0 / S::BN] = make_float2(m, sum);
  }
}

// The logits become the loss's gradient with respect to them, but for the target's
// column, which goes to `patch`.  From lse it is one exponential a logit; 8192 x 1536 by
// 32768 with a soft cap 855 us under a trace, 512 MB of gradients written.
template <class S, bool CAP, bool EXACT>
__device__ __forceinline__ void gradient_tile(f32x16 (&acc)[S::FQ][S::FP], const ProductArgs& a, const Tile& t, int tid,
                                              Patch<S>& patch) {
  const int tt = fresh(tid);
  const int lane = tt & 63, w = tt >> 6, wq = w % S::WN, wp = w / S::WN;
  const int c0 = wq * S::WTQ + 4 * (lane >> 5);
  const SoftCap cap = soft_cap(a);
#pragma unroll
  for (int i = 0; i < S::FP; ++i) {
    const int r = min(wp * S::WTP + 32 * i + (lane & 31), t.m - 1) + t.i0;
    const int target = target_of(a, r) - t.j0;
    const float lse = a.lse[r] * LOG2E, ga = a.ga[r];
    const bool mine = target >= wq * S::WTQ && target < (wq + 1) * S::WTQ && ((target >> 2) & 1) == (lane >> 5);
    patch.col[i] = mine ? target : -1;
    patch.value[i] = 0.f;
    if (__any(mine)) {
      float l = 0.f;
#pragma unroll
      for (int j = 0; j < S::FQ; ++j)
#pragma unroll
        for (int v = 0; v < 16; ++v) l = target == c0 + 32 * j + 8 * (v >> 2) + (v & 3) ? acc[j][i][v] : l;
      if constexpr (CAP) {
        const float q = cap_r(l, cap);
        patch.value[i] = (ga * __builtin_amdgcn_exp2f(capped_y<EXACT>(l, q, cap) - lse) - a.gb[r]) * cap_slope(q);
      } else {
        patch.value[i] = ga * __builtin_amdgcn_exp2f(__builtin_fmaf(l, LOG2E, -lse)) - a.gb[r];
      }
      if (!S::F32 && mine) a.rest[r] = rest_of(patch.value[i]);
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int j = 0; j < S::FQ; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) {
        const float l = acc[j][i][v];
        if constexpr (CAP) {
          const float q = cap_r(l, cap);
          acc[j][i][v] = ga * (cap_slope(q) * __builtin_amdgcn_exp2f(capped_y<EXACT>(l, q, cap) - lse));
        } else {
          acc[j][i][v] = ga * __builtin_amdgcn_exp2f(__builtin_fmaf(l, LOG2E, -lse));
        }
        if (v % 8 == 7) __builtin_amdgcn_sched_barrier(0);
      }
  }
}

// grad_W = dl^T x (TN): the rests of the tile's rows of k whose target is among its rows of
// C, as a product of its own: 64 such rows of k at a time, in a fixed order, one element each
// (rounded to bfloat16: 2^-16 of the target's element), with their rows of x.  How many there
// are differs by target, all rows may have one; 8192 rows over 32768 columns are a stage or two
// a tile.  8192 x 1536 by 32768 677 us, 662 without (under a trace); 1337 x 333 by 20011, 60 %
// ignored, 31 and 26: the waits for targets, rests and rows of x.
template <class S>
__device__ __forceinline__ void add_targets_tn(f32x16 (&acc)[S::FQ][S::FP], const ProductArgs& a, const Tile& t, char* smem,
                                               int* wave_sum, int tid) {
  using LY = Layout<S, FORM_TN>;
  constexpr int PER = 16, CHUNK = S::NT * PER;
  static_assert(!S::F32 && LY::BUF + CHUNK * 4 <= LY::BYTES, "the list lies in the second buffer");
  uint32_t* list = reinterpret_cast<uint32_t*>(smem + LY::BUF);       // row of k 256 + row of C
  tid = fresh(tid);
  const int lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6), wq = w % S::WN, wp = w / S::WN;
  const int first = t.lo + t.k0, end = first + t.k, c0 = a.col0 + t.i0, m = min(t.m, S::BM);
  const char* q = reinterpret_cast<const char*>(a.q) + t.j0 * 2;
  // a wave looks through 64 rows of every `step`: its own, or, where there are few, all of them
  const bool few = end - first <= 64 * PER;
  const int step = few ? 64 : S::NT;
#pragma unroll 1
  for (int b = first; b < end; b += CHUNK) {
    const int r0 = b + (few ? lane : tid);
    int target[PER], count = 0, at = 0;
#pragma unroll
    for (int e = 0; e < PER; ++e) {
      target[e] = c0 - 1;
      if (b + step * e < end) target[e] = gmem(a.target)[min(r0 + step * e, end - 1)];
    }
#pragma unroll
    for (int e = 0; e < PER; ++e) {
      const int v = target[e] - c0;
      target[e] = r0 + step * e < end && v < m ? v : -1;
    }
#pragma unroll
    for (int e = 0; e < PER; ++e) count += __popcll(__ballot(target[e] >= 0));
    if (few) {
      if (count == 0) return;         // all waves
    } else {
      if (lane == 0) wave_sum[w] = count;
      lds_barrier();
      count = 0;
#pragma unroll
      for (int x = 0; x < S::NT / 64; ++x) {
        if (x < w) at += wave_sum[x];
        count += wave_sum[x];
      }
      count = __builtin_amdgcn_readfirstlane(count);
    }
    if (!few || w == 0) {
#pragma unroll
      for (int e = 0; e < PER; ++e) {
        const uint64_t votes = __ballot(target[e] >= 0);
        if (target[e] >= 0) list[at + __popcll(votes & ((uint64_t(1) << lane) - 1))] = uint32_t(r0 + step * e) << 8 | uint32_t(target[e]);
        at += __popcll(votes);
      }
    }
#pragma unroll 1
    for (int e0 = 0; e0 < count; e0 += S::KE) {
      lds_barrier();                  // the list is there, the stage before has been read
      // chunks as in a stage: x's rows, and rows of zeros but for a rest
      u32x4 x[S::CQ];
#pragma unroll
      for (int i = 0; i < S::CQ; ++i) {
        int row, byte;
        chunk_at<S, S::BN, true>(tid + S::NT * i, row, byte);
        const uint32_t r = e0 + row < count ? list[e0 + row] >> 8 : first;
        x[i] = *reinterpret_cast<gload16*>((gchar*)(q + int64_t(r) * a.ld_q * 2 + (byte < t.n * 2 ? byte : 0)));
      }
#pragma unroll
      for (int i = 0; i < S::CP; ++i) {
        int row, byte;
        chunk_at<S, S::BM, true>(tid + S::NT * i, row, byte);
        const uint32_t e = e0 + row < count ? list[e0 + row] : ~0u;
        const int d = int(e & 255) * 2 - byte;
        u32x4 v = {0, 0, 0, 0};
        if (e != ~0u && d >= 0 && d < 16) {
          const uint32_t bits = uint32_t(float_to_bf16_bits(a.rest[e >> 8])) << 8 * (d & 2);
#pragma unroll
          for (int z = 0; z < 4; ++z) v[z] = d >> 2 == z ? bits : 0;
        }
        *reinterpret_cast<u32x4*>(smem + row * LY::LP::pitch + byte) = v;
      }
#pragma unroll
      for (int i = 0; i < S::CQ; ++i) {
        int row, byte;
        chunk_at<S, S::BN, true>(tid + S::NT * i, row, byte);
        if (e0 + row >= count) x[i] = u32x4{0, 0, 0, 0};
        *reinterpret_cast<u32x4*>(smem + LY::LP::bytes + row * LY::LQ::pitch + byte) = x[i];
      }
      lds_barrier();
      lchar* fp = (lchar*)smem + frag_lds<S, S::BM, true>(wp * S::WTP, lane);
      lchar* fq = (lchar*)smem + LY::LP::bytes + frag_lds<S, S::BN, true>(wq * S::WTQ, lane);
#pragma unroll 1
      for (int ks = 0; ks < S::SLABS; ++ks) {
        if (e0 + 16 * ks >= count) break;
        u32x4 f[S::FQ + S::FP];
        read_frags<S, S::BN, true, S::FQ>(f, fq, 0);
        read_frags<S, S::BM, true, S::FP>(f + S::FQ, fp, 0);
        fq += 16 * LY::LQ::pitch;
        fp += 16 * LY::LP::pitch;
#pragma unroll
        for (int j = 0; j < S::FQ; ++j)
#pragma unroll
          for (int i = 0; i < S::FP; ++i) mfma(acc[j][i], f[j], f[S::FQ + i]);
      }
    }
    lds_barrier();                    // list and wave_sum have been read
  }
}

// ------------------------------------------------------------------ kernel

// Tiles of C go through the columns in bands of BAND rows of tiles, so that the
// tiles that run together on an XCD (32 or more) share panels of P and Q in its L2.
constexpr int BAND = 8;

// Tile number t.  NT, NN: pre counts the groups' tiles of rows; chunks of k follow each
// other, all tiles of one before those of the next.  TN: pre counts their pieces of k.
template <class S, int FORM>
__device__ __forceinline__ Tile tile_at(const ProductArgs& a, const int* pre, int chunk, int t) {
  Tile r;
  const int nt = (a.n + S::BN - 1) / S::BN;
  int mt, piece = 0;        // tiles of rows of the group (TN: of C)
  const int all = FORM == FORM_TN ? 0 : __builtin_amdgcn_readfirstlane(pre[a.groups]) * nt;
  if constexpr (FORM != FORM_TN) {
    piece = t / all;
    t -= piece * all;
  }
  mt = FORM == FORM_TN ? (a.m + S::BM - 1) / S::BM : 1;
  const int u = t / (mt * nt);
  int lo = 0, hi = a.groups;          // pre[lo] <= u < pre[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (pre[mid] <= u) lo = mid;
    else hi = mid;
  }
  r.g = __builtin_amdgcn_readfirstlane(lo);
  const int before = __builtin_amdgcn_readfirstlane(pre[r.g]), of = __builtin_amdgcn_readfirstlane(pre[r.g + 1]) - before;
  int slot = 2 * (before - r.g);
  if constexpr (FORM == FORM_TN) {
    if (a.queue) {
      const int32_t* order = a.queue + QUEUE_PRE + a.groups + 1;
      r.g = __builtin_amdgcn_readfirstlane(order[r.g]);
      slot = __builtin_amdgcn_readfirstlane(order[a.groups + r.g]);
    }
  }
  if constexpr (FORM == FORM_TN) {
    piece = u - before;
    t -= u * mt * nt;
  } else {
    mt = of;
    t -= before * nt;
  }
  const int b = t / (BAND * nt), rows = min(BAND, mt - b * BAND), v = t - b * BAND * nt;
  r.i0 = (b * BAND + v % rows) * S::BM;
  r.j0 = v / rows * S::BN;
  int first, end;
  group_range(a, r.g, first, end);
  first = __builtin_amdgcn_readfirstlane(first);
  end = __builtin_amdgcn_readfirstlane(end);
  r.lo = first < end ? first : 0;      // TN: a group without rows reads the tensor's first row, as zeros
  r.n = a.n - r.j0;
  const int k = FORM == FORM_TN ? end - first : a.k;
  r.m = FORM == FORM_TN ? a.m - r.i0 : end - first - r.i0;
  r.k0 = piece * chunk;                // below 2^31: a group's pieces end with its rows
  r.k = min(chunk, k - r.k0);
  if constexpr (FORM == FORM_TN) r.part = of > 1 ? slot + piece : -1;
  else r.part = k > chunk ? piece : -1;
  return r;
}

// The queue of TN's tiles.  Strips of consecutive tiles, a column of a band each, belong
// to the XCDs in turn, so that an XCD's tiles share panels in its L2; when all of its own
// are taken a workgroup goes on with the other XCDs'.  Which workgroup has a tile changes
// nothing in it.
template <class S>
__device__ __forceinline__ int strip_of(const ProductArgs& a) {
  return min(BAND, (a.m + S::BM - 1) / S::BM);
}
__device__ __forceinline__ int queue_tile(const ProductArgs& a, int xcd, int strip, int end) {
  for (int x = 0; x < QUEUE_XCD; ++x) {
    const int got = __hip_atomic_fetch_add(a.queue + xcd * QUEUE_STEP, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    const int64_t t = (int64_t(got / strip) * QUEUE_XCD + xcd) * strip + got % strip;
    if (t < end) return int(t);
    xcd = (xcd + 1) % QUEUE_XCD;
  }
  return end;                        // none is left
}

template <class S, int FORM, int EPI, bool WHOLE>
__global__ __launch_bounds__(S::NT) void product_kernel(const ProductArgs a) {
  using LY = Layout<S, FORM>;
  constexpr bool PK = LY::PK, QK = LY::QK;
  extern __shared__ __attribute__((aligned(16))) char smem[];
  int* pre = reinterpret_cast<int*>(smem + LY::BYTES);
  const int tid = threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6), wq = w % S::WN, wp = w / S::WN;

  // Which tiles are this workgroup's: workgroup b runs on XCD b % 8.  Tiles of equal
  // work (NT, NN): a contiguous eighth of them for each XCD.  TN, where k differs from
  // group to group: the grid takes as many consecutive tiles at a time as it has
  // workgroups, so that a long group is spread over all of them; or, with a queue, each
  // takes the next tile as it comes free, the longest ones first (queue_tile).
  const int xcd = blockIdx.x % NUM_XCD, slot = blockIdx.x / NUM_XCD, slots = gridDim.x / NUM_XCD;
  __shared__ int wave_sum[S::NT / 64];
  int tile, step, end, chunk = a.chunk;
  __shared__ int taken;
  if constexpr (FORM == FORM_TN) {
    if (a.queue) {
      chunk = a.queue[QUEUE_CHUNK];
      for (int g = tid; g <= a.groups; g += S::NT) pre[g] = a.queue[QUEUE_PRE + g];
      __syncthreads();
    } else {
      chunk = __builtin_amdgcn_readfirstlane(safe_chunk<S::NT>(a, pre, wave_sum, tid));
      group_sums<S::NT>(a.groups, pre, wave_sum, tid, [&](int g) {
        int lo, hi;
        group_range(a, g, lo, hi);
        return pieces_of(hi - lo, chunk);
      });
    }
    end = __builtin_amdgcn_readfirstlane(pre[a.groups]) * ((a.m + S::BM - 1) / S::BM) * ((a.n + S::BN - 1) / S::BN);
    tile = xcd * slots + slot;
    step = gridDim.x;
    if (a.queue) {
      if (tid == 0) taken = queue_tile(a, xcd, strip_of<S>(a), end);
      __syncthreads();
      tile = __builtin_amdgcn_readfirstlane(taken);
    }
  } else {
    group_sums<S::NT>(a.groups, pre, wave_sum, tid, [&](int g) {
      int lo, hi;
      group_range(a, g, lo, hi);
      return (hi - lo + S::BM - 1) / S::BM;
    });
    const int total = __builtin_amdgcn_readfirstlane(pre[a.groups]) * ((a.n + S::BN - 1) / S::BN) *
                      (epi_store(EPI) ? (a.k + chunk - 1) / chunk : 1);
    const int per = (total + NUM_XCD - 1) / NUM_XCD;
    tile = xcd * per + slot;
    end = min((xcd + 1) * per, total);
    step = slots;
  }
  if (tile >= end) return;

  // One register for each operand's stores and fragment reads; everything else is an
  // immediate (opaque, or the compiler keeps one register for each sum)
  lchar* put_at_p = (lchar*)smem + chunk_lds<S, S::BM, PK>(tid);
  lchar* put_at_q = (lchar*)smem + LY::LP::bytes + chunk_lds<S, S::BN, QK>(tid);
  lchar* frag_p = (lchar*)smem + frag_lds<S, S::BM, PK>(wp * S::WTP, lane);
  lchar* frag_q = (lchar*)smem + LY::LP::bytes + frag_lds<S, S::BN, QK>(wq * S::WTQ, lane);
  asm volatile("" : "+v"(put_at_p), "+v"(put_at_q), "+v"(frag_p), "+v"(frag_q));
  int turn = S::SINGLE ? 0 : LY::BUF;       // to the other buffer
  u32x4 rp[S::CP], rq[S::CQ];
  Loads<S::CP> lp;
  Loads<S::CQ> lq;
  // bytes from one stage of an operand in k-row form to the next: 64 k-rows of 2^25 bytes,
  // or 32 of 2^26, 2^31 at most
  const uint32_t step_p = uint32_t(S::KE * a.ld_p * S::ESZ), step_q = uint32_t(S::KE * a.ld_q * S::ESZ);
  // (a group without rows has one of zeros)
  auto stages = [](const Tile& t) { return max(1, (t.k + S::KE - 1) / S::KE); };
  // the first stage of a tile, into registers
  auto load_first = [&](const Tile& u) {
    const Source sp = source_of<S, FORM, 0>(a, u), sq = source_of<S, FORM, 1>(a, u);
    if (stages(u) > 1) {
      first_loads<S, S::BM, PK>(lp, sp, tid);
      first_loads<S, S::BN, QK>(lq, sq, tid);
    } else {
      last_loads<S, S::BM, PK, WHOLE>(lp, sp, 0, u.k, tid);
      last_loads<S, S::BN, QK, WHOLE>(lq, sq, 0, u.k, tid);
    }
    load_chunks(rp, lp);
    load_chunks(rq, lq);
  };
  // the addresses that stage g >= 1 of tile u is loaded from
  auto address = [&](const Tile& u, int g) {
    if (g < stages(u) - 1) {
      lp.at += PK ? step_p : KB;
      lq.at += QK ? step_q : KB;
    } else {
      last_loads<S, S::BM, PK, WHOLE>(lp, source_of<S, FORM, 0>(a, u), g, u.k, tid);
      last_loads<S, S::BN, QK, WHOLE>(lq, source_of<S, FORM, 1>(a, u), g, u.k, tid);
    }
  };
  constexpr int HP = (S::CP + 1) / 2, HQ = (S::CQ + 1) / 2, HF = (S::FP + 1) / 2;
  // chunks i0 .. i1 - 1 of an operand's stage g of tile u to LDS; last: g may be the last
  // stage
  auto put_p = [&](bool last, const Tile& u, int g, int i0, int i1) {
    if (last) store_last<S, S::BM, PK, WHOLE>(rp, source_of<S, FORM, 0>(a, u), g, u.k, put_at_p, tid, i0, i1);
    else store_chunks<S, S::BM, PK>(rp, put_at_p, i0, i1);
  };
  auto put_q = [&](bool last, const Tile& u, int g, int i0, int i1) {
    if (last) store_last<S, S::BN, QK, WHOLE>(rq, source_of<S, FORM, 1>(a, u), g, u.k, put_at_q, tid, i0, i1);
    else store_chunks<S, S::BN, QK>(rq, put_at_q, i0, i1);
  };
  // from one stage to the next the buffers that are stored to and read from change places
  auto swap_put = [&] {
    put_at_p += turn;
    put_at_q += turn;
    turn = -turn;
  };
  // The first stage of a tile, loaded before, to LDS; the second one into registers.
  // Before it, stores and reads point at one buffer; after it, at one each.
  auto prime = [&](const Tile& u) {
    const int n = stages(u);
    put_p(n == 1, u, 0, 0, S::CP);
    put_q(n == 1, u, 0, 0, S::CQ);
    swap_put();
    if (n > 1) {
      address(u, 1);
      load_chunks(rp, lp);
      load_chunks(rq, lq);
    }
  };
  Tile t = tile_at<S, FORM>(a, pre, chunk, tile);
  load_first(t);
  prime(t);

#pragma unroll 1
  while (true) {
    const int nk = stages(t);
    f32x16 acc[S::FQ][S::FP];
#pragma unroll
    for (int j = 0; j < S::FQ; ++j)
#pragma unroll
      for (int i = 0; i < S::FP; ++i)
#pragma unroll
        for (int v = 0; v < 16; ++v) acc[j][i][v] = 0.f;

    int ntile = tile + step;
    bool more = ntile < end;
    Tile tn = t;
    // the next tile's first stage, if there is one.  (TN: taken a stage before, and known to
    // all after a barrier)
    auto take = [&] {
      if constexpr (FORM == FORM_TN) {
        if (a.queue && fresh(tid) == 0) taken = queue_tile(a, blockIdx.x % NUM_XCD, strip_of<S>(a), end);
      }
    };
    auto load_next = [&] {
      if constexpr (FORM == FORM_TN) {
        if (a.queue) {
          ntile = __builtin_amdgcn_readfirstlane(taken);
          more = ntile < end;
        }
      }
      if (!more) return;
      tn = tile_at<S, FORM>(a, pre, chunk, ntile);
      load_first(tn);
    };

    lds_barrier();       // the first stage is in LDS, the tile before has left it
    {
      u32x4 F[2][S::PARTS * (S::FQ + S::FP)];
      auto frags = [&](u32x4* f, int ks) {
        read_frags<S, S::BN, QK, S::FQ>(f, frag_q, ks);
        read_frags<S, S::BM, PK, S::FP>(f + S::PARTS * S::FQ, frag_p, ks);
      };
      auto multiply = [&](const u32x4* f, int h) {
        // parts of Q and P, the small products first
        constexpr int QPART[6] = {0, 2, 1, 0, 1, 0}, PPART[6] = {2, 0, 1, 1, 0, 0};
#pragma unroll
        for (int x = S::F32 ? 0 : 5; x < 6; ++x)
#pragma unroll
          for (int j = 0; j < S::FQ; ++j)
#pragma unroll
            for (int i = 0; i < S::FP; ++i)
              if (i / HF == h) mfma(acc[j][i], f[QPART[x] * S::FQ + j], f[S::PARTS * S::FQ + PPART[x] * S::FP + i]);
      };
      // binary32: the splitting of the next stage (some 7 instructions a value) goes between
      // `mfmas` MFMAs, a few at a time: behind them it would wait for the last one, and
      // they for it
      auto interleave = [&](auto mfmas) {
        constexpr int N = decltype(mfmas)::value, CHUNKS = S::CP + S::CQ, VALU = CHUNKS * 26 / N + 1;
#pragma unroll
        for (int i = 0; i < N; ++i) {
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
          __builtin_amdgcn_sched_group_barrier(0x002, VALU, 0);
          __builtin_amdgcn_sched_group_barrier(0x200, (CHUNKS * 3 + N - 1) / N, 0);
        }
      };
      // One stage, kt: its MFMAs, the LDS writes of stage kt + 1 and the loads of stage kt + 2.
      // MODE 0: both in this tile; 1: stage kt + 1 is the last one, the loads are the
      // next tile's first stage (TN: in the last stage); 2: kt is the last one.
      auto stage = [&](const int kt, auto mode_c) {
        constexpr int MODE = decltype(mode_c)::value;
        constexpr bool LAST = MODE == 1;
        constexpr int NEXT = FORM == FORM_TN ? 2 : 1;
        if constexpr (MODE == 1) take();
        if constexpr (S::SINGLE) {
          // On entry F holds the stage's two slabs (the second one's reads may be on their
          // way).  The barriers: every wave has the stage, which may be overwritten; the
          // next one is there.
          multiply(F[0], 0);
          __builtin_amdgcn_sched_barrier(0);
          lds_barrier();
          multiply(F[0], 1);
          if constexpr (MODE != 2) {
            put_p(LAST, t, kt + 1, 0, S::CP);
            put_q(LAST, t, kt + 1, 0, S::CQ);
          }
          if constexpr (MODE == 0) interleave(std::integral_constant<int, 6 * S::FQ * (S::FP - HF)>{});
          __builtin_amdgcn_sched_barrier(0);
          if constexpr (MODE == 0) {
            address(t, kt + 2);
            load_chunks(rp, lp);
            load_chunks(rq, lq);
          }
          if constexpr (MODE == NEXT) load_next();
          if constexpr (MODE != 2) lds_barrier();
          if constexpr (MODE == 0) frags(F[0], 0);
          __builtin_amdgcn_sched_barrier(0);
          multiply(F[1], 0);
          multiply(F[1], 1);
          __builtin_amdgcn_sched_barrier(0);
          if constexpr (MODE == 0) frags(F[1], 1);
          __builtin_amdgcn_sched_barrier(0);
          return;
        }
        // the other buffer is published, and this one's readers are done
        auto turn_over = [&] {
          lds_barrier();
          frag_p -= turn;
          frag_q -= turn;
          if constexpr (MODE != 2) swap_put();
          if constexpr (MODE == 0) frags(F[0], 0);
          __builtin_amdgcn_sched_barrier(0);
        };
        frags(F[1], 1);
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (S::SLABS == 2) {
          multiply(F[0], 0);
          multiply(F[0], 1);
          if constexpr (MODE != 2) {
            put_p(LAST, t, kt + 1, 0, S::CP);
            put_q(LAST, t, kt + 1, 0, S::CQ);
          }
          if constexpr (MODE == 0) interleave(std::integral_constant<int, 6 * S::FQ * S::FP>{});
          __builtin_amdgcn_sched_barrier(0);
          if constexpr (MODE == 0) {
            address(t, kt + 2);
            load_chunks(rp, lp);
            load_chunks(rq, lq);
          }
          if constexpr (MODE == NEXT) load_next();
          turn_over();
          multiply(F[1], 0);
          multiply(F[1], 1);
          __builtin_amdgcn_sched_barrier(0);
          return;
        }
        multiply(F[0], 0);
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (MODE != 2) put_p(LAST, t, kt + 1, 0, HP);
        __builtin_amdgcn_sched_barrier(0);
        multiply(F[0], 1);
        __builtin_amdgcn_sched_barrier(0);
        frags(F[0], 2);
        __builtin_amdgcn_sched_barrier(0);
        multiply(F[1], 0);
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (MODE != 2) {
          put_p(LAST, t, kt + 1, HP, S::CP);
          put_q(LAST, t, kt + 1, 0, HQ);
        }
        __builtin_amdgcn_sched_barrier(0);
        multiply(F[1], 1);
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (MODE == 0) {
          address(t, kt + 2);
          load_chunks(rp, lp);
        }
        __builtin_amdgcn_sched_barrier(0);
        frags(F[1], 3);
        __builtin_amdgcn_sched_barrier(0);
        multiply(F[0], 0);
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (MODE != 2) put_q(LAST, t, kt + 1, HQ, S::CQ);
        __builtin_amdgcn_sched_barrier(0);
        multiply(F[0], 1);
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (MODE == 0) load_chunks(rq, lq);
        if constexpr (MODE == NEXT) load_next();
        turn_over();
        multiply(F[1], 0);
        multiply(F[1], 1);
        __builtin_amdgcn_sched_barrier(0);
      };
      if (nk > 1) {
        int kt = 0;
        frags(F[0], 0);
        if constexpr (S::SINGLE) frags(F[1], 1);
#pragma unroll 1
        for (; kt + 2 < nk; ++kt) stage(kt, std::integral_constant<int, 0>{});
        stage(kt, std::integral_constant<int, 1>{});
      } else if constexpr (FORM == FORM_TN) {
        take();
        lds_barrier();
      } else {
        load_next();
      }
      // (its first fragments are read here, not across the branches: they would go
      // through scratch memory)
      frags(F[0], 0);
      if constexpr (S::SINGLE) frags(F[1], 1);
      stage(nk - 1, std::integral_constant<int, 2>{});
    }

    constexpr bool EXACT = S::F32 || EPI == EPI_LSE_LARGE_CAP || EPI == EPI_DZ_LARGE_CAP;
    if constexpr (epi_lse(EPI)) {
      lse_tile<S, epi_cap(EPI), EXACT>(acc, a, t, smem, tid);
    } else if constexpr (epi_dz(EPI)) {
      Patch<S> patch;
      gradient_tile<S, epi_cap(EPI), EXACT>(acc, a, t, tid, patch);
      store_tile<S, S::F32, S::F32, LY::BYTES>(acc, out_of<FORM>(a, t), false, t, smem, tid, &patch);
    } else {
      if constexpr (EPI == EPI_STORE_TARGET && FORM == FORM_TN) add_targets_tn<S>(acc, a, t, smem, wave_sum, tid);
      const Out out = out_of<FORM>(a, t);
      if constexpr (S::F32) store_tile<S, true, true, LY::BYTES>(acc, out, a.add_f32, t, smem, tid);
      else {
        constexpr bool TARGET = EPI == EPI_STORE_TARGET && FORM == FORM_NN;
        if (a.out_f32 || t.part >= 0) store_tile<S, true, true, LY::BYTES, TARGET>(acc, out, a.add_f32, t, smem, tid, nullptr, &a);
        else if (a.add) store_tile<S, false, true, LY::BYTES, TARGET>(acc, out, a.add_f32, t, smem, tid, nullptr, &a);
        else store_tile<S, false, false, LY::BYTES, TARGET>(acc, out, false, t, smem, tid, nullptr, &a);
      }
    }
    if (!more) break;
    lds_barrier();
    prime(tn);
    tile = ntile;
    t = tn;
  }
}

template <class S, int FORM, int EPI, bool WHOLE>
hipError_t launch_whole(const ProductArgs& a, int cus, hipStream_t stream) {
  using LY = Layout<S, FORM>;
  const size_t lds = LY::BYTES + (size_t(a.groups) + 1) * 4;
  const int64_t nt = (a.n + S::BN - 1) / S::BN;
  // tiles of rows and pieces of k, at most
  const int64_t mt = FORM == FORM_TN ? (a.groups + int64_t(a.rows / a.chunk)) * ((a.m + S::BM - 1) / S::BM)
                                     : (a.rows / S::BM + int64_t(std::min(a.groups, a.rows))) *
                                           (epi_store(EPI) ? (a.k + a.chunk - 1) / a.chunk : 1);
  // workgroups that a compute unit holds: by its LDS, and by waves (8 a unit at 256 registers)
  const int fit = std::max(1, std::min(int((160 * 1024) / (lds + 64)), 2048 / S::NT / 4));
  const int64_t grid = std::min<int64_t>((mt * nt + NUM_XCD - 1) / NUM_XCD * NUM_XCD,
                                         int64_t(cus) / NUM_XCD * NUM_XCD * fit);
  if (grid <= 0) return hipSuccess;
  hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(&product_kernel<S, FORM, EPI, WHOLE>),
                                     hipFuncAttributeMaxDynamicSharedMemorySize, int(lds));
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((product_kernel<S, FORM, EPI, WHOLE>), dim3(unsigned(grid)), dim3(S::NT), lds, stream, a);
  return hipGetLastError();
}

// Two kernels: for operands whose 16-byte chunks end where their rows (k-row form), or
// k (row form), end, and for any others, whose last stage is shifted and masked (2 %
// slower on 8192 x 1536 by 32768 x 1536: 780 us against 764).
template <class S, int FORM, int EPI>
hipError_t launch_shape(const ProductArgs& a, int cus, hipStream_t stream) {
  constexpr int V = 16 / S::ESZ;
  const bool whole = FORM == FORM_TN ? a.m % V == 0 && a.n % V == 0 : a.k % V == 0 && (FORM == FORM_NT || a.n % V == 0);
  return whole ? launch_whole<S, FORM, EPI, true>(a, cus, stream) : launch_whole<S, FORM, EPI, false>(a, cus, stream);
}

// The shapes.  A stage of 256 x 256 needs half the loads and LDS reads a product of 128 x
// 128, and one workgroup of it fills a compute unit's registers (128 accumulators a lane)
// and LDS; the matrix cores are busy half the time at 1.7 to 2.0 GHz, to which their load
// brings the clock.  The smaller ones are for what does not fill the GPU with these.
//   bfloat16, 8192 rows, 1536 and 32768: logits (NT) 755 us, 1.09 PFLOP/s (tiles of 128
//   x 128 896); dl W (NN, cut in four) 725 to 755 with the sums; dl^T x (TN) 660 to 690, 1.2
//   16384 rows of eight groups, 1536 and 6144: NT 266 to 320 us by the groups' last tiles
//   binary32, 717 rows (1024, 30 % ignored), 768 and 10007: TN 71 to 77 us, 128 x 128 tiles
//   10 % more; 142 to 155 TFLOP/s of binary32 products, six times that of bfloat16 ones
// Narrow (128 x 64, four waves, two workgroups a unit) is for few columns (Kind).
// Medium: 1337 x 333 to 20011 of 60 % ignored rows, NN 24 us.  Small (32 rows), for few:
// 64 experts of 24 rows, 1536 to 2048, 78 us, 89 without it; 32 of 24, 768 to 256, 8.6 and 17.5;
// the loss of 17 to 64 rows of 1536 by 32768 24.5 and 28, of 768 by 10007 14 and 19.5 (bfloat16).
using Large = Shape<256, 256, 2, 4, false>;
using Medium = Shape<128, 128, 2, 2, false>;
using MediumTn = Shape<128, 256, 2, 4, false>;
using Small = Shape<32, 128, 1, 4, false>;
using Narrow = Shape<128, 64, 2, 2, false>;
using LargeF32 = Shape<256, 128, 4, 2, true>;
using MediumF32 = Shape<128, 128, 2, 4, true>;
using SmallF32 = Shape<32, 128, 1, 4, true>;

}  // namespace
}  // namespace muon
