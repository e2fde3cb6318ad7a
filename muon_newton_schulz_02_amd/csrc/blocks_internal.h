// Types shared by the host side of the block operators and their kernels
// (stacks of blocks with min(rows, cols) <= 128; see muon_blocks.h).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace muon {

constexpr int BLOCK_MAX_M = 128;

enum BlockFlags : uint32_t {
  BF_X_BF16 = 1,      // x is bfloat16 (else binary32)
  BF_Y_BF16 = 2,
  BF_OUT_BF16 = 4,
  BF_TR = 8,          // rows > cols: element (i, j) of the wide block is at j * ld + i
  BF_WRITEBACK = 16   // apply: out is a weight, out <- rnd(out * d - t * O)
};

// One stack as the kernels see it, at one stage of the computation.
struct BlockStack {
  const void* x;      // input, gradient of the step, or iterate of an earlier stage
  int64_t x_ld, x_bs;
  const void* y;      // gradient: cotangent; step: momentum (binary32, written by the gram pass)
  int64_t y_ld, y_bs;
  void* out;
  int64_t out_ld, out_bs;
  float* upd;         // exported update, blocks x rows x cols contiguous, or null
  int64_t part0;      // first float of the stack's Gram partials
  int64_t part;       // floats from one workgroup's partial to the next (the same at every stage)
  int32_t m, n;       // wide shape
  int32_t cols;       // row length of upd
  int32_t block0;     // index of the stack's first block in the launch
  int32_t goff, gsplit, gchunk;  // gram workgroups: first, per block, columns of each
  int32_t aoff, asplit, achunk;  // apply workgroups
  uint32_t flags;
  float t, d;         // write-back scalars
  int32_t blocks;
};

// First workgroups (and blocks) of the stacks, by kernel: what a workgroup
// searches for its stack.
enum BlockKey : int { KEY_GRAM = 0, KEY_BLOCK = 1, KEY_APPLY = 2, KEY_COUNT = 3 };

// The stacks of a launch: up to BLOCK_INLINE in the kernel's arguments, else
// in a device table (written by block_table_kernel, so that a call needs no
// host-to-device copy): ext_keys holds KEY_COUNT lists of `count` keys.
constexpr int BLOCK_INLINE = 16;
struct BlockTable {
  const BlockStack* ext;
  const int32_t* ext_keys;
  int32_t count;
  int32_t first;      // number of the launch's first workgroup (or block): a launch may take a part of them
  int32_t keys[KEY_COUNT][BLOCK_INLINE];
  BlockStack inl[BLOCK_INLINE];
};
static_assert(sizeof(BlockTable) + 512 <= 4096, "kernel arguments stay below 4 KiB");

// Momentum of the step: M <- beta M + g1 G, U = nesterov ? g1 G + beta M : M
// with g1 = 1 (heavy ball) or fl32(1 - beta) (EMA).
struct BlockMom {
  float beta, g1;
  int32_t nesterov, ema;
};

// The steps of one stage of the m x m recursion.
constexpr int BLOCK_STAGE_STEPS = 32;
struct BlockSteps {
  float a[BLOCK_STAGE_STEPS], b[BLOCK_STAGE_STEPS], c[BLOCK_STAGE_STEPS];
  int32_t steps;
  int32_t first;      // x is not normalised yet: fold 1 / (||x|| + eps)
};

enum BlockKind : int { BK_X = 0, BK_STEP = 1, BK_VJP = 2 };

// Row tiles of 16 that a block of m rows is padded to: 2, 4 or 8 (the
// kernels' template sizes; 32, 64 or 128 rows).
constexpr int block_mt(int m) { return m <= 32 ? 2 : m <= 64 ? 4 : 8; }
// Floats of a Gram partial: the upper triangle of 16 x 16 tiles, and for the
// gradient all tiles of y x^T.
constexpr int block_part_floats(int mt, int kind) {
  return ((mt / 2) * (mt + 1) + (kind == BK_VJP ? mt * mt : 0)) * 256;
}
// The gram and apply passes work on tiles of all 16 MT rows by this many
// columns, 8192 elements, 16 for each of the 512 threads.
constexpr int BLOCK_THREADS = 512;
constexpr int block_kc(int mt) { return 512 / mt; }
// Element offsets within a tile are 32-bit byte offsets: at most 256 rows
// apart by this row stride.
constexpr int64_t BLOCK_MAX_LD = int64_t(1) << 21;
// Type of x known when a kernel is compiled, or read from the flags.
enum BlockXType : int { BX_F32 = 0, BX_BF16 = 1, BX_ANY = 2 };

// One launch of block_table_kernel: runs of stacks that differ in their
// pointers only, each given by its first member.
constexpr int BLOCK_BATCH = 96, BLOCK_CLASSES = 4;
struct BlockTableBatch {
  int32_t n;
  int32_t first[BLOCK_CLASSES];   // first entry of each run (runs not used: n)
  BlockStack cls[BLOCK_CLASSES];
  const void* x[BLOCK_BATCH];
  const void* y[BLOCK_BATCH];
  void* out[BLOCK_BATCH];
  float* upd[BLOCK_BATCH];
};
static_assert(sizeof(BlockTableBatch) <= 4096, "kernel arguments stay below 4 KiB");

// The launchers.  pl: bfloat16 parts of an element of x (1, 2, 3); pp: parts
// of an element of P (2, 3); xbf: x is bfloat16 in every stack.
// Writes a table of `count` stacks and its keys to device memory.
hipError_t launch_block_table(const BlockStack* host, int32_t count, BlockStack* dev, int32_t* keys,
                              hipStream_t stream);
hipError_t launch_block_gram(int mt, int pl, int kind, bool xbf, const BlockTable& tab, int32_t wgs, float* partials,
                             const BlockMom& mom, hipStream_t stream);
// Sums the partials of every block, runs the recursion and writes P (and, for
// the gradient, T) as pp planes of bfloat16 parts, mp x mp each.  scratch: 2
// mp x mp binary32 matrices per block (gradient only).
hipError_t launch_block_iterate(int mt, int pp, int kind, const BlockTable& tab, int32_t blocks,
                                const float* partials, uint16_t* p_out, uint16_t* t_out, float* scratch,
                                const BlockSteps& steps, hipStream_t stream);
hipError_t launch_block_apply(int mt, int pl, int pp, int kind, bool xbf, const BlockTable& tab, int32_t wgs,
                              const uint16_t* p, const uint16_t* t, const BlockMom& mom, hipStream_t stream);

}  // namespace muon
