// Types shared by the host side of the expert products and of the head's loss
// (muon_experts.h, muon_head.h) and their kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace muon {

// C[i][j] = sum_k P[i][k] Q[j][k] (i < m, j < n), the form of every product
// here.  An operand lies in row form (k contiguous) or in k-row form (the rows of
// C, or its columns, contiguous):
//   NT  P and Q in row form      y = x W^T, logits
//   NN  P row form, Q k-row      grad_x = grad_y W
//   TN  both k-row form          grad_W = grad_y^T x
enum ProductForm : int { FORM_NT = 0, FORM_NN = 1, FORM_TN = 2 };

// What becomes of C.
//   STORE  out = C + addend, rounded to out's type
//   LSE    a maximum and a sum of exponentials for every row and tile of columns,
//          and the target's logit
//   DZ     the gradient of the loss with respect to the logits C
//   STORE_TARGET  (NN, TN of bfloat16 gradients of the logits) C with what these hold of
//          their targets made whole by `rest`, stored
// (_CAP: with a soft cap, _LARGE_CAP: of bfloat16 operands above FAST_CAP; product_epilogue
// chooses.)
enum ProductEpilogue : int {
  EPI_STORE = 0, EPI_LSE = 1, EPI_DZ = 2, EPI_LSE_CAP = 3, EPI_DZ_CAP = 4, EPI_LSE_LARGE_CAP = 5, EPI_DZ_LARGE_CAP = 6,
  EPI_STORE_TARGET = 7
};
constexpr bool epi_store(int e) { return e == EPI_STORE || e == EPI_STORE_TARGET; }
constexpr bool epi_lse(int e) { return e == EPI_LSE || e == EPI_LSE_CAP || e == EPI_LSE_LARGE_CAP; }
constexpr bool epi_dz(int e) { return e == EPI_DZ || e == EPI_DZ_CAP || e == EPI_DZ_LARGE_CAP; }
constexpr bool epi_cap(int e) { return e >= EPI_LSE_CAP && e <= EPI_DZ_LARGE_CAP; }
// Up to this cap logits of bfloat16 operands take the soft cap's short form, whose error of
// 5 2^-24 cap is then no more than that of a binary32 logit of the cap's size (8192 x 1536 by
// 32768: loss 772 us, gradient 2415; the exact form 842 and 2495).
constexpr float FAST_CAP = 32.f;

// One launch.  Groups (experts) split the rows of P and C for NT and NN, and k
// for TN: group g has rows [offsets[g], offsets[g + 1]) of P (TN: of P and Q),
// offsets clamped to [0, rows].  Strides are in elements.
struct ProductArgs {
  const void* p;
  const void* q;
  void* out;
  const void* add;             // addend, in add's type and out's layout (no map), or null
  const int32_t* offsets;      // groups + 1, or null: one group of all rows
  const int32_t* map;          // row of `out` for a row of C, or null
  int64_t ld_p, ld_q, ld_out, ld_add;
  int64_t es_q, es_out;        // from one group's Q (NT, NN) or out (TN) to the next
  int64_t p_elems;             // elements from p's first to the end of its last row
  int64_t q_elems;             // the same for q (NT, NN: for one group's)
  int32_t groups, rows;
  int32_t m, n, k;             // m: TN; k: NT and NN
  int32_t chunk;               // k values of a tile at most (STORE only; see ProductPlan)
  float* part;                 // partial tiles of what is cut along k
  int32_t* queue;              // TN: the tiles in the order of product_order_kernel, taken as
                               // workgroups come free; null: every workgroup has its own
  int32_t f32;                 // type of p and q: 1 binary32, 0 bfloat16
  int32_t out_f32, add_f32;
  // head
  float cap, inv_cap;          // soft cap (0: none)
  int32_t col0;                // vocabulary index of column 0
  int32_t stat_tiles;          // tiles of columns of a row of `stats`
  const int32_t* target;       // of every row of C; null: targets
  const int64_t* targets;      // the caller's
  const float* lse;
  const float* ga;             // grad_loss + grad_lse
  const float* gb;             // grad_loss
  // bfloat16 gradients of the logits: what the rounding leaves of every row's element in the
  // target's column, by far the largest (0.9999 of the sum of squares in the d24 head's
  // gradient).  DZ writes it, STORE of NN (P) and TN (P) adds it; null: binary32
  float* rest;
  float* logit;                // the target's logit (soft-capped)
  float2* stats;               // [row][tile], with y = z log2 e: maximum of y, sum of 2^(y - maximum)
};

// Tile shapes.
enum ProductShape : int { SHAPE_NAIVE = 0, SHAPE_SMALL = 1, SHAPE_MEDIUM = 2, SHAPE_LARGE = 3, SHAPE_NARROW = 4, SHAPE_STREAM = 5 };
hipError_t launch_nt(int shape, int epi, const ProductArgs& a, int cus, hipStream_t stream);
hipError_t launch_nn(int shape, int epi, const ProductArgs& a, int cus, hipStream_t stream);
hipError_t launch_tn(int shape, int epi, const ProductArgs& a, int cus, hipStream_t stream);
// NT, STORE (without an addend or a map, out of the operands' type) and LSE, k a multiple
// of 16 bytes.
hipError_t launch_stream(int epi, const ProductArgs& a, hipStream_t stream);
constexpr int STREAM_TILE_N = 32, NAIVE_TILE_N = 16;

// How a product runs.  k may be cut into chunks, so that few tiles fill the GPU and
// one long group does not hold up the rest: a tile then takes `chunk` of k, writes
// binary32 partial sums, and a second kernel adds them, in order.
//   NT, NN  every tile is cut alike: partial sums are (chunk of k) x rows x n
//   TN      a group of more than `chunk` rows is cut into n_g pieces; with s_g the sum of
//           n - 1 over the groups before it, its partial matrices (m x n) are 2 s_g,
//           2 s_g + 1, .. (n <= 2 (n - 1), so groups do not meet), and there are 2 rows /
//           chunk of them at most.  Offsets whose groups overlap, and have more rows in
//           all than there are, are not cut.
struct ProductPlan {
  int shape;
  int32_t chunk;               // k of a chunk, whole stages
  size_t bytes;                // workspace that launch_product needs: partial sums,
  size_t queue;                // and these bytes before them (ProductArgs::queue)
};
ProductPlan product_plan(int form, int epi, const ProductArgs& a, int cus);
// STORE, LSE or DZ with the kind of soft cap that `a` has.
int product_epilogue(int epi, const ProductArgs& a);
// The queue, in int32_t: NUM_XCD counters of tiles taken, QUEUE_STEP apart (a line of
// memory each), the chunk, then pre[groups + 1] (sums of pieces, the groups with most rows
// first), order[groups] and slot[groups] (2 s_g).
constexpr int QUEUE_XCD = 8, QUEUE_STEP = 32, QUEUE_CHUNK = QUEUE_XCD * QUEUE_STEP, QUEUE_PRE = QUEUE_CHUNK + 1;
constexpr int64_t part_ld(int64_t n) { return (n + 3) / 4 * 4; }

// Columns of a tile of `stats` that launch_product writes.
int32_t product_tile_n(int form, int epi, const ProductArgs& a, int cus);
// `ws`: 256-byte aligned, product_plan's bytes.
hipError_t launch_product(int form, int epi, const ProductArgs& a, int cus, char* ws, hipStream_t stream);

// The head's rows that have a target, packed: offsets = {0, their number}, and
// for each its row, target, and (gradient) lse, ga and gb; the rows of x copied to
// xc.  Writes what rows without a target get: loss and lse (forward), grad_x.
struct HeadRows {
  const void* x;
  const int64_t* targets;
  const float* lse_in;
  const float* grad_loss;
  const float* grad_lse;       // may be null
  void* xc;
  int32_t* offsets;
  int32_t* row;
  int32_t* target;
  float* lse_c;
  float* ga;
  float* gb;
  float* loss;                 // forward: written where there is no target
  float* lse_out;
  void* grad_x;                // gradient: zeroed where there is no target; may be null
  int64_t ld_x, ld_xc, ld_grad_x;
  int64_t ignore_index, vocab;
  int32_t rows, dim, f32;
  int32_t chunk;               // rows of a workgroup
};
hipError_t launch_head_rows(const HeadRows& a, hipStream_t stream);

// loss and lse from the tiles' maxima and sums: of the packed rows (`targets` null), or
// of all rows, with what those without a target get.
struct HeadFinish {
  const float2* stats;
  const float* logit;
  const int32_t* offsets;
  const int32_t* row;
  const int64_t* targets;
  int64_t ignore_index, vocab;
  float* loss;
  float* lse;
  int32_t tiles, rows;
};
hipError_t launch_head_finish(const HeadFinish& a, hipStream_t stream);

}  // namespace muon
