/*
 * muon_experts.h -- C ABI of libmuon_mi355x.so, continued: products grouped by
 * expert, with their gradients.
 *
 * A layer of experts is one stack of weights W_0 .. W_{E-1}, out_dim x in_dim
 * each (the stack that muon_step_blocks takes for narrow experts, or the
 * matrices that muon_step_batched takes).  Its input is a packed matrix of
 * rows sorted by expert: rows offsets[e] .. offsets[e + 1] - 1 belong to
 * expert e, any number of them, none included.  For a row r of expert e
 *
 *   y[r]      = W_e x[r]                              muon_experts_product
 *   grad_x[r] = W_e^T grad_y[r]                       muon_experts_product_vjp
 *   grad_W_e  = sum over the rows r of e of grad_y[r] x[r]^T
 *
 * Conventions are those of muon.h (device memory of the current device, row
 * strides in elements, validation before anything is enqueued, no
 * synchronisation, status codes), and:
 *   - offsets is a device array of experts + 1 int32, read when the kernels
 *     run, so a router on the GPU needs no synchronisation.  Offsets are taken
 *     as at most `rows` and at least 0, and an expert whose end is not above
 *     its start as one without rows: no value of theirs makes a call read or
 *     write out of range.  Rows that lie in more than one range get any values in
 *     y and grad_x.
 *   - Rows before offsets[0] and from offsets[experts] on belong to no expert:
 *     what they hold does not matter, and y and grad_x stay as they were there.
 *   - An expert without rows has grad_W_e = 0 (accumulate: unchanged).
 *   - Elements outside the matrices (row padding, what lies between experts) are
 *     not written, and do not change results.  They, and rows of no expert, may be
 *     read within the tensor, from its first element to its last.
 *   - Tensors overlap (ALIAS where one of them is written) where their address
 *     ranges, first element to last, do: columns of one buffer beside each other
 *     are refused, though their elements are apart.
 *   - bfloat16 tensors are multiplied on the bfloat16 matrix cores (products
 *     exact), binary32 ones to binary32 accuracy: a product is off by 2^-24 of
 *     itself at most, and elements below 2^-110 in magnitude count with an error
 *     of up to 2^-134.  Sums are binary32, and results are rounded once.
 *   - A NaN or an infinity reaches the results whose sums it takes part in (the
 *     row, or the expert's grad_W) and no others.  They are NaN or infinite, as the
 *     formulas have it; with binary32 tensors also NaN where the formula is infinite.
 *   - The same call gives the same bits every time, captured or not.
 *   - Workspace: with workspace = NULL the library keeps one per device (grown
 *     on demand, freed by muon_release_workspace), and calls of this header and
 *     of muon_head.h that use it run one after another on a device, in the
 *     order they were made, whatever their streams.  With a workspace of the
 *     caller's (256-byte aligned device memory of
 *     muon_experts_workspace_bytes bytes) calls with different workspaces may
 *     overlap; those that share one must not.  A call that needs none (0
 *     bytes) may overlap any other.
 *   - While launches are timed (muon_timing_enable) products count as
 *     MUON_KC_COMBINE, logits as MUON_KC_GRAM, the head's packing as
 *     MUON_KC_MOMENTUM and its last pass as MUON_KC_NORM.
 *   - Capture: a call on a capturing stream that needs a workspace needs one of
 *     the caller's (UNSUPPORTED without).  It records kernels on `stream` only.
 */
#ifndef MUON_MI355X_EXPERTS_H
#define MUON_MI355X_EXPERTS_H

#include "muon.h"

#ifdef __cplusplus
extern "C" {
#endif

/* How a weight lies in memory.                                              */
typedef enum muon_weight_order {
  MUON_WEIGHT_OUT_IN = 0,  /* out_dim rows of in_dim contiguous elements     */
  MUON_WEIGHT_IN_OUT = 1   /* in_dim rows of out_dim contiguous elements     */
} muon_weight_order;

/* experts in [0, 2048]; rows (of x, y and their gradients) in [0, 2^24];
 * in_dim, out_dim in [1, 65536].  Row strides >= the row's length (any where
 * there is one row) and at most 2^21; expert strides stride_* >= 0 (the
 * weights; 0: one weight for all), for grad_w so that experts do not share
 * elements.  dtype: F32 or BF16, of x, w, y, grad_y and grad_x;
 * grad_w_dtype: F32, or BF16 where dtype is.  grad_w has w's order.
 * accumulate: 0, or 1: grad_w is added to.  Fields that a call does not use
 * are ignored.  reserved: 0.                                                */
typedef struct muon_experts_desc {
  int64_t experts, rows, in_dim, out_dim;
  int64_t ld_x, ld_y;                  /* ld_y: y, or grad_y               */
  int64_t ld_w, stride_w;
  int64_t ld_grad_x;
  int64_t ld_grad_w, stride_grad_w;
  int32_t dtype, grad_w_dtype;
  int32_t w_order;                     /* a muon_weight_order               */
  int32_t accumulate;
  int64_t reserved;
} muon_experts_desc;

/* y[r] = W_e x[r].
 * Errors: INVALID_ARGUMENT (null pointer, bad size or stride, workspace too
 * small), UNSUPPORTED (dtype, alignment, size cap, capture without a workspace),
 * ALIAS (y overlaps another buffer), OUT_OF_MEMORY, HIP.                    */
muon_status muon_experts_product(const void* x, const void* w, const int32_t* offsets, void* y,
                                 const muon_experts_desc* desc, void* workspace, uint64_t workspace_bytes,
                                 void* stream);

/* The gradients of <muon_experts_product(x, w), grad_y>.  grad_x or grad_w may
 * be NULL and is then not computed; x is needed (and read) for grad_w only, w
 * for grad_x only, and either may be NULL else.  Errors as
 * muon_experts_product.                                                     */
muon_status muon_experts_product_vjp(const void* x, const void* w, const int32_t* offsets, const void* grad_y,
                                     void* grad_x, void* grad_w, const muon_experts_desc* desc, void* workspace,
                                     uint64_t workspace_bytes, void* stream);

/* The calls, for muon_experts_workspace_bytes.                              */
typedef enum muon_experts_op {
  MUON_EXPERTS_PRODUCT = 0,
  MUON_EXPERTS_GRAD_X = 1,
  MUON_EXPERTS_GRAD_W = 2,
  MUON_EXPERTS_GRAD_X_W = 3
} muon_experts_op;

/* Workspace bytes of a call of `op` (a muon_experts_op) on the current device;
 * 0 for a call that needs none, and on error.                               */
uint64_t muon_experts_workspace_bytes(int32_t op, const muon_experts_desc* desc);

#ifdef __cplusplus
}
#endif

#endif /* MUON_MI355X_EXPERTS_H */
