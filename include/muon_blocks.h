/*
 * muon_blocks.h -- C ABI of libmuon_mi355x.so, continued: Newton-Schulz
 * orthogonalisation of stacks of small blocks, its gradient, and the Muon
 * step on such stacks.
 *
 * A stack is `blocks` matrices of rows x cols inside one tensor, a fixed
 * stride apart: the heads of an attention projection (consecutive rows, or
 * consecutive columns), the low-rank factors of adapters, the experts of a
 * narrow layer.  Every block is orthogonalised by itself, and
 * min(rows, cols) <= 128 (larger matrices: muon_ns_batched and
 * muon_step_batched in muon.h).
 *
 * With x one block, oriented m x n with m <= n (blocks with rows > cols are
 * transposed and transposed back),
 *
 *   X <- x / (||x||_F + 1e-7)
 *   repeat ns_steps times:  A <- X X^T ; X <- (a I + b A + c A A) X
 *   NS(x) = X
 *
 * as in muon.h (the polynomial Newton-Schulz iteration; N. J. Higham,
 * Functions of Matrices, ch. 8).  Every iterate is a polynomial in A_0 =
 * X_0 X_0^T times X_0, so a block needs one Gram product over n, a recursion
 * on m x m matrices
 *
 *   Q_j = a I + b A_j + c A_j^2 ; A_{j+1} = Q_j A_j Q_j ; P <- Q_j P
 *
 * and one product P X_0 over n, whatever the number of steps.  Gram matrices
 * square the condition number, so the recursion starts again from the Gram
 * matrix of the current iterate (one more pass over the block) before the
 * steps since the last one multiply small singular values by more than a
 * limit.  With g the growth by all steps (1.5 a cubic step, 3.4445 one of the
 * usual quintic):
 *   - bfloat16 results: 512, so that five quintic steps (g = 485) are one pass;
 *     150 where g is more; 48 for blocks of up to four rows, and of up to 16
 *     with n < 4 m;
 *   - binary32 results: sqrt(3.5 g), at least 12 and at most 48 (five quintic
 *     steps 3 + 2, eight cubic ones 4 + 4); 12 where g is more than 512, and for
 *     blocks of few rows as above or with n < 2 m, whose gradient takes a Gram
 *     matrix for every step.
 * There are as few stages as that allows, as even as can be.  Measured against
 * float64:
 *   - bfloat16 results and gradients are off by their rounding and up to 3e-3
 *     more (one singular value 100 to 3000 times the others); where x is
 *     binary32 and of rank one alone, by 2^-18 g;
 *   - binary32 ones by up to about five times what the same iteration carried
 *     out in binary32 is, and 5e-6 beside (most 1e-6 to 1e-5; rank one alone
 *     some 2^-24 g, and so is that iteration).  Five quintic steps leave more
 *     where one singular value is about 20 times the others, 2e-5 to 4e-5, and
 *     as much for gradients there and up to 50 times; ones alone up to 6e-5.
 *
 * Conventions are those of muon.h (device memory of the current device,
 * strides in elements, validation before anything is enqueued, no
 * synchronisation, status codes), and:
 *   - Block b of a tensor starts stride_* * b elements after its pointer; its
 *     rows are ld_* apart and contiguous.  Written tensors' blocks must not
 *     share elements: stride >= (rows - 1) ld + cols, or side by side in the
 *     same rows: stride >= cols and (blocks - 1) stride + cols <= ld.
 *     Read-only tensors take any stride >= 0 (0: one block for all).
 *   - Blocks of one tensor may lie between those of another (query, key and
 *     value heads in turns in one weight).  Where one of the two is written,
 *     such tensors need equal strides, or equal row strides and columns apart;
 *     others whose address ranges meet are ALIAS.
 *   - Elements outside the blocks (row padding, other columns) are neither
 *     read nor written.
 *   - A block that holds a NaN or an infinity, or whose squared norm
 *     overflows binary32, gives NaN (its own block only).  A zero block gives
 *     zeros, and a zero gradient through the norm.
 *     With respect to a block of norm above 2^60 the gradient, 2^-60 of the
 *     cotangent and less, loses bits to the range of binary32.
 *   - Products over n run on the bfloat16 matrix cores on operands split into
 *     bfloat16 parts, with binary32 sums: bfloat16 inputs are one part
 *     (exact), binary32 values two parts (17 bits) where results are bfloat16
 *     and three parts (24 bits) where they are binary32.  The recursion runs
 *     on two binary16 parts (24 bits).  Results do not depend on the other
 *     stacks of a call or on their order, except that the Gram sums over n
 *     are split by the number of blocks in the call; the same call gives the
 *     same bits every time, captured or not.
 *   - Workspace: with workspace = NULL the library keeps one per device (grown
 *     on demand, freed by muon_release_workspace), and calls on a device that
 *     use it run one after another in the order they were made, whatever
 *     their streams.  With a workspace of the caller's (256-byte aligned
 *     device memory of muon_blocks_workspace_bytes bytes) the call only
 *     launches kernels, on `stream`: calls or graphs with different workspaces
 *     may overlap; those that share one must not.
 *   - Capture: a call on a capturing stream needs a workspace of the caller's
 *     (UNSUPPORTED without) and records kernels on `stream` only.  Pointers,
 *     sizes, coefficients, rates and decay are those of the capture.
 *   - Streams: a call with the library's workspace may run parts of a large
 *     group of blocks on further streams of the library's (up to two a device,
 *     at the default priority).  They start after what `stream` held before
 *     the call, and `stream` goes on after them.
 */
#ifndef MUON_MI355X_BLOCKS_H
#define MUON_MI355X_BLOCKS_H

#include "muon.h"

#ifdef __cplusplus
extern "C" {
#endif

/* One stack.  blocks in [0, 2^20] (0: skipped; at most 2^21 in a call), rows
 * and cols in [1, 65536] with min(rows, cols) <= 128, row strides up to 2^21.
 * Which tensors the three groups of fields describe is said at each call; a
 * group that a call does not name is ignored.  reserved: 0.                 */
typedef struct muon_block_desc {
  int64_t blocks, rows, cols;
  int64_t ld_param, ld_grad, ld_mom;             /* row strides, >= cols; any where rows = 1 */
  int64_t stride_param, stride_grad, stride_mom; /* from block to block      */
  int32_t param_dtype, grad_dtype, mom_dtype;
  int32_t reserved;
} muon_block_desc;

/* NS of every block.  x_in[i]: grad fields (F32 or BF16), read only.
 * x_out[i]: param fields (F32 or BF16), written.  ns_schedule: NULL, or a
 * host array of ns_steps triples used in place of ns_coeffs, read during the
 * call.  ns_steps = 0 gives the normalised blocks.
 * Errors: INVALID_ARGUMENT (null pointer, bad size or stride, non-finite
 * coefficient, ns_steps outside [0, 1000], workspace too small), UNSUPPORTED
 * (dtype, alignment, min(rows, cols) > 128, size cap, capture without a
 * workspace), ALIAS (a written buffer overlaps another, or itself),
 * OUT_OF_MEMORY, HIP.                                                       */
muon_status muon_ns_blocks(const void* const* x_in, void* const* x_out, const muon_block_desc* stacks,
                           int32_t count, muon_ns_coeffs ns_coeffs, int32_t ns_steps,
                           const muon_ns_coeffs* ns_schedule, void* workspace, uint64_t workspace_bytes,
                           void* stream);

/* The gradient of muon_ns_blocks: grad_in[i] = d<NS(x), y>/dx for x =
 * x_in[i] and y = grad_out[i], block by block, the normalisation included.
 *   dX_0 = P y + 2 L X_0 ;  dx = (dX_0 - X_0 <dX_0, X_0>/(||x|| inv)) inv
 * with inv = 1/(||x||_F + 1e-7) and L the derivative of the polynomial P(A)
 * at A_0 in direction sym(y X_0^T), carried along the recursion as its
 * tangent.  x_in[i]: grad fields, y: mom fields (F32 or BF16 each), both read
 * only; grad_in[i]: param fields (F32 or BF16), written, not accumulated
 * into.  Nothing is kept from the forward call: the recursion is run again.
 * Errors as muon_ns_blocks.                                                 */
muon_status muon_ns_blocks_vjp(const void* const* x_in, const void* const* grad_out, void* const* grad_in,
                               const muon_block_desc* stacks, int32_t count, muon_ns_coeffs ns_coeffs,
                               int32_t ns_steps, const muon_ns_coeffs* ns_schedule, void* workspace,
                               uint64_t workspace_bytes, void* stream);

/* One Muon step in which every block of every stack is a matrix of its own:
 * momentum, NS and the scaled write-back of muon_step_batched_v2, with s of
 * the scale rule from the block's rows and cols.  params[i]: param fields
 * (F32 or BF16), grads[i]: grad fields (F32 or BF16, read only), momenta[i]:
 * mom fields (F32).  The momentum and the write-back are bit-exact as in
 * muon_step_batched.  hparams->options may give ns_schedule, weight_decay,
 * momentum_kind, and lr_per_matrix and scale_per_matrix with one entry per
 * stack; launch_mode and tile_mode must be AUTO (0).  updates_out: NULL, or
 * per stack NULL or the binary32 update O that the write-back used, blocks x
 * rows x cols contiguous, as exact as results of the parameters' type are
 * before they are rounded.  Errors as muon_ns_blocks.                       */
muon_status muon_step_blocks(void* const* params, const void* const* grads, void* const* momenta,
                             const muon_block_desc* stacks, int32_t count, const muon_step_hparams* hparams,
                             float* const* updates_out, void* workspace, uint64_t workspace_bytes, void* stream);

/* The calls, for muon_blocks_workspace_bytes.                               */
typedef enum muon_blocks_op {
  MUON_BLOCKS_NS = 0,
  MUON_BLOCKS_VJP = 1,
  MUON_BLOCKS_STEP = 2
} muon_blocks_op;

/* Workspace bytes of a call of `op` (a muon_blocks_op) on these stacks with
 * these coefficients, on the current device; 0 on error (and for a call that
 * needs none).                                                              */
uint64_t muon_blocks_workspace_bytes(int32_t op, const muon_block_desc* stacks, int32_t count,
                                     muon_ns_coeffs ns_coeffs, int32_t ns_steps,
                                     const muon_ns_coeffs* ns_schedule);

#ifdef __cplusplus
}
#endif

#endif /* MUON_MI355X_BLOCKS_H */
