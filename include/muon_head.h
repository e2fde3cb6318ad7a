/*
 * muon_head.h -- C ABI of libmuon_mi355x.so, continued: the softmax cross
 * entropy of an output head over a large vocabulary, with its gradient.
 *
 * The head is the matrix W (vocab x dim) that muon_adamw_batched updates; its
 * gradient is made here.  With x the rows x dim input of the head and t_r the
 * target of row r,
 *
 *   l_rj  = <x_r, W_j>
 *   z_rj  = softcap tanh(l_rj / softcap), or l_rj where softcap = 0
 *   lse_r = log sum_j exp z_rj
 *   loss_r = lse_r - z_r,t_r
 *
 * and, for the cotangents g of loss and h of lse, with p_rj = exp(z_rj - lse_r),
 *
 *   dl_rj = ((g_r + h_r) p_rj - g_r [j = t_r]) (1 - (z_rj / softcap)^2)
 *   grad_x = dl W,  grad_W = dl^T x
 *
 * (the last factor only with a soft cap).  The soft cap is the logit soft-cap
 * 15 tanh(x / 15) that "开发者千美元训3.8B模型 击败GPT-2" (aiproducthub.cn),
 * paragraph 影响, lists.
 *
 * The loss keeps no logits: it reduces every tile of them to a maximum and a sum
 * a row, 8 bytes of workspace for 16 to 256 columns.  The gradient computes them again, a piece
 * of the vocabulary at a time, and holds one piece's dl: 512 MiB of workspace at
 * most, or 2048 columns where that is more.  Conventions are those of muon_experts.h (workspace,
 * capture and padding included; the two share the library's workspace), and:
 *   - targets is a device array of rows int64.  A row whose target is
 *     ignore_index has loss = lse = 0 and takes no part in the gradients, whatever x,
 *     grad_loss and grad_lse hold there (its grad_x is 0).  Any other target outside
 *     [0, vocab) gives loss = lse = NaN, and a row that takes no part in the
 *     gradients either (its grad_x is 0).
 *   - bfloat16: logits, their softmax and all sums are binary32; dl is rounded
 *     to bfloat16 for the two products (relative 2^-8 at most, independent from
 *     element to element), but for the target's element of every row, by far the
 *     largest, which is kept to 2^-16.  binary32: to
 *     binary32 accuracy throughout (products as in muon_experts.h).
 *   - A row with a NaN or an infinity among its logits has the values that the
 *     formulas give, NaN or infinite, and so have gradients that it takes part in.
 *     (Soft-capped) logits from 2^127 on in magnitude count as infinite.
 *   - The soft cap itself is off by 2^-21 cap at most, and by 18 2^-24 of the logit
 *     (bfloat16: with caps above 32), however large the cap.
 */
#ifndef MUON_MI355X_HEAD_H
#define MUON_MI355X_HEAD_H

#include "muon.h"

#ifdef __cplusplus
extern "C" {
#endif

/* rows in [0, 2^20], dim in [1, 65536], vocab in [1, 2^24].  Row strides >= dim
 * (any where there is one row), at most 2^21.  dtype: F32 or BF16, of x, w,
 * grad_x and grad_w.  softcap: 0 or a finite positive value of at least 1e-3.
 * ld_grad_* are used by the gradient only.  reserved: 0.                    */
typedef struct muon_head_desc {
  int64_t rows, dim, vocab;
  int64_t ld_x, ld_w, ld_grad_x, ld_grad_w;
  int64_t ignore_index;
  float softcap;
  int32_t dtype;
  int64_t reserved;
} muon_head_desc;

/* loss[r] and lse[r], binary32 arrays of `rows`.
 * Errors: INVALID_ARGUMENT (null pointer, bad size, stride or softcap, workspace
 * too small), UNSUPPORTED (dtype, alignment, size cap, capture without a
 * workspace), ALIAS (a written buffer overlaps another), OUT_OF_MEMORY, HIP. */
muon_status muon_head_loss(const void* x, const void* w, const int64_t* targets, float* loss, float* lse,
                           const muon_head_desc* desc, void* workspace, uint64_t workspace_bytes, void* stream);

/* The gradients of <loss, grad_loss> + <lse, grad_lse> from muon_head_loss's
 * lse.  grad_loss, grad_lse: binary32 arrays of `rows`; grad_lse may be NULL
 * (zeros).  grad_x or grad_w may be NULL and is then not computed.  Errors as
 * muon_head_loss.                                                           */
muon_status muon_head_loss_vjp(const void* x, const void* w, const int64_t* targets, const float* lse,
                               const float* grad_loss, const float* grad_lse, void* grad_x, void* grad_w,
                               const muon_head_desc* desc, void* workspace, uint64_t workspace_bytes, void* stream);

/* The calls, for muon_head_workspace_bytes.                                 */
typedef enum muon_head_op {
  MUON_HEAD_LOSS = 0,
  MUON_HEAD_GRAD_X = 1,
  MUON_HEAD_GRAD_W = 2,
  MUON_HEAD_GRAD_X_W = 3
} muon_head_op;

/* Workspace bytes of a call of `op` (a muon_head_op) on the current device; 0
 * for a call that needs none, and on error.                                 */
uint64_t muon_head_workspace_bytes(int32_t op, const muon_head_desc* desc);

#ifdef __cplusplus
}
#endif

#endif /* MUON_MI355X_HEAD_H */
