// Host side of the products grouped by expert (muon_experts.h).
#include "muon_experts.h"

#include <hip/hip_runtime.h>

#include <algorithm>

#include "op_workspace.h"
#include "products_internal.h"

namespace muon {
namespace {

constexpr int64_t MAX_EXPERTS = 2048, MAX_ROWS = 1 << 24, MAX_DIM = 65536, MAX_LD = 1 << 21;
constexpr int64_t MAX_STRIDE = int64_t(1) << 40;

struct Call {
  int op = MUON_EXPERTS_PRODUCT;
  const void* x = nullptr;
  const void* w = nullptr;
  const int32_t* offsets = nullptr;
  const void* gy = nullptr;      // vjp
  void* out = nullptr;           // y, or grad_x
  void* gw = nullptr;
  const muon_experts_desc* desc = nullptr;
  void* ws = nullptr;
  uint64_t ws_bytes = 0;
  hipStream_t stream = nullptr;
  bool need_x() const { return op == MUON_EXPERTS_PRODUCT || (op & MUON_EXPERTS_GRAD_W); }
  bool need_w() const { return op == MUON_EXPERTS_PRODUCT || (op & MUON_EXPERTS_GRAD_X); }
};

int esize(int32_t dt) { return dt == MUON_DTYPE_BF16 ? 2 : 4; }

// A matrix of the call: `rows` rows of `cols` elements, ld apart.
int64_t row_stride(int64_t rows, int64_t cols, int64_t ld) { return rows <= 1 ? cols : ld; }
int64_t span(int64_t rows, int64_t cols, int64_t ld) { return rows < 1 ? 0 : (rows - 1) * row_stride(rows, cols, ld) + cols; }

struct Weight {
  int64_t rows, cols;
};
Weight weight_of(const muon_experts_desc& d) {
  return d.w_order == MUON_WEIGHT_OUT_IN ? Weight{d.out_dim, d.in_dim} : Weight{d.in_dim, d.out_dim};
}

muon_status check_ld(const char* what, int64_t rows, int64_t cols, int64_t ld) {
  if (rows <= 1) return MUON_OK;
  if (ld < cols) return op_fail(MUON_ERR_INVALID_ARGUMENT, "%s: row stride %lld below %lld", what, (long long)ld, (long long)cols);
  if (ld > MAX_LD) return op_fail(MUON_ERR_UNSUPPORTED, "%s: row stride %lld above 2^21", what, (long long)ld);
  return MUON_OK;
}

muon_status check_stride(const char* what, int64_t stride) {
  if (stride < 0 || stride > MAX_STRIDE)
    return op_fail(MUON_ERR_INVALID_ARGUMENT, "%s: expert stride %lld out of [0, 2^40]", what, (long long)stride);
  return MUON_OK;
}

muon_status check_desc(const Call& c) {
  if (!c.desc) return op_fail(MUON_ERR_INVALID_ARGUMENT, "desc is NULL");
  const muon_experts_desc& d = *c.desc;
  if (d.reserved != 0) return op_fail(MUON_ERR_INVALID_ARGUMENT, "reserved must be 0");
  if (d.experts < 0 || d.rows < 0 || d.in_dim < 1 || d.out_dim < 1)
    return op_fail(MUON_ERR_INVALID_ARGUMENT, "bad size: %lld experts, %lld rows, %lld x %lld weights",
                   (long long)d.experts, (long long)d.rows, (long long)d.out_dim, (long long)d.in_dim);
  if (d.experts > MAX_EXPERTS || d.rows > MAX_ROWS || d.in_dim > MAX_DIM || d.out_dim > MAX_DIM)
    return op_fail(MUON_ERR_UNSUPPORTED, "at most 2048 experts, 2^24 rows and 65536 x 65536 weights (got %lld, %lld, "
                   "%lld x %lld)", (long long)d.experts, (long long)d.rows, (long long)d.out_dim, (long long)d.in_dim);
  if (d.dtype != MUON_DTYPE_F32 && d.dtype != MUON_DTYPE_BF16)
    return op_fail(MUON_ERR_UNSUPPORTED, "dtype %d is not F32 or BF16", d.dtype);
  if (d.w_order != MUON_WEIGHT_OUT_IN && d.w_order != MUON_WEIGHT_IN_OUT)
    return op_fail(MUON_ERR_INVALID_ARGUMENT, "unknown w_order %d", d.w_order);
  const Weight w = weight_of(d);
  muon_status st = MUON_OK;
  if (c.need_x()) st = check_ld("x", d.rows, d.in_dim, d.ld_x);
  if (st == MUON_OK) st = check_ld(c.op == MUON_EXPERTS_PRODUCT ? "y" : "grad_y", d.rows, d.out_dim, d.ld_y);
  if (st == MUON_OK && c.need_w()) st = check_ld("w", w.rows, w.cols, d.ld_w);
  if (st == MUON_OK && c.need_w()) st = check_stride("w", d.stride_w);
  if (st == MUON_OK && (c.op & MUON_EXPERTS_GRAD_X)) st = check_ld("grad_x", d.rows, d.in_dim, d.ld_grad_x);
  if (st == MUON_OK && (c.op & MUON_EXPERTS_GRAD_W)) {
    st = check_ld("grad_w", w.rows, w.cols, d.ld_grad_w);
    if (st == MUON_OK) st = check_stride("grad_w", d.stride_grad_w);
    if (st != MUON_OK) return st;
    if (d.grad_w_dtype != MUON_DTYPE_F32 && !(d.grad_w_dtype == MUON_DTYPE_BF16 && d.dtype == MUON_DTYPE_BF16))
      return op_fail(MUON_ERR_UNSUPPORTED, "grad_w_dtype %d with dtype %d", d.grad_w_dtype, d.dtype);
    if (d.accumulate != 0 && d.accumulate != 1)
      return op_fail(MUON_ERR_INVALID_ARGUMENT, "accumulate must be 0 or 1");
    const int64_t ld = row_stride(w.rows, w.cols, d.ld_grad_w);
    const bool apart = d.stride_grad_w >= span(w.rows, w.cols, ld);
    const bool beside = d.stride_grad_w >= w.cols && (d.experts - 1) * d.stride_grad_w + w.cols <= ld;
    if (d.experts > 1 && !apart && !beside)
      return op_fail(MUON_ERR_ALIAS, "experts of grad_w share elements (row stride %lld, expert stride %lld)",
                     (long long)ld, (long long)d.stride_grad_w);
  }
  return st;
}

muon_status check_ptr(const char* what, const void* p, int esz, bool needed) {
  if (!p && needed) return op_fail(MUON_ERR_INVALID_ARGUMENT, "%s is NULL", what);
  if (reinterpret_cast<uintptr_t>(p) % uintptr_t(esz) != 0)
    return op_fail(MUON_ERR_UNSUPPORTED, "%s is not aligned to %d bytes", what, esz);
  return MUON_OK;
}

muon_status check_buffers(const Call& c) {
  const muon_experts_desc& d = *c.desc;
  const Weight w = weight_of(d);
  OpRange r[7];
  int n = 0;
  muon_status st = MUON_OK;
  auto add = [&](const char* what, const void* p, int64_t elems, int esz, bool written) {
    if (st != MUON_OK) return;
    st = check_ptr(what, p, esz, elems > 0);
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    if (elems > 0) r[n++] = {lo, lo + uintptr_t(elems) * uintptr_t(esz), written, what};
  };
  const int esz = esize(d.dtype);
  const bool product = c.op == MUON_EXPERTS_PRODUCT;
  if (c.need_x()) add("x", c.x, span(d.rows, d.in_dim, d.ld_x), esz, false);
  if (c.need_w())
    add("w", c.w, d.rows == 0 ? 0 : (d.experts - 1) * d.stride_w + span(w.rows, w.cols, d.ld_w), esz, false);
  add("offsets", c.offsets, d.experts + 1, 4, false);
  if (product) {
    add("y", c.out, span(d.rows, d.out_dim, d.ld_y), esz, true);
  } else {
    add("grad_y", c.gy, span(d.rows, d.out_dim, d.ld_y), esz, false);
    if (c.op & MUON_EXPERTS_GRAD_X) add("grad_x", c.out, span(d.rows, d.in_dim, d.ld_grad_x), esz, true);
    if (c.op & MUON_EXPERTS_GRAD_W)
      add("grad_w", c.gw, (d.experts - 1) * d.stride_grad_w + span(w.rows, w.cols, d.ld_grad_w), esize(d.grad_w_dtype), true);
  }
  if (c.ws) {
    if (reinterpret_cast<uintptr_t>(c.ws) % 256 != 0) return op_fail(MUON_ERR_UNSUPPORTED, "workspace is not aligned to 256 bytes");
    add("workspace", c.ws, int64_t(c.ws_bytes), 1, true);
  }
  return st != MUON_OK ? st : op_check_alias(r, n);
}

// The product of `op` (one of PRODUCT, GRAD_X, GRAD_W).
int product_args(const Call& c, int op, ProductArgs& a) {
  const muon_experts_desc& d = *c.desc;
  const Weight w = weight_of(d);
  const bool oi = d.w_order == MUON_WEIGHT_OUT_IN;
  const int64_t ldx = row_stride(d.rows, d.in_dim, d.ld_x), ldy = row_stride(d.rows, d.out_dim, d.ld_y);
  const int64_t ldw = row_stride(w.rows, w.cols, d.ld_w);
  a = ProductArgs{};
  a.offsets = c.offsets;
  a.groups = int32_t(d.experts);
  a.rows = int32_t(d.rows);
  a.f32 = d.dtype == MUON_DTYPE_F32;
  a.out_f32 = a.f32;
  if (op == MUON_EXPERTS_GRAD_W) {
    // grad_W = grad_y^T x, or its transpose x^T grad_y
    a.p = oi ? c.gy : c.x;
    a.q = oi ? c.x : c.gy;
    a.ld_p = oi ? ldy : ldx;
    a.ld_q = oi ? ldx : ldy;
    a.m = int32_t(w.rows);
    a.n = int32_t(w.cols);
    a.p_elems = span(d.rows, w.rows, a.ld_p);
    a.q_elems = span(d.rows, w.cols, a.ld_q);
    a.out = c.gw;
    a.ld_out = a.ld_add = row_stride(w.rows, w.cols, d.ld_grad_w);
    a.es_out = d.stride_grad_w;
    a.out_f32 = a.add_f32 = d.grad_w_dtype == MUON_DTYPE_F32;
    a.add = d.accumulate ? c.gw : nullptr;
    return FORM_TN;
  }
  const bool product = op == MUON_EXPERTS_PRODUCT;
  a.p = product ? c.x : c.gy;
  a.ld_p = product ? ldx : ldy;
  a.k = int32_t(product ? d.in_dim : d.out_dim);
  a.n = int32_t(product ? d.out_dim : d.in_dim);
  a.p_elems = span(d.rows, a.k, a.ld_p);
  a.q = c.w;
  a.ld_q = ldw;
  a.es_q = d.stride_w;
  a.q_elems = span(w.rows, w.cols, ldw);
  a.out = c.out;
  a.ld_out = product ? ldy : row_stride(d.rows, d.in_dim, d.ld_grad_x);
  return product == oi ? FORM_NT : FORM_NN;
}

// The calls of one op run in turn and share it.
size_t workspace_need(const Call& c, int cus) {
  size_t need = 0;
  for (int op : {MUON_EXPERTS_GRAD_X, MUON_EXPERTS_GRAD_W, MUON_EXPERTS_PRODUCT}) {
    if (op == MUON_EXPERTS_PRODUCT ? c.op != op : !(c.op & op)) continue;
    ProductArgs a;
    const int form = product_args(c, op, a);
    need = std::max(need, op_align256(product_plan(form, EPI_STORE, a, cus).bytes));
  }
  return need;
}

muon_status run(const Call& c) {
  muon_status st = check_desc(c);
  if (st != MUON_OK) return st;
  if (c.desc->experts == 0) return MUON_OK;
  if ((st = check_buffers(c)) != MUON_OK) return st;
  if (c.desc->rows == 0 && !(c.op & MUON_EXPERTS_GRAD_W)) return MUON_OK;
  int cus = 0;
  if ((st = op_device(&cus)) != MUON_OK) return st;
  return op_run(workspace_need(c, cus), c.ws, c.ws_bytes, c.stream, [&](char* ws, bool capturing) {
    auto one = [&](int op) -> hipError_t {
      ProductArgs a;
      const int form = product_args(c, op, a);
      auto launch = [&] { return launch_product(form, EPI_STORE, a, cus, ws, c.stream); };
      return capturing ? launch() : api_timed(MUON_KC_COMBINE, c.stream, launch);
    };
    hipError_t e = hipSuccess;
    if (c.op == MUON_EXPERTS_PRODUCT) return one(c.op);
    if ((c.op & MUON_EXPERTS_GRAD_X) && c.desc->rows > 0) e = one(MUON_EXPERTS_GRAD_X);
    if (e == hipSuccess && (c.op & MUON_EXPERTS_GRAD_W)) e = one(MUON_EXPERTS_GRAD_W);
    return e;
  });
}

}  // namespace
}  // namespace muon

using namespace muon;

extern "C" {

muon_status muon_experts_product(const void* x, const void* w, const int32_t* offsets, void* y,
                                 const muon_experts_desc* desc, void* workspace, uint64_t workspace_bytes,
                                 void* stream) {
  return op_guarded([&] {
    Call c;
    c.x = x;
    c.w = w;
    c.offsets = offsets;
    c.out = y;
    c.desc = desc;
    c.ws = workspace;
    c.ws_bytes = workspace_bytes;
    c.stream = reinterpret_cast<hipStream_t>(stream);
    return run(c);
  });
}

muon_status muon_experts_product_vjp(const void* x, const void* w, const int32_t* offsets, const void* grad_y,
                                     void* grad_x, void* grad_w, const muon_experts_desc* desc, void* workspace,
                                     uint64_t workspace_bytes, void* stream) {
  return op_guarded([&]() -> muon_status {
    if (!grad_x && !grad_w && !(desc && desc->rows == 0))
      return api_fail(MUON_ERR_INVALID_ARGUMENT, "grad_x and grad_w are both NULL");
    Call c;
    c.op = (grad_x ? MUON_EXPERTS_GRAD_X : 0) | (grad_w ? MUON_EXPERTS_GRAD_W : 0);
    if (c.op == 0) c.op = MUON_EXPERTS_GRAD_X;
    c.x = x;
    c.w = w;
    c.offsets = offsets;
    c.gy = grad_y;
    c.out = grad_x;
    c.gw = grad_w;
    c.desc = desc;
    c.ws = workspace;
    c.ws_bytes = workspace_bytes;
    c.stream = reinterpret_cast<hipStream_t>(stream);
    return run(c);
  });
}

uint64_t muon_experts_workspace_bytes(int32_t op, const muon_experts_desc* desc) {
  uint64_t need = 0;
  (void)op_guarded([&]() -> muon_status {
    if (op < MUON_EXPERTS_PRODUCT || op > MUON_EXPERTS_GRAD_X_W)
      return op_fail(MUON_ERR_INVALID_ARGUMENT, "unknown op %d", op);
    Call c;
    c.op = op;
    c.desc = desc;
    muon_status st = check_desc(c);
    int cus = 0;
    if (st == MUON_OK) st = op_device(&cus);
    if (st == MUON_OK) need = workspace_need(c, cus);
    return st;
  });
  return need;
}

}  // extern "C"
