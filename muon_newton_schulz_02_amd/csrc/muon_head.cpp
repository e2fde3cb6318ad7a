// Host side of the head's loss (muon_head.h).
#include "muon_head.h"

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "op_workspace.h"
#include "products_internal.h"

namespace muon {
namespace {

constexpr int64_t MAX_ROWS = 1 << 20, MAX_DIM = 65536, MAX_VOCAB = 1 << 24, MAX_LD = 1 << 21;
// Bytes of a piece's gradients with respect to the logits, or PIECE_LEAST columns of them
// where that is more: with the most rows 4 GiB of bfloat16, 8 of binary32.
constexpr int64_t PIECE_BYTES = int64_t(512) << 20, PIECE_LEAST = 2048;
// The products reach the rows of a tile (256 at most, of those that there are) by 32-bit
// offsets: those of the caller's tensors, and of a piece, which is wide where rows are few
// (up to MAX_VOCAB columns, rounded up to whole tiles).
static_assert(256 * MAX_LD * 4 < int64_t(1) << 32 && 256 * (PIECE_LEAST + 255) * 4 < int64_t(1) << 32 &&
              PIECE_BYTES + 256 * 255 * 4 < int64_t(1) << 32, "offsets in a tile");

// Up to so many rows the forward pass takes x as it lies, the rows without a target
// among them: packing would be a launch of its own (8 us of 42 for one row over 32768 x
// 1536), for less work in products that read W at the rate of memory anyway.
constexpr int64_t DIRECT_ROWS = 256;

struct Call {
  int op = MUON_HEAD_LOSS;
  const void* x = nullptr;
  const void* w = nullptr;
  const int64_t* targets = nullptr;
  const float* grad_loss = nullptr;
  const float* grad_lse = nullptr;
  float* loss = nullptr;
  float* lse = nullptr;          // written, or (gradient) read
  void* gx = nullptr;
  void* gw = nullptr;
  const muon_head_desc* desc = nullptr;
  void* ws = nullptr;
  uint64_t ws_bytes = 0;
  hipStream_t stream = nullptr;
};

int esize(int32_t dt) { return dt == MUON_DTYPE_BF16 ? 2 : 4; }
int64_t row_stride(int64_t rows, int64_t cols, int64_t ld) { return rows <= 1 ? cols : ld; }
int64_t span(int64_t rows, int64_t cols, int64_t ld) { return rows < 1 ? 0 : (rows - 1) * row_stride(rows, cols, ld) + cols; }
int64_t round_up(int64_t v, int64_t m) { return (v + m - 1) / m * m; }

muon_status check_ld(const char* what, int64_t rows, int64_t cols, int64_t ld) {
  if (rows <= 1) return MUON_OK;
  if (ld < cols) return op_fail(MUON_ERR_INVALID_ARGUMENT, "%s: row stride %lld below %lld", what, (long long)ld, (long long)cols);
  if (ld > MAX_LD) return op_fail(MUON_ERR_UNSUPPORTED, "%s: row stride %lld above 2^21", what, (long long)ld);
  return MUON_OK;
}

muon_status check_desc(const Call& c) {
  if (!c.desc) return op_fail(MUON_ERR_INVALID_ARGUMENT, "desc is NULL");
  const muon_head_desc& d = *c.desc;
  if (d.reserved != 0) return op_fail(MUON_ERR_INVALID_ARGUMENT, "reserved must be 0");
  if (d.rows < 0 || d.dim < 1 || d.vocab < 1)
    return op_fail(MUON_ERR_INVALID_ARGUMENT, "bad size: %lld rows of %lld, vocabulary of %lld", (long long)d.rows,
                   (long long)d.dim, (long long)d.vocab);
  if (d.rows > MAX_ROWS || d.dim > MAX_DIM || d.vocab > MAX_VOCAB)
    return op_fail(MUON_ERR_UNSUPPORTED, "at most 2^20 rows of 65536 and a vocabulary of 2^24 (got %lld, %lld, %lld)",
                   (long long)d.rows, (long long)d.dim, (long long)d.vocab);
  if (d.dtype != MUON_DTYPE_F32 && d.dtype != MUON_DTYPE_BF16)
    return op_fail(MUON_ERR_UNSUPPORTED, "dtype %d is not F32 or BF16", d.dtype);
  if (!(d.softcap == 0.f || (std::isfinite(d.softcap) && d.softcap >= 1e-3f)))
    return op_fail(MUON_ERR_INVALID_ARGUMENT, "softcap must be 0 or finite and at least 1e-3 (got %g)", double(d.softcap));
  muon_status st = check_ld("x", d.rows, d.dim, d.ld_x);
  if (st == MUON_OK) st = check_ld("w", d.vocab, d.dim, d.ld_w);
  if (st == MUON_OK && (c.op & MUON_HEAD_GRAD_X)) st = check_ld("grad_x", d.rows, d.dim, d.ld_grad_x);
  if (st == MUON_OK && (c.op & MUON_HEAD_GRAD_W)) st = check_ld("grad_w", d.vocab, d.dim, d.ld_grad_w);
  return st;
}

muon_status check_buffers(const Call& c) {
  const muon_head_desc& d = *c.desc;
  OpRange r[9];
  int n = 0;
  muon_status st = MUON_OK;
  auto add = [&](const char* what, const void* p, int64_t elems, int esz, bool written) {
    if (st != MUON_OK) return;
    if (!p && elems > 0) {
      st = op_fail(MUON_ERR_INVALID_ARGUMENT, "%s is NULL", what);
    } else if (reinterpret_cast<uintptr_t>(p) % uintptr_t(esz) != 0) {
      st = op_fail(MUON_ERR_UNSUPPORTED, "%s is not aligned to %d bytes", what, esz);
    } else if (elems > 0) {
      const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
      r[n++] = {lo, lo + uintptr_t(elems) * uintptr_t(esz), written, what};
    }
  };
  const int esz = esize(d.dtype);
  const bool fwd = c.op == MUON_HEAD_LOSS;
  add("x", c.x, span(d.rows, d.dim, d.ld_x), esz, false);
  add("w", c.w, d.rows == 0 ? 0 : span(d.vocab, d.dim, d.ld_w), esz, false);
  add("targets", c.targets, d.rows, 8, false);
  add("lse", c.lse, d.rows, 4, fwd);
  if (fwd) {
    add("loss", c.loss, d.rows, 4, true);
  } else {
    add("grad_loss", c.grad_loss, d.rows, 4, false);
    if (c.grad_lse) add("grad_lse", c.grad_lse, d.rows, 4, false);
    if (c.op & MUON_HEAD_GRAD_X) add("grad_x", c.gx, span(d.rows, d.dim, d.ld_grad_x), esz, true);
    if (c.op & MUON_HEAD_GRAD_W) add("grad_w", c.gw, span(d.vocab, d.dim, d.ld_grad_w), esz, true);
  }
  if (c.ws) {
    if (st == MUON_OK && reinterpret_cast<uintptr_t>(c.ws) % 256 != 0)
      return op_fail(MUON_ERR_UNSUPPORTED, "workspace is not aligned to 256 bytes");
    add("workspace", c.ws, int64_t(c.ws_bytes), 1, true);
  }
  return st != MUON_OK ? st : op_check_alias(r, n);
}

// Where everything lies in the workspace.
struct Plan {
  size_t offsets, row, target, xc, lse, ga, gb, rest, logit, stats, dz, acc, part, bytes;
  int64_t ld_xc;       // elements of a packed row of x (and of acc)
  int64_t piece;       // columns of a piece of the vocabulary
  int64_t ld_dz;
  int32_t tiles;       // tiles of columns of the whole vocabulary (forward)
  bool direct;         // the rows are not packed
};

// What the product of the logits of columns [c0, c0 + n) takes.
ProductArgs logits_args(const Call& c, const Plan& p, char* ws, int64_t c0, int64_t n) {
  const muon_head_desc& d = *c.desc;
  ProductArgs a = {};
  const int64_t ldw = row_stride(d.vocab, d.dim, d.ld_w);
  a.p = ws + p.xc;
  a.ld_p = p.ld_xc;
  a.p_elems = span(d.rows, d.dim, p.ld_xc);
  a.q = reinterpret_cast<const char*>(c.w) + size_t(c0) * size_t(ldw) * size_t(esize(d.dtype));
  a.ld_q = ldw;
  a.q_elems = span(n, d.dim, ldw);
  a.offsets = reinterpret_cast<const int32_t*>(ws + p.offsets);
  a.target = reinterpret_cast<const int32_t*>(ws + p.target);
  if (p.direct) {
    a.p = c.x;
    a.ld_p = row_stride(d.rows, d.dim, d.ld_x);
    a.p_elems = span(d.rows, d.dim, d.ld_x);
    a.offsets = nullptr;
    a.target = nullptr;
    a.targets = c.targets;
  }
  a.groups = 1;
  a.rows = int32_t(d.rows);
  a.n = int32_t(n);
  a.k = int32_t(d.dim);
  a.f32 = a.out_f32 = a.add_f32 = d.dtype == MUON_DTYPE_F32;
  a.cap = d.softcap;
  a.inv_cap = d.softcap != 0.f ? 1.f / d.softcap : 0.f;
  a.col0 = int32_t(c0);
  a.logit = reinterpret_cast<float*>(ws + p.logit);
  a.stats = reinterpret_cast<float2*>(ws + p.stats);
  a.stat_tiles = p.tiles;
  a.lse = reinterpret_cast<const float*>(ws + p.lse);
  a.ga = reinterpret_cast<const float*>(ws + p.ga);
  a.gb = reinterpret_cast<const float*>(ws + p.gb);
  return a;
}

// The logits' gradients of a piece.
ProductArgs dz_args(const Call& c, const Plan& p, char* ws, int64_t c0, int64_t n) {
  ProductArgs a = logits_args(c, p, ws, c0, n);
  a.out = ws + p.dz;
  if (!a.f32) a.rest = reinterpret_cast<float*>(ws + p.rest);
  a.ld_out = p.ld_dz;
  return a;
}

// grad_x from the piece that `a` makes: binary32 sums over the pieces, the last one's
// rounded into grad_x.
ProductArgs grad_x_args(const Call& c, const Plan& p, char* ws, const ProductArgs& a) {
  const muon_head_desc& d = *c.desc;
  const bool first = a.col0 == 0, last = a.col0 + int64_t(a.n) == d.vocab;
  ProductArgs b = {};
  b.p = a.out;
  b.ld_p = p.ld_dz;
  b.p_elems = span(d.rows, a.n, p.ld_dz);
  b.q = a.q;
  b.ld_q = a.ld_q;
  b.q_elems = a.q_elems;
  b.offsets = a.offsets;
  b.groups = 1;
  b.rows = a.rows;
  b.n = int32_t(d.dim);
  b.k = a.n;
  b.f32 = a.f32;
  b.target = a.target;
  b.col0 = a.col0;
  b.rest = a.rest;
  b.out = last ? c.gx : ws + p.acc;
  b.map = last ? reinterpret_cast<const int32_t*>(ws + p.row) : nullptr;
  b.out_f32 = last ? a.f32 : 1;
  b.ld_out = last ? row_stride(d.rows, d.dim, d.ld_grad_x) : p.ld_xc;
  b.add = first ? nullptr : ws + p.acc;
  b.add_f32 = 1;
  b.ld_add = p.ld_xc;
  return b;
}

// The rows of grad_w that the piece makes.
ProductArgs grad_w_args(const Call& c, const Plan& p, const ProductArgs& a) {
  const muon_head_desc& d = *c.desc;
  ProductArgs b = {};
  b.p = a.out;
  b.ld_p = p.ld_dz;
  b.p_elems = span(d.rows, a.n, p.ld_dz);
  b.q = a.p;
  b.ld_q = p.ld_xc;
  b.q_elems = a.p_elems;
  b.offsets = a.offsets;
  b.groups = 1;
  b.rows = a.rows;
  b.m = a.n;
  b.n = int32_t(d.dim);
  b.f32 = b.out_f32 = a.f32;
  b.target = a.target;
  b.col0 = a.col0;
  b.rest = a.rest;
  b.ld_out = row_stride(d.vocab, d.dim, d.ld_grad_w);
  b.out = reinterpret_cast<char*>(c.gw) + size_t(a.col0) * size_t(b.ld_out) * size_t(esize(d.dtype));
  return b;
}

Plan plan_of(const Call& c, int cus) {
  const muon_head_desc& d = *c.desc;
  Plan p = {};
  size_t at = 0;
  auto take = [&](int64_t bytes) {
    const size_t r = at;
    at += op_align256(size_t(bytes));
    return r;
  };
  const int64_t t = d.rows, esz = esize(d.dtype);
  p.direct = c.op == MUON_HEAD_LOSS && t <= DIRECT_ROWS;
  p.ld_xc = round_up(d.dim, 64);
  if (!p.direct) {
    p.offsets = take(8);
    p.row = take(4 * t);
    p.target = take(4 * t);
    p.xc = take(t * p.ld_xc * esz);
  }
  if (c.op == MUON_HEAD_LOSS) {
    const ProductArgs a = logits_args(c, p, nullptr, 0, d.vocab);
    const int tn = product_tile_n(FORM_NT, EPI_LSE, a, cus);
    p.tiles = int32_t((d.vocab + tn - 1) / tn);
    p.logit = take(4 * t);
    p.stats = take(8 * t * p.tiles);
  } else {
    p.lse = take(4 * t);
    p.ga = take(4 * t);
    p.gb = take(4 * t);
    if (d.dtype != MUON_DTYPE_F32) p.rest = take(4 * t);
    const int64_t most = std::max(PIECE_LEAST, PIECE_BYTES / (std::max<int64_t>(t, 1) * esz));
    // pieces of one size, whole tiles of 256 columns
    const int64_t pieces = (d.vocab + most - 1) / most;
    p.piece = round_up((d.vocab + pieces - 1) / pieces, 256);
    p.ld_dz = p.piece;
    p.dz = take(t * p.ld_dz * esz);
    if ((c.op & MUON_HEAD_GRAD_X) && p.piece < d.vocab) p.acc = take(t * p.ld_xc * 4);
    size_t part = 0;
    for (int64_t c0 : {int64_t(0), (d.vocab - 1) / p.piece * p.piece}) {      // a whole piece, and the last one
      const ProductArgs a = dz_args(c, p, nullptr, c0, std::min(p.piece, d.vocab - c0));
      if (c.op & MUON_HEAD_GRAD_X) part = std::max(part, product_plan(FORM_NN, EPI_STORE, grad_x_args(c, p, nullptr, a), cus).bytes);
      if (c.op & MUON_HEAD_GRAD_W) part = std::max(part, product_plan(FORM_TN, EPI_STORE, grad_w_args(c, p, a), cus).bytes);
    }
    p.part = take(int64_t(part));
  }
  p.bytes = at;
  return p;
}

hipError_t enqueue(const Call& c, const Plan& p, char* ws, int cus, bool capturing) {
  const muon_head_desc& d = *c.desc;
  const bool fwd = c.op == MUON_HEAD_LOSS;
  auto timed = [&](int kc, const std::function<hipError_t()>& launch) -> hipError_t {
    return capturing ? launch() : api_timed(kc, c.stream, launch);
  };
  HeadRows h = {};
  h.f32 = d.dtype == MUON_DTYPE_F32;
  h.x = c.x;
  h.targets = c.targets;
  h.lse_in = fwd ? nullptr : c.lse;
  h.grad_loss = c.grad_loss;
  h.grad_lse = c.grad_lse;
  h.xc = ws + p.xc;
  h.offsets = reinterpret_cast<int32_t*>(ws + p.offsets);
  h.row = reinterpret_cast<int32_t*>(ws + p.row);
  h.target = reinterpret_cast<int32_t*>(ws + p.target);
  h.lse_c = reinterpret_cast<float*>(ws + p.lse);
  h.ga = reinterpret_cast<float*>(ws + p.ga);
  h.gb = reinterpret_cast<float*>(ws + p.gb);
  h.loss = fwd ? c.loss : nullptr;
  h.lse_out = fwd ? c.lse : nullptr;
  h.grad_x = c.gx;
  h.ld_x = row_stride(d.rows, d.dim, d.ld_x);
  h.ld_xc = p.ld_xc;
  h.ld_grad_x = row_stride(d.rows, d.dim, d.ld_grad_x);
  h.ignore_index = d.ignore_index;
  h.vocab = d.vocab;
  h.rows = int32_t(d.rows);
  h.dim = int32_t(d.dim);
  h.chunk = int32_t(std::max<int64_t>(4, (d.rows + 1023) / 1024));
  hipError_t e = p.direct ? hipSuccess : timed(MUON_KC_MOMENTUM, [&] { return launch_head_rows(h, c.stream); });
  if (e != hipSuccess) return e;
  if (fwd) {
    const ProductArgs a = logits_args(c, p, ws, 0, d.vocab);
    e = timed(MUON_KC_GRAM, [&] { return launch_product(FORM_NT, EPI_LSE, a, cus, ws + p.part, c.stream); });
    if (e != hipSuccess) return e;
    HeadFinish f = {};
    f.stats = a.stats;
    f.logit = a.logit;
    f.offsets = a.offsets;
    f.row = h.row;
    f.targets = p.direct ? c.targets : nullptr;
    f.ignore_index = d.ignore_index;
    f.vocab = d.vocab;
    f.loss = c.loss;
    f.lse = c.lse;
    f.tiles = p.tiles;
    f.rows = h.rows;
    return timed(MUON_KC_NORM, [&] { return launch_head_finish(f, c.stream); });
  }
  for (int64_t c0 = 0; c0 < d.vocab && e == hipSuccess; c0 += p.piece) {
    const int64_t n = std::min(p.piece, d.vocab - c0);
    const ProductArgs a = dz_args(c, p, ws, c0, n);
    e = timed(MUON_KC_GRAM, [&] { return launch_product(FORM_NT, EPI_DZ, a, cus, ws + p.part, c.stream); });
    if (e == hipSuccess && c.gx) {
      const ProductArgs b = grad_x_args(c, p, ws, a);
      e = timed(MUON_KC_COMBINE, [&] { return launch_product(FORM_NN, EPI_STORE, b, cus, ws + p.part, c.stream); });
    }
    if (e == hipSuccess && c.gw) {
      const ProductArgs b = grad_w_args(c, p, a);
      e = timed(MUON_KC_COMBINE, [&] { return launch_product(FORM_TN, EPI_STORE, b, cus, ws + p.part, c.stream); });
    }
  }
  return e;
}

// Without rows: the weight's gradient is zero.
hipError_t enqueue_empty(const Call& c, int cus) {
  const muon_head_desc& d = *c.desc;
  ProductArgs b = {};
  b.groups = 1;
  b.m = int32_t(d.vocab);
  b.n = int32_t(d.dim);
  b.f32 = b.out_f32 = d.dtype == MUON_DTYPE_F32;
  b.ld_out = row_stride(d.vocab, d.dim, d.ld_grad_w);
  b.out = c.gw;
  return launch_product(FORM_TN, EPI_STORE, b, cus, nullptr, c.stream);
}

muon_status run(const Call& c) {
  muon_status st = check_desc(c);
  if (st != MUON_OK) return st;
  if ((st = check_buffers(c)) != MUON_OK) return st;
  const bool empty = c.desc->rows == 0;
  if (empty && !(c.op & MUON_HEAD_GRAD_W)) return MUON_OK;
  int cus = 0;
  if ((st = op_device(&cus)) != MUON_OK) return st;
  if (empty)
    return op_run(0, c.ws, c.ws_bytes, c.stream, [&](char*, bool) { return enqueue_empty(c, cus); });
  const Plan p = plan_of(c, cus);
  return op_run(p.bytes, c.ws, c.ws_bytes, c.stream,
                [&](char* ws, bool capturing) { return enqueue(c, p, ws, cus, capturing); });
}

}  // namespace
}  // namespace muon

using namespace muon;

extern "C" {

muon_status muon_head_loss(const void* x, const void* w, const int64_t* targets, float* loss, float* lse,
                           const muon_head_desc* desc, void* workspace, uint64_t workspace_bytes, void* stream) {
  return op_guarded([&] {
    Call c;
    c.x = x;
    c.w = w;
    c.targets = targets;
    c.loss = loss;
    c.lse = lse;
    c.desc = desc;
    c.ws = workspace;
    c.ws_bytes = workspace_bytes;
    c.stream = reinterpret_cast<hipStream_t>(stream);
    return run(c);
  });
}

muon_status muon_head_loss_vjp(const void* x, const void* w, const int64_t* targets, const float* lse,
                               const float* grad_loss, const float* grad_lse, void* grad_x, void* grad_w,
                               const muon_head_desc* desc, void* workspace, uint64_t workspace_bytes, void* stream) {
  return op_guarded([&]() -> muon_status {
    if (!grad_x && !grad_w && !(desc && desc->rows == 0))
      return api_fail(MUON_ERR_INVALID_ARGUMENT, "grad_x and grad_w are both NULL");
    Call c;
    c.op = (grad_x ? MUON_HEAD_GRAD_X : 0) | (grad_w ? MUON_HEAD_GRAD_W : 0);
    if (c.op == 0) c.op = MUON_HEAD_GRAD_X;
    c.x = x;
    c.w = w;
    c.targets = targets;
    c.lse = const_cast<float*>(lse);
    c.grad_loss = grad_loss;
    c.grad_lse = grad_lse;
    c.gx = grad_x;
    c.gw = grad_w;
    c.desc = desc;
    c.ws = workspace;
    c.ws_bytes = workspace_bytes;
    c.stream = reinterpret_cast<hipStream_t>(stream);
    return run(c);
  });
}

uint64_t muon_head_workspace_bytes(int32_t op, const muon_head_desc* desc) {
  uint64_t need = 0;
  (void)op_guarded([&]() -> muon_status {
    if (op < MUON_HEAD_LOSS || op > MUON_HEAD_GRAD_X_W) return op_fail(MUON_ERR_INVALID_ARGUMENT, "unknown op %d", op);
    Call c;
    c.op = op;
    c.desc = desc;
    muon_status st = check_desc(c);
    int cus = 0;
    if (st == MUON_OK) st = op_device(&cus);
    if (st == MUON_OK && desc->rows > 0) need = plan_of(c, cus).bytes;
    return st;
  });
  return need;
}

}  // extern "C"
