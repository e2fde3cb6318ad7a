// Host side of the block operators (muon_blocks.h): validation, the stages
// of the recursion, the workspace and the launches.
//
// A call is a sequence of stages; each runs three kernels over every block of
// a group of stacks: the Gram pass, the m x m recursion and the apply pass.
// Stacks are grouped by what selects a kernel's template: padded m, types and
// the stage limit.
#include "muon_blocks.h"

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <map>
#include <new>
#include <tuple>
#include <vector>

#include "api_internal.h"
#include "blocks_internal.h"

namespace muon {
namespace {

constexpr int64_t MAX_DIM = 65536;
constexpr int64_t MAX_BLOCKS = 1 << 20;
constexpr int32_t MAX_COUNT = 1 << 20;
constexpr int32_t MAX_NS_STEPS = 1000;
constexpr int64_t MAX_STRIDE = int64_t(1) << 40;

// Largest growth of small singular values between two Gram matrices.  The
// Gram matrix holds eigenvalues down to about 2^-24 of its trace, and the
// recursion carries its error on with the square of that growth, and so do the
// stages behind it in their turn.  Errors measured against float64; "one large"
// is a block of one singular value and m - 1 others at 1/20 to 1/3000 of it.
//
// bfloat16 results: one stage up to a growth of 512 by all steps (five quintic
// ones, 485, spectra from flat to i^-3 and rank-16 spikes 1e-4 to 6e-4, one
// large and its gradient 3e-3 beside the rounding of the result), stages of up
// to 150 where there is more (eight quintic steps, one large at 1/200 in binary32
// arithmetic: 5 + 3 steps 4e-3 and the gradient 3e-2, 4 + 4 2e-4 and 1e-3).
constexpr double LIMIT_BF16 = 512.0, LIMIT_BF16_MORE = 150.0;
// Binary32 results: 12 where the growth by all steps is more than 512 (six
// quintic steps, gradient of Gaussian blocks of 128 x 257: 3 + 3 steps 4e-5, 2 +
// 2 + 2 6e-6, binary32 iterates 4e-6), else the square root of RATIO times it,
// between 12 and 48: binary32 iterates lose with the whole growth, a stage with
// its square.  Cubic steps on 64 x 200: eight as one stage 2e-6 (Gaussian), 8e-6
// (plus 10) and 1.7e-5 (plus 100), as 4 + 4 7e-7, 1.4e-6 and 3e-6, binary32
// iterates 2e-7, 7e-7 and 2e-6; nine 2e-6, 1e-5 and 2.4e-5, as 5 + 4 8e-7, 1.3e-6
// and 3e-6.  Three quintic steps as one 1.5e-6, 4e-6 and 1.3e-5, as 2 + 1 1.3e-6,
// 1.0e-6 and 5e-6.  Five quintic steps are 3 + 2: 2e-6 to 8e-6, but one large at
// 1/20 2e-5 to 4e-5 and its gradient 4e-5, where binary32 iterates give 2e-6;
// 2 + 2 + 1 would give that too, at 1.3 to 1.5 times the time.
constexpr double LIMIT_F32 = 48.0, LIMIT_F32_LEAST = 12.0, RATIO_F32 = 3.5;
// Blocks of so few rows that a single bad direction counts (m <= 4; m <= 16
// up to n < 4 m) take LIMIT_F32 for bfloat16 results, and for binary32 ones
// the limits of nearly square blocks: the worst of 300000 random 2 x 3 blocks
// 2e-2 with LIMIT_BF16, 3.6e-3 so (2 x 4: 6e-3 and 3.7e-3; half a step of the
// result is up to 3.9e-3); binary32, 3 x 212 with a singular value 100 times
// the rest, 8e-6 with LIMIT_F32, 1.9e-6 so, binary32 iterates 2.0e-6.
constexpr int64_t FEW_ROWS = 4, FEW_ROWS_SHORT = 16;
// Binary32 results of nearly square blocks (n < 2 m), whose singular values
// reach down to zero: LIMIT_F32_LEAST, two quintic steps a stage, for the
// orthogonalisation, one step for its gradient (sixty random blocks, six steps,
// largest error: 2e-5 against 3e-5 with LIMIT_F32, and for the gradient the
// ninetieth percentile 6e-6 against 2e-5; binary32 iterates 2e-5 and 6e-6).
constexpr double LIMIT_VJP_SQUARE = 1.0;

muon_status fail(muon_status s, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  return api_fail(s, buf);
}

int64_t round_up(int64_t v, int64_t m) { return (v + m - 1) / m * m; }
size_t align256(size_t v) { return (v + 255) & ~size_t(255); }
// A row stride as the descriptor gives it, or of blocks of one row, where it
// may be anything, their length.
int64_t row_stride(const muon_block_desc& d, int64_t ld) { return d.rows == 1 ? d.cols : ld; }
int esize(int32_t dt) { return dt == MUON_DTYPE_BF16 ? 2 : 4; }

struct Call {
  int op = MUON_BLOCKS_NS;
  const void* const* x = nullptr;   // grad fields
  const void* const* y = nullptr;   // mom fields: cotangent (VJP) or momentum (STEP, written)
  void* const* out = nullptr;       // param fields
  float* const* upd = nullptr;
  const muon_block_desc* stacks = nullptr;
  int32_t count = 0;
  muon_ns_coeffs co = {0.f, 0.f, 0.f};
  int32_t ns_steps = 0;
  const muon_ns_coeffs* schedule = nullptr;
  const muon_step_hparams* hp = nullptr;
  void* ws = nullptr;
  uint64_t ws_bytes = 0;
  hipStream_t stream = nullptr;
};

// ------------------------------------------------------------- validation

// Bytes a tensor of blocks may touch: runs of `run` bytes, at lo + i bs + r rs
// for i < blocks and r < rows; and the grid its rows lie on: rows start `row`
// bytes apart from the first and are `win` bytes long (row = 0: no such grid).
struct Region {
  uintptr_t lo, hi;
  int64_t blocks, bs, rows, rs, run;
  uint64_t row, win;
  bool written;
  int32_t idx;
  const char* what;
};

Region region_of(const void* p, const muon_block_desc& d, int64_t ld, int64_t stride, int esz, bool written,
                 int32_t idx, const char* what) {
  ld = row_stride(d, ld);
  Region r;
  r.lo = reinterpret_cast<uintptr_t>(p);
  r.hi = r.lo + uint64_t((d.blocks - 1) * stride + (d.rows - 1) * ld + d.cols) * uint64_t(esz);
  r.blocks = stride > 0 ? d.blocks : 1;
  r.bs = stride * esz;
  r.rows = d.rows;
  r.rs = ld * esz;
  r.run = d.cols * esz;
  r.row = r.win = 0;
  if (d.blocks == 1 || stride % ld == 0) {
    r.row = uint64_t(ld) * esz;
    r.win = uint64_t(d.cols) * esz;
  } else if ((d.blocks - 1) * stride + d.cols <= ld) {
    r.row = uint64_t(ld) * esz;
    r.win = uint64_t((d.blocks - 1) * stride + d.cols) * esz;
  }
  r.written = written;
  r.idx = idx;
  r.what = what;
  return r;
}

int64_t floor_div(int64_t a, int64_t b) { return a / b - (a % b < 0 ? 1 : 0); }  // b > 0

// Whether two tensors of equal strides share a byte, exactly: whether their
// distance is x bs + y rs + z with x, y and z among the differences of two
// block numbers, row numbers and places in a run.  A stride that one of them
// does not use (one block, one row) is the other's.  Of the larger stride's
// differences few can be met where blocks lie apart or side by side; true
// where strides differ or many would have to be tried (read-only tensors).
bool runs_meet(const Region& a, const Region& b) {
  if ((a.blocks > 1 && b.blocks > 1 && a.bs != b.bs) || (a.rows > 1 && b.rows > 1 && a.rs != b.rs)) return true;
  struct Axis {
    int64_t step, lo, hi;  // differences lo .. hi, `step` bytes each
  };
  Axis o = {a.blocks > 1 ? a.bs : b.bs, 1 - b.blocks, a.blocks - 1};
  Axis i = {a.rows > 1 ? a.rs : b.rs, 1 - b.rows, a.rows - 1};
  for (Axis* x : {&o, &i})
    if (x->lo == x->hi || x->step == 0) *x = {1, 0, 0};
  if (o.step < i.step) std::swap(o, i);
  const int64_t d = int64_t(b.lo - a.lo), zlo = 1 - b.run, zhi = a.run - 1;
  const int64_t x0 = std::max(o.lo, -floor_div(i.hi * i.step + zhi - d, o.step));
  const int64_t x1 = std::min(o.hi, floor_div(d - i.lo * i.step - zlo, o.step));
  if (x1 - x0 > 64) return true;
  for (int64_t x = x0; x <= x1; ++x) {
    const int64_t e = d - x * o.step;  // y step + z
    const int64_t y0 = std::max(i.lo, -floor_div(zhi - e, i.step)), y1 = std::min(i.hi, floor_div(e - zlo, i.step));
    if (y0 <= y1) return true;
  }
  return false;
}

bool share_bytes(const Region& a, const Region& b) {  // a.lo <= b.lo
  if (b.lo >= a.hi) return false;
  if (!runs_meet(a, b)) return false;
  if (a.row == 0 || a.row != b.row) return true;
  // rows on one grid: disjoint if the windows are
  const uint64_t d = (b.lo - a.lo) % a.row;
  return !(d >= a.win && d + b.win <= a.row);
}

muon_status check_alias(std::vector<Region>& v) {
  std::sort(v.begin(), v.end(), [](const Region& a, const Region& b) { return a.lo < b.lo; });
  for (size_t i = 0; i < v.size(); ++i)
    for (size_t j = i + 1; j < v.size() && v[j].lo < v[i].hi; ++j)
      if ((v[i].written || v[j].written) && share_bytes(v[i], v[j]))
        return fail(MUON_ERR_ALIAS, "%s of stack %d overlaps %s of stack %d", v[j].what, v[j].idx, v[i].what, v[i].idx);
  return MUON_OK;
}

muon_status check_view(int32_t i, const char* what, const muon_block_desc& d, int64_t ld, int64_t stride,
                       int32_t dtype, bool f32_only, bool written) {
  if (dtype != MUON_DTYPE_F32 && (f32_only || dtype != MUON_DTYPE_BF16))
    return fail(MUON_ERR_UNSUPPORTED, "stack %d: %s dtype %d is not %s", i, what, dtype, f32_only ? "F32" : "F32 or BF16");
  ld = row_stride(d, ld);
  if (ld < d.cols || ld > BLOCK_MAX_LD)
    return fail(ld < d.cols ? MUON_ERR_INVALID_ARGUMENT : MUON_ERR_UNSUPPORTED,
                "stack %d: %s row stride %lld out of [cols = %lld, 2^21]", i, what, (long long)ld, (long long)d.cols);
  if (stride < 0 || stride > MAX_STRIDE)
    return fail(MUON_ERR_INVALID_ARGUMENT, "stack %d: %s block stride %lld out of [0, 2^40]", i, what,
                (long long)stride);
  if (written && d.blocks > 1) {
    const bool apart = stride >= (d.rows - 1) * ld + d.cols;
    const bool beside = stride >= d.cols && (d.blocks - 1) * stride + d.cols <= ld;
    if (!apart && !beside)
      return fail(MUON_ERR_ALIAS, "stack %d: blocks of %s share elements (rows %lld, cols %lld, row stride %lld, block "
                  "stride %lld)", i, what, (long long)d.rows, (long long)d.cols, (long long)ld, (long long)stride);
  }
  return MUON_OK;
}

muon_status check_ptr(int32_t i, const char* what, const void* p, int esz) {
  if (!p) return fail(MUON_ERR_INVALID_ARGUMENT, "stack %d: %s pointer is NULL", i, what);
  if (reinterpret_cast<uintptr_t>(p) % uintptr_t(esz) != 0)
    return fail(MUON_ERR_UNSUPPORTED, "stack %d: %s pointer is not aligned to %d bytes", i, what, esz);
  return MUON_OK;
}

bool finite3(const muon_ns_coeffs& c) { return std::isfinite(c.a) && std::isfinite(c.b) && std::isfinite(c.c); }

muon_status check_steps(const Call& c) {
  if (c.ns_steps < 0 || c.ns_steps > MAX_NS_STEPS)
    return fail(MUON_ERR_INVALID_ARGUMENT, "ns_steps %d out of range [0, %d]", c.ns_steps, MAX_NS_STEPS);
  if (!finite3(c.co)) return fail(MUON_ERR_INVALID_ARGUMENT, "ns_coeffs must be finite");
  if (c.schedule)
    for (int32_t k = 0; k < c.ns_steps; ++k)
      if (!finite3(c.schedule[k])) return fail(MUON_ERR_INVALID_ARGUMENT, "ns_schedule[%d] is not finite", k);
  return MUON_OK;
}

// Sizes, dtypes and strides of every stack (no pointers).
muon_status check_descs(const Call& c) {
  int64_t total = 0;
  for (int32_t i = 0; i < c.count; ++i) {
    const muon_block_desc& d = c.stacks[i];
    if (d.blocks < 0 || d.blocks > MAX_BLOCKS)
      return fail(d.blocks < 0 ? MUON_ERR_INVALID_ARGUMENT : MUON_ERR_UNSUPPORTED,
                  "stack %d: %lld blocks out of [0, 2^20]", i, (long long)d.blocks);
    if (d.rows < 1 || d.cols < 1)
      return fail(MUON_ERR_INVALID_ARGUMENT, "stack %d: rows and cols must be >= 1 (got %lld x %lld)", i,
                  (long long)d.rows, (long long)d.cols);
    if (d.rows > MAX_DIM || d.cols > MAX_DIM)
      return fail(MUON_ERR_UNSUPPORTED, "stack %d: rows and cols must be <= %lld", i, (long long)MAX_DIM);
    if (std::min(d.rows, d.cols) > BLOCK_MAX_M)
      return fail(MUON_ERR_UNSUPPORTED, "stack %d: blocks of %lld x %lld; min(rows, cols) must be <= %d (larger "
                  "matrices: muon_ns_batched, muon_step_batched)", i, (long long)d.rows, (long long)d.cols, BLOCK_MAX_M);
    if (d.reserved != 0) return fail(MUON_ERR_INVALID_ARGUMENT, "stack %d: reserved must be 0", i);
    muon_status st = check_view(i, c.op == MUON_BLOCKS_STEP ? "grad" : "x_in", d, d.ld_grad, d.stride_grad,
                                d.grad_dtype, false, false);
    if (st == MUON_OK)
      st = check_view(i, c.op == MUON_BLOCKS_STEP ? "param" : c.op == MUON_BLOCKS_VJP ? "grad_in" : "x_out", d,
                      d.ld_param, d.stride_param, d.param_dtype, false, true);
    if (st == MUON_OK && c.op == MUON_BLOCKS_VJP)
      st = check_view(i, "grad_out", d, d.ld_mom, d.stride_mom, d.mom_dtype, false, false);
    if (st == MUON_OK && c.op == MUON_BLOCKS_STEP)
      st = check_view(i, "momentum", d, d.ld_mom, d.stride_mom, d.mom_dtype, true, true);
    if (st != MUON_OK) return st;
    total += d.blocks;
    // the numbers of workgroups fit 31 bits: in a call of so many blocks one has
    // one gram workgroup and at most 2^16 / (6 * 64) apply workgroups
    if (total > (int64_t(1) << 21))
      return fail(MUON_ERR_UNSUPPORTED, "more than 2^21 blocks in one call");
  }
  return MUON_OK;
}

muon_status check_hparams(const Call& c) {
  if (!c.hp) return fail(MUON_ERR_INVALID_ARGUMENT, "hparams is NULL");
  const muon_step_hparams& h = *c.hp;
  if (!std::isfinite(h.lr)) return fail(MUON_ERR_INVALID_ARGUMENT, "lr is not finite");
  if (!(h.beta >= 0.f && h.beta < 1.f)) return fail(MUON_ERR_INVALID_ARGUMENT, "beta must be in [0, 1)");
  if (h.nesterov != 0 && h.nesterov != 1) return fail(MUON_ERR_INVALID_ARGUMENT, "nesterov must be 0 or 1");
  if (h.scale_rule < MUON_SCALE_NONE || h.scale_rule > MUON_SCALE_RMS_MATCH)
    return fail(MUON_ERR_INVALID_ARGUMENT, "unknown scale_rule %d", h.scale_rule);
  if (!h.options) return MUON_OK;
  const muon_step_options& o = *h.options;
  if (!std::isfinite(o.weight_decay) || o.weight_decay < 0.f)
    return fail(MUON_ERR_INVALID_ARGUMENT, "weight_decay must be finite and >= 0");
  if (o.momentum_kind != MUON_MOMENTUM_HEAVY_BALL && o.momentum_kind != MUON_MOMENTUM_EMA)
    return fail(MUON_ERR_INVALID_ARGUMENT, "unknown momentum_kind %d", o.momentum_kind);
  if (o.launch_mode < MUON_LAUNCH_AUTO || o.launch_mode > MUON_LAUNCH_CHAIN)
    return fail(MUON_ERR_INVALID_ARGUMENT, "unknown launch_mode %d", o.launch_mode);
  if (o.tile_mode < MUON_TILES_AUTO || o.tile_mode > MUON_TILES_SMALL)
    return fail(MUON_ERR_INVALID_ARGUMENT, "unknown tile_mode %d", o.tile_mode);
  if (o.launch_mode != MUON_LAUNCH_AUTO || o.tile_mode != MUON_TILES_AUTO)
    return fail(MUON_ERR_UNSUPPORTED, "launch_mode and tile_mode must be AUTO for blocks");
  for (int32_t i = 0; i < c.count; ++i) {
    if (o.lr_per_matrix && !std::isfinite(o.lr_per_matrix[i]))
      return fail(MUON_ERR_INVALID_ARGUMENT, "lr_per_matrix[%d] is not finite", i);
    if (o.scale_per_matrix && !std::isfinite(o.scale_per_matrix[i]))
      return fail(MUON_ERR_INVALID_ARGUMENT, "scale_per_matrix[%d] is not finite", i);
  }
  return MUON_OK;
}

muon_status validate(const Call& c) {
  if (c.count < 0 || c.count > MAX_COUNT)
    return fail(MUON_ERR_INVALID_ARGUMENT, "count %d out of range [0, %d]", c.count, MAX_COUNT);
  muon_status st;
  if (c.op == MUON_BLOCKS_STEP && (st = check_hparams(c)) != MUON_OK) return st;
  if ((st = check_steps(c)) != MUON_OK) return st;
  if (c.count == 0) return MUON_OK;
  if (!c.stacks) return fail(MUON_ERR_INVALID_ARGUMENT, "stacks is NULL");
  const bool vjp = c.op == MUON_BLOCKS_VJP, step = c.op == MUON_BLOCKS_STEP;
  if (!c.x || !c.out || ((vjp || step) && !c.y)) return fail(MUON_ERR_INVALID_ARGUMENT, "a pointer array is NULL");
  if ((st = check_descs(c)) != MUON_OK) return st;
  std::vector<Region> reg;
  reg.reserve(size_t(c.count) * 3 + 1);
  for (int32_t i = 0; i < c.count; ++i) {
    const muon_block_desc& d = c.stacks[i];
    if (d.blocks == 0) continue;
    const char* xn = step ? "grad" : "x_in";
    const char* yn = step ? "momentum" : "grad_out";
    const char* on = step ? "param" : vjp ? "grad_in" : "x_out";
    if ((st = check_ptr(i, xn, c.x[i], esize(d.grad_dtype))) != MUON_OK) return st;
    if ((st = check_ptr(i, on, c.out[i], esize(d.param_dtype))) != MUON_OK) return st;
    reg.push_back(region_of(c.x[i], d, d.ld_grad, d.stride_grad, esize(d.grad_dtype), false, i, xn));
    reg.push_back(region_of(c.out[i], d, d.ld_param, d.stride_param, esize(d.param_dtype), true, i, on));
    if (vjp || step) {
      if ((st = check_ptr(i, yn, c.y[i], esize(d.mom_dtype))) != MUON_OK) return st;
      reg.push_back(region_of(c.y[i], d, d.ld_mom, d.stride_mom, esize(d.mom_dtype), step, i, yn));
    }
    if (c.upd && c.upd[i]) {
      if ((st = check_ptr(i, "update", c.upd[i], 4)) != MUON_OK) return st;
      reg.push_back(region_of(c.upd[i], d, d.cols, d.rows * d.cols, 4, true, i, "update"));
    }
  }
  if (c.ws) {
    if (reinterpret_cast<uintptr_t>(c.ws) % 256 != 0)
      return fail(MUON_ERR_UNSUPPORTED, "workspace is not aligned to 256 bytes");
    const uintptr_t lo = reinterpret_cast<uintptr_t>(c.ws);
    reg.push_back({lo, lo + c.ws_bytes, 1, 0, 1, 0, int64_t(c.ws_bytes), 0, 0, true, -1, "workspace"});
  }
  return check_alias(reg);
}

// ------------------------------------------------------------------ stages

// Largest |a + b l + c l^2| over the squared singular values an iterate has
// (the usual quintic's stay below 1.45), at least 1.
double step_gain(const muon_ns_coeffs& k) {
  const double a = k.a, b = k.b, c = k.c, hi = 1.5;
  double q = std::max({1.0, std::fabs(a), std::fabs(a + b * hi + c * hi * hi)});
  if (c != 0) {
    const double v = -b / (2 * c);
    if (v > 0 && v < hi) q = std::max(q, std::fabs(a + b * v + c * v * v));
  }
  return q;
}

struct Stage {
  int32_t first, steps;
};

double step_gain_of(const Call& c, int32_t j) { return step_gain(c.schedule ? c.schedule[j] : c.co); }

// The limits of blocks that are neither of few rows nor nearly square.
struct Limits {
  double bf16, f32;
};
Limits limits_of(const Call& c) {
  double total = 1.0;
  for (int32_t j = 0; j < c.ns_steps && total <= LIMIT_BF16; ++j) total *= step_gain_of(c, j);
  if (total > LIMIT_BF16) return {LIMIT_BF16_MORE, LIMIT_F32_LEAST};
  return {LIMIT_BF16, std::min(LIMIT_F32, std::max(LIMIT_F32_LEAST, std::sqrt(RATIO_F32 * total)))};
}

// Stages as long as the limit allows.
std::vector<Stage> cut_stages(const std::vector<double>& gains, double limit) {
  std::vector<Stage> out;
  const int32_t n = int32_t(gains.size());
  for (int32_t j = 0; j < n;) {
    int32_t r = 1;
    double gain = gains[size_t(j)];
    while (j + r < n && r < BLOCK_STAGE_STEPS && gain * gains[size_t(j + r)] <= limit) gain *= gains[size_t(j + r++)];
    out.push_back({j, r});
    j += r;
  }
  if (out.empty()) out.push_back({0, 0});
  return out;
}

// As few stages as the limit allows, and these as even as can be: the least
// limit that gives as many.
std::vector<Stage> stages_of(const Call& c, double limit) {
  std::vector<double> gains;
  for (int32_t j = 0; j < c.ns_steps; ++j) gains.push_back(step_gain_of(c, j));
  std::vector<Stage> best = cut_stages(gains, limit);
  double lo = 0.0, hi = std::log2(limit);
  for (int32_t k = 0; k < 24 && best.size() > 1; ++k) {
    const double mid = 0.5 * (lo + hi);
    std::vector<Stage> s = cut_stages(gains, std::exp2(mid));
    if (s.size() > best.size()) {
      lo = mid;
    } else {
      hi = mid;
      best = std::move(s);
    }
  }
  return best;
}

// ------------------------------------------------------------------ groups

struct Group {
  int mt = 2;
  bool f32 = false, xbf = false, ybf = false;  // result class, input types
  double limit = LIMIT_BF16;
  std::vector<int32_t> members;     // stacks of the call
  int64_t blocks = 0;
  std::vector<Stage> stages;
  int32_t gram_wgs = 0, apply_wgs = 0;
  int parts = 1;                    // of a call with the library's workspace
  std::vector<BlockStack> base;     // sizes and splits; views are filled per stage
  std::vector<size_t> stage_off;    // per member: byte offset of its binary32 copy in a stage buffer
  size_t stage_bytes = 0;           // one stage buffer
  int32_t stage_bufs = 0, tables = 0;
  // byte offsets in the workspace
  size_t o_tab = 0, o_part = 0, o_p = 0, o_t = 0, o_scr = 0, o_stage = 0, end = 0;
};

// Parts of a group that a call with the library's workspace runs on streams of
// their own.  Measured,
// time on one stream over time in two, three and four parts:
//  - several stages (binary32): the gradient 130 blocks 0.97 to 1.04, 216 to
//    600 1.03 to 1.20 in two; forward at 128 rows 130 to 200 0.97 to 1.01, 300
//    to 600 1.04 to 1.06 in two; at 64 rows 576 0.96 to 1.00, 1200 1.04;
//  - the bfloat16 step at 128 rows 400 blocks 0.99, 0.96, 1.03; 520 to 1500
//    1.00 to 1.04, 1.02 to 1.09, 0.99 to 1.05;
//  - the other bfloat16 calls at 128 rows gain where a second round of the
//    recursion (a compute unit holds two blocks, of the gradient one) would be
//    nearly empty: the gradient 260 to 330 1.10 to 1.13 in two, 400 0.98, 200
//    0.93, 640 1.00; forward 520 to 576 1.01 to 1.04, 640 0.91, 1152 0.97;
//  - the same at 64 rows 0.95 to 0.98.
constexpr int MAX_PARTS = 3;
int parts_of(const Group& g, int op, int64_t cus) {
  const bool vjp = op == MUON_BLOCKS_VJP;
  if (g.stages.size() > 1) return g.blocks >= (vjp ? cus * 3 / 4 : g.mt == 8 ? cus : 4 * cus) ? 2 : 1;
  if (g.mt != 8) return 1;
  const int64_t round = vjp ? cus : 2 * cus;
  if (op == MUON_BLOCKS_STEP) return g.blocks > round ? 3 : 1;
  return g.blocks > round && g.blocks <= round + cus * 3 / 8 ? 2 : 1;
}

int64_t ld_of_stage(const muon_block_desc& d) { return round_up(d.cols, 4); }

// A device table and its keys.
size_t table_bytes(size_t n) { return align256(sizeof(BlockStack) * n) + align256(sizeof(int32_t) * KEY_COUNT * n); }

// Splits the call into groups and lays out the workspace (the groups run one
// after another and share it).  Returns its size.
size_t plan_groups(const Call& c, int cus, std::vector<Group>& groups) {
  std::map<std::vector<int64_t>, size_t> where;
  const bool vjp = c.op == MUON_BLOCKS_VJP;
  const Limits limits = limits_of(c);
  for (int32_t i = 0; i < c.count; ++i) {
    const muon_block_desc& d = c.stacks[i];
    if (d.blocks == 0) continue;
    const int64_t m = std::min(d.rows, d.cols), n = std::max(d.rows, d.cols);
    Group g;
    g.mt = block_mt(int(m));
    g.f32 = d.param_dtype == MUON_DTYPE_F32;
    g.xbf = d.grad_dtype == MUON_DTYPE_BF16;
    g.ybf = vjp && d.mom_dtype == MUON_DTYPE_BF16;
    const bool few = m <= FEW_ROWS || (m <= FEW_ROWS_SHORT && n < 4 * m), square = few || n < 2 * m;
    g.limit = !g.f32 ? (few ? LIMIT_F32 : limits.bf16)
              : !square ? limits.f32 : vjp ? LIMIT_VJP_SQUARE : LIMIT_F32_LEAST;
    int64_t limit_bits;
    memcpy(&limit_bits, &g.limit, sizeof(limit_bits));
    const std::vector<int64_t> key = {g.mt, g.f32, g.xbf, g.ybf, limit_bits};
    auto it = where.find(key);
    if (it == where.end()) {
      it = where.emplace(key, groups.size()).first;
      groups.push_back(g);
    }
    Group& q = groups[it->second];
    q.members.push_back(i);
    q.blocks += d.blocks;
  }
  size_t need = 0;
  for (Group& g : groups) {
    const int kc = block_kc(g.mt), mp = 16 * g.mt;
    const int kind = vjp ? BK_VJP : c.op == MUON_BLOCKS_STEP ? BK_STEP : BK_X;
    g.stages = stages_of(c, g.limit);
    // members of equal shapes and strides next to each other: runs that differ
    // in their pointers only take one entry of a table launch
    auto key = [&](int32_t i) {
      const muon_block_desc& d = c.stacks[i];
      return std::make_tuple(d.rows, d.cols, d.blocks, d.ld_grad, d.ld_param, d.ld_mom, d.stride_grad, d.stride_param,
                             d.stride_mom);
    };
    std::stable_sort(g.members.begin(), g.members.end(), [&](int32_t a, int32_t b) { return key(a) < key(b); });
    // gram workgroups enough to fill the GPU once, two to a compute unit, each
    // with two tiles of columns at least: more even ones write more partials
    // (128 rows: 36 KB each, the gradient's 100), which the recursion reads;
    // two a block, up to where even those are many rounds.  Both passes with 8,
    // 4, 2 and 1 workgroups a compute unit: the gradient of 288 bfloat16 blocks
    // of 128 x 1536 420, 378, 361 and 356 us, 576 of them forward 227, 219, 218
    // and 218; the step of 48 79, 79, 76 and 79, of 1152 (two a block, one, one
    // and one) 714, 728, 725 and 721; 576 binary32 blocks of 64 x 768 (four a
    // block, two, one and one) 51, 49, 50 and 49, the step's Gram pass 78 with
    // one and 72 us with two.  The apply pass takes four times as many.
    g.parts = parts_of(g, c.op, cus);
    const int64_t launch = (g.blocks + g.parts - 1) / g.parts;
    const int64_t per = std::max<int64_t>((2 * int64_t(cus) + launch - 1) / launch, launch < 8 * cus ? 2 : 1);
    const int64_t aper = (8 * int64_t(cus) + g.blocks - 1) / g.blocks;
    auto chunk = [&](int64_t n, int64_t split) {
      return int32_t(std::max<int64_t>(round_up((n + split - 1) / split, kc), 2 * kc));
    };
    int64_t goff = 0, aoff = 0, block0 = 0, part = 0;
    for (int32_t i : g.members) {
      const muon_block_desc& d = c.stacks[i];
      BlockStack s;
      memset(&s, 0, sizeof(s));
      const bool tr = d.rows > d.cols;
      s.m = int32_t(std::min(d.rows, d.cols));
      s.n = int32_t(std::max(d.rows, d.cols));
      s.cols = int32_t(d.cols);
      s.blocks = int32_t(d.blocks);
      s.block0 = int32_t(block0);
      s.flags = tr ? BF_TR : 0;
      s.gchunk = chunk(s.n, per);
      s.gsplit = (s.n + s.gchunk - 1) / s.gchunk;
      // apply workgroups of six tiles at most: what runs at a time lies closer
      // together in memory (1152 blocks of 128 x 1536, the step's: 2 tiles 500
      // us, 4 488, 6 482, 12 494, 24 534)
      s.achunk = std::min(chunk(s.n, aper), 6 * kc);
      // one tile each where every compute unit has one at most (two tiles and
      // one: 12 blocks of 64 x 768 5.3 and 4.3 us, 12 binary32 ones of 16 rows
      // 7.9 and 5.4, their gradient 11.2 and 7.3; with two workgroups a
      // compute unit no gain, the gradient 15.1 and 17.7).  A gram pass so cut
      // gains 0.8 us and the recursion, which adds up its partials, loses 1
      if (g.blocks * ((s.n + kc - 1) / kc) <= cus) s.achunk = kc;
      s.asplit = (s.n + s.achunk - 1) / s.achunk;
      s.goff = int32_t(goff);
      s.aoff = int32_t(aoff);
      s.part0 = part;
      s.part = block_part_floats(g.mt, kind);
      s.d = 1.f;
      goff += d.blocks * s.gsplit;
      aoff += d.blocks * s.asplit;
      part += d.blocks * s.gsplit * s.part;
      block0 += d.blocks;
      g.base.push_back(s);
      g.stage_off.push_back(g.stage_bytes);
      g.stage_bytes += align256(size_t(d.blocks) * size_t(d.rows) * size_t(ld_of_stage(d)) * 4);
    }
    g.gram_wgs = int32_t(goff);
    g.apply_wgs = int32_t(aoff);
    const int32_t nst = int32_t(g.stages.size());
    g.tables = vjp ? 2 * nst - 1 : nst;
    g.stage_bufs = nst == 1 ? 0 : vjp ? nst : 1;
    const int pp = g.f32 ? 3 : 2;
    size_t o = 0;
    g.o_tab = o;
    if (g.base.size() > size_t(BLOCK_INLINE)) o += table_bytes(g.base.size()) * size_t(g.tables);
    g.o_part = o;
    o += align256(size_t(part) * 4);
    g.o_p = o;
    o += align256(size_t(g.blocks) * pp * mp * mp * 2);
    if (vjp) {
      g.o_t = o;
      o += align256(size_t(g.blocks) * pp * mp * mp * 2);
      g.o_scr = o;
      o += align256(size_t(g.blocks) * 2 * mp * mp * 4);
    }
    g.o_stage = o;
    o += g.stage_bytes * size_t(g.stage_bufs);
    g.end = o;
    need = std::max(need, o);
  }
  return need;
}

double rule_scale(int rule, int64_t rows, int64_t cols) {
  if (rule == MUON_SCALE_SQRT_ASPECT) return std::sqrt(std::max(1.0, double(rows) / double(cols)));
  if (rule == MUON_SCALE_RMS_MATCH) return 0.2 * std::sqrt(double(std::max(rows, cols)));
  return 1.0;
}

// One stage's three launches.
struct Phase {
  BlockTable tab;
  int kind = BK_X, pl = 1;
  bool xbf = false;
  BlockSteps steps;
};

// The stages of a group in order, with their tables (written on the call's
// stream where they are in device memory).
hipError_t group_phases(const Call& c, const Group& g, char* ws, std::vector<Phase>& out) {
  const bool vjp = c.op == MUON_BLOCKS_VJP, step = c.op == MUON_BLOCKS_STEP;
  const int32_t nst = int32_t(g.stages.size());

  // views of a member: the caller's tensors, or stage buffer `buf`
  auto set_x = [&](BlockStack& s, size_t k, int buf) {
    const int32_t i = g.members[k];
    const muon_block_desc& d = c.stacks[i];
    if (buf < 0) {
      s.x = c.x[i];
      s.x_ld = row_stride(d, d.ld_grad);
      s.x_bs = d.stride_grad;
      if (g.xbf) s.flags |= BF_X_BF16;
    } else {
      s.x = ws + g.o_stage + size_t(buf) * g.stage_bytes + g.stage_off[k];
      s.x_ld = ld_of_stage(d);
      s.x_bs = d.rows * s.x_ld;
    }
  };
  auto set_y = [&](BlockStack& s, size_t k, int buf) {
    const int32_t i = g.members[k];
    const muon_block_desc& d = c.stacks[i];
    if (buf < 0) {
      s.y = c.y[i];
      s.y_ld = row_stride(d, d.ld_mom);
      s.y_bs = d.stride_mom;
      if (d.mom_dtype == MUON_DTYPE_BF16) s.flags |= BF_Y_BF16;
    } else {
      s.y = ws + g.o_stage + size_t(buf) * g.stage_bytes + g.stage_off[k];
      s.y_ld = ld_of_stage(d);
      s.y_bs = d.rows * s.y_ld;
    }
  };
  auto set_out = [&](BlockStack& s, size_t k, int buf) {
    const int32_t i = g.members[k];
    const muon_block_desc& d = c.stacks[i];
    if (buf < 0) {
      s.out = c.out[i];
      s.out_ld = row_stride(d, d.ld_param);
      s.out_bs = d.stride_param;
      if (!g.f32) s.flags |= BF_OUT_BF16;
      if (step) {
        s.flags |= BF_WRITEBACK;
        s.upd = c.upd ? c.upd[i] : nullptr;
        const muon_step_options* o = c.hp->options;
        const float lr = o && o->lr_per_matrix ? o->lr_per_matrix[i] : c.hp->lr;
        const double sc = o && o->scale_per_matrix ? double(o->scale_per_matrix[i])
                                                   : rule_scale(c.hp->scale_rule, d.rows, d.cols);
        s.t = float(double(lr) * sc);
        const float wd = o ? o->weight_decay : 0.f;
        const float lw = lr * wd;
        s.d = wd != 0.f ? 1.f - lw : 1.f;
      }
    } else {
      s.out = ws + g.o_stage + size_t(buf) * g.stage_bytes + g.stage_off[k];
      s.out_ld = ld_of_stage(d);
      s.out_bs = d.rows * s.out_ld;
    }
  };

  int32_t table = 0;
  auto set_table = [&](BlockTable& tab, const std::vector<BlockStack>& v) -> hipError_t {
    memset(&tab, 0, sizeof(tab));
    tab.count = int32_t(v.size());
    if (v.size() <= size_t(BLOCK_INLINE)) {
      memcpy(tab.inl, v.data(), sizeof(BlockStack) * v.size());
      for (size_t k = 0; k < v.size(); ++k) {
        tab.keys[KEY_GRAM][k] = v[k].goff;
        tab.keys[KEY_BLOCK][k] = v[k].block0;
        tab.keys[KEY_APPLY][k] = v[k].aoff;
      }
      return hipSuccess;
    }
    char* at = ws + g.o_tab + size_t(table++) * table_bytes(v.size());
    BlockStack* dev = reinterpret_cast<BlockStack*>(at);
    int32_t* keys = reinterpret_cast<int32_t*>(at + align256(sizeof(BlockStack) * v.size()));
    tab.ext = dev;
    tab.ext_keys = keys;
    return launch_block_table(v.data(), int32_t(v.size()), dev, keys, c.stream);
  };
  auto steps_of = [&](const Stage& st, bool first) {
    BlockSteps s;
    memset(&s, 0, sizeof(s));
    s.steps = st.steps;
    s.first = first;
    for (int32_t k = 0; k < st.steps; ++k) {
      const muon_ns_coeffs& co = c.schedule ? c.schedule[st.first + k] : c.co;
      s.a[k] = co.a;
      s.b[k] = co.b;
      s.c[k] = co.c;
    }
    return s;
  };

  // forward stages; for the gradient all but the last, into a buffer each
  const int32_t fwd = vjp ? nst - 1 : nst;
  out.resize(size_t(fwd + (vjp ? nst : 0)));
  size_t at = 0;
  for (int32_t i = 0; i < fwd; ++i) {
    Phase& p = out[at++];
    std::vector<BlockStack> v = g.base;
    const bool user_u = step && i == 0;
    const int src = i == 0 ? -1 : vjp ? i - 1 : 0;
    const int dst = vjp ? i : i == nst - 1 ? -1 : 0;
    for (size_t k = 0; k < v.size(); ++k) {
      set_x(v[k], k, src);
      if (user_u) set_y(v[k], k, -1);
      set_out(v[k], k, dst);
    }
    p.kind = user_u ? BK_STEP : BK_X;
    p.pl = g.f32 ? 3 : (user_u || i > 0 || !g.xbf) ? 2 : 1;
    p.xbf = i == 0 && g.xbf;
    p.steps = steps_of(g.stages[size_t(i)], i == 0);
    const hipError_t e = set_table(p.tab, v);
    if (e != hipSuccess) return e;
  }
  if (!vjp) return hipSuccess;
  // backward stages: the cotangent of stage i's input, in place in the last buffer
  for (int32_t i = nst - 1; i >= 0; --i) {
    Phase& p = out[at++];
    std::vector<BlockStack> v = g.base;
    for (size_t k = 0; k < v.size(); ++k) {
      set_x(v[k], k, i - 1);
      set_y(v[k], k, i == nst - 1 ? -1 : nst - 1);
      set_out(v[k], k, i == 0 ? -1 : nst - 1);
    }
    p.kind = BK_VJP;
    p.xbf = i == 0 && g.xbf;
    p.pl = g.f32 ? 3 : (p.xbf && i == nst - 1 && g.ybf) ? 1 : 2;
    p.steps = steps_of(g.stages[size_t(i)], i == 0);
    const hipError_t e = set_table(p.tab, v);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// First gram and apply workgroup of block b (the group's count for b = all).
void workgroups_at(const Group& g, int64_t b, int32_t& gram, int32_t& apply) {
  gram = g.gram_wgs;
  apply = g.apply_wgs;
  for (size_t k = g.base.size(); k-- > 0;) {
    const BlockStack& s = g.base[k];
    if (b < s.block0 || b >= s.block0 + s.blocks) continue;
    gram = s.goff + int32_t(b - s.block0) * s.gsplit;
    apply = s.aoff + int32_t(b - s.block0) * s.asplit;
  }
}

// Launches workgroups [first, end) of a pass over `tab` by launch(how many).
// HIP takes fewer than 2^32 threads a launch (2^21 blocks of 1 x 5000 are 2^23
// apply workgroups of 512): more run in slices, which the table's first
// workgroup allows.
template <class Launch>
hipError_t in_slices(BlockTable& tab, int32_t first, int32_t end, Launch&& launch) {
  constexpr int32_t SLICE = 1 << 22;
  hipError_t e = hipSuccess;
  for (int32_t at = first; at < end && e == hipSuccess; at += std::min(SLICE, end - at)) {
    tab.first = at;
    e = launch(std::min(SLICE, end - at));
  }
  return e;
}

// Enqueues phase `p` for blocks [b0, b1) on `stream`; every launch goes
// through run(kernel class, launch).  `after`, where not null, is recorded
// behind the gram pass.
template <class Run>
hipError_t enqueue_phase(const Call& c, const Group& g, Phase& p, char* ws, int64_t b0, int64_t b1, hipStream_t stream,
                         hipEvent_t after, Run&& run) {
  const bool vjp = c.op == MUON_BLOCKS_VJP;
  const int pp = g.f32 ? 3 : 2;
  float* parts = reinterpret_cast<float*>(ws + g.o_part);
  uint16_t* P = reinterpret_cast<uint16_t*>(ws + g.o_p);
  uint16_t* T = vjp ? reinterpret_cast<uint16_t*>(ws + g.o_t) : nullptr;
  float* scr = vjp ? reinterpret_cast<float*>(ws + g.o_scr) : nullptr;
  BlockMom mom = {0.f, 1.f, 0, 0};
  if (p.kind == BK_STEP) {
    mom.beta = c.hp->beta;
    mom.nesterov = c.hp->nesterov;
    mom.ema = c.hp->options && c.hp->options->momentum_kind == MUON_MOMENTUM_EMA;
    mom.g1 = mom.ema ? 1.f - c.hp->beta : 1.f;
  }
  int32_t g0, g1, a0, a1;
  workgroups_at(g, b0, g0, a0);
  workgroups_at(g, b1, g1, a1);
  hipError_t e = run(p.kind == BK_STEP ? MUON_KC_MOMENTUM : MUON_KC_GRAM, [&] {
    return in_slices(p.tab, g0, g1, [&](int32_t wgs) {
      return launch_block_gram(g.mt, p.pl, p.kind, p.xbf, p.tab, wgs, parts, mom, stream);
    });
  });
  if (e == hipSuccess && after) e = hipEventRecord(after, stream);
  if (e != hipSuccess) return e;
  p.tab.first = int32_t(b0);
  e = run(MUON_KC_POLY, [&] {
    return launch_block_iterate(g.mt, pp, p.kind == BK_VJP ? BK_VJP : BK_X, p.tab, int32_t(b1 - b0), parts, P, T, scr,
                                p.steps, stream);
  });
  if (e != hipSuccess) return e;
  return run(MUON_KC_COMBINE, [&] {
    return in_slices(p.tab, a0, a1, [&](int32_t wgs) {
      return launch_block_apply(g.mt, p.pl, pp, p.kind, p.xbf, p.tab, wgs, P, T, mom, stream);
    });
  });
}

// -------------------------------------------------------------- workspaces

struct BlockDevice {
  int cus = 0;
  void* ws = nullptr;
  size_t ws_bytes = 0;
  hipEvent_t last = nullptr;   // after the last call that used ws
  bool recorded = false;
  // the further streams of a large call and their events
  hipStream_t side[MAX_PARTS - 1] = {};
  hipEvent_t fork[MAX_PARTS - 1] = {}, join[MAX_PARTS - 1] = {};
};
std::map<int, BlockDevice> g_blocks;  // under api_mutex()

void release_blocks() {
  for (auto& kv : g_blocks) {
    if (hipSetDevice(kv.first) != hipSuccess) continue;
    (void)hipDeviceSynchronize();
    if (kv.second.ws) (void)hipFree(kv.second.ws);
    if (kv.second.last) (void)hipEventDestroy(kv.second.last);
    for (int k = 0; k < MAX_PARTS - 1; ++k) {
      if (kv.second.side[k]) (void)hipStreamDestroy(kv.second.side[k]);
      if (kv.second.fork[k]) (void)hipEventDestroy(kv.second.fork[k]);
      if (kv.second.join[k]) (void)hipEventDestroy(kv.second.join[k]);
    }
  }
  g_blocks.clear();
}
struct HookRelease {
  HookRelease() { api_release_hook = release_blocks; }
} g_hook_release;

muon_status current_device(BlockDevice** out) {
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess) {
    (void)hipGetLastError();
    return fail(MUON_ERR_HIP, "hipGetDevice failed (no HIP device?)");
  }
  BlockDevice& bd = g_blocks[dev];
  if (bd.cus == 0) {
    int cus = 0;
    if (hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || cus <= 0) {
      (void)hipGetLastError();
      return fail(MUON_ERR_HIP, "cannot query the compute-unit count of device %d", dev);
    }
    bd.cus = cus;
  }
  *out = &bd;
  return MUON_OK;
}

// The streams of `parts` parts and their events; without them a call runs on
// its own stream.
bool side_streams(BlockDevice& bd, int parts) {
  for (int k = 0; k < parts - 1; ++k) {
    if (!bd.side[k] && hipStreamCreateWithFlags(&bd.side[k], hipStreamNonBlocking) != hipSuccess) bd.side[k] = nullptr;
    if (!bd.fork[k] && hipEventCreateWithFlags(&bd.fork[k], hipEventDisableTiming) != hipSuccess) bd.fork[k] = nullptr;
    if (!bd.join[k] && hipEventCreateWithFlags(&bd.join[k], hipEventDisableTiming) != hipSuccess) bd.join[k] = nullptr;
    if (!bd.side[k] || !bd.fork[k] || !bd.join[k]) {
      (void)hipGetLastError();
      return false;
    }
  }
  return true;
}

// Enqueues one group.  The recursion keeps the matrix cores busy and the other
// two passes the memory, so a group may be cut into parts: each but the first
// runs on a stream of its own, behind the gram pass of the part before, and
// one part's recursion runs beside another's passes over memory.  The streams
// are the device's: only calls with the library's workspace use them, which
// run one after another anyway.  A call with a workspace of its own would wait
// behind whatever an earlier call's parts still wait for.
hipError_t enqueue_group(const Call& c, const Group& g, char* ws, BlockDevice& bd, bool capturing) {
  std::vector<Phase> phases;
  hipError_t e = group_phases(c, g, ws, phases);
  const bool split = g.parts > 1 && !c.ws && !api_timing() && side_streams(bd, g.parts);
  const int parts = split ? g.parts : 1;
  auto run = [&](int kc, auto&& launch) -> hipError_t {
    return capturing ? launch() : api_timed(kc, c.stream, launch);
  };
  int used = 1;
  for (size_t i = 0; i < phases.size() && e == hipSuccess; ++i)
    for (int k = 0; k < parts && e == hipSuccess; ++k) {
      hipStream_t s = k == 0 ? c.stream : bd.side[k - 1];
      if (i == 0 && k > 0) {
        e = hipStreamWaitEvent(s, bd.fork[k - 1], 0);
        if (e != hipSuccess) break;
        used = k + 1;
      }
      e = enqueue_phase(c, g, phases[i], ws, g.blocks * k / parts, g.blocks * (k + 1) / parts, s,
                        i == 0 && k + 1 < parts ? bd.fork[k] : nullptr, run);
    }
  // also after a failed launch: what was enqueued belongs to this call
  for (int k = 1; k < used; ++k) {
    const hipError_t j = hipEventRecord(bd.join[k - 1], bd.side[k - 1]);
    const hipError_t w = j == hipSuccess ? hipStreamWaitEvent(c.stream, bd.join[k - 1], 0) : j;
    if (e == hipSuccess) e = w;
  }
  return e;
}

muon_status run_call(const Call& c) {
  muon_status st = validate(c);
  if (st != MUON_OK) return st;
  bool any = false;
  for (int32_t i = 0; i < c.count && !any; ++i) any = c.stacks[i].blocks > 0;
  if (!any) return MUON_OK;
  std::lock_guard<std::mutex> lock(api_mutex());
  BlockDevice* bd = nullptr;
  if ((st = current_device(&bd)) != MUON_OK) return st;
  std::vector<Group> groups;
  const size_t need = plan_groups(c, bd->cus, groups);

  hipStreamCaptureStatus cap = hipStreamCaptureStatusNone;
  if (hipStreamIsCapturing(c.stream, &cap) != hipSuccess) {
    // the null stream while another stream captures
    (void)hipGetLastError();
    return fail(MUON_ERR_HIP, "the stream cannot be used during another stream's capture");
  }
  const bool capturing = cap != hipStreamCaptureStatusNone;
  char* ws = reinterpret_cast<char*>(c.ws);
  if (c.ws) {
    if (c.ws_bytes < need)
      return fail(MUON_ERR_INVALID_ARGUMENT, "the workspace holds %llu bytes; this call needs %zu",
                  (unsigned long long)c.ws_bytes, need);
  } else {
    if (capturing)
      return fail(MUON_ERR_UNSUPPORTED, "a captured call needs a workspace of the caller's "
                  "(muon_blocks_workspace_bytes: %zu bytes)", need);
    if (need > bd->ws_bytes) {
      if (hipDeviceSynchronize() != hipSuccess)
        return fail(MUON_ERR_HIP, "hipDeviceSynchronize failed: %s", hipGetErrorString(hipGetLastError()));
      if (bd->ws) (void)hipFree(bd->ws);
      bd->ws = nullptr;
      bd->ws_bytes = 0;
      void* p = nullptr;
      if (api_device_alloc(&p, need) != hipSuccess) {
        (void)hipGetLastError();
        return fail(MUON_ERR_OUT_OF_MEMORY, "workspace allocation of %zu bytes failed", need);
      }
      bd->ws = p;
      bd->ws_bytes = need;
    }
    if (!bd->last && hipEventCreateWithFlags(&bd->last, hipEventDisableTiming) != hipSuccess) {
      bd->last = nullptr;
      return fail(MUON_ERR_HIP, "hipEventCreate failed: %s", hipGetErrorString(hipGetLastError()));
    }
    if (bd->recorded && hipStreamWaitEvent(c.stream, bd->last, 0) != hipSuccess)
      return fail(MUON_ERR_HIP, "ordering after the device's previous call failed: %s",
                  hipGetErrorString(hipGetLastError()));
    ws = reinterpret_cast<char*>(bd->ws);
  }

  // an error that an earlier call of the thread's left would be taken for one of
  // the first launch, whose kernel runs all the same
  (void)hipGetLastError();
  hipError_t e = hipSuccess;
  for (const Group& g : groups) {
    e = enqueue_group(c, g, ws, *bd, capturing);
    if (e != hipSuccess) break;
  }
  if (!c.ws && hipEventRecord(bd->last, c.stream) == hipSuccess) bd->recorded = true;
  if (e != hipSuccess) return fail(MUON_ERR_HIP, "kernel launch failed: %s", hipGetErrorString(e));
  return MUON_OK;
}

// Nothing crosses the ABI as an exception.
muon_status guarded(const Call& c) {
  api_clear_error();
  try {
    return run_call(c);
  } catch (const std::bad_alloc&) {
    return api_fail(MUON_ERR_OUT_OF_MEMORY, "host memory allocation failed");
  } catch (...) {
    return api_fail(MUON_ERR_HIP, "unexpected failure on the host");
  }
}

}  // namespace
}  // namespace muon

using namespace muon;

extern "C" {

muon_status muon_ns_blocks(const void* const* x_in, void* const* x_out, const muon_block_desc* stacks,
                           int32_t count, muon_ns_coeffs ns_coeffs, int32_t ns_steps,
                           const muon_ns_coeffs* ns_schedule, void* workspace, uint64_t workspace_bytes,
                           void* stream) {
  Call c;
  c.op = MUON_BLOCKS_NS;
  c.x = x_in;
  c.out = x_out;
  c.stacks = stacks;
  c.count = count;
  c.co = ns_coeffs;
  c.ns_steps = ns_steps;
  c.schedule = ns_schedule;
  c.ws = workspace;
  c.ws_bytes = workspace_bytes;
  c.stream = reinterpret_cast<hipStream_t>(stream);
  return guarded(c);
}

muon_status muon_ns_blocks_vjp(const void* const* x_in, const void* const* grad_out, void* const* grad_in,
                               const muon_block_desc* stacks, int32_t count, muon_ns_coeffs ns_coeffs,
                               int32_t ns_steps, const muon_ns_coeffs* ns_schedule, void* workspace,
                               uint64_t workspace_bytes, void* stream) {
  Call c;
  c.op = MUON_BLOCKS_VJP;
  c.x = x_in;
  c.y = grad_out;
  c.out = grad_in;
  c.stacks = stacks;
  c.count = count;
  c.co = ns_coeffs;
  c.ns_steps = ns_steps;
  c.schedule = ns_schedule;
  c.ws = workspace;
  c.ws_bytes = workspace_bytes;
  c.stream = reinterpret_cast<hipStream_t>(stream);
  return guarded(c);
}

muon_status muon_step_blocks(void* const* params, const void* const* grads, void* const* momenta,
                             const muon_block_desc* stacks, int32_t count, const muon_step_hparams* hparams,
                             float* const* updates_out, void* workspace, uint64_t workspace_bytes, void* stream) {
  Call c;
  c.op = MUON_BLOCKS_STEP;
  c.x = grads;
  c.y = momenta;
  c.out = params;
  c.upd = updates_out;
  c.stacks = stacks;
  c.count = count;
  c.hp = hparams;
  if (hparams) {
    c.co = hparams->ns_coeffs;
    c.ns_steps = hparams->ns_steps;
    c.schedule = hparams->options ? hparams->options->ns_schedule : nullptr;
  }
  c.ws = workspace;
  c.ws_bytes = workspace_bytes;
  c.stream = reinterpret_cast<hipStream_t>(stream);
  return guarded(c);
}

uint64_t muon_blocks_workspace_bytes(int32_t op, const muon_block_desc* stacks, int32_t count,
                                     muon_ns_coeffs ns_coeffs, int32_t ns_steps,
                                     const muon_ns_coeffs* ns_schedule) {
  api_clear_error();
  if (op < MUON_BLOCKS_NS || op > MUON_BLOCKS_STEP) {
    (void)fail(MUON_ERR_INVALID_ARGUMENT, "unknown op %d", op);
    return 0;
  }
  try {
    Call c;
    c.op = op;
    c.stacks = stacks;
    c.count = count;
    c.co = ns_coeffs;
    c.ns_steps = ns_steps;
    c.schedule = ns_schedule;
    if (count < 0 || count > MAX_COUNT || (count > 0 && !stacks)) {
      (void)fail(MUON_ERR_INVALID_ARGUMENT, "bad count or NULL stacks");
      return 0;
    }
    if (check_steps(c) != MUON_OK || check_descs(c) != MUON_OK) return 0;
    std::lock_guard<std::mutex> lock(api_mutex());
    BlockDevice* bd = nullptr;
    if (current_device(&bd) != MUON_OK) return 0;
    std::vector<Group> groups;
    return plan_groups(c, bd->cus, groups);
  } catch (...) {
    (void)api_fail(MUON_ERR_OUT_OF_MEMORY, "host memory allocation failed");
    return 0;
  }
}

}  // extern "C"
