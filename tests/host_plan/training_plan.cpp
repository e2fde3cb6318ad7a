// Which kernels the expert products and the head's loss run on: muon_experts.cpp,
// muon_head.cpp and products_plan.cpp compiled for the host, with launchers that print
// the plan of every product instead of launching it.  Reads calls from stdin, one a line:
//   head NAME rows dim vocab f32 cap
//   experts NAME experts rows in out f32 in_out grad_w_f32
// and prints "NAME form epilogue shape f32 cut queued" for every product of the call and
// of its gradients.  Run by tests/test_training_cpu.py.
#include <cstdio>
#include <cstring>
#include <iostream>
#include <string>

#include "muon_experts.h"
#include "muon_head.h"
#include "op_workspace.h"
#include "products_internal.h"

static std::string g_name;
static size_t g_need = 0;

namespace muon {
muon_status api_fail(muon_status s, const char* text) noexcept {
  std::printf("FAIL %s: %s\n", g_name.c_str(), text);
  return s;
}
void api_clear_error() {}
hipError_t api_timed(int, hipStream_t, const std::function<hipError_t()>& launch) { return launch(); }
muon_status op_fail(muon_status s, const char* fmt, ...) { return api_fail(s, fmt); }
muon_status op_device(int* cus) {
  *cus = 256;
  return MUON_OK;
}
muon_status op_check_alias(const OpRange*, int) { return MUON_OK; }
muon_status op_run(size_t need, void*, uint64_t, hipStream_t, const std::function<hipError_t(char*, bool)>& launch) {
  g_need = need;
  return launch(reinterpret_cast<char*>(uintptr_t(1) << 40), true) == hipSuccess ? MUON_OK : MUON_ERR_HIP;
}
hipError_t launch_head_rows(const HeadRows&, hipStream_t) { return hipSuccess; }
hipError_t launch_head_finish(const HeadFinish&, hipStream_t) { return hipSuccess; }
hipError_t launch_product(int form, int epi, const ProductArgs& a, int cus, char* ws, hipStream_t) {
  const ProductPlan p = product_plan(form, epi, a, cus);
  const size_t at = reinterpret_cast<uintptr_t>(ws) - (uintptr_t(1) << 40);
  std::printf("%s %d %d %d %d %d %d%s\n", g_name.c_str(), form, product_epilogue(epi, a), p.shape, a.f32, p.bytes > p.queue ? 1 : 0,
              p.queue ? 1 : 0, p.bytes > 0 && at + p.bytes > g_need ? " OUTSIDE" : "");
  return hipSuccess;
}
}  // namespace muon

int main() {
  void* p[8];
  for (int i = 0; i < 8; ++i) p[i] = reinterpret_cast<void*>(uintptr_t(2 + i) << 42);
  const auto f = [&](int i) { return static_cast<float*>(p[i]); };
  std::string kind;
  while (std::cin >> kind >> g_name) {
    muon_status st = MUON_ERR_INVALID_ARGUMENT;
    if (kind == "head") {
      muon_head_desc d = {};
      int f32;
      std::cin >> d.rows >> d.dim >> d.vocab >> f32 >> d.softcap;
      d.ld_x = d.ld_w = d.ld_grad_x = d.ld_grad_w = d.dim;
      d.ignore_index = -100;
      d.dtype = f32 ? MUON_DTYPE_F32 : MUON_DTYPE_BF16;
      const auto* t = static_cast<const int64_t*>(p[2]);
      st = muon_head_loss(p[0], p[1], t, f(3), f(4), &d, nullptr, 0, nullptr);
      if (st == MUON_OK) st = muon_head_loss_vjp(p[0], p[1], t, f(3), f(4), nullptr, p[5], p[6], &d, nullptr, 0, nullptr);
    } else if (kind == "experts") {
      muon_experts_desc d = {};
      int f32, in_out, gw;
      std::cin >> d.experts >> d.rows >> d.in_dim >> d.out_dim >> f32 >> in_out >> gw;
      d.ld_x = d.ld_grad_x = d.in_dim;
      d.ld_y = d.out_dim;
      d.ld_w = d.ld_grad_w = in_out ? d.out_dim : d.in_dim;
      d.stride_w = d.stride_grad_w = d.in_dim * d.out_dim;
      d.w_order = in_out ? MUON_WEIGHT_IN_OUT : MUON_WEIGHT_OUT_IN;
      d.dtype = f32 ? MUON_DTYPE_F32 : MUON_DTYPE_BF16;
      d.grad_w_dtype = gw ? MUON_DTYPE_F32 : MUON_DTYPE_BF16;
      const auto* o = static_cast<const int32_t*>(p[2]);
      st = muon_experts_product(p[0], p[1], o, p[3], &d, nullptr, 0, nullptr);
      if (st == MUON_OK) st = muon_experts_product_vjp(p[0], p[1], o, p[3], p[4], p[5], &d, nullptr, 0, nullptr);
    }
    if (st != MUON_OK) return std::printf("FAIL %s\n", g_name.c_str()), 1;
  }
  return 0;
}
