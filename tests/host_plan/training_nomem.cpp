// The C entries of the expert products and of the head's loss without host memory:
// operator new fails from a chosen allocation on, and no call may end in an
// exception.  Run by tests/test_training_cpu.py with the library's path.
#include <dlfcn.h>

#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <new>

#include "muon_experts.h"
#include "muon_head.h"

namespace {
long g_left = -1;  // allocations that still succeed; -1: all
}

void* operator new(size_t n) {
  if (g_left == 0) throw std::bad_alloc();
  if (g_left > 0) --g_left;
  if (void* p = std::malloc(n)) return p;
  throw std::bad_alloc();
}
void operator delete(void* p) noexcept { std::free(p); }
void operator delete(void* p, size_t) noexcept { std::free(p); }

int main(int argc, char** argv) {
  void* lib = argc > 1 ? dlopen(argv[1], RTLD_NOW) : nullptr;
  if (!lib) return std::printf("cannot load the library: %s\n", dlerror()), 2;
  const auto product = reinterpret_cast<decltype(&muon_experts_product)>(dlsym(lib, "muon_experts_product"));
  const auto vjp = reinterpret_cast<decltype(&muon_experts_product_vjp)>(dlsym(lib, "muon_experts_product_vjp"));
  const auto ebytes = reinterpret_cast<decltype(&muon_experts_workspace_bytes)>(dlsym(lib, "muon_experts_workspace_bytes"));
  const auto loss = reinterpret_cast<decltype(&muon_head_loss)>(dlsym(lib, "muon_head_loss"));
  const auto lvjp = reinterpret_cast<decltype(&muon_head_loss_vjp)>(dlsym(lib, "muon_head_loss_vjp"));
  const auto hbytes = reinterpret_cast<decltype(&muon_head_workspace_bytes)>(dlsym(lib, "muon_head_workspace_bytes"));
  muon_experts_desc e = {};
  e.experts = 2;
  e.rows = 10;
  e.in_dim = e.out_dim = e.ld_x = e.ld_y = e.ld_w = e.ld_grad_x = e.ld_grad_w = 16;
  e.stride_w = e.stride_grad_w = 256;
  muon_experts_desc ebad = e;
  ebad.rows = -1;
  muon_head_desc h = {};
  h.rows = 10;
  h.vocab = 20;
  h.dim = h.ld_x = h.ld_w = h.ld_grad_x = h.ld_grad_w = 16;
  muon_head_desc hbad = h;
  hbad.softcap = -1.f;
  // validation reads no element, and outputs overlap inputs: no call gets to a kernel
  char* a = reinterpret_cast<char*>(uintptr_t(1) << 40);
  float* f = reinterpret_cast<float*>(a);
  const auto* o = reinterpret_cast<const int32_t*>(a);
  const auto* t = reinterpret_cast<const int64_t*>(a);
  int thrown = 0, calls = 0;
  for (long n = 0; n < 6; ++n)
    for (int k = 0; k < 12; ++k) {
      const muon_experts_desc* ed = k % 2 ? &ebad : &e;
      const muon_head_desc* hd = k % 2 ? &hbad : &h;
      g_left = n;
      try {
        switch (k / 2) {
          case 0: product(a, a, o, a, ed, nullptr, 0, nullptr); break;
          case 1: vjp(a, a, o, a, a, a, ed, nullptr, 0, nullptr); break;
          case 2: ebytes(k % 2 ? 7 : 2, ed); break;
          case 3: loss(a, a, t, f, f, hd, nullptr, 0, nullptr); break;
          case 4: lvjp(a, a, t, f, f, f, a, a, hd, nullptr, 0, nullptr); break;
          case 5: hbytes(k % 2 ? 7 : 3, hd); break;
        }
      } catch (...) {
        g_left = -1;
        std::printf("call %d with %ld allocations threw\n", k, n);
        ++thrown;
      }
      g_left = -1;
      ++calls;
    }
  std::printf("%d calls, %d threw\n", calls, thrown);
  return thrown ? 1 : 0;
}
