// The block operators' C entries without host memory: operator new fails from a
// chosen allocation on, and no call may end in an exception.  Run by
// tests/test_blocks_cpu.py with the library's path.
#include <dlfcn.h>

#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <new>

#include "muon_blocks.h"

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
  const auto ns = reinterpret_cast<decltype(&muon_ns_blocks)>(dlsym(lib, "muon_ns_blocks"));
  const auto vjp = reinterpret_cast<decltype(&muon_ns_blocks_vjp)>(dlsym(lib, "muon_ns_blocks_vjp"));
  const auto step = reinterpret_cast<decltype(&muon_step_blocks)>(dlsym(lib, "muon_step_blocks"));
  const auto bytes = reinterpret_cast<decltype(&muon_blocks_workspace_bytes)>(dlsym(lib, "muon_blocks_workspace_bytes"));
  const muon_ns_coeffs co = {1.5f, -0.5f, 0.f};
  muon_block_desc bad = {4, 200, 200, 200, 200, 200, 40000, 40000, 40000, 0, 0, 0, 0};  // min(rows, cols) > 128
  muon_block_desc good = {4, 20, 200, 200, 200, 200, 4000, 4000, 4000, 0, 0, 0, 0};
  void* a = reinterpret_cast<void*>(uintptr_t(1) << 40);  // validation reads no element, and its output overlaps its input
  muon_step_hparams hp = {};
  hp.lr = 0.02f;
  hp.ns_coeffs = co;
  hp.ns_steps = 3;
  int thrown = 0, calls = 0;
  for (long n = 0; n < 6; ++n)
    for (int k = 0; k < 9; ++k) {
      const void* x[1] = {a};
      void* y[1] = {a};
      const muon_block_desc* d = k % 2 ? &bad : &good;
      g_left = n;
      try {
        switch (k) {
          case 0: case 1: ns(x, y, d, 1, co, 3, nullptr, nullptr, 0, nullptr); break;
          case 2: case 3: vjp(x, x, y, d, 1, co, 3, nullptr, nullptr, 0, nullptr); break;
          case 4: case 5: step(y, x, y, d, 1, &hp, nullptr, nullptr, 0, nullptr); break;
          case 6: bytes(17, d, 1, co, 3, nullptr); break;
          case 7: bytes(MUON_BLOCKS_NS, d, 1, co, 3, nullptr); break;
          case 8: bytes(MUON_BLOCKS_NS, nullptr, 1, co, 3, nullptr); break;
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
