// The workspace that the expert products and the head's loss share on a device,
// and the way from an entry point to its launches.  Not part of the ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <cstdarg>
#include <functional>
#include <new>

#include "api_internal.h"

namespace muon {

// Sets the thread's last error from a format.
muon_status op_fail(muon_status s, const char* fmt, ...);

// Compute units of the current device (0 and an error where there is none).
muon_status op_device(int* cus);

// Runs `launch` on `need` bytes: the caller's workspace, or the device's own, behind
// the device's previous call that used it.  need = 0: neither.
muon_status op_run(size_t need, void* ws, uint64_t ws_bytes, hipStream_t stream,
                   const std::function<hipError_t(char* ws, bool capturing)>& launch);

// Address ranges [lo, hi) of a call's tensors.
struct OpRange {
  uintptr_t lo, hi;
  bool written;
  const char* what;
};
// ALIAS where a written range meets another.
muon_status op_check_alias(const OpRange* r, int n);

// Nothing crosses the ABI as an exception.
template <class F>
muon_status op_guarded(F&& f) {
  api_clear_error();
  try {
    return f();
  } catch (const std::bad_alloc&) {
    return api_fail(MUON_ERR_OUT_OF_MEMORY, "host memory allocation failed");
  } catch (...) {
    return api_fail(MUON_ERR_HIP, "unexpected failure on the host");
  }
}

inline size_t op_align256(size_t v) { return (v + 255) & ~size_t(255); }

}  // namespace muon
