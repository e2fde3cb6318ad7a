// What muon_api.cpp shares with the other host files of the library: the
// thread-local error, the lock of the per-device state, the allocation fault
// hook, the timing hook and the release hook.  Not part of the ABI.
#pragma once

#include <hip/hip_runtime.h>

#include <functional>
#include <mutex>

#include "muon.h"

namespace muon {

// Sets the calling thread's last error (none if there is no memory for the
// text) and returns `s`.
muon_status api_fail(muon_status s, const char* text) noexcept;
void api_clear_error();
std::mutex& api_mutex();
// hipMalloc behind MUON_FAULT_ALLOC.
hipError_t api_device_alloc(void** p, size_t bytes);
// Runs `launch` as kernel class `kc` of muon_timing_read (lock held).
hipError_t api_timed(int kc, hipStream_t stream, const std::function<hipError_t()>& launch);
// Whether launches are being timed (lock held).
bool api_timing();
// Called by muon_release_workspace with the lock held; null if unused.  A file
// that sets it calls what it held before.
extern void (*api_release_hook)();

}  // namespace muon
