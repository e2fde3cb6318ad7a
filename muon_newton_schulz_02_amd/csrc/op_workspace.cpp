#include "op_workspace.h"

#include <cstdio>
#include <map>

namespace muon {
namespace {

struct OpDevice {
  int cus = 0;
  void* ws = nullptr;
  size_t bytes = 0;
  hipEvent_t last = nullptr;   // after the last call that used ws
  bool recorded = false;
};
std::map<int, OpDevice> g_devices;       // under api_mutex()
void (*g_next_release)() = nullptr;

void release_ops() {
  for (auto& kv : g_devices) {
    if (hipSetDevice(kv.first) != hipSuccess) continue;
    (void)hipDeviceSynchronize();
    if (kv.second.ws) (void)hipFree(kv.second.ws);
    if (kv.second.last) (void)hipEventDestroy(kv.second.last);
  }
  g_devices.clear();
  if (g_next_release) g_next_release();
}
struct HookRelease {
  HookRelease() {
    g_next_release = api_release_hook;
    api_release_hook = release_ops;
  }
} g_hook_release;

muon_status current(OpDevice** out) {
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess) {
    (void)hipGetLastError();
    return op_fail(MUON_ERR_HIP, "hipGetDevice failed (no HIP device?)");
  }
  OpDevice& d = g_devices[dev];
  if (d.cus == 0) {
    int cus = 0;
    if (hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || cus <= 0) {
      (void)hipGetLastError();
      return op_fail(MUON_ERR_HIP, "cannot query the compute-unit count of device %d", dev);
    }
    d.cus = cus;
  }
  *out = &d;
  return MUON_OK;
}

}  // namespace

muon_status op_fail(muon_status s, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  return api_fail(s, buf);
}

muon_status op_device(int* cus) {
  std::lock_guard<std::mutex> lock(api_mutex());
  OpDevice* d = nullptr;
  const muon_status st = current(&d);
  if (st == MUON_OK) *cus = d->cus;
  return st;
}

muon_status op_check_alias(const OpRange* r, int n) {
  for (int i = 0; i < n; ++i)
    for (int j = i + 1; j < n; ++j)
      if ((r[i].written || r[j].written) && r[i].lo < r[j].hi && r[j].lo < r[i].hi)
        return op_fail(MUON_ERR_ALIAS, "%s overlaps %s", r[i].what, r[j].what);
  return MUON_OK;
}

muon_status op_run(size_t need, void* ws, uint64_t ws_bytes, hipStream_t stream,
                   const std::function<hipError_t(char* ws, bool capturing)>& launch) {
  std::lock_guard<std::mutex> lock(api_mutex());
  OpDevice* d = nullptr;
  const muon_status st = current(&d);
  if (st != MUON_OK) return st;
  hipStreamCaptureStatus cap = hipStreamCaptureStatusNone;
  if (hipStreamIsCapturing(stream, &cap) != hipSuccess) {
    // the null stream while another stream captures
    (void)hipGetLastError();
    return op_fail(MUON_ERR_HIP, "the stream cannot be used during another stream's capture");
  }
  const bool capturing = cap != hipStreamCaptureStatusNone;
  char* at = reinterpret_cast<char*>(ws);
  const bool shared = need > 0 && !ws;
  if (ws && ws_bytes < need)
    return op_fail(MUON_ERR_INVALID_ARGUMENT, "the workspace holds %llu bytes; this call needs %zu",
                   (unsigned long long)ws_bytes, need);
  if (shared) {
    if (capturing)
      return op_fail(MUON_ERR_UNSUPPORTED, "a captured call needs a workspace of the caller's (%zu bytes)", need);
    if (need > d->bytes) {
      if (hipDeviceSynchronize() != hipSuccess)
        return op_fail(MUON_ERR_HIP, "hipDeviceSynchronize failed: %s", hipGetErrorString(hipGetLastError()));
      if (d->ws) (void)hipFree(d->ws);
      d->ws = nullptr;
      d->bytes = 0;
      void* p = nullptr;
      if (api_device_alloc(&p, need) != hipSuccess) {
        (void)hipGetLastError();
        return op_fail(MUON_ERR_OUT_OF_MEMORY, "workspace allocation of %zu bytes failed", need);
      }
      d->ws = p;
      d->bytes = need;
    }
    if (!d->last && hipEventCreateWithFlags(&d->last, hipEventDisableTiming) != hipSuccess) {
      d->last = nullptr;
      return op_fail(MUON_ERR_HIP, "hipEventCreate failed: %s", hipGetErrorString(hipGetLastError()));
    }
    if (d->recorded && hipStreamWaitEvent(stream, d->last, 0) != hipSuccess)
      return op_fail(MUON_ERR_HIP, "ordering after the device's previous call failed: %s",
                     hipGetErrorString(hipGetLastError()));
    at = reinterpret_cast<char*>(d->ws);
  }
  // an error that an earlier call of the thread's left would be taken for one of
  // the first launch, whose kernel runs all the same
  (void)hipGetLastError();
  const hipError_t e = launch(at, capturing);
  if (shared && hipEventRecord(d->last, stream) == hipSuccess) d->recorded = true;
  if (e != hipSuccess) return op_fail(MUON_ERR_HIP, "kernel launch failed: %s", hipGetErrorString(e));
  return MUON_OK;
}

}  // namespace muon
