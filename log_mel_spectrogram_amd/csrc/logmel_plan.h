// A plan and what every entry point of the C-ABI layer does around a call.
#pragma once
#include <hip/hip_runtime_api.h>

#include <cstdlib>

#include "logmel.h"

struct logmel_plan {
  logmel_config cfg;
  double* tables = nullptr;  // device, kTabBytes
  int resident_waves = 0;    // wavefronts of the transform kernel resident at once: one per SIMD
};

namespace {

struct DeviceGuard {
  int prev = -1;
  bool ok = true;
  explicit DeviceGuard(int dev) {
    if (hipGetDevice(&prev) != hipSuccess) { ok = false; return; }
    if (prev != dev && hipSetDevice(dev) != hipSuccess) ok = false;
  }
  ~DeviceGuard() {
    int cur = -1;
    if (prev >= 0 && hipGetDevice(&cur) == hipSuccess && cur != prev) (void)hipSetDevice(prev);
  }
};

bool env_validate() {
  const char* v = std::getenv("LOGMEL_VALIDATE");
  return v && v[0] && v[0] != '0';
}

}  // namespace
