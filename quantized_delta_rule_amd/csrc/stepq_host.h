// stepq_host.h -- what the host entry points share beside the kernels' interface.  Not part of the public
// ABI, and not one of the decode kernels' sources.
#pragma once
#include <hip/hip_runtime.h>

namespace stepq {

// Makes a device current and restores the caller's on scope exit; when it is already
// current (the usual case) no device switch is made either way.
struct DeviceGuard {
  int prev = -1;
  bool ok_ = false;
  explicit DeviceGuard(int dev) {
    if (hipGetDevice(&prev) != hipSuccess) {
      prev = -1;
      return;
    }
    if (prev == dev) {
      prev = -1;
      ok_ = true;
      return;
    }
    if (hipSetDevice(dev) == hipSuccess) ok_ = true;
  }
  ~DeviceGuard() {
    if (prev >= 0) (void)hipSetDevice(prev);
  }
};

}  // namespace stepq
