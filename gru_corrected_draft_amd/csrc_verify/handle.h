// Host helpers of the handles behind domino_verify.h.  Messages go to fixed
// buffers and nothing here throws, so no C++ exception reaches a C caller.
#pragma once
#include <hip/hip_runtime.h>
#include <stdarg.h>
#include <stdio.h>
#include <string.h>

#include "../../include/domino_rollout.h"

namespace {

struct HandleBase {
  int device = 0;
  void* alloc_[4] = {};
  int allocs = 0;
  char err[256] = "";

  void* take(size_t bytes) {
    void* p = nullptr;
    if (allocs == 4 || hipMalloc(&p, bytes < 256 ? 256 : bytes) != hipSuccess) {
      (void)hipGetLastError();
      return nullptr;
    }
    alloc_[allocs++] = p;
    return p;
  }
  void release() {
    for (int i = 0; i < allocs; ++i) (void)hipFree(alloc_[i]);
    allocs = 0;
  }
};

template <size_t N>
__attribute__((format(printf, 3, 4))) domino_status_t say(char (&err)[N], domino_status_t st,
                                                          const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(err, N, fmt, ap);
  va_end(ap);
  return st;
}

template <size_t N>
domino_status_t check_device(char (&err)[N], int* dev) {
  if (hipGetDevice(dev) != hipSuccess) {
    (void)hipGetLastError();
    return say(err, DOMINO_ERR_UNSUPPORTED, "create: no HIP device");
  }
  hipDeviceProp_t prop;
  if (hipGetDeviceProperties(&prop, *dev) != hipSuccess) {
    (void)hipGetLastError();
    return say(err, DOMINO_ERR_HIP, "create: hipGetDeviceProperties failed");
  }
  if (strncmp(prop.gcnArchName, "gfx950", 6) != 0)
    return say(err, DOMINO_ERR_UNSUPPORTED, "create: device is %s, the library runs on gfx950 only",
               prop.gcnArchName);
  return DOMINO_OK;
}

// makes the handle's device current for the life of the guard
struct DeviceGuard {
  int prev = -1, want;
  explicit DeviceGuard(int d) : want(d) {
    if (hipGetDevice(&prev) == hipSuccess && prev != want) (void)hipSetDevice(want);
  }
  ~DeviceGuard() {
    if (prev >= 0 && prev != want) (void)hipSetDevice(prev);
  }
};

}  // namespace
