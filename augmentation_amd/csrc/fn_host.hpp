// fn_host.hpp -- what every entry point of libfn.so does on the host: the
// thread's error message, the checks of device pointers, cached device
// properties and the status of a launch.
#pragma once
#include <hip/hip_runtime.h>

#include <atomic>
#include <cstdarg>
#include <cstdint>
#include <cstdio>

#include "fn.h"

#define FN_EXPORT extern "C" __attribute__((visibility("default")))

namespace fnhost {

// the last error message of this thread: a fixed buffer, so that recording
// an error never allocates (and nothing can throw across the C ABI)
inline thread_local char g_last_error[512];

inline int fail(int code, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_last_error, sizeof(g_last_error), fmt, ap);
  va_end(ap);
  return code;
}

inline int ok() {
  g_last_error[0] = '\0';
  return FN_OK;
}

inline bool in_unit(float p) { return p >= 0.0f && p <= 1.0f; }  // false for NaN

// The calling thread's current device.
inline int current_device(int* dev) {
  if (hipGetDevice(dev) != hipSuccess) {
    (void)hipGetLastError();
    return fail(FN_EHIP, "hipGetDevice failed");
  }
  return FN_OK;
}

// The buffer [p, p + bytes) must be device memory of the current device,
// inside one allocation.  *dev caches the current device across the checks
// of one call (-1: not queried yet).  Failed queries leave no sticky HIP
// error behind.
inline int check_device_range(const void* p, size_t bytes, const char* name, int* dev) {
  if (p == nullptr) return fail(FN_EINVAL, "%s is NULL", name);
  if (*dev < 0) {
    const int rc = current_device(dev);
    if (rc) return rc;
  }
  hipPointerAttribute_t attr;
  hipError_t e = hipPointerGetAttributes(&attr, p);
  if (e != hipSuccess) {
    (void)hipGetLastError();
    return fail(FN_EINVAL, "%s is not device memory (%s)", name, hipGetErrorString(e));
  }
  if (attr.type != hipMemoryTypeDevice)
    return fail(FN_EINVAL, "%s is not device memory (memory type %d)", name, (int)attr.type);
  if (attr.device != *dev)
    return fail(FN_EINVAL, "%s lives on device %d, the current device is %d", name, attr.device,
                *dev);
  hipDeviceptr_t base = nullptr;
  size_t size = 0;
  e = hipMemGetAddressRange(&base, &size, (hipDeviceptr_t)p);
  if (e != hipSuccess) {
    (void)hipGetLastError();
    return fail(FN_EINVAL, "%s: cannot determine its allocation (%s)", name, hipGetErrorString(e));
  }
  const uintptr_t lo = (uintptr_t)base, hi = lo + size, b = (uintptr_t)p;
  if (b < lo || bytes > hi - b)
    return fail(FN_EINVAL, "%s: %zu bytes needed, %zu available in its allocation", name, bytes,
                (size_t)(hi - b));
  return FN_OK;
}

inline int launch_status(const char* what) {
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return fail(FN_EHIP, "%s: %s", what, hipGetErrorString(e));
  return ok();
}

// HIP starts fewer than 2^32 threads along a dimension of a launch.  More are
// refused, or silently taken modulo 2^32.
constexpr int64_t kMaxThreads = 0xFFFFFFFF;

inline unsigned blocks_for(int64_t items, int64_t per_block) {
  return (unsigned)((items + per_block - 1) / per_block);
}

// Compute units of device `dev`, queried once per device.
inline int device_cu_count(int dev, int* cus) {
  static std::atomic<int> cache[64];
  if (dev >= 0 && dev < 64 && cache[dev].load(std::memory_order_relaxed) > 0) {
    *cus = cache[dev].load(std::memory_order_relaxed);
    return FN_OK;
  }
  int v = 0;
  const hipError_t e = hipDeviceGetAttribute(&v, hipDeviceAttributeMultiprocessorCount, dev);
  if (e != hipSuccess || v <= 0) {
    (void)hipGetLastError();
    return fail(FN_EHIP, "cannot query the compute unit count: %s", hipGetErrorString(e));
  }
  if (dev >= 0 && dev < 64) cache[dev].store(v, std::memory_order_relaxed);
  *cus = v;
  return FN_OK;
}

}  // namespace fnhost
