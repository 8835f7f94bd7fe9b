// Host-side checks shared by the C-ABI entry points: the current device, where
// a pointer lives, alignment, and small integer helpers.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>
#include <string.h>

#include <atomic>
#include <mutex>

#include "../../include/mxgemm.h"

namespace mxg {
namespace host {

constexpr int kMaxDevices = 64;

struct DeviceInfo {
  std::atomic<int> checked{0};  // 0 unknown, 1 gfx950, -1 other; set after cus
  int cus = 0;
};

inline DeviceInfo g_dev[kMaxDevices];
inline std::mutex g_dev_mutex;

inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

inline bool fits_i32(int64_t v) { return v >= 0 && v <= 0x7FFFFFFFLL; }

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned_to(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// Takes MXG_TRUSTED_POINTERS out of a call's flags.
inline bool take_trust(unsigned* flags) {
  const bool trusted = (*flags & MXG_TRUSTED_POINTERS) != 0;
  *flags &= ~(unsigned)MXG_TRUSTED_POINTERS;
  return trusted;
}

// launch(first, count) for `blocks` workgroups in runs of 2^22 at most, for kernels of up to 512 threads.  A launch has
// fewer than 2^32 work items in a dimension; one of more is not refused but runs the remainder by 2^32 alone.  (Two
// dimensions in place of runs cost every call of the quantiser 0.2 to 0.4 us.)
template <class F>
inline void launch_runs(int64_t blocks, F launch) {
  constexpr int64_t kRun = 1 << 22;
  for (int64_t first = 0; first < blocks; first += kRun) launch(first, (unsigned)(blocks - first < kRun ? blocks - first : kRun));
}

// Current device must be gfx950; returns its CU count through *cus.
inline int device_check(int* dev_out, int* cus) {
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) return MXG_ERR_DEVICE;
  DeviceInfo& d = g_dev[dev];
  if (d.checked == 0) {
    std::lock_guard<std::mutex> lock(g_dev_mutex);
    if (d.checked == 0) {
      hipDeviceProp_t prop;
      if (hipGetDeviceProperties(&prop, dev) != hipSuccess) return MXG_ERR_DEVICE;
      d.cus = prop.multiProcessorCount;
      d.checked = strncmp(prop.gcnArchName, "gfx950", 6) == 0 ? 1 : -1;
    }
  }
  if (d.checked != 1) return MXG_ERR_DEVICE;
  *dev_out = dev;
  *cus = d.cus;
  return MXG_OK;
}

// Device memory of `dev` (or managed memory) is accepted; host memory is not.
inline bool on_device(const void* p, int dev) {
  hipPointerAttribute_t attr;
  if (hipPointerGetAttributes(&attr, p) != hipSuccess) {
    (void)hipGetLastError();
    return false;
  }
  if (attr.type != hipMemoryTypeDevice && attr.type != hipMemoryTypeManaged) return false;
  return attr.device == dev;
}

}  // namespace host
}  // namespace mxg
