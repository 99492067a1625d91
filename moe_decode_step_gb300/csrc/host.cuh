// What the C entry points beside the layer share: the device's properties, how
// a call begins and ends.
#pragma once

#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdint>

#include "moe_decode.h"

namespace moe_internal {
int cuda_fail(cudaError_t e);
}

namespace moe {

using moe_internal::cuda_fail;

constexpr int kMaxDevices = 64;

struct Device {
  std::atomic<bool> known{false};   // set after the others
  std::atomic<bool> sm103{false};
  std::atomic<int> n_sm{0};
};

// The current device's properties, asked for once per device: a host-side
// query whose answer cannot change.
inline int this_device(const Device** out) {
  static Device devices[kMaxDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e);
  if (dev < 0 || dev >= kMaxDevices) return MOE_ERR_UNSUPPORTED;
  Device& d = devices[dev];
  if (!d.known.load(std::memory_order_acquire)) {
    int major = 0, minor = 0, n_sm = 0;
    if ((e = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev)) ||
        (e = cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev)) ||
        (e = cudaDeviceGetAttribute(&n_sm, cudaDevAttrMultiProcessorCount, dev)))
      return cuda_fail(e);
    // threads whose first calls meet store the same values
    d.sm103.store(major == 10 && minor == 3, std::memory_order_relaxed);
    d.n_sm.store(n_sm, std::memory_order_relaxed);
    d.known.store(true, std::memory_order_release);
  }
  *out = &d;
  return d.sm103 ? MOE_OK : MOE_ERR_UNSUPPORTED;
}

// What every call starts with: an error left pending by earlier work is
// reported as it is, not blamed on this call's launches.
inline int begin(const Device** dev) {
  const cudaError_t e = cudaPeekAtLastError();
  if (e != cudaSuccess) return cuda_fail(e);
  return this_device(dev);
}

inline int end() {
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? MOE_OK : cuda_fail(e);
}

inline bool misaligned(const void* p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) != 0; }

}  // namespace moe
