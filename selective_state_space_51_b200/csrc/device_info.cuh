// What the handle-free entry points need to know of a device, looked up once.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "../../include/ssm_scan.h"

namespace ssm {

inline bool aligned(const void *p, size_t a) {
  return (reinterpret_cast<uintptr_t>(p) % a) == 0;
}

// The multiprocessor count of a B200; SSM_ERR_ARCH on another architecture.
inline int device_sms(int device, int *sms) {
  constexpr int kMaxDevices = 64;
  static std::atomic<int> known[kMaxDevices];
  if (device < 0 || device >= kMaxDevices) return SSM_ERR_INVALID;
  int n = known[device].load(std::memory_order_relaxed);
  if (n == 0) {
    int count = 0, major = 0, minor = 0;
    if (cudaGetDeviceCount(&count) != cudaSuccess) {
      cudaGetLastError();
      return SSM_ERR_CUDA;
    }
    if (device >= count) return SSM_ERR_INVALID;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor,
                               device) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor,
                               device) != cudaSuccess ||
        cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, device) !=
            cudaSuccess) {
      cudaGetLastError();
      return SSM_ERR_CUDA;
    }
    if (major != 10 || minor != 0) return SSM_ERR_ARCH;
    known[device].store(n, std::memory_order_relaxed);
  }
  *sms = n;
  return SSM_OK;
}

// The same, and that the device is the current one of this thread.
inline int device_ready(int device, int *sms) {
  const int rc = device_sms(device, sms);
  if (rc != SSM_OK) return rc;
  int cur = -1;
  if (cudaGetDevice(&cur) != cudaSuccess) {
    cudaGetLastError();
    return SSM_ERR_CUDA;
  }
  return cur == device ? SSM_OK : SSM_ERR_INVALID;
}

}  // namespace ssm
