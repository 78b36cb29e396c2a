// What the handle-free entry points need to know of a device, looked up once.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>
#include <initializer_list>

#include "../../include/ssm_scan.h"

namespace ssm {

inline bool aligned(const void *p, size_t a) {
  return (reinterpret_cast<uintptr_t>(p) % a) == 0;
}

// Device memory from `at` on (nullptr: none).
struct Span {
  const void *at;
  size_t bytes;
};

// Whether something of `writes` shares memory with another entry of it or with
// one of `reads` (`same`: but for reads that start where the write does, for
// calls that read each element before they write it).
inline bool clash(std::initializer_list<Span> writes,
                  std::initializer_list<Span> reads, bool same = false) {
  auto meet = [](const Span &a, const Span &b) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.at),
                    y = reinterpret_cast<uintptr_t>(b.at);
    return x && y && x < y + b.bytes && y < x + a.bytes;
  };
  for (const Span *w = writes.begin(); w != writes.end(); ++w) {
    for (const Span *o = w + 1; o != writes.end(); ++o)
      if (meet(*w, *o)) return true;
    for (const Span &r : reads)
      if (meet(*w, r) && !(same && w->at == r.at)) return true;
  }
  return false;
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
