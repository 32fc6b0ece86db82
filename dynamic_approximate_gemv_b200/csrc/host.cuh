// Host helpers shared by the files that implement the C ABI.
#pragma once
#include <cuda_runtime.h>

#include "../../include/effort.h"

namespace effort {

inline size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

// Device memory, counted against the library's cap (api.cu).
bool within_cap(size_t bytes);
effort_status_t dev_alloc(void** p, size_t bytes);
void dev_free(void* p, size_t bytes);

struct DevBuf {
  void* p = nullptr;
  size_t bytes = 0;
  effort_status_t alloc(size_t b) {
    bytes = b;
    return dev_alloc(&p, b);
  }
  void release() {
    dev_free(p, bytes);
    p = nullptr;
    bytes = 0;
  }
};

// Makes a device current for the length of a call.
struct DeviceGuard {
  int prev = -1;
  explicit DeviceGuard(int dev) {
    if (cudaGetDevice(&prev) == cudaSuccess && prev != dev) cudaSetDevice(dev);
    else prev = -1;
  }
  ~DeviceGuard() {
    if (prev >= 0) cudaSetDevice(prev);
  }
};

}  // namespace effort
