// Host-side helpers shared by every translation unit of libpagedkv: the
// status and error text of the C ABI, the launch count, and device queries.
#pragma once

#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdarg>
#include <cstdint>

#include "pagedkv.h"

namespace pagedkv {

// Record a thread-local description of a failure and return its status.
pa_status fail(pa_status s, const char* fmt, ...)
    __attribute__((format(printf, 2, 3)));

// Count one kernel launch issued by the library.
void count_launch();

// Clear the thread-local description (called on entry of each API call).
void clear_error();

// SM count of the current device, looked up once per device ordinal (the
// launch paths ask on every call).
int device_sm_count();

// The driver's cuTensorMapEncodeTiled, or nullptr if it is unavailable.
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();

// Which devices a kernel's attributes were set on: a static one of these
// beside a launch spares the runtime calls on every later one.
struct OncePerDevice {
  std::atomic<uint64_t> mask{0};
  // True if not yet marked for the current device.
  bool needed() const {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return true;
    return !(mask.load(std::memory_order_acquire) >> dev & 1u);
  }
  void mark() {
    int dev = 0;
    if (cudaGetDevice(&dev) == cudaSuccess && dev >= 0 && dev < 64)
      mask.fetch_or(uint64_t(1) << dev, std::memory_order_release);
  }
};

// Address at which the current device reaches `p`: device memory of this
// device, or mapped page-locked host memory.  nullptr for anything else
// (pageable host memory, another device's memory).
void* device_view(const void* p);

inline bool aligned16(const void* p) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0;
}

}  // namespace pagedkv
