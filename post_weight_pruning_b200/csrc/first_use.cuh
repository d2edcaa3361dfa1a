// Per-device settings of kernels, made at a kernel's first use (host code only).
#pragma once

#include <cuda_runtime_api.h>

#include <atomic>

namespace pwp {

// Runs `set` (a callable that returns cudaError_t) unless a call for the current device with
// this flag word has returned cudaSuccess.  Kernel attributes (dynamic shared memory limits)
// are per device, so each device of a multi-GPU process sets them once; devices past 63 set
// them at every call.  The flag follows the setting: whoever finds it raised may launch, two
// threads that come first together both set (the attributes are the same), and a setting that
// failed is made again by the next call.
template <typename F>
cudaError_t on_first_use(std::atomic<unsigned long long>& done, F set) {
  int dev = 0;
  const cudaError_t at = cudaGetDevice(&dev);
  if (at != cudaSuccess) return at;
  const unsigned long long bit = dev >= 0 && dev < 64 ? 1ull << dev : 0;
  if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  const cudaError_t e = set();
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

}  // namespace pwp
