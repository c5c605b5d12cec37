// per_device.h -- what a launch needs to know or set once for each device:
// kept by device, and only once it has succeeded (a failure, say in a first
// call during a stream capture, is tried again by the next).
#pragma once

#include <atomic>
#include <cstdint>
#include <cuda_runtime.h>

namespace qgemv {

constexpr int kMaxDevices = 64;

// The current device and its number of SMs.
inline cudaError_t current_device(int* dev, int* sms) {
  static std::atomic<int> known[kMaxDevices];
  cudaError_t e = cudaGetDevice(dev);
  if (e == cudaSuccess && (*dev < 0 || *dev >= kMaxDevices)) e = cudaErrorInvalidDevice;
  if (e != cudaSuccess) return e;
  *sms = known[*dev].load(std::memory_order_relaxed);
  if (*sms > 0) return cudaSuccess;
  e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, *dev);
  if (e == cudaSuccess && *sms <= 0) e = cudaErrorInvalidDevice;
  if (e == cudaSuccess) known[*dev].store(*sms, std::memory_order_relaxed);
  else cudaGetLastError();
  return e;
}

// A kernel's limit of dynamic shared memory on device `dev`, which must be the
// current one (set twice by two threads does no harm).
template <typename K>
cudaError_t allow_shared_memory(std::atomic<uint64_t>& done, int dev, K* kernel, int bytes) {
  const uint64_t bit = uint64_t(1) << dev;
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  else cudaGetLastError();
  return e;
}

}  // namespace qgemv
