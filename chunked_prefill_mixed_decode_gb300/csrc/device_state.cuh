// Per-device host state (devices 0 .. kMaxDevices - 1), kept by the translation
// unit that launches: which of its kernels have had their shared-memory limit
// raised.  Safe to use from several host threads: every entry is computed the
// same way by whoever gets there first.
#pragma once

#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "mixed_step.h"

namespace {

constexpr int kMaxDevices = 64;
std::atomic<uint32_t> g_smem_attr_set[kMaxDevices];

inline int current_device() {
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return -1;
  return dev;
}

// Raise `kernel`'s dynamic shared-memory limit on the current device once (bit
// `slot` of the device's mask), to the most that any of its launches uses: a
// launch may then ask for less, and no call changes the limit under another.
template <typename Kernel>
int ensure_smem_limit(Kernel kernel, int slot, int bytes) {
  const int dev = current_device();
  if (dev < 0) return MS_ERR_CUDA;
  if (g_smem_attr_set[dev].load(std::memory_order_acquire) & (1u << slot)) return MS_OK;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess)
    return MS_ERR_CUDA;
  g_smem_attr_set[dev].fetch_or(1u << slot, std::memory_order_release);
  return MS_OK;
}

}  // namespace
