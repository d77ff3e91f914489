// What the C entry points of several translation units share: the per-device
// state behind the status word and the tensor-map encoder, and the check of
// device pointers (defined in fa_api.cu).
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>
#include <mutex>

#include "fa.h"

namespace fa {

struct HostDevice {
  int dev;               // the current device
  int sms;               // its SM count
  unsigned int* status;  // its status words {code, site, index}
};

// Looks the current device up (first call: the one-time set-up described at
// the top of fa.h).  FA_OK, FA_ERR_CUDA or FA_ERR_UNSUPPORTED.
int host_device(HostDevice* out);

// Device pointer on `dev` (or managed memory)?
bool host_is_device_ptr(const void* p, int dev);

// Tensor map of bytes (e4m3 codes): rank dims, strides in bytes of dims 1..,
// box, shared-memory swizzle of 128 or 64 bytes.  After host_device().
int host_encode_bytes(CUtensorMap* m, const void* base, int rank, const uint64_t* dims, const uint64_t* strides,
                      const uint32_t* box, int swizzle);

// Lets `kernel` use `smem` bytes of dynamic shared memory, once a device.
inline int allow_smem(const void* kernel, int smem, bool (&ready)[64]) {
  static std::mutex mutex;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return FA_ERR_CUDA;
  std::lock_guard<std::mutex> lock(mutex);
  if (!ready[dev]) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
      return FA_ERR_CUDA;
    ready[dev] = true;
  }
  return FA_OK;
}

}  // namespace fa
