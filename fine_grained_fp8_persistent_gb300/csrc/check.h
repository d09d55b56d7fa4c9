// check.h -- host-side checks shared by the ABI's translation units.
#pragma once
#include <cstdint>
#include <initializer_list>

#include <cuda_runtime.h>

#include "../../include/fgf8.h"
#include "fgf8_internal.h"

namespace fgf8 {

// Every tensor pointer is 16-byte aligned device (or managed) memory of the current
// device, checked before anything is launched.
inline int check_pointers(const char* who, std::initializer_list<const void*> ptrs) {
  for (const void* p : ptrs) {
    if (p == nullptr) return set_error(FGF8_ERR_INVALID_ARG, "%s: null pointer", who);
    if ((reinterpret_cast<uintptr_t>(p) & 15u) != 0)
      return set_error(FGF8_ERR_MISALIGNED, "%s: pointers must be 16-byte aligned", who);
  }
  int dev = 0;
  const cudaError_t ed = cudaGetDevice(&dev);
  if (ed != cudaSuccess) return set_error(FGF8_ERR_CUDA, "cudaGetDevice: %s", cudaGetErrorString(ed));
  int i = 0;
  for (const void* p : ptrs) {
    cudaPointerAttributes at;
    const cudaError_t e = cudaPointerGetAttributes(&at, p);
    if (e != cudaSuccess) {
      cudaGetLastError();  // the failed query also sets the runtime's last error; clear it
      return set_error(FGF8_ERR_INVALID_ARG, "%s: pointer %d: %s", who, i, cudaGetErrorString(e));
    }
    if (at.type != cudaMemoryTypeDevice && at.type != cudaMemoryTypeManaged)
      return set_error(FGF8_ERR_INVALID_ARG, "%s: pointer %d is not device memory", who, i);
    if (at.type == cudaMemoryTypeDevice && at.device != dev)
      return set_error(FGF8_ERR_INVALID_ARG, "%s: pointer %d is on device %d, the current device is %d", who, i,
                       at.device, dev);
    ++i;
  }
  return FGF8_OK;
}

}  // namespace fgf8
