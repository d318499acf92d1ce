// Host helpers of the C entry points that live outside api.cpp: error text,
// argument checks and device allocations, with the behaviour of api.cpp's own.
#pragma once

#include <cstdarg>
#include <cstddef>
#include <cstdint>
#include <cstdio>

#include <cuda_runtime.h>

#include "ling_moe.h"

namespace lingmoe {

void set_last_error(const char* msg);  // api.cpp: the calling thread's message

inline int fail_arg(int code, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  set_last_error(buf);
  return code;
}
inline int fail_cuda(cudaError_t e, const char* what) {
  return fail_arg(e == cudaErrorMemoryAllocation ? LING_MOE_ERR_OOM : LING_MOE_ERR_CUDA, "%s: %s (%s)", what,
                  cudaGetErrorName(e), cudaGetErrorString(e));
}
inline bool is_aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline bool ranges_overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
  return a0 < b0 + nb && b0 < a0 + na;
}
// The current device's ordinal and SM count; LING_MOE_ERR_UNSUPPORTED unless it is an sm_100 GPU.
inline int check_device(int* dev, int* sms) {
  cudaError_t e = cudaGetDevice(dev);
  if (e != cudaSuccess) return fail_cuda(e, "cudaGetDevice");
  int major = 0;
  e = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, *dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, *dev);
  if (e != cudaSuccess) return fail_cuda(e, "cudaDeviceGetAttribute");
  if (major != 10) return fail_arg(LING_MOE_ERR_UNSUPPORTED, "needs an sm_100 GPU (got sm_%d)", major * 10);
  return LING_MOE_OK;
}
// A handle's calls belong to the device that was current when it was created.
inline int check_same_device(int device) {
  int dev = -1;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return fail_cuda(e, "cudaGetDevice");
  if (dev != device)
    return fail_arg(LING_MOE_ERR_INVALID_ARG, "the handle belongs to device %d, the current device is %d", device, dev);
  return LING_MOE_OK;
}

}  // namespace lingmoe
