// Argument checks shared by the entry points (internal to libmoe).
#pragma once
#include <hip/hip_runtime.h>

#include "../../include/moe.h"
#include "status.h"

namespace moe {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Device of a stream (NULL stream: the current device).
inline moe_status stream_device(hipStream_t s, int* dev) {
  hipError_t e = s ? hipStreamGetDevice(s, dev) : hipGetDevice(dev);
  if (e != hipSuccess) {
    (void)hipGetLastError();
    return fail(MOE_ERR_HIP, "cannot query the stream's device: %s", hipGetErrorString(e));
  }
  return MOE_OK;
}

// The pointer must be device (or managed) memory of device `dev` (the ordinal,
// not only the kind: arc PR #89, Stage 0).
inline moe_status check_dev(const void* p, int dev, const char* name) {
  if (!p) return MOE_OK;
  hipPointerAttribute_t a;
  hipError_t e = hipPointerGetAttributes(&a, p);
  if (e != hipSuccess) {
    (void)hipGetLastError();
    return fail(MOE_ERR_DEVICE, "%s is not HIP device memory", name);
  }
  if (a.type != hipMemoryTypeDevice && a.type != hipMemoryTypeManaged)
    return fail(MOE_ERR_DEVICE, "%s is not device memory (memory type %d)", name, (int)a.type);
  if (a.device != dev)
    return fail(MOE_ERR_DEVICE, "%s lives on device %d but the stream runs on device %d", name, a.device, dev);
  return MOE_OK;
}

struct DevCheck {
  int dev = 0;
  moe_status st = MOE_OK;
  void operator()(const void* p, const char* name) {
    if (st == MOE_OK) st = check_dev(p, dev, name);
  }
};

inline moe_status hip_fail(hipError_t e, const char* what) {
  (void)hipGetLastError();
  return fail(MOE_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

}  // namespace moe
