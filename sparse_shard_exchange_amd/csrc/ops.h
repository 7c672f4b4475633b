// Host checks shared by the plan-less operators (balance.hip, moe_grad.hip,
// norm.hip): they take a descriptor, buffers, a workspace and a stream.
#pragma once

#include <math.h>

#include "device.h"
#include "runtime.h"

namespace pw {

inline size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }

// The caller's workspace holds `need` bytes (need 0: none is looked at).
inline int check_workspace(const void* ws, size_t ws_bytes, size_t need) {
  if (need == 0) return PW_OK;
  if (!ws) return fail(PW_ERR_INVALID, "this call needs a workspace of %zu bytes", need);
  if ((uintptr_t)ws % 256) return fail(PW_ERR_INVALID, "the workspace must be 256-byte aligned");
  if (ws_bytes < need) return fail(PW_ERR_NOMEM, "workspace of %zu bytes, %zu needed", ws_bytes, need);
  return PW_OK;
}

// The stream belongs to the current device (kernels are launched there).
inline int check_stream(hipStream_t s) {
  int cur = -1;
  hipError_t e = hipGetDevice(&cur);
  if (e != hipSuccess) return hip_fail(e, "hipGetDevice");
  if (!s) return PW_OK;
  hipDevice_t dev = cur;
  e = hipStreamGetDevice(s, &dev);
  if (e != hipSuccess) return hip_fail(e, "hipStreamGetDevice");
  if (dev != cur) return fail(PW_ERR_STATE, "the stream is on device %d, the current device is %d", dev, cur);
  return PW_OK;
}

}  // namespace pw
