// What the plan-less operators share (balance.hip, moe_grad.hip, norm.hip): sums
// and maxima over lanes, and the host checks of buffers, workspace and stream.
#pragma once

#include <math.h>

#include <initializer_list>

#include "device.h"
#include "runtime.h"

namespace pw {

// The value of the lane that differs in bit M of its number, once the lanes
// below have been joined (all lanes of an aligned group of M agree): quad
// permutes and row mirrors inside 16 lanes, an LDS exchange beyond. All lanes of
// the aligned group of 2 M are active.
template <int M>
__device__ __forceinline__ float across(float v) {
  if constexpr (M >= 16) return __shfl_xor(v, M);
  constexpr int ctrl = M == 1 ? 0xB1 : M == 2 ? 0x4E : M == 4 ? 0x141 : 0x140;
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), ctrl, 0xf, 0xf, true));
}

// Sum over each aligned group of L lanes; every lane gets it.
template <int L, int M = 1>
__device__ __forceinline__ float lanes_sum(float v) {
  if constexpr (M < L) return lanes_sum<L, 2 * M>(v + across<M>(v));
  return v;
}
template <int L, int M = 1>
__device__ __forceinline__ float lanes_max(float v) {
  if constexpr (M < L) return lanes_max<L, 2 * M>(fmaxf(v, across<M>(v)));
  return v;
}

// Workgroups of a launch at most: a dimension of the grid holds fewer than 2^32
// threads, of workgroups of up to 1024. Kernels that are launched with one
// workgroup for each piece of work walk on from there in steps of the grid.
constexpr uint32_t kMaxGrid = 1u << 21;

inline size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }

// Whether an address is no multiple of `bytes` (NULL is one).
inline bool misaligned(std::initializer_list<const void*> ps, uintptr_t bytes) {
  uintptr_t v = 0;
  for (const void* p : ps) v |= (uintptr_t)p;
  return v % bytes != 0;
}

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
