// Keys of the routing's choice: one 32-bit integer that orders an expert by a
// float and names it.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace pw {

// Order-preserving integers of floats other than negative zero.
__host__ __device__ __forceinline__ int32_t ordered(float f) {
  const int32_t b = __builtin_bit_cast(int32_t, f);
  return b ^ (b >> 31 & 0x7fffffff);
}
__host__ __device__ __forceinline__ float unordered(int32_t i) { return __builtin_bit_cast(float, i ^ (i >> 31 & 0x7fffffff)); }

// The higher key is the higher value, as far as the bits outside `names` (2^n - 1, at
// least the experts' count less one) tell, and of equal ones the lower expert.
__host__ __device__ __forceinline__ int32_t route_key(float v, uint32_t expert, uint32_t names) {
  return (int32_t)(((uint32_t)ordered(v) & ~names) | ((names - expert) & names));
}

// What a key does not hold of its value (0: it holds all). Of the number's own bits: those
// of ordered() are all ones where a negative number has zeros.
__host__ __device__ __forceinline__ uint32_t key_lacks(float v, uint32_t names) { return __builtin_bit_cast(uint32_t, v) & names; }

}  // namespace pw
