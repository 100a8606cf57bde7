// past.hpp - loads and stores of what is too large to find again in the
// caches: marked as passing through, so that they leave what is there.
#pragma once

#include "common.hpp"

namespace qmv {

typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(4)));

// Four floats at p, 4-byte aligned; `past` is uniform.
__device__ __forceinline__ void store_four(float* p, const float (&v)[4], bool past) {
  u32x4 x;
  __builtin_memcpy(&x, v, 16);
  if (past) __builtin_nontemporal_store(x, reinterpret_cast<u32x4_any*>(p));
  else __builtin_memcpy(__builtin_assume_aligned(p, 4), &x, 16);
}
__device__ __forceinline__ u32x4 load_past(const float* p) {
  return __builtin_nontemporal_load(reinterpret_cast<const u32x4_any*>(p));
}

}  // namespace qmv
