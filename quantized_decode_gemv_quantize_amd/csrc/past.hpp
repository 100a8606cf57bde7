// past.hpp - loads and stores of what is too large to find again in the
// caches: marked as passing through, so that they leave what is there.
//
// Past the caches (non-temporal) means past the last-level one, too, where the
// next reader would have found it: that pays where all of it does not fit
// there. Through the L2 means that the line is written on and is not kept
// there: the reader finds it in the last-level cache.
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
// The same through the L2. A store of more than 64 bits reads its registers for
// two more wait states, which the compiler sees to for its own only.
__device__ __forceinline__ void store_four_through(float* p, const float (&v)[4]) {
  u32x4 x;
  __builtin_memcpy(&x, v, 16);
  asm volatile("global_store_dwordx4 %0, %1, off sc1\n\ts_nop 1" ::"v"(p), "v"(x) : "memory");
}
__device__ __forceinline__ u32x4 load_past(const float* p) {
  return __builtin_nontemporal_load(reinterpret_cast<const u32x4_any*>(p));
}

}  // namespace qmv
