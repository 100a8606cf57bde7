// reduce64.hpp - wave reductions of 64-bit values by DPP and lane swaps, two
// 32-bit moves a step (an LDS permute would be a round trip of some 100
// cycles a step and half).
#pragma once

#include "common.hpp"

namespace qmv {

template <int CTRL>
__device__ __forceinline__ int dpp_i(int v) {
  return __builtin_amdgcn_update_dpp(0, v, CTRL, 0xF, 0xF, false);
}
template <int CTRL>
__device__ __forceinline__ double dpp_d(double v) {
  return __hiloint2double(dpp_i<CTRL>(__double2hiint(v)), dpp_i<CTRL>(__double2loint(v)));
}
// Partner across lane bit 5 (MASK 32) or 4 (MASK 16).
template <int MASK>
__device__ __forceinline__ uint32_t swap_partner(uint32_t v) {
  if constexpr (MASK == 32) {
    const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    return lane_id() & 32 ? r[0] : r[1];
  } else {
    const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    return lane_id() & 16 ? r[0] : r[1];
  }
}
template <int MASK>
__device__ __forceinline__ double swap_d(double v) {
  return __hiloint2double(static_cast<int>(swap_partner<MASK>(static_cast<uint32_t>(__double2hiint(v)))),
                          static_cast<int>(swap_partner<MASK>(static_cast<uint32_t>(__double2loint(v)))));
}
// Over the wave, the same in all lanes.
__device__ __forceinline__ double wave_sum(double v) {
  v += dpp_d<kDppXor1>(v);
  v += dpp_d<kDppXor2>(v);
  v += dpp_d<kDppMirror8>(v);
  v += dpp_d<kDppMirror16>(v);
  v += swap_d<16>(v);
  v += swap_d<32>(v);
  return v;
}

}  // namespace qmv
