// draw.hpp - what drawing from a row of logits rests on: exponentials in 64
// bits, the largest logit at its lowest index, and scans over a wave.
#pragma once

#include "reduce64.hpp"

namespace qmv {

// 2^t for t <= 0: the integer part by rounding in the sum with 1.5 * 2^52, 2^f
// of the rest, |f| <= 1/2, by the Taylor polynomial of degree 12 of
// exp(f ln 2): its next term is below 2 10^-16. NaN and -inf give 0.
struct Exp2 {
  double c[13];
  // The coefficients in scalar registers: as literals each step of the
  // polynomial would first move its own into a vector register.
  __device__ __forceinline__ Exp2() {
    double v = 1.0;
#pragma unroll
    for (int i = 0; i <= 12; ++i) {
      c[i] = v;
      v = v * 0.69314718055994530941723212145818 / (i + 1);
    }
#pragma unroll
    for (int i = 0; i <= 12; ++i) asm("" : "+s"(c[i]));
  }
  __device__ __forceinline__ double operator()(double t) const {
    constexpr double kRound = 6755399441055744.0;
    t = fmax(t, -1080.0);                      // below the smallest double
    const double k = t + kRound, f = t - (k - kRound);
    double p = c[12];
#pragma unroll
    for (int i = 11; i >= 0; --i) p = fma(p, f, c[i]);
    return __builtin_ldexp(p, static_cast<int>(__double2loint(k)));
  }
};

__device__ __forceinline__ void take_top(float& top, int& at, float t, int i) {
  const bool take = t > top || (t == top && i < at);
  top = take ? t : top;
  at = take ? i : at;
}
__device__ __forceinline__ void wave_top(float& top, int& at) {
  take_top(top, at, dpp_f<kDppXor1>(top), dpp_i<kDppXor1>(at));
  take_top(top, at, dpp_f<kDppXor2>(top), dpp_i<kDppXor2>(at));
  take_top(top, at, dpp_f<kDppMirror8>(top), dpp_i<kDppMirror8>(at));
  take_top(top, at, dpp_f<kDppMirror16>(top), dpp_i<kDppMirror16>(at));
  take_top(top, at, __uint_as_float(swap_partner<16>(__float_as_uint(top))),
           static_cast<int>(swap_partner<16>(static_cast<uint32_t>(at))));
  take_top(top, at, __uint_as_float(swap_partner<32>(__float_as_uint(top))),
           static_cast<int>(swap_partner<32>(static_cast<uint32_t>(at))));
}

// Value of the lane CTRL names, 0 where there is none or the row is masked out.
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp_zero_d(double v) {
  return __hiloint2double(__builtin_amdgcn_update_dpp(0, __double2hiint(v), CTRL, ROWS, 0xF, false),
                          __builtin_amdgcn_update_dpp(0, __double2loint(v), CTRL, ROWS, 0xF, false));
}
// Inclusive sums over the lanes: within rows of 16 by shifts, then the rows'
// last lanes handed on.
__device__ __forceinline__ double wave_scan(double v) {
  v += dpp_zero_d<0x111, 0xF>(v);              // row_shr:1
  v += dpp_zero_d<0x112, 0xF>(v);
  v += dpp_zero_d<0x114, 0xF>(v);
  v += dpp_zero_d<0x118, 0xF>(v);
  v += dpp_zero_d<0x142, 0xA>(v);              // row_bcast:15 to rows 1 and 3
  v += dpp_zero_d<0x143, 0xC>(v);              // row_bcast:31 to rows 2 and 3
  return v;
}

// The sums before each lane, from the inclusive ones. (Those less the lane's own
// value would lose in it what is far smaller.)
__device__ __forceinline__ double wave_before(double up) { return dpp_zero_d<0x138, 0xF>(up); }   // wave_shr:1

template <int CTRL, int ROWS>
__device__ __forceinline__ int dpp_zero_i(int v) {
  return __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xF, false);
}
__device__ __forceinline__ int wave_scan(int v) {
  v += dpp_zero_i<0x111, 0xF>(v);
  v += dpp_zero_i<0x112, 0xF>(v);
  v += dpp_zero_i<0x114, 0xF>(v);
  v += dpp_zero_i<0x118, 0xF>(v);
  v += dpp_zero_i<0x142, 0xA>(v);
  v += dpp_zero_i<0x143, 0xC>(v);
  return v;
}
// Four elements at i, `fill` behind the row's end.
__device__ __forceinline__ void load_quad(const float* row, int i, int n, float fill, float (&v)[4]) {
  if (n >= 4) {
    const int at = i + 4 <= n ? i : n - 4;     // no branch, so that loads go out together
    const u32x4 r = ld_x4(reinterpret_cast<const uint8_t*>(row + at));
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int from = i + e - at;             // 0..3 where the element exists
      const uint32_t x = from <= 0 ? r[0] : from == 1 ? r[1] : from == 2 ? r[2] : r[3];
      v[e] = i + e < n ? __uint_as_float(x) : fill;
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = i + e < n ? row[i + e] : fill;
  }
}

}  // namespace qmv
