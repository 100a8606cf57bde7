// embed.hip - rows of an embedding table, in any weight format.
//
//   out[t][i] = scale * W[ids[t]][i], in fp32
//
// A product of a block's scale and a code fits fp32 (at most 23 bits), so the
// formats without an offset take one fp32 product with `scale`, which rounds
// once. Those with one (d q + m, d sc q - dmin m) go through 64 bits and round
// those, 2^-52 off, to fp32. Every byte of a row is read once and every output
// written once; the writes are most of it and bound it: 4096 rows of 4096 take
// 11.9 (Q4_0) to 15.9 us (Q5_K), 15.2 from Q4_K (5.0 TB/s), 30.3 from F32 (4.4
// TB/s). One row is a launch's latency and two loads', 3 us. A wave takes kEPiece values of a row, in runs of four a lane, so that
// a store is 1 KB side by side and a short row does not leave a workgroup
// idle; what the lanes of a block share comes from the caches.
#include "launch.hpp"
#include "past.hpp"
#include "serve_args.hpp"

namespace qmv {

constexpr int kEThreads = 256;
constexpr int kEWaves = kEThreads / kWave;
constexpr int kEQuads = 4;                     // runs of four values a lane
constexpr int kEPiece = kWave * 4 * kEQuads;   // values of a row a wave takes

// A run of four consecutive values of a row, i a multiple of 4.
__device__ __forceinline__ uint32_t bytes4(const uint8_t* p) {   // 2-byte aligned
  uint32_t v;
  __builtin_memcpy(&v, __builtin_assume_aligned(p, 2), 4);
  return v;
}

// Six-bit scale and min of sub-block t of the 12 packed bytes.
__device__ __forceinline__ void k_scales(const uint8_t* s, int t, int& sc, int& m) {
  if (t < 4) {
    sc = s[t] & 63;
    m = s[t + 4] & 63;
  } else {
    sc = (s[t + 4] & 15) | (s[t - 4] >> 6 << 4);
    m = (s[t + 4] >> 4) | (s[t] >> 6 << 4);
  }
}

__device__ __forceinline__ void scaled(const float (&v)[4], float scale, float (&y)[4]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) y[e] = v[e] * scale;
}
// scale * (d q + m), the sum in 64 bits
__device__ __forceinline__ void scaled_offset(float d, const int (&q)[4], float m, float scale, float (&y)[4]) {
#pragma unroll
  for (int e = 0; e < 4; ++e)
    y[e] = static_cast<float>(fma(static_cast<double>(d), static_cast<double>(q[e]), static_cast<double>(m)) *
                              static_cast<double>(scale));
}

template <int TYPE>
__device__ __forceinline__ void table_run(const uint8_t* row, int i, int K, float scale, float (&y)[4]) {
  if constexpr (TYPE == MMVQ_F32 || TYPE == MMVQ_F16 || TYPE == MMVQ_BF16) {
    float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int at = i + e < K ? i + e : K - 1;
      if constexpr (TYPE == MMVQ_F32) v[e] = reinterpret_cast<const float*>(row)[at];
      else if constexpr (TYPE == MMVQ_F16) v[e] = h2f(ld_u16(row + 2 * static_cast<int64_t>(at)));
      else v[e] = __uint_as_float(ld_u16(row + 2 * static_cast<int64_t>(at)) << 16);
    }
    scaled(v, scale, y);
  } else if constexpr (TYPE == MMVQ_Q8_0) {
    const uint8_t* b = row + static_cast<int64_t>(i >> 5) * 34;
    const float d = h2f(ld_u16(b));
    const uint32_t w = bytes4(b + 2 + (i & 31));
    float v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = d * static_cast<float>(static_cast<int8_t>(w >> (8 * e)));
    scaled(v, scale, y);
  } else if constexpr (TYPE == MMVQ_Q4_0 || TYPE == MMVQ_Q4_1 || TYPE == MMVQ_Q5_0 || TYPE == MMVQ_Q5_1) {
    constexpr bool kMin = TYPE == MMVQ_Q4_1 || TYPE == MMVQ_Q5_1, kFifth = TYPE == MMVQ_Q5_0 || TYPE == MMVQ_Q5_1;
    constexpr int kHigh = kMin ? 4 : 2, kCodes = kHigh + (kFifth ? 4 : 0), kSize = kCodes + 16;
    const uint8_t* b = row + static_cast<int64_t>(i >> 5) * kSize;
    const int j = i & 31;
    const float d = h2f(ld_u16(b));
    const uint32_t w = bytes4(b + kCodes + (j & 15)) >> (j & 16 ? 4 : 0);
    uint32_t fifth = 0;
    if constexpr (kFifth) fifth = bytes4(b + kHigh) >> j;
    int q[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) q[e] = static_cast<int>((w >> (8 * e)) & 15) | static_cast<int>(((fifth >> e) & 1) << 4);
    if constexpr (kMin) {
      scaled_offset(d, q, h2f(ld_u16(b + 2)), scale, y);
    } else {
      float v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = d * static_cast<float>(q[e] - (kFifth ? 16 : 8));
      scaled(v, scale, y);
    }
  } else if constexpr (TYPE == MMVQ_Q4_K || TYPE == MMVQ_Q5_K) {
    constexpr int kCodes = TYPE == MMVQ_Q4_K ? 16 : 48;
    const uint8_t* b = row + static_cast<int64_t>(i >> 8) * (kCodes + 128);
    const int t = (i & 255) >> 5, l = i & 31;
    const uint32_t dm = ld_u32(b);
    int sc, m;
    k_scales(b + 4, t, sc, m);
    const uint32_t w = ld_u32(b + kCodes + 32 * (t >> 1) + l) >> (t & 1 ? 4 : 0);
    uint32_t fifth = 0;
    if constexpr (TYPE == MMVQ_Q5_K) fifth = ld_u32(b + 16 + l) >> t;
    int q[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) q[e] = static_cast<int>((w >> (8 * e)) & 15) | static_cast<int>(((fifth >> (8 * e)) & 1) << 4);
    scaled_offset(h2f(dm) * static_cast<float>(sc), q, -(h2f(dm >> 16) * static_cast<float>(m)), scale, y);
  } else {
    static_assert(TYPE == MMVQ_Q6_K);
    const uint8_t* b = row + static_cast<int64_t>(i >> 8) * 210;
    const int j = i & 255, h = j >> 7, g = (j >> 5) & 3, l = j & 31;
    const float d = h2f(ld_u16(b + 208)) * static_cast<float>(static_cast<int8_t>(b[192 + (j >> 4)]));
    const uint32_t low = bytes4(b + 64 * h + 32 * (g & 1) + l) >> (g & 2 ? 4 : 0);
    const uint32_t high = bytes4(b + 128 + 32 * h + l) >> (2 * g);
    float v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      v[e] = d * static_cast<float>(static_cast<int>((low >> (8 * e)) & 15) + static_cast<int>(((high >> (8 * e)) & 3) << 4) - 32);
    scaled(v, scale, y);
  }
}

template <int TYPE>
__global__ void __launch_bounds__(kEThreads) embed_kernel(EmbedArgs a) {
  for (int64_t unit = static_cast<int64_t>(blockIdx.x) * kEWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); unit < a.units;
       unit += static_cast<int64_t>(gridDim.x) * kEWaves) {
    const int64_t t = unit / a.pieces;
    const int first = static_cast<int>(unit - t * a.pieces) * kEPiece + 4 * lane_id();
    const int id = a.ids[t];
    const bool real = id >= 0 && id < a.vocab;
    const uint8_t* row = a.table + static_cast<int64_t>(real ? id : 0) * a.row_bytes;
    float* out = a.out + t * a.ldo;
    float y[kEQuads][4];
#pragma unroll
    for (int k = 0; k < kEQuads; ++k) {
      const int i = first + 4 * kWave * k;
      if (real && i < a.K) {
        table_run<TYPE>(row, i, a.K, a.scale, y[k]);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) y[k][e] = 0.0f;
      }
    }
#pragma unroll
    for (int k = 0; k < kEQuads; ++k) {
      const int i = first + 4 * kWave * k;
      if (i + 4 <= a.K) {
        if (a.through) store_four_through(out + i, y[k]);
        else store_four(out + i, y[k], a.past);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (i + e < a.K) out[i + e] = y[k][e];
      }
    }
  }
}

constexpr int64_t kMaxEmbedGrid = 1 << 20;     // workgroups; more pieces share them

int launch_embed(int type, const EmbedArgs& given, hipStream_t st) {
  EmbedArgs a = given;
  a.pieces = (a.K + kEPiece - 1) / kEPiece;
  a.units = a.n * a.pieces;
  a.past = past_caches(a.n, a.K, kEmbedPast);
  a.through = !a.past && past_caches(a.n, a.K, kL2) && a.ldo % 32 == 0 && reinterpret_cast<uintptr_t>(a.out) % 128 == 0;
  const int64_t blocks = (a.units + kEWaves - 1) / kEWaves;
  const dim3 grid(static_cast<unsigned>(blocks < kMaxEmbedGrid ? blocks : kMaxEmbedGrid)), block(kEThreads);
  switch (type) {
    case MMVQ_F32: hipLaunchKernelGGL(embed_kernel<MMVQ_F32>, grid, block, 0, st, a); break;
    case MMVQ_F16: hipLaunchKernelGGL(embed_kernel<MMVQ_F16>, grid, block, 0, st, a); break;
    case MMVQ_BF16: hipLaunchKernelGGL(embed_kernel<MMVQ_BF16>, grid, block, 0, st, a); break;
    case MMVQ_Q4_0: hipLaunchKernelGGL(embed_kernel<MMVQ_Q4_0>, grid, block, 0, st, a); break;
    case MMVQ_Q4_1: hipLaunchKernelGGL(embed_kernel<MMVQ_Q4_1>, grid, block, 0, st, a); break;
    case MMVQ_Q5_0: hipLaunchKernelGGL(embed_kernel<MMVQ_Q5_0>, grid, block, 0, st, a); break;
    case MMVQ_Q5_1: hipLaunchKernelGGL(embed_kernel<MMVQ_Q5_1>, grid, block, 0, st, a); break;
    case MMVQ_Q8_0: hipLaunchKernelGGL(embed_kernel<MMVQ_Q8_0>, grid, block, 0, st, a); break;
    case MMVQ_Q4_K: hipLaunchKernelGGL(embed_kernel<MMVQ_Q4_K>, grid, block, 0, st, a); break;
    case MMVQ_Q5_K: hipLaunchKernelGGL(embed_kernel<MMVQ_Q5_K>, grid, block, 0, st, a); break;
    case MMVQ_Q6_K: hipLaunchKernelGGL(embed_kernel<MMVQ_Q6_K>, grid, block, 0, st, a); break;
    default: return MMVQ_ERR_TYPE;
  }
  return check_launch();
}

}  // namespace qmv
