// norm.hip - residual addition, RMS norm and q8_1 quantization in one pass,
// and q8_1 columns read back.
//
//   h = x + residual (fp32), r = 1/sqrt(sum(h^2)/K + eps), y = h r w
//
// The sum, the root and the two products are in 64 bits and y is rounded to
// fp32 once: a q8_1 code depends on which side of a border y lies, and with
// 64 bits the order of the sum does not decide it. The extra arithmetic (a
// 64-bit fma and two 64-bit products a value, at half the fp32 rate) hides
// behind the memory traffic.
//
// One workgroup owns a column and keeps it in registers between the sum and
// the products, so each input is read once and each output written once. It
// is bound by memory bandwidth from about a hundred columns (256 of 14336
// with all outputs but y: 12.4 us, 3.9 TB/s) and by the latency of one
// column's load, reduction and store below (one of 4096: 3.4 us).
#include "decode_args.hpp"
#include "launch.hpp"
#include "q8.hpp"
#include "reduce64.hpp"

namespace qmv {

__device__ __forceinline__ void st_x4(float* p, const float (&v)[4]) {   // p 4-byte aligned
  __builtin_memcpy(__builtin_assume_aligned(p, 4), v, 16);
}

// Up to four values at element i of a row of K.
__device__ __forceinline__ void load4(const float* row, int i, int K, float (&v)[4]) {
  if (i + 4 <= K) {
    const u32x4 r = ld_x4(reinterpret_cast<const uint8_t*>(row + i));
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = __uint_as_float(r[e]);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = i + e < K ? row[i + e] : 0.0f;
  }
}

__device__ __forceinline__ void store4(float* row, int i, int K, const float (&v)[4]) {
  if (i + 4 <= K) {
    st_x4(row + i, v);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (i + e < K) row[i + e] = v[e];
  }
}

// Sum over the workgroup's T lanes, the same in every lane.
template <int T>
__device__ __forceinline__ double block_sum(double v, double* lds) {
  v = wave_sum(v);
  if (T > kWave) {
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.0;
#pragma unroll
    for (int w = 0; w < T / kWave; ++w) v += lds[w];
  }
  return v;
}

// 1 / sqrt(a) by the hardware's estimate and two Newton steps (each doubles
// its 26 bits): some 15 operations where the exact root and quotient take
// 60 in a row, while every lane of the workgroup waits.
__device__ __forceinline__ double rsqrt64(double a) {
  double r = __builtin_amdgcn_rsq(a);
  const double half = 0.5 * a;
  r = r * fma(-half * r, r, 1.5);
  r = r * fma(-half * r, r, 1.5);
  return a < INFINITY ? r : a == INFINITY ? 0.0 : a;
}

// The q8_1 block of a group of 8 lanes that hold 4 values each.
__device__ __forceinline__ void store_q8_1(uint8_t* col, int i, const float (&y)[4]) {
  const u32x4 raw[1] = {{__float_as_uint(y[0]), __float_as_uint(y[1]), __float_as_uint(y[2]), __float_as_uint(y[3])}};
  float amax = absmax4(raw[0]);
  amax = fmaxf(amax, dpp_f<kDppXor1>(amax));
  amax = fmaxf(amax, dpp_f<kDppXor2>(amax));
  amax = fmaxf(amax, dpp_f<kDppMirror8>(amax));
  const float d = q8_scale_product(amax);
  int sq = 0;
  uint32_t packed[1];
  q8_quant_block(raw, d, packed, sq);
  sq += __builtin_amdgcn_update_dpp(0, sq, kDppXor1, 0xF, 0xF, false);
  sq += __builtin_amdgcn_update_dpp(0, sq, kDppXor2, 0xF, 0xF, false);
  sq += __builtin_amdgcn_update_dpp(0, sq, kDppMirror8, 0xF, 0xF, false);
  uint8_t* yb = col + static_cast<int64_t>(i >> 5) * kQ8Bytes;
  *reinterpret_cast<uint32_t*>(yb + 4 + (i & 31)) = packed[0];
  if ((i & 31) == 0) *reinterpret_cast<uint32_t*>(yb) = f2h_bits(d) | (f2h_bits(q8_s(d, sq)) << 16);
}

__device__ __forceinline__ void weights4(const float* w, int i, int K, float (&v)[4]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = 1.0f;
  if (w) load4(w, i, K, v);
}

__device__ __forceinline__ void scale4(const float (&h)[4], double r, const float (&wv)[4], float (&y)[4]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) y[e] = static_cast<float>(static_cast<double>(h[e]) * r * static_cast<double>(wv[e]));
}

__device__ __forceinline__ void out4(const NormArgs& a, int64_t j, int i, const float (&y)[4]) {
  if (a.y) store4(a.y + j * a.ldy, i, a.K, y);
  if (a.yq) store_q8_1(a.yq + j * (static_cast<int64_t>(a.K / 32) * kQ8Bytes), i, y);
}

// T lanes hold a column, 4 V values each.
template <int T, int V>
__global__ void __launch_bounds__(T) norm_kernel(NormArgs a) {
  __shared__ double lds[2][T / kWave];
  int turn = 0;
  for (int64_t j = blockIdx.x; j < a.n; j += gridDim.x, turn ^= 1) {
    const float* x = a.x + j * a.ldx;
    const float* res = a.res ? a.res + j * a.ldr : nullptr;
    float h[V][4], w[V][4];
    double ss = 0.0;
#pragma unroll
    for (int v = 0; v < V; ++v) load4(x, 4 * (v * T + static_cast<int>(threadIdx.x)), a.K, h[v]);
    if (res) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float t[4];
        load4(res, 4 * (v * T + static_cast<int>(threadIdx.x)), a.K, t);
#pragma unroll
        for (int e = 0; e < 4; ++e) h[v][e] += t[e];
      }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) weights4(a.w, 4 * (v * T + static_cast<int>(threadIdx.x)), a.K, w[v]);   // on their way meanwhile
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int e = 0; e < 4; ++e) ss = fma(static_cast<double>(h[v][e]), static_cast<double>(h[v][e]), ss);
    if (a.sum) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int i = 4 * (v * T + static_cast<int>(threadIdx.x));
        if (i < a.K) store4(a.sum + j * a.lds, i, a.K, h[v]);
      }
    }
    const double r = rsqrt64(fma(block_sum<T>(ss, lds[turn]), a.inv_K, a.eps));
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int i = 4 * (v * T + static_cast<int>(threadIdx.x));
      if (i < a.K) {
        float y[4];
        scale4(h[v], r, w[v], y);
        out4(a, j, i, y);
      }
    }
  }
}

// Columns that do not fit the registers of a workgroup: h is formed again
// (or read back from sum, which may be x itself) in the second pass.
template <int T>
__global__ void __launch_bounds__(T) norm_long_kernel(NormArgs a) {
  __shared__ double lds[2][T / kWave];
  int turn = 0;
  for (int64_t j = blockIdx.x; j < a.n; j += gridDim.x, turn ^= 1) {
    const float* x = a.x + j * a.ldx;
    const float* res = a.res ? a.res + j * a.ldr : nullptr;
    float* sum = a.sum ? a.sum + j * a.lds : nullptr;
    double ss = 0.0;
    for (int i = 4 * static_cast<int>(threadIdx.x); i < a.K; i += 4 * T) {
      float h[4], t[4];
      load4(x, i, a.K, h);
      if (res) {
        load4(res, i, a.K, t);
#pragma unroll
        for (int e = 0; e < 4; ++e) h[e] += t[e];
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) ss = fma(static_cast<double>(h[e]), static_cast<double>(h[e]), ss);
      if (sum) store4(sum, i, a.K, h);
    }
    const double r = rsqrt64(fma(block_sum<T>(ss, lds[turn]), a.inv_K, a.eps));
    for (int i = 4 * static_cast<int>(threadIdx.x); i < a.K; i += 4 * T) {
      float h[4], t[4], w[4], y[4];
      weights4(a.w, i, a.K, w);
      load4(sum ? sum : x, i, a.K, h);
      if (res && !sum) {
        load4(res, i, a.K, t);
#pragma unroll
        for (int e = 0; e < 4; ++e) h[e] += t[e];
      }
      scale4(h, r, w, y);
      out4(a, j, i, y);
    }
  }
}

constexpr int64_t kMaxNormGrid = 1 << 20;   // workgroups; more columns share them

int launch_norm(const NormArgs& a, hipStream_t st) {
  const dim3 grid(static_cast<unsigned>(a.n < kMaxNormGrid ? a.n : kMaxNormGrid));
  const int quads = (a.K + 3) / 4;
  if (quads <= 256) hipLaunchKernelGGL((norm_kernel<256, 1>), grid, dim3(256), 0, st, a);
  else if (quads <= 512) hipLaunchKernelGGL((norm_kernel<256, 2>), grid, dim3(256), 0, st, a);
  else if (quads <= 1024) hipLaunchKernelGGL((norm_kernel<1024, 1>), grid, dim3(1024), 0, st, a);
  else if (quads <= 2048) hipLaunchKernelGGL((norm_kernel<1024, 2>), grid, dim3(1024), 0, st, a);
  else if (quads <= 4096) hipLaunchKernelGGL((norm_kernel<1024, 4>), grid, dim3(1024), 0, st, a);
  else hipLaunchKernelGGL((norm_long_kernel<1024>), grid, dim3(1024), 0, st, a);
  return check_launch();
}

// Four values a lane: one code word and, shared by 8 lanes, the block's d.
__global__ void __launch_bounds__(256) dequantize_q8_1_kernel(const uint8_t* __restrict__ yq, int64_t nb, int64_t n,
                                                              float* __restrict__ x, int64_t ldx) {
  const int64_t step = static_cast<int64_t>(gridDim.x) * 256;
  for (int64_t g = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; g < n * nb * 8; g += step) {
    const int64_t blk = g >> 3, j = blk / nb, b = blk - j * nb;
    const int sub = static_cast<int>(g & 7);
    const float d = h2f(ld_u16(yq + blk * kQ8Bytes));
    const uint32_t c = ld_u32(yq + blk * kQ8Bytes + 4 + 4 * sub);
    float v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = d * static_cast<float>(sbfe(c, 8 * e, 8));
    st_x4(x + j * ldx + 32 * b + 4 * sub, v);
  }
}

int launch_dequantize_q8_1(const uint8_t* yq, int64_t K, int64_t n, float* x, int64_t ldx, hipStream_t st) {
  const int64_t want = (n * (K / 32) * 8 + 255) / 256, most = 1 << 16;
  hipLaunchKernelGGL(dequantize_q8_1_kernel, dim3(static_cast<unsigned>(want < most ? want : most)), dim3(256), 0, st,
                     yq, K / 32, n, x, ldx);
  return check_launch();
}

}  // namespace qmv
