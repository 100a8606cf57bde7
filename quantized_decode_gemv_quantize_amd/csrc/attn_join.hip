// attn_join.hip - the join of the ranges that a long cache is cut into.
#include "attn_kernel.hpp"

namespace qmv {

__device__ __forceinline__ float wave_max(float v) {
  v = fmaxf(v, dpp_f<kDppXor1>(v));
  v = fmaxf(v, dpp_f<kDppXor2>(v));
  v = fmaxf(v, dpp_f<kDppMirror8>(v));
  v = fmaxf(v, dpp_f<kDppMirror16>(v));
  return row_max(v);
}
__device__ __forceinline__ float wave_sum(float v) {
  v += dpp_f<kDppXor1>(v);
  v += dpp_f<kDppXor2>(v);
  v += dpp_f<kDppMirror8>(v);
  v += dpp_f<kDppMirror16>(v);
  return row_sum(v);
}

// One workgroup a row: its lanes hold four dims each and share the splits. A
// row's launch is one chain of latencies (its ranges' M and l, their joint
// maximum, the weighted sum of O), so every wave forms the factors for itself
// and the O values are on their way meanwhile (4.0 -> 3.1 us, 32 ranges of
// 32 heads).
template <int D, int SHIFT>
__global__ void __launch_bounds__(kAttnThreads) attn_join_kernel(AttnArgs a) {
  constexpr int L = D / 4, P = kAttnThreads / L;   // lanes a share, shares
  constexpr int AHEAD = 4;
  __shared__ float f_s[kAttnThreads / kWave][kMaxSplits];
  __shared__ __attribute__((aligned(16))) float acc_s[P * D];
  const int tid = threadIdx.x, token = blockIdx.x, head = blockIdx.y, splits = static_cast<int>(a.splits.d);
  const int wave = tid >> 6, lane = lane_id(), d = 4 * (tid % L), share = tid / L;
  const int row0 = a.b.token_start[0], row1 = a.b.token_start[a.b.n_seqs];
  const int64_t at = (static_cast<int64_t>(token) * a.n_heads + head) * splits;
  // (of a row outside the batch, whatever is there)
  const float2 none = make_float2(-INFINITY, 0.0f);
  const float2 p0 = lane < splits ? a.part_ml[at + lane] : none;
  const float2 p1 = lane + kWave < splits ? a.part_ml[at + lane + kWave] : none;
  const float* src = a.part_o + at * D + d;
  f32x4 x[AHEAD];
#pragma unroll
  for (int k = 0; k < AHEAD; ++k)
    x[k] = share < P && share + k * P < splits ? *reinterpret_cast<const f32x4*>(src + static_cast<int64_t>(share + k * P) * D)
                                               : f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  const float m = wave_max(fmaxf(p0.x, p1.x)), from = m == -INFINITY ? 0.0f : m;
  const float f0 = __builtin_amdgcn_exp2f(p0.x - from), f1 = __builtin_amdgcn_exp2f(p1.x - from);
  const float l = wave_sum(fmaf(p0.y, f0, p1.y * f1));
  f_s[wave][lane] = f0;
  if (kMaxSplits > kWave) f_s[wave][lane + kWave] = f1;
  if (token < row0 || token >= row1) return;       // the whole workgroup
  __builtin_amdgcn_wave_barrier();                 // the wave's own factors: LDS keeps its order
  f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
  if (share < P) {
    for (int i = share; i < splits; i += AHEAD * P) {
#pragma unroll
      for (int k = 0; k < AHEAD; ++k) {
        const int now = i + k * P, then = now + AHEAD * P;
        const float f = now < splits ? f_s[wave][now] : 0.0f;
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[e] = fmaf(x[k][e], f, acc[e]);
        if (then < splits) x[k] = *reinterpret_cast<const f32x4*>(src + static_cast<int64_t>(then) * D);
      }
    }
    *reinterpret_cast<f32x4*>(&acc_s[share * D + d]) = acc;
  }
  __syncthreads();
  if (tid < D) {
    float v = 0.0f;
#pragma unroll
    for (int p = 0; p < P; ++p) v += acc_s[p * D + tid];
    const float f = row_factor(a, head, m, l, static_cast<float>(SHIFT));
    a.out[token * a.ldo + static_cast<int64_t>(head) * D + tid] = f == 0.0f ? 0.0f : v * f;
  }
}

template <int SHIFT>
int launch_join_as(const AttnArgs& a, hipStream_t st) {
  const dim3 grid(static_cast<unsigned>(a.b.n_tokens), static_cast<unsigned>(a.n_heads));
  switch (a.head_dim) {
    case 64: hipLaunchKernelGGL((attn_join_kernel<64, SHIFT>), grid, dim3(kAttnThreads), 0, st, a); break;
    case 96: hipLaunchKernelGGL((attn_join_kernel<96, SHIFT>), grid, dim3(kAttnThreads), 0, st, a); break;
    case 128: hipLaunchKernelGGL((attn_join_kernel<128, SHIFT>), grid, dim3(kAttnThreads), 0, st, a); break;
    case 256: hipLaunchKernelGGL((attn_join_kernel<256, SHIFT>), grid, dim3(kAttnThreads), 0, st, a); break;
    default: return MMVQ_ERR_SHAPE;
  }
  return check_launch();
}

int launch_attn_join(const AttnArgs& a, bool f16, hipStream_t st) {
  return f16 ? launch_join_as<static_cast<int>(weight_shift(kKvF16))>(a, st) : launch_join_as<static_cast<int>(weight_shift(kKvQ8))>(a, st);
}

}  // namespace qmv
