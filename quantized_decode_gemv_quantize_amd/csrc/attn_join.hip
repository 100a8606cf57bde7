// attn_join.hip - the shape of an attention launch, and the join of the
// ranges that a long cache is cut into.
#include "attn_kernel.hpp"

namespace qmv {

constexpr int kMaxSplits = 128;                 // at most the lanes of a join's workgroup
constexpr int kSplitKeys = 256;                 // fewest keys worth a workgroup of their own
constexpr int kTargetGroups = 512;              // two workgroups for each of the 256 compute units

// Rows of one key/value head (new tokens times query heads that share it):
// up to 16 or 32 fit the tiles of one wave, and the four waves share the
// keys; beyond 64 each wave takes rows of its own. The keys are cut until
// about two workgroups a compute unit exist, no finer than kSplitKeys.
AttnShape attn_shape(int kind, int nb, int n_seqs, int n_kv_heads, int group, int max_new, int max_len, int window) {
  (void)kind;
  const int64_t rows = static_cast<int64_t>(max_new) * group;
  AttnShape s;
  s.rows = rows > 64;
  s.mt = nb < 8 && rows > 16 ? 2 : 1;
  if (nb == 2 && rows > 32 && rows <= 48) s.mt = 3;
  const int rt = 16 * s.mt * (s.rows ? 4 : 1);
  s.tiles = static_cast<int>((rows + rt - 1) / rt);
  const int64_t groups = static_cast<int64_t>(n_seqs) * n_kv_heads * s.tiles;
  const int64_t keys = window > 0 && window + static_cast<int64_t>(max_new) < max_len
                           ? window + static_cast<int64_t>(max_new) : max_len;
  const char* e1=getenv("ATG"); const char* e2=getenv("ASK");
  const int tg=e1?atoi(e1):kTargetGroups, sk=e2?atoi(e2):kSplitKeys;
  int64_t splits = (tg + groups - 1) / groups;
  const int64_t most = (keys + sk - 1) / sk;
  if (splits > most) splits = most;
  if (splits > kMaxSplits) splits = kMaxSplits;
  s.splits = static_cast<int>(splits < 1 ? 1 : splits);
  return s;
}

// One workgroup a row: its lanes hold four dims each and share the splits.
template <int D, int SHIFT>
__global__ void __launch_bounds__(kAttnThreads) attn_join_kernel(AttnArgs a) {
  constexpr int L = D / 4, P = kAttnThreads / L;   // lanes a share, shares
  __shared__ float2 ml[kMaxSplits];
  __shared__ float acc_s[P * D];
  const int tid = threadIdx.x, token = blockIdx.x, head = blockIdx.y, splits = static_cast<int>(a.splits.d);
  const int64_t at = (static_cast<int64_t>(token) * a.n_heads + head) * splits;
  const int row0 = a.b.token_start[0], row1 = a.b.token_start[a.b.n_seqs];
  if (tid < splits) ml[tid] = a.part_ml[at + tid];   // (of a row outside, whatever is there)
  __syncthreads();
  if (token < row0 || token >= row1) return;
  float m = -INFINITY;
  for (int i = 0; i < splits; ++i) m = fmaxf(m, ml[i].x);
  const float from = m == -INFINITY ? 0.0f : m;
  float l = 0.0f;
  for (int i = 0; i < splits; ++i) l = fmaf(ml[i].y, __builtin_amdgcn_exp2f(ml[i].x - from), l);
  const int d = 4 * (tid % L), share = tid / L;
  f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
  if (share < P)
    for (int i = share; i < splits; i += P) {
      const float f = __builtin_amdgcn_exp2f(ml[i].x - from);
      const f32x4 x = *reinterpret_cast<const f32x4*>(a.part_o + (at + i) * D + d);
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[e] = fmaf(x[e], f, acc[e]);
    }
  if (share < P) *reinterpret_cast<f32x4*>(&acc_s[share * D + d]) = acc;
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
