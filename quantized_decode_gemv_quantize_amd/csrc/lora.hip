// lora.hip - low-rank adapters of many requests beside a shared projection.
//
//   v = A_a x[t] (r numbers a row), out[t] = base[t] + scale_a * B_a v
//
// Two launches: shrink (v, in ranges of K) and expand (v of all ranges
// summed, B_a v, the addition). Up to 16 rows of one adapter, out of 64
// consecutive ones, share its weights: the tile of a 16x16x32 bf16 matrix
// product, whose other side is 16 rows of A or B. Rows of one adapter are
// found in the ids of the 64 by a ballot, so that nothing has to be sorted
// or listed first; single tokens of as many adapters leave 15 of a tile's 16
// columns empty, but then the weights are all there is to read, and the
// products wait for them anyway.
//
// fp32 values enter a product as three bf16 parts by truncation, x = x1 + x2 +
// x3 exactly (8 bits each); weights as one (bf16), two (fp16: 11 bits) or
// three (fp32). All products of parts but that of the two last of three and
// three (2^-28 of the whole) are formed: fp32 products, for three, six or
// eight matrix instructions where one of fp32 takes the time of sixteen.
#include "launch.hpp"
#include "serve_args.hpp"

namespace qmv {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kLThreads = 256;
constexpr int kLWaves = kLThreads / kWave;
constexpr int kLBlock = 64;                    // consecutive rows among which tiles are formed
constexpr int kLTile = 16;                     // rows of a tile
constexpr int kLStep = 32;                     // of K, or ranks, a matrix product

__device__ __forceinline__ f32x4 mfma_bf16(u32x4 a, u32x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// High halves of two words: two bf16 by truncation.
__device__ __forceinline__ uint32_t high_halves(float lo, float hi) {
  return __builtin_amdgcn_perm(__float_as_uint(hi), __float_as_uint(lo), 0x07060302u);
}
__device__ __forceinline__ float truncated(float v) { return __uint_as_float(__float_as_uint(v) & 0xFFFF0000u); }

// The first N bf16 parts of eight values.
template <int N>
__device__ __forceinline__ void split8(const float (&v)[8], u32x4 (&part)[N]) {
  float rest[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) rest[e] = v[e];
#pragma unroll
  for (int p = 0; p < N; ++p) {
#pragma unroll
    for (int e = 0; e < 8; e += 2) part[p][e / 2] = high_halves(rest[e], rest[e + 1]);
    if (p + 1 < N) {
#pragma unroll
      for (int e = 0; e < 8; ++e) rest[e] -= truncated(rest[e]);
    }
  }
}

// Eight consecutive weights at element i, as bf16 parts; those from `valid` on 0.
template <int TYPE>
struct Weights {
  static constexpr int kParts = TYPE == MMVQ_BF16 ? 1 : TYPE == MMVQ_F16 ? 2 : 3;
  static constexpr int kBytes = TYPE == MMVQ_F32 ? 4 : 2;
  static __device__ __forceinline__ void load(const uint8_t* m, int64_t i, int valid, u32x4 (&part)[kParts]) {
    const uint8_t* p = m + i * kBytes;
    float v[8];
    if constexpr (TYPE == MMVQ_F32) {
      const u32x4 a = ld_a16_x4(p), b = ld_a16_x4(p + 16);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[e] = __uint_as_float(a[e]);
        v[e + 4] = __uint_as_float(b[e]);
      }
    } else {
      const u32x4 a = ld_a16_x4(p);
      if constexpr (TYPE == MMVQ_BF16) {
        part[0] = a;
        if (valid < 8) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            part[0][e] = a[e] & ((2 * e < valid ? 0x0000FFFFu : 0u) | (2 * e + 1 < valid ? 0xFFFF0000u : 0u));
        }
        return;
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[2 * e] = h2f(a[e]);
        v[2 * e + 1] = h2f(a[e] >> 16);
      }
    }
    if (valid < 8) {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = e < valid ? v[e] : 0.0f;
    }
    split8<kParts>(v, part);
  }
};

// c += weights x values over their parts, largest last.
template <int PARTS>
__device__ __forceinline__ f32x4 multiply(const u32x4 (&w)[PARTS], const u32x4 (&x)[3], f32x4 c) {
#pragma unroll
  for (int order = 3; order >= 0; --order)     // parts p and q are below 2^-7(p + q) of the product
#pragma unroll
    for (int p = PARTS - 1; p >= 0; --p)
      if (order - p >= 0 && order - p <= 2) c = mfma_bf16(w[p], x[order - p], c);
  return c;
}

// The tile that row `lead` of a block of 64 leads, the same in every wave.
struct Tile {
  int adapter;             // -1: none
  int rank;
  int count;               // rows; 0: none
  int row;                 // of the lane's column (lane % 16), valid below count
  float scale;
};

__device__ __forceinline__ int adapter_of(const LoraArgs& a, int t) {
  const int s = a.row_seq ? a.row_seq[t] : t;
  if (s < 0 || s >= a.n_seqs) return -1;
  const int id = a.adapter[s];
  return id >= 0 && id < a.n_adapters ? id : -1;
}

// Adapters of the block's rows, one a lane; -2 behind the last row.
__device__ __forceinline__ int block_ids(const LoraArgs& a, int block) {
  const int t = block * kLBlock + lane_id();
  return t < a.n ? adapter_of(a, t) : -2;
}

__device__ __forceinline__ Tile tile_of(const LoraArgs& a, int block, int ids, int lead) {
  Tile tile{__builtin_amdgcn_readlane(ids, lead), 0, 0, 0, 0.0f};
  const uint64_t same = __ballot(ids == tile.adapter);
  const int ahead = __builtin_popcountll(same & ((uint64_t(1) << lead) - 1));
  if (tile.adapter == -2 || ahead % kLTile) return tile;
  const int left = __builtin_popcountll(same) - ahead;
  tile.count = left < kLTile ? left : kLTile;
  const int lane = lane_id(), mine = __builtin_popcountll(same & ((uint64_t(1) << lane) - 1)) - ahead;
  const bool member = ids == tile.adapter && mine >= 0 && mine < kLTile;
  const int pushed = __builtin_amdgcn_ds_permute(4 * (member ? mine : kWave - 1), block * kLBlock + lane);
  tile.row = __shfl(pushed, lane % kLTile);
  if (tile.adapter >= 0) {
    const int r = a.rank ? a.rank[tile.adapter] : a.max_rank;
    tile.rank = r < 0 ? 0 : r > a.max_rank ? a.max_rank : r;
    tile.scale = a.scale ? a.scale[tile.adapter] : 1.0f;
  }
  return tile;
}

// Eight fp32 values at element i of a row (4-byte aligned).
__device__ __forceinline__ void values8(const float* p, float (&v)[8]) {
  const u32x4 a = ld_x4(reinterpret_cast<const uint8_t*>(p)), b = ld_x4(reinterpret_cast<const uint8_t*>(p + 4));
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    v[e] = __uint_as_float(a[e]);
    v[e + 4] = __uint_as_float(b[e]);
  }
}

// v of a tile over a range of K, up to 16 RT ranks at a time. The four waves
// share the range.
template <int TYPE, int RT>
__global__ void __launch_bounds__(kLThreads) lora_shrink_kernel(LoraArgs a) {
  using W = Weights<TYPE>;
  __shared__ f32x4 lds[kLWaves][RT][kWave];
  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), g = lane / 16;
  const int block = blockIdx.x, per_y = kLBlock / gridDim.y, split = blockIdx.z;
  const int ids = block_ids(a, block);
  const int steps = static_cast<int>((a.K + kLStep - 1) / kLStep);
  const int s0 = (split * kLWaves + wave) * a.steps, s1 = s0 + a.steps < steps ? s0 + a.steps : steps;
  for (int lead = blockIdx.y * per_y; lead < static_cast<int>(blockIdx.y + 1) * per_y; ++lead) {
    const Tile tile = tile_of(a, block, ids, lead);
    if (tile.count == 0 || tile.rank == 0) continue;       // uniform
    const bool live = lane % 16 < tile.count;
    const float* x = a.x + (live ? tile.row : 0) * a.ldx;
    const uint8_t* A = a.A + tile.adapter * a.stride_a * W::kBytes;
    for (int r0 = 0; r0 < tile.rank; r0 += 16 * RT) {
      f32x4 acc[RT];
#pragma unroll
      for (int t = 0; t < RT; ++t) acc[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 2
      for (int s = s0; s < s1; ++s) {
        const int k = s * kLStep + 8 * g;
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = 0.0f;
        if (live && k < a.K) values8(x + k, v);
        u32x4 w[RT][W::kParts], xp[3];
#pragma unroll
        for (int t = 0; t < RT; ++t) {
          const int j = r0 + 16 * t + lane % 16;
#pragma unroll
          for (int p = 0; p < W::kParts; ++p) w[t][p] = u32x4{0, 0, 0, 0};
          if (j < tile.rank && k < a.K) W::load(A, j * a.K + k, 8, w[t]);
        }
        split8<3>(v, xp);
#pragma unroll
        for (int t = 0; t < RT; ++t) acc[t] = multiply<W::kParts>(w[t], xp, acc[t]);
      }
      __syncthreads();                         // the sums before are read
#pragma unroll
      for (int t = 0; t < RT; ++t) lds[wave][t][lane] = acc[t];
      __syncthreads();
      for (int t = wave; t < RT; t += kLWaves) {
        const int j = r0 + 16 * t + 4 * g;
        f32x4 sum = lds[0][t][lane];
#pragma unroll
        for (int w = 1; w < kLWaves; ++w) sum += lds[w][t][lane];
        if (live && j < a.max_rank)
          *reinterpret_cast<f32x4*>(a.part + (static_cast<int64_t>(split) * a.n + tile.row) * a.max_rank + j) = sum;
      }
    }
  }
}

// base + scale * B v of a tile, for a slice of M; up to 32 RC ranks.
template <int TYPE, int RC>
__global__ void __launch_bounds__(kLThreads) lora_expand_kernel(LoraArgs a) {
  using W = Weights<TYPE>;
  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), g = lane / 16;
  const int block = blockIdx.x, per_y = kLBlock / gridDim.y;
  const int ids = block_ids(a, block);
  const int64_t m_step = static_cast<int64_t>(gridDim.z) * kLWaves * 16, m_first = (static_cast<int64_t>(blockIdx.z) * kLWaves + wave) * 16;
  for (int lead = blockIdx.y * per_y; lead < static_cast<int>(blockIdx.y + 1) * per_y; ++lead) {
    const Tile tile = tile_of(a, block, ids, lead);
    if (tile.count == 0 || (tile.rank == 0 && a.base == a.out)) continue;   // uniform
    const bool live = lane % 16 < tile.count;
    u32x4 v[RC][3];
#pragma unroll
    for (int c = 0; c < RC; ++c) {
      const int j = kLStep * c + 8 * g;
      float sum[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) sum[e] = 0.0f;
      if (live && j < tile.rank)
        for (int s = 0; s < a.splits; ++s) {
          float one[8];
          values8(a.part + (static_cast<int64_t>(s) * a.n + tile.row) * a.max_rank + j, one);
#pragma unroll
          for (int e = 0; e < 8; ++e) sum[e] += one[e];
        }
      split8<3>(sum, v[c]);
    }
    const uint8_t* B = a.B + (tile.adapter < 0 ? 0 : tile.adapter) * a.stride_b * W::kBytes;
    const float* base = a.base + (live ? tile.row : 0) * a.ldb;
    float* out = a.out + (live ? tile.row : 0) * a.ldo;
    for (int64_t m0 = m_first; m0 < a.M; m0 += m_step) {
      const int64_t m = m0 + lane % 16, o = m0 + 4 * g;
      f32x4 acc{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int c = 0; c < RC; ++c) {
        const int j = kLStep * c + 8 * g;
        if (kLStep * c < tile.rank) {          // uniform
          u32x4 w[W::kParts];
#pragma unroll
          for (int p = 0; p < W::kParts; ++p) w[p] = u32x4{0, 0, 0, 0};
          if (m < a.M && j < tile.rank) W::load(B, m * a.max_rank + j, tile.rank - j, w);
          acc = multiply<W::kParts>(w, v[c], acc);
        }
      }
      if (live && o + 4 <= a.M) {
        const u32x4 b = ld_x4(reinterpret_cast<const uint8_t*>(base + o));
        f32x4 y;
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = __uint_as_float(b[e]) + tile.scale * acc[e];
        __builtin_memcpy(__builtin_assume_aligned(out + o, 4), &y, 16);
      } else if (live) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (o + e < a.M) out[o + e] = base[o + e] + tile.scale * acc[e];
      }
    }
  }
}

// Launch shape. Ranges of K until the chip is filled, of two products a wave
// at least; slices of M likewise, of 64 outputs at least.
struct LoraShape {
  int blocks, leads, splits, steps, slices;
};
inline LoraShape lora_shape(int64_t n, int64_t K, int64_t M) {
  LoraShape s;
  s.blocks = static_cast<int>((n + kLBlock - 1) / kLBlock);
  s.leads = s.blocks <= 8 ? 64 : s.blocks <= 32 ? 16 : 4;
  const int64_t tiles = (n + kLTile - 1) / kLTile, want = (4 * kCus + tiles - 1) / tiles;
  const int64_t steps = (K + kLStep - 1) / kLStep, most = (steps + 2 * kLWaves - 1) / (2 * kLWaves);
  int64_t splits = want < most ? want : most;
  if (splits > 16) splits = 16;
  s.steps = static_cast<int>((steps + splits * kLWaves - 1) / (splits * kLWaves));
  s.splits = static_cast<int>((steps + static_cast<int64_t>(s.steps) * kLWaves - 1) / (s.steps * kLWaves));
  const int64_t groups = (M + 63) / 64;
  s.slices = static_cast<int>(want < groups ? want : groups);
  if (s.slices > 64) s.slices = 64;
  return s;
}

int64_t lora_bytes(int64_t n, int64_t K, int64_t M, int max_rank) {
  if (n == 0) return 0;
  return lora_shape(n, K, M).splits * n * max_rank * static_cast<int64_t>(sizeof(float));
}

template <int TYPE, int RT>
int launch_ranks(const LoraArgs& a, const LoraShape& s, hipStream_t st) {
  hipLaunchKernelGGL((lora_shrink_kernel<TYPE, RT>), dim3(s.blocks, s.leads, s.splits), dim3(kLThreads), 0, st, a);
  const int rc = check_launch();
  if (rc) return rc;
  constexpr int RC = (RT + 1) / 2;
  const dim3 grid(s.blocks, s.leads, s.slices);
  if constexpr (RT == 8) {
    if (a.max_rank > 128) {
      hipLaunchKernelGGL((lora_expand_kernel<TYPE, 2 * RC>), grid, dim3(kLThreads), 0, st, a);
      return check_launch();
    }
  }
  hipLaunchKernelGGL((lora_expand_kernel<TYPE, RC>), grid, dim3(kLThreads), 0, st, a);
  return check_launch();
}

template <int TYPE>
int launch_type(const LoraArgs& given, hipStream_t st) {
  LoraArgs a = given;
  const LoraShape s = lora_shape(a.n, a.K, a.M);
  a.splits = s.splits;
  a.steps = s.steps;
  if (a.max_rank <= 16) return launch_ranks<TYPE, 1>(a, s, st);
  if (a.max_rank <= 32) return launch_ranks<TYPE, 2>(a, s, st);
  if (a.max_rank <= 64) return launch_ranks<TYPE, 4>(a, s, st);
  return launch_ranks<TYPE, 8>(a, s, st);
}

int launch_lora(int type, const LoraArgs& a, hipStream_t st) {
  switch (type) {
    case MMVQ_F16: return launch_type<MMVQ_F16>(a, st);
    case MMVQ_BF16: return launch_type<MMVQ_BF16>(a, st);
    case MMVQ_F32: return launch_type<MMVQ_F32>(a, st);
    default: return MMVQ_ERR_TYPE;
  }
}

}  // namespace qmv
