// lora.hip - low-rank adapters of many requests beside a shared projection.
//
//   v = A_a x[t] (r numbers a row), out[t] = base[t] + scale_a * B_a v
//
// Two launches: shrink (v, in ranges of K) and expand (v of all ranges
// summed, B_a v, the addition). Up to 16 rows of one adapter (32 in large
// batches), out of 64 consecutive ones, share its weights: a side of 16x16x32
// bf16 matrix products, whose other side is 16 rows of A or B. Rows of one adapter are
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

constexpr int kLBlock = 64;                    // consecutive rows among which tiles are formed
constexpr int kLStep = 32;                     // of K, or ranks, a matrix product
constexpr int kLColumns = 16;                  // rows of x a matrix product
constexpr int kAWaves = 8, kBWaves = 4;        // of a workgroup of shrink and of expand

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

// Eight consecutive weights: as they are stored, and as bf16 parts.
template <int TYPE>
struct Weights {
  static constexpr int kParts = TYPE == MMVQ_BF16 ? 1 : TYPE == MMVQ_F16 ? 2 : 3;
  static constexpr int kBytes = TYPE == MMVQ_F32 ? 4 : 2;
  static constexpr int kQuads = TYPE == MMVQ_F32 ? 2 : 1;
  u32x4 raw[kQuads];
  __device__ __forceinline__ void load(const uint8_t* m, int64_t i) {
#pragma unroll
    for (int q = 0; q < kQuads; ++q) raw[q] = ld_a16_x4(m + i * kBytes + 16 * q);
  }
  // Those from `valid` on become 0 (8 and more: none).
  __device__ __forceinline__ void cut(int valid) {
#pragma unroll
    for (int q = 0; q < kQuads; ++q)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if constexpr (TYPE == MMVQ_F32) raw[q][e] = 4 * q + e < valid ? raw[q][e] : 0u;
        else raw[q][e] &= (2 * e < valid ? 0x0000FFFFu : 0u) | (2 * e + 1 < valid ? 0xFFFF0000u : 0u);
      }
  }
  __device__ __forceinline__ void split(u32x4 (&part)[kParts]) const {
    if constexpr (TYPE == MMVQ_BF16) {
      part[0] = raw[0];
    } else {
      float v[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if constexpr (TYPE == MMVQ_F32) {
          v[e] = __uint_as_float(raw[0][e]);
          v[e + 4] = __uint_as_float(raw[1][e]);
        } else {
          v[2 * e] = h2f(raw[0][e]);
          v[2 * e + 1] = h2f(raw[0][e] >> 16);
        }
      }
      split8<kParts>(v, part);
    }
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
template <int CT>
struct Tile {
  int adapter;             // -1: none
  int rank;
  int count;               // rows; 0: none
  int row[CT];             // of the lane's columns lane % 16 + 16 c; the first one's behind count
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

template <int CT>
__device__ __forceinline__ Tile<CT> tile_of(const LoraArgs& a, int block, int ids, int lead) {
  constexpr int kRows = kLColumns * CT;
  Tile<CT> tile{__builtin_amdgcn_readlane(ids, lead), 0, 0, {}, 0.0f};
  const uint64_t same = __ballot(ids == tile.adapter);
  const int ahead = __builtin_popcountll(same & ((uint64_t(1) << lead) - 1));
  if (tile.adapter == -2 || ahead % kRows) return tile;
  const int left = __builtin_popcountll(same) - ahead;
  tile.count = left < kRows ? left : kRows;
  const int lane = lane_id(), mine = __builtin_popcountll(same & ((uint64_t(1) << lane) - 1)) - ahead;
  const bool member = ids == tile.adapter && mine >= 0 && mine < kRows;
  const int pushed = __builtin_amdgcn_ds_permute(4 * (member ? mine : kWave - 1), lane);
#pragma unroll
  for (int c = 0; c < CT; ++c) {
    const int column = lane % kLColumns + kLColumns * c;
    tile.row[c] = block * kLBlock + __shfl(pushed, column < tile.count ? column : 0);
  }
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

// v of a tile over a range of K, 16 RT ranks at a time. The waves share the
// range. Columns behind the tile's count and ranks behind the adapter's repeat
// real ones, so that no load waits for a condition; what comes of them is
// not stored, or not used.
template <int TYPE, int RT, int CT>
__global__ void __launch_bounds__(kAWaves * kWave) lora_shrink_kernel(LoraArgs a) {
  using W = Weights<TYPE>;
  constexpr int kRegs = 8 * CT + 4 * W::kQuads * RT, kAhead = kRegs <= 24 ? 4 : kRegs <= 48 ? 2 : 1;   // steps on their way
  __shared__ f32x4 lds[kAWaves][RT][kWave];
  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), g = lane / 16;
  const int block = blockIdx.x, split = blockIdx.z;
  const int ids = block_ids(a, block);
  const int steps = static_cast<int>((a.K + kLStep - 1) / kLStep), whole = static_cast<int>(a.K / kLStep);
  const int s0 = (split * kAWaves + wave) * a.steps, s1 = s0 + a.steps < steps ? s0 + a.steps : steps;
  for (int lead = blockIdx.y * a.leads, end = lead + a.leads; lead < end; ++lead) {
    const Tile<CT> tile = tile_of<CT>(a, block, ids, lead);
    if (tile.count == 0 || tile.rank == 0) continue;       // uniform
    const float* x[CT];
#pragma unroll
    for (int c = 0; c < CT; ++c) x[c] = a.x + tile.row[c] * a.ldx + 8 * g;
    const uint8_t* A = a.A + tile.adapter * a.stride_a * W::kBytes;
    for (int r0 = 0; r0 < tile.rank; r0 += 16 * RT) {
      f32x4 acc[RT][CT];
      int64_t w0[RT];                          // element of the lane's rank
#pragma unroll
      for (int t = 0; t < RT; ++t) {
        const int j = r0 + 16 * t + lane % 16;
        w0[t] = (j < tile.rank ? j : tile.rank - 1) * a.K + 8 * g;
#pragma unroll
        for (int c = 0; c < CT; ++c) acc[t][c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      }
      const auto products = [&](const float (&v)[CT][8], W (&w)[RT]) QMV_INLINE {
        u32x4 xp[CT][3];
#pragma unroll
        for (int c = 0; c < CT; ++c) split8<3>(v[c], xp[c]);
#pragma unroll
        for (int t = 0; t < RT; ++t)
          if (RT == 1 || r0 + 16 * t < tile.rank) {        // uniform
            u32x4 wp[W::kParts];
            w[t].split(wp);
#pragma unroll
            for (int c = 0; c < CT; ++c) acc[t][c] = multiply<W::kParts>(wp, xp[c], acc[t][c]);
          }
      };
      int s = s0;
      for (const int last = s1 < whole ? s1 : whole; s < last; s += kAhead) {
        float v[kAhead][CT][8];
        W w[kAhead][RT];
#pragma unroll
        for (int q = 0; q < kAhead; ++q) {
          const int k = (s + q < last ? s + q : last - 1) * kLStep;
#pragma unroll
          for (int c = 0; c < CT; ++c) values8(x[c] + k, v[q][c]);
#pragma unroll
          for (int t = 0; t < RT; ++t)
            if (RT == 1 || r0 + 16 * t < tile.rank) w[q][t].load(A, w0[t] + k);
        }
#pragma unroll
        for (int q = 0; q < kAhead; ++q)
          if (s + q < last) products(v[q], w[q]);           // uniform
      }
      if (whole < s1 && s0 <= whole) {                     // the rest of K: 8, 16 or 24 values
        float v[1][CT][8];
        W w[1][RT];
        const int k = whole * kLStep, back = k + 8 * g < a.K ? 0 : 8 * g;   // lanes behind it repeat the first's, times 0
#pragma unroll
        for (int c = 0; c < CT; ++c) {
          values8(x[c] + k - back, v[0][c]);
#pragma unroll
          for (int e = 0; e < 8; ++e) v[0][c][e] = back ? 0.0f : v[0][c][e];
        }
#pragma unroll
        for (int t = 0; t < RT; ++t) {
          w[0][t].load(A, w0[t] + k - back);
          w[0][t].cut(back ? 0 : 8);
        }
        products(v[0], w[0]);
      }
#pragma unroll
      for (int c = 0; c < CT; ++c) {
        __syncthreads();                       // the sums before are read
#pragma unroll
        for (int t = 0; t < RT; ++t) lds[wave][t][lane] = acc[t][c];
        __syncthreads();
        for (int t = wave; t < RT; t += kAWaves) {
          const int j = r0 + 16 * t + 4 * g;
          f32x4 sum = lds[0][t][lane];
#pragma unroll
          for (int w = 1; w < kAWaves; ++w) sum += lds[w][t][lane];
          if (lane % kLColumns + kLColumns * c < tile.count && j < a.max_rank)
            *reinterpret_cast<f32x4*>(a.part + (static_cast<int64_t>(split) * a.n + tile.row[c]) * a.max_rank + j) = sum;
        }
      }
    }
  }
}

// base + scale * B v of a tile, for a slice of M; up to 32 RC ranks.
template <int TYPE, int RC, int CT>
__global__ void __launch_bounds__(kBWaves * kWave) lora_expand_kernel(LoraArgs a) {
  using W = Weights<TYPE>;
  constexpr int kAhead = RC * W::kQuads * (CT + 1) <= 4 ? 4 : RC * W::kQuads <= 4 ? 2 : 1;   // tiles of 16 outputs on their way
  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), g = lane / 16;
  const int block = blockIdx.x;
  const int ids = block_ids(a, block);
  constexpr int kPiece = 16 * kAhead;          // outputs a wave takes at a time, side by side
  const int64_t m_first = (static_cast<int64_t>(blockIdx.z) * kBWaves + wave) * kPiece, m_step = static_cast<int64_t>(gridDim.z) * kBWaves * kPiece;
  for (int lead = blockIdx.y * a.leads, end = lead + a.leads; lead < end; ++lead) {
    const Tile<CT> tile = tile_of<CT>(a, block, ids, lead);
    if (tile.count == 0 || (tile.rank == 0 && a.base == a.out)) continue;   // uniform
    const float* base[CT];
    float* out[CT];
    bool live[CT];
#pragma unroll
    for (int c = 0; c < CT; ++c) {
      live[c] = lane % kLColumns + kLColumns * c < tile.count;
      base[c] = a.base + tile.row[c] * a.ldb + 4 * g;
      out[c] = a.out + tile.row[c] * a.ldo + 4 * g;
    }
    const uint8_t* B = a.B + (tile.adapter < 0 ? 0 : tile.adapter) * a.stride_b * W::kBytes;
    W w[kAhead][RC];
    f32x4 old[kAhead][CT];
    const auto fetch = [&](int64_t m0) QMV_INLINE {
#pragma unroll
      for (int t = 0; t < kAhead; ++t) {
        const int64_t m = m0 + 16 * t + lane % 16, row = (m < a.M ? m : a.M - 1) * a.max_rank;
#pragma unroll
        for (int q = 0; q < RC; ++q) {
          const int j = kLStep * q + 8 * g;
          if (kLStep * q < tile.rank) w[t][q].load(B, row + (j < a.max_rank ? j : 0));   // uniform
        }
#pragma unroll
        for (int c = 0; c < CT; ++c)
          if (live[c] && m0 + 16 * t + 4 * g + 4 <= a.M) {
            const u32x4 b = ld_x4(reinterpret_cast<const uint8_t*>(base[c] + m0 + 16 * t));
            old[t][c] = f32x4{__uint_as_float(b[0]), __uint_as_float(b[1]), __uint_as_float(b[2]), __uint_as_float(b[3])};
          }
      }
    };
    if (m_first < a.M) fetch(m_first);         // on their way while v is summed
    u32x4 v[CT][RC][3];
#pragma unroll
    for (int c = 0; c < CT; ++c)
#pragma unroll
      for (int q = 0; q < RC; ++q) {
        const int j = kLStep * q + 8 * g;
        float sum[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[e] = 0.0f;
        if (j < tile.rank) {
          const float* part = a.part + static_cast<int64_t>(tile.row[c]) * a.max_rank + j;
          const int64_t step = static_cast<int64_t>(a.n) * a.max_rank;
#pragma unroll 4
          for (int s = 0; s < a.splits; ++s) {
            float one[8];
            values8(part + s * step, one);
#pragma unroll
            for (int e = 0; e < 8; ++e) sum[e] += one[e];
          }
        }
        // (ranks behind the adapter's have sums of others' weights)
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[e] = j + e < tile.rank ? sum[e] : 0.0f;
        split8<3>(sum, v[c][q]);
      }
    const bool cuts = tile.rank % kLStep != 0;   // uniform
    for (int64_t m0 = m_first; m0 < a.M; m0 += m_step) {
      if (m0 > m_first) fetch(m0);
#pragma unroll
      for (int t = 0; t < kAhead; ++t) {
        f32x4 acc[CT];
#pragma unroll
        for (int c = 0; c < CT; ++c) acc[c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int q = 0; q < RC; ++q) {
          if (kLStep * q < tile.rank) {        // uniform
            if (cuts) w[t][q].cut(tile.rank - kLStep * q - 8 * g);
            u32x4 wp[W::kParts];
            w[t][q].split(wp);
#pragma unroll
            for (int c = 0; c < CT; ++c) acc[c] = multiply<W::kParts>(wp, v[c][q], acc[c]);
          }
        }
        const int64_t o = m0 + 16 * t;
#pragma unroll
        for (int c = 0; c < CT; ++c) {
          if (live[c] && o + 4 * g + 4 <= a.M) {
            f32x4 y;
#pragma unroll
            for (int e = 0; e < 4; ++e) y[e] = old[t][c][e] + tile.scale * acc[c][e];
            __builtin_memcpy(__builtin_assume_aligned(out[c] + o, 4), &y, 16);
          } else if (live[c]) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (o + 4 * g + e < a.M) out[c][o + e] = base[c][o + e] + tile.scale * acc[c][e];
          }
        }
      }
    }
  }
}

// Launch shape. How many tiles there are the host cannot see: it counts on
// rows of their own adapters in one block of rows, of one adapter beyond.
// Ranges of K until the chip is filled, of two products a wave at least, and
// slices of M likewise. Of many rows tiles take 32, which halves the reads of
// the weights.
struct LoraShape {
  int blocks, leads, groups, splits, steps, slices, ct;
};
inline LoraShape lora_shape(int64_t n, int64_t K, int64_t M, int max_rank) {
  LoraShape s;
  s.ct = n >= 1024 && max_rank <= 64 ? 2 : 1;
  s.blocks = static_cast<int>((n + kLBlock - 1) / kLBlock);
  s.leads = s.blocks <= 8 ? 1 : s.blocks <= 32 ? 4 : kLColumns * s.ct;   // rows of a block that a workgroup looks for tiles at
  const int rows = n < kLBlock ? static_cast<int>(n) : kLBlock;
  s.groups = (rows + s.leads - 1) / s.leads;
  int64_t tiles = (n + kLColumns * s.ct - 1) / (kLColumns * s.ct);
  if (tiles < rows) tiles = rows;
  const int64_t want = (2 * kCus + tiles - 1) / tiles;
  const int64_t steps = (K + kLStep - 1) / kLStep, most = (steps + 2 * kAWaves - 1) / (2 * kAWaves);
  int64_t splits = want < most ? want : most;
  if (splits > 16) splits = 16;
  s.steps = static_cast<int>((steps + splits * kAWaves - 1) / (splits * kAWaves));
  s.splits = static_cast<int>((steps + static_cast<int64_t>(s.steps) * kAWaves - 1) / (s.steps * kAWaves));
  const int64_t pieces = (M + 32 * kBWaves - 1) / (32 * kBWaves);
  s.slices = static_cast<int>(2 * want < pieces ? 2 * want : pieces);
  if (s.slices > 64) s.slices = 64;
  return s;
}

int64_t lora_bytes(int64_t n, int64_t K, int64_t M, int max_rank) {
  if (n == 0) return 0;
  return lora_shape(n, K, M, max_rank).splits * n * max_rank * static_cast<int64_t>(sizeof(float));
}

template <int TYPE, int RT, int RC, int CT>
int launch_ranks(const LoraArgs& a, const LoraShape& s, hipStream_t st) {
  hipLaunchKernelGGL((lora_shrink_kernel<TYPE, RT, CT>), dim3(s.blocks, s.groups, s.splits), dim3(kAWaves * kWave), 0, st, a);
  const int rc = check_launch();
  if (rc) return rc;
  hipLaunchKernelGGL((lora_expand_kernel<TYPE, RC, CT>), dim3(s.blocks, s.groups, s.slices), dim3(kBWaves * kWave), 0, st, a);
  return check_launch();
}

template <int TYPE>
int launch_type(const LoraArgs& given, hipStream_t st) {
  LoraArgs a = given;
  const LoraShape s = lora_shape(a.n, a.K, a.M, a.max_rank);
  a.splits = s.splits;
  a.steps = s.steps;
  a.leads = s.leads;
  if (s.ct == 2) {
    if (a.max_rank <= 16) return launch_ranks<TYPE, 1, 1, 2>(a, s, st);
    if (a.max_rank <= 32) return launch_ranks<TYPE, 2, 1, 2>(a, s, st);
    return launch_ranks<TYPE, 4, 2, 2>(a, s, st);
  }
  if (a.max_rank <= 16) return launch_ranks<TYPE, 1, 1, 1>(a, s, st);
  if (a.max_rank <= 32) return launch_ranks<TYPE, 2, 1, 1>(a, s, st);
  if (a.max_rank <= 64) return launch_ranks<TYPE, 4, 2, 1>(a, s, st);
  if (a.max_rank <= 128) return launch_ranks<TYPE, 8, 4, 1>(a, s, st);
  return launch_ranks<TYPE, 8, 8, 1>(a, s, st);
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
